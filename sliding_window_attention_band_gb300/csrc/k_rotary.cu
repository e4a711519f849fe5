// k_rotary.cu -- rotary positions on queries and keys, their gradient, and the
// same fused with the write of K and V into the paged cache.
//
// Pair k of a head, channels (a, b), turns by t = 2 pi frac(p * turns[k] / 2^64):
//     y_a = m (x_a cos t - x_b sin t),   y_b = m (x_b cos t + x_a sin t),
// the gradient by -t.  The frequency is a 64-bit fixed-point fraction of a
// turn, so the product with the position, taken modulo 2^64, IS the fraction
// of the turn: one integer multiply, exact at any distance, where an fp32
// product is off by 0.06 rad at position 10^6.  Its upper bits become the
// argument of sincospif (relative rounding 2^-24, so at most 2^-25 pi rad).
//
// A block takes a few tokens: it fills a table of their cosines and sines in
// shared memory (one sincospi for a pair and token, shared by all the heads),
// then walks the head rows; a thread owns one place in the row (16 bytes of
// each member of its pairs, 16 bytes of both when interleaved) and keeps two
// rows' loads in flight, so consecutive threads read whole lines.
// HBM-bound: every value is read once and written once.
#include "swab_internal.h"

static constexpr unsigned kSwabFile = 11;   // site id of the bounds checks

namespace swab {
namespace {

constexpr int kThreads = 256;

// One row of work: a head of Q or K (turned) or of V (copied).
struct Row {
    const char *src;
    char *dst;       // null: nothing to write (no slot)
    bool turn;
};

template <typename T> struct VecOf {
    static constexpr int kN = 16 / sizeof(T);   // elements of 16 bytes
};

template <typename T>
__device__ __forceinline__ void unpack16(const uint4 &v, float *f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (sizeof(T) == 4) {
            f[k] = __uint_as_float(w[k]);
        } else {
            f[2 * k] = lo16<T>(w[k]);
            f[2 * k + 1] = hi16<T>(w[k]);
        }
    }
}
template <typename T>
__device__ __forceinline__ uint4 pack16(const float *f) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (sizeof(T) == 4) w[k] = __float_as_uint(f[k]);
        else w[k] = pack2<T>(f[2 * k], f[2 * k + 1]);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 load16(const void *p) { return *reinterpret_cast<const uint4 *>(p); }

// Row `idx` of token t: heads of Q, then of K, then (append) of V.
template <typename T, bool kAppend>
__device__ __forceinline__ Row row_of(const RotaryArgs &p, long long t, int idx) {
    const unsigned bb = (unsigned)t / (unsigned)p.n, i = (unsigned)t - bb * (unsigned)p.n;
    Row r;
    if (idx < p.hq) {
        r.src = (const char *)p.Q + ((long long)bb * p.sq[0] + (long long)i * p.sq[1] + (long long)idx * p.sq[2]) * (int)sizeof(T);
        r.dst = (char *)p.Qo + ((long long)bb * p.sqo[0] + (long long)i * p.sqo[1] + (long long)idx * p.sqo[2]) * (int)sizeof(T);
        r.turn = true;
        return r;
    }
    idx -= p.hq;
    const bool is_v = kAppend && idx >= p.hk;
    if (is_v) idx -= p.hk;
    const long long *s = is_v ? p.sv : p.sk;
    r.src = (const char *)(is_v ? p.V : p.K) + ((long long)bb * s[0] + (long long)i * s[1] + (long long)idx * s[2]) * (int)sizeof(T);
    r.turn = !is_v;
    if constexpr (kAppend) {
        const int slot = *GP(p.bnd, p.slots + t);
        r.dst = nullptr;
        if (slot >= 0 && slot < p.n_slots) {
            const unsigned blk = (unsigned)slot >> p.page_log2, off = (unsigned)slot & ((1u << p.page_log2) - 1u);
            const long long line = (((long long)blk * p.hk + idx) << p.page_log2) + off;
            r.dst = (char *)(is_v ? p.Vc : p.Kc) + line * p.hd * (int)sizeof(T);
        } else if (slot != -1) {
            atomicOr(p.err, kErrInvalid);
        }
    } else {
        r.dst = (char *)p.Ko + ((long long)bb * p.sko[0] + (long long)i * p.sko[1] + (long long)idx * p.sko[2]) * (int)sizeof(T);
    }
    return r;
}

// kMode: 0 = halves in 16-byte pieces, 1 = interleaved in 16-byte pieces,
// 2 = element by element (a pair does not start on a 16-byte piece).
template <typename T, int kMode, bool kAppend>
__global__ void __launch_bounds__(kThreads) k_rotary(const __grid_constant__ RotaryArgs p) {
    constexpr int kV = VecOf<T>::kN;
    extern __shared__ float tab[];           // [tile][2][rot / 2]: cos, sin of each token
    const int half = p.rot / 2;
    const int rows = p.hq + p.hk * (kAppend ? 2 : 1);
    // places of a row: those whose pairs turn, then those copied
    const int nturn = kMode == 0 ? half / kV : kMode == 1 ? p.rot / kV : half;
    const int ncopy = kMode == 2 ? p.hd - p.rot : (p.hd - p.rot) / kV;
    const int places = nturn + ncopy;
    const int per_pass = places >= kThreads ? 1 : kThreads / places;   // rows of a pass

    for (long long t0 = (long long)blockIdx.x * p.tile; t0 < p.tokens; t0 += (long long)gridDim.x * p.tile) {
        const int nt = (int)(p.tokens - t0 < p.tile ? p.tokens - t0 : p.tile);
        for (int e = threadIdx.x; e < nt * half; e += kThreads) {
            const int tt = e / half, k = e - tt * half;
            const long long t = t0 + tt;
            const long long at = (p.pos ? (long long)*GP(p.bnd, p.pos + t) : t % p.n) + p.pos0;
            const long long frac = (long long)((unsigned long long)at * *GP(p.bnd, p.turns + k));
            float sn, cs;
            sincospif((float)frac * 0x1p-63f, &sn, &cs);   // in half turns: [-1, 1)
            tab[(2 * tt) * half + k] = cs * p.scale;
            tab[(2 * tt + 1) * half + k] = sn * (p.backward ? -p.scale : p.scale);
        }
        __syncthreads();
        // head rows of the block's share: blockIdx.y of gridDim.y slices of the heads
        const int lo = (int)((long long)rows * blockIdx.y / gridDim.y), hi = (int)((long long)rows * (blockIdx.y + 1) / gridDim.y);
        const int mine = hi - lo, total = nt * mine;
        for (int place = threadIdx.x % places, q0 = threadIdx.x / places;;) {
            if (places < kThreads && q0 >= per_pass) break;      // the odd threads of a pass
            for (int q = q0; q < total; q += per_pass) {
                const int tt = q / mine;
                const Row r = row_of<T, kAppend>(p, t0 + tt, lo + q - tt * mine);
                if (r.dst == nullptr) continue;
                const float *cs = tab + (2 * tt) * half, *sn = cs + half;
                if constexpr (kMode == 2) {
                    const T *x = reinterpret_cast<const T *>(r.src);
                    T *y = reinterpret_cast<T *>(r.dst);
                    if (place >= nturn) {
                        *GP(p.bnd, y + p.rot + place - nturn) = *GP(p.bnd, x + p.rot + place - nturn);
                    } else {
                        const int a = p.interleaved ? 2 * place : place, b = p.interleaved ? 2 * place + 1 : place + half;
                        const T xa = *GP(p.bnd, x + a), xb = *GP(p.bnd, x + b);
                        if (r.turn) {
                            const float fa = Elt<T>::to_f(xa), fb = Elt<T>::to_f(xb), c = cs[place], s = sn[place];
                            *GP(p.bnd, y + a) = Elt<T>::from_f(fa * c - fb * s);
                            *GP(p.bnd, y + b) = Elt<T>::from_f(fb * c + fa * s);
                        } else {
                            *GP(p.bnd, y + a) = xa;
                            *GP(p.bnd, y + b) = xb;
                        }
                    }
                } else if (place >= nturn) {
                    const int at = (p.rot + (place - nturn) * kV) * (int)sizeof(T);
                    if (r.src != r.dst) *reinterpret_cast<uint4 *>(GPN(p.bnd, r.dst + at, 16)) = load16(GPN(p.bnd, r.src + at, 16));
                } else if constexpr (kMode == 0) {
                    const int a = 16 * place, b = a + half * (int)sizeof(T);
                    uint4 va = load16(GPN(p.bnd, r.src + a, 16)), vb = load16(GPN(p.bnd, r.src + b, 16));
                    if (r.turn) {
                        float fa[kV], fb[kV], ya[kV], yb[kV];
                        unpack16<T>(va, fa);
                        unpack16<T>(vb, fb);
#pragma unroll
                        for (int e = 0; e < kV; ++e) {
                            const float c = cs[place * kV + e], s = sn[place * kV + e];
                            ya[e] = fa[e] * c - fb[e] * s;
                            yb[e] = fb[e] * c + fa[e] * s;
                        }
                        va = pack16<T>(ya);
                        vb = pack16<T>(yb);
                    }
                    *reinterpret_cast<uint4 *>(GPN(p.bnd, r.dst + a, 16)) = va;
                    *reinterpret_cast<uint4 *>(GPN(p.bnd, r.dst + b, 16)) = vb;
                } else {
                    const int a = 16 * place;
                    uint4 v = load16(GPN(p.bnd, r.src + a, 16));
                    if (r.turn) {
                        float f[kV], y[kV];
                        unpack16<T>(v, f);
#pragma unroll
                        for (int e = 0; e < kV / 2; ++e) {
                            const float c = cs[place * (kV / 2) + e], s = sn[place * (kV / 2) + e];
                            y[2 * e] = f[2 * e] * c - f[2 * e + 1] * s;
                            y[2 * e + 1] = f[2 * e + 1] * c + f[2 * e] * s;
                        }
                        v = pack16<T>(y);
                    }
                    *reinterpret_cast<uint4 *>(GPN(p.bnd, r.dst + a, 16)) = v;
                }
            }
            place += kThreads;                                    // rows longer than the block
            if (places < kThreads || place >= places) break;
        }
        __syncthreads();
    }
}

template <typename T, bool kAppend>
cudaError_t launch_t(const RotaryArgs &a, int mode, dim3 grid, size_t smem, cudaStream_t st) {
    switch (mode) {
        case 0: k_rotary<T, 0, kAppend><<<grid, kThreads, smem, st>>>(a); break;
        case 1: k_rotary<T, 1, kAppend><<<grid, kThreads, smem, st>>>(a); break;
        default: k_rotary<T, 2, kAppend><<<grid, kThreads, smem, st>>>(a); break;
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rotary(DType dt, bool append, RotaryArgs a, cudaStream_t st) {
    const int es = dt == kF32 ? 4 : 2, vec = 16 / es;
    const int mode = a.rot == 0 ? 0 : a.interleaved ? (a.rot % vec == 0 ? 1 : 2) : (a.rot / 2 % vec == 0 ? 0 : 2);
    const int rows = a.hq + a.hk * (append ? 2 : 1);
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidValue;
    a.tile = a.tokens >= 8LL * 4 * sms ? 4 : 1;
    const long long tiles = (a.tokens + a.tile - 1) / a.tile;
    const dim3 grid((unsigned)(tiles < 8LL * sms ? tiles : 8LL * sms), 1);
    const size_t smem = (size_t)a.tile * a.rot * sizeof(float);
    (void)rows;
    if (dt == kF32) return append ? launch_t<float, true>(a, mode, grid, smem, st) : launch_t<float, false>(a, mode, grid, smem, st);
    if (dt == kF16) return append ? launch_t<__half, true>(a, mode, grid, smem, st) : launch_t<__half, false>(a, mode, grid, smem, st);
    return append ? launch_t<__nv_bfloat16, true>(a, mode, grid, smem, st) : launch_t<__nv_bfloat16, false>(a, mode, grid, smem, st);
}

}  // namespace swab
