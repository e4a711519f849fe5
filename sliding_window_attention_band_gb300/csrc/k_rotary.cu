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
// A block takes a few tokens.  It lists their head rows (where from, where to)
// and fills a table of their cosines and sines in shared memory -- one sincospi
// for a pair and token, shared by all the heads, so the divisions and the
// trigonometry cost one thread-step a row and a pair.  Then a thread owns one
// place in a row (16 bytes of each member of its pairs, 16 bytes of both when
// interleaved) and walks the rows four at a time, their loads in flight
// together; consecutive threads cover whole lines.
// HBM-bound: every value is read once and written once.
#include <algorithm>

#include "swab_internal.h"

static constexpr unsigned kSwabFile = 11;   // site id of the bounds checks

namespace swab {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = 512;        // listed rows of a block at a time
constexpr int kMaxTile = 16;        // tokens of a block (Row::token)
constexpr int kUnroll = 4;            // rows of a thread in flight

// One row of work: a head of Q or K (turned) or of V (copied).  The addresses
// are multiples of 16, so their low bits carry the token of the tile and
// whether the row turns.
struct Row {
    uintptr_t s, d;  // d = 0: nothing to write (no slot)
    __device__ __forceinline__ const char *src() const { return reinterpret_cast<const char *>(s & ~(uintptr_t)15); }
    __device__ __forceinline__ char *dst() const { return reinterpret_cast<char *>(d & ~(uintptr_t)15); }
    __device__ __forceinline__ int token() const { return (int)(s & 15u); }
    __device__ __forceinline__ bool turn() const { return d & 1u; }
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
__device__ __forceinline__ Row row_of(const RotaryArgs &p, unsigned t, int tt, int idx) {
    const unsigned bb = t / (unsigned)p.n, i = t - bb * (unsigned)p.n;
    const char *src;
    char *dst;
    bool turn = true;
    if (idx < p.hq) {
        src = (const char *)p.Q + ((long long)bb * p.sq[0] + (long long)i * p.sq[1] + (long long)idx * p.sq[2]) * (int)sizeof(T);
        dst = (char *)p.Qo + ((long long)bb * p.sqo[0] + (long long)i * p.sqo[1] + (long long)idx * p.sqo[2]) * (int)sizeof(T);
    } else {
        idx -= p.hq;
        const bool is_v = kAppend && idx >= p.hk;
        if (is_v) idx -= p.hk;
        const long long *s = is_v ? p.sv : p.sk;
        src = (const char *)(is_v ? p.V : p.K) + ((long long)bb * s[0] + (long long)i * s[1] + (long long)idx * s[2]) * (int)sizeof(T);
        turn = !is_v;
        if constexpr (kAppend) {
            const int slot = *GP(p.bnd, p.slots + t);
            dst = nullptr;
            if (slot >= 0 && slot < p.n_slots) {
                const unsigned blk = (unsigned)slot >> p.page_log2, off = (unsigned)slot & ((1u << p.page_log2) - 1u);
                const long long line = (((long long)blk * p.hk + idx) << p.page_log2) + off;
                dst = (char *)(is_v ? p.Vc : p.Kc) + line * p.hd * (int)sizeof(T);
            } else if (slot != -1) {
                atomicOr(p.err, kErrInvalid);
            }
        } else {
            dst = (char *)p.Ko + ((long long)bb * p.sko[0] + (long long)i * p.sko[1] + (long long)idx * p.sko[2]) * (int)sizeof(T);
        }
    }
    const uintptr_t d = reinterpret_cast<uintptr_t>(dst);
    return Row{reinterpret_cast<uintptr_t>(src) + tt, d && turn ? d + 1 : d};
}

// kMode: 0 = halves in 16-byte pieces, 1 = interleaved in 16-byte pieces,
// 2 = a pair a place (the pairs do not start on 16-byte pieces; the channels
// behind them are copied 16 bytes at a time where they do).
template <typename T, int kMode, bool kAppend>
__global__ void __launch_bounds__(kThreads) k_rotary(const __grid_constant__ RotaryArgs p) {
    constexpr int kV = VecOf<T>::kN, kB = (int)sizeof(T);
    constexpr int kLoads = kMode == 0 ? 2 : 1;
    extern __shared__ float tab[];           // [tile][2][rot / 2]: cos, sin of each token
    __shared__ Row list[kMaxRows];
    const int half = p.rot / 2;
    const int rows = p.hq + p.hk * (kAppend ? 2 : 1);
    const bool vcopy = kMode != 2 || p.rot * kB % 16 == 0;
    // places of a row: those whose pairs turn, then those copied
    const int nturn = kMode == 0 ? half / kV : kMode == 1 ? p.rot / kV : half;
    const int places = nturn + (vcopy ? (p.hd - p.rot) / kV : p.hd - p.rot);
    const int per_pass = places >= kThreads ? 1 : kThreads / places;   // rows of a pass
    const int place0 = threadIdx.x % places, q0 = threadIdx.x / places;
    // the block's share of the heads: gridDim.y slices
    const int lo = (int)((long long)rows * blockIdx.y / gridDim.y), mine = (int)((long long)rows * (blockIdx.y + 1) / gridDim.y) - lo;

    for (long long t0 = (long long)blockIdx.x * p.tile; t0 < p.tokens; t0 += (long long)gridDim.x * p.tile) {
        const int nt = (int)(p.tokens - t0 < p.tile ? p.tokens - t0 : p.tile);
        const int total = nt * mine;
        for (int e = threadIdx.x; e < total; e += kThreads) {
            const int tt = e / mine;
            list[e] = row_of<T, kAppend>(p, (unsigned)t0 + tt, tt, lo + e - tt * mine);
        }
        for (int e = threadIdx.x; e < nt * half; e += kThreads) {
            const int tt = e / half, k = e - tt * half;
            const unsigned t = (unsigned)t0 + tt;
            const long long at = (p.pos ? (long long)*GP(p.bnd, p.pos + t) : (long long)(t % (unsigned)p.n)) + p.pos0;
            const long long frac = (long long)((unsigned long long)at * *GP(p.bnd, p.turns + k));
            float sn, cs;
            sincospif((float)frac * 0x1p-63f, &sn, &cs);   // in half turns: [-1, 1)
            tab[(2 * tt) * half + k] = cs * p.scale;
            tab[(2 * tt + 1) * half + k] = sn * (p.backward ? -p.scale : p.scale);
        }
        __syncthreads();
        for (int place = place0; place < places; place += kThreads) {
            if (places < kThreads && q0 >= per_pass) break;      // the threads left over by a pass
            const bool copies = place >= nturn;
            const int at = copies ? (vcopy ? (p.rot + (place - nturn) * kV) * kB : (p.rot + place - nturn) * kB) : 16 * place;
            for (int q = q0; q < total; q += kUnroll * per_pass) {
                if constexpr (kMode == 2) {
                    if (!(copies && vcopy)) {                     // element by element
#pragma unroll
                        for (int u = 0; u < kUnroll; ++u) {
                            const int e = q + u * per_pass;
                            if (e >= total || !list[e].d) continue;
                            const T *x = reinterpret_cast<const T *>(list[e].src());
                            T *y = reinterpret_cast<T *>(list[e].dst());
                            if (copies) {
                                *GP(p.bnd, y + at / kB) = *GP(p.bnd, x + at / kB);
                                continue;
                            }
                            const int a = p.interleaved ? 2 * place : place, b = p.interleaved ? 2 * place + 1 : place + half;
                            const T xa = *GP(p.bnd, x + a), xb = *GP(p.bnd, x + b);
                            T ya = xa, yb = xb;
                            if (list[e].turn()) {
                                const float *cs = tab + 2 * list[e].token() * half;
                                const float fa = Elt<T>::to_f(xa), fb = Elt<T>::to_f(xb), c = cs[place], s = cs[half + place];
                                ya = Elt<T>::from_f(fa * c - fb * s);
                                yb = Elt<T>::from_f(fb * c + fa * s);
                            }
                            *GP(p.bnd, y + a) = ya;
                            *GP(p.bnd, y + b) = yb;
                        }
                        continue;
                    }
                }
                uint4 v[kUnroll][kLoads];
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    const int e = q + u * per_pass;
                    if (e >= total || !list[e].d) continue;
                    v[u][0] = load16(GPN(p.bnd, list[e].src() + at, 16));
                    if (kMode == 0 && !copies) v[u][kLoads - 1] = load16(GPN(p.bnd, list[e].src() + at + half * kB, 16));
                }
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    const int e = q + u * per_pass;
                    if (e >= total) break;
                    const Row r = list[e];
                    if (!r.d) continue;
                    char *out = r.dst();
                    if (kMode != 2 && !copies && r.turn()) {
                        const float *cs = tab + 2 * r.token() * half, *sn = cs + half;
                        if constexpr (kMode == 0) {
                            float fa[kV], fb[kV], ya[kV], yb[kV];
                            unpack16<T>(v[u][0], fa);
                            unpack16<T>(v[u][1], fb);
#pragma unroll
                            for (int k = 0; k < kV; ++k) {
                                const float c = cs[place * kV + k], s = sn[place * kV + k];
                                ya[k] = fa[k] * c - fb[k] * s;
                                yb[k] = fb[k] * c + fa[k] * s;
                            }
                            v[u][0] = pack16<T>(ya);
                            v[u][1] = pack16<T>(yb);
                        } else if constexpr (kMode == 1) {
                            float f[kV], y[kV];
                            unpack16<T>(v[u][0], f);
#pragma unroll
                            for (int k = 0; k < kV / 2; ++k) {
                                const float c = cs[place * (kV / 2) + k], s = sn[place * (kV / 2) + k];
                                y[2 * k] = f[2 * k] * c - f[2 * k + 1] * s;
                                y[2 * k + 1] = f[2 * k + 1] * c + f[2 * k] * s;
                            }
                            v[u][0] = pack16<T>(y);
                        }
                    }
                    *reinterpret_cast<uint4 *>(GPN(p.bnd, out + at, 16)) = v[u][0];
                    if (kMode == 0 && !copies) *reinterpret_cast<uint4 *>(GPN(p.bnd, out + at + half * kB, 16)) = v[u][kLoads - 1];
                }
            }
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
    // tokens of a block: about four rows a thread, but blocks enough for the GPU
    const int places = (mode == 0 ? a.rot / 2 : a.rot) / (mode == 2 ? 2 : vec) + (a.hd - a.rot) / vec;
    const long long items = (long long)rows * (places > 0 ? places : 1);
    long long tile = 4LL * kThreads / items;
    tile = std::min(tile, a.tokens / (4LL * sms));
    tile = std::max(1LL, std::min(tile, (long long)kMaxTile));
    int slices = 1;                          // of the heads
    if (rows > kMaxRows) slices = (rows + kMaxRows - 1) / kMaxRows, tile = 1;
    else tile = std::max(1LL, std::min(tile, (long long)kMaxRows / rows));
    a.tile = (int)tile;
    const long long tiles = (a.tokens + a.tile - 1) / a.tile;
    const dim3 grid((unsigned)std::min(tiles, 64LL * sms), (unsigned)slices);
    const size_t smem = (size_t)a.tile * a.rot * sizeof(float);
    if (dt == kF32) return append ? launch_t<float, true>(a, mode, grid, smem, st) : launch_t<float, false>(a, mode, grid, smem, st);
    if (dt == kF16) return append ? launch_t<__half, true>(a, mode, grid, smem, st) : launch_t<__half, false>(a, mode, grid, smem, st);
    return append ? launch_t<__nv_bfloat16, true>(a, mode, grid, smem, st) : launch_t<__nv_bfloat16, false>(a, mode, grid, smem, st);
}

}  // namespace swab
