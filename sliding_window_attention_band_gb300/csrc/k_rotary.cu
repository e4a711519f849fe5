// k_rotary.cu -- rotary positions on queries and keys, their gradient, and the
// same fused with the write of K and V into the paged cache.
//
// Pair k of a head, channels (a, b), turns by t = 2 pi frac(p * turns[k] / 2^64):
//     y_a = m (x_a cos t - x_b sin t),   y_b = m (x_b cos t + x_a sin t),
// the gradient by -t.  The frequency is a 64-bit fixed-point fraction of a
// turn, so the product with the position, taken modulo 2^64, IS the fraction
// of the turn: one integer multiply, exact at any distance, where an fp32
// product is off by 0.06 rad at position 10^6.  Its upper 32 bits (2 pi 2^-32
// rad), the nearest quarter turn taken off, become the argument of sincospif
// (rounded to fp32: 2^-27 pi rad at most, a small angle relatively).
//
// A block takes a few tokens at a time.  It lists their head rows (where from,
// where to) and fills a table of their cosines and sines in shared memory -- one
// sincospi for a pair and token, shared by all the heads, so the divisions and
// the trigonometry cost one thread-step a row and a pair.  Then a thread owns one
// place in a row (16 bytes of each member of its pairs, 16 bytes of both when
// interleaved) and walks the rows with four loads in flight; consecutive threads
// cover whole lines.  List and table of the next tokens are made under the first
// loads of these (two buffers, one barrier a tile).
//
// HBM-bound: every value is read once and written once.  8192 tokens of 32 + 8
// heads of 128: 28 us (168 MB, 6.0 TB/s); 12 x 1365 tokens of 24 heads of 64,
// half turned, adjacent pairs: 18.8 us (101 MB, 5.3 TB/s; 19.8 with one buffer);
// 8.9k tokens into the cache: 17.1 us (82 MB).  The short rows are bound by
// instructions: 16 bytes a thread carry the same addresses as 32.
#include <algorithm>

#include "swab_internal.h"

static constexpr unsigned kSwabFile = 11;   // site id of the bounds checks

namespace swab {
namespace {

constexpr int kThreads = 256;
constexpr int kBlocks = 5;           // of an SM
constexpr int kMaxRows = 512;        // listed rows of a block at a time
constexpr int kMaxTile = 16;        // tokens of a block (Row::token)

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

// N floats of the table, 16 or 8 bytes at a time
template <int N>
__device__ __forceinline__ void take(const float *src, float (&f)[N]) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int k = 0; k < N; k += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(src + k);
            f[k] = v.x, f[k + 1] = v.y, f[k + 2] = v.z, f[k + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < N; k += 2) {
            const float2 v = *reinterpret_cast<const float2 *>(src + k);
            f[k] = v.x, f[k + 1] = v.y;
        }
    }
}

// Row `idx` of token t: heads of Q, then of K, then (append) of V.  Strides
// are in units of 16 bytes, their sums below 2^32 (checked by the caller).
template <bool kAppend>
__device__ __forceinline__ Row row_of(const RotaryArgs &p, unsigned t, unsigned tt, int idx) {
    unsigned bb = 0, i = t;
    if (p.n < p.tokens) {
        bb = t / (unsigned)p.n;
        i = t - bb * (unsigned)p.n;
    }
    const bool is_q = idx < p.hq;
    unsigned head = is_q ? idx : idx - p.hq;
    const bool is_v = kAppend && !is_q && head >= (unsigned)p.hk;
    if (is_v) head -= p.hk;
    const unsigned *s = is_q ? p.sq : is_v ? p.sv : p.sk;
    const char *src = (const char *)(is_q ? p.Q : is_v ? p.V : p.K) + (unsigned long long)(bb * s[0] + i * s[1] + head * s[2]) * 16u;
    char *dst;
    if (kAppend && !is_q) {
        const int slot = *GP(p.bnd, p.slots + t);
        dst = nullptr;
        if (slot >= 0 && slot < p.n_slots) {
            const unsigned blk = (unsigned)slot >> p.page_log2, off = (unsigned)slot & ((1u << p.page_log2) - 1u);
            const unsigned line = ((blk * (unsigned)p.hk + head) << p.page_log2) + off;     // below 2^32
            dst = (char *)(is_v ? p.Vc : p.Kc) + (unsigned long long)line * p.row_bytes;
        } else if (slot != -1) {
            atomicOr(p.err, kErrInvalid);
        }
    } else {
        const unsigned *so = is_q ? p.sqo : p.sko;
        dst = (char *)(is_q ? p.Qo : p.Ko) + (unsigned long long)(bb * so[0] + i * so[1] + head * so[2]) * 16u;
    }
    const uintptr_t d = reinterpret_cast<uintptr_t>(dst);
    return Row{reinterpret_cast<uintptr_t>(src) + tt, d && !is_v ? d + 1 : d};
}

// kMode: 0 = halves in 16-byte pieces, 1 = interleaved in 16-byte pieces,
// 2 = a pair a place (the pairs do not start on 16-byte pieces; the channels
// behind them are copied 16 bytes at a time where they do).
template <typename T, int kMode, bool kAppend>
__global__ void __launch_bounds__(kThreads, kBlocks) k_rotary(const __grid_constant__ RotaryArgs p) {
    constexpr int kV = VecOf<T>::kN, kB = (int)sizeof(T);
    constexpr int kLoads = kMode == 0 ? 2 : 1, kUnroll = 4 / kLoads;   // rows of a thread in flight
    extern __shared__ __align__(16) float tabs[];      // two of [tile][2][rot / 2]: cos, sin of each token
    __shared__ Row lists[2][kMaxRows];
    const int half = p.rot / 2;
    const bool vcopy = kMode != 2 || p.rot * kB % 16 == 0;
    // places of a row: those whose pairs turn, then those copied
    const int nturn = kMode == 0 ? half / kV : kMode == 1 ? p.rot / kV : half;
    const int places = nturn + (vcopy ? (p.hd - p.rot) / kV : p.hd - p.rot);
    const int per_pass = places >= kThreads ? 1 : kThreads / places;   // rows of a pass
    const int place0 = threadIdx.x % places, q0 = threadIdx.x / places;
    const bool active = places >= kThreads || q0 < per_pass;           // not one of the threads left over
    // the block's share of the heads: gridDim.y slices
    const int lo = (int)((long long)p.rows * blockIdx.y / gridDim.y), mine = (int)((long long)p.rows * (blockIdx.y + 1) / gridDim.y) - lo;
    // x / mine and x / half for x < 2^15 by one multiplication
    const unsigned by_mine = 0xffffffffu / mine + 1u, by_half = half > 1 ? 0xffffffffu / half + 1u : 0u;

    // byte offset of a place in its row
    auto place_at = [&](int place) {
        return place < nturn ? 16 * place : vcopy ? (p.rot + (place - nturn) * kV) * kB : (p.rot + place - nturn) * kB;
    };
    auto fetch = [&](const Row *list, Row (&r)[kUnroll], uint4 (&v)[kUnroll][kLoads], int q, int at, bool copies, int total) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int e = q + u * per_pass;
            r[u].d = 0;
            if (e < total) r[u] = list[e];
            if (!r[u].d) continue;
            v[u][0] = load16(GPN(p.bnd, r[u].src() + at, 16));
            if (kMode == 0 && !copies) v[u][kLoads - 1] = load16(GPN(p.bnd, r[u].src() + at + half * kB, 16));
        }
    };
    // the rows and the table of the tile at token t0
    auto prepare = [&](long long t0, Row *list, float *tab) {
        const int nt = (int)(p.tokens - t0 < p.tile ? p.tokens - t0 : p.tile);
        for (int e = threadIdx.x; e < nt * mine; e += kThreads) {
            const unsigned tt = mine > 1 ? __umulhi(e, by_mine) : e;
            list[e] = row_of<kAppend>(p, (unsigned)t0 + tt, tt, lo + e - tt * mine);
        }
        for (int e = kThreads - 1 - threadIdx.x; e < nt * half; e += kThreads) {   // (the threads without a row first)
            const unsigned tt = half > 1 ? __umulhi(e, by_half) : e, k = e - tt * half, t = (unsigned)t0 + tt;
            const long long at = (p.pos ? (long long)*GP(p.bnd, p.pos + t) : (long long)(t % p.n)) + p.pos0;
            // the upper 32 bits of the fraction of a turn, less the nearest quarter:
            // at most an eighth of a turn is rounded to a float, not the whole angle
            const unsigned frac = (unsigned)(((unsigned long long)at * *GP(p.bnd, p.turns + k)) >> 32);
            const unsigned quarter = (frac + 0x20000000u) >> 30;
            float sn, cs;
            sincospif((float)(int)(frac - (quarter << 30)) * 0x1p-31f, &sn, &cs);
            if (quarter & 1u) {
                const float x = cs;
                cs = -sn;
                sn = x;
            }
            if (quarter & 2u) {
                cs = -cs;
                sn = -sn;
            }
            tab[(2 * tt) * half + k] = cs * p.scale;
            tab[(2 * tt + 1) * half + k] = sn * (p.backward ? -p.scale : p.scale);
        }
    };

    pdl_wait();
    pdl_trigger();
    const long long step = (long long)gridDim.x * p.tile;
    int buf = 0;
    prepare((long long)blockIdx.x * p.tile, lists[0], tabs);
    for (long long t0 = (long long)blockIdx.x * p.tile; t0 < p.tokens; t0 += step, buf ^= 1) {
        const int total = (int)(p.tokens - t0 < p.tile ? p.tokens - t0 : p.tile) * mine;
        const Row *list = lists[buf];
        const float *tab = tabs + buf * p.tile * p.rot;
        __syncthreads();                 // this tile is prepared, the other buffer is free
        // the next tile is prepared under this one's first loads
        const bool ahead = active && (kMode != 2 || (place0 >= nturn && vcopy));
        Row r[kUnroll];
        uint4 v[kUnroll][kLoads];
        if (ahead) fetch(list, r, v, q0, place_at(place0), place0 >= nturn, total);
        if (t0 + step < p.tokens) prepare(t0 + step, lists[buf ^ 1], tabs + (buf ^ 1) * p.tile * p.rot);
        for (int place = place0; place < places; place += kThreads) {
            if (!active) break;                  // the threads left over by a pass
            const bool copies = place >= nturn;
            const int at = place_at(place);
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
                if (!(ahead && place == place0 && q == q0)) fetch(list, r, v, q, at, copies, total);
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    if (!r[u].d) continue;
                    if (kMode != 2 && !copies && (!kAppend || r[u].turn())) {
                        constexpr int kPairs = kMode == 0 ? kV : kV / 2;
                        const float *tc = tab + 2 * r[u].token() * half + place * kPairs;
                        float c[kPairs], s[kPairs];
                        take<kPairs>(tc, c);
                        take<kPairs>(tc + half, s);
                        if constexpr (kMode == 0) {
                            float fa[kV], fb[kV];
                            unpack16<T>(v[u][0], fa);
                            unpack16<T>(v[u][kLoads - 1], fb);
#pragma unroll
                            for (int k = 0; k < kV; ++k) {
                                const float x = fa[k];
                                fa[k] = x * c[k] - fb[k] * s[k];
                                fb[k] = fb[k] * c[k] + x * s[k];
                            }
                            v[u][0] = pack16<T>(fa);
                            v[u][kLoads - 1] = pack16<T>(fb);
                        } else if constexpr (kMode == 1) {
                            float f[kV];
                            unpack16<T>(v[u][0], f);
#pragma unroll
                            for (int k = 0; k < kPairs; ++k) {
                                const float x = f[2 * k];
                                f[2 * k] = x * c[k] - f[2 * k + 1] * s[k];
                                f[2 * k + 1] = f[2 * k + 1] * c[k] + x * s[k];
                            }
                            v[u][0] = pack16<T>(f);
                        }
                    }
                    char *out = r[u].dst();
                    *reinterpret_cast<uint4 *>(GPN(p.bnd, out + at, 16)) = v[u][0];
                    if (kMode == 0 && !copies) *reinterpret_cast<uint4 *>(GPN(p.bnd, out + at + half * kB, 16)) = v[u][kLoads - 1];
                }
            }
        }
    }
}

template <typename T, bool kAppend>
cudaError_t launch_t(const RotaryArgs &a, int mode, dim3 grid, size_t smem, cudaStream_t st) {
    const auto fn = mode == 0 ? &k_rotary<T, 0, kAppend> : mode == 1 ? &k_rotary<T, 1, kAppend> : &k_rotary<T, 2, kAppend>;
    return launch_dependent(fn, grid, kThreads, smem, st, a);
}

}  // namespace

cudaError_t launch_rotary(DType dt, bool append, RotaryArgs a, cudaStream_t st) {
    const int es = dt == kF32 ? 4 : 2, vec = 16 / es;
    const int mode = a.rot == 0 ? 0 : a.interleaved ? (a.rot % vec == 0 ? 1 : 2) : (a.rot / 2 % vec == 0 ? 0 : 2);
    const int rows = a.hq + a.hk * (append ? 2 : 1);
    a.rows = rows;
    a.row_bytes = a.hd * es;
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidValue;
    // tokens of a block: about four rows a thread, but blocks enough for the GPU
    const int places = (mode == 0 ? a.rot / 2 : a.rot) / (mode == 2 ? 2 : vec) + (a.hd - a.rot) / vec;
    const long long items = (long long)rows * (places > 0 ? places : 1);
    const long long full = (long long)kBlocks * sms;          // blocks the GPU holds
    long long tile = std::min(4LL * kThreads / items, (a.tokens + full - 1) / full);
    tile = std::max(1LL, std::min(tile, (long long)kMaxTile));
    if (a.rot > 0) tile = std::min(tile, 32768LL / (2 * a.rot * (long long)sizeof(float)));   // two tables, 32 KB
    int slices = 1;                          // of the heads
    if (rows > kMaxRows) slices = (rows + kMaxRows - 1) / kMaxRows, tile = 1;
    else tile = std::max(1LL, std::min(tile, (long long)kMaxRows / rows));
    a.tile = (int)tile;
    const long long tiles = (a.tokens + a.tile - 1) / a.tile;
    // the GPU full once: the set-up of a block is then paid for by several tiles
    // (12 x 1365 tokens of 24 heads of 64: 19.8 us against 21.7 with a block a tile)
    const dim3 grid((unsigned)std::min(tiles, full), (unsigned)slices);
    const size_t smem = (size_t)2 * a.tile * a.rot * sizeof(float);
    if (dt == kF32) return append ? launch_t<float, true>(a, mode, grid, smem, st) : launch_t<float, false>(a, mode, grid, smem, st);
    if (dt == kF16) return append ? launch_t<__half, true>(a, mode, grid, smem, st) : launch_t<__half, false>(a, mode, grid, smem, st);
    return append ? launch_t<__nv_bfloat16, true>(a, mode, grid, smem, st) : launch_t<__nv_bfloat16, false>(a, mode, grid, smem, st);
}

}  // namespace swab
