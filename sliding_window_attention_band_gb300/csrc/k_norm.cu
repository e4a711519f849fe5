// k_norm.cu -- norms of queries and keys, a head at a time, with rotary positions
// in the same pass; the same fused with the write of K and V into the paged cache,
// in the tensors' type or in 4 bits; and the gradient.
//
// Forward.  A row x of head_dim channels becomes R(p) [x_c r v_c] with
//     r = 1 / sqrt(mean x^2 + eps),  v_c = w_c + offset
// and R the rotation of k_rotary.cu.  The channels of a pair have to meet, and a
// row's squares have to be summed: a row belongs to a group of 4 to 32 lanes of a
// warp, each with 16 bytes of either member of its pairs (any two pieces where
// the pairs are adjacent channels), so the rotation stays inside a lane and the
// sum is log2(lanes) shuffles.  Rows whose pairs do not start on 16 bytes, or wider
// than 32 lanes hold, go a warp a row through shared memory (kMode 2).
//
// A block takes a few tokens at a time: it lists their rows and fills a table of
// cosines and sines shared by all the heads, one buffer ahead (as k_rotary does);
// the weights lie in shared memory as floats.
//
// 4 bits.  A group of 32 channels is four pieces of 16-bit values, so four lanes:
// the value of largest magnitude is a maximum over the integers (bits << 1 | sign
// positive), two shuffles; the quotient x / s is decided exactly: the values have at
// most 11 significant bits and s 5, so a quotient that is no tie is 2^-13 off one,
// and fma(x, 1 / s, 768) rounds it to a multiple of 2^-14 before it is rounded to
// a whole number.
//
// Backward.  g = R^T dy, dx_c = r (g_c v_c - x_c r^2 mean(g v x)): two sums a row,
// one pass over x and dy.  dw_c = sum over rows of g_c x_c r: a lane adds up its
// channels over all its rows, a block writes one row of sums, a second kernel adds
// the blocks' in a fixed order.
//
// All of it is HBM-bound: every value read once and written once.
#include <algorithm>

#include "swab_rows.cuh"

static constexpr unsigned kSwabFile = 17;   // site id of the bounds checks

namespace swab {
namespace {

constexpr int kThreads = 256;
constexpr int kBlocks = 4;           // of an SM
constexpr int kMaxRows = 256;        // listed rows of a block at a time
constexpr int kMaxTile = 16;         // tokens of a block (Row::token)
constexpr int kIsQ = 1, kIsK = 2, kIsV = 3;

// One row of work: where from, where to.  Addresses are multiples of 16; the low
// bits carry the token of the tile and the kind of the row.  A row of a cache in 4
// bits has the number of its line in place of an address.  d = 0: nothing to write.
struct Row {
    uintptr_t s, d;
    __device__ __forceinline__ const char *src() const { return reinterpret_cast<const char *>(s & ~(uintptr_t)15); }
    __device__ __forceinline__ char *dst() const { return reinterpret_cast<char *>(d & ~(uintptr_t)15); }
    __device__ __forceinline__ unsigned line() const { return (unsigned)(d >> 4); }
    __device__ __forceinline__ int token() const { return (int)(s & 15u); }
    __device__ __forceinline__ int kind() const { return (int)(d & 15u); }
};

__device__ __forceinline__ unsigned long long row_units(const RotaryArgs &p, unsigned t, const unsigned *s, unsigned head) {
    unsigned bb = 0, i = t;
    if (p.n < p.tokens) {
        bb = t / p.n;
        i = t - bb * p.n;
    }
    return (unsigned long long)(bb * s[0] + i * s[1] + head * s[2]) * 16u;    // below 2^36 (checked by the caller)
}

// Row `idx` of token t: heads of Q, then of K, then (cache write) of V.
template <int kKind>
__device__ __forceinline__ Row row_of(const RotaryArgs &p, unsigned t, unsigned tt, int idx) {
    const bool is_q = idx < p.hq;
    unsigned head = is_q ? idx : idx - p.hq;
    const bool is_v = kKind > 0 && !is_q && head >= (unsigned)p.hk;
    if (is_v) head -= p.hk;
    const char *src = (const char *)(is_q ? p.Q : is_v ? p.V : p.K) + row_units(p, t, is_q ? p.sq : is_v ? p.sv : p.sk, head);
    const int kind = is_q ? kIsQ : is_v ? kIsV : kIsK;
    uintptr_t d = 0;
    if (kKind > 0 && !is_q) {
        const int slot = *GP(p.bnd, p.slots + t);
        if (slot >= 0 && slot < p.n_slots) {
            const unsigned blk = (unsigned)slot >> p.page_log2, off = (unsigned)slot & ((1u << p.page_log2) - 1u);
            const unsigned line = ((blk * (unsigned)p.hk + head) << p.page_log2) + off;     // below 2^32
            if (kKind == 2) d = ((uintptr_t)line << 4) + kind;
            else d = reinterpret_cast<uintptr_t>((char *)(is_v ? p.Vc : p.Kc) + (unsigned long long)line * p.row_bytes) + kind;
        } else if (slot != -1) {
            atomicOr(p.err, kErrInvalid);
        }
    } else {
        d = reinterpret_cast<uintptr_t>((char *)(is_q ? p.Qo : p.Ko) + row_units(p, t, is_q ? p.sqo : p.sko, head)) + kind;
    }
    return Row{reinterpret_cast<uintptr_t>(src) + tt, d};
}

// ---------------------------------------------------------------------------
// 4 bits
// ---------------------------------------------------------------------------
// Order of magnitude, the positive of two equal ones first: (|x| as bits) << 1 | x > 0.
__device__ __forceinline__ unsigned rank_of(float x) {
    const unsigned b = __float_as_uint(x);
    return (b << 1) | (~b >> 31);
}
template <typename T> struct Scale4;
template <> struct Scale4<__half> {
    static constexpr int kFloor = -24;       // a scale is a multiple of 2 to this ...
    static constexpr float kMost = 2560.f;   // ... and at most that
};
template <> struct Scale4<__nv_bfloat16> {
    static constexpr int kFloor = -120;
    static constexpr float kMost = 0x1.4p123f;
};
template <> struct Scale4<float> {
    static constexpr int kFloor = -120;
    static constexpr float kMost = 0x1.4p123f;
};
// The scale of a group whose largest value has this rank: m / -8 in 5 significant
// bits (ties to even); NaN where m is not finite.
template <typename T> __device__ __forceinline__ float scale_of(unsigned rank) {
    constexpr float kSmall = Scale4<T>::kFloor == -24 ? 0x1p-20f : 0x1p-116f;    // below: a multiple of the floor
    constexpr float kMagic = Scale4<T>::kFloor == -24 ? 0x1.8p-1f : 0x1.8p-97f;  // 1.5 * 2^23 floors
    const unsigned mag = rank >> 1;
    if (mag >= 0x7f800000u) return __uint_as_float(0x7fffffffu);
    const float a = __uint_as_float(mag) * 0.125f;
    const unsigned b = __float_as_uint(a);
    float s = __uint_as_float((b + 0x3ffffu + ((b >> 19) & 1u)) & ~0x7ffffu);
    if (a < kSmall) s = __fsub_rn(__fadd_rn(a, kMagic), kMagic);
    s = fminf(s, Scale4<T>::kMost);
    return (rank & 1u) && s != 0.f ? -s : s;
}
// Code of x under scale s: inv = 1 / s, or 0 (code 8) where s is 0 or NaN.
__device__ __forceinline__ int code_of(float x, float inv) {
    const float t = __fsub_rn(__fmaf_rn(x, inv, 768.f), 768.f);     // |x / s| < 26: a multiple of 2^-14
    const int n = (int)(__float_as_uint(__fadd_rn(t, 12582912.f)) - 0x4b400000u);   // to the nearest, ties to even
    return min(max(n, -8), 7) + 8;
}

// A lane's 16 bytes of a group as 16-bit values (already rounded): eight codes as a
// word, and the group's scale.  Four adjacent lanes hold the group.
template <typename T>
__device__ __forceinline__ uint32_t quantise8(const float (&x)[8], float &s) {
    unsigned rank = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) rank = max(rank, rank_of(x[k]));
    rank = max(rank, __shfl_xor_sync(0xffffffffu, rank, 1));
    rank = max(rank, __shfl_xor_sync(0xffffffffu, rank, 2));
    s = scale_of<T>(rank);
    const bool none = !(fabsf(s) > 0.f);                             // 0 or NaN
    const float inv = none ? 0.f : __frcp_rn(s);
    uint32_t w = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) w |= (uint32_t)code_of(none ? 0.f : x[k], inv) << (4 * k);
    return w;
}

// 1 / sqrt(mean of squares + eps)
__device__ __forceinline__ float inverse_norm(float sum, float hd, float eps) { return __frsqrt_rn(__fdiv_rn(sum, hd) + eps); }

// A pair turned, rounded as k_rotary does (so that the cache holds the same bits
// with and without norms, in either width): pieces, and pair by pair.
__device__ __forceinline__ void turn(float &a, float &b, float c, float s, bool by_pairs = false) {
    const float x = a;
    a = __fmaf_rn(x, c, -__fmul_rn(b, s));
    b = by_pairs ? __fmaf_rn(b, c, __fmul_rn(x, s)) : __fmaf_rn(x, s, __fmul_rn(b, c));
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
// kMode: 0 = halves in 16-byte pieces, 1 = adjacent pairs in 16-byte pieces, 2 = a
// warp a row.  kKind: 0 = Q, K -> Qo, Ko; 1 = into the cache; 2 = into the cache in
// 4 bits (kMode 0, 1: 16-bit types, groups on four lanes).
template <typename T, int kMode, int kKind>
__global__ void __launch_bounds__(kThreads, kBlocks) k_norm(const __grid_constant__ NormArgs a) {
    constexpr int kV = VecOf<T>::kN, kUnroll = 2;
    const RotaryArgs &p = a.r;
    extern __shared__ __align__(16) float smem[];      // two tables [tile][2][rot / 2]; weights [2][hd]; (mode 2) a row a warp
    __shared__ Row lists[2][kMaxRows];
    const int half = p.rot / 2;
    float *wtab = smem + 2 * p.tile * p.rot;
    const int lo = (int)((long long)p.rows * blockIdx.y / gridDim.y), mine = (int)((long long)p.rows * (blockIdx.y + 1) / gridDim.y) - lo;
    const unsigned by_mine = 0xffffffffu / mine + 1u, by_half = half > 1 ? 0xffffffffu / half + 1u : 0u;   // x / mine, x / half for x < 2^15

    // the lanes of a row and this lane's two pieces of it
    const int L = a.lanes, sub = threadIdx.x & (L - 1), q0 = threadIdx.x / L, per_pass = kThreads / L;
    const int pieces = p.hd / kV, nturn = kMode == 0 ? half / kV : 0;
    const bool active = sub < pieces / 2;
    const int pa = sub < nturn ? sub : nturn + sub, pb = sub < nturn ? sub + nturn : pieces / 2 + sub;

    // the rows and the table of the tile at token t0
    auto prepare = [&](long long t0, Row *list, float *tab) {
        const int nt = (int)(p.tokens - t0 < p.tile ? p.tokens - t0 : p.tile);
        for (int e = threadIdx.x; e < nt * mine; e += kThreads) {
            const unsigned tt = mine > 1 ? __umulhi(e, by_mine) : e;
            list[e] = row_of<kKind>(p, (unsigned)t0 + tt, tt, lo + e - tt * mine);
        }
        for (int e = kThreads - 1 - threadIdx.x; e < nt * half; e += kThreads) {   // (the threads without a row first)
            const unsigned tt = half > 1 ? __umulhi(e, by_half) : e, k = e - tt * half, t = (unsigned)t0 + tt;
            const long long at = (p.pos ? (long long)*GP(p.bnd, p.pos + t) : (long long)(t % p.n)) + p.pos0;
            float cs, sn;
            cos_sin(at, *GP(p.bnd, p.turns + k), cs, sn);
            tab[(2 * tt) * half + k] = cs * p.scale;
            tab[(2 * tt + 1) * half + k] = sn * p.scale;
        }
    };

    pdl_wait();
    pdl_trigger();
    for (int c = threadIdx.x; c < 2 * p.hd; c += kThreads) {
        const T *w = reinterpret_cast<const T *>(c < p.hd ? a.wq : a.wk);
        wtab[c] = w ? Elt<T>::to_f(*GP(p.bnd, w + (c < p.hd ? c : c - p.hd))) + a.offset : 1.f;
    }
    const long long step = (long long)gridDim.x * p.tile;
    int buf = 0;
    prepare((long long)blockIdx.x * p.tile, lists[0], smem);
    for (long long t0 = (long long)blockIdx.x * p.tile; t0 < p.tokens; t0 += step, buf ^= 1) {
        const int total = (int)(p.tokens - t0 < p.tile ? p.tokens - t0 : p.tile) * mine;
        const Row *list = lists[buf];
        const float *tab = smem + buf * p.tile * p.rot;
        __syncthreads();                 // this tile is prepared, the other buffer is free
        if constexpr (kMode < 2) {
            Row r[kUnroll];
            uint4 va[kUnroll], vb[kUnroll];
            auto fetch = [&](int q) {
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    const int e = q + q0 + u * per_pass;
                    r[u].s = r[u].d = 0;
                    va[u] = vb[u] = make_uint4(0, 0, 0, 0);
                    if (e < total) r[u] = list[e];
                    if (!r[u].d || !active) continue;
                    va[u] = load16(GPN(p.bnd, r[u].src() + pa * 16, 16));
                    vb[u] = load16(GPN(p.bnd, r[u].src() + pb * 16, 16));
                }
            };
            // the next tile is prepared under this one's first loads
            fetch(0);
            if (t0 + step < p.tokens) prepare(t0 + step, lists[buf ^ 1], smem + (buf ^ 1) * p.tile * p.rot);
            for (int q = 0; q < total; q += kUnroll * per_pass) {
                if (q > 0) fetch(q);
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    const int kind = r[u].kind();
                    float fa[kV], fb[kV];
                    unpack16<T>(va[u], fa);
                    unpack16<T>(vb[u], fb);
                    if (a.norm) {
                        float sum = 0.f;
#pragma unroll
                        for (int k = 0; k < kV; ++k) sum = fmaf(fa[k], fa[k], fmaf(fb[k], fb[k], sum));
                        for (int d = L / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                        if (kKind == 0 || kind != kIsV) {
                            const float rn = inverse_norm(sum, (float)p.hd, a.eps);
                            const float *w = wtab + (kind == kIsQ ? 0 : p.hd);
                            if (active) {
                                float c[kV];
                                take<kV>(w + pa * kV, c);
#pragma unroll
                                for (int k = 0; k < kV; ++k) fa[k] *= rn * c[k];
                                take<kV>(w + pb * kV, c);
#pragma unroll
                                for (int k = 0; k < kV; ++k) fb[k] *= rn * c[k];
                            }
                        }
                    }
                    if (active && (kKind == 0 || kind != kIsV)) {
                        const float *cs = tab + 2 * r[u].token() * half;
                        if constexpr (kMode == 0) {
                            if (sub < nturn) {
                                float c[kV], s[kV];
                                take<kV>(cs + pa * kV, c);
                                take<kV>(cs + half + pa * kV, s);
#pragma unroll
                                for (int k = 0; k < kV; ++k) turn(fa[k], fb[k], c[k], s[k]);
                            }
                        } else {
                            auto turn_piece = [&](float (&f)[kV], int piece) {
                                if (piece * kV >= p.rot) return;
                                float c[kV / 2], s[kV / 2];
                                take<kV / 2>(cs + piece * (kV / 2), c);
                                take<kV / 2>(cs + half + piece * (kV / 2), s);
#pragma unroll
                                for (int k = 0; k < kV / 2; ++k) turn(f[2 * k], f[2 * k + 1], c[k], s[k]);
                            };
                            turn_piece(fa, pa);
                            turn_piece(fb, pb);
                        }
                    }
                    const uint4 ya = pack16<T>(fa), yb = pack16<T>(fb);
                    if constexpr (kKind == 2 && sizeof(T) == 2) {
                        if (__any_sync(0xffffffffu, kind >= kIsK)) {
                            float s0, s1;
                            unpack16<T>(ya, fa);                     // as the cache of this type would hold them
                            unpack16<T>(yb, fb);
                            const uint32_t wa = quantise8<T>(fa, s0), wb = quantise8<T>(fb, s1);
                            if (kind >= kIsK && active) {
                                const unsigned long long line = r[u].line();
                                char *codes = (char *)(kind == kIsV ? p.Vc : p.Kc) + line * (p.hd / 2);
                                T *sc = (T *)(kind == kIsV ? a.Vs : a.Ks) + line * (p.hd / kGroup4);
                                *reinterpret_cast<uint32_t *>(GPN(p.bnd, codes + pa * 4, 4)) = wa;
                                *reinterpret_cast<uint32_t *>(GPN(p.bnd, codes + pb * 4, 4)) = wb;
                                if ((sub & 3) == 0) {
                                    *GP(p.bnd, sc + pa / 4) = Elt<T>::from_f(s0);
                                    *GP(p.bnd, sc + pb / 4) = Elt<T>::from_f(s1);
                                }
                            }
                        }
                    }
                    if (!r[u].d || !active || (kKind == 2 && kind != kIsQ)) continue;
                    *reinterpret_cast<uint4 *>(GPN(p.bnd, r[u].dst() + pa * 16, 16)) = ya;
                    *reinterpret_cast<uint4 *>(GPN(p.bnd, r[u].dst() + pb * 16, 16)) = yb;
                }
            }
        } else {
            if (t0 + step < p.tokens) prepare(t0 + step, lists[buf ^ 1], smem + (buf ^ 1) * p.tile * p.rot);
            const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
            float *x = wtab + 2 * p.hd + warp * p.hd;
            for (int e = warp; e < total; e += kThreads / 32) {
                const Row r = list[e];
                if (!r.d) continue;
                const int kind = r.kind();
                const T *src = reinterpret_cast<const T *>(r.src());
                for (int c = lane; c < p.hd; c += 32) x[c] = Elt<T>::to_f(*GP(p.bnd, src + c));
                if (kind != kIsV) {
                    if (a.norm) {
                        __syncwarp();
                        float sum = 0.f;
                        if (a.sum_lanes) {               // in the order of the lanes that own pieces
                            const int na = a.sum_turn, la = lane < na ? lane : na + lane, lb = lane < na ? lane + na : pieces / 2 + lane;
                            if (lane < pieces / 2)
                                for (int k = 0; k < kV; ++k) sum = fmaf(x[la * kV + k], x[la * kV + k], fmaf(x[lb * kV + k], x[lb * kV + k], sum));
                            for (int d = a.sum_lanes / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                            sum = __shfl_sync(0xffffffffu, sum, 0);
                        } else {
                            for (int c = lane; c < p.hd; c += 32) sum = fmaf(x[c], x[c], sum);
#pragma unroll
                            for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                        }
                        __syncwarp();
                        const float rn = inverse_norm(sum, (float)p.hd, a.eps);
                        const float *w = wtab + (kind == kIsQ ? 0 : p.hd);
                        for (int c = lane; c < p.hd; c += 32) x[c] *= rn * w[c];
                    }
                    __syncwarp();
                    const float *cs = tab + 2 * r.token() * half;
                    for (int k = lane; k < half; k += 32) {
                        const int one = p.interleaved ? 2 * k : k, two = p.interleaved ? 2 * k + 1 : k + half;
                        float xa = x[one], xb = x[two];
                        turn(xa, xb, cs[k], cs[half + k], a.by_pairs);
                        x[one] = xa;
                        x[two] = xb;
                    }
                }
                __syncwarp();
                if (kKind == 2 && kind != kIsQ) {
                    const unsigned long long line = r.line();
                    char *codes = (char *)(kind == kIsV ? p.Vc : p.Kc) + line * (p.hd / 2);
                    T *sc = (T *)(kind == kIsV ? a.Vs : a.Ks) + line * (p.hd / kGroup4);
                    for (int g = 0; g < p.hd / kGroup4; ++g) {       // a lane a channel
                        const float f = Elt<T>::to_f(Elt<T>::from_f(x[g * kGroup4 + lane]));
                        const float s = scale_of<T>(__reduce_max_sync(0xffffffffu, rank_of(f)));
                        // (fp32 quotients have ties of their own: divided as they are)
                        const float y = fabsf(s) > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(f, s)), -8.f), 7.f) : 0.f;
                        uint32_t w = (uint32_t)((int)y + 8) << (4 * (lane & 7));
                        w |= __shfl_xor_sync(0xffffffffu, w, 1);
                        w |= __shfl_xor_sync(0xffffffffu, w, 2);
                        w |= __shfl_xor_sync(0xffffffffu, w, 4);
                        if ((lane & 7) == 0) *reinterpret_cast<uint32_t *>(GPN(p.bnd, codes + g * 16 + lane / 2, 4)) = w;
                        if (lane == 0) *GP(p.bnd, sc + g) = Elt<T>::from_f(s);
                    }
                } else {
                    T *dst = reinterpret_cast<T *>(r.dst());
                    for (int c = lane; c < p.hd; c += 32) *GP(p.bnd, dst + c) = Elt<T>::from_f(x[c]);
                }
                __syncwarp();
            }
        }
    }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
struct BwdRow {
    uintptr_t g, x, d;         // of dy (low bits: the token of the tile), x, dx (0: none)
};
constexpr int kBwdRows = 256;

// Blocks 0 .. blocks_q - 1 take the rows of Q, the others those of K: each has the
// weight gradient of one of them.  kMode as above.
template <typename T, int kMode>
__global__ void __launch_bounds__(kThreads, 2) k_norm_bwd(const __grid_constant__ NormArgs a) {
    constexpr int kV = VecOf<T>::kN, kUnroll = sizeof(T) == 2 && kMode < 2 ? 2 : 1;
    const RotaryArgs &p = a.r;
    extern __shared__ __align__(16) float smem[];      // two tables [tile][2][rot / 2]; weights [hd]; sums [kThreads / L][hd] or, mode 2, rows
    __shared__ BwdRow lists[2][kBwdRows];
    const int which = blockIdx.x >= a.blocks_q, heads = which ? p.hk : p.hq;
    const int first = which ? blockIdx.x - a.blocks_q : blockIdx.x, nblocks = which ? a.blocks - a.blocks_q : a.blocks_q;
    const int tile = a.tile[which], slices = a.slices[which];
    const long long work = (long long)a.tiles[which] * slices;
    const int half = p.rot / 2;
    const int table = 2 * max(a.tile[0], a.tile[1]) * p.rot;
    float *wtab = smem + table, *sums = wtab + p.hd;

    const int L = a.lanes, sub = threadIdx.x & (L - 1), q0 = threadIdx.x / L, per_pass = kThreads / L;
    const int pieces = p.hd / kV, nturn = kMode == 0 ? half / kV : 0;
    const bool active = sub < pieces / 2;
    const int pa = sub < nturn ? sub : nturn + sub, pb = sub < nturn ? sub + nturn : pieces / 2 + sub;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

    // unit of work u: the heads of slice u % slices of the tokens of tile u / slices
    auto prepare = [&](long long u, BwdRow *list, float *tab) -> int {
        const int slice = (int)(u % slices), lo = (int)((long long)heads * slice / slices), mine = (int)((long long)heads * (slice + 1) / slices) - lo;
        const long long t0 = u / slices * tile;
        const int nt = (int)(p.tokens - t0 < tile ? p.tokens - t0 : tile);
        const unsigned *sg = which ? p.sk : p.sq, *sd = which ? p.sko : p.sqo;
        for (int e = threadIdx.x; e < nt * mine; e += kThreads) {
            const unsigned tt = e / mine, head = lo + e - tt * mine, t = (unsigned)t0 + tt;
            list[e].g = reinterpret_cast<uintptr_t>((const char *)(which ? p.K : p.Q) + row_units(p, t, sg, head)) + tt;
            list[e].x = reinterpret_cast<uintptr_t>((const char *)a.X[which] + row_units(p, t, a.sx[which], head));
            list[e].d = reinterpret_cast<uintptr_t>((char *)(which ? p.Ko : p.Qo) + row_units(p, t, sd, head));
        }
        for (int e = kThreads - 1 - threadIdx.x; e < nt * half; e += kThreads) {
            const unsigned tt = e / half, k = e - tt * half, t = (unsigned)t0 + tt;
            const long long at = (p.pos ? (long long)*GP(p.bnd, p.pos + t) : (long long)(t % p.n)) + p.pos0;
            float cs, sn;
            cos_sin(at, *GP(p.bnd, p.turns + k), cs, sn);
            tab[(2 * tt) * half + k] = cs * p.scale;
            tab[(2 * tt + 1) * half + k] = sn * p.scale;
        }
        return nt * mine;
    };
    // R^T on a lane's pieces
    auto back = [&](const float *cs, float (&ga)[kV], float (&gb)[kV]) {
        if constexpr (kMode == 0) {
            if (sub < nturn) {
                float c[kV], s[kV];
                take<kV>(cs + pa * kV, c);
                take<kV>(cs + half + pa * kV, s);
#pragma unroll
                for (int k = 0; k < kV; ++k) {
                    const float x = ga[k];
                    ga[k] = x * c[k] + gb[k] * s[k];
                    gb[k] = gb[k] * c[k] - x * s[k];
                }
            }
        } else {
            auto turn = [&](float (&f)[kV], int piece) {
                if (piece * kV >= p.rot) return;
                float c[kV / 2], s[kV / 2];
                take<kV / 2>(cs + piece * (kV / 2), c);
                take<kV / 2>(cs + half + piece * (kV / 2), s);
#pragma unroll
                for (int k = 0; k < kV / 2; ++k) {
                    const float x = f[2 * k];
                    f[2 * k] = x * c[k] + f[2 * k + 1] * s[k];
                    f[2 * k + 1] = f[2 * k + 1] * c[k] - x * s[k];
                }
            };
            turn(ga, pa);
            turn(gb, pb);
        }
    };

    pdl_wait();
    pdl_trigger();
    const T *w = reinterpret_cast<const T *>(which ? a.wk : a.wq);
    for (int c = threadIdx.x; c < p.hd; c += kThreads) wtab[c] = w ? Elt<T>::to_f(*GP(p.bnd, w + c)) + a.offset : 1.f;
    float da[kV], db[kV];              // this lane's share of dw (mode 2: in shared memory, a row a warp)
#pragma unroll
    for (int k = 0; k < kV; ++k) da[k] = db[k] = 0.f;
    float *dsum = sums + warp * 3 * p.hd, *sx = dsum + p.hd, *sg = sx + p.hd;     // mode 2
    if constexpr (kMode == 2)
        for (int c = lane; c < p.hd; c += 32) dsum[c] = 0.f;

    int buf = 0, total = prepare(first, lists[0], smem);
    for (long long u0 = first; u0 < work; u0 += nblocks, buf ^= 1) {
        const BwdRow *list = lists[buf];
        const float *tab = smem + buf * (table / 2);
        const bool more = u0 + nblocks < work;
        int next = 0;
        __syncthreads();                 // this tile is prepared, the other buffer is free
        if constexpr (kMode < 2) {
            BwdRow r[kUnroll];
            uint4 xa[kUnroll], xb[kUnroll], ga[kUnroll], gb[kUnroll];
            auto fetch = [&](int q) {
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    const int e = q + q0 + u * per_pass;
                    r[u].d = r[u].g = 0;
                    xa[u] = xb[u] = ga[u] = gb[u] = make_uint4(0, 0, 0, 0);
                    if (e >= total || !active) continue;
                    r[u] = list[e];
                    const char *x = reinterpret_cast<const char *>(r[u].x), *g = reinterpret_cast<const char *>(r[u].g & ~(uintptr_t)15);
                    xa[u] = load16(GPN(p.bnd, x + pa * 16, 16));
                    xb[u] = load16(GPN(p.bnd, x + pb * 16, 16));
                    ga[u] = load16(GPN(p.bnd, g + pa * 16, 16));
                    gb[u] = load16(GPN(p.bnd, g + pb * 16, 16));
                }
            };
            fetch(0);
            if (more) next = prepare(u0 + nblocks, lists[buf ^ 1], smem + (buf ^ 1) * (table / 2));
            for (int q = 0; q < total; q += kUnroll * per_pass) {
                if (q > 0) fetch(q);
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    float fa[kV], fb[kV], ya[kV], yb[kV], va[kV], vb[kV];
                    unpack16<T>(xa[u], fa);
                    unpack16<T>(xb[u], fb);
                    unpack16<T>(ga[u], ya);
                    unpack16<T>(gb[u], yb);
#pragma unroll
                    for (int k = 0; k < kV; ++k) va[k] = vb[k] = 0.f;
                    if (active) {
                        back(tab + 2 * (int)(r[u].g & 15u) * half, ya, yb);
                        take<kV>(wtab + pa * kV, va);
                        take<kV>(wtab + pb * kV, vb);
                    }
                    float sum = 0.f, dot = 0.f;
#pragma unroll
                    for (int k = 0; k < kV; ++k) {
                        sum = fmaf(fa[k], fa[k], fmaf(fb[k], fb[k], sum));
                        va[k] *= ya[k];
                        vb[k] *= yb[k];
                        dot = fmaf(va[k], fa[k], fmaf(vb[k], fb[k], dot));
                    }
                    for (int d = L / 2; d > 0; d >>= 1) {
                        sum += __shfl_xor_sync(0xffffffffu, sum, d);
                        dot += __shfl_xor_sync(0xffffffffu, dot, d);
                    }
                    if (!r[u].d) continue;
                    const float rn = inverse_norm(sum, (float)p.hd, a.eps), c2 = dot / (float)p.hd * rn * rn;
#pragma unroll
                    for (int k = 0; k < kV; ++k) {
                        da[k] = fmaf(ya[k], fa[k] * rn, da[k]);
                        db[k] = fmaf(yb[k], fb[k] * rn, db[k]);
                        fa[k] = rn * fmaf(-c2, fa[k], va[k]);
                        fb[k] = rn * fmaf(-c2, fb[k], vb[k]);
                    }
                    char *d = reinterpret_cast<char *>(r[u].d);
                    *reinterpret_cast<uint4 *>(GPN(p.bnd, d + pa * 16, 16)) = pack16<T>(fa);
                    *reinterpret_cast<uint4 *>(GPN(p.bnd, d + pb * 16, 16)) = pack16<T>(fb);
                }
            }
        } else {
            if (more) next = prepare(u0 + nblocks, lists[buf ^ 1], smem + (buf ^ 1) * (table / 2));
            for (int e = warp; e < total; e += kThreads / 32) {
                const BwdRow r = list[e];
                const T *x = reinterpret_cast<const T *>(r.x), *g = reinterpret_cast<const T *>(r.g & ~(uintptr_t)15);
                const float *cs = tab + 2 * (int)(r.g & 15u) * half;
                float sum = 0.f, dot = 0.f;
                for (int c = lane; c < p.hd; c += 32) {
                    const float f = Elt<T>::to_f(*GP(p.bnd, x + c));
                    sum = fmaf(f, f, sum);
                    sx[c] = f;
                    sg[c] = Elt<T>::to_f(*GP(p.bnd, g + c));
                }
                __syncwarp();
                for (int k = lane; k < half; k += 32) {
                    const int one = p.interleaved ? 2 * k : k, two = p.interleaved ? 2 * k + 1 : k + half;
                    const float y1 = sg[one], y2 = sg[two], c = cs[k], s = cs[half + k];
                    sg[one] = y1 * c + y2 * s;
                    sg[two] = y2 * c - y1 * s;
                }
                __syncwarp();
                for (int c = lane; c < p.hd; c += 32) dot = fmaf(sg[c] * wtab[c], sx[c], dot);
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) {
                    sum += __shfl_xor_sync(0xffffffffu, sum, d);
                    dot += __shfl_xor_sync(0xffffffffu, dot, d);
                }
                const float rn = inverse_norm(sum, (float)p.hd, a.eps), c2 = dot / (float)p.hd * rn * rn;
                T *d = reinterpret_cast<T *>(r.d);
                for (int c = lane; c < p.hd; c += 32) {
                    dsum[c] = fmaf(sg[c], sx[c] * rn, dsum[c]);
                    *GP(p.bnd, d + c) = Elt<T>::from_f(rn * fmaf(-c2, sx[c], sg[c] * wtab[c]));
                }
                __syncwarp();
            }
        }
        total = next;
    }
    if (!a.dw[which]) return;
    // the block's sums, in the order of its row groups
    int rows = kThreads / 32, stride = 3 * p.hd;
    if constexpr (kMode < 2) {
        rows = per_pass;
        stride = p.hd;
        if (active) {
#pragma unroll
            for (int k = 0; k < kV; ++k) {
                sums[q0 * p.hd + pa * kV + k] = da[k];
                sums[q0 * p.hd + pb * kV + k] = db[k];
            }
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.hd; c += kThreads) {
        float s = 0.f;
        for (int q = 0; q < rows; ++q) s += sums[q * stride + c];
        *GP(p.bnd, a.part + (long long)blockIdx.x * p.hd + c) = s;
    }
}

// dw: the blocks' sums added, 32 channels a block, 32 threads a channel.
__global__ void __launch_bounds__(1024) k_norm_dw(const __grid_constant__ NormArgs a) {
    __shared__ float s[32][33];
    const RotaryArgs &p = a.r;
    const int which = blockIdx.y, c = blockIdx.x * 32 + (threadIdx.x & 31), seg = threadIdx.x >> 5;
    const int lo = which ? a.blocks_q : 0, hi = which ? a.blocks : a.blocks_q;
    pdl_wait();
    pdl_trigger();
    if (!a.dw[which]) return;
    float x = 0.f;
    if (c < p.hd) {
#pragma unroll 8
        for (int b = lo + seg; b < hi; b += 32) x += *GP(p.bnd, a.part + (long long)b * p.hd + c);
    }
    s[seg][threadIdx.x & 31] = x;
    __syncthreads();
    x = s[threadIdx.x & 31][seg];                        // a warp a channel now
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    if ((threadIdx.x & 31) == 0 && blockIdx.x * 32 + seg < p.hd) *GP(p.bnd, a.dw[which] + blockIdx.x * 32 + seg) = x;
}

// ---------------------------------------------------------------------------
// rows of a cache in 4 bits as values: a thread a word of codes (8 channels)
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(kThreads) k_read4(const __grid_constant__ Read4Args p) {
    const int words = p.hd / 8;
    const long long per_token = 2LL * p.hk * words, items = per_token * p.tokens;
    pdl_wait();
    pdl_trigger();
    for (long long e = (long long)blockIdx.x * kThreads + threadIdx.x; e < items; e += (long long)gridDim.x * kThreads) {
        const long long t = e / per_token;
        const int in = (int)(e - t * per_token), is_v = in >= p.hk * words, row = (is_v ? in - p.hk * words : in) / words;
        const int word = in % words;
        const int slot = *GP(p.bnd, p.slots + t);
        if (slot < 0 || slot >= p.n_slots) {
            if (slot != -1 && in == 0) atomicOr(p.err, kErrInvalid);
            continue;
        }
        const unsigned blk = (unsigned)slot >> p.page_log2, off = (unsigned)slot & ((1u << p.page_log2) - 1u);
        const unsigned long long line = ((blk * (unsigned)p.hk + row) << p.page_log2) + off;
        const uint32_t w = *GP(p.bnd, reinterpret_cast<const uint32_t *>(is_v ? p.Vc : p.Kc) + line * words + word);
        const float s = Elt<T>::to_f(*GP(p.bnd, reinterpret_cast<const T *>(is_v ? p.Vs : p.Ks) + line * (p.hd / kGroup4) + word / 4));
        float f[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = s * (float)((int)((w >> (4 * k)) & 15u) - 8);
        T *dst = reinterpret_cast<T *>(is_v ? p.V : p.K) + (t * p.hk + row) * p.hd + word * 8;
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<uint4 *>(GPN(p.bnd, dst, 16)) = pack16<T>(f);
            *reinterpret_cast<uint4 *>(GPN(p.bnd, dst + 4, 16)) = pack16<T>(f + 4);
        } else {
            *reinterpret_cast<uint4 *>(GPN(p.bnd, dst, 16)) = pack16<T>(f);
        }
    }
}

// Which kernel takes the rows: halves or adjacent pairs in 16-byte pieces on at
// most 32 lanes (and, into 4 bits, 16-bit types whose groups lie on four lanes),
// else a warp a row.  lanes: of a row, a power of two from 4.
int mode_of(const RotaryArgs &r, int es, bool bits4, int *lanes, NormArgs *a = nullptr) {
    const int vec = 16 / es, pieces = r.hd / vec, half = r.rot / 2;
    int L = 4;
    while (L < pieces / 2) L *= 2;
    *lanes = L;
    const int nturn = r.interleaved || r.rot == 0 ? 0 : half / vec;
    const bool on_pieces = r.interleaved || r.rot == 0 ? r.rot % vec == 0 : half % vec == 0;
    bool fits = pieces % 2 == 0 && L <= 32 && on_pieces;
    if (a) {
        a->by_pairs = !on_pieces;
        a->sum_lanes = fits ? L : 0;
        a->sum_turn = nturn;
    }
    if (bits4) fits = fits && es == 2 && nturn % 4 == 0 && (pieces - 2 * nturn) % 8 == 0;
    if (!fits) *lanes = 32;
    return !fits ? 2 : r.interleaved ? 1 : 0;
}

template <typename T, int kKind>
cudaError_t launch_t(const NormArgs &a, int mode, dim3 grid, size_t smem, cudaStream_t st) {
    if constexpr (kKind == 2 && sizeof(T) == 4) return launch_dependent(&k_norm<T, 2, kKind>, grid, kThreads, smem, st, a);
    else {
        const auto fn = mode == 0 ? &k_norm<T, 0, kKind> : mode == 1 ? &k_norm<T, 1, kKind> : &k_norm<T, 2, kKind>;
        return launch_dependent(fn, grid, kThreads, smem, st, a);
    }
}
template <typename T>
cudaError_t launch_kind(int kind, const NormArgs &a, int mode, dim3 grid, size_t smem, cudaStream_t st) {
    return kind == 0 ? launch_t<T, 0>(a, mode, grid, smem, st) : kind == 1 ? launch_t<T, 1>(a, mode, grid, smem, st)
                                                                           : launch_t<T, 2>(a, mode, grid, smem, st);
}

constexpr long long kTable = 16384;      // bytes of the two tables at most

// tokens of a block at a time and slices of the heads: about four rows a lane group,
// but units enough for `full` blocks
void tile_of(const RotaryArgs &r, int rows, int lanes, long long full, int most_rows, int *tile_out, int *slices_out) {
    long long tile = std::min(4LL * kThreads / ((long long)rows * lanes), (r.tokens + full - 1) / full);
    tile = std::max(1LL, std::min(tile, (long long)kMaxTile));
    if (r.rot > 0) tile = std::min(tile, kTable / (2 * r.rot * (long long)sizeof(float)));
    int slices = 1;
    if (rows > most_rows) slices = (rows + most_rows - 1) / most_rows, tile = 1;
    else tile = std::max(1LL, std::min(tile, (long long)most_rows / rows));
    *tile_out = (int)tile;
    *slices_out = slices;
}

}  // namespace

cudaError_t launch_norm(DType dt, int kind, NormArgs a, cudaStream_t st) {
    const int es = dt == kF32 ? 4 : 2;
    const int mode = mode_of(a.r, es, kind == 2, &a.lanes, &a);
    a.r.rows = a.r.hq + a.r.hk * (kind ? 2 : 1);
    a.r.row_bytes = a.r.hd * es;
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidValue;
    const long long full = (long long)kBlocks * sms;
    int slices = 1;
    tile_of(a.r, a.r.rows, a.lanes, full, kMaxRows, &a.r.tile, &slices);
    const long long tiles = ((long long)a.r.tokens + a.r.tile - 1) / a.r.tile;
    const dim3 grid((unsigned)std::min(tiles, full), (unsigned)slices);
    const size_t smem = ((size_t)2 * a.r.tile * a.r.rot + 2 * a.r.hd + (mode == 2 ? kThreads / 32 * a.r.hd : 0)) * sizeof(float);
    if (dt == kF32) return launch_kind<float>(kind, a, mode, grid, smem, st);
    if (dt == kF16) return launch_kind<__half>(kind, a, mode, grid, smem, st);
    return launch_kind<__nv_bfloat16>(kind, a, mode, grid, smem, st);
}

namespace {
template <typename T>
cudaError_t launch_bwd_t(const NormArgs &a, int mode, size_t smem, cudaStream_t st) {
    const auto fn = mode == 0 ? &k_norm_bwd<T, 0> : mode == 1 ? &k_norm_bwd<T, 1> : &k_norm_bwd<T, 2>;
    const cudaError_t e = ensure_smem(reinterpret_cast<const void *>(fn), (int)smem);
    if (e != cudaSuccess) return e;
    return launch_dependent(fn, dim3((unsigned)a.blocks), kThreads, smem, st, a);
}
}  // namespace

cudaError_t launch_norm_bwd(DType dt, NormArgs a, cudaStream_t st) {
    const int es = dt == kF32 ? 4 : 2;
    const int mode = mode_of(a.r, es, false, &a.lanes);
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidValue;
    const long long full = std::min(2LL * sms, (long long)kNormBlocks - 2);
    long long work[2] = {0, 0};
    for (int k = 0; k < 2; ++k) {
        const int heads = k ? a.r.hk : a.r.hq;
        a.tile[k] = a.slices[k] = 1;
        if (heads == 0) continue;
        tile_of(a.r, heads, a.lanes, full, kBwdRows, &a.tile[k], &a.slices[k]);
        a.tiles[k] = (int)(((long long)a.r.tokens + a.tile[k] - 1) / a.tile[k]);
        work[k] = (long long)a.tiles[k] * a.slices[k];
    }
    // blocks shared by how many rows there are
    const long long all = a.r.hq + a.r.hk;
    const long long kq = std::max(1LL, std::min(work[0], full * a.r.hq / all));
    const long long kk = a.r.hk ? std::max(1LL, std::min(work[1], full - full * a.r.hq / all)) : 0;
    a.blocks_q = (int)kq;
    a.blocks = (int)(kq + kk);
    const int rows = mode == 2 ? kThreads / 32 * 3 : kThreads / a.lanes;
    const size_t smem = ((size_t)2 * std::max(a.tile[0], a.tile[1]) * a.r.rot + a.r.hd + (size_t)rows * a.r.hd) * sizeof(float);
    const cudaError_t e = dt == kF32   ? launch_bwd_t<float>(a, mode, smem, st)
                          : dt == kF16 ? launch_bwd_t<__half>(a, mode, smem, st)
                                       : launch_bwd_t<__nv_bfloat16>(a, mode, smem, st);
    if (e != cudaSuccess || (!a.dw[0] && !a.dw[1])) return e;
    return launch_dependent(&k_norm_dw, dim3((unsigned)((a.r.hd + 31) / 32), a.dw[1] ? 2u : 1u), 1024, 0, st, a);
}

cudaError_t launch_read4(DType dt, const Read4Args &a, cudaStream_t st) {
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidValue;
    const long long items = 2LL * a.hk * (a.hd / 8) * a.tokens;
    const dim3 grid((unsigned)std::min((items + kThreads - 1) / kThreads, 32LL * sms));
    if (dt == kF32) return launch_dependent(&k_read4<float>, grid, kThreads, 0, st, a);
    if (dt == kF16) return launch_dependent(&k_read4<__half>, grid, kThreads, 0, st, a);
    return launch_dependent(&k_read4<__nv_bfloat16>, grid, kThreads, 0, st, a);
}

}  // namespace swab
