// k_decode4.cu -- banded attention of a few new tokens a request over a paged
// cache held in 4 bits: a code c of a channel stands for s (c - 8), s the scale of
// its 32 adjacent channels.
//
// k_decode4_rows: fp16 / bf16 with head_dim 64 or 128, on the tensor cores.  The
// query heads that share a key head, of all the new tokens of a request, are the
// rows of one tile, so every code is read from memory once for all of them.
//
// HBM-bound by bytes, but a byte carries four times the arithmetic of one in 16
// bits: what counts is instructions a code.  So
//  * the products are transposed: S^T = K Q^T and O^T = V^T P^T, the cache the A
//    operand (16 keys or channels) and the few rows its 8 columns; half as many
//    products as with the rows as A, and the values are made once for all rows;
//  * a code becomes a value by two instructions for two of them: shifted so that it
//    lies behind the exponent of 16 (x = 16 + c), masked and joined with it in one
//    operation, then x s - 24 s = s (c - 8), exact because s has 5 significant bits;
//  * codes stay as they lie: A's k order is any order that B's shares.  A lane takes
//    32 (16) adjacent channels of a key, one group, in K; 16 (8) adjacent channels of
//    four keys in V, whose words are joined by halves so that a register holds two
//    keys of one channel.
// A warp owns groups of 32 keys and runs on its own: lines looked up one stage
// ahead, codes and scales brought in with cp.async into a ring of its own.  Which
// key of a group sits in which row of the product (slot_of) and where a piece of a
// line lies in the ring are chosen so that no read of the ring has bank conflicts.
// Absent keys are zero-filled, scale and all: their values are 0 whatever the cache
// holds there.
// The softmax is that of k_decode_rows: the running maximum raised only when a
// score passes it by 2^8, weights rounded to 16 bits for the product, sums fp32.
//
// k_decode4_general: every type and head size (a multiple of 32), fp32 arithmetic.
#include <type_traits>

#include "swab_internal.h"
#include "swab_decode.cuh"

static constexpr unsigned kSwabFile = 18;   // site id of the bounds checks

namespace swab {
namespace {

constexpr int kKeys = 32;          // keys of a group
constexpr float kSlack = 8.f;      // log2 headroom of the running maximum

template <int HD, int kN, int kWarps> struct Shape4 {
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kBlocks = (kN == 1 ? 16 : 12) / kWarps;   // an SM holds, by registers and shared memory
    static constexpr int kStages = HD == 128 ? 3 : 4;
    static constexpr int kLine = HD / 2;                            // bytes of codes of a key
    static constexpr int kScale = HD / 16;                          // bytes of its scales
    static constexpr int kCodes = kKeys * kLine, kScales = kKeys * kScale;
    static constexpr int kStage = 2 * (kCodes + kScales);          // codes of K, of V, scales of K, of V
    static constexpr int kRing = kStages * kStage;
    static constexpr int kSmem = kWarps * kRing + 128;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
template <int N> __device__ __forceinline__ void cp_async_small(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<T, __half>::value)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 8 x 8 16-bit values, a row on four lanes: transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Codes to values, two at a time.
template <typename T> struct Two;
template <> struct Two<__half> {
    // codes n and n + 4 of a word as 16 + c: bits 6..9 of a half behind the exponent of 16
    template <int n> __device__ static __forceinline__ uint32_t biased(uint32_t w) {
        const uint32_t x = n == 0 ? w << 6 : n == 1 ? w << 2 : n == 2 ? w >> 2 : w >> 6;
        return (x & 0x03c003c0u) | 0x4c004c00u;
    }
    __device__ static __forceinline__ uint32_t fma(uint32_t x, uint32_t s, uint32_t b) {
        uint32_t y;
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(x), "r"(s), "r"(b));
        return y;
    }
    __device__ static __forceinline__ uint32_t bias(uint32_t s) {       // -24 s, exact
        uint32_t y;
        asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(s), "r"(0xce00ce00u));
        return y;
    }
};
template <> struct Two<__nv_bfloat16> {
    template <int n> __device__ static __forceinline__ uint32_t biased(uint32_t w) {     // bits 3..6
        const uint32_t x = n == 0 ? w << 3 : n == 1 ? w >> 1 : n == 2 ? w >> 5 : w >> 9;
        return (x & 0x00780078u) | 0x41804180u;
    }
    __device__ static __forceinline__ uint32_t fma(uint32_t x, uint32_t s, uint32_t b) {
        uint32_t y;
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(x), "r"(s), "r"(b));
        return y;
    }
    __device__ static __forceinline__ uint32_t bias(uint32_t s) {
        uint32_t y;
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(s), "r"(0xc1c0c1c0u));
        return y;
    }
};
// word -> {value n, value n + 4} for n = 0..3
template <typename T> __device__ __forceinline__ void values(uint32_t w, uint32_t s, uint32_t b, uint32_t (&v)[4]) {
    v[0] = Two<T>::fma(Two<T>::template biased<0>(w), s, b);
    v[1] = Two<T>::fma(Two<T>::template biased<1>(w), s, b);
    v[2] = Two<T>::fma(Two<T>::template biased<2>(w), s, b);
    v[3] = Two<T>::fma(Two<T>::template biased<3>(w), s, b);
}

// Key (of 8) in row p of a product: the even rows take the first four, the odd ones
// the others backwards.
__device__ __forceinline__ int slot_of(int p) { return (p & 1) ? 4 + ((p >> 1) ^ 3) : p >> 1; }

// Grid: (piece, key head and tile of 8 kN rows, request).  kWarps: the warps that
// share a piece.
template <typename T, int HD, int kN, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, Shape4<HD, kN, kWarps>::kBlocks) k_decode4_rows(const __grid_constant__ DecodeArgs p) {
    using S = Shape4<HD, kN, kWarps>;
    constexpr int kThreads = S::kThreads, kRows = 8 * kN;
    constexpr int kWords = HD / 32;                        // words of codes of a lane's share of a key (K)
    constexpr int kSteps = HD / 16, kTiles = HD / 16;      // products of 16 channels (S), of 16 channels (O)
    constexpr int kChunks = S::kLine / 16, kPer = 32 / kChunks;   // 16-byte pieces of a line; lines of a copy instruction
    constexpr int kPad = HD + 8;                           // floats of a row in the final exchange
    static_assert(kRows * kPad * 4 <= S::kRing, "a warp's O fits its ring");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~static_cast<uintptr_t>(127));
    __shared__ float2 sml[kWarps][kRows];
    __shared__ float swt[kWarps][kRows];
    __shared__ float2 stot[kRows];
    __shared__ uint32_t sok[kWarps][S::kStages];           // which keys of the group in a stage are there
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int split = blockIdx.x, r = blockIdx.z;
    const int kvh = (int)(blockIdx.y % (unsigned)p.hk), tile0 = (int)(blockIdx.y / (unsigned)p.hk);
    const int tiles_y = gridDim.y / p.hk;
    pdl_wait();
    pdl_trigger();
    const Request q = request_of(p, r);
    uint8_t *ring = smem + warp * S::kRing;
    const uint32_t ring_s = smem_u32(ring);
    const char *kbase = reinterpret_cast<const char *>(p.Kc) + lane % kChunks * 16;
    const char *vbase = reinterpret_cast<const char *>(p.Vc) + lane % kChunks * 16;
    // where a copied piece goes: piece c of line i at c ^ (2 (i / 2 mod 2)) of the line
    // (64-byte lines; 32-byte ones as they are)
    const uint32_t copy_row = lane / kChunks;
    const uint32_t copy_to = copy_row * S::kLine + ((lane % kChunks) ^ (HD == 128 ? (copy_row & 2) : 0)) * 16;
    // what this lane reads: in K keys slot_of(g) and + 8 of each 16, in V keys t4 and 7 - t4 and + 8
    const int k_slot = slot_of(g), v_even = t4, v_odd = 4 + (t4 ^ 3);
    const uint32_t k_at = k_slot * S::kLine + (HD == 128 ? (t4 ^ (k_slot & 2)) * 16 : t4 * 8);
    auto v_place = [&](int slot) { return (uint32_t)(slot * S::kLine + (HD == 128 ? ((g >> 1) ^ (slot & 2)) * 16 + (g & 1) * 8 : g * 4)); };
    const uint32_t ve_at = S::kCodes + v_place(v_even), vo_at = S::kCodes + v_place(v_odd);
    const uint32_t ks_at = 2 * S::kCodes + k_slot * S::kScale + (HD == 128 ? t4 : t4 >> 1) * 2;
    const int v_group = HD == 128 ? g >> 1 : g >> 2;
    const uint32_t ves_at = 2 * S::kCodes + S::kScales + v_even * S::kScale + v_group * 2;
    const uint32_t vos_at = 2 * S::kCodes + S::kScales + v_odd * S::kScale + v_group * 2;
    // scores are scaled by |scale| inside the exponent; a negative one turns Q
    // round (exact), zero clears it
    const float scale = p.scale_log2 == 0.f ? 1.f : fabsf(p.scale_log2);
    const uint32_t q_and = p.scale_log2 == 0.f ? 0u : 0xffffffffu, q_xor = p.scale_log2 < 0.f ? 0x80008000u : 0u;
    // tiles of rows: with a key stride each token has its own
    const int per_tok = (p.group + kRows - 1) / kRows;
    const int ntiles = p.stride == 1 ? (q.m * p.group + kRows - 1) / kRows : q.m * per_tok;

    for (int tile = tile0; tile < ntiles; tile += tiles_y) {
        int row0, nrows;
        if (p.stride == 1) {
            row0 = tile * kRows;
            nrows = min(kRows, q.m * p.group - row0);
        } else {
            const int part = tile % per_tok;
            row0 = tile / per_tok * p.group + part * kRows;
            nrows = min(kRows, p.group - part * kRows);
        }
        const int a_lo = row0 / p.group, a_hi = (row0 + nrows - 1) / p.group;
        const KeyList keys = keys_of(p, q, a_lo, a_hi);
        const int lo = min((long long)split * p.chunk, (long long)keys.count);
        const int hi = split == p.nsplit - 1 ? keys.count : (int)min((long long)lo + p.chunk, (long long)keys.count);
        const int groups = (int)(((long long)hi - lo + kKeys - 1) / kKeys);
        const int mine = groups > warp ? (groups - warp + kWarps - 1) / kWarps : 0;   // of this warp

        // line of key `lane` of the warp's group n
        auto look_up = [&](int n) -> uint32_t {
            // (unsigned: past the end of the longest list the sum passes 2^31)
            const unsigned u = (unsigned)kKeys * (unsigned)(warp + kWarps * n) + (unsigned)lane;
            return n < mine && u < (unsigned)(hi - lo) ? key_line(p, q, keys.at(lo + (int)u), kvh) : kNoLine;
        };
        auto load = [&](int stage, uint32_t line) {
            const uint32_t there = __ballot_sync(0xffffffffu, line != kNoLine);
            if (lane == 0) sok[warp][stage] = there;
            const uint32_t at = ring_s + stage * S::kStage, to = at + copy_to;
#pragma unroll
            for (int i = 0; i < kKeys / kPer; ++i) {
                const uint32_t ln = __shfl_sync(0xffffffffu, line, i * kPer + lane / kChunks);
                const uint32_t bytes = ln != kNoLine ? 16u : 0u;
                const unsigned long long from = (unsigned long long)(ln != kNoLine ? ln : 0u) * S::kLine;
                cp_async16(to + i * kPer * S::kLine, GPN(p.bnd, kbase + from, 16), bytes);
                cp_async16(to + i * kPer * S::kLine + S::kCodes, GPN(p.bnd, vbase + from, 16), bytes);
            }
            const uint32_t bytes = line != kNoLine ? (uint32_t)S::kScale : 0u;
            const unsigned long long from = (unsigned long long)(line != kNoLine ? line : 0u) * S::kScale;
            const uint32_t sc = at + 2 * S::kCodes + lane * S::kScale;
            cp_async_small<S::kScale>(sc, GPN(p.bnd, reinterpret_cast<const char *>(p.Ks) + from, S::kScale), bytes);
            cp_async_small<S::kScale>(sc + S::kScales, GPN(p.bnd, reinterpret_cast<const char *>(p.Vs) + from, S::kScale), bytes);
        };

        // fill the ring; the lines of the stage after it are looked up meanwhile
        uint32_t first[S::kStages];
#pragma unroll
        for (int s = 0; s < S::kStages; ++s) first[s] = look_up(s);
#pragma unroll
        for (int s = 0; s < S::kStages - 1; ++s) {
            if (s < mine) load(s, first[s]);
            cp_commit();
        }
        uint32_t next = first[S::kStages - 1];

        // Q of the tile as B operands: row 8 n + g, in the k order of a lane's words (8 w +
        // {2 e, 2 e + 4}, {2 e + 1, 2 e + 5} of its channels in step 2 w + e)
        uint32_t qb[kN][kSteps][2];
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            const int rr = 8 * n + g;
            const bool live = rr < nrows;
            const int row = row0 + (live ? rr : 0), a = row / p.group, hh = kvh * p.group + row - a * p.group;
            const T *src = reinterpret_cast<const T *>(p.Q) + (long long)(q.row0 + a) * p.q_stride + (long long)hh * HD + t4 * (HD / 4);
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
                const uint4 x = *reinterpret_cast<const uint4 *>(GPN(p.bnd, src + 8 * w, 16));
                const uint32_t v[4] = {live ? (x.x & q_and) ^ q_xor : 0u, live ? (x.y & q_and) ^ q_xor : 0u,
                                       live ? (x.z & q_and) ^ q_xor : 0u, live ? (x.w & q_and) ^ q_xor : 0u};
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    qb[n][2 * w + e][0] = __byte_perm(v[e], v[2 + e], 0x5410);
                    qb[n][2 * w + e][1] = __byte_perm(v[e], v[2 + e], 0x7632);
                }
            }
        }
        // positions of this lane's rows (row 8 n + 2 t4 + e)
        int pos[kN][2];
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) pos[n][e] = q.i0 + (row0 + min(8 * n + 2 * t4 + e, nrows - 1)) / p.group;
        const int pos_lo = q.i0 + a_lo, pos_hi = q.i0 + a_hi;

        // O^T: channels kTiles g' .. of row 2 t4 + e: o[n][i][e] is channel 2 i, o[n][i][2 + e] 2 i + 1
        float o[kN][kTiles][4], m[kN][2], l[kN][2];
#pragma unroll
        for (int n = 0; n < kN; ++n) {
#pragma unroll
            for (int d = 0; d < kTiles; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][d][e] = 0.f;
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
        }

        int stage = 0;
        for (int n_it = 0; n_it < mine; ++n_it) {
            // the ring's free stage takes group n_it + kStages - 1
            const uint32_t ahead = look_up(n_it + S::kStages);
            if (n_it + S::kStages - 1 < mine) load(stage == 0 ? S::kStages - 1 : stage - 1, next);
            cp_commit();
            next = ahead;
            cp_wait<S::kStages - 1>();
            __syncwarp();
            const uint8_t *st = ring + stage * S::kStage;

            // scores: c[n][x]: keys 16 x + slot_of(g) (e = 0, 1: rows) and + 8 (e = 2, 3)
            float c[kN][2][4];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
                for (int n = 0; n < kN; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) c[n][x][e] = 0.f;
                uint32_t w[2][kWords], s[2], b[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint8_t *at = st + (16 * x + 8 * h) * S::kLine + k_at;
                    if constexpr (HD == 128) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(at);
                        w[h][0] = v.x, w[h][1] = v.y, w[h][kWords - 2] = v.z, w[h][kWords - 1] = v.w;
                    } else {
                        const uint2 v = *reinterpret_cast<const uint2 *>(at);
                        w[h][0] = v.x, w[h][1] = v.y;
                    }
                    const uint32_t sc = *reinterpret_cast<const uint16_t *>(st + (16 * x + 8 * h) * S::kScale + ks_at);
                    s[h] = sc | sc << 16;
                    b[h] = Two<T>::bias(s[h]);
                }
#pragma unroll
                for (int k = 0; k < kWords; ++k) {
                    uint32_t va[4], vb[4];
                    values<T>(w[0][k], s[0], b[0], va);
                    values<T>(w[1][k], s[1], b[1], vb);
#pragma unroll
                    for (int n = 0; n < kN; ++n) {
                        mma16816<T>(c[n][x], va[0], vb[0], va[1], vb[1], qb[n][2 * k][0], qb[n][2 * k][1]);
                        mma16816<T>(c[n][x], va[2], vb[2], va[3], vb[3], qb[n][2 * k + 1][0], qb[n][2 * k + 1][1]);
                    }
                }
            }
            // which of the group's keys each row attends to
            const int u0 = lo + kKeys * (warp + kWarps * n_it);
            const uint32_t ok = sok[warp][stage];
            const int j_lo = keys.at(u0), j_hi = keys.at(u0 + kKeys - 1);
            const bool all = ok == 0xffffffffu && j_hi <= pos_lo && (j_hi < p.n_sink || (long long)pos_hi - j_lo <= (long long)p.w * p.stride);
            if (!all) {
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int slot = 16 * x + 8 * h + k_slot, j = keys.at(u0 + slot);
                        const bool here = (ok >> slot) & 1u;
#pragma unroll
                        for (int n = 0; n < kN; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                if (!(here && attends(p, pos[n][e], j))) c[n][x][2 * h + e] = -INFINITY;
                    }
            }
            float best[kN][2];
            bool up = false;
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    best[n][e] = fmaxf(max3(c[n][0][e], c[n][0][2 + e], c[n][1][e]), c[n][1][2 + e]) * scale;
                    up |= best[n][e] > m[n][e] + kSlack;
                }
            if (__any_sync(0xffffffffu, up)) {   // raise the maxima, scale what was summed so far
#pragma unroll
                for (int n = 0; n < kN; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = best[n][e];
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                        const float mn = fmaxf(m[n][e], mx);
                        const float f = m[n][e] == -INFINITY ? 0.f : ex2(m[n][e] - mn);
                        m[n][e] = mn;
                        l[n][e] *= f;
#pragma unroll
                        for (int d = 0; d < kTiles; ++d) {
                            o[n][d][e] *= f;
                            o[n][d][2 + e] *= f;
                        }
                    }
            }
            // weights, as B operands: keys 2 t4, 2 t4 + 1 (rows of the first product) of row g
            uint32_t pb[kN][2][2];
#pragma unroll
            for (int n = 0; n < kN; ++n) {
                const float m0 = m[n][0] == -INFINITY ? 0.f : m[n][0], m1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float p0 = ex2(fmaf(c[n][x][2 * h], scale, -m0)), p1 = ex2(fmaf(c[n][x][2 * h + 1], scale, -m1));
                        l[n][0] += p0;
                        l[n][1] += p1;
                        pb[n][x][h] = transpose8(pack2<T>(p0, p1));
                    }
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                // v[h]: keys 16 x + 8 h + v_even, v_odd
                uint32_t we[2][HD / 64], wo[2][HD / 64], s[2], b[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint8_t *at = st + (16 * x + 8 * h) * S::kLine;
                    if constexpr (HD == 128) {
                        const uint2 ve = *reinterpret_cast<const uint2 *>(at + ve_at), vo = *reinterpret_cast<const uint2 *>(at + vo_at);
                        we[h][0] = ve.x, we[h][HD / 64 - 1] = ve.y;
                        wo[h][0] = vo.x, wo[h][HD / 64 - 1] = vo.y;
                    } else {
                        we[h][0] = *reinterpret_cast<const uint32_t *>(at + ve_at);
                        wo[h][0] = *reinterpret_cast<const uint32_t *>(at + vo_at);
                    }
                    const uint8_t *sc = st + (16 * x + 8 * h) * S::kScale;
                    s[h] = *reinterpret_cast<const uint16_t *>(sc + ves_at) | (uint32_t)*reinterpret_cast<const uint16_t *>(sc + vos_at) << 16;
                    b[h] = Two<T>::bias(s[h]);
                }
#pragma unroll
                for (int k = 0; k < HD / 64; ++k)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        // four channels (8 k + 4 half + 0..3 of the lane's) of two keys
                        uint32_t va[4], vb[4];
                        values<T>(__byte_perm(we[0][k], wo[0][k], half ? 0x7632 : 0x5410), s[0], b[0], va);
                        values<T>(__byte_perm(we[1][k], wo[1][k], half ? 0x7632 : 0x5410), s[1], b[1], vb);
                        const int i = 4 * k + 2 * half;
#pragma unroll
                        for (int n = 0; n < kN; ++n) {
                            mma16816<T>(o[n][i], va[0], va[1], vb[0], vb[1], pb[n][x][0], pb[n][x][1]);
                            mma16816<T>(o[n][i + 1], va[2], va[3], vb[2], vb[3], pb[n][x][0], pb[n][x][1]);
                        }
                    }
            }
            __syncwarp();                        // every lane has read the stage
            stage = stage + 1 == S::kStages ? 0 : stage + 1;
        }
        cp_wait<0>();
        __syncwarp();

        // join the warps: O of each into its own ring, then all threads sum
        float *mine_o = reinterpret_cast<float *>(ring);
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float s = l[n][e];
                s += __shfl_xor_sync(0xffffffffu, s, 4);
                s += __shfl_xor_sync(0xffffffffu, s, 8);
                s += __shfl_xor_sync(0xffffffffu, s, 16);
                const int row = 8 * n + 2 * t4 + e;
                if (g == 0) sml[warp][row] = make_float2(m[n][e], s);
#pragma unroll
                for (int d = 0; d < kTiles; ++d)
                    *reinterpret_cast<float2 *>(mine_o + row * kPad + g * (HD / 8) + 2 * d) = make_float2(o[n][d][e], o[n][d][2 + e]);
            }
        __syncthreads();
        if (threadIdx.x < kRows) {
            const int row = threadIdx.x;
            float M = -INFINITY, L = 0.f;
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sml[w][row].x);
            for (int w = 0; w < kWarps; ++w) {
                const float f = sml[w][row].x == -INFINITY ? 0.f : ex2(sml[w][row].x - M);
                swt[w][row] = f;
                L = fmaf(sml[w][row].y, f, L);
            }
            stot[row] = make_float2(M, L);
            if (row < nrows) {
                const int a = (row0 + row) / p.group, hh = kvh * p.group + row0 + row - a * p.group;
                const long long th = (long long)(q.row0 + a) * p.h + hh;
                if (p.nparts > 1) *GP(p.bnd, p.pml + th * p.nparts + split) = make_float2(M, L);
                else if (p.lse) *GP(p.bnd, p.lse + th) = lse_of(M, L);
            }
        }
        __syncthreads();
        for (int e = threadIdx.x; e < nrows * (HD / 4); e += kThreads) {
            const int row = e / (HD / 4), c4 = e % (HD / 4) * 4;
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = swt[w][row];
                const float4 v = *reinterpret_cast<const float4 *>(reinterpret_cast<float *>(smem + w * S::kRing) + row * kPad + c4);
                y.x = fmaf(v.x, f, y.x);
                y.y = fmaf(v.y, f, y.y);
                y.z = fmaf(v.z, f, y.z);
                y.w = fmaf(v.w, f, y.w);
            }
            const int a = (row0 + row) / p.group, hh = kvh * p.group + row0 + row - a * p.group;
            const long long tok = q.row0 + a, th = tok * p.h + hh;
            if (p.nparts > 1) {
                *reinterpret_cast<float4 *>(GPN(p.bnd, p.po + (th * p.nparts + split) * HD + c4, 16)) = y;
            } else {
                const float inv = inverse_of(stot[row].y);
                *reinterpret_cast<uint2 *>(GPN(p.bnd, reinterpret_cast<T *>(p.O) + tok * p.o_stride + (long long)hh * HD + c4, 8)) =
                    make_uint2(pack2<T>(y.x * inv, y.y * inv), pack2<T>(y.z * inv, y.w * inv));
            }
        }
        __syncthreads();                         // the rings are free for the next tile
    }
}

// ---------------------------------------------------------------------------
// every type and head size
// ---------------------------------------------------------------------------
constexpr int kThreadsG = 128;

// A key belongs to a group of kLanes lanes, 8 channels (a word of codes) a lane;
// kThreadsG / kLanes keys at a time.  A block answers kR query heads that share the
// key head, so a key is loaded and unpacked once for them.
template <typename T, int kLanes, int kR>
__global__ void __launch_bounds__(kThreadsG, kR == 1 ? 8 : 4) k_decode4_general(const __grid_constant__ DecodeArgs p) {
    constexpr int kGroups = kThreadsG / kLanes, kU = 4;
    __shared__ float so[kGroups][kLanes * 8];
    __shared__ float2 sml[kGroups];
    const int per = (p.group + kR - 1) / kR;                       // blocks of a key head
    const int split = blockIdx.x, kvh = blockIdx.y / per, g0 = blockIdx.y % per * kR, r = blockIdx.z;
    const int head0 = kvh * p.group + g0, nr = min(kR, p.group - g0);
    const int sub = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
    const int words = p.hd / 8;
    const bool active = lane < words;
    pdl_wait();
    pdl_trigger();
    const Request q = request_of(p, r);
    for (int a = 0; a < q.m; ++a) {
        const KeyList keys = keys_of(p, q, a, a);
        const long long n = keys.count, lo = (long long)split * p.chunk;
        const long long hi = split == p.nsplit - 1 ? n : min(n, lo + p.chunk);
        const long long row = q.row0 + a;
        float qf[kR][8], o[kR][8], m[kR], l[kR];
#pragma unroll
        for (int t = 0; t < kR; ++t) {
            m[t] = -INFINITY;
            l[t] = 0.f;
            const T *qrow = reinterpret_cast<const T *>(p.Q) + row * p.q_stride + (long long)(head0 + min(t, nr - 1)) * p.hd + lane * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                qf[t][e] = active ? Elt<T>::to_f(*GP(p.bnd, qrow + e)) : 0.f;
                o[t][e] = 0.f;
            }
        }
        // every lane group makes the same number of steps (the shuffles below
        // need the whole warp), kU keys a step with all their loads in flight
        const long long span = hi - lo;
        const int steps = span > 0 ? (int)((span + kGroups * kU - 1) / (kGroups * kU)) : 0;
        for (int s = 0; s < steps; ++s) {
            uint32_t line[kU], kw[kU], vw[kU];
            float ks[kU], vs[kU];
#pragma unroll
            for (int i = 0; i < kU; ++i) {
                const long long u = lo + ((long long)s * kU + i) * kGroups + sub;
                line[i] = u < hi ? key_line(p, q, keys.at((int)u), kvh) : kNoLine;
            }
#pragma unroll
            for (int i = 0; i < kU; ++i) {
                kw[i] = vw[i] = 0;
                ks[i] = vs[i] = 0.f;
                if (line[i] != kNoLine && active) {
                    const unsigned long long at = (unsigned long long)line[i] * words + lane, sc = (unsigned long long)line[i] * (p.hd / kGroup4) + lane / 4;
                    kw[i] = *GP(p.bnd, reinterpret_cast<const uint32_t *>(p.Kc) + at);
                    vw[i] = *GP(p.bnd, reinterpret_cast<const uint32_t *>(p.Vc) + at);
                    ks[i] = Elt<T>::to_f(*GP(p.bnd, reinterpret_cast<const T *>(p.Ks) + sc));
                    vs[i] = Elt<T>::to_f(*GP(p.bnd, reinterpret_cast<const T *>(p.Vs) + sc));
                }
            }
            float x[kR][kU];
#pragma unroll
            for (int i = 0; i < kU; ++i) {
                float kf[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) kf[e] = ks[i] * (float)((int)((kw[i] >> (4 * e)) & 15u) - 8);
#pragma unroll
                for (int t = 0; t < kR; ++t) {
                    x[t][i] = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[t][i] = fmaf(qf[t][e], kf[e], x[t][i]);
                }
            }
#pragma unroll
            for (int d = kLanes / 2; d > 0; d >>= 1)
#pragma unroll
                for (int t = 0; t < kR; ++t)
#pragma unroll
                    for (int i = 0; i < kU; ++i) x[t][i] += __shfl_xor_sync(0xffffffffu, x[t][i], d);
#pragma unroll
            for (int t = 0; t < kR; ++t) {
                float mn = m[t];
#pragma unroll
                for (int i = 0; i < kU; ++i) {
                    x[t][i] = line[i] == kNoLine ? -INFINITY : x[t][i] * p.scale_log2;
                    mn = fmaxf(mn, x[t][i]);
                }
                const float mb = mn == -INFINITY ? 0.f : mn;                 // no key yet
                const float corr = m[t] == -INFINITY ? 0.f : exp2f(m[t] - mb);
                m[t] = mn;
                l[t] *= corr;
#pragma unroll
                for (int e = 0; e < 8; ++e) o[t][e] *= corr;
#pragma unroll
                for (int i = 0; i < kU; ++i) {
                    x[t][i] = exp2f(x[t][i] - mb);                           // 0 for an absent key
                    l[t] += x[t][i];
                }
            }
#pragma unroll
            for (int i = 0; i < kU; ++i) {
                float vf[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) vf[e] = vs[i] * (float)((int)((vw[i] >> (4 * e)) & 15u) - 8);
#pragma unroll
                for (int t = 0; t < kR; ++t)
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[t][e] = fmaf(x[t][i], vf[e], o[t][e]);
            }
        }
#pragma unroll
        for (int t = 0; t < kR; ++t) {
            if (t >= nr) break;
            __syncthreads();             // the previous head's reads of the buffers
#pragma unroll
            for (int e = 0; e < 8; ++e) so[sub][lane * 8 + e] = o[t][e];
            if (lane == 0) sml[sub] = make_float2(m[t], l[t]);
            __syncthreads();
            float M = -INFINITY, L = 0.f;
            for (int g = 0; g < kGroups; ++g) M = fmaxf(M, sml[g].x);
            for (int g = 0; g < kGroups; ++g) L = fmaf(sml[g].y, sml[g].x == -INFINITY ? 0.f : exp2f(sml[g].x - M), L);
            const int head = head0 + t;
            const long long th = row * p.h + head;
            for (int c = threadIdx.x; c < p.hd; c += kThreadsG) {
                float y = 0.f;
                for (int g = 0; g < kGroups; ++g) y = fmaf(so[g][c], sml[g].x == -INFINITY ? 0.f : exp2f(sml[g].x - M), y);
                if (p.nparts > 1)
                    *GP(p.bnd, p.po + (th * p.nparts + split) * p.hd + c) = y;
                else
                    *GP(p.bnd, reinterpret_cast<T *>(p.O) + row * p.o_stride + (long long)head * p.hd + c) =
                        Elt<T>::from_f(L == 0.f ? 0.f : y / L);
            }
            if (threadIdx.x == 0) {
                if (p.nparts > 1) *GP(p.bnd, p.pml + th * p.nparts + split) = make_float2(M, L);
                else if (p.lse) *GP(p.bnd, p.lse + th) = lse_of(M, L);
            }
        }
    }
}

template <typename T, int HD, int kN, int kWarps>
cudaError_t launch_w(const DecodeArgs &a, cudaStream_t st) {
    using S = Shape4<HD, kN, kWarps>;
    const auto fn = &k_decode4_rows<T, HD, kN, kWarps>;
    const cudaError_t e = ensure_smem(reinterpret_cast<const void *>(fn), S::kSmem);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)a.nsplit, (unsigned)(a.hk * a.row_tiles), (unsigned)a.batch);
    return launch_dependent(fn, grid, S::kThreads, S::kSmem, st, a);
}
template <typename T, int HD>
cudaError_t launch_hd(const DecodeArgs &a, cudaStream_t st) {
    return a.tile_rows == 8 ? launch_w<T, HD, 1, 4>(a, st) : launch_w<T, HD, 2, 4>(a, st);
}

template <typename T, int kR>
cudaError_t launch_general_r(const DecodeArgs &a, cudaStream_t st) {
    const dim3 grid((unsigned)a.nsplit, (unsigned)(a.hk * ((a.group + kR - 1) / kR)), (unsigned)a.batch);
    if (a.hd <= 32) return launch_dependent(&k_decode4_general<T, 4, kR>, grid, kThreadsG, 0, st, a);
    if (a.hd <= 64) return launch_dependent(&k_decode4_general<T, 8, kR>, grid, kThreadsG, 0, st, a);
    if (a.hd <= 128) return launch_dependent(&k_decode4_general<T, 16, kR>, grid, kThreadsG, 0, st, a);
    return launch_dependent(&k_decode4_general<T, 32, kR>, grid, kThreadsG, 0, st, a);
}
template <typename T>
cudaError_t launch_general_t(const DecodeArgs &a, cudaStream_t st) {
    return a.group == 1 ? launch_general_r<T, 1>(a, st) : launch_general_r<T, 4>(a, st);
}

}  // namespace

cudaError_t launch_decode4_rows(DType dt, const DecodeArgs &a, cudaStream_t st) {
    if (dt == kF16) return a.hd == 64 ? launch_hd<__half, 64>(a, st) : launch_hd<__half, 128>(a, st);
    return a.hd == 64 ? launch_hd<__nv_bfloat16, 64>(a, st) : launch_hd<__nv_bfloat16, 128>(a, st);
}
cudaError_t launch_decode4_general(DType dt, const DecodeArgs &a, cudaStream_t st) {
    return dt == kF32 ? launch_general_t<float>(a, st) : dt == kF16 ? launch_general_t<__half>(a, st) : launch_general_t<__nv_bfloat16>(a, st);
}

}  // namespace swab
