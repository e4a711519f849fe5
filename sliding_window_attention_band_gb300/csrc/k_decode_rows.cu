// k_decode_rows.cu -- banded attention of a few new tokens a request over the
// paged cache, fp16 / bf16 with head_dim 64 or 128: the query heads that share
// a key head, of all the new tokens of a request, are the rows of one tile, so
// every key and value is read from memory once for all of them.
//
// HBM-bound (4 flops a row for every 2 bytes): what counts is bytes in flight.
// A warp owns groups of 16 keys (group g of the block's piece goes to warp
// g mod kWarps) and runs on its own: it looks the 16 lines up in the block table
// one stage ahead, brings them in with 16-byte cp.async into a ring of its own,
// and waits for nobody until the end.  A group is 16 rows x 16 keys of mma.sync
// m16n8k16 (the rows are few: a 128-row tcgen05 tile would be 7/8 padding and
// would need the gathered lines staged for it; 32 of these instructions a group
// are 256 cycles of an SM quarter, a fifth of what the memory takes): S = Q K^T
// with Q in registers, the softmax on the accumulator, O += P V with P repacked
// in registers (the accumulator's layout is the A operand's).  The running
// maximum is raised only when a score exceeds it by 2^8, so the usual group
// needs no exchange between lanes; a weight is rounded to 16 bits for the
// product (at most 2^8, inside fp16; the tensor cores take no wider operand at
// this rate), the sums stay fp32.  Piece c of line r lies at place c xor (r mod
// 8), so the eight lines of an ldmatrix miss each other's banks.  Absent keys are
// zero-filled, so whatever the cache holds there cannot reach a product.
//
// More than 16 rows are several tiles, in blocks of their own beside each other:
// the keys then come out of L2 for the second one.  (Tiles of 32 rows, 255
// registers and 8 warps an SM: 93 against 68 us for 48 requests of 4k, 32 rows
// over 4 key heads of 128; 99 against 115 for 32 requests of 4k to 8k.)
//
// The warps' (m, l, O) are joined in shared memory; the pieces of a split key
// list (few requests, long contexts) go to the workspace and are joined by
// k_decode_join; the parts of a shared prefix, up to 16 of them, are joined here
// where all blocks fit at once.
//
// 12 warps an SM (168 registers, 16 KB of ring each) in blocks that all fit at
// once, so that no second wave pays the chain lengths -> table -> keys again:
// 48 requests of 8 key heads of 128 under a window of 4096 take 110 us (733 MB:
// 6.7 TB/s) with 384 blocks of 4 warps on 456 places, 128 us cut into three
// pieces; 8 warps an SM with 3 stages took 149 us.  512 blocks of 4096 keys:
// 161 us (6.7 TB/s) with 3 warps a block, 208 with 4.  One context of 131072: 80
// us for 57 x 8 pieces, 85 with the join.
#include <type_traits>

#include "swab_internal.h"
#include "swab_decode.cuh"

static constexpr unsigned kSwabFile = 15;   // site id of the bounds checks

namespace swab {
namespace {

constexpr int kKeys = 16;          // keys of a group
constexpr float kSlack = 8.f;      // log2 headroom of the running maximum

template <int HD, int kWarps> struct Shape {
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kBlocks = 12 / kWarps;              // an SM holds, by registers and shared memory
    static constexpr int kStages = HD == 128 ? 2 : 4;
    static constexpr int kTile = kKeys * HD * 2;             // bytes of 16 lines
    static constexpr int kStage = 2 * kTile;                 // K and V
    static constexpr int kRing = kStages * kStage;           // of a warp
    static constexpr int kSmem = kWarps * kRing + 256;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<T, __half>::value)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Grid: (piece, key head and 16-row tile, request).  kWarps: the warps that share
// a piece.
template <typename T, int HD, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, Shape<HD, kWarps>::kBlocks) k_decode_rows(const __grid_constant__ DecodeArgs p) {
    using S = Shape<HD, kWarps>;
    constexpr int kThreads = S::kThreads;
    constexpr int kRows = 16, kSteps = HD / 16, kPieces = HD / 8;   // 16-byte pieces of a line
    constexpr int kPer = 32 / kPieces;                                   // lines of a copy instruction
    constexpr int kPad = HD + 8;                                         // floats of a row in the final exchange
    static_assert(kRows * kPad * 4 <= S::kRing, "a warp's O fits its ring");
    extern __shared__ uint8_t smem_raw[];
    // (the xors below need the rings at multiples of 256 bytes)
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 255) & ~static_cast<uintptr_t>(255));
    __shared__ float2 sml[kWarps][kRows];
    __shared__ float swt[kWarps][kRows];
    __shared__ float2 stot[kRows];
    __shared__ float2 spre[kMaxFold][kRows];       // the prefix's parts, joined here: (max, sum), then the weight
    __shared__ uint32_t sok[kWarps][S::kStages];   // which keys of the group in a stage are there
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int split = blockIdx.x, r = blockIdx.z;
    const int kvh = (int)(blockIdx.y % (unsigned)p.hk), tile0 = (int)(blockIdx.y / (unsigned)p.hk);
    const int tiles_y = gridDim.y / p.hk;
    if (p.npre == 0) {
        pdl_wait();
    } else {
        // Behind the prefix kernel this block does not wait for that kernel's end.
        // A thread of it that has passed its own wait, so that all that was written
        // before the call is visible to it, has set the block's word (release);
        // seen here (acquire), and past the barrier, the same holds for this block.
        // Not seen, it waits for the end after all.  The word is cleared for the
        // next call, which may be a replay with the same token.
        if (threadIdx.x == 0) {
            unsigned long long *go = GP(p.bnd, p.go + ((long long)blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x);
            bool seen = false;
            for (int k = 0; k < 32 && !seen; ++k) seen = load_acquire(go) == p.token;
            if (!seen) pdl_wait();
            *go = 0;
        }
        __syncthreads();
    }
    pdl_trigger();
    const Request q = request_of(p, r);
    uint8_t *ring = smem + warp * S::kRing;
    const uint32_t ring_s = smem_u32(ring);
    // this lane's piece of a line in memory, where a copy of it goes, and the
    // lines an ldmatrix reads: the place of piece 2k + b of line r is that of
    // piece b, xor 2k
    const char *kbase = reinterpret_cast<const char *>(p.Kc) + lane % kPieces * 16;
    const char *vbase = reinterpret_cast<const char *>(p.Vc) + lane % kPieces * 16;
    const uint32_t copy_row = lane / kPieces, copy_to = copy_row * (HD * 2) + (((lane % kPieces) ^ copy_row) << 4);
    const uint32_t krow = (lane & 7) + ((lane >> 4) << 3), vrow = (lane & 7) + (((lane >> 3) & 1) << 3);
    const uint32_t kat = krow * (HD * 2) + ((((lane >> 3) & 1) ^ (krow & 7)) << 4);
    const uint32_t vat = S::kTile + vrow * (HD * 2) + (((lane >> 4) ^ (vrow & 7)) << 4);
    // scores are scaled by |scale| inside the exponent; a negative one turns Q
    // round (exact), zero clears it
    const float scale = p.scale_log2 == 0.f ? 1.f : fabsf(p.scale_log2);
    const uint32_t q_and = p.scale_log2 == 0.f ? 0u : 0xffffffffu, q_xor = p.scale_log2 < 0.f ? 0x80008000u : 0u;
    // tiles of rows: with a key stride each token has its own
    const int per_tok = (p.group + kRows - 1) / kRows;
    const int ntiles = p.stride == 1 ? (q.m * p.group + kRows - 1) / kRows : q.m * per_tok;

    for (int tile = tile0; tile < ntiles; tile += tiles_y) {
        // row 0 of the tile and how many there are, counted over (token, head of the group)
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
        const int groups = (hi - lo + kKeys - 1) / kKeys;
        const int mine = groups > warp ? (groups - warp + kWarps - 1) / kWarps : 0;   // of this warp

        // line of key (lane mod 16) of the warp's group n
        auto look_up = [&](int n) -> uint32_t {
            const int u = lo + kKeys * (warp + kWarps * n) + (lane & 15);
            return n < mine && u < hi ? key_line(p, q, keys.at(u), kvh) : kNoLine;
        };
        // the 16 lines into a stage: copy i brings lines i * kPer.. ; piece c of
        // line r goes to place c ^ (r mod 8) of the line
        auto load = [&](int stage, uint32_t line) {
            const uint32_t there = __ballot_sync(0xffffffffu, line != kNoLine) & 0xffffu;
            if (lane == 0) sok[warp][stage] = there;
            const uint32_t to = ring_s + stage * S::kStage + copy_to;
#pragma unroll
            for (int i = 0; i < kKeys / kPer; ++i) {
                const uint32_t ln = __shfl_sync(0xffffffffu, line, i * kPer + lane / kPieces);
                const uint32_t bytes = ln != kNoLine ? 16u : 0u;
                const unsigned long long at = (unsigned long long)(ln != kNoLine ? ln : 0u) * (HD * 2);
                const uint32_t dst = (to + i * kPer * HD * 2) ^ (((i * kPer) & 7) << 4);
                cp_async16(dst, GPN(p.bnd, kbase + at, 16), bytes);
                cp_async16(dst + S::kTile, GPN(p.bnd, vbase + at, 16), bytes);
            }
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

        // Q of the tile as A operands
        uint32_t qa[kSteps][4];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int rr = g + 8 * half;
                const bool live = rr < nrows;
                const int row = row0 + (live ? rr : 0), a = row / p.group, hh = kvh * p.group + row - a * p.group;
                const T *src = reinterpret_cast<const T *>(p.Q) + (long long)(q.row0 + a) * p.q_stride + (long long)hh * HD + 2 * t4;
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                    const uint32_t x0 = *GP(p.bnd, reinterpret_cast<const uint32_t *>(src + 16 * k));
                    const uint32_t x1 = *GP(p.bnd, reinterpret_cast<const uint32_t *>(src + 16 * k + 8));
                    qa[k][half] = live ? (x0 & q_and) ^ q_xor : 0u;
                    qa[k][half + 2] = live ? (x1 & q_and) ^ q_xor : 0u;
                }
            }
        // positions of this lane's rows (row g + 8 e)
        int pos[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) pos[e] = q.i0 + (row0 + min(g + 8 * e, nrows - 1)) / p.group;
        const int pos_lo = q.i0 + a_lo, pos_hi = q.i0 + a_hi;

        float o[HD / 8][4], m[2], l[2];
#pragma unroll
        for (int d = 0; d < HD / 8; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[d][e] = 0.f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;

        int stage = 0;
        for (int n = 0; n < mine; ++n) {
            // the ring's free stage takes group n + kStages - 1
            const uint32_t ahead = look_up(n + S::kStages);
            if (n + S::kStages - 1 < mine) load(stage == 0 ? S::kStages - 1 : stage - 1, next);
            cp_commit();
            next = ahead;
            cp_wait<S::kStages - 1>();
            __syncwarp();
            const uint32_t kt = ring_s + stage * S::kStage + kat, vt = ring_s + stage * S::kStage + vat;

            float c[2][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) c[0][e] = c[1][e] = 0.f;
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                uint32_t b[4];
                ldsm4(kt ^ (k << 5), b);
                mma16816<T>(c[0], qa[k], b[0], b[1]);
                mma16816<T>(c[1], qa[k], b[2], b[3]);
            }
            // which of the group's keys each row attends to
            const int u0 = lo + kKeys * (warp + kWarps * n);
            const uint32_t ok = sok[warp][stage];
            const int j_lo = keys.at(u0), j_hi = keys.at(u0 + kKeys - 1);
            const bool all = ok == 0xffffu && j_hi <= pos_lo && (j_hi < p.n_sink || (long long)pos_hi - j_lo <= (long long)p.w * p.stride);
            if (!all) {
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int col = 8 * x + 2 * t4 + e, j = keys.at(u0 + col);
                        const bool here = (ok >> col) & 1u;
#pragma unroll
                            for (int r2 = 0; r2 < 2; ++r2)
                                if (!(here && attends(p, pos[r2], j))) c[x][2 * r2 + e] = -INFINITY;
                    }
            }
            float best[2];
            bool up = false;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    best[e] = fmaxf(max3(c[0][2 * e], c[0][2 * e + 1], c[1][2 * e]), c[1][2 * e + 1]) * scale;
                    up |= best[e] > m[e] + kSlack;
                }
            if (__any_sync(0xffffffffu, up)) {   // raise the maxima, scale what was summed so far
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = best[e];
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                        const float mn = fmaxf(m[e], mx);
                        const float f = m[e] == -INFINITY ? 0.f : ex2(m[e] - mn);
                        m[e] = mn;
                        l[e] *= f;
#pragma unroll
                        for (int d = 0; d < HD / 8; ++d) {
                            o[d][2 * e] *= f;
                            o[d][2 * e + 1] *= f;
                        }
                    }
            }
            uint32_t pa[4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float mb = m[e] == -INFINITY ? 0.f : m[e];
                    const float p0 = ex2(fmaf(c[0][2 * e], scale, -mb)), p1 = ex2(fmaf(c[0][2 * e + 1], scale, -mb));
                    const float p2 = ex2(fmaf(c[1][2 * e], scale, -mb)), p3 = ex2(fmaf(c[1][2 * e + 1], scale, -mb));
                    l[e] += (p0 + p1) + (p2 + p3);
                    pa[e] = pack2<T>(p0, p1);
                    pa[e + 2] = pack2<T>(p2, p3);
                }
#pragma unroll
            for (int d = 0; d < kSteps; ++d) {
                uint32_t b[4];
                ldsm4t(vt ^ (d << 5), b);
                mma16816<T>(o[2 * d], pa, b[0], b[1]);
                mma16816<T>(o[2 * d + 1], pa, b[2], b[3]);
            }
            __syncwarp();                        // every lane has read the stage
            stage = stage + 1 == S::kStages ? 0 : stage + 1;
        }
        cp_wait<0>();
        __syncwarp();

        // join the warps: O of each into its own ring, then all threads sum
        float *mine_o = reinterpret_cast<float *>(ring);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float s = l[e];
                s += __shfl_xor_sync(0xffffffffu, s, 1);
                s += __shfl_xor_sync(0xffffffffu, s, 2);
                const int row = g + 8 * e;
                if (t4 == 0) sml[warp][row] = make_float2(m[e], s);
#pragma unroll
                for (int d = 0; d < HD / 8; ++d)
                    *reinterpret_cast<float2 *>(mine_o + row * kPad + 8 * d + 2 * t4) = make_float2(o[d][2 * e], o[d][2 * e + 1]);
            }
        if (p.fold) {
            pdl_wait();                          // the prefix's parts are there
            for (int e = threadIdx.x; e < kRows * p.npre; e += kThreads) {
                const int row = e % kRows, s = e / kRows;
                if (row >= nrows) continue;
                const int a = (row0 + row) / p.group, hh = kvh * p.group + row0 + row - a * p.group;
                spre[s][row] = *GP(p.bnd, p.pml + ((long long)(q.row0 + a) * p.h + hh) * p.nparts + 1 + s);
            }
        }
        __syncthreads();
        if (threadIdx.x < kRows) {
            const int row = threadIdx.x;
            const int a = (row0 + row) / p.group, hh = kvh * p.group + row0 + row - a * p.group;
            const long long th = (long long)(q.row0 + a) * p.h + hh;
            float M = -INFINITY, L = 0.f;
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sml[w][row].x);
            if (p.fold && row < nrows) {
                for (int s = 0; s < p.npre; ++s) M = fmaxf(M, spre[s][row].x);
                for (int s = 0; s < p.npre; ++s) {
                    const float f = spre[s][row].x == -INFINITY ? 0.f : ex2(spre[s][row].x - M);
                    L = fmaf(spre[s][row].y, f, L);
                    spre[s][row].x = f;
                }
            }
            for (int w = 0; w < kWarps; ++w) {
                const float f = sml[w][row].x == -INFINITY ? 0.f : ex2(sml[w][row].x - M);
                swt[w][row] = f;
                L = fmaf(sml[w][row].y, f, L);
            }
            stot[row] = make_float2(M, L);
            if (row < nrows) {
                if (p.nparts > 1 && !p.fold) *GP(p.bnd, p.pml + th * p.nparts + split) = make_float2(M, L);
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
            if (p.fold) {
                const float *po = p.po + (th * p.nparts + 1) * HD + c4;
#pragma unroll 8
                for (int s = 0; s < p.npre; ++s) {
                    const float f = spre[s][row].x;
                    // (the values of an empty part are not written)
                    const float4 v = f == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                                              : *reinterpret_cast<const float4 *>(GPN(p.bnd, po + (long long)s * HD, 16));
                    y.x = fmaf(v.x, f, y.x);
                    y.y = fmaf(v.y, f, y.y);
                    y.z = fmaf(v.z, f, y.z);
                    y.w = fmaf(v.w, f, y.w);
                }
            }
            if (p.nparts > 1 && !p.fold) {
                *reinterpret_cast<float4 *>(GPN(p.bnd, p.po + (th * p.nparts + split) * HD + c4, 16)) = y;
            } else {
                const float inv = inverse_of(stot[row].y);
                *reinterpret_cast<uint2 *>(GPN(p.bnd, reinterpret_cast<T *>(p.O) + tok * p.o_stride + (long long)hh * HD + c4, 8)) =
                    make_uint2(pack2<T>(y.x * inv, y.y * inv), pack2<T>(y.z * inv, y.w * inv));
            }
        }
        __syncthreads();                         // the rings are free for the next tile
    }
    // What follows waits for this grid alone: with a shared prefix it must end
    // after that kernel.  One block sees to it, the others make room.
    if (p.npre > 0 && (p.fold || (blockIdx.x | blockIdx.y | blockIdx.z) == 0)) pdl_wait();
}

template <typename T, int HD, int kWarps>
cudaError_t launch_w(const DecodeArgs &a, cudaStream_t st) {
    using S = Shape<HD, kWarps>;
    const auto fn = &k_decode_rows<T, HD, kWarps>;
    const cudaError_t e = ensure_smem(reinterpret_cast<const void *>(fn), S::kSmem);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)a.nsplit, (unsigned)(a.hk * a.row_tiles), (unsigned)a.batch);
    return launch_dependent(fn, grid, S::kThreads, S::kSmem, st, a);
}

template <typename T, int HD>
cudaError_t launch_hd(const DecodeArgs &a, cudaStream_t st) {
    if (a.row_warps == 2) return launch_w<T, HD, 2>(a, st);
    if (a.row_warps == 3) return launch_w<T, HD, 3>(a, st);
    return launch_w<T, HD, 4>(a, st);
}

}  // namespace

cudaError_t launch_decode_rows(DType dt, const DecodeArgs &a, cudaStream_t st) {
    if (dt == kF16) return a.hd == 64 ? launch_hd<__half, 64>(a, st) : launch_hd<__half, 128>(a, st);
    return a.hd == 64 ? launch_hd<__nv_bfloat16, 64>(a, st) : launch_hd<__nv_bfloat16, 128>(a, st);
}

}  // namespace swab
