// k_decode_prefix.cu -- the shared prefix of a batch, attended to by all its
// new tokens at once: for each key head a dense product of M = tokens x heads
// of the group rows with the prefix's keys, fp16 / bf16, head_dim 64 or 128.
//
// With R = tokens * group rows a key costs 4 R hd flops and 4 hd bytes: bound
// by the tensor cores above R = bf16 rate / copy rate = 281 rows, by memory
// below.  tcgen05 with the accumulators in tensor memory, so both can be
// reached: a block owns 128 rows of one key head and a run of 128-key chunks
// (the prefix is split so that the blocks fill the SMs once).
//
// Per chunk: S = Q K^T (M = 128 rows, N = 128 keys) into one of two
// tensor-memory buffers; eight softmax warps, two for each 32-row quarter, 64
// keys each (thread = row), take S to registers, p = 2^(x - m) with a
// reference m of their own that is raised only by more than 2^8, and put P,
// 16 bits wide, back over their half of S; O_h += P V for each half h into the
// half's own fp32 accumulator (two of them, joined at the end like two pieces
// of a split list).  The prefix needs no mask but at its very end and for
// absent blocks: there the scores are set to never win, and the values of
// those keys, which may be anything, are zeroed in shared memory.
//
// A block of the cache is one TMA box of `page` lines; the tiles of 128 keys,
// K and V in turn, run through a ring.  Warps: 0 = TMA (each lane fetches one
// page of a tile), 1 = tensor memory and MMA, 2..9 = softmax.  Every wait is
// bounded; a wait that gives up raises the block's abort flag and the status
// word, and everybody leaves after the copies and products in flight.
#include <type_traits>

#include "swab_internal.h"
#include "swab_decode.cuh"

static constexpr unsigned kSwabFile = 16;   // site id of the bounds checks

namespace swab {
namespace {

constexpr int kBQ = 128, kBK = 128;
constexpr int kWorkers = 8;                     // softmax warps
constexpr int kThreads = 64 + 32 * kWorkers;
constexpr uint32_t kCols = 512;                 // tensor-memory columns
constexpr float kSlack = 8.f;

template <int HD> struct Shape {
    static constexpr int kHalves = HD / 64;              // 64-channel tiles of 128-byte lines
    static constexpr int kTile = kBK * HD * 2;           // K or V of a chunk
    static constexpr int kSlots = HD == 128 ? 6 : 8;     // ring of such tiles
    static constexpr int kQ = kBQ * HD * 2;
    static constexpr int kSmem = kQ + kSlots * kTile + 512 + 1024;
    static constexpr uint32_t kColS = 0, kColO = 256;    // S_b at 128 b (P_b over it), O_h at 256 + HD h
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <typename T, int HD>
__global__ void __launch_bounds__(kThreads, 1)
    k_decode_prefix(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                    const __grid_constant__ CUtensorMap mapV, const __grid_constant__ DecodeArgs p) {
    using S = Shape<HD>;
    constexpr int kSlots = S::kSlots;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *qtile = base;                       // [HD / 64] x 128 lines
    uint8_t *ring = base + S::kQ;
    uint64_t *bars = reinterpret_cast<uint64_t *>(ring + kSlots * S::kTile);
    uint64_t *qfull = bars, *full = bars + 1, *empty = full + kSlots;
    uint64_t *sfull = empty + kSlots;            // [2] S_b written
    uint64_t *pfull = sfull + 2;                 // [2] P_b in place: one arrival a softmax warp
    uint64_t *pempty = pfull + 2;                // [2] the product that read P_b is done
    uint64_t *mlbar = pempty + 2;                // [4] per quarter, its two warps
    uint64_t *done = mlbar + 4;
    uint32_t *holder = reinterpret_cast<uint32_t *>(done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(holder + 1);
    volatile int *no_abort = abort_flag + 1;
    volatile uint32_t *okmask = holder + 4;      // [8] the pages of chunk c that are there, at c mod 8

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tile = blockIdx.x / p.npre, split = blockIdx.x - tile * p.npre, kvh = blockIdx.y;
    const int nchunks = (p.prefix_len + kBK - 1) / kBK;
    const int c0 = split * p.pre_chunks, c1 = min(nchunks, c0 + p.pre_chunks), n = c1 - c0;
    const int ppt = 128 >> p.page_log2;          // pages of a tile

    if (threadIdx.x == 0) {
        mbar_init(qfull, 1);
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sfull[i], 1);
            mbar_init(&pfull[i], kWorkers);
            mbar_init(&pempty[i], 1);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&mlbar[i], 2);
        mbar_init(done, 1);
        *abort_flag = 0;
        *no_abort = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(holder, kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *holder;
    pdl_trigger();                               // the requests' own keys may start beside this

    if (warp == 0) {
        // ---------------- TMA: lane k fetches page k of a tile ----------------
        if (lane == 0) {
            tma_prefetch_desc(&mapK);
            tma_prefetch_desc(&mapV);
            mbar_arrive_expect_tx(qfull, (uint32_t)(p.pre_tokens * p.group) * 128u * S::kHalves);
            for (int h = 0; h < S::kHalves; ++h)
                tma_load_3d(qtile + h * (kBQ * 128), &mapQ, qfull, 64 * h, kvh * p.group, tile * p.pre_tokens);
        }
        __syncwarp();
        int it = 0;
        bool ok = true;
        int id = -1;
        auto page_id = [&](int c) -> int {       // this lane's page of chunk c, -1: none
            const int j = (c * ppt + lane) << p.page_log2;
            if (lane >= ppt || c >= c1 || j >= p.prefix_len) return -1;
            const int x = *GP(p.bnd, p.ptable + (j >> p.page_log2));
            if ((unsigned)x < (unsigned)p.n_blocks) return x;
            if (x != -1) atomicOr(p.err, kErrInvalid);
            return -1;
        };
        id = page_id(c0);
        for (int c = c0; c < c1 && ok; ++c) {
            const int ahead = page_id(c + 1);
            const uint32_t there = __ballot_sync(0xffffffffu, id >= 0);
            const uint32_t bytes = (uint32_t)__popc(there) * ((uint32_t)HD * 2u << p.page_log2);
            for (int v = 0; v < 2 && ok; ++v, ++it) {
                const int slot = it % kSlots;
                ok = __all_sync(0xffffffffu, mbar_wait(&empty[slot], ((it / kSlots) & 1) ^ 1, abort_flag, p.err));
                if (!ok) break;
                uint8_t *dst = ring + slot * S::kTile + ((lane << p.page_log2) * 128);
                if (lane == 0) {
                    // (rewritten 8 chunks later, long after the softmax warps
                    // have read it: they are at most 4 chunks behind)
                    okmask[(c - c0) & 7] = there;
                    mbar_arrive_expect_tx(&full[slot], bytes);
                }
                __syncwarp();
                if (id >= 0)
                    for (int h = 0; h < S::kHalves; ++h)
                        tma_load_3d(dst + h * (kBK * 128), v ? &mapV : &mapK, &full[slot], 64 * h, 0, id * p.hk + kvh);
                __syncwarp();
            }
            id = ahead;
        }
        // every copy issued lands before the block may exit
        if (lane == 0) {
            for (int k = it > kSlots ? it - kSlots : 0; k < it; ++k)
                mbar_wait(&full[k % kSlots], (k / kSlots) & 1, no_abort, nullptr, 100000000ull);
            mbar_wait(qfull, 0, no_abort, nullptr, 100000000ull);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr bool kBf16 = !std::is_same<T, __half>::value;
            constexpr uint32_t idesc_s = idesc_f16(kBQ, kBK, kBf16, false, false);
            constexpr uint32_t idesc_o = idesc_f16(kBQ, HD, kBf16, false, true);
            const uint64_t qdesc = sdesc_sw128(smem_u32(qtile), 16, 1024);
            const uint64_t kdesc = sdesc_sw128(smem_u32(ring), 16, 1024);
            // V as an MN-major operand: 64-channel blocks one tile half apart
            const uint64_t vdesc = sdesc_sw128(smem_u32(ring), kBK * 128, 1024);
            bool ok = mbar_wait(qfull, 0, abort_flag, p.err);
            auto product = [&](int c) -> bool {      // O_h += P V of chunk c (counted from 0)
                const int b = c & 1, it = 2 * c + 1, slot = it % kSlots;
                if (!mbar_wait(&full[slot], (it / kSlots) & 1, abort_flag, p.err)) return false;
                if (!mbar_wait(&pfull[b], (c >> 1) & 1, abort_flag, p.err)) return false;
                tc_fence_after();
                const uint64_t va = vdesc + (uint64_t)((slot * S::kTile) >> 4);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_f16_ts(tmem + S::kColO + HD * h, tmem + S::kColS + kBK * b + 64 * h + 8 * k,
                                   va + (uint64_t)((2048 * (4 * h + k)) >> 4), idesc_o, (c == 0 && k == 0) ? 0u : 1u);
                mma_commit(&pempty[b]);
                mma_commit(&empty[slot]);
                return true;
            };
            for (int c = 0; c < n && ok; ++c) {
                const int b = c & 1, it = 2 * c, slot = it % kSlots;
                ok = mbar_wait(&full[slot], (it / kSlots) & 1, abort_flag, p.err);
                if (!ok) break;
                // S_b holds P of chunk c - 2: its product has to be done
                if (c >= 2 && !(ok = mbar_wait(&pempty[b], ((c >> 1) & 1) ^ 1, abort_flag, p.err))) break;
                tc_fence_after();
                const uint64_t ka = kdesc + (uint64_t)((slot * S::kTile) >> 4);
#pragma unroll
                for (int h = 0; h < S::kHalves; ++h)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_f16_ss(tmem + S::kColS + kBK * b, qdesc + (uint64_t)((h * kBQ * 128) >> 4) + 2 * k,
                                   ka + (uint64_t)((h * kBK * 128) >> 4) + 2 * k, idesc_s, (h > 0 || k > 0) ? 1u : 0u);
                mma_commit(&empty[slot]);
                mma_commit(&sfull[b]);
                if (c > 0) ok = product(c - 1);
            }
            if (ok && n > 0) product(n - 1);
            mma_commit(done);                    // nothing is in flight when tensor memory is freed
            mbar_wait(done, 0, no_abort, nullptr, 100000000ull);
        }
    } else {
        // ---------------- softmax: thread = row, half h of the keys ----------------
        const int quarter = warp & 3, half = (warp - 2) >> 2, row = 32 * quarter + lane;
        const uint32_t lane_base = tmem_addr(tmem, quarter * 32, 0);
        const float xs = p.scale_log2;
        const bool neg = xs < 0.f;
        const float never = neg ? INFINITY : -INFINITY;
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        for (int c = 0; c < n; ++c) {
            const int b = c & 1;
            if (!__all_sync(0xffffffffu, mbar_wait(&sfull[b], (c >> 1) & 1, abort_flag, p.err))) {
                ok = false;
                break;
            }
            tc_fence_after();
            // keys of this half that are there, 32 a word
            uint32_t vm[2] = {0xffffffffu, 0xffffffffu};
            const int j0 = (c0 + c) * kBK;
            const uint32_t there = okmask[c & 7];
            const bool whole = there == (1u << ppt) - 1u && j0 + kBK <= p.prefix_len;
            if (!whole) {
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const int j = 64 * half + 32 * w;        // in the chunk
                    vm[w] = (((there >> (j >> p.page_log2)) & 1u) ? 0xffffu : 0u) |
                            (((there >> ((j + 16) >> p.page_log2)) & 1u) ? 0xffff0000u : 0u);
                    const int left = p.prefix_len - j0 - j;
                    if (left < 32) vm[w] &= left <= 0 ? 0u : (1u << left) - 1u;
                }
            }
            uint32_t x[64];
            tmem_ld32(lane_base + S::kColS + kBK * b + 64 * half, *reinterpret_cast<uint32_t (*)[32]>(x));
            tmem_ld32(lane_base + S::kColS + kBK * b + 64 * half + 32, *reinterpret_cast<uint32_t (*)[32]>(x + 32));
            tmem_ld_wait();
            if (!whole) {
#pragma unroll
                for (int i = 0; i < 64; ++i)
                    if (!((vm[i >> 5] >> (i & 31)) & 1u)) x[i] = __float_as_uint(never);
                // V lines of absent keys become zeros: this warp's quarter of the
                // lines of its half, once the tile has landed
                const int it = 2 * c + 1, slot = it % kSlots;
                if (!__all_sync(0xffffffffu, mbar_wait(&full[slot], (it / kSlots) & 1, abort_flag, p.err))) {
                    ok = false;
                    break;
                }
                for (int k = quarter; k < 64; k += 4) {
                    if ((vm[k >> 5] >> (k & 31)) & 1u) continue;
                    const int line = 64 * half + k;
                    for (int i = lane; i < HD / 8; i += 32)
                        *reinterpret_cast<uint4 *>(ring + slot * S::kTile + (i >> 3) * (kBK * 128) + line * 128 + (i & 7) * 16) =
                            make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
            }
            float ext[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t *y = x + 16 * k;
                float a = __uint_as_float(y[0]);
#pragma unroll
                for (int i = 1; i < 15; i += 2)
                    a = neg ? min3(a, __uint_as_float(y[i]), __uint_as_float(y[i + 1]))
                            : max3(a, __uint_as_float(y[i]), __uint_as_float(y[i + 1]));
                ext[k] = neg ? fminf(a, __uint_as_float(y[15])) : fmaxf(a, __uint_as_float(y[15]));
            }
            const float best = neg ? fminf(fminf(ext[0], ext[1]), fminf(ext[2], ext[3]))
                                   : fmaxf(fmaxf(ext[0], ext[1]), fmaxf(ext[2], ext[3]));
            const float cmax = best == never ? -INFINITY : best * xs;
            const bool raise = cmax > m + kSlack;            // the first time too: m is -inf
            const float mref = raise ? cmax : m;
            const float mb = mref == -INFINITY ? 0.f : mref;
            const uint64_t xs2 = f2(xs, xs), nb2 = f2(-mb, -mb);
            uint64_t ls[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                uint32_t pk[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float y0, y1;
                    f2split(fma2(f2(__uint_as_float(x[32 * v + 2 * e]), __uint_as_float(x[32 * v + 2 * e + 1])), xs2, nb2), y0, y1);
                    const float p0 = ex2(y0), p1 = ex2(y1);
                    ls[e & 1] = add2(ls[e & 1], f2(p0, p1));
                    pk[e] = pack2<T>(p0, p1);
                }
                tmem_st16(lane_base + S::kColS + kBK * b + 64 * half + 16 * v, pk);
            }
            float l0, l1;
            f2split(add2(ls[0], ls[1]), l0, l1);
            const bool rescale = raise && m != -INFINITY;
            const float corr = rescale ? ex2(m - mref) : 1.f;
            l = l * corr + (l0 + l1);
            if (__any_sync(0xffffffffu, rescale)) {
                // O_h must not move under a product: wait for chunk c - 1's
                if (!__all_sync(0xffffffffu, mbar_wait(&pempty[b ^ 1], ((c - 1) >> 1) & 1, abort_flag, p.err))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
#pragma unroll 1
                for (int k = 0; k < HD / 32; ++k) {
                    uint32_t o[32];
                    tmem_ld32(lane_base + S::kColO + HD * half + 32 * k, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * corr);
                    tmem_st32(lane_base + S::kColO + HD * half + 32 * k, o);
                }
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive_warp(&pfull[b]);
            m = mref;
        }
        // the two halves of a row, then the part of this block
        if (ok && n > 0) {
            ok = __all_sync(0xffffffffu, mbar_wait(&pempty[(n - 1) & 1], ((n - 1) >> 1) & 1, abort_flag, p.err));
            if (ok) {
                tc_fence_after();
                float2 *ml = reinterpret_cast<float2 *>(qtile);      // Q is done with
                ml[half * kBQ + row] = make_float2(m, l);
                mbar_arrive_warp(&mlbar[quarter]);
                ok = __all_sync(0xffffffffu, mbar_wait(&mlbar[quarter], 0, abort_flag, p.err));
                if (ok) {
                    const float2 e0 = ml[row], e1 = ml[kBQ + row];
                    const float M = fmaxf(e0.x, e1.x);
                    const float f0 = e0.x == -INFINITY ? 0.f : ex2(e0.x - M), f1 = e1.x == -INFINITY ? 0.f : ex2(e1.x - M);
                    const int tok = tile * p.pre_tokens + row / p.group, hh = kvh * p.group + row % p.group;
                    const bool live = row < p.pre_tokens * p.group && tok < p.tokens;
                    const long long at = ((long long)tok * p.h + hh) * p.nparts + p.nsplit + split;
                    if (live && half == 0) *GP(p.bnd, p.pml + at) = make_float2(M, e0.y * f0 + e1.y * f1);
#pragma unroll 1
                    for (int k = 0; k < HD / 32; ++k) {          // 16 channels of this half's share
                        uint32_t o0[16], o1[16];
                        const int ch = half * (HD / 2) + 16 * k;
                        tmem_ld16(lane_base + S::kColO + ch, o0);
                        tmem_ld16(lane_base + S::kColO + HD + ch, o1);
                        tmem_ld_wait();
                        if (live) {
                            float *dst = p.po + at * HD + ch;
#pragma unroll
                            for (int v = 0; v < 4; ++v) {
                                float4 y;
                                y.x = fmaf(__uint_as_float(o1[4 * v]), f1, __uint_as_float(o0[4 * v]) * f0);
                                y.y = fmaf(__uint_as_float(o1[4 * v + 1]), f1, __uint_as_float(o0[4 * v + 1]) * f0);
                                y.z = fmaf(__uint_as_float(o1[4 * v + 2]), f1, __uint_as_float(o0[4 * v + 2]) * f0);
                                y.w = fmaf(__uint_as_float(o1[4 * v + 3]), f1, __uint_as_float(o0[4 * v + 3]) * f0);
                                *reinterpret_cast<float4 *>(GPN(p.bnd, dst + 4 * v, 16)) = y;
                            }
                        }
                    }
                }
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, kCols);
}

template <typename T, int HD>
cudaError_t launch_t(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, const DecodeArgs &a, cudaStream_t st) {
    const cudaError_t e = ensure_smem(reinterpret_cast<const void *>(&k_decode_prefix<T, HD>), Shape<HD>::kSmem);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(a.npre * ((a.tokens + a.pre_tokens - 1) / a.pre_tokens)), (unsigned)a.hk);
    k_decode_prefix<T, HD><<<grid, kThreads, Shape<HD>::kSmem, st>>>(mq, mk, mv, a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode_prefix(DType dt, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, const DecodeArgs &a,
                                 cudaStream_t st) {
    if (dt == kF16) return a.hd == 64 ? launch_t<__half, 64>(mq, mk, mv, a, st) : launch_t<__half, 128>(mq, mk, mv, a, st);
    return a.hd == 64 ? launch_t<__nv_bfloat16, 64>(mq, mk, mv, a, st) : launch_t<__nv_bfloat16, 128>(mq, mk, mv, a, st);
}

}  // namespace swab
