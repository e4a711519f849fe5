// k_decode_prefix.cu -- the shared prefix of a batch, attended to by all its
// new tokens at once: for each key head a dense product of M = tokens x heads
// of the group rows with the prefix's keys, fp16 / bf16, head_dim 64 or 128.
//
// With R = tokens * group rows a key costs 4 R hd flops and 4 hd bytes: bound
// by the tensor cores above R = bf16 rate / copy rate = 281 rows, by memory
// below.  tcgen05 with the accumulators in tensor memory, so both can be
// reached: a block owns 128 rows of one key head and a run of 128-key chunks
// (as many pieces as the host finds best: the SMs left over go to the requests'
// own keys, whose kernel runs beside this one).
//
// Two streams of work go through the tensor cores in turn, so that one stream's
// softmax runs under the other's products: with more than 128 rows two row
// tiles over the same chunks (kPair; K and V are fetched once for both), with
// fewer the one tile's even and odd chunks, whose results are two parts.  Each
// stream has a score buffer and an fp32 accumulator in tensor memory (2 x 128 +
// 2 x hd columns, all 512 at hd 128).  Per chunk of a stream: S = Q K^T; four
// softmax warps (thread = row) take S to registers and make p = 2^(x - m)
// against the reference m so far; only when a weight passes 2^8 is the maximum
// found, the accumulator rescaled and the weights made again.  P goes, 16 bits
// wide, back over S; O += P V (A from tensor memory).  The next S of the stream
// is issued once that product is done, so it may overwrite P, and the softmax
// may rescale O without waiting.  The prefix needs no mask but at its very end
// and for absent blocks: there the scores are set to never win, and the values
// of those keys, which may be anything, are zeroed in shared memory.
//
// 128 requests x 32 heads over 8 key heads of 128, 16384 keys (34 GFLOP, 68 MB)
// with all SMs to it: 36 us on 144, 0.95 PFLOP/s; 31 to the last product.  5 us
// go to the first tiles, 5 to the parts (19 MB in whole sectors), 1.75 to a pair
// of chunks, of which the four products are 1.0.  (The plan gives it 96 there, 42
// us, and the rest to the requests' own keys.)  Tensor memory has no room for a
// second score buffer a stream, so a stream's softmax, product and scores follow
// one another.  Steps on the way: the halves of one tile's keys as
// streams 45 us; steps of 64 keys with two score buffers 60 (N = 64 costs the
// tensor cores as much as N = 128); the issuing loop under one lane 45.
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

template <int HD, bool kPair> struct Shape {
    static constexpr int kHalves = HD / 64;              // 64-channel tiles of 128-byte lines
    static constexpr int kTile = kBK * HD * 2;           // K or V of a chunk
    static constexpr int kQ1 = kBQ * HD * 2;             // Q of a row tile
    static constexpr int kQ = (kPair ? 2 : 1) * kQ1;
    static constexpr int kSlots = HD == 64 ? 10 : kPair ? 5 : 6;   // ring of K and V tiles
    static constexpr int kSmem = kQ + kSlots * kTile + 512 + 1024;
    static constexpr uint32_t kColS = 0, kColO = 256;    // S_g at 128 g (P_g over it), O_g at 256 + HD g
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// one lane of a converged warp
__device__ __forceinline__ bool elect_one() {
    uint32_t yes;
    asm volatile(
        "{\n"
        " .reg .pred p;\n"
        " elect.sync _|p, 0xffffffff;\n"
        " selp.u32 %0, 1, 0, p;\n"
        "}\n"
        : "=r"(yes));
    return yes != 0;
}
// a whole 32-byte sector: rows of parts lie far apart, so a warp's store
// fills 32 of them
__device__ __forceinline__ void stg32(float *dst, const uint32_t *v) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                 "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

template <typename T, int HD, bool kPair>
__global__ void __launch_bounds__(kThreads, 1)
    k_decode_prefix(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                    const __grid_constant__ CUtensorMap mapV, const __grid_constant__ DecodeArgs p) {
    using S = Shape<HD, kPair>;
    constexpr int kSlots = S::kSlots;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *qtile = base;                       // [row tiles][HD / 64] x 128 lines
    uint8_t *ring = base + S::kQ;
    uint64_t *bars = reinterpret_cast<uint64_t *>(ring + kSlots * S::kTile);
    uint64_t *qfull = bars, *full = bars + 1, *empty = full + kSlots;
    uint64_t *sfull = empty + kSlots;            // [2] a stream's S is written
    uint64_t *pfull = sfull + 2;                 // [2] its P is in place: one arrival a softmax warp
    uint64_t *odone = pfull + 2;                 // [2] its product is done
    uint64_t *done = odone + 2;
    uint32_t *holder = reinterpret_cast<uint32_t *>(done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(holder + 1);
    volatile int *no_abort = abort_flag + 1;
    volatile uint32_t *okmask = holder + 4;      // [8] the pages of chunk c that are there, at c mod 8

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int block = blockIdx.x / p.pre_pieces, split = blockIdx.x - block * p.pre_pieces, kvh = blockIdx.y;
    const int nchunks = (p.prefix_len + kBK - 1) / kBK;
    const int c0 = split * p.pre_chunks, c1 = min(nchunks, c0 + p.pre_chunks), n = c1 - c0;
    const int ppt = 128 >> p.page_log2;          // pages of a tile

    // this lane's page of chunk c, -1: none (warp 0)
    auto page_id = [&](int c) -> int {
        const int j = (c * ppt + lane) << p.page_log2;
        if (lane >= ppt || c >= c1 || j >= p.prefix_len) return -1;
        const int x = *GP(p.bnd, p.ptable + (j >> p.page_log2));
        if ((unsigned)x < (unsigned)p.n_blocks) return x;
        if (x != -1) atomicOr(p.err, kErrInvalid);
        return -1;
    };
    if (threadIdx.x == 0) {
        mbar_init(qfull, 1);
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sfull[i], 1);
            mbar_init(&pfull[i], kWorkers / 2);
            mbar_init(&odone[i], 1);
        }
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
    pdl_wait();
    if (warp == 2) {
        // The requests' own keys may start beside this: every block of their kernel
        // finds its word set by a thread that has passed the wait above.
        const long long blocks = (long long)gridDim.x * gridDim.y;
        for (long long k = (long long)blockIdx.y * gridDim.x + blockIdx.x + blocks * lane; k < p.row_blocks; k += 32 * blocks)
            store_release(GP(p.bnd, p.go + k), p.token);
        __syncwarp();
        if (lane == 0) pdl_trigger();
    }

    if (warp == 0) {
        // ---------------- TMA: lane k fetches page k of a tile ----------------
        if (lane == 0) {
            tma_prefetch_desc(&mapK);
            tma_prefetch_desc(&mapV);
            mbar_arrive_expect_tx(qfull, (uint32_t)(p.pre_tokens * p.group) * 128u * S::kHalves * (kPair ? 2u : 1u));
            for (int t = 0; t < (kPair ? 2 : 1); ++t)      // a tile past the last token reads zeros
                for (int h = 0; h < S::kHalves; ++h)
                    tma_load_3d(qtile + t * S::kQ1 + h * (kBQ * 128), &mapQ, qfull, 64 * h, kvh * p.group,
                                (block * (kPair ? 2 : 1) + t) * p.pre_tokens);
        }
        __syncwarp();
        int it = 0, id = page_id(c0);
        bool ok = true;
        for (int c = c0; c < c1 && ok; ++c) {
            const int ahead = page_id(c + 1);
            const uint32_t there = __ballot_sync(0xffffffffu, id >= 0);
            const uint32_t bytes = (uint32_t)__popc(there) * ((uint32_t)HD * 2u << p.page_log2);
            for (int v = 0; v < 2; ++v, ++it) {
                const int slot = it % kSlots;
                ok = __all_sync(0xffffffffu, mbar_wait(&empty[slot], ((it / kSlots) & 1) ^ 1, abort_flag, p.err));
                if (!ok) break;
                uint8_t *dst = ring + slot * S::kTile + ((lane << p.page_log2) * 128);
                if (lane == 0) {
                    // (rewritten 8 chunks later, when the softmax warps, at most
                    // kSlots / 2 chunks behind, have long read it)
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
        // The whole warp walks the loop and one lane issues: descriptors and
        // addresses then stay in uniform registers.  With the loop itself under
        // one lane each instruction moved its six operands there first and 16 of
        // them took 2100 cycles against the 1024 of the tensor cores.
        constexpr bool kBf16 = !std::is_same<T, __half>::value;
        constexpr uint32_t idesc_s = idesc_f16(kBQ, kBK, kBf16, false, false);
        constexpr uint32_t idesc_o = idesc_f16(kBQ, HD, kBf16, false, true);
        const bool leader = elect_one();
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint64_t qdesc = sdesc_sw128(smem_u32(qtile), 16, 1024);
        const uint64_t kdesc = sdesc_sw128(smem_u32(ring), 16, 1024);
        // V as an MN-major operand: 64-channel blocks one tile half apart
        const uint64_t vdesc = sdesc_sw128(smem_u32(ring), kBK * 128, 1024);
        auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, p.err));
        };
        // ring position and phase of a tile
        struct Place {
            int slot;
            uint32_t phase;
            __device__ __forceinline__ void step(int by) {
                slot += by;
                if (slot >= kSlots) {
                    slot -= kSlots;
                    phase ^= 1u;
                }
            }
        };
        auto scores = [&](int g, const Place &k_at, bool last_use) {       // S = Q K^T
            const uint64_t qa = qdesc + (uint64_t)((kPair ? g * S::kQ1 : 0) >> 4);
            const uint64_t ka = kdesc + (uint64_t)((k_at.slot * S::kTile) >> 4);
            tc_fence_after();
            if (leader) {
#pragma unroll
                for (int h = 0; h < S::kHalves; ++h)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_f16_ss(tm + S::kColS + kBK * g, qa + (uint64_t)((h * kBQ * 128) >> 4) + 2 * k,
                                   ka + (uint64_t)((h * kBK * 128) >> 4) + 2 * k, idesc_s, (h > 0 || k > 0) ? 1u : 0u);
                mma_commit(&sfull[g]);
                if (last_use) mma_commit(&empty[k_at.slot]);
            }
            __syncwarp();
        };
        auto product = [&](int g, const Place &v_at, uint32_t more, bool last_use) {      // O += P V
            const uint64_t va = vdesc + (uint64_t)((v_at.slot * S::kTile) >> 4);
            tc_fence_after();
            if (leader) {
#pragma unroll
                for (int k = 0; k < kBK / 16; ++k)
                    mma_f16_ts(tm + S::kColO + HD * g, tm + S::kColS + kBK * g + 8 * k, va + (uint64_t)((2048 * k) >> 4), idesc_o,
                               k == 0 ? more : 1u);
                mma_commit(&odone[g]);
                if (last_use) mma_commit(&empty[v_at.slot]);
            }
            __syncwarp();
        };
        bool ok = wait(qfull, 0);
        if constexpr (kPair) {
            // both streams over the chunks: a tile is waited for by the first one
            Place k_at{0, 0}, v_at{1, 0};
            if (ok && (ok = wait(&full[0], 0))) {
                scores(0, k_at, false);
                scores(1, k_at, true);
            }
            for (int i = 0; i < n && ok; ++i) {
                const uint32_t par = i & 1;
                const bool go = i + 1 < n;
                ok = wait(&full[v_at.slot], v_at.phase) && wait(&pfull[0], par);
                if (!ok) break;
                product(0, v_at, i > 0, false);
                if (go) {
                    k_at.step(2);
                    if (!(ok = wait(&full[k_at.slot], k_at.phase) && wait(&odone[0], par))) break;
                    scores(0, k_at, false);
                }
                if (!(ok = wait(&pfull[1], par))) break;
                product(1, v_at, i > 0, true);
                if (go) {
                    if (!(ok = wait(&odone[1], par))) break;
                    scores(1, k_at, true);
                    v_at.step(2);
                }
            }
        } else {
            // the streams take the chunks in turn
            Place k_at{0, 0}, v_at{1, 0};        // of the next scores, of the next product
            for (int c = 0; c < n && c < 2 && ok; ++c) {
                if (!(ok = wait(&full[k_at.slot], k_at.phase))) break;
                scores(c, k_at, true);
                k_at.step(2);
            }
            for (int c = 0; c < n && ok; ++c) {
                const int g = c & 1;
                const uint32_t par = (c >> 1) & 1;
                if (!(ok = wait(&full[v_at.slot], v_at.phase) && wait(&pfull[g], par))) break;
                product(g, v_at, c > 1, true);
                v_at.step(2);
                if (c + 2 < n) {
                    if (!(ok = wait(&full[k_at.slot], k_at.phase) && wait(&odone[g], par))) break;
                    scores(g, k_at, true);
                    k_at.step(2);
                }
            }
        }
        if (leader) {
            mma_commit(done);                    // nothing is in flight when tensor memory is freed
            mbar_wait(done, 0, no_abort, nullptr, 100000000ull);
        }
        __syncwarp();
    } else {
        // ---------------- softmax: thread = row of stream g ----------------
        const int quarter = warp & 3, g = (warp - 2) >> 2, row = 32 * quarter + lane;
        const int mine = kPair ? n : (n - g + 1) / 2;            // chunks of the stream
        const uint32_t lane_base = tmem_addr(tmem, quarter * 32, 0);
        const uint32_t at_s = lane_base + S::kColS + kBK * g, at_o = lane_base + S::kColO + HD * g;
        // (scale 0: small enough for equal weights, and -inf stays -inf)
        const float xs = p.scale_log2 == 0.f ? 1e-37f : p.scale_log2;
        const bool neg = xs < 0.f;
        const float never = neg ? INFINITY : -INFINITY;
        const bool real = row < p.pre_tokens * p.group;          // not one of the tile's spare rows, which hold anything
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        for (int i = 0; i < mine; ++i) {
            const int c = kPair ? i : 2 * i + g;
            if (!__all_sync(0xffffffffu, mbar_wait(&sfull[g], i & 1, abort_flag, p.err))) {
                ok = false;
                break;
            }
            tc_fence_after();
            const int j0 = (c0 + c) * kBK;
            const uint32_t there = okmask[c & 7];
            const bool whole = there == (1u << ppt) - 1u && j0 + kBK <= p.prefix_len;
            // keys that are there, 32 a word
            uint32_t vm[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
            if (!whole) {
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int j = 32 * w, left = p.prefix_len - j0 - j;
                    vm[w] = (((there >> (j >> p.page_log2)) & 1u) ? 0xffffu : 0u) |
                            (((there >> ((j + 16) >> p.page_log2)) & 1u) ? 0xffff0000u : 0u);
                    if (left < 32) vm[w] &= left <= 0 ? 0u : (1u << left) - 1u;
                }
                // V lines of absent keys become zeros, once the tile has landed: a
                // quarter of them for each warp
                const int it = 2 * c + 1, slot = it % kSlots;
                if (!__all_sync(0xffffffffu, mbar_wait(&full[slot], (it / kSlots) & 1, abort_flag, p.err))) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    for (int k = quarter; k < 32; k += 4) {
                        if ((vm[w] >> k) & 1u) continue;
                        if (lane < HD / 8)
                            *reinterpret_cast<uint4 *>(ring + slot * S::kTile + (lane >> 3) * (kBK * 128) + (32 * w + k) * 128 +
                                                       (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                fence_proxy_async_smem();
            }
            // 32 scores of this row; those of absent keys never win
            auto take = [&](int v, uint32_t (&x)[32]) {
                tmem_ld32(at_s + 32 * v, x);
                tmem_ld_wait();
                if (!whole) {
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (!((vm[v] >> k) & 1u)) x[k] = __float_as_uint(never);
                }
            };
            // P of the chunk against the reference mb, its sum and largest weight
            uint32_t pk[kBK / 2];
            auto weigh = [&](float mb, float &sum) -> float {
                const uint64_t xs2 = f2(xs, xs), nb2 = f2(-mb, -mb);
                uint64_t ls[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
                float top[2] = {0.f, 0.f};
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    uint32_t x[32];
                    take(v, x);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float y0, y1;
                        f2split(fma2(f2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), xs2, nb2), y0, y1);
                        const float p0 = ex2(y0), p1 = ex2(y1);
                        top[e & 1] = max3(top[e & 1], p0, p1);
                        ls[e & 1] = add2(ls[e & 1], f2(p0, p1));
                        pk[16 * v + e] = pack2<T>(p0, p1);
                    }
                }
                float l0, l1;
                f2split(add2(ls[0], ls[1]), l0, l1);
                sum = l0 + l1;
                return fmaxf(top[0], top[1]);
            };
            // Almost always no weight passes 2^8 against the reference so far, and
            // no maximum is needed; else it is found and the weights made again.
            float sum, corr = 1.f;
            bool made = false;
            if (__all_sync(0xffffffffu, m != -INFINITY || !real)) {
                const float top = weigh(real ? m : 0.f, sum);
                made = !__any_sync(0xffffffffu, real && top > 256.f);
            }
            if (!made) {
                float best = never;
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    uint32_t x[32];
                    take(v, x);
#pragma unroll
                    for (int e = 0; e < 32; e += 2)
                        best = neg ? min3(best, __uint_as_float(x[e]), __uint_as_float(x[e + 1]))
                                   : max3(best, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
                }
                const float cmax = best == never ? -INFINITY : best * xs;
                const bool raise = cmax > m + kSlack;        // the first time too: m is -inf
                const bool rescale = raise && m != -INFINITY;
                corr = rescale ? ex2(m - cmax) : 1.f;
                if (raise) m = cmax;
                if (__any_sync(0xffffffffu, rescale)) {
                    // (the product before this S is done: see the issuing warp)
#pragma unroll 1
                    for (int k = 0; k < HD / 32; ++k) {
                        uint32_t o[32];
                        tmem_ld32(at_o + 32 * k, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
                        tmem_st32(at_o + 32 * k, o);
                    }
                }
                weigh(m == -INFINITY ? 0.f : m, sum);
            }
#pragma unroll
            for (int v = 0; v < 2; ++v) tmem_st32(at_s + 32 * v, *reinterpret_cast<const uint32_t (*)[32]>(pk + 32 * v));
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive_warp(&pfull[g]);
            l = l * corr + sum;
        }
        // the stream's part
        const int tok = (block * (kPair ? 2 : 1) + (kPair ? g : 0)) * p.pre_tokens + row / p.group;
        const int hh = kvh * p.group + row % p.group;
        const bool live = real && tok < p.tokens;
        const long long at = ((long long)tok * p.h + hh) * p.nparts + p.nsplit + (kPair ? split : 2 * split + g);
        if (ok && mine > 0) ok = __all_sync(0xffffffffu, mbar_wait(&odone[g], (mine - 1) & 1, abort_flag, p.err));
        if (ok) {
            tc_fence_after();
            if (live) *GP(p.bnd, p.pml + at) = make_float2(m, l);
            if (mine > 0) {
#pragma unroll 1
                for (int k = 0; k < HD / 32; ++k) {
                    uint32_t o[32];
                    tmem_ld32(at_o + 32 * k, o);
                    tmem_ld_wait();
                    if (live) {
                        float *dst = p.po + at * HD + 32 * k;
#pragma unroll
                        for (int v = 0; v < 4; ++v) stg32(GPN(p.bnd, dst + 8 * v, 32), o + 8 * v);
                    }
                }
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, kCols);
}

template <typename T, int HD, bool kPair>
cudaError_t launch_t(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, const DecodeArgs &a, cudaStream_t st) {
    using S = Shape<HD, kPair>;
    const cudaError_t e = ensure_smem(reinterpret_cast<const void *>(&k_decode_prefix<T, HD, kPair>), S::kSmem);
    if (e != cudaSuccess) return e;
    const int tokens = a.pre_tokens * (kPair ? 2 : 1);           // of a block
    const dim3 grid((unsigned)(a.pre_pieces * ((a.tokens + tokens - 1) / tokens)), (unsigned)a.hk);
    return launch_dependent(&k_decode_prefix<T, HD, kPair>, grid, kThreads, S::kSmem, st, mq, mk, mv, a);
}

template <typename T>
cudaError_t launch_hd(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, const DecodeArgs &a, cudaStream_t st) {
    const bool pair = a.tokens > a.pre_tokens;
    if (a.hd == 64) return pair ? launch_t<T, 64, true>(mq, mk, mv, a, st) : launch_t<T, 64, false>(mq, mk, mv, a, st);
    return pair ? launch_t<T, 128, true>(mq, mk, mv, a, st) : launch_t<T, 128, false>(mq, mk, mv, a, st);
}

}  // namespace

cudaError_t launch_decode_prefix(DType dt, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, const DecodeArgs &a,
                                 cudaStream_t st) {
    return dt == kF16 ? launch_hd<__half>(mq, mk, mv, a, st) : launch_hd<__nv_bfloat16>(mq, mk, mv, a, st);
}

}  // namespace swab
