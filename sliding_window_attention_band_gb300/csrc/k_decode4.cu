// k_decode4.cu -- banded attention of a few new tokens a request over a paged
// cache held in 4 bits: a code c of a channel stands for s (c - 8), s the scale of
// its 32 adjacent channels.
//
// k_decode4_rows: fp16 / bf16 with head_dim 64 or 128, and 96 where keys are not apart
// (no dilation), on the tensor cores.  The query heads that share a key head, of all the new tokens of a request, are the
// rows of one tile, so every code is read from memory once for all of them.
//
// A byte of codes carries four times the arithmetic of a byte in 16 bits, and what
// bounds the kernel is instructions, not memory: 32 keys of 8 heads' rows cost a warp
// about 700 (K 248 and V 268 of them, the rest scores, softmax and lookups), and the
// copies alone would take 29 of 43 us.  So
//  * the products are transposed: S^T = K Q^T and O^T = V^T P^T, the cache the A
//    operand (16 keys or channels) and the few rows its 8 columns; half as many
//    products as with the rows as A, and the values are made once for all rows;
//  * a code becomes a value by three instructions for two of them: shifted so that it
//    lies behind the exponent of 16 (x = 16 + c), masked and joined with it in one
//    operation, then x s - 24 s = s (c - 8), exact because s has 5 significant bits;
//  * codes stay as they lie: A's k order is any order that B's shares.  A lane takes
//    32 (16) adjacent channels of a key, one group, in K; 16 (8) adjacent channels of
//    four keys in V, whose words are joined by halves so that a register holds two
//    keys of one channel.  Three groups (96) do not go round four lanes: there a word
//    of each group (K) and four channels of each (V), with the scales of all three;
//  * a warp owns groups of 64 keys and runs on its own, with a ring of two stages (three
//    for head_dim 64).  Undilated (kRun) a group is four halves of 16 adjacent keys,
//    which never cross a block's end, as pages are multiples of 16: 16 lanes each start
//    one bulk copy (codes or scales, of K or of V) on the stage's mbarrier.  Lines are
//    looked up 32 halves at a time, a lane a half (one group ahead: 109 and 57 us for the
//    two cases that this brought to 88 and 47).  With a dilation keys lie apart: cp.async,
//    a key's line by its pieces.
// Lines lie in the ring as in memory: the reads of K meet no bank twice (slot_of says
// which key sits in which row of the product), V's of 8 bytes are spread by the same
// order over its key pairs.
// A key that no row attends to, or that is not there, has a score of -inf and, in the
// ring, a scale of 0 for its V: it adds 0 whatever the cache holds there.
// The softmax is that of k_decode_rows: the running maximum raised only when a
// score passes it by 2^8, weights rounded to 16 bits for the product (what the tensor
// cores take; as in decode over 16 bits), sums fp32.
//
// Measured (8 heads of 128, 32 query heads, bf16): one request of 131072 tokens 42.5 us,
// 3.6 TB/s of codes and scales; 57 requests x 4096 61 us, 4.4 TB/s; with 16 rows a tile
// 84 us, 3.2 TB/s.  16 requests of 3000 to 5000, 24 heads over 8 of 96: 28 us, where
// the general kernel took 143.  A single step of one short request 4.4 us, of which
// launch and join are most.
//
// k_decode4_general: every type and head size (a multiple of 32), fp32 arithmetic.
#include <type_traits>

#include "swab_internal.h"
#include "swab_decode.cuh"

static constexpr unsigned kSwabFile = 18;   // site id of the bounds checks

namespace swab {
namespace {

constexpr int kGroup = 64;         // keys of a group, which a warp takes at a time
constexpr float kSlack = 8.f;      // log2 headroom of the running maximum

template <int HD, int kN, int kWarps> struct Shape4 {
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kBlocks = (HD == 64 && kN == 1 ? 16 : 12) / kWarps;   // an SM holds, by registers and shared memory
    static constexpr int kStages = HD == 64 ? 3 : 2;
    static constexpr int kLine = HD / 2;                            // bytes of codes of a key
    static constexpr int kScale = HD / 16;                          // bytes of its scales
    static constexpr int kCodes = kGroup * kLine, kScales = kGroup * kScale;
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

// Codes to values, two at a time.  (x & mask) | magic is one instruction when both
// constants are in registers: an immediate for each makes two of it, so they are
// held where the compiler does not see what they are.
struct Masks {
    uint32_t mask, magic;
};
template <typename T> __device__ __forceinline__ Masks masks_of() {
    constexpr bool kHalf = std::is_same<T, __half>::value;      // 16 + c: bits 6..9 of a half, or 3..6
    Masks k;
    asm volatile("mov.b32 %0, %2;\n mov.b32 %1, %3;" : "=r"(k.mask), "=r"(k.magic)
                 : "n"(kHalf ? 0x03c003c0 : 0x00780078), "n"(kHalf ? 0x4c004c00 : 0x41804180));
    return k;
}
// codes n and n + 4 of a word as 16 + c
template <typename T, int n> __device__ __forceinline__ uint32_t biased(uint32_t w, const Masks &k) {
    constexpr int left = std::is_same<T, __half>::value ? 6 - 4 * n : 3 - 4 * n;
    const uint32_t x = left >= 0 ? w << (left & 31) : w >> (-left & 31);
    uint32_t y;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(x), "r"(k.mask), "r"(k.magic));
    return y;
}
template <typename T> __device__ __forceinline__ uint32_t fma_two(uint32_t x, uint32_t s, uint32_t b) {
    uint32_t y;
    if constexpr (std::is_same<T, __half>::value) asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(x), "r"(s), "r"(b));
    else asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(x), "r"(s), "r"(b));
    return y;
}
template <typename T> __device__ __forceinline__ uint32_t bias_of(uint32_t s) {       // -24 s, exact
    uint32_t y;
    if constexpr (std::is_same<T, __half>::value) asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(s), "r"(0xce00ce00u));
    else asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(s), "r"(0xc1c0c1c0u));
    return y;
}
// word -> {value n, value n + 4} for n = 0..3
template <typename T> __device__ __forceinline__ void values(uint32_t w, uint32_t s, uint32_t b, const Masks &k, uint32_t (&v)[4]) {
    v[0] = fma_two<T>(biased<T, 0>(w, k), s, b);
    v[1] = fma_two<T>(biased<T, 1>(w, k), s, b);
    v[2] = fma_two<T>(biased<T, 2>(w, k), s, b);
    v[3] = fma_two<T>(biased<T, 3>(w, k), s, b);
}

// Key (of 8) in row p of a product: the even rows take the first four, the odd ones
// the others backwards.
__device__ __forceinline__ int slot_of(int p) { return (p & 1) ? 4 + ((p >> 1) ^ 3) : p >> 1; }

// A warp's copies of one stage have arrived: bounded, never trapping (the context
// stays usable, the status word says so).
struct Waiter {
    volatile int *abort_flag;
    unsigned *err;
    __device__ __forceinline__ void wait(uint64_t *bar, uint32_t parity) const { mbar_wait(bar, parity, abort_flag, err); }
};
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}

// The positions that a tile's rows attend to, undilated, as halves of 16: those with
// sinks, then those of the band.
struct Halves {
    int count, nsink, band_lo, hi, sink_halves, band_half;
    __device__ __forceinline__ int at(int u) const { return (u < sink_halves ? u : band_half + (u - sink_halves)) << 4; }
    __device__ __forceinline__ bool has(int j) const { return j < nsink || (j >= band_lo && j <= hi); }
};
__device__ __forceinline__ Halves halves_of(const DecodeArgs &p, const Request &q, int a_lo, int a_hi) {
    Halves k;
    const int lo = q.i0 + a_lo;
    k.hi = min(q.i0 + a_hi, q.last);
    k.nsink = max(min(p.n_sink, k.hi + 1), 0);
    k.band_lo = (int)max((long long)lo - p.w, (long long)p.n_sink);
    k.sink_halves = (int)(((unsigned)k.nsink + 15u) >> 4);
    k.band_half = max(k.band_lo >> 4, k.sink_halves);
    k.count = k.sink_halves + max((k.hi >> 4) - k.band_half + 1, 0);
    return k;
}

// Grid: (piece, key head and tile of 8 kN rows, request).  kWarps: the warps that
// share a piece.  kRun: undilated, whole halves of a block at a time.
template <typename T, int HD, int kN, int kWarps, bool kRun>
__global__ void __launch_bounds__(32 * kWarps, Shape4<HD, kN, kWarps>::kBlocks) k_decode4_rows(const __grid_constant__ DecodeArgs p) {
    using S = Shape4<HD, kN, kWarps>;
    constexpr int kThreads = S::kThreads, kRows = 8 * kN;
    constexpr int kWords = HD / 32;                        // words of codes of a lane's share of a key (K)
    constexpr int kSteps = HD / 16, kTiles = HD / 16;      // products of 16 channels (S), of 16 channels (O)
    constexpr int kQuads = HD / 32;                        // of four channels: a lane's share of a key (V)
    // With three groups a lane's share cannot be one of them: word t4 of each group (K), quad g
    // of each (V) instead of adjacent ones, and the scales of all groups.
    constexpr bool kThree = HD == 96;
    static_assert(!kThree || kRun, "lines of 48 bytes come by bulk copies only");
    constexpr int kChunks = S::kLine / 16, kPer = 32 / kChunks;   // 16-byte pieces of a line; lines of a copy instruction
    constexpr int kPad = HD + 8;                           // floats of a row in the final exchange
    static_assert(kRows * kPad * 4 <= S::kRing, "a warp's O fits its ring");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~static_cast<uintptr_t>(127));
    __shared__ float2 sml[kWarps][kRows];
    __shared__ float swt[kWarps][kRows];
    __shared__ float2 stot[kRows];
    __shared__ uint2 sok[kRun ? 1 : kWarps][S::kStages];   // which keys of the group in a stage are there
    __shared__ uint64_t sbar[kRun ? kWarps : 1][S::kStages];
    __shared__ int sabort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int split = blockIdx.x, r = blockIdx.z;
    const int kvh = (int)(blockIdx.y % (unsigned)p.hk), tile0 = (int)(blockIdx.y / (unsigned)p.hk);
    const int tiles_y = gridDim.y / p.hk;
    if constexpr (kRun) {
        if (threadIdx.x == 0) sabort = 0;
        if (lane < S::kStages) mbar_init(&sbar[warp][lane], 1);
        fence_barrier_init();
        __syncthreads();
    }
    const Waiter waiter{&sabort, p.err};
    pdl_wait();
    pdl_trigger();
    const Request q = request_of(p, r);
    uint8_t *ring = smem + warp * S::kRing;
    const uint32_t ring_s = smem_u32(ring);
    // what this lane reads: in K keys slot_of(g) and + 8 of each 16, in V keys t4 and 7 - t4 and + 8
    const int k_slot = slot_of(g), v_even = t4, v_odd = 4 + (t4 ^ 3);
    const uint32_t k_at = k_slot * S::kLine + t4 * (kThree ? 4 : HD / 8);
    const uint32_t v_unit = kThree ? 2 : HD / 16;
    const uint32_t ve_at = S::kCodes + v_even * S::kLine + g * v_unit, vo_at = S::kCodes + v_odd * S::kLine + g * v_unit;
    const uint32_t ks_at = k_slot * S::kScale + (HD == 128 ? t4 : HD == 64 ? t4 >> 1 : 0) * 2;
    const int v_group = HD == 128 ? g >> 1 : HD == 64 ? g >> 2 : 0;
    const uint32_t ves_at = S::kScales + v_even * S::kScale + v_group * 2;
    const uint32_t vos_at = S::kScales + v_odd * S::kScale + v_group * 2;
    // scores are scaled by |scale| inside the exponent; a negative one turns Q
    // round (exact), zero clears it
    const float scale = p.scale_log2 == 0.f ? 1.f : fabsf(p.scale_log2);
    const uint32_t q_and = p.scale_log2 == 0.f ? 0u : 0xffffffffu, q_xor = p.scale_log2 < 0.f ? 0x80008000u : 0u;
    // tiles of rows: with a key stride each token has its own
    const int per_tok = (p.group + kRows - 1) / kRows;
    const int ntiles = kRun ? (q.m * p.group + kRows - 1) / kRows : q.m * per_tok;
    const Masks masks = masks_of<T>();
    int to_fill = 0, to_read = 0;                          // stages
    uint32_t phase = 0;                                    // of the barriers (kRun)
    // kRun: lane 4 half + what copies codes of K, of V, scales of K, of V (what) of a half
    const uint32_t copy_unit = t4 < 2 ? S::kLine : S::kScale, copy_half = (lane >> 2) & 3;
    const char *copy_from = reinterpret_cast<const char *>(t4 == 0 ? p.Kc : t4 == 1 ? p.Vc : t4 == 2 ? p.Ks : p.Vs);
    const uint32_t copy_to = ring_s + (t4 < 2 ? t4 * S::kCodes : 2 * S::kCodes + (t4 - 2) * S::kScales) + copy_half * 16 * copy_unit;

    // a tile of rows row0 .. row0 + nrows - 1, at most 8 N
    auto run = [&](auto tag, int row0, int nrows) {
        constexpr int N = decltype(tag)::value;
        const int a_lo = row0 / p.group, a_hi = (row0 + nrows - 1) / p.group;
        Halves halves;
        KeyList keys;
        int lo, hi;                                        // of the list of halves, or of keys
        if constexpr (kRun) {
            halves = halves_of(p, q, a_lo, a_hi);
            const int per = p.chunk >> 4;
            lo = (int)min((long long)split * per, (long long)halves.count);
            hi = split == p.nsplit - 1 ? halves.count : (int)min((long long)lo + per, (long long)halves.count);
        } else {
            keys = keys_of(p, q, a_lo, a_hi);
            lo = (int)min((long long)split * p.chunk, (long long)keys.count);
            hi = split == p.nsplit - 1 ? keys.count : (int)min((long long)lo + p.chunk, (long long)keys.count);
        }
        constexpr int kUnit = kRun ? kGroup / 16 : kGroup;   // entries of the list a group takes
        const int groups = (int)(((long long)hi - lo + kUnit - 1) / kUnit);
        const int mine = groups > warp ? (groups - warp + kWarps - 1) / kWarps : 0;   // of this warp

        const int pos_lo = q.i0 + a_lo, pos_hi = q.i0 + a_hi;

        // kRun.  The warp's halves are looked up 32 at a time, a lane a half (8 groups),
        // the block ids of the next ones while these are used: their lines, and
        // which are there and attended to by every row.
        int next_id = -1, batch = 0;
        uint32_t lines = kNoLine, there = 0, full = 0, there_before = 0, full_before = 0;
        auto half_of = [&](int batch_, int &j0) -> bool {
            // (unsigned: past the end of the longest list the sum passes 2^31)
            const int n = 8 * batch_ + (lane >> 2);
            const unsigned u = 4u * (unsigned)(warp + kWarps * n) + (unsigned)(lane & 3);
            if (!(n < mine && u < (unsigned)(hi - lo))) return false;
            j0 = halves.at(lo + (int)u);
            return true;
        };
        auto fetch_ids = [&](int batch_) {
            int j0 = 0, col = -1;
            if (half_of(batch_, j0)) col = key_column(p, q, j0);
            next_id = col < 0 ? -1 : *GP(p.bnd, q.trow + col);
        };
        auto take_ids = [&](int batch_) {
            int j0 = 0;
            const bool in = half_of(batch_, j0);
            lines = in ? block_line(p, next_id, j0 & ((1 << p.page_log2) - 1), kvh) : kNoLine;
            bool here = lines != kNoLine;
#if SWAB_BOUNDS_CHECK
            // (a copy that would leave its buffer is left out)
            const unsigned long long ln = lines;
            auto inside = [&](const void *base, int unit) {
                const char *src = reinterpret_cast<const char *>(base) + ln * unit;
                return GPN(p.bnd, src, 16 * unit) == src;
            };
            if (here && !(inside(p.Kc, S::kLine) && inside(p.Vc, S::kLine) && inside(p.Ks, S::kScale) && inside(p.Vs, S::kScale))) here = false;
#endif
            there_before = there;
            full_before = full;
            there = __ballot_sync(0xffffffffu, here);
            full = __ballot_sync(0xffffffffu, here && j0 + 15 <= pos_lo && (j0 + 15 < p.n_sink || (long long)pos_hi - j0 <= p.w));
            batch = batch_;
            fetch_ids(batch_ + 1);
        };
        // lines of keys `lane` and `lane` + 32 of the warp's group n
        auto look_up = [&](int n) -> uint2 {
            const unsigned u = (unsigned)kGroup * (unsigned)(warp + kWarps * n) + (unsigned)lane;
            uint2 line = make_uint2(kNoLine, kNoLine);
            if (n < mine && u < (unsigned)(hi - lo)) line.x = key_line(p, q, keys.at(lo + (int)u), kvh);
            if (n < mine && u + 32u < (unsigned)(hi - lo)) line.y = key_line(p, q, keys.at(lo + (int)u + 32), kvh);
            return line;
        };
        // the warp's group n into the next stage; `line`: of its keys (not kRun)
        auto issue = [&](int n, const uint2 &line) {
            if (n < mine) {
                if constexpr (kRun) {
                    if ((n & 7) == 0) take_ids(n >> 3);
                    const uint32_t have = there >> (4 * (n & 7)) & 15u;
                    const uint32_t ln = __shfl_sync(0xffffffffu, lines, 4 * (n & 7) + copy_half);
                    uint64_t *bar = &sbar[warp][to_fill];
                    if (lane == 0) mbar_arrive_expect_tx(bar, __popc(have) * (S::kStage / 4));
                    __syncwarp();
                    if (lane < 16 && (have >> copy_half & 1u))
                        bulk_load(copy_to + to_fill * S::kStage, copy_from + (unsigned long long)ln * copy_unit, 16 * copy_unit, bar);
                } else {
                    const uint2 have = make_uint2(__ballot_sync(0xffffffffu, line.x != kNoLine), __ballot_sync(0xffffffffu, line.y != kNoLine));
                    if (lane == 0) sok[warp][to_fill] = have;
                    const uint32_t at = ring_s + to_fill * S::kStage, to = at + lane * 16;
#pragma unroll
                    for (int i = 0; i < kGroup / kPer; ++i) {
                        const uint32_t ln = __shfl_sync(0xffffffffu, i * kPer < 32 ? line.x : line.y, (i * kPer & 31) + lane / kChunks);
                        const uint32_t bytes = ln != kNoLine ? 16u : 0u;
                        const unsigned long long from = (unsigned long long)(ln != kNoLine ? ln : 0u) * S::kLine + lane % kChunks * 16;
                        cp_async16(to + i * kPer * S::kLine, GPN(p.bnd, reinterpret_cast<const char *>(p.Kc) + from, 16), bytes);
                        cp_async16(to + i * kPer * S::kLine + S::kCodes, GPN(p.bnd, reinterpret_cast<const char *>(p.Vc) + from, 16), bytes);
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t ln = i ? line.y : line.x, bytes = ln != kNoLine ? (uint32_t)S::kScale : 0u;
                        const unsigned long long from = (unsigned long long)(ln != kNoLine ? ln : 0u) * S::kScale;
                        const uint32_t sc = at + 2 * S::kCodes + (32 * i + lane) * S::kScale;
                        cp_async_small<S::kScale>(sc, GPN(p.bnd, reinterpret_cast<const char *>(p.Ks) + from, S::kScale), bytes);
                        cp_async_small<S::kScale>(sc + S::kScales, GPN(p.bnd, reinterpret_cast<const char *>(p.Vs) + from, S::kScale), bytes);
                    }
                }
                to_fill = to_fill + 1 == S::kStages ? 0 : to_fill + 1;
            }
            if constexpr (!kRun) cp_commit();
        };

        // fill the ring; the lines of the stage after it are looked up meanwhile
        uint2 next = make_uint2(kNoLine, kNoLine);
        if constexpr (kRun) {
            fetch_ids(0);
#pragma unroll
            for (int s = 0; s < S::kStages - 1; ++s) issue(s, next);
        } else {
            uint2 first[S::kStages];
#pragma unroll
            for (int s = 0; s < S::kStages; ++s) first[s] = look_up(s);
#pragma unroll
            for (int s = 0; s < S::kStages - 1; ++s) issue(s, first[s]);
            next = first[S::kStages - 1];
        }

        // Q of the tile as B operands: row 8 n + g, in the k order of a lane's words (8 w +
        // {2 e, 2 e + 4}, {2 e + 1, 2 e + 5} of its channels in step 2 w + e)
        uint32_t qb[N][kSteps][2];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int rr = 8 * n + g;
            const bool live = rr < nrows;
            const int row = row0 + (live ? rr : 0), a = row / p.group, hh = kvh * p.group + row - a * p.group;
            const T *src = reinterpret_cast<const T *>(p.Q) + (long long)(q.row0 + a) * p.q_stride + (long long)hh * HD + t4 * (kThree ? 8 : HD / 4);
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
                const uint4 x = *reinterpret_cast<const uint4 *>(GPN(p.bnd, src + (kThree ? 32 : 8) * w, 16));
                const uint32_t v[4] = {live ? (x.x & q_and) ^ q_xor : 0u, live ? (x.y & q_and) ^ q_xor : 0u,
                                       live ? (x.z & q_and) ^ q_xor : 0u, live ? (x.w & q_and) ^ q_xor : 0u};
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    qb[n][2 * w + e][0] = __byte_perm(v[e], v[2 + e], 0x5410);
                    qb[n][2 * w + e][1] = __byte_perm(v[e], v[2 + e], 0x7632);
                }
            }
        }

        // O^T of row 2 t4 + e: of the lane's channels o[n][i][e] is 2 i, o[n][i][2 + e] 2 i + 1
        float o[N][kTiles][4], m[N][2], l[N][2];
#pragma unroll
        for (int n = 0; n < N; ++n) {
#pragma unroll
            for (int d = 0; d < kTiles; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][d][e] = 0.f;
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
        }

        for (int n_it = 0; n_it < mine; ++n_it) {
            // the ring's free stage takes group n_it + kStages - 1
            uint2 ahead = make_uint2(kNoLine, kNoLine);
            if constexpr (!kRun) ahead = look_up(n_it + S::kStages);
            issue(n_it + S::kStages - 1, next);
            next = ahead;
            const uint8_t *stage = ring + to_read * S::kStage;
            // which of the group's halves (not kRun: keys) are there; halves that every row attends to
            uint32_t there4 = 0, full4 = 0;
            uint2 there64 = make_uint2(0u, 0u);
            if constexpr (kRun) {
                const bool now = n_it >> 3 == batch;
                there4 = (now ? there : there_before) >> (4 * (n_it & 7)) & 15u;
                full4 = (now ? full : full_before) >> (4 * (n_it & 7)) & 15u;
                waiter.wait(&sbar[warp][to_read], phase);
            } else {
                cp_wait<S::kStages - 1>();
                __syncwarp();
                there64 = sok[warp][to_read];
            }
            if (++to_read == S::kStages) {
                to_read = 0;
                phase ^= 1u;
            }

            // kX blocks of 16 keys at a time: all four for 8 rows (more products in flight: 128k
            // keys 42.5 us, two at a time 43.9), two where tiles may have 16 (registers: with four for
            // those of 8 among them the window of 48 requests takes 87.6 us, so 86.5)
            constexpr int kX = kN == 1 ? 4 : 2;
#pragma unroll 1
            for (int x0 = 0; x0 < 4; x0 += kX) {
                const int u0 = lo + kUnit * (warp + kWarps * n_it) + x0 * (kUnit / 4);
                const uint8_t *st = stage + x0 * 16 * S::kLine, *sc = stage + 2 * S::kCodes + x0 * 16 * S::kScale;
                uint32_t ok[kX / 2];                       // which keys are there, 32 at a time
                bool all;
                if constexpr (kRun) {
                    const uint32_t have = there4 >> x0 & ((1u << kX) - 1u);
                    if (have == 0u) continue;              // (absent blocks: the next ones may be there)
                    all = (full4 >> x0 & ((1u << kX) - 1u)) == (1u << kX) - 1u;
                    if (!all) {
                        // scales of the values that no row attends to: 0, whatever is there
#pragma unroll
                        for (int i = 0; i < kX / 2; ++i) {
                            const int x = 2 * i + (lane >> 4);
                            const bool here = (have >> x & 1u) && halves.has(halves.at(u0 + x) + (lane & 15));
                            ok[i] = __ballot_sync(0xffffffffu, here);
                            if (!here) {
                                uint8_t *zero = const_cast<uint8_t *>(sc) + S::kScales + (32 * i + lane) * S::kScale;
                                if constexpr (HD == 128) *reinterpret_cast<uint2 *>(zero) = make_uint2(0u, 0u);
                                else if constexpr (kThree) for (int k = 0; k < 3; ++k) reinterpret_cast<uint16_t *>(zero)[k] = 0;
                                else *reinterpret_cast<uint32_t *>(zero) = 0u;
                            }
                        }
                        fence_proxy_async_smem();          // (before the stage's next copies)
                        __syncwarp();
                    }
                } else {
                    if (kX == 4) ok[0] = there64.x, ok[kX / 2 - 1] = there64.y;
                    else ok[0] = x0 ? there64.y : there64.x;
                    uint32_t every = ok[0];
                    if (kX == 4) every &= ok[kX / 2 - 1];
                    const int j_lo = keys.at(u0), j_hi = keys.at(u0 + 16 * kX - 1);
                    all = every == 0xffffffffu && j_hi <= pos_lo && (j_hi < p.n_sink || (long long)pos_hi - j_lo <= (long long)p.w * p.stride);
                }

                // scores: c[n][x]: keys 16 x + slot_of(g) (e = 0, 1: rows) and + 8 (e = 2, 3)
                float c[N][kX][4];
#pragma unroll
                for (int n = 0; n < N; ++n)
#pragma unroll
                    for (int x = 0; x < kX; ++x)
#pragma unroll
                        for (int e = 0; e < 4; ++e) c[n][x][e] = 0.f;
                uint32_t w[kX][2][kWords], s[kX][2], b[kX][2];
                auto k_scale = [&](int x, int h, int k) {  // of word k
                    const uint32_t one = *reinterpret_cast<const uint16_t *>(sc + (16 * x + 8 * h) * S::kScale + ks_at + (kThree ? 2 * k : 0));
                    s[x][h] = __byte_perm(one, one, 0x1010);
                    b[x][h] = bias_of<T>(s[x][h]);
                };
#pragma unroll
                for (int x = 0; x < kX; ++x)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint8_t *at = st + (16 * x + 8 * h) * S::kLine + k_at;
                        if constexpr (HD == 128) {
                            const uint4 v = *reinterpret_cast<const uint4 *>(at);
                            w[x][h][0] = v.x, w[x][h][1] = v.y, w[x][h][kWords - 2] = v.z, w[x][h][kWords - 1] = v.w;
                        } else if constexpr (kThree) {
#pragma unroll
                            for (int k = 0; k < kWords; ++k) w[x][h][k] = *reinterpret_cast<const uint32_t *>(at + 16 * k);
                        } else {
                            const uint2 v = *reinterpret_cast<const uint2 *>(at);
                            w[x][h][0] = v.x, w[x][h][1] = v.y;
                        }
                        if (!kThree) k_scale(x, h, 0);
                    }
#pragma unroll
                for (int k = 0; k < kWords; ++k)
#pragma unroll
                    for (int x = 0; x < kX; ++x) {
                        if (kThree) k_scale(x, 0, k), k_scale(x, 1, k);
                        uint32_t va[4], vb[4];
                        values<T>(w[x][0][k], s[x][0], b[x][0], masks, va);
                        values<T>(w[x][1][k], s[x][1], b[x][1], masks, vb);
#pragma unroll
                        for (int n = 0; n < N; ++n) mma16816<T>(c[n][x], va[0], vb[0], va[1], vb[1], qb[n][2 * k][0], qb[n][2 * k][1]);
#pragma unroll
                        for (int n = 0; n < N; ++n) mma16816<T>(c[n][x], va[2], vb[2], va[3], vb[3], qb[n][2 * k + 1][0], qb[n][2 * k + 1][1]);
                    }
                if (!all) {
                    __syncwarp();                          // (a branch: predicated, this costs every group 70 instructions)
                    // positions of this lane's rows (row 8 n + 2 t4 + e)
                    int pos[N][2];
#pragma unroll
                    for (int n = 0; n < N; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) pos[n][e] = q.i0 + (row0 + min(8 * n + 2 * t4 + e, nrows - 1)) / p.group;
#pragma unroll
                    for (int x = 0; x < kX; ++x)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int slot = 16 * x + 8 * h + k_slot;
                            const int j = kRun ? halves.at(u0 + x) + 8 * h + k_slot : keys.at(u0 + slot);
                            const bool here = (ok[x / 2] >> (slot & 31)) & 1u;
#pragma unroll
                            for (int n = 0; n < N; ++n)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    if (!(here && attends(p, pos[n][e], j))) c[n][x][2 * h + e] = -INFINITY;
                        }
                }
                float best[N][2];
                bool up = false;
#pragma unroll
                for (int n = 0; n < N; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = c[n][0][e];
#pragma unroll
                        for (int x = 0; x < kX; ++x) mx = x == 0 ? fmaxf(mx, c[n][0][2 + e]) : max3(mx, c[n][x][e], c[n][x][2 + e]);
                        best[n][e] = mx * scale;
                        up |= best[n][e] > m[n][e] + kSlack;
                    }
                if (__any_sync(0xffffffffu, up)) {   // raise the maxima, scale what was summed so far
#pragma unroll
                    for (int n = 0; n < N; ++n)
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
                uint32_t pb[N][kX][2];
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const float m0 = m[n][0] == -INFINITY ? 0.f : m[n][0], m1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
#pragma unroll
                    for (int x = 0; x < kX; ++x)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float p0 = ex2(fmaf(c[n][x][2 * h], scale, -m0)), p1 = ex2(fmaf(c[n][x][2 * h + 1], scale, -m1));
                            l[n][0] += p0;
                            l[n][1] += p1;
                            pb[n][x][h] = transpose8(pack2<T>(p0, p1));
                        }
                }
#pragma unroll
                for (int x = 0; x < kX; ++x) {
                    // keys 16 x + 8 h + v_even, v_odd
                    uint32_t we[2][kWords], wo[2][kWords], vs[2], vb[2];     // (kThree: a quad in each)
                    auto v_scales = [&](int h, int k) {    // of both keys, quad k
                        const uint8_t *of = sc + (16 * x + 8 * h) * S::kScale + (kThree ? 2 * k : 0);
                        vs[h] = __byte_perm(*reinterpret_cast<const uint16_t *>(of + ves_at), *reinterpret_cast<const uint16_t *>(of + vos_at), 0x5410);
                        vb[h] = bias_of<T>(vs[h]);
                    };
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint8_t *at = st + (16 * x + 8 * h) * S::kLine;
                        if constexpr (HD == 128) {
                            const uint2 ve = *reinterpret_cast<const uint2 *>(at + ve_at), vo = *reinterpret_cast<const uint2 *>(at + vo_at);
                            we[h][0] = ve.x, we[h][1] = ve.y;
                            wo[h][0] = vo.x, wo[h][1] = vo.y;
                        } else if constexpr (kThree) {
#pragma unroll
                            for (int k = 0; k < kQuads; ++k) {
                                we[h][k] = *reinterpret_cast<const uint16_t *>(at + ve_at + 16 * k);
                                wo[h][k] = *reinterpret_cast<const uint16_t *>(at + vo_at + 16 * k);
                            }
                        } else {
                            we[h][0] = *reinterpret_cast<const uint32_t *>(at + ve_at);
                            wo[h][0] = *reinterpret_cast<const uint32_t *>(at + vo_at);
                        }
                        if (!kThree) v_scales(h, 0);
                    }
#pragma unroll
                    for (int k = 0; k < kQuads; ++k) {
                        // four channels (quad k of the lane's) of two keys
                        const int word = kThree ? k : k / 2;
                        const uint32_t pick = !kThree && k % 2 ? 0x7632 : 0x5410;
                        if (kThree) v_scales(0, k), v_scales(1, k);
                        uint32_t a0[4], a1[4];
                        values<T>(__byte_perm(we[0][word], wo[0][word], pick), vs[0], vb[0], masks, a0);
                        values<T>(__byte_perm(we[1][word], wo[1][word], pick), vs[1], vb[1], masks, a1);
#pragma unroll
                        for (int n = 0; n < N; ++n) {
                            mma16816<T>(o[n][2 * k], a0[0], a0[1], a1[0], a1[1], pb[n][x][0], pb[n][x][1]);
                            mma16816<T>(o[n][2 * k + 1], a0[2], a0[3], a1[2], a1[3], pb[n][x][0], pb[n][x][1]);
                        }
                    }
                }
            }
            __syncwarp();                        // every lane has read the stage
        }
        if constexpr (!kRun) cp_wait<0>();
        __syncwarp();

        // join the warps: O of each into its own ring, then all threads sum
        float *mine_o = reinterpret_cast<float *>(ring);
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = l[n][e];
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                const int row = 8 * n + 2 * t4 + e;
                if (g == 0) sml[warp][row] = make_float2(m[n][e], sum);
#pragma unroll
                for (int d = 0; d < kTiles; ++d)
                    *reinterpret_cast<float2 *>(mine_o + row * kPad + (kThree ? d / 2 * 32 + g * 4 + d % 2 * 2 : g * (HD / 8) + 2 * d)) = make_float2(o[n][d][e], o[n][d][2 + e]);
            }
        __syncthreads();
        if (threadIdx.x < 8 * N) {
            const int row = threadIdx.x;
            float M = -INFINITY, L = 0.f;
            for (int w2 = 0; w2 < kWarps; ++w2) M = fmaxf(M, sml[w2][row].x);
            for (int w2 = 0; w2 < kWarps; ++w2) {
                const float f = sml[w2][row].x == -INFINITY ? 0.f : ex2(sml[w2][row].x - M);
                swt[w2][row] = f;
                L = fmaf(sml[w2][row].y, f, L);
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
            for (int w2 = 0; w2 < kWarps; ++w2) {
                const float f = swt[w2][row];
                const float4 v = *reinterpret_cast<const float4 *>(reinterpret_cast<float *>(smem + w2 * S::kRing) + row * kPad + c4);
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
        if constexpr (kRun) fence_proxy_async_smem();
        __syncthreads();                         // the rings are free for the next tile
    };

    for (int tile = tile0; tile < ntiles; tile += tiles_y) {
        int row0, nrows;
        if constexpr (kRun) {
            row0 = tile * kRows;
            nrows = min(kRows, q.m * p.group - row0);
        } else {
            const int part = tile % per_tok;
            row0 = tile / per_tok * p.group + part * kRows;
            nrows = min(kRows, p.group - part * kRows);
        }
        if (kN == 1 || nrows <= 8) run(std::integral_constant<int, 1>{}, row0, nrows);
        else run(std::integral_constant<int, kN>{}, row0, nrows);
    }
}

// ---------------------------------------------------------------------------
// every type and head size
// ---------------------------------------------------------------------------
constexpr int kThreadsG = 128;

// The eight codes of a word less 8, exact: behind the exponent of 2^23 by one
// operation (its second constant held in a register), and 2^23 + 8 taken off.
__device__ __forceinline__ void codes_of(uint32_t w, uint32_t magic, float (&f)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        uint32_t x;
        asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(x) : "r"(w >> (4 * e)), "r"(15u), "r"(magic));
        f[e] = __uint_as_float(x) - 8388616.f;
    }
}

// A key belongs to a group of kLanes lanes, 8 channels (a word of codes) a lane;
// kThreadsG / kLanes keys at a time.  A block answers kR query heads that share the
// key head, so a key is loaded and unpacked once for them.  The channels of a
// word share a scale: it multiplies the word's sum in K, and the weight in V.  Bound by
// instructions: 16 requests of 3000 to 5000, 12 heads of 64, fp32: 50 us, 1.2 TB/s (with
// every value scaled by itself 56); 32 heads over 8 of 128, 10000 to 20000: 382 us.
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
    uint32_t magic;
    asm volatile("mov.b32 %0, 0x4b000000;" : "=r"(magic));
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
                codes_of(kw[i], magic, kf);
#pragma unroll
                for (int t = 0; t < kR; ++t) {
                    x[t][i] = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[t][i] = fmaf(qf[t][e], kf[e], x[t][i]);
                    x[t][i] *= ks[i];
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
                codes_of(vw[i], magic, vf);
#pragma unroll
                for (int t = 0; t < kR; ++t) {
                    const float weight = x[t][i] * vs[i];
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[t][e] = fmaf(weight, vf[e], o[t][e]);
                }
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
    auto fn = &k_decode4_rows<T, HD, kN, kWarps, true>;
    if constexpr (HD != 96)
        if (a.stride > 1) fn = &k_decode4_rows<T, HD, kN, kWarps, false>;
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
    auto launch = [&](auto of) {
        using T = decltype(of);
        return a.hd == 64 ? launch_hd<T, 64>(a, st) : a.hd == 96 ? launch_hd<T, 96>(a, st) : launch_hd<T, 128>(a, st);
    };
    return dt == kF16 ? launch(__half()) : launch(__nv_bfloat16());
}
cudaError_t launch_decode4_general(DType dt, const DecodeArgs &a, cudaStream_t st) {
    return dt == kF32 ? launch_general_t<float>(a, st) : dt == kF16 ? launch_general_t<__half>(a, st) : launch_general_t<__nv_bfloat16>(a, st);
}

}  // namespace swab
