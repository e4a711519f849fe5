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
// than 32 lanes hold, go a warp a row through shared memory.
//
// A warp takes a token at a time (or a slice of its heads, where there are fewer
// tokens than warps): it makes the token's cosines and sines once, each lane keeps those
// of its pairs in registers for all the heads, and rows are loaded some
// steps ahead, across tokens.  No block-wide barrier, no list of rows.  (With a block a
// tile of tokens, rows listed and tables in shared memory, the gradient of 12 x 1365
// tokens took 48 us: every tile waited for its list, its table and its first rows.)
//
// 4 bits.  A group of 32 channels is four pieces of 16-bit values, on four adjacent lanes
// where the pairs of the rotation leave it so: the value of largest magnitude is a
// maximum over the integers (bits << 1 | sign positive), two shuffles; the quotient x / s is decided exactly: the values have at
// most 11 significant bits and s 5, so a quotient that is no tie is 2^-13 off one,
// and fma(x, 1 / s, 768) rounds it to a multiple of 2^-14 before it is rounded to
// a whole number.
//
// Backward.  g = R^T dy, dx_c = r (g_c v_c - x_c r^2 mean(g v x)): two sums a row,
// one pass over x and dy.  dw_c = sum over rows of g_c x_c r: a lane adds up its
// channels over all its rows, a block writes one row of sums, a second kernel adds
// the blocks' in a fixed order.
//
// Every value is read once and written once.  Neither memory (27 to 47 % of its rate in
// ncu) nor issue slots (51 to 66 %) are full: what bounds the calls is how much is in flight,
// and that is what registers hold, 12 to 20 warps an SM with one or two row groups
// each (more warps, or more rows ahead in registers, were slower: 2 rows ahead 38 us for
// the prompt, 4 ahead 46, addresses that step by additions 34).
// Measured: a prompt of 8192 tokens, 32 + 8 heads of 128, bf16: 34 us, 4.9 TB/s (the same
// without the norms 28), fp32 62 us, 5.4 TB/s; prompts of 8.9k tokens, 12 + 12 + 12 heads of
// 64, fp16, into the cache 20 us, 4.1 TB/s; of 32 + 8 + 8 heads of 128, bf16, into a cache
// in 4 bits 48 us, 4.0 TB/s (fp32, a warp a row, 278 us, 1.4 TB/s); the gradient of 12 x
// 1365 tokens, 24 heads of 64, fp16, with both weights' 39 us, 3.9 TB/s (Q and K in blocks
// of their own 45 to 48), of 8192 tokens, 32 + 8 heads of 128, bf16, 57 us, 4.4 TB/s.
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
// Two fp32 at a time (fma.rn.f32x2 and its kin): the rows are bound by instructions
// before they are by memory where each value is handled alone.
template <typename T> __device__ __forceinline__ void unpack2(const uint4 &v, uint64_t (&f)[VecOf<T>::kN / 2]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (sizeof(T) == 4) {
        f[0] = f2(__uint_as_float(w[0]), __uint_as_float(w[1]));
        f[1] = f2(__uint_as_float(w[2]), __uint_as_float(w[3]));
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = f2(lo16<T>(w[k]), hi16<T>(w[k]));
    }
}
template <typename T> __device__ __forceinline__ uint4 repack2(const uint64_t (&f)[VecOf<T>::kN / 2]) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < VecOf<T>::kN / 2; ++k) {
        float lo, hi;
        f2split(f[k], lo, hi);
        if constexpr (sizeof(T) == 4) w[2 * k] = __float_as_uint(lo), w[2 * k + 1] = __float_as_uint(hi);
        else w[k] = pack2<T>(lo, hi);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// N pairs from shared memory
template <int N> __device__ __forceinline__ void take2(const float *src, uint64_t (&f)[N]) {
    if constexpr (N % 2 == 0) {
#pragma unroll
        for (int k = 0; k < N; k += 2) {
            const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(src + 2 * k);
            f[k] = v.x, f[k + 1] = v.y;
        }
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k) f[k] = *reinterpret_cast<const unsigned long long *>(src + 2 * k);
    }
}
__device__ __forceinline__ uint64_t negate2(uint64_t x) { return x ^ 0x8000000080000000ull; }
__device__ __forceinline__ float sum2(uint64_t x) {
    float lo, hi;
    f2split(x, lo, hi);
    return lo + hi;
}

// The largest rank of a lane's eight 16-bit values (already rounded), in 16 bits, two
// values at a time.
__device__ __forceinline__ uint32_t rank8(const uint4 &y) {
    const uint32_t w[4] = {y.x, y.y, y.z, y.w};
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) top = __vmaxu2(top, ((w[k] << 1) & 0xfffefffeu) | ((~w[k] >> 15) & 0x00010001u));
    return max(top & 0xffffu, top >> 16);
}
// The ranks of the groups that a lane's two pieces belong to.  kAdjacent: four adjacent
// lanes hold a group.  Else a row's groups, four at most, lie over its `lanes` lanes as
// the pairs of the rotation want it: every lane puts what it has in its groups' places
// of two words, whose maxima all take (8.9k tokens of 32 + 8 + 8 heads of 96 with their
// reading back 61 us, a warp a row 221; of 128, a quarter turned, 67 and 254).
template <bool kAdjacent>
__device__ __forceinline__ void group_ranks(uint32_t &ra, uint32_t &rb, int pa, int pb, int lanes) {
    if constexpr (kAdjacent) {
#pragma unroll
        for (int d = 1; d <= 2; d <<= 1) {
            ra = max(ra, __shfl_xor_sync(0xffffffffu, ra, d));
            rb = max(rb, __shfl_xor_sync(0xffffffffu, rb, d));
        }
    } else {
        const int sa = pa / 4 * 16 & 16, sb = pb / 4 * 16 & 16;
        const bool ha = pa >= 8, hb = pb >= 8;
        uint32_t lo = __vmaxu2(ha ? 0u : ra << sa, hb ? 0u : rb << sb), hi = __vmaxu2(ha ? ra << sa : 0u, hb ? rb << sb : 0u);
        for (int d = 1; d < lanes; d <<= 1) {
            lo = __vmaxu2(lo, __shfl_xor_sync(0xffffffffu, lo, d));
            hi = __vmaxu2(hi, __shfl_xor_sync(0xffffffffu, hi, d));
        }
        ra = (ha ? hi : lo) >> sa & 0xffffu;
        rb = (hb ? hi : lo) >> sb & 0xffffu;
    }
}
// The eight codes of a piece, and the scale of its group from the group's rank.  A
// quotient is rounded to a multiple of 2^-14 by the fma and to the nearest whole
// number, plus 8, by the addition (12582920 = 1.5 * 2^23 + 8, even as 8 is, so that ties
// stay with the even quotient).
template <typename T>
__device__ __forceinline__ uint32_t quantise8(const uint4 &y, uint32_t rank, float &s) {
    s = scale_of<T>((__float_as_uint(lo16<T>(rank >> 1)) << 1) | (rank & 1u));
    const bool none = !(fabsf(s) > 0.f);                             // 0 or NaN
    const float inv = none ? 0.f : __frcp_rn(s);
    const uint64_t by = f2(inv, inv), far = f2(768.f, 768.f), near = f2(12582920.f - 768.f, 12582920.f - 768.f);
    uint64_t x[4];
    unpack2<T>(y, x);
    uint32_t u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float lo, hi;
        f2split(add2(fma2(x[k], by, far), near), lo, hi);
        const uint32_t n = __vimin_s16x2_relu(__byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x5410), 0x000f000fu);   // into 0..15
        u[k] = n | n >> 12;
    }
    const uint32_t codes = __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
    return none ? 0x88888888u : codes;
}

// 1 / sqrt(mean of squares + eps), within 2 ulp
__device__ __forceinline__ float inverse_norm(float sum, float by_hd, float eps) { return rsqrtf(__fmaf_rn(sum, by_hd, eps)); }

// r^2 mean(g v x) of the gradient.  Where the squares pass fp32's range r is 0, and so
// is all of the row: the products may have passed it too, and infinity times 0 is NaN.
__device__ __forceinline__ float mean_part(float dot, float by_hd, float rn) { return rn == 0.f ? 0.f : dot * by_hd * rn * rn; }

// A pair turned, rounded as k_rotary does (so that the cache holds the same bits
// with and without norms, in either width): pieces, and pair by pair.
__device__ __forceinline__ void turn(float &a, float &b, float c, float s, bool by_pairs = false) {
    const float x = a;
    a = __fmaf_rn(x, c, -__fmul_rn(b, s));
    b = by_pairs ? __fmaf_rn(b, c, __fmul_rn(x, s)) : __fmaf_rn(x, s, __fmul_rn(b, c));
}
// the same for two pairs (pieces)
__device__ __forceinline__ void turn2(uint64_t &a, uint64_t &b, uint64_t c, uint64_t s) {
    const uint64_t x = a;
    a = fma2(x, c, negate2(mul2(b, s)));
    b = fma2(x, s, mul2(b, c));
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
// Rows on lane groups: kInter: adjacent pairs in 16-byte pieces, else halves.  kKind: 0
// = Q, K -> Qo, Ko; 1 = into the cache; 2 = into the cache in 4 bits (16-bit types,
// groups on four adjacent lanes), 3 = the same with groups anywhere in the row.
constexpr int kWarps = 4;
constexpr int kAhead = 2;            // rows of a lane group loaded ahead

// This lane's two pieces of a row, and its place in the row group.
struct Lane {
    int sub, row, pa, pb;
    bool active, turns;
};
template <bool kInter> __device__ __forceinline__ Lane lane_of(int lanes, int pieces, int turning) {
    const int lane = threadIdx.x & 31, nturn = kInter ? 0 : turning;
    Lane l;
    l.sub = lane & (lanes - 1);
    l.row = lane / lanes;
    l.active = l.sub < pieces / 2;
    l.pa = l.sub < nturn ? l.sub : nturn + l.sub;
    l.pb = l.sub < nturn ? l.sub + nturn : pieces / 2 + l.sub;
    l.turns = l.active && (kInter || l.sub < nturn);
    return l;
}
// A token's cosines and sines by the warp, then those of this lane's pairs: c, s.
template <typename T, bool kInter>
__device__ __forceinline__ void token_turns(const RotaryArgs &p, const Lane &l, long long at, const unsigned long long *turns, float *cs,
                                            uint64_t (&c)[VecOf<T>::kN / 2], uint64_t (&s)[VecOf<T>::kN / 2]) {
    constexpr int kV = VecOf<T>::kN, kH = kV / 2;
    const int half = p.rot / 2;
    __syncwarp();                        // (the token before is done with the table)
    for (int k = threadIdx.x & 31; k < half; k += 32) {
        float x, y;
        cos_sin(at, turns[k], x, y);
        cs[k] = x * p.scale;
        cs[half + k] = y * p.scale;
    }
    __syncwarp();
    if (!l.turns) return;
    if constexpr (kInter) {
        // kH pairs of either piece
        uint64_t *to[2] = {c, s};
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int k = 0; k < kH / 2; ++k) {
                if (l.pa * kV < p.rot) to[w][k] = *reinterpret_cast<const unsigned long long *>(cs + w * half + l.pa * kH + 2 * k);
                if (l.pb * kV < p.rot) to[w][kH / 2 + k] = *reinterpret_cast<const unsigned long long *>(cs + w * half + l.pb * kH + 2 * k);
            }
    } else {
        take2<kH>(cs + l.pa * kV, c);
        take2<kH>(cs + half + l.pa * kV, s);
    }
}
// Position of token t.
__device__ __forceinline__ long long position_of(const RotaryArgs &p, unsigned t) {
    return (p.pos ? (long long)*GP(p.bnd, p.pos + t) : (long long)(t % p.n)) + p.pos0;
}
// x / d for x < 2^31: by = (2^32 - 1) / d gives it or one less.
__device__ __forceinline__ unsigned divide(unsigned x, unsigned d, unsigned by) {
    const unsigned q = __umulhi(x, by);
    return x - q * d >= d ? q + 1u : q;
}
// Token t of sequence bb, its i-th; where it lies in a tensor, in units of 16 bytes.
struct Token {
    unsigned bb, i;
    __device__ __forceinline__ unsigned units(const unsigned *s) const { return bb * s[0] + i * s[1]; }
};
// Unit u of the work: slice `slice` of the rows of a token.
struct Unit {
    unsigned t, slice;
};
__device__ __forceinline__ Unit unit_of(unsigned u, unsigned split, unsigned by_split) {
    if (split == 1) return Unit{u, 0u};
    const unsigned t = divide(u, split, by_split);
    return Unit{t, u - t * split};
}
__device__ __forceinline__ Token token_of(const RotaryArgs &p, unsigned t, unsigned by_n) {
    if (p.n == p.tokens) return Token{0u, t};
    const unsigned bb = divide(t, p.n, by_n);
    return Token{bb, t - bb * p.n};
}

template <typename T, bool kInter, int kKind>
__global__ void __launch_bounds__(32 * kWarps, 5) k_norm(const __grid_constant__ NormArgs a) {
    constexpr int kV = VecOf<T>::kN, kH = kV / 2;
    constexpr unsigned kNever = 0xffffffffu;
    const RotaryArgs &p = a.r;
    extern __shared__ __align__(16) float smem[];      // turns [rot / 2]; weights [2][hd]; [rot] a warp
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, L = a.lanes, pad = (p.rot + 3) / 4 * 4;
    const unsigned group = 32 / L, hq = p.hq, hqk = p.hq + p.hk, rows = p.rows;
    unsigned long long *turns = reinterpret_cast<unsigned long long *>(smem);
    float *wtab = smem + pad, *cs = wtab + 2 * p.hd + warp * pad;
    const Lane l = lane_of<kInter>(L, p.hd / kV, p.rot / 2 / kV);
    const float by_hd = 1.f / (float)p.hd;
    // units of work: the `its` row groups of slice u % split of token u / split
    const unsigned split = a.split, its = a.its, units = p.tokens * split, step = gridDim.x * kWarps;
    const unsigned by_split = 0xffffffffu / split, by_n = 0xffffffffu / p.n;
    unsigned u = blockIdx.x * kWarps + warp;

    // A lane's row e of a token moves on by a row group at a time: its address by a
    // fixed step until it passes `bound`, into the heads of the next tensor.
    // The loads run kAhead row groups ahead: row le at `from`.
    unsigned lu = u, li = 0, le = 0, lbound = 0, lstep = 0;
    const char *from = nullptr;
    Token ltok{0, 0};
    auto aim_row = [&]() {
        const bool is_q = le < hq, is_v = kKind > 0 && le >= hqk;
        const unsigned *s = is_q ? p.sq : is_v ? p.sv : p.sk;
        const unsigned at = ltok.units(s) + (is_q ? le : is_v ? le - hqk : le - hq) * s[2];
        from = (const char *)(is_q ? p.Q : is_v ? p.V : p.K) + (unsigned long long)at * 16u;
        lstep = s[2] * group;
        lbound = le >= rows || !l.active ? 0 : is_q ? hq : is_v || kKind == 0 ? rows : hqk;     // 0: no row
    };
    auto aim = [&]() {                                 // the loads at unit lu
        lbound = 0;
        if (lu >= units) return;
        const Unit x = unit_of(lu, split, by_split);
        ltok = token_of(p, x.t, by_n);
        le = x.slice * its * group + l.row;
        aim_row();
    };
    auto load = [&](uint4 &va, uint4 &vb) {
        va = vb = make_uint4(0, 0, 0, 0);
        if (lbound) {
            va = load16(GPN(p.bnd, from + l.pa * 16, 16));
            vb = load16(GPN(p.bnd, from + l.pb * 16, 16));
            le += group;
            from += (unsigned long long)lstep * 16u;
            if (le >= lbound) aim_row();
        }
        if (++li == its) {
            li = 0;
            lu += step;
            aim();
        }
    };

    pdl_wait();
    pdl_trigger();
    uint4 va[kAhead], vb[kAhead];
    aim();
#pragma unroll
    for (int k = 0; k < kAhead; ++k) load(va[k], vb[k]);
    Unit now = unit_of(u, split, by_split);
    long long at = u < units ? position_of(p, now.t) : 0;
    int slot = kKind > 0 && u < units ? *GP(p.bnd, p.slots + now.t) : -1;
    for (int k = threadIdx.x; k < p.rot / 2; k += 32 * kWarps) turns[k] = *GP(p.bnd, p.turns + k);
    for (int c = threadIdx.x; c < 2 * p.hd; c += 32 * kWarps) {
        const T *w = reinterpret_cast<const T *>(c < p.hd ? a.wq : a.wk);
        wtab[c] = w ? Elt<T>::to_f(*GP(p.bnd, w + (c < p.hd ? c : c - p.hd))) + a.offset : 1.f;
    }
    __syncthreads();

    for (; u < units; u += step) {
        const Token tok = token_of(p, now.t, by_n);
        unsigned e = now.slice * its * group + l.row;
        uint64_t c[kH], s[kH];
        token_turns<T, kInter>(p, l, at, turns, cs, c, s);
        const int here = slot;
        if (u + step < units) {
            now = unit_of(u + step, split, by_split);
            at = position_of(p, now.t);
            if (kKind > 0) slot = *GP(p.bnd, p.slots + now.t);
        }
        const bool kept = kKind == 0 || (here >= 0 && here < p.n_slots);
        if (kKind > 0 && !kept && here != -1 && lane == 0) atomicOr(p.err, kErrInvalid);

        // the same for what is written: row e to `dst` (4 bits: its codes), scales to `sc`
        unsigned bound = 0;
        char *dst = nullptr;
        unsigned long long dstep = 0;
        T *sc = nullptr;
        auto aim_out = [&]() {
            bound = kNever;                            // (rows past the last one move nowhere)
            if (e >= rows) return;
            const bool is_q = e < hq, is_v = kKind > 0 && e >= hqk;
            bound = is_q ? hq : is_v || kKind == 0 ? rows : hqk;
            if (is_q || kKind == 0) {
                const unsigned *so = is_q ? p.sqo : p.sko;
                dst = (char *)(is_q ? p.Qo : p.Ko) + (unsigned long long)(tok.units(so) + (is_q ? e : e - hq) * so[2]) * 16u;
                dstep = (unsigned long long)(so[2] * group) * 16u;
            } else {
                const unsigned blk = (unsigned)here >> p.page_log2, off = (unsigned)here & ((1u << p.page_log2) - 1u), head = e - (is_v ? hqk : hq);
                const unsigned long long line = ((blk * (unsigned)p.hk + head) << p.page_log2) + off;     // below 2^32
                const unsigned width = kKind >= 2 ? p.hd / 2 : p.row_bytes;
                dst = (char *)(is_v ? p.Vc : p.Kc) + line * width;
                dstep = (unsigned long long)(group << p.page_log2) * width;
                if (kKind >= 2) sc = (T *)(is_v ? a.Vs : a.Ks) + line * (p.hd / kGroup4);
            }
        };
        aim_out();

        for (unsigned i = 0; i < its; ++i) {
            const bool there = e < rows && l.active, is_q = e < hq, as_is = kKind > 0 && e >= hqk;
            const uint4 xa = va[0], xb = vb[0];
#pragma unroll
            for (int m = 0; m + 1 < kAhead; ++m) va[m] = va[m + 1], vb[m] = vb[m + 1];
            load(va[kAhead - 1], vb[kAhead - 1]);
            uint64_t fa[kH], fb[kH];
            unpack2<T>(xa, fa);
            unpack2<T>(xb, fb);
            if (a.norm) {
                uint64_t squares = 0;
#pragma unroll
                for (int m = 0; m < kH; ++m) squares = fma2(fa[m], fa[m], fma2(fb[m], fb[m], squares));
                float sum = sum2(squares);
                for (int d = L / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                if (!as_is && l.active) {
                    const float rn = inverse_norm(sum, by_hd, a.eps);
                    const uint64_t rn2 = f2(rn, rn);
                    const float *w = wtab + (is_q ? 0 : p.hd);
                    uint64_t v[kH];
                    take2<kH>(w + l.pa * kV, v);
#pragma unroll
                    for (int m = 0; m < kH; ++m) fa[m] = mul2(fa[m], mul2(rn2, v[m]));
                    take2<kH>(w + l.pb * kV, v);
#pragma unroll
                    for (int m = 0; m < kH; ++m) fb[m] = mul2(fb[m], mul2(rn2, v[m]));
                }
            }
            if (l.turns && !as_is) {
                if constexpr (kInter) {
                    auto turn_piece = [&](uint64_t (&f)[kH], int piece, int first) {
                        if (piece * kV >= p.rot) return;
#pragma unroll
                        for (int m = 0; m < kH; ++m) {
                            float x, y, c0, c1, s0, s1;
                            f2split(f[m], x, y);
                            f2split(c[first + m / 2], c0, c1);
                            f2split(s[first + m / 2], s0, s1);
                            turn(x, y, m & 1 ? c1 : c0, m & 1 ? s1 : s0);
                            f[m] = f2(x, y);
                        }
                    };
                    turn_piece(fa, l.pa, 0);
                    turn_piece(fb, l.pb, kH / 2);
                } else {
#pragma unroll
                    for (int m = 0; m < kH; ++m) turn2(fa[m], fb[m], c[m], s[m]);
                }
            }
            const uint4 ya = as_is ? xa : repack2<T>(fa), yb = as_is ? xb : repack2<T>(fb);
            bool whole = there && (is_q || kept);      // a row of the tensors' type to write
            if constexpr (kKind >= 2 && sizeof(T) == 2) {
                if (__any_sync(0xffffffffu, there && !is_q)) {
                    float s0, s1;                      // (ya, yb: as the cache of this type would hold them)
                    uint32_t ra = l.active ? rank8(ya) : 0u, rb = l.active ? rank8(yb) : 0u;
                    group_ranks<kKind == 2>(ra, rb, l.pa, l.pb, L);
                    const uint32_t wa = quantise8<T>(ya, ra, s0), wb = quantise8<T>(yb, rb, s1);
                    if (there && !is_q && kept) {
                        *reinterpret_cast<uint32_t *>(GPN(p.bnd, dst + l.pa * 4, 4)) = wa;
                        *reinterpret_cast<uint32_t *>(GPN(p.bnd, dst + l.pb * 4, 4)) = wb;
                        if ((l.pa & 3) == 0) *GP(p.bnd, sc + l.pa / 4) = Elt<T>::from_f(s0);
                        if ((l.pb & 3) == 0) *GP(p.bnd, sc + l.pb / 4) = Elt<T>::from_f(s1);
                    }
                    sc += (unsigned long long)(group << p.page_log2) * (p.hd / kGroup4);
                }
                whole = there && is_q;
            }
            if (whole) {
                *reinterpret_cast<uint4 *>(GPN(p.bnd, dst + l.pa * 16, 16)) = ya;
                *reinterpret_cast<uint4 *>(GPN(p.bnd, dst + l.pb * 16, 16)) = yb;
            }
            e += group;
            dst += dstep;
            if (e >= bound) aim_out();
        }
    }
}

// The rows that do not lie on lane groups: a warp a row, through shared memory.  A block
// takes a few tokens at a time: it lists their rows and fills a table of cosines and
// sines shared by all the heads, one buffer ahead.
template <typename T, int kKind>
__global__ void __launch_bounds__(kThreads, kBlocks) k_norm_rows(const __grid_constant__ NormArgs a) {
    constexpr int kV = VecOf<T>::kN;
    const RotaryArgs &p = a.r;
    const float by_hd = 1.f / (float)p.hd;
    extern __shared__ __align__(16) float smem[];      // two tables [tile][2][rot / 2]; weights [2][hd]; a row a warp
    __shared__ Row lists[2][kMaxRows];
    const int half = p.rot / 2;
    float *wtab = smem + 2 * p.tile * p.rot;
    const int lo = (int)((long long)p.rows * blockIdx.y / gridDim.y), mine = (int)((long long)p.rows * (blockIdx.y + 1) / gridDim.y) - lo;
    const unsigned by_mine = 0xffffffffu / mine + 1u, by_half = half > 1 ? 0xffffffffu / half + 1u : 0u;   // x / mine, x / half for x < 2^15

    const int pieces = p.hd / kV, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float *x = wtab + 2 * p.hd + warp * p.hd;

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
        if (t0 + step < p.tokens) prepare(t0 + step, lists[buf ^ 1], smem + (buf ^ 1) * p.tile * p.rot);
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
                        if (lane < pieces / 2) {
                            float odd = 0.f;
                            for (int k = 0; k < kV; k += 2) {
                                const float *xa = x + la * kV + k, *xb = x + lb * kV + k;
                                sum = __fmaf_rn(xa[0], xa[0], __fmaf_rn(xb[0], xb[0], sum));
                                odd = __fmaf_rn(xa[1], xa[1], __fmaf_rn(xb[1], xb[1], odd));
                            }
                            sum += odd;
                        }
                        for (int d = a.sum_lanes / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                        sum = __shfl_sync(0xffffffffu, sum, 0);
                    } else {
                        for (int c = lane; c < p.hd; c += 32) sum = fmaf(x[c], x[c], sum);
#pragma unroll
                        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                    }
                    __syncwarp();
                    const float rn = inverse_norm(sum, by_hd, a.eps);
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

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// One row group is loaded ahead; a lane adds up both weights' gradients.
template <typename T, bool kInter>
__global__ void __launch_bounds__(32 * kWarps, 3) k_norm_bwd(const __grid_constant__ NormArgs a) {
    constexpr int kV = VecOf<T>::kN, kH = kV / 2;
    constexpr unsigned kNever = 0xffffffffu;
    const RotaryArgs &p = a.r;
    extern __shared__ __align__(16) float smem[];      // turns [rot / 2]; [rot] a warp; weights [2][hd]; sums [32 kWarps / lanes][hd]
    const int warp = threadIdx.x >> 5, L = a.lanes, pad = (p.rot + 3) / 4 * 4;
    const unsigned group = 32 / L, hq = p.hq, rows = p.rows;
    unsigned long long *turns = reinterpret_cast<unsigned long long *>(smem);
    float *cs = smem + pad + warp * pad, *wtab = smem + pad + kWarps * pad, *sums = wtab + 2 * p.hd;
    const Lane l = lane_of<kInter>(L, p.hd / kV, p.rot / 2 / kV);
    const float by_hd = 1.f / (float)p.hd;
    const unsigned split = a.split, its = a.its, units = p.tokens * split, step = gridDim.x * kWarps;
    const unsigned by_split = 0xffffffffu / split, by_n = 0xffffffffu / p.n;
    unsigned u = blockIdx.x * kWarps + warp;

    // the loads, a row group ahead: row le at from_x, from_g (as in k_norm)
    unsigned lu = u, li = 0, le = 0, lbound = 0, step_x = 0, step_g = 0;
    const char *from_x = nullptr, *from_g = nullptr;
    Token ltok{0, 0};
    auto aim_row = [&]() {
        const bool is_q = le < hq;
        const unsigned *sx = a.sx[is_q ? 0 : 1], *sg = is_q ? p.sq : p.sk, head = is_q ? le : le - hq;
        from_x = (const char *)a.X[is_q ? 0 : 1] + (unsigned long long)(ltok.units(sx) + head * sx[2]) * 16u;
        from_g = (const char *)(is_q ? p.Q : p.K) + (unsigned long long)(ltok.units(sg) + head * sg[2]) * 16u;
        step_x = sx[2] * group;
        step_g = sg[2] * group;
        lbound = le >= rows || !l.active ? 0 : is_q ? hq : rows;               // 0: no row
    };
    auto aim = [&]() {
        lbound = 0;
        if (lu >= units) return;
        const Unit x = unit_of(lu, split, by_split);
        ltok = token_of(p, x.t, by_n);
        le = x.slice * its * group + l.row;
        aim_row();
    };
    uint4 rxa, rxb, rga, rgb;
    auto load = [&]() {
        rxa = rxb = rga = rgb = make_uint4(0, 0, 0, 0);
        if (lbound) {
            rxa = load16(GPN(p.bnd, from_x + l.pa * 16, 16));
            rxb = load16(GPN(p.bnd, from_x + l.pb * 16, 16));
            rga = load16(GPN(p.bnd, from_g + l.pa * 16, 16));
            rgb = load16(GPN(p.bnd, from_g + l.pb * 16, 16));
            le += group;
            from_x += (unsigned long long)step_x * 16u;
            from_g += (unsigned long long)step_g * 16u;
            if (le >= lbound) aim_row();
        }
        if (++li == its) {
            li = 0;
            lu += step;
            aim();
        }
    };

    pdl_wait();
    pdl_trigger();
    aim();
    load();
    Unit now = unit_of(u, split, by_split);
    long long at = u < units ? position_of(p, now.t) : 0;
    for (int k = threadIdx.x; k < p.rot / 2; k += 32 * kWarps) turns[k] = *GP(p.bnd, p.turns + k);
    for (int c = threadIdx.x; c < 2 * p.hd; c += 32 * kWarps) {
        const T *w = reinterpret_cast<const T *>(c < p.hd ? a.wq : a.wk);
        wtab[c] = w ? Elt<T>::to_f(*GP(p.bnd, w + (c < p.hd ? c : c - p.hd))) + a.offset : 1.f;
    }
    uint64_t dqa[kH], dqb[kH], dka[kH], dkb[kH];       // this lane's share of dwq, dwk
#pragma unroll
    for (int k = 0; k < kH; ++k) dqa[k] = dqb[k] = dka[k] = dkb[k] = 0;
    __syncthreads();

    for (; u < units; u += step) {
        const Token tok = token_of(p, now.t, by_n);
        unsigned e = now.slice * its * group + l.row;
        uint64_t c[kH], s[kH];
        token_turns<T, kInter>(p, l, at, turns, cs, c, s);
        if (u + step < units) {
            now = unit_of(u + step, split, by_split);
            at = position_of(p, now.t);
        }
        unsigned bound = 0, dstep = 0;
        char *dst = nullptr;
        auto aim_out = [&]() {
            bound = kNever;
            if (e >= rows) return;
            const bool is_q = e < hq;
            const unsigned *so = is_q ? p.sqo : p.sko;
            bound = is_q ? hq : rows;
            dst = (char *)(is_q ? p.Qo : p.Ko) + (unsigned long long)(tok.units(so) + (is_q ? e : e - hq) * so[2]) * 16u;
            dstep = so[2] * group;
        };
        aim_out();
        for (unsigned i = 0; i < its; ++i) {
            const bool there = e < rows && l.active, is_q = e < hq;
            uint64_t fa[kH], fb[kH], ya[kH], yb[kH], va[kH], vb[kH];
            unpack2<T>(rxa, fa);
            unpack2<T>(rxb, fb);
            unpack2<T>(rga, ya);
            unpack2<T>(rgb, yb);
            load();
            if (l.turns) {                             // R^T
                if constexpr (kInter) {
                    auto turn_back = [&](uint64_t (&f)[kH], int piece, int first) {
                        if (piece * kV >= p.rot) return;
#pragma unroll
                        for (int m = 0; m < kH; ++m) {
                            float x, y, c0, c1, s0, s1;
                            f2split(f[m], x, y);
                            f2split(c[first + m / 2], c0, c1);
                            f2split(s[first + m / 2], s0, s1);
                            const float co = m & 1 ? c1 : c0, si = m & 1 ? s1 : s0;
                            f[m] = f2(x * co + y * si, y * co - x * si);
                        }
                    };
                    turn_back(ya, l.pa, 0);
                    turn_back(yb, l.pb, kH / 2);
                } else {
#pragma unroll
                    for (int m = 0; m < kH; ++m) {
                        const uint64_t x = ya[m];
                        ya[m] = fma2(x, c[m], mul2(yb[m], s[m]));
                        yb[m] = fma2(yb[m], c[m], negate2(mul2(x, s[m])));
                    }
                }
            }
            uint64_t squares = 0, products = 0;
            if (l.active) {
                take2<kH>(wtab + (is_q ? 0 : p.hd) + l.pa * kV, va);
                take2<kH>(wtab + (is_q ? 0 : p.hd) + l.pb * kV, vb);
            } else {
#pragma unroll
                for (int m = 0; m < kH; ++m) va[m] = vb[m] = 0;
            }
#pragma unroll
            for (int m = 0; m < kH; ++m) {
                squares = fma2(fa[m], fa[m], fma2(fb[m], fb[m], squares));
                va[m] = mul2(va[m], ya[m]);
                vb[m] = mul2(vb[m], yb[m]);
                products = fma2(va[m], fa[m], fma2(vb[m], fb[m], products));
            }
            float sum = sum2(squares), dot = sum2(products);
            for (int d = L / 2; d > 0; d >>= 1) {
                sum += __shfl_xor_sync(0xffffffffu, sum, d);
                dot += __shfl_xor_sync(0xffffffffu, dot, d);
            }
            if (there) {
                const float rn = inverse_norm(sum, by_hd, a.eps), c2 = mean_part(dot, by_hd, rn);
                const uint64_t rn2 = f2(rn, rn), less = f2(-c2, -c2);
#pragma unroll
                for (int m = 0; m < kH; ++m) {
                    ya[m] = mul2(ya[m], mul2(fa[m], rn2));             // this row's term of dw
                    yb[m] = mul2(yb[m], mul2(fb[m], rn2));
                    fa[m] = mul2(rn2, fma2(less, fa[m], va[m]));
                    fb[m] = mul2(rn2, fma2(less, fb[m], vb[m]));
                }
                *reinterpret_cast<uint4 *>(GPN(p.bnd, dst + l.pa * 16, 16)) = repack2<T>(fa);
                *reinterpret_cast<uint4 *>(GPN(p.bnd, dst + l.pb * 16, 16)) = repack2<T>(fb);
                if (is_q) {
#pragma unroll
                    for (int m = 0; m < kH; ++m) dqa[m] = add2(dqa[m], ya[m]), dqb[m] = add2(dqb[m], yb[m]);
                } else {
#pragma unroll
                    for (int m = 0; m < kH; ++m) dka[m] = add2(dka[m], ya[m]), dkb[m] = add2(dkb[m], yb[m]);
                }
            }
            e += group;
            dst += (unsigned long long)dstep * 16u;
            if (e >= bound) aim_out();
        }
    }
    // the block's sums, in the order of its row groups
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        if (!a.dw[which]) continue;
        __syncthreads();
        if (l.active) {
            float *mine = sums + (warp * group + l.row) * p.hd;
#pragma unroll
            for (int k = 0; k < kH; ++k) {
                *reinterpret_cast<unsigned long long *>(mine + l.pa * kV + 2 * k) = which ? dka[k] : dqa[k];
                *reinterpret_cast<unsigned long long *>(mine + l.pb * kV + 2 * k) = which ? dkb[k] : dqb[k];
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < p.hd; c += 32 * kWarps) {
            float sum = 0.f;
            for (unsigned q = 0; q < kWarps * group; ++q) sum += sums[q * p.hd + c];
            *GP(p.bnd, a.part + (2LL * blockIdx.x + which) * p.hd + c) = sum;
        }
    }
}

// The rows that do not lie on lane groups: a warp a row.  Blocks 0 .. blocks_q - 1
// take the rows of Q, the others those of K: each has the weight gradient of one of them.
struct BwdRow {
    uintptr_t g, x, d;         // of dy (low bits: the token of the tile), x, dx (0: none)
};
constexpr int kBwdRows = 256;

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) k_norm_bwd_rows(const __grid_constant__ NormArgs a) {
    const RotaryArgs &p = a.r;
    const float by_hd = 1.f / (float)p.hd;
    extern __shared__ __align__(16) float smem[];      // two tables [tile][2][rot / 2]; weights [hd]; sums, x, g [3][hd] a warp
    __shared__ BwdRow lists[2][kBwdRows];
    const int which = blockIdx.x >= a.blocks_q, heads = which ? p.hk : p.hq;
    const int first = which ? blockIdx.x - a.blocks_q : blockIdx.x, nblocks = which ? a.blocks - a.blocks_q : a.blocks_q;
    const int tile = a.tile[which], slices = a.slices[which];
    const long long work = (long long)a.tiles[which] * slices;
    const int half = p.rot / 2;
    const unsigned by_half = half > 1 ? 0xffffffffu / half + 1u : 0u;      // x / half for x < 2^15
    const int table = 2 * max(a.tile[0], a.tile[1]) * p.rot;
    float *wtab = smem + table, *sums = wtab + p.hd;

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

    // unit of work u: the heads of slice u % slices of the tokens of tile u / slices
    auto prepare = [&](long long u, BwdRow *list, float *tab) -> int {
        const int slice = (int)(u % slices), lo = (int)((long long)heads * slice / slices), mine = (int)((long long)heads * (slice + 1) / slices) - lo;
        const long long t0 = u / slices * tile;
        const int nt = (int)(p.tokens - t0 < tile ? p.tokens - t0 : tile);
        const unsigned *sg = which ? p.sk : p.sq, *sd = which ? p.sko : p.sqo;
        const unsigned by_mine = 0xffffffffu / mine + 1u;  // x / mine for x < 2^15
        for (int e = threadIdx.x; e < nt * mine; e += kThreads) {
            const unsigned tt = mine > 1 ? __umulhi(e, by_mine) : e, head = lo + e - tt * mine, t = (unsigned)t0 + tt;
            list[e].g = reinterpret_cast<uintptr_t>((const char *)(which ? p.K : p.Q) + row_units(p, t, sg, head)) + tt;
            list[e].x = reinterpret_cast<uintptr_t>((const char *)a.X[which] + row_units(p, t, a.sx[which], head));
            list[e].d = reinterpret_cast<uintptr_t>((char *)(which ? p.Ko : p.Qo) + row_units(p, t, sd, head));
        }
        for (int e = kThreads - 1 - threadIdx.x; e < nt * half; e += kThreads) {
            const unsigned tt = half > 1 ? __umulhi(e, by_half) : e, k = e - tt * half, t = (unsigned)t0 + tt;
            const long long at = (p.pos ? (long long)*GP(p.bnd, p.pos + t) : (long long)(t % p.n)) + p.pos0;
            float cs, sn;
            cos_sin(at, *GP(p.bnd, p.turns + k), cs, sn);
            tab[(2 * tt) * half + k] = cs * p.scale;
            tab[(2 * tt + 1) * half + k] = sn * p.scale;
        }
        return nt * mine;
    };
    pdl_wait();
    pdl_trigger();
    const T *w = reinterpret_cast<const T *>(which ? a.wk : a.wq);
    for (int c = threadIdx.x; c < p.hd; c += kThreads) wtab[c] = w ? Elt<T>::to_f(*GP(p.bnd, w + c)) + a.offset : 1.f;
    float *dsum = sums + warp * 3 * p.hd, *sx = dsum + p.hd, *sg = sx + p.hd;
    for (int c = lane; c < p.hd; c += 32) dsum[c] = 0.f;

    int buf = 0, total = prepare(first, lists[0], smem);
    for (long long u0 = first; u0 < work; u0 += nblocks, buf ^= 1) {
        const BwdRow *list = lists[buf];
        const float *tab = smem + buf * (table / 2);
        const bool more = u0 + nblocks < work;
        int next = 0;
        __syncthreads();                 // this tile is prepared, the other buffer is free
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
            const float rn = inverse_norm(sum, by_hd, a.eps), c2 = mean_part(dot, by_hd, rn);
            T *d = reinterpret_cast<T *>(r.d);
            for (int c = lane; c < p.hd; c += 32) {
                dsum[c] = fmaf(sg[c], sx[c] * rn, dsum[c]);
                *GP(p.bnd, d + c) = Elt<T>::from_f(rn * fmaf(-c2, sx[c], sg[c] * wtab[c]));
            }
            __syncwarp();
        }
        total = next;
    }
    if (!a.dw[which]) return;
    // the block's sums, in the order of its warps
    __syncthreads();
    for (int c = threadIdx.x; c < p.hd; c += kThreads) {
        float s = 0.f;
        for (int q = 0; q < kThreads / 32; ++q) s += sums[q * 3 * p.hd + c];
        *GP(p.bnd, a.part + (long long)blockIdx.x * p.hd + c) = s;
    }
}

// dw: the blocks' sums added, 32 channels a block, 32 threads a channel.
__global__ void __launch_bounds__(1024) k_norm_dw(const __grid_constant__ NormArgs a) {
    __shared__ float s[32][33];
    const RotaryArgs &p = a.r;
    const int which = blockIdx.y, c = blockIdx.x * 32 + (threadIdx.x & 31), seg = threadIdx.x >> 5;
    // rows of sums: two a block, or one (blocks of Q, then of K)
    const int lo = a.both ? which : which ? a.blocks_q : 0, hi = a.both || which ? a.blocks : a.blocks_q, by = a.both ? 2 : 1;
    pdl_wait();
    pdl_trigger();
    if (!a.dw[which]) return;
    float x = 0.f;
    if (c < p.hd) {
#pragma unroll 8
        for (int b = lo + by * seg; b < hi; b += 32 * by) x += *GP(p.bnd, a.part + (long long)b * p.hd + c);
    }
    s[seg][threadIdx.x & 31] = x;
    __syncthreads();
    x = s[threadIdx.x & 31][seg];                        // a warp a channel now
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    if ((threadIdx.x & 31) == 0 && blockIdx.x * 32 + seg < p.hd) *GP(p.bnd, a.dw[which] + blockIdx.x * 32 + seg) = x;
}

// ---------------------------------------------------------------------------
// rows of a cache in 4 bits as values: a thread a word of codes (8 channels).  8.9k
// tokens of 8 heads of 128, bf16, take 16 us, 2.9 TB/s, by instructions: 137 of a warp for
// 32 words, as each divides for its row and has a slot, a scale and three addresses.
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(kThreads) k_read4(const __grid_constant__ Read4Args p) {
    constexpr int kFlight = 4;                           // words of a thread in flight: slot -> codes is a chain
    const unsigned words = p.hd / 8, per_kind = p.hk * words, per_token = 2 * per_kind;   // at most 2^23
    const unsigned by_words = 0xffffffffu / words + 1u;  // for x / words
    const long long step = (long long)gridDim.x * kThreads, first = (long long)blockIdx.x * kThreads + threadIdx.x;
    const unsigned step_t = (unsigned)(step / per_token), step_in = (unsigned)(step - (long long)step_t * per_token);
    long long t = first / per_token;
    unsigned in = (unsigned)(first - t * per_token);
    pdl_wait();
    pdl_trigger();
    while (t < p.tokens) {
        uint32_t w[kFlight];
        T scale[kFlight];
        T *dst[kFlight];
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
            dst[i] = nullptr;
            if (t < p.tokens) {
                const int slot = *GP(p.bnd, p.slots + t);
                if (slot >= 0 && slot < p.n_slots) {
                    const bool is_v = in >= per_kind;
                    const unsigned x = is_v ? in - per_kind : in;
                    unsigned row = __umulhi(x, by_words);
                    if (row * words > x) --row;          // (the product may be one too large past 2^32 / words)
                    const unsigned word = x - row * words, blk = (unsigned)slot >> p.page_log2, off = (unsigned)slot & ((1u << p.page_log2) - 1u);
                    const unsigned long long line = ((blk * (unsigned)p.hk + row) << p.page_log2) + off;
                    w[i] = *GP(p.bnd, reinterpret_cast<const uint32_t *>(is_v ? p.Vc : p.Kc) + line * words + word);
                    scale[i] = *GP(p.bnd, reinterpret_cast<const T *>(is_v ? p.Vs : p.Ks) + line * (words / 4) + word / 4);
                    dst[i] = reinterpret_cast<T *>(is_v ? p.V : p.K) + (t * p.hk + row) * p.hd + word * 8;
                } else if (slot != -1 && in == 0) {
                    atomicOr(p.err, kErrInvalid);
                }
                t += step_t;
                in += step_in;
                if (in >= per_token) {
                    in -= per_token;
                    ++t;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
            if (!dst[i]) continue;
            const float s = Elt<T>::to_f(scale[i]);
            float f[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] = s * (float)((int)((w[i] >> (4 * k)) & 15u) - 8);
            if constexpr (sizeof(T) == 4) {
                *reinterpret_cast<uint4 *>(GPN(p.bnd, dst[i], 16)) = pack16<T>(f);
                *reinterpret_cast<uint4 *>(GPN(p.bnd, dst[i] + 4, 16)) = pack16<T>(f + 4);
            } else {
                *reinterpret_cast<uint4 *>(GPN(p.bnd, dst[i], 16)) = pack16<T>(f);
            }
        }
    }
}

// Which kernel takes the rows: halves or adjacent pairs in 16-byte pieces on at
// most 32 lanes (and, into 4 bits, 16-bit types whose groups lie on four adjacent lanes or
// are four at most), else a warp a row.  lanes: of a row, a power of two from 4.
int mode_of(const RotaryArgs &r, int es, int *kind, int *lanes, NormArgs *a = nullptr) {
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
    if (*kind == 2) {
        const bool adjacent = nturn % 4 == 0 && (pieces - 2 * nturn) % 8 == 0;
        fits = fits && es == 2 && (adjacent || pieces <= 16);
        if (fits && !adjacent) *kind = 3;
    }
    if (!fits) *lanes = 32;
    return !fits ? 2 : r.interleaved ? 1 : 0;
}

template <typename T, int kKind>
cudaError_t launch_t(const NormArgs &a, int mode, dim3 grid, size_t smem, cudaStream_t st) {
    if constexpr (kKind < 2 || sizeof(T) == 2) {
        if (mode == 0) return launch_dependent(&k_norm<T, false, kKind>, grid, 32 * kWarps, smem, st, a);
        if (mode == 1) return launch_dependent(&k_norm<T, true, kKind>, grid, 32 * kWarps, smem, st, a);
    }
    return launch_dependent(&k_norm_rows<T, kKind == 3 ? 2 : kKind>, grid, kThreads, smem, st, a);
}
template <typename T>
cudaError_t launch_kind(int kind, const NormArgs &a, int mode, dim3 grid, size_t smem, cudaStream_t st) {
    if (kind == 0) return launch_t<T, 0>(a, mode, grid, smem, st);
    if (kind == 1) return launch_t<T, 1>(a, mode, grid, smem, st);
    if constexpr (sizeof(T) == 2)
        if (kind == 3) return launch_t<T, 3>(a, mode, grid, smem, st);
    return launch_t<T, 2>(a, mode, grid, smem, st);
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

// Slices of a token's `all` row groups, and row groups of a slice: more than one slice
// where there are fewer tokens than warps.
void split_of(const RotaryArgs &r, long long all, long long warps, int *split, int *its) {
    const long long want = std::max(1LL, std::min(all, warps / r.tokens));
    *its = (int)((all + want - 1) / want);
    *split = (int)((all + *its - 1) / *its);
}

template <typename T>
cudaError_t launch_bwd_t(const NormArgs &a, int mode, size_t smem, cudaStream_t st) {
    if (mode == 0) return launch_dependent(&k_norm_bwd<T, false>, dim3((unsigned)a.blocks_q), 32 * kWarps, smem, st, a);
    if (mode == 1) return launch_dependent(&k_norm_bwd<T, true>, dim3((unsigned)a.blocks_q), 32 * kWarps, smem, st, a);
    const auto fn = &k_norm_bwd_rows<T>;
    const cudaError_t e = ensure_smem(reinterpret_cast<const void *>(fn), (int)smem);
    if (e != cudaSuccess) return e;
    return launch_dependent(fn, dim3((unsigned)a.blocks), kThreads, smem, st, a);
}

}  // namespace

cudaError_t launch_norm(DType dt, int kind, NormArgs a, cudaStream_t st) {
    const int es = dt == kF32 ? 4 : 2;
    const int mode = mode_of(a.r, es, &kind, &a.lanes, &a);
    a.r.rows = a.r.hq + a.r.hk * (kind ? 2 : 1);
    a.r.row_bytes = a.r.hd * es;
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidValue;
    dim3 grid;
    size_t smem;
    if (mode < 2) {
        const long long full = 5LL * sms, pad = (a.r.rot + 3) / 4 * 4, group = 32 / a.lanes;
        split_of(a.r, (a.r.rows + group - 1) / group, full * kWarps, &a.split, &a.its);
        grid = dim3((unsigned)std::min(((long long)a.r.tokens * a.split + kWarps - 1) / kWarps, full));
        smem = (size_t)((1 + kWarps) * pad + 2 * a.r.hd) * sizeof(float);
    } else {
        const long long full = (long long)kBlocks * sms;
        int slices = 1;
        tile_of(a.r, a.r.rows, 32, full, kMaxRows, &a.r.tile, &slices);
        grid = dim3((unsigned)std::min(((long long)a.r.tokens + a.r.tile - 1) / a.r.tile, full), (unsigned)slices);
        smem = ((size_t)2 * a.r.tile * a.r.rot + 2 * a.r.hd + kThreads / 32 * a.r.hd) * sizeof(float);
    }
    if (dt == kF32) return launch_kind<float>(kind, a, mode, grid, smem, st);
    if (dt == kF16) return launch_kind<__half>(kind, a, mode, grid, smem, st);
    return launch_kind<__nv_bfloat16>(kind, a, mode, grid, smem, st);
}

cudaError_t launch_norm_bwd(DType dt, NormArgs a, cudaStream_t st) {
    const int es = dt == kF32 ? 4 : 2;
    int kind = 0;
    const int mode = mode_of(a.r, es, &kind, &a.lanes);
    a.r.rows = a.r.hq + a.r.hk;
    a.both = mode < 2;
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidValue;
    size_t smem;
    if (mode < 2) {
        const long long full = std::min(3LL * sms, (long long)kNormRows / 2), group = 32 / a.lanes;
        split_of(a.r, (a.r.rows + group - 1) / group, full * kWarps, &a.split, &a.its);
        a.blocks_q = (int)std::min(((long long)a.r.tokens * a.split + kWarps - 1) / kWarps, full);
        a.blocks = 2 * a.blocks_q;                 // (rows of sums)
        smem = ((size_t)(1 + kWarps) * ((a.r.rot + 3) / 4 * 4) + (size_t)(32 * kWarps / a.lanes + 2) * a.r.hd) * sizeof(float);
    } else {
        const long long full = std::min(2LL * sms, (long long)kNormRows - 2), all = a.r.rows;
        long long blocks[2] = {0, 0};
        for (int k = 0; k < 2; ++k) {
            const int heads = k ? a.r.hk : a.r.hq;
            a.tile[k] = a.slices[k] = 1;
            if (heads == 0) continue;
            // blocks shared by how many rows there are
            const long long share = std::max(1LL, k ? full - full * a.r.hq / all : full * a.r.hq / all);
            tile_of(a.r, heads, 32, full, kBwdRows, &a.tile[k], &a.slices[k]);
            a.tiles[k] = (int)(((long long)a.r.tokens + a.tile[k] - 1) / a.tile[k]);
            blocks[k] = std::min((long long)a.tiles[k] * a.slices[k], share);
        }
        a.blocks_q = (int)blocks[0];
        a.blocks = (int)(blocks[0] + blocks[1]);
        smem = ((size_t)2 * std::max(a.tile[0], a.tile[1]) * a.r.rot + a.r.hd + (size_t)kThreads / 32 * 3 * a.r.hd) * sizeof(float);
    }
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
    const dim3 grid((unsigned)std::min((items + kThreads - 1) / kThreads, 8LL * sms));
    if (dt == kF32) return launch_dependent(&k_read4<float>, grid, kThreads, 0, st, a);
    if (dt == kF16) return launch_dependent(&k_read4<__half>, grid, kThreads, 0, st, a);
    return launch_dependent(&k_read4<__nv_bfloat16>, grid, kThreads, 0, st, a);
}

}  // namespace swab
