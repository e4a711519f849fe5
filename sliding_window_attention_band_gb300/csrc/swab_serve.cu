// swab_serve.cu -- the entry points of include/swab.h for answering with the
// banded attention: rotary positions, block tables, the cache write, decode.
// Arguments are validated on the host before any CUDA call.
#include <algorithm>
#include <atomic>
#include <chrono>
#include <cmath>

#include "swab_internal.h"

namespace swab {
namespace {

bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
cudaStream_t as_stream(void *s) { return reinterpret_cast<cudaStream_t>(s); }
long long elt(int dtype) { return dtype == SWAB_F32 ? 4 : 2; }
bool good_dtype(int dtype) { return dtype == SWAB_F32 || dtype == SWAB_F16 || dtype == SWAB_BF16; }

swab_status check_tensors(std::initializer_list<const void *> ptrs) {
    for (const void *p : ptrs) {
        if (!p) return SWAB_ERR_INVALID_ARG;
        if (!aligned(p, 16)) return SWAB_ERR_MISALIGNED;
    }
    return SWAB_OK;
}
swab_status check_ints(std::initializer_list<const void *> ptrs) {
    for (const void *p : ptrs) {
        if (!p) return SWAB_ERR_INVALID_ARG;
        if (!aligned(p, 4)) return SWAB_ERR_MISALIGNED;
    }
    return SWAB_OK;
}

#if SWAB_BOUNDS_CHECK
#define SERVE_BOUNDS(target, ...) call_extents((target), {__VA_ARGS__})
#else
#define SERVE_BOUNDS(target, ...) SWAB_OK
#endif

int log2_of(int page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : page == 128 ? 7 : -1; }

// ---------------------------------------------------------------------------
// rotary
// ---------------------------------------------------------------------------

// Strides of a [b, n, heads, hd] tensor in units of 16 bytes: the given ones,
// or contiguous.  An output's rows must not overlap: sorted by stride, each
// dimension has to step over all that the smaller ones span.
swab_status take_strides(const swab_rotary_desc *d, int heads, const int64_t *given, bool output, unsigned *units) {
    const long long vec = 16 / elt(d->dtype), size[3] = {d->b, d->n, heads};
    long long s[3];
    if (given[0] == 0 && given[1] == 0 && given[2] == 0) {
        s[2] = d->head_dim;
        s[1] = s[2] * heads;
        s[0] = s[1] * d->n;
        output = false;
    } else {
        for (int k = 0; k < 3; ++k) {
            if (given[k] < 0) return SWAB_ERR_INVALID_ARG;
            if (given[k] % vec != 0) return SWAB_ERR_MISALIGNED;
            s[k] = given[k];
        }
    }
    if (output) {
        int order[3] = {0, 1, 2};
        std::sort(order, order + 3, [&](int x, int y) { return s[x] < s[y]; });
        long long span = d->head_dim;
        for (int k : order) {
            if (size[k] == 1) continue;
            if (s[k] < span) return SWAB_ERR_INVALID_ARG;
            if (s[k] > (1ll << 40)) return SWAB_ERR_UNSUPPORTED;
            span += s[k] * (size[k] - 1);
        }
    }
    long long last = 0;                      // of a row, in units of 16 bytes
    for (int k = 0; k < 3; ++k) {
        const long long u = size[k] == 1 ? 0 : s[k] / vec;
        if (u > 0xffffffffll) return SWAB_ERR_UNSUPPORTED;
        if (size[k] > 1 && u > (0xffffffffll - last) / (size[k] - 1)) return SWAB_ERR_UNSUPPORTED;
        last += u * (size[k] - 1);
        units[k] = (unsigned)u;
    }
    return SWAB_OK;
}

[[maybe_unused]] size_t strided_bytes(const swab_rotary_desc *d, int heads, const unsigned *s) {
    return ((size_t)s[0] * (d->b - 1) + (size_t)s[1] * (d->n - 1) + (size_t)s[2] * (heads - 1)) * 16 + d->head_dim * elt(d->dtype);
}

swab_status check_rotary(const swab_rotary_desc *d, const uint64_t *turns, const int32_t *pos, RotaryArgs *a) {
    if (!d) return SWAB_ERR_INVALID_ARG;
    if (d->b < 1 || d->n < 1 || d->h < 1 || d->hk < 0 || d->head_dim < 1 || d->pos0 < 0) return SWAB_ERR_INVALID_ARG;
    if (d->rot_dim < 0 || d->rot_dim > d->head_dim || d->rot_dim % 2 != 0) return SWAB_ERR_INVALID_ARG;
    if (d->interleaved != 0 && d->interleaved != 1) return SWAB_ERR_INVALID_ARG;
    if (!good_dtype(d->dtype) || !std::isfinite(d->scale)) return SWAB_ERR_INVALID_ARG;
    if (d->head_dim * elt(d->dtype) % 16 != 0 || d->head_dim > 512) return SWAB_ERR_UNSUPPORTED;
    if (d->h > 65535 || d->hk > 65535) return SWAB_ERR_UNSUPPORTED;
    if ((long long)d->b * d->n > 0x7fffffffll) return SWAB_ERR_UNSUPPORTED;
    if (d->rot_dim > 0) {
        if (!turns) return SWAB_ERR_INVALID_ARG;
        if (!aligned(turns, 8)) return SWAB_ERR_MISALIGNED;
    }
    if (pos && !aligned(pos, 4)) return SWAB_ERR_MISALIGNED;
    a->turns = reinterpret_cast<const unsigned long long *>(turns);
    a->pos = pos;
    a->tokens = (unsigned)d->b * (unsigned)d->n;
    a->n = (unsigned)d->n;
    a->hq = d->h;
    a->hk = d->hk;
    a->hd = d->head_dim;
    a->rot = d->rot_dim;
    a->interleaved = d->interleaved;
    a->pos0 = d->pos0;
    a->scale = d->scale;
    return SWAB_OK;
}

swab_status rotary_common(const swab_rotary_desc *d, const uint64_t *turns, const int32_t *pos, const void *Q,
                          const void *K, void *Qo, void *Ko, bool backward, void *stream) {
    RotaryArgs a{};
    swab_status s = check_rotary(d, turns, pos, &a);
    if (s != SWAB_OK) return s;
    if ((s = take_strides(d, d->h, d->q_stride, false, a.sq)) != SWAB_OK) return s;
    if ((s = take_strides(d, d->h, d->qo_stride, true, a.sqo)) != SWAB_OK) return s;
    if ((s = check_tensors({Q, Qo})) != SWAB_OK) return s;
    if (d->hk > 0) {
        if ((s = take_strides(d, d->hk, d->k_stride, false, a.sk)) != SWAB_OK) return s;
        if ((s = take_strides(d, d->hk, d->ko_stride, true, a.sko)) != SWAB_OK) return s;
        if ((s = check_tensors({K, Ko})) != SWAB_OK) return s;
    }
    a.Q = Q;
    a.K = K;
    a.Qo = Qo;
    a.Ko = Ko;
    a.backward = backward;
    if ((s = SERVE_BOUNDS(&a.bnd, {Q, strided_bytes(d, d->h, a.sq)}, {Qo, strided_bytes(d, d->h, a.sqo)},
                          {d->hk ? K : nullptr, strided_bytes(d, d->hk, a.sk)},
                          {d->hk ? Ko : nullptr, strided_bytes(d, d->hk, a.sko)},
                          {d->rot_dim ? turns : nullptr, (size_t)d->rot_dim / 2 * 8}, {pos, (size_t)a.tokens * 4})) != SWAB_OK)
        return s;
    return status_of(launch_rotary(static_cast<DType>(d->dtype), false, a, as_stream(stream)));
}

// ---------------------------------------------------------------------------
// cache
// ---------------------------------------------------------------------------
swab_status check_cache(const swab_cache_desc *c) {
    if (!c) return SWAB_ERR_INVALID_ARG;
    if (c->batch < 1 || c->n_blocks < 1 || c->cols < 1) return SWAB_ERR_INVALID_ARG;
    if (c->ring != 0 && c->ring != 1) return SWAB_ERR_INVALID_ARG;
    if (c->pinned < 0 || c->pinned >= (c->ring ? c->cols : 1) || c->max_new < 0) return SWAB_ERR_INVALID_ARG;
    if (log2_of(c->page) < 0 || c->batch > 65535) return SWAB_ERR_UNSUPPORTED;
    if ((long long)c->n_blocks * c->page > 0x7fffff00ll) return SWAB_ERR_UNSUPPORTED;
    return SWAB_OK;
}

[[maybe_unused]] size_t cache_bytes(const swab_cache_desc *c, int hk, int hd, int dtype) {
    return (size_t)c->n_blocks * c->page * hk * hd * elt(dtype);
}
[[maybe_unused]] size_t table_bytes(const swab_cache_desc *c) { return (size_t)c->batch * c->cols * 4; }

// ---------------------------------------------------------------------------
// decode
// ---------------------------------------------------------------------------
constexpr long long kSms = 152;      // of a GB300 (the plan sizes the workspace, and that needs no device)

struct DecodePlan {
    bool rows;                       // tensor-core kernels (fp16 / bf16, head_dim 64 or 128)
    int nsplit, chunk, nparts;
    int npre, pre_pieces, pre_chunks, pre_tokens;
    int row_warps;
    bool fold;                       // no join launch: the rows kernel adds the prefix's parts
    int row_tiles;                   // of a request, in the rows kernel's grid
    long long row_blocks;            // of that grid
    size_t parts_bytes, ml_bytes, bytes;   // workspace: the parts, their (max, sum), a word a block of rows behind a prefix
};

swab_status check_decode(const swab_decode_desc *d) {
    if (!d) return SWAB_ERR_INVALID_ARG;
    const swab_cache_desc *c = &d->cache;
    const swab_status s = check_cache(c);
    if (s == SWAB_ERR_INVALID_ARG) return s;
    if (d->tokens < 1 || d->h < 1 || d->hk < 1 || d->head_dim < 1 || d->max_q < 1 || d->max_len < 1) return SWAB_ERR_INVALID_ARG;
    if (d->w < 0 || d->w > (1 << 30) || d->dilation < 0 || d->n_sink < 0 || d->prefix_len < 0) return SWAB_ERR_INVALID_ARG;
    if (!good_dtype(d->dtype) || d->h % d->hk != 0) return SWAB_ERR_INVALID_ARG;
    if (d->prefix_len > (long long)c->n_blocks * c->page) return SWAB_ERR_INVALID_ARG;
    const long long width = (long long)d->h * d->head_dim, vec = 16 / elt(d->dtype);
    for (const int64_t rs : {d->q_row_stride, d->out_row_stride})
        if (rs < 0 || (rs > 0 && rs < width)) return SWAB_ERR_INVALID_ARG;
    if (c->ring) {
        const long long reach = (long long)d->w * (d->dilation + 1) + d->max_q;
        if (reach > (long long)(c->cols - c->pinned - 1) * c->page + 1) return SWAB_ERR_INVALID_ARG;
        if (d->n_sink > (long long)c->pinned * c->page) return SWAB_ERR_INVALID_ARG;
    }
    if (s != SWAB_OK) return s;
    if (d->head_dim % vec != 0 || d->head_dim > 256 || d->dilation > SWAB_MAX_DILATION) return SWAB_ERR_UNSUPPORTED;
    if ((long long)c->n_blocks * c->page * d->hk >= 0xffffffffll) return SWAB_ERR_UNSUPPORTED;
    if (d->h / d->hk > 128 || d->h > 65535 || (long long)d->tokens * d->h > 0x7fffffffll) return SWAB_ERR_UNSUPPORTED;
    for (const int64_t rs : {d->q_row_stride, d->out_row_stride}) {
        if (rs % vec != 0) return SWAB_ERR_MISALIGNED;
        if (rs > (1ll << 36)) return SWAB_ERR_UNSUPPORTED;
    }
    return SWAB_OK;
}

// How many of its own positions a query (a request's queries, undilated) can
// attend to.
long long most_keys(const swab_decode_desc *d) {
    const long long band = (long long)d->w + 1 + (d->dilation == 0 ? d->max_q - 1 : 0);
    return std::min<long long>(d->max_len, d->n_sink + band);
}

// Pieces of the prefix, and whether the rows kernel joins its parts (fold).  The
// prefix kernel keeps an SM a block to itself; the rows kernel starts beside it
// on the SMs left over, and takes all of them when it has ended.  More pieces
// end sooner but leave fewer SMs and more parts to join; with fold the rows
// kernel's blocks stay where they are until the prefix is there, without it they
// make room for more and a third launch joins.  The time of each choice is
// estimated (us; `blocks` of the rows kernel with `keys` keys each): a block of
// the prefix 5.6 + 1.6 a chunk (0.8 of a single row tile; two thirds with
// head_dim 64), a block of rows 3.3 + 1 every 45 KB, parts 1 MB a us, 1.25 in
// a launch of their own that costs 1.3 more.  The numbers were fitted to shapes
// measured with every choice; on 162 of them (2 to 256 requests, prefixes of 256
// to 32768, head_dim 64 and 128; profiles/prefix_plan.md) theirs are 3.8 %
// slower than the best on average, all SMs to the prefix and fold wherever it
// goes 9.0 % (256 requests with 2048
// shared keys: 49 us with one piece of a tile, 54 with four, 61 with four and
// fold; 64 with 8192: 33 with 7 pieces, 36 with 16 and fold, 41 without).
void plan_prefix(const swab_decode_desc *d, long long blocks, long long keys, DecodePlan *p) {
    const long long group = d->h / d->hk;
    p->pre_tokens = (int)(128 / group);
    const bool pair = d->tokens > p->pre_tokens;
    const long long per = p->pre_tokens * (pair ? 2 : 1), tiles = (d->tokens + per - 1) / per * d->hk;
    const long long chunks = ((long long)d->prefix_len + 127) / 128;
    const long long most = std::min(std::max<long long>(1, kSms / tiles), (chunks + 1) / 2);
    const double chunk_us = (pair ? 1.6 : 0.8) * (d->head_dim + 64) / 192, slots = 12 / p->row_warps;
    const double block_us = 3.3 + (double)keys * d->head_dim * 4 / 45e3, part_us = (double)d->tokens * d->h * d->head_dim * 4 / 1e6;
    double best = 0.0;
    for (long long eighth = 8; eighth >= 1; --eighth) {
        const long long want = std::max<long long>(1, most * eighth / 8), pre_chunks = (chunks + want - 1) / want;
        const long long pieces = (chunks + pre_chunks - 1) / pre_chunks, npre = pieces * (pair ? 1 : 2);
        const double pre = 5.6 + chunk_us * pre_chunks, beside = std::max<long long>(0, kSms - tiles * pieces) * slots;
        for (int fold = p->nsplit == 1 && npre <= kMaxFold; fold >= 0; --fold) {
            double us = fold ? part_us * npre : 1.3 + part_us * (npre + p->nsplit) * 0.8;
            if (blocks <= beside) us += std::max(pre, block_us);
            else if (fold) us += pre + std::max((blocks - beside) / (kSms * slots), 0.8) * block_us;
            else us += pre + std::max((blocks - beside * pre / block_us) / (kSms * slots), 0.1) * block_us;
            if (best > 0.0 && us >= best) continue;
            best = us;
            p->pre_chunks = (int)pre_chunks;
            p->pre_pieces = (int)pieces;
            p->npre = (int)npre;
            p->fold = fold;
        }
    }
}

DecodePlan plan_decode(const swab_decode_desc *d) {
    DecodePlan p{};
    const long long group = d->h / d->hk, batch = d->cache.batch;
    p.rows = d->dtype != SWAB_F32 && (d->head_dim == 64 || d->head_dim == 128);
    // the key list of a query (general kernel) or of a request's rows is cut
    // where there are fewer blocks than the GPU holds
    long long keys = most_keys(d), blocks = batch, hold, least;
    if (p.rows) {
        const long long rows = d->dilation == 0 ? d->max_q * group : group;
        const long long tiles = (rows + 15) / 16 * (d->dilation == 0 ? 1 : d->max_q);
        blocks *= d->hk * tiles;
        p.row_tiles = (int)std::min<long long>(tiles, 65535 / d->hk);
        // An SM holds 12 warps.  Long lists want all of them in one go: four warps
        // a block where the blocks fit at once, else three or two; with more
        // blocks than that, four (two for lists too short to share).  Where they
        // leave a quarter of the warps free, blocks of three or two and a list cut
        // once more may fill them (256 blocks of 8k keys: 94 us against 111).
        p.row_warps = blocks <= 3 * kSms ? 4 : blocks <= 4 * kSms ? 3 : blocks <= 6 * kSms ? 2 : keys <= 256 ? 2 : 4;
        hold = 3 * kSms;
        for (int w = 3; w >= 2 && keys >= 2048; --w) {
            const long long now = std::max<long long>(1, hold / blocks) * p.row_warps, then = 12 / w * kSms / blocks * w;
            if (4 * then >= 5 * now && blocks <= 3 * kSms) {
                p.row_warps = w;
                hold = 12 / w * kSms;
            }
        }
        // Pieces of 128 keys (8 key heads of 128, a context of 2000: 7.0 us against
        // 8.4 with 256 and 26 in one piece); of 64 where up to 24 blocks have up to
        // 1024 keys (8 x 600: 5.9 against 6.5 us, 8 x 1500: 7.2 against 6.5).  Lists
        // up to 256 whole: the second launch costs as much (12 x 200: 4.7 against
        // 4.9 in pieces of 64).  Up to 512 too where there are more than 64 blocks
        // or a prefix whose parts could be joined without it (192 x 400: 7.3
        // against 8.2; 32 x 400: 8.4 against 6.7).
        const bool whole = keys <= 256 || (keys <= 512 && (blocks > 64 || d->prefix_len > 0));
        least = whole ? 512 : keys <= 1024 && blocks <= 24 ? 64 : 128;
    } else {
        keys += d->prefix_len;
        blocks *= d->hk * ((group + 3) / 4);
        hold = 8 * kSms;
        least = 64;
    }
    const long long want = std::max<long long>(1, hold / blocks);
    const long long chunk = std::max<long long>(least, ((keys + want - 1) / want + 63) / 64 * 64);
    p.nsplit = (int)((keys + chunk - 1) / chunk);
    p.chunk = (int)std::min<long long>(chunk, 0x7fffffff);
    if (p.rows && d->prefix_len > 0) plan_prefix(d, blocks * p.nsplit, std::min<long long>(keys, p.chunk), &p);
    p.nparts = p.nsplit + p.npre;
    if (p.nparts > 1) {
        const size_t lines = (size_t)d->tokens * d->h * p.nparts;
        p.parts_bytes = (lines * d->head_dim * 4 + 255) / 256 * 256;
        p.ml_bytes = lines * 8;
        p.bytes = p.parts_bytes + p.ml_bytes + 256;     // the parts start on a multiple of 256 bytes
    }
    if (p.npre > 0) {
        p.row_blocks = p.nsplit * (long long)d->hk * p.row_tiles * batch;
        p.bytes += (size_t)p.row_blocks * 8;
    }
    return p;
}

// A number that no other call of this process, nor memory by chance, holds: the
// workspace's contents on entry do not matter, and a word left in it must not
// be taken for one that this call's prefix kernel has set.
unsigned long long next_token() {
    static std::atomic<unsigned long long> count{(unsigned long long)std::chrono::steady_clock::now().time_since_epoch().count()};
    unsigned long long x = count.fetch_add(1, std::memory_order_relaxed) * 0x9e3779b97f4a7c15ull;   // odd: a bijection
    x ^= x >> 32;
    x *= 0xd6e8feb86659fd93ull;
    return (x ^ (x >> 32)) | 1ull;
}

// Tensor maps of the prefix kernel: Q as {hd, h, tokens}, a tile the heads of a
// group for pre_tokens tokens; the cache as {hd, page, n_blocks * hk}, a block
// of one key head at a time; 64 channels (128 bytes) wide.
bool prefix_maps(const swab_decode_desc *d, const DecodeArgs &a, DType dt, CUtensorMap *mq, CUtensorMap *mk, CUtensorMap *mv) {
    const cuuint64_t hd = (cuuint64_t)d->head_dim;
    const cuuint64_t qd[3] = {hd, (cuuint64_t)d->h, (cuuint64_t)d->tokens}, qs[2] = {hd * 2, (cuuint64_t)a.q_stride * 2};
    const cuuint32_t qb[3] = {64, (cuuint32_t)a.group, (cuuint32_t)a.pre_tokens};
    const cuuint64_t page = (cuuint64_t)d->cache.page;
    const cuuint64_t kd[3] = {hd, page, (cuuint64_t)d->cache.n_blocks * d->hk}, ks[2] = {hd * 2, page * hd * 2};
    const cuuint32_t kb[3] = {64, (cuuint32_t)page, 1};
    return encode_tiled(mq, dt, 3, a.Q, qd, qs, qb) && encode_tiled(mk, dt, 3, a.Kc, kd, ks, kb) &&
           encode_tiled(mv, dt, 3, a.Vc, kd, ks, kb);
}

}  // namespace
}  // namespace swab

using namespace swab;

extern "C" {

SWAB_API swab_status rotary_frequencies(int32_t rot_dim, double base, int32_t scaling, double factor, double original,
                                        double low, double high, uint64_t *turns, float *scale) {
    if (rot_dim < 2 || rot_dim % 2 != 0 || !turns || !scale) return SWAB_ERR_INVALID_ARG;
    if (!(base > 1.0) || !std::isfinite(base) || !(factor >= 1.0) || !std::isfinite(factor)) return SWAB_ERR_INVALID_ARG;
    if (scaling < SWAB_ROTARY_NONE || scaling > SWAB_ROTARY_BANDS) return SWAB_ERR_INVALID_ARG;
    const bool blends = scaling == SWAB_ROTARY_YARN || scaling == SWAB_ROTARY_BANDS;
    if (blends && !(original > 0.0 && std::isfinite(original) && low > 0.0 && low < high && std::isfinite(high)))
        return SWAB_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586476925, r = rot_dim;
    *scale = 1.f;
    double ramp_lo = 0.0, ramp_hi = 0.0;
    if (scaling == SWAB_ROTARY_NTK && rot_dim > 2) base *= std::pow(factor, r / (r - 2.0));
    if (scaling == SWAB_ROTARY_YARN) {
        // the pair that turns `t` times within the original context
        auto pair = [&](double t) { return r * std::log(original / (t * two_pi)) / (2.0 * std::log(base)); };
        ramp_lo = std::max(std::floor(pair(high)), 0.0);
        ramp_hi = std::min(std::ceil(pair(low)), r - 1.0);
        *scale = (float)(0.1 * std::log(factor) + 1.0);
    }
    for (int k = 0; k < rot_dim / 2; ++k) {
        double f = std::pow(base, -2.0 * k / r);
        if (scaling == SWAB_ROTARY_LINEAR) {
            f /= factor;
        } else if (scaling == SWAB_ROTARY_YARN) {
            const double m = std::min(std::max((k - ramp_lo) / std::max(ramp_hi - ramp_lo, 0.001), 0.0), 1.0);
            f = f / factor * m + f * (1.0 - m);
        } else if (scaling == SWAB_ROTARY_BANDS) {
            const double m = std::min(std::max((original * f / two_pi - low) / (high - low), 0.0), 1.0);
            f = (1.0 - m) * f / factor + m * f;
        }
        turns[k] = (uint64_t)(std::ldexp(f / two_pi, 64) + 0.5);   // f <= 1: below 2^64 / 6
    }
    return SWAB_OK;
}

SWAB_API swab_status rotary(const swab_rotary_desc *desc, const uint64_t *turns, const int32_t *pos, const void *Q,
                            const void *K, void *Qo, void *Ko, void *stream) {
    return rotary_common(desc, turns, pos, Q, K, Qo, Ko, false, stream);
}

SWAB_API swab_status rotary_bwd(const swab_rotary_desc *desc, const uint64_t *turns, const int32_t *pos,
                                const void *dQo, const void *dKo, void *dQ, void *dK, void *stream) {
    return rotary_common(desc, turns, pos, dQo, dKo, dQ, dK, true, stream);
}

SWAB_API swab_status cache_slots(const swab_cache_desc *cache, int32_t tokens, int32_t pos0, const int32_t *lens,
                                 const int32_t *n_new, int32_t *table, const int32_t *free_list, int32_t n_free,
                                 const int32_t *used, int32_t *lens_out, int32_t *used_out, int32_t *q_start,
                                 int32_t *slots, int32_t *pos, void *stream) {
    swab_status s = check_cache(cache);
    if (s != SWAB_OK) return s;
    if (tokens < 0 || pos0 < 0 || n_free < 0) return SWAB_ERR_INVALID_ARG;
    if ((s = check_ints({lens, n_new, table, used, lens_out, used_out, q_start})) != SWAB_OK) return s;
    if (tokens > 0 && (s = check_ints({slots, pos})) != SWAB_OK) return s;
    if (n_free > 0 && (s = check_ints({free_list})) != SWAB_OK) return s;
    if (lens_out == n_new || q_start == lens || q_start == n_new || q_start == lens_out || (tokens > 0 && slots == pos))
        return SWAB_ERR_INVALID_ARG;
    CacheSlotsArgs a{};
    a.lens = lens;
    a.n_new = n_new;
    a.free_list = free_list;
    a.used = used;
    a.table = table;
    a.lens_out = lens_out;
    a.used_out = used_out;
    a.q_start = q_start;
    a.slots = slots;
    a.pos = pos;
    a.batch = cache->batch;
    a.page_log2 = log2_of(cache->page);
    a.n_blocks = cache->n_blocks;
    a.cols = cache->cols;
    a.ring = cache->ring;
    a.pinned = cache->pinned;
    a.max_new = cache->max_new;
    a.n_free = n_free;
    a.tokens = tokens;
    a.pos0 = pos0;
    const size_t b4 = (size_t)cache->batch * 4;
    (void)b4;
    if ((s = SERVE_BOUNDS(&a.bnd, {lens, b4}, {n_new, b4}, {table, table_bytes(cache)}, {free_list, (size_t)n_free * 4},
                          {used, 4}, {lens_out, b4}, {used_out, 8}, {q_start, b4 + 4}, {slots, (size_t)tokens * 4},
                          {pos, (size_t)tokens * 4})) != SWAB_OK)
        return s;
    if (!(a.err = device_status_word())) return SWAB_ERR_CUDA;
    return status_of(launch_cache_slots(a, as_stream(stream)));
}

SWAB_API swab_status rotary_append(const swab_rotary_desc *desc, const swab_cache_desc *cache, const uint64_t *turns,
                                   const int32_t *pos, const int32_t *slots, const void *Q, const void *K, const void *V,
                                   void *Qo, void *Kc, void *Vc, void *stream) {
    RotaryArgs a{};
    swab_status s = check_rotary(desc, turns, pos, &a);
    if (s != SWAB_OK) return s;
    if ((s = check_cache(cache)) != SWAB_OK) return s;
    if (desc->hk < 1 || !Q != !Qo) return SWAB_ERR_INVALID_ARG;
    if ((long long)cache->n_blocks * cache->page * desc->hk >= 0xffffffffll) return SWAB_ERR_UNSUPPORTED;
    if (desc->rot_dim > 0 && !pos) return SWAB_ERR_INVALID_ARG;
    if (Q) {
        if ((s = take_strides(desc, desc->h, desc->q_stride, false, a.sq)) != SWAB_OK) return s;
        if ((s = take_strides(desc, desc->h, desc->qo_stride, true, a.sqo)) != SWAB_OK) return s;
        if ((s = check_tensors({Q, Qo})) != SWAB_OK) return s;
    } else {
        a.hq = 0;
    }
    if ((s = take_strides(desc, desc->hk, desc->k_stride, false, a.sk)) != SWAB_OK) return s;
    if ((s = take_strides(desc, desc->hk, desc->v_stride, false, a.sv)) != SWAB_OK) return s;
    if ((s = check_tensors({K, V, Kc, Vc})) != SWAB_OK) return s;
    if ((s = check_ints({slots})) != SWAB_OK) return s;
    if (Kc == Vc) return SWAB_ERR_INVALID_ARG;
    a.Q = Q;
    a.K = K;
    a.V = V;
    a.Qo = Qo;
    a.Kc = Kc;
    a.Vc = Vc;
    a.slots = slots;
    a.page_log2 = log2_of(cache->page);
    a.n_slots = cache->n_blocks * cache->page;
    if ((s = SERVE_BOUNDS(&a.bnd, {Q, strided_bytes(desc, desc->h, a.sq)}, {Qo, strided_bytes(desc, desc->h, a.sqo)},
                          {K, strided_bytes(desc, desc->hk, a.sk)}, {V, strided_bytes(desc, desc->hk, a.sv)},
                          {Kc, cache_bytes(cache, desc->hk, desc->head_dim, desc->dtype)},
                          {Vc, cache_bytes(cache, desc->hk, desc->head_dim, desc->dtype)},
                          {desc->rot_dim ? turns : nullptr, (size_t)desc->rot_dim / 2 * 8}, {pos, (size_t)a.tokens * 4},
                          {slots, (size_t)a.tokens * 4})) != SWAB_OK)
        return s;
    if (!(a.err = device_status_word())) return SWAB_ERR_CUDA;
    return status_of(launch_rotary(static_cast<DType>(desc->dtype), true, a, as_stream(stream)));
}

SWAB_API size_t band_decode_workspace(const swab_decode_desc *desc) {
    return check_decode(desc) == SWAB_OK ? plan_decode(desc).bytes : 0;
}

SWAB_API swab_status band_decode(const swab_decode_desc *desc, float scale, const void *Q, const void *Kc, const void *Vc,
                                 const int32_t *table, const int32_t *lens, const int32_t *q_start,
                                 const int32_t *prefix_table, void *O, float *lse, void *workspace, void *stream) {
    swab_status s = check_decode(desc);
    if (s != SWAB_OK) return s;
    const swab_cache_desc *c = &desc->cache;
    if (!std::isfinite(scale)) return SWAB_ERR_INVALID_ARG;
    if ((s = check_tensors({Q, Kc, Vc, O})) != SWAB_OK) return s;
    if ((s = check_ints({table, lens, q_start})) != SWAB_OK) return s;
    if (desc->prefix_len > 0 && (s = check_ints({prefix_table})) != SWAB_OK) return s;
    if (lse && !aligned(lse, 16)) return SWAB_ERR_MISALIGNED;
    const DecodePlan plan = plan_decode(desc);
    if (plan.bytes > 0 && (s = check_tensors({workspace})) != SWAB_OK) return s;
    DecodeArgs a{};
    a.Q = Q;
    a.Kc = Kc;
    a.Vc = Vc;
    a.O = O;
    a.lse = lse;
    a.table = table;
    a.lens = lens;
    a.q_start = q_start;
    a.ptable = prefix_table;
    char *parts = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(workspace) + 255) & ~static_cast<uintptr_t>(255));
    a.po = reinterpret_cast<float *>(parts);
    a.pml = reinterpret_cast<float2 *>(parts + plan.parts_bytes);
    a.go = reinterpret_cast<unsigned long long *>(parts + plan.parts_bytes + plan.ml_bytes);
    a.token = plan.npre > 0 ? next_token() : 0;
    a.row_blocks = plan.row_blocks;
    a.row_tiles = plan.row_tiles;
    a.q_stride = desc->q_row_stride ? desc->q_row_stride : (long long)desc->h * desc->head_dim;
    a.o_stride = desc->out_row_stride ? desc->out_row_stride : (long long)desc->h * desc->head_dim;
    a.batch = c->batch;
    a.tokens = desc->tokens;
    a.h = desc->h;
    a.hk = desc->hk;
    a.group = desc->h / desc->hk;
    a.hd = desc->head_dim;
    a.w = desc->w;
    a.stride = desc->dilation + 1;
    a.n_sink = desc->n_sink;
    a.prefix_len = desc->prefix_len;
    a.page_log2 = log2_of(c->page);
    a.n_blocks = c->n_blocks;
    a.cols = c->cols;
    a.ring = c->ring;
    a.pinned = c->pinned;
    a.nsplit = plan.nsplit;
    a.chunk = plan.chunk;
    a.nparts = plan.nparts;
    a.npre = plan.npre;
    a.pre_pieces = plan.pre_pieces;
    a.pre_chunks = plan.pre_chunks;
    a.fold = plan.fold;
    a.row_warps = plan.row_warps;
    a.pre_tokens = plan.pre_tokens;
    a.scale_log2 = scale * 1.4426950408889634f;
    const DType dt = static_cast<DType>(desc->dtype);
    const size_t es = (size_t)elt(desc->dtype), width = (size_t)desc->h * desc->head_dim;
    (void)es;
    (void)width;
    if ((s = SERVE_BOUNDS(&a.bnd, {Q, ((size_t)(desc->tokens - 1) * a.q_stride + width) * es},
                          {O, ((size_t)(desc->tokens - 1) * a.o_stride + width) * es},
                          {Kc, cache_bytes(c, desc->hk, desc->head_dim, desc->dtype)},
                          {Vc, cache_bytes(c, desc->hk, desc->head_dim, desc->dtype)}, {table, table_bytes(c)},
                          {lens, (size_t)c->batch * 4}, {q_start, (size_t)(c->batch + 1) * 4},
                          {desc->prefix_len ? prefix_table : nullptr, (size_t)(desc->prefix_len + c->page - 1) / c->page * 4},
                          {lse, (size_t)desc->tokens * desc->h * 4}, {plan.bytes ? workspace : nullptr, plan.bytes})) != SWAB_OK)
        return s;
    if (!(a.err = device_status_word())) return SWAB_ERR_CUDA;
    cudaError_t e = cudaSuccess;
    if (plan.npre > 0) {
        CUtensorMap mq, mk, mv;
        if (!prefix_maps(desc, a, dt, &mq, &mk, &mv)) return status_of(cudaErrorInvalidValue);
        e = launch_decode_prefix(dt, mq, mk, mv, a, as_stream(stream));
    }
    if (e == cudaSuccess)
        e = plan.rows ? launch_decode_rows(dt, a, as_stream(stream)) : launch_decode_general(dt, a, as_stream(stream));
    if (e == cudaSuccess && a.nparts > 1 && !a.fold) e = launch_decode_join(dt, a, as_stream(stream));
    return status_of(e);
}

}  // extern "C"
