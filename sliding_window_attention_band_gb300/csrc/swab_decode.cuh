// swab_decode.cuh -- what the decode kernels share: a request's rows, the list
// of positions its queries attend to, and where a position lies in the cache.
#pragma once

#include "swab_internal.h"

namespace swab {

// The new tokens of request r: m rows from row0, the first at position i0 of a
// context of `len` positions.
struct Request {
    int r, m, row0, len, i0;
    const int *trow;     // its row of the block table
    int ring_lo;         // recycled positions below this one are gone
    int last;            // last position with a column: a context longer than its table (recorded) ends there
};

constexpr unsigned kDecodeFile = 14;   // site id of the bounds checks in this header

__device__ __forceinline__ Request request_of(const DecodeArgs &p, int r) {
    [[maybe_unused]] constexpr unsigned kSwabFile = kDecodeFile;
    Request q;
    // (any two values: both ends are brought into 0..tokens before they are
    // subtracted, and the difference of the values as they are takes 33 bits)
    const int first = *GP(p.bnd, p.q_start + r), end = *GP(p.bnd, p.q_start + r + 1);
    const int a = min(max(first, 0), p.tokens), b = min(max(end, 0), p.tokens);
    q.r = r;
    q.row0 = a;
    q.m = max(b - a, 0);
    q.len = max(*GP(p.bnd, p.lens + r), 0);
    q.i0 = (int)max((long long)q.len - ((long long)end - first), -0x7fffffffLL);
    q.trow = p.table + (long long)r * p.cols;
    q.ring_lo = 0;
    const long long room = (long long)p.cols << p.page_log2;
    q.last = p.ring || q.len <= room ? 0x7fffffff : (int)room - 1;
    if (q.last != 0x7fffffff && threadIdx.x == 0) atomicOr(p.err, kErrInvalid);
    if (p.ring && q.len > 0) q.ring_lo = max(((q.len - 1) >> p.page_log2) - (p.cols - p.pinned) + 1, 0) << p.page_log2;
    return q;
}

// Positions that at least one of the queries a_lo..a_hi attends to, ascending:
// the sinks 0..nsink-1, then band_lo, band_lo + step, ...  With a key stride
// the queries have keys of their own, so the list is made for one (a_lo = a_hi).
struct KeyList {
    int count, nsink, band_lo, step;
    __device__ __forceinline__ int at(int u) const { return u < nsink ? u : band_lo + (u - nsink) * step; }
};

__device__ __forceinline__ KeyList keys_of(const DecodeArgs &p, const Request &q, int a_lo, int a_hi) {
    KeyList k;
    const int lo = q.i0 + a_lo, hi = min(q.i0 + a_hi, q.last);
    k.step = p.stride;
    k.nsink = max(min(p.n_sink, hi + 1), 0);
    int cnt = 0;
    k.band_lo = 0;
    if (p.stride == 1) {
        k.band_lo = (int)max((long long)lo - p.w, (long long)p.n_sink);
        cnt = max(hi - k.band_lo + 1, 0);
    } else if (lo >= p.n_sink) {
        k.band_lo = lo - min((lo - p.n_sink) / p.stride, p.w) * p.stride;
        if (k.band_lo <= hi) cnt = (hi - k.band_lo) / p.stride + 1;
    }
    k.count = k.nsink + cnt;
    return k;
}

// Does the query at position i attend to position j of such a list?
__device__ __forceinline__ bool attends(const DecodeArgs &p, int i, int j) {
    return j <= i && (j < p.n_sink || (long long)i - j <= (long long)p.w * p.stride);
}

// Line (row of head_dim values) of head kvh at row `off` of block `id`, or
// kNoLine: an absent column, or an id outside the cache (recorded).  The lines
// of a cache number less than 2^32 - 1 (checked by the caller).
constexpr uint32_t kNoLine = 0xffffffffu;
__device__ __forceinline__ uint32_t block_line(const DecodeArgs &p, int id, int off, int kvh) {
    if ((unsigned)id >= (unsigned)p.n_blocks) {
        if (id != -1) atomicOr(p.err, kErrInvalid);
        return kNoLine;
    }
    return (((uint32_t)id * (uint32_t)p.hk + (uint32_t)kvh) << p.page_log2) + (uint32_t)off;
}
// Column of position j of a list, or -1 when its block has been recycled.
__device__ __forceinline__ int key_column(const DecodeArgs &p, const Request &q, int j) {
    const int lb = j >> p.page_log2;
    if (lb >= p.pinned && j < q.ring_lo) return -1;
    return lb < p.cols ? lb : p.pinned + (lb - p.pinned) % (p.cols - p.pinned);
}
__device__ __forceinline__ uint32_t key_line(const DecodeArgs &p, const Request &q, int j, int kvh) {
    [[maybe_unused]] constexpr unsigned kSwabFile = kDecodeFile;
    const int col = key_column(p, q, j);
    return col < 0 ? kNoLine : block_line(p, *GP(p.bnd, q.trow + col), j & ((1 << p.page_log2) - 1), kvh);
}
__device__ __forceinline__ uint32_t prefix_line(const DecodeArgs &p, int j, int kvh) {
    [[maybe_unused]] constexpr unsigned kSwabFile = kDecodeFile;
    return block_line(p, *GP(p.bnd, p.ptable + (j >> p.page_log2)), j & ((1 << p.page_log2) - 1), kvh);
}

// A maximum leaves NaN out (fmaxf, max.f32), a sum keeps it: a row with keys
// whose scores are NaN has m = -inf and l = NaN, one without keys m = -inf and
// l = 0.  So it is the sum that says whether there was a key, and a part with m =
// -inf weighs 0 but its sum is still added (NaN * 0 is NaN).
__device__ __forceinline__ float inverse_of(float L) { return L == 0.f ? 0.f : 1.f / L; }
// log-sum-exp from the maximum (log2 units) and the sum
__device__ __forceinline__ float lse_of(float M, float L) {
    return L == 0.f ? -INFINITY : M * 0.6931471805599453f + logf(L);
}

}  // namespace swab
