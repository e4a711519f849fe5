// k_cache.cu -- block tables and slot maps from request lengths.
//
// With have = ceil(len / page) and want = ceil((len + new) / page) columns
// (both at most `cols`), two running sums over the requests place everything:
// the sum of `new` is where a request's tokens start in the flat batch, the
// sum of want - have is where its blocks start in the free list.  Latency-
// bound (a step of 64 requests moves 1.5 KB), so one launch does it all and no
// block waits for another: every block repeats the two sums over all the
// requests (a request a thread, 1024 at a time) and then writes its own share
// of the new table columns and of the tokens, each finding its request by
// binary search in the sums held in shared memory.  A new column is read from
// the free list itself, never from the table that another block may be
// writing.  64 requests, a token each: 4.3 us in a graph, of which an empty
// launch is 2.2; 256 requests with 64k tokens (63 blocks): 5.0 us.
#include "swab_internal.h"

static constexpr unsigned kSwabFile = 12;   // site id of the bounds checks

namespace swab {
namespace {

constexpr int kThreads = 1024;

struct Chunk {                       // the requests of one pass
    long long tok[kThreads + 1];     // running sum of new tokens
    long long blk[kThreads + 1];     // running sum of blocks wanted
    int len[kThreads], have[kThreads], fresh[kThreads];   // fresh = -1: not served
    int total[kThreads];
    long long wsum[2][32];
};

// last r in [0, n) with sum[r] <= x (sum[0] <= x < sum[n])
__device__ __forceinline__ int owner(const long long *sum, int n, long long x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sum[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ int clamp32(long long x) { return x > 0x7fffffffLL ? 0x7fffffff : (int)x; }

// exclusive running sums of (a, b) over the block, plus the carried-in start
__device__ __forceinline__ void scan2(long long &a, long long &b, Chunk &c, long long a0, long long b0) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long va = a, vb = b;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long ya = __shfl_up_sync(0xffffffffu, a, d), yb = __shfl_up_sync(0xffffffffu, b, d);
        if (lane >= d) {
            a += ya;
            b += yb;
        }
    }
    if (lane == 31) {
        c.wsum[0][warp] = a;
        c.wsum[1][warp] = b;
    }
    __syncthreads();
    if (warp == 0) {                     // the warps' sums, summed the same way
        long long wa = c.wsum[0][lane], wb = c.wsum[1][lane];
        const long long ua = wa, ub = wb;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long ya = __shfl_up_sync(0xffffffffu, wa, d), yb = __shfl_up_sync(0xffffffffu, wb, d);
            if (lane >= d) {
                wa += ya;
                wb += yb;
            }
        }
        c.wsum[0][lane] = a0 + wa - ua;
        c.wsum[1][lane] = b0 + wb - ub;
    }
    __syncthreads();
    a += c.wsum[0][warp];
    b += c.wsum[1][warp];
    c.tok[threadIdx.x + 1] = a;
    c.blk[threadIdx.x + 1] = b;
    if (threadIdx.x == 0) {
        c.tok[0] = a0;
        c.blk[0] = b0;
    }
    a -= va;
    b -= vb;
}

__global__ void __launch_bounds__(kThreads) k_cache_slots(const __grid_constant__ CacheSlotsArgs p) {
    __shared__ Chunk c;
    __shared__ unsigned long long sh_taken, sh_missing;
    const int tid = threadIdx.x;
    pdl_wait();
    pdl_trigger();
    const int used0 = max(*GP(p.bnd, p.used), 0);
    const long long avail = p.n_free > used0 ? p.n_free - used0 : 0;
    if (tid == 0) sh_taken = sh_missing = 0;
    // this block's share of the tokens
    const long long per = ((long long)p.tokens + gridDim.x - 1) / gridDim.x;
    const long long t_lo = min((long long)p.tokens, per * blockIdx.x), t_hi = min((long long)p.tokens, t_lo + per);
    const int page = 1 << p.page_log2, cyc = p.cols - p.pinned;
    long long tok0 = 0, blk0 = 0;

    for (int r0 = 0; r0 < p.batch; r0 += kThreads) {
        const int r = r0 + tid, nr = min(kThreads, p.batch - r0);
        long long m = 0, need = 0, total = 0, over = 0;
        int len = 0, have = 0;
        bool fits = true, many = false;
        if (tid < nr) {
            len = max(*GP(p.bnd, p.lens + r), 0);
            m = max(*GP(p.bnd, p.n_new + r), 0);
            total = len + m;
            const long long hb = ((long long)len + page - 1) >> p.page_log2, wb = (total + page - 1) >> p.page_log2;
            have = (int)min(hb, (long long)p.cols);
            many = p.max_new > 0 && m > p.max_new;
            fits = total <= 0x7fffffffLL && (p.ring || wb <= p.cols) && !many;
            if (fits) need = min(wb, (long long)p.cols) - have;
            else over = max(wb - p.cols, 1LL);
        }
        long long ts = m, bs = need;
        __syncthreads();                 // the previous pass has read the chunk
        scan2(ts, bs, c, tok0, blk0);
        // (a request past the rows takes no block, and none after it does)
        const bool rows = p.max_new == 0 || m == 0 || ts + m <= p.tokens;
        const bool served = fits && rows && (need == 0 || bs + need <= avail);
        c.len[tid] = len;
        c.have[tid] = have;
        c.total[tid] = served ? (int)total : 0;
        c.fresh[tid] = served ? (int)need : -1;
        if (tid < nr && p.state) {
            if (blockIdx.x == 0) {
                *GP(p.bnd, p.q_start + r) = clamp32(ts);
                *GP(p.bnd, p.lens_out + r) = served ? (int)total : len;
                if (served && need) atomicMax(&sh_taken, (unsigned long long)(bs + need));
                if (!served) atomicAdd(&sh_missing, (unsigned long long)max(need + over, 1LL));
                if (many || !rows) atomicOr(p.err, kErrInvalid);
            }
        }
        __syncthreads();
        tok0 = c.tok[kThreads];
        blk0 = c.blk[kThreads];
        if (p.table_pass) {
            // new table columns: the blocks of the list in order, spread over the grid
            const long long b_hi = min(c.blk[nr], avail);
            for (long long x = c.blk[0] + (long long)blockIdx.x * kThreads + tid; x < b_hi; x += (long long)gridDim.x * kThreads) {
                const int q = owner(c.blk, nr, x);
                if (c.fresh[q] <= 0) continue;
                const long long at = (long long)(r0 + q) * p.cols + c.have[q] + (x - c.blk[q]);
                *GP(p.bnd, p.table + at) = *GP(p.bnd, p.free_list + used0 + x);
            }
            // this block's tokens among the chunk's
            const long long e_hi = min(t_hi, c.tok[nr]);
            for (long long t = max(t_lo, c.tok[0]) + tid; t < e_hi; t += kThreads) {
                const int q = owner(c.tok, nr, t);
                const long long j = c.len[q] + (t - c.tok[q]);
                int slot = -1;
                const int fresh = c.fresh[q];
                if (fresh >= 0) {
                    const int lb = (int)(j >> p.page_log2), last = (c.total[q] - 1) >> p.page_log2;
                    const int col = lb < p.cols ? lb : p.pinned + (lb - p.pinned) % cyc;
                    // a block that this very step recycles again keeps its last round only
                    if (lb < p.pinned || lb > last - cyc) {
                        const int id = col >= c.have[q] ? *GP(p.bnd, p.free_list + used0 + c.blk[q] + (col - c.have[q]))
                                                        : *GP(p.bnd, p.table + (long long)(r0 + q) * p.cols + col);
                        if (id >= 0 && id < p.n_blocks) slot = (id << p.page_log2) + (int)(j & (page - 1));
                        else atomicOr(p.err, kErrInvalid);
                    }
                }
                *GP(p.bnd, p.slots + t) = slot;
                *GP(p.bnd, p.pos + t) = clamp32(j + p.pos0);
            }
        }
    }
    if (p.table_pass)
        for (long long t = max(t_lo, tok0) + tid; t < t_hi; t += kThreads) {   // padding
            *GP(p.bnd, p.slots + t) = -1;
            *GP(p.bnd, p.pos + t) = 0;
        }
    __syncthreads();
    if (p.state && blockIdx.x == 0 && tid == 0) {
        *GP(p.bnd, p.q_start + p.batch) = clamp32(tok0);
        *GP(p.bnd, p.used_out) = used0 + (int)sh_taken;
        *GP(p.bnd, p.used_out + 1) = clamp32((long long)sh_missing);
    }
}

}  // namespace

cudaError_t launch_cache_slots(CacheSlotsArgs a, cudaStream_t st) {
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidValue;
    const long long want = ((long long)a.tokens + kThreads - 1) / kThreads;
    const int blocks = (int)(want < 1 ? 1 : want < 2LL * sms ? want : 2LL * sms);
    // Lengths or counters updated in place must not change while another block
    // still reads them: with several blocks they are written by a second launch.
    const bool in_place = a.lens_out == a.lens || a.used_out == a.used;
    a.table_pass = 1;
    a.state = !(in_place && blocks > 1);
    cudaError_t e = launch_dependent(&k_cache_slots, dim3((unsigned)blocks), kThreads, 0, st, a);
    if (e == cudaSuccess && !a.state) {
        a.table_pass = 0;
        a.state = 1;
        e = launch_dependent(&k_cache_slots, dim3(1), kThreads, 0, st, a);
    }
    return e;
}

}  // namespace swab
