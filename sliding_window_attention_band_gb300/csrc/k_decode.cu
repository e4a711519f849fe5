// k_decode.cu -- banded attention of a few new tokens a request over the paged
// cache: the general kernel (every type and head size) and the joining of the
// parts of a split key axis.
//
// A query's keys are a list: the shared prefix, the leading global tokens, the
// band (ascending).  The list is cut into pieces; a block takes a request, up to
// four query heads of a key head and a piece, and runs through it once with the running maximum m and
// sum l of the softmax, in log2 units and fp32:
//     m' = max(m, x),  l' = l 2^(m - m') + 2^(x - m'),  o' = o 2^(m - m') + 2^(x - m') v.
// The pieces are joined as O = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s.
// fp32 is exact to fp32 rounding here (no tf32).  HBM-bound with a head of its
// own (16 requests of 3 to 5k, 12 heads of 64, fp32: 62 us, 6.0 TB/s), bound by
// instructions where a key serves several heads (24 heads of 96 over 8, bf16:
// 122 us, a quarter of the copy rate); joining 57 parts of 32 heads takes 5 us.
#include "swab_internal.h"
#include "swab_decode.cuh"

static constexpr unsigned kSwabFile = 13;   // site id of the bounds checks

namespace swab {
namespace {

constexpr int kThreads = 128;

template <typename T>
__device__ __forceinline__ void widen16(const uint4 &v, float *f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (sizeof(T) == 4) {
            f[k] = __uint_as_float(w[k]);
        } else {
            f[2 * k] = lo16<T>(w[k]);
            f[2 * k + 1] = hi16<T>(w[k]);
        }
    }
}

// A key belongs to a group of kLanes lanes, 16 bytes of its row a lane (kVec
// times when the row has more than 32 pieces); kThreads / kLanes keys at a time.
// A block answers kR query heads that share the key head, so a key is loaded
// once for them.
// Blocks an SM holds: the plan cuts the lists for 8.  Left to itself the compiler
// gave one query head 52 to 72 registers and four of them 96 to 168, by what the
// code around the loop happened to be, and the loads in flight went with them (16
// requests of 3 to 5k, 12 heads of 64, fp32: 67 to 83 us, 62 with 8 blocks; 12
// of 96 in 16 bits 83 to 104, 69; 24 over 8 of 96 in 16 bits 120 to 134, 122 with 4).
// Fewer where that would spill: 4 lanes a key are 32 keys at a time.
template <typename T, int kLanes, int kR>
constexpr int kResident = kR == 1 ? (kLanes == 4 ? 6 : 8) : sizeof(T) == 2 && kLanes == 4 ? 3 : 4;

template <typename T, int kLanes, int kVec, int kR>
__global__ void __launch_bounds__(kThreads, kResident<T, kLanes, kR>) k_decode_general(const __grid_constant__ DecodeArgs p) {
    constexpr int kV = 16 / sizeof(T), kE = kV * kVec, kGroups = kThreads / kLanes, kU = kVec == 1 ? 4 : 2;
    __shared__ float so[kGroups][kLanes * kE];
    __shared__ float2 sml[kGroups];
    const int per = (p.group + kR - 1) / kR;                       // blocks of a key head
    const int split = blockIdx.x, kvh = blockIdx.y / per, g0 = blockIdx.y % per * kR, r = blockIdx.z;
    const int head0 = kvh * p.group + g0, nr = min(kR, p.group - g0);
    const int sub = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
    const int pieces = p.hd / kV;
    pdl_wait();
    pdl_trigger();
    const Request q = request_of(p, r);
    for (int a = 0; a < q.m; ++a) {
        const KeyList keys = keys_of(p, q, a, a);
        const long long n = (long long)keys.count + p.prefix_len, lo = (long long)split * p.chunk;
        const long long hi = split == p.nsplit - 1 ? n : min(n, lo + p.chunk);
        const long long row = q.row0 + a;
        float qf[kR][kE], o[kR][kE], m[kR], l[kR];
#pragma unroll
        for (int t = 0; t < kR; ++t) {
            m[t] = -INFINITY;
            l[t] = 0.f;
            const T *qrow = reinterpret_cast<const T *>(p.Q) + row * p.q_stride + (long long)(head0 + min(t, nr - 1)) * p.hd;
#pragma unroll
            for (int v = 0; v < kVec; ++v) {
                const int piece = lane + v * kLanes;
                uint4 raw = make_uint4(0, 0, 0, 0);
                if (piece < pieces) raw = *reinterpret_cast<const uint4 *>(GPN(p.bnd, qrow + piece * kV, 16));
                widen16<T>(raw, qf[t] + v * kV);
            }
#pragma unroll
            for (int e = 0; e < kE; ++e) o[t][e] = 0.f;
        }
        // every lane group makes the same number of steps (the shuffles below
        // need the whole warp), kU keys a step with all their loads in flight
        const long long span = hi - lo;
        const int steps = span > 0 ? (int)((span + kGroups * kU - 1) / (kGroups * kU)) : 0;
        for (int s = 0; s < steps; ++s) {
            uint32_t line[kU];
            uint4 kr[kU][kVec], vr[kU][kVec];
#pragma unroll
            for (int i = 0; i < kU; ++i) {
                const long long u = lo + ((long long)s * kU + i) * kGroups + sub;
                line[i] = kNoLine;
                if (u < hi) line[i] = u < p.prefix_len ? prefix_line(p, (int)u, kvh) : key_line(p, q, keys.at((int)(u - p.prefix_len)), kvh);
            }
#pragma unroll
            for (int i = 0; i < kU; ++i)
#pragma unroll
                for (int v = 0; v < kVec; ++v) {
                    const int piece = lane + v * kLanes;
                    kr[i][v] = vr[i][v] = make_uint4(0, 0, 0, 0);
                    if (line[i] != kNoLine && piece < pieces) {
                        const long long at = (long long)line[i] * p.hd + piece * kV;
                        kr[i][v] = ldg16(GPN(p.bnd, reinterpret_cast<const T *>(p.Kc) + at, 16));
                        vr[i][v] = ldg16(GPN(p.bnd, reinterpret_cast<const T *>(p.Vc) + at, 16));
                    }
                }
            float x[kR][kU];
#pragma unroll
            for (int i = 0; i < kU; ++i) {
                float kf[kE];
#pragma unroll
                for (int v = 0; v < kVec; ++v) widen16<T>(kr[i][v], kf + v * kV);
#pragma unroll
                for (int t = 0; t < kR; ++t) {
                    x[t][i] = 0.f;
#pragma unroll
                    for (int e = 0; e < kE; ++e) x[t][i] = fmaf(qf[t][e], kf[e], x[t][i]);
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
                for (int e = 0; e < kE; ++e) o[t][e] *= corr;
#pragma unroll
                for (int i = 0; i < kU; ++i) {
                    x[t][i] = exp2f(x[t][i] - mb);                           // 0 for an absent key
                    l[t] += x[t][i];
                }
            }
#pragma unroll
            for (int i = 0; i < kU; ++i) {
                float vf[kE];
#pragma unroll
                for (int v = 0; v < kVec; ++v) widen16<T>(vr[i][v], vf + v * kV);
#pragma unroll
                for (int t = 0; t < kR; ++t)
#pragma unroll
                    for (int e = 0; e < kE; ++e) o[t][e] = fmaf(x[t][i], vf[e], o[t][e]);
            }
        }
#pragma unroll
        for (int t = 0; t < kR; ++t) {
            if (t >= nr) break;
            __syncthreads();             // the previous head's reads of the buffers
#pragma unroll
            for (int e = 0; e < kE; ++e) so[sub][lane * kE + e] = o[t][e];
            if (lane == 0) sml[sub] = make_float2(m[t], l[t]);
            __syncthreads();
            float M = -INFINITY, L = 0.f;
            for (int g = 0; g < kGroups; ++g) M = fmaxf(M, sml[g].x);
            for (int g = 0; g < kGroups; ++g) L = fmaf(sml[g].y, sml[g].x == -INFINITY ? 0.f : exp2f(sml[g].x - M), L);
            const int head = head0 + t;
            const long long th = row * p.h + head;
            for (int c = threadIdx.x; c < p.hd; c += kThreads) {
                const int piece = c / kV, at = piece % kLanes * kE + piece / kLanes * kV + c % kV;
                float y = 0.f;
                for (int g = 0; g < kGroups; ++g) y = fmaf(so[g][at], sml[g].x == -INFINITY ? 0.f : exp2f(sml[g].x - M), y);
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

// Joins the parts of one (token, head): kW warps share them (a warp where there
// are few; four, over shared memory, where a long context was cut into many).
// A lane holds 4 adjacent channels, and 4 more of heads over 128.
template <typename T, int kW>
__global__ void __launch_bounds__(kThreads) k_decode_join(const __grid_constant__ DecodeArgs p) {
    constexpr int kPairs = kThreads / 32 / kW, kVecs = 2, kFlight = 8;      // head_dim <= 256
    __shared__ float4 so[kW > 1 ? kW : 1][kVecs * 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part0 = warp % kW;
    const long long th = (long long)blockIdx.x * kPairs + warp / kW;
    const long long row = th / p.h;
    const int head = (int)(th - row * p.h);
    if (row >= p.tokens) return;                                  // with kW = 4: the whole block
    const float2 *ml = p.pml + th * p.nparts;
    const float *po = p.po + th * p.nparts * p.hd;
    pdl_wait();                                                   // the parts are there
    pdl_trigger();
    // the requests' rows (a first start behind the second one says nothing of the others)
    const int start = *GP(p.bnd, p.q_start), first = start <= *GP(p.bnd, p.q_start + 1) ? start : 0;
    const int live = *GP(p.bnd, p.q_start + p.batch);
    float M = -INFINITY, L = 0.f;
    const float2 none = make_float2(-INFINITY, 0.f);
    // the first 64 parts' (max, sum), two a lane
    const float2 near[2] = {lane < p.nparts ? *GP(p.bnd, ml + lane) : none, lane + 32 < p.nparts ? *GP(p.bnd, ml + lane + 32) : none};
    M = fmaxf(near[0].x, near[1].x);
    for (int s = 64 + lane; s < p.nparts; s += 32) M = fmaxf(M, GP(p.bnd, ml + s)->x);
    if (row < first || row >= live) return;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    float4 o[kVecs];
#pragma unroll
    for (int e = 0; e < kVecs; ++e) o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    // 32 parts at a time, a weight a lane, so that the loads of the values
    // depend on no load before them; eight of them in flight
    for (int s0 = 0; s0 < p.nparts; s0 += 32) {
        const int left = min(p.nparts - s0, 32);
        const float2 v = s0 == 0 ? near[0] : s0 == 32 ? near[1] : lane < left ? *GP(p.bnd, ml + s0 + lane) : none;
        const float mine = v.x == -INFINITY ? 0.f : exp2f(v.x - M);
        L = fmaf(v.y, mine, L);
        for (int k0 = part0; k0 < left; k0 += kFlight * kW) {
#pragma unroll
            for (int e = 0; e < kVecs; ++e) {
                const int c = 4 * (lane + 32 * e);
                if (32 * 4 * e >= p.hd) break;
                float4 x[kFlight];
                float f[kFlight];
#pragma unroll
                for (int i = 0; i < kFlight; ++i) {
                    const int k = k0 + i * kW;
                    f[i] = __shfl_sync(0xffffffffu, mine, k & 31);
                    if (k >= left) f[i] = 0.f;
                    x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    // (the values of an empty part are not written)
                    if (f[i] != 0.f && c < p.hd) x[i] = *reinterpret_cast<const float4 *>(GPN(p.bnd, po + (long long)(s0 + k) * p.hd + c, 16));
                }
#pragma unroll
                for (int i = 0; i < kFlight; ++i) {
                    o[e].x = fmaf(x[i].x, f[i], o[e].x);
                    o[e].y = fmaf(x[i].y, f[i], o[e].y);
                    o[e].z = fmaf(x[i].z, f[i], o[e].z);
                    o[e].w = fmaf(x[i].w, f[i], o[e].w);
                }
            }
        }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) L += __shfl_xor_sync(0xffffffffu, L, d);
    if constexpr (kW > 1) {
#pragma unroll
        for (int e = 0; e < kVecs; ++e) so[warp][lane + 32 * e] = o[e];
        __syncthreads();
        if (warp > 0) return;
#pragma unroll
        for (int e = 0; e < kVecs; ++e)
#pragma unroll
            for (int w = 1; w < kW; ++w) {
                const float4 x = so[w][lane + 32 * e];
                o[e].x += x.x;
                o[e].y += x.y;
                o[e].z += x.z;
                o[e].w += x.w;
            }
    }
    const float inv = inverse_of(L);
    T *out = reinterpret_cast<T *>(p.O) + row * p.o_stride + (long long)head * p.hd;
#pragma unroll
    for (int e = 0; e < kVecs; ++e) {
        const int c = 4 * (lane + 32 * e);
        if (c >= p.hd) break;
        const float4 y = make_float4(o[e].x * inv, o[e].y * inv, o[e].z * inv, o[e].w * inv);
        if constexpr (sizeof(T) == 4) *reinterpret_cast<float4 *>(GPN(p.bnd, out + c, 16)) = y;
        else *reinterpret_cast<uint2 *>(GPN(p.bnd, out + c, 8)) = make_uint2(pack2<T>(y.x, y.y), pack2<T>(y.z, y.w));
    }
    if (lane == 0 && p.lse) *GP(p.bnd, p.lse + th) = lse_of(M, L);
}

template <typename T, int kR>
cudaError_t launch_general_r(const DecodeArgs &a, cudaStream_t st) {
    const dim3 grid((unsigned)a.nsplit, (unsigned)(a.hk * ((a.group + kR - 1) / kR)), (unsigned)a.batch);
    const int pieces = a.hd * (int)sizeof(T) / 16;
    if (pieces <= 4) return launch_dependent(&k_decode_general<T, 4, 1, kR>, grid, kThreads, 0, st, a);
    if (pieces <= 8) return launch_dependent(&k_decode_general<T, 8, 1, kR>, grid, kThreads, 0, st, a);
    if (pieces <= 16) return launch_dependent(&k_decode_general<T, 16, 1, kR>, grid, kThreads, 0, st, a);
    if constexpr (sizeof(T) == 4)
        if (pieces > 32) return launch_dependent(&k_decode_general<T, 32, 2, kR>, grid, kThreads, 0, st, a);
    return launch_dependent(&k_decode_general<T, 32, 1, kR>, grid, kThreads, 0, st, a);
}

template <typename T>
cudaError_t launch_general_t(const DecodeArgs &a, cudaStream_t st) {
    return a.group == 1 ? launch_general_r<T, 1>(a, st) : launch_general_r<T, 4>(a, st);
}

template <typename T>
cudaError_t launch_join_t(const DecodeArgs &a, cudaStream_t st) {
    const long long pairs = (long long)a.tokens * a.h;
    if (a.nparts > 8 && pairs <= 2048) return launch_dependent(&k_decode_join<T, 4>, dim3((unsigned)pairs), kThreads, 0, st, a);
    return launch_dependent(&k_decode_join<T, 1>, dim3((unsigned)((pairs + 3) / 4)), kThreads, 0, st, a);
}

}  // namespace

cudaError_t launch_decode_general(DType dt, const DecodeArgs &a, cudaStream_t st) {
    return dt == kF32 ? launch_general_t<float>(a, st) : dt == kF16 ? launch_general_t<__half>(a, st) : launch_general_t<__nv_bfloat16>(a, st);
}

cudaError_t launch_decode_join(DType dt, const DecodeArgs &a, cudaStream_t st) {
    return dt == kF32 ? launch_join_t<float>(a, st) : dt == kF16 ? launch_join_t<__half>(a, st) : launch_join_t<__nv_bfloat16>(a, st);
}

}  // namespace swab
