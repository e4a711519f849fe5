// swab_rows.cuh -- what the kernels over the rows of heads share (rotary
// positions, norms, the cache write): 16 bytes of a row at a time, and the angle
// of a position.
#pragma once

#include "swab_internal.h"

namespace swab {

template <typename T> struct VecOf {
    static constexpr int kN = 16 / sizeof(T);   // elements of 16 bytes
};

template <typename T>
__device__ __forceinline__ void unpack16(const uint4 &v, float *f) {
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
template <typename T>
__device__ __forceinline__ uint4 pack16(const float *f) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (sizeof(T) == 4) w[k] = __float_as_uint(f[k]);
        else w[k] = pack2<T>(f[2 * k], f[2 * k + 1]);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 load16(const void *p) { return *reinterpret_cast<const uint4 *>(p); }

// N floats of the table, 16 or 8 bytes at a time
template <int N>
__device__ __forceinline__ void take(const float *src, float (&f)[N]) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int k = 0; k < N; k += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(src + k);
            f[k] = v.x, f[k + 1] = v.y, f[k + 2] = v.z, f[k + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < N; k += 2) {
            const float2 v = *reinterpret_cast<const float2 *>(src + k);
            f[k] = v.x, f[k + 1] = v.y;
        }
    }
}

// Cosine and sine of 2 pi frac(at * turns / 2^64): the upper 32 bits of the
// fraction of a turn, less the nearest quarter, so that at most an eighth of a
// turn is rounded to a float, not the whole angle.
__device__ __forceinline__ void cos_sin(long long at, unsigned long long turns, float &cs, float &sn) {
    const unsigned frac = (unsigned)(((unsigned long long)at * turns) >> 32);
    const unsigned quarter = (frac + 0x20000000u) >> 30;
    sincospif((float)(int)(frac - (quarter << 30)) * 0x1p-31f, &sn, &cs);
    if (quarter & 1u) {
        const float x = cs;
        cs = -sn;
        sn = x;
    }
    if (quarter & 2u) {
        cs = -cs;
        sn = -sn;
    }
}

}  // namespace swab
