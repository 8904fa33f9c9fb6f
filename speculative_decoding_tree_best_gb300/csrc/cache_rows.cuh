// cache_rows.cuh -- rows of keys and values in registers: 16-byte pieces as
// numbers, and the quotients of the 8-bit rows (paged_cache.cu, rope.cu).
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace spec {

namespace {

// lanes per row and values per lane: 16 bytes of the I/O type each
template <int IO, int D> struct geo {
    static constexpr int VEC = 16 / sizeof(typename io_t<IO>::T);
    static constexpr int LPR = D / VEC;
};

template <int IO>
__device__ __forceinline__ void unpack(const uint4& u,
                                       float (&x)[16 / sizeof(typename io_t<IO>::T)]) {
    if constexpr (IO == SPEC_IO_F32) {
        x[0] = __uint_as_float(u.x);
        x[1] = __uint_as_float(u.y);
        x[2] = __uint_as_float(u.z);
        x[3] = __uint_as_float(u.w);
    } else {
        const uint32_t r[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(r[i] << 16);
            x[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
        }
    }
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// x / y from r, 1 / y rounded: one Newton step on the quotient's remainder, which
// rounds it correctly (Markstein 1990).
__device__ __forceinline__ float quotient(float x, float y, float r) {
    const float q = x * r;
    return fmaf(fmaf(-q, y, x), r, q);
}

// two quotients by the same y
__device__ __forceinline__ float2 quotients(float2 x, float y, float r) {
    const float2 r2 = make_float2(r, r), q = __fmul2_rn(x, r2);
    return __ffma2_rn(__ffma2_rn(q, make_float2(-y, -y), x), r2, q);
}

// an 8-bit row's scale from its largest magnitude (the bits of it)
__device__ __forceinline__ float row_scale(uint32_t most) {
    float scale = fmaxf(quotient(__uint_as_float(most), 448.0f, 1.0f / 448.0f), 0x1p-100f);
    if (most == 0u) scale = 1.0f;
    if (most >= 0x7f800000u) scale = __uint_as_float(0x7fffffffu);
    return scale;
}

// e4m3 codes of four values by the scale and its rounded reciprocal (where the
// quotients' remainder underflows the code is 0 whatever it is)
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float scale,
                                           float inv) {
    const float2 lo = quotients(make_float2(a, b), scale, inv);
    const float2 hi = quotients(make_float2(c, d), scale, inv);
    return (uint32_t)__nv_cvt_float2_to_fp8x2(lo, __NV_SATFINITE, __NV_E4M3) |
           ((uint32_t)__nv_cvt_float2_to_fp8x2(hi, __NV_SATFINITE, __NV_E4M3) << 16);
}

// the 16-byte piece of rounded values
template <int IO>
__device__ __forceinline__ uint4 pack(const float (&x)[16 / sizeof(typename io_t<IO>::T)]) {
    if constexpr (IO == SPEC_IO_F32)
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                          __float_as_uint(x[3]));
    else
        return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                          pack_bf16(x[6], x[7]));
}

}  // namespace

}  // namespace spec
