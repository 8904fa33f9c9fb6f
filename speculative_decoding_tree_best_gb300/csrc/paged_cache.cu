// paged_cache.cu -- the paged key/value cache written and read back.
//
// A row (one token's key or value of one head, D values) is handled by the
// lanes of one half- or quarter-warp group, 16 bytes of the I/O type per lane,
// so that its maximum is a few shuffles and its codes leave in one piece.
//
// Written with 8 bits: scale = max(amax / 448, 2^-100), code = e4m3(x / scale).
// 448 is e4m3's largest value, so the row's largest value keeps all three
// mantissa bits; a rounding is at most 2^-4 of a value (2^-10 scale below the
// normal range).  The floor keeps 1 / scale in fp32's range.  Rows of zeros
// take scale 1, rows with a non-finite value a NaN scale and NaN codes.
#include <math.h>

#include "paged.cuh"

namespace spec {

namespace {

constexpr int NT = 256;

// lanes per row and values per lane: 16 bytes of the I/O type each
template <int IO, int D> struct geo {
    static constexpr int VEC = 16 / sizeof(typename io_t<IO>::T);
    static constexpr int LPR = D / VEC;
};

template <int IO>
__device__ __forceinline__ void unpack(const uint4& u, float (&x)[16 / sizeof(typename io_t<IO>::T)]) {
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

template <int IO, int KV, int D>
__global__ void __launch_bounds__(NT)
append_rows(PageMap pm, int B, int T, const uint4* __restrict__ k_new,
            const uint4* __restrict__ v_new, const int32_t* __restrict__ n_new, void* k_pages,
            void* v_pages, float* k_scale, float* v_scale, void* ws) {
    using G = geo<IO, D>;
    const int64_t rows = (int64_t)B * T * pm.Hkv;
    const int64_t r = ((int64_t)blockIdx.x * NT + threadIdx.x) / G::LPR;
    const int lane = threadIdx.x % G::LPR;
    const bool is_v = blockIdx.y != 0;
    if (r >= rows) return;                         // whole row groups leave together
    const int h = (int)(r % pm.Hkv);
    const int64_t bi = r / pm.Hkv;
    const int b = (int)(bi / T), i = (int)(bi % T);
    uint32_t bits = 0;
    const int n = new_rows(n_new, b, T, bits);
    const int L = pm.kv_len[b];
    if (L < 0 || L > pm.cap() - n) bits |= SPEC_DEV_OVERFLOW;
    if (bits && lane == 0 && i == 0 && h == 0) raise_status(ws, bits);
    if ((bits & SPEC_DEV_OVERFLOW) || i >= n) return;
    const int64_t dst = pm.row(b, L + i, h);
    if (dst < 0) {
        if (lane == 0) raise_status(ws, SPEC_DEV_BADPAGE);
        return;
    }
    const uint4 u = (is_v ? v_new : k_new)[r * G::LPR + lane];
    void* pages = is_v ? v_pages : k_pages;
    if constexpr (KV == SPEC_KV_IO) {
        reinterpret_cast<uint4*>(pages)[dst * G::LPR + lane] = u;
    } else {
        float x[G::VEC], amax = 0.0f, bad = 0.0f;
        unpack<IO>(u, x);
#pragma unroll
        for (int j = 0; j < G::VEC; ++j) {
            amax = fmaxf(amax, fabsf(x[j]));
            bad += x[j] - x[j];                    // NaN for a non-finite value, else 0
        }
        const unsigned grp = G::LPR == 32 ? 0xffffffffu
                                          : ((1u << (G::LPR & 31)) - 1u)
                                                << ((threadIdx.x & 31) & ~(G::LPR - 1));
#pragma unroll
        for (int o = G::LPR / 2; o > 0; o >>= 1) {
            amax = fmaxf(amax, __shfl_xor_sync(grp, amax, o));
            bad += __shfl_xor_sync(grp, bad, o);
        }
        float scale = amax == 0.0f ? 1.0f : fmaxf(__fdiv_rn(amax, 448.0f), 0x1p-100f);
        if (bad != 0.0f) scale = __int_as_float(0x7fffffff);   // bad is 0 or NaN
        uint32_t w[G::VEC / 4];
#pragma unroll
        for (int j = 0; j < G::VEC / 4; ++j) {
            const float2 a = make_float2(__fdiv_rn(x[4 * j], scale), __fdiv_rn(x[4 * j + 1], scale));
            const float2 c = make_float2(__fdiv_rn(x[4 * j + 2], scale),
                                         __fdiv_rn(x[4 * j + 3], scale));
            w[j] = (uint32_t)__nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3) |
                   ((uint32_t)__nv_cvt_float2_to_fp8x2(c, __NV_SATFINITE, __NV_E4M3) << 16);
        }
        if constexpr (G::VEC == 8)
            reinterpret_cast<uint2*>(pages)[dst * G::LPR + lane] = make_uint2(w[0], w[1]);
        else
            reinterpret_cast<uint32_t*>(pages)[dst * G::LPR + lane] = w[0];
        if (lane == 0) (is_v ? v_scale : k_scale)[dst] = scale;
    }
}

template <int IO, int KV, int D>
__global__ void __launch_bounds__(NT)
read_rows(PageMap pm, int B, int Lmax, const void* __restrict__ k_pages,
          const void* __restrict__ v_pages, const float* __restrict__ k_scale,
          const float* __restrict__ v_scale, uint4* __restrict__ k_out, uint4* __restrict__ v_out,
          void* ws) {
    using G = geo<IO, D>;
    const int64_t rows = (int64_t)B * Lmax * pm.Hkv;
    const int64_t r = ((int64_t)blockIdx.x * NT + threadIdx.x) / G::LPR;
    const int lane = threadIdx.x % G::LPR;
    const bool is_v = blockIdx.y != 0;
    if (r >= rows) return;
    const int h = (int)(r % pm.Hkv);
    const int64_t bi = r / pm.Hkv;
    const int b = (int)(bi / Lmax), i = (int)(bi % Lmax);
    int L = pm.kv_len[b];
    const int most = min(Lmax, pm.cap());
    if (L < 0 || L > most) {
        if (lane == 0 && i == 0 && h == 0) raise_status(ws, SPEC_DEV_OVERFLOW);
        L = L < 0 ? 0 : most;
    }
    if (i >= L) return;
    const int64_t src = pm.row(b, i, h);
    if (src < 0) {
        if (lane == 0) raise_status(ws, SPEC_DEV_BADPAGE);
        return;
    }
    const void* pages = is_v ? v_pages : k_pages;
    uint4 u;
    if constexpr (KV == SPEC_KV_IO) {
        u = reinterpret_cast<const uint4*>(pages)[src * G::LPR + lane];
    } else {
        const float scale = (is_v ? v_scale : k_scale)[src];
        const uint8_t* cp = reinterpret_cast<const uint8_t*>(pages) + src * D + lane * G::VEC;
        uint32_t w[G::VEC / 4];
#pragma unroll
        for (int j = 0; j < G::VEC / 4; ++j) w[j] = reinterpret_cast<const uint32_t*>(cp)[j];
        float x[G::VEC];
#pragma unroll
        for (int j = 0; j < G::VEC; ++j)
            x[j] = e4m3_to_float((uint8_t)(w[j / 4] >> (8 * (j % 4)))) * scale;
        if constexpr (IO == SPEC_IO_F32)
            u = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                           __float_as_uint(x[3]));
        else
            u = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                           pack_bf16(x[6], x[7]));
    }
    (is_v ? v_out : k_out)[r * G::LPR + lane] = u;
}

template <int IO, int KV, int D>
cudaError_t append_t(const spec_paged_cfg& c, const spec_paged_kv& kv, const void* k_new,
                     const void* v_new, const int32_t* n_new, void* ws, cudaStream_t st) {
    const int64_t lanes = (int64_t)c.B * c.T * c.Hkv * geo<IO, D>::LPR;
    const int64_t ctas = (lanes + NT - 1) / NT;
    if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
    return launch_k(false, append_rows<IO, KV, D>, dim3((unsigned)ctas, 2), dim3(NT), 0, st,
                    page_map(c, kv), c.B, c.T, static_cast<const uint4*>(k_new),
                    static_cast<const uint4*>(v_new), n_new, kv.k_pages, kv.v_pages, kv.k_scale,
                    kv.v_scale, ws);
}

template <int IO, int KV, int D>
cudaError_t read_t(const spec_paged_cfg& c, const spec_paged_kv& kv, int Lmax, void* k_out,
                   void* v_out, void* ws, cudaStream_t st) {
    const int64_t lanes = (int64_t)c.B * Lmax * c.Hkv * geo<IO, D>::LPR;
    const int64_t ctas = (lanes + NT - 1) / NT;
    if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
    return launch_k(false, read_rows<IO, KV, D>, dim3((unsigned)ctas, 2), dim3(NT), 0, st,
                    page_map(c, kv), c.B, Lmax, kv.k_pages, kv.v_pages, kv.k_scale, kv.v_scale,
                    static_cast<uint4*>(k_out), static_cast<uint4*>(v_out), ws);
}

}  // namespace


cudaError_t launch_page_append(const spec_paged_cfg& c, const spec_paged_kv& kv, const void* k_new,
                               const void* v_new, const int32_t* n_new, void* ws,
                               cudaStream_t st) {
    SPEC_PAGED_DISPATCH(append_t, c, kv, k_new, v_new, n_new, ws, st);
}

cudaError_t launch_page_read(const spec_paged_cfg& c, const spec_paged_kv& kv, int Lmax,
                             void* k_out, void* v_out, void* ws, cudaStream_t st) {
    SPEC_PAGED_DISPATCH(read_t, c, kv, Lmax, k_out, v_out, ws, st);
}

}  // namespace spec
