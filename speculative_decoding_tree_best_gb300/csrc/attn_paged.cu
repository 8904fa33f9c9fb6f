// attn_paged.cu -- attention of a step's new tokens over the paged cache.
//
// One warp per (request, new token, q-head): one pass over the row's keys with
// the running maximum and sum of the softmax, the head dimension split over
// the lanes.
#include <math.h>

#include "paged.cuh"

namespace spec {

namespace {

constexpr int WARPS = 4;

template <int IO, int KV, int D>
__global__ void __launch_bounds__(32 * WARPS)
attn_rows(PageMap pm, int B, int T, int Hq, const typename io_t<IO>::T* __restrict__ q,
          const void* __restrict__ k_pages, const void* __restrict__ v_pages,
          const float* __restrict__ k_scale, const float* __restrict__ v_scale,
          const int32_t* __restrict__ n_new, typename io_t<IO>::T* __restrict__ o, float qk_scale,
          void* ws) {
    constexpr int E = D / 32;
    const int64_t w = (int64_t)blockIdx.x * WARPS + threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    if (w >= (int64_t)B * T * Hq) return;
    const int h = (int)(w % Hq);
    const int b = (int)(w / Hq / T), i = (int)(w / Hq % T);
    const int hk = h / (Hq / pm.Hkv);
    uint32_t bits = 0;
    const int n = new_rows(n_new, b, T, bits);
    int L = pm.kv_len[b];
    if (L < 0 || L > pm.cap() - n) {
        bits |= SPEC_DEV_OVERFLOW;
        L = L < 0 ? 0 : min(L, pm.cap());
    }
    const int end = i < n ? min(L + i + 1, pm.cap()) : 0;
    float qr[E], acc[E], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int j = 0; j < E; ++j) {
        qr[j] = io_t<IO>::ld(q, w * D + lane * E + j) * qk_scale;
        acc[j] = 0.0f;
    }
    using KT = typename kv_t<IO, KV>::T;
    const KT* kp = static_cast<const KT*>(k_pages);
    const KT* vp = static_cast<const KT*>(v_pages);
    for (int pos = 0; pos < end; ++pos) {
        const int64_t r = pm.row(b, pos, hk);
        if (r < 0) {
            bits |= SPEC_DEV_BADPAGE;
            continue;
        }
        float s = 0.0f, v[E];
#pragma unroll
        for (int j = 0; j < E; ++j) {
            if constexpr (KV == SPEC_KV_E4M3) {
                s += qr[j] * e4m3_to_float(kp[r * D + lane * E + j]);
                v[j] = e4m3_to_float(vp[r * D + lane * E + j]) * v_scale[r];
            } else {
                s += qr[j] * io_t<IO>::ld(kp, r * D + lane * E + j);
                v[j] = io_t<IO>::ld(vp, r * D + lane * E + j);
            }
        }
        s = warp_sum(s);
        if constexpr (KV == SPEC_KV_E4M3) s *= k_scale[r];
        const float nm = fmaxf(m, s), base = nm == -INFINITY ? 0.0f : nm;
        const float f = expf(m - base), p = expf(s - base);
        l = l * f + p;
#pragma unroll
        for (int j = 0; j < E; ++j) acc[j] = acc[j] * f + p * v[j];
        m = nm;
    }
#pragma unroll
    for (int j = 0; j < E; ++j) {
        const float x = l == 0.0f ? 0.0f : acc[j] / l;
        if (!(fabsf(x) <= 3.4028234663852886e38f)) bits |= SPEC_DEV_RANGE;
        io_t<IO>::st(o, w * D + lane * E + j, x);
    }
    if (bits) raise_status(ws, bits);
}

template <int IO, int KV, int D>
cudaError_t attn_t(const spec_paged_cfg& c, const spec_paged_kv& kv, const void* q,
                   const int32_t* n_new, void* o, void* ws, cudaStream_t st) {
    using T = typename io_t<IO>::T;
    const int64_t ctas = ((int64_t)c.B * c.T * c.Hq + WARPS - 1) / WARPS;
    return launch_k(false, attn_rows<IO, KV, D>, dim3((unsigned)ctas), dim3(32 * WARPS), 0, st,
                    page_map(c, kv), c.B, c.T, c.Hq, static_cast<const T*>(q), kv.k_pages,
                    kv.v_pages, kv.k_scale, kv.v_scale, n_new, static_cast<T*>(o),
                    1.0f / sqrtf((float)D), ws);
}

}  // namespace

cudaError_t launch_attn_paged(const spec_paged_cfg& c, const spec_paged_kv& kv, const void* q,
                              const int32_t* n_new, void* o, void* ws, cudaStream_t st) {
    SPEC_PAGED_DISPATCH(attn_t, c, kv, q, n_new, o, ws, st);
}

}  // namespace spec
