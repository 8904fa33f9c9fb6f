// serving.cuh -- checks and launchers of the calls around a serving step: page
// tables (page_tables.cu), rotary positions (rope.cu), sampling (token_sample.cu).
#pragma once

#include "paged.cuh"

namespace spec {

inline int check_pool(const spec_page_pool* p) {
    if (!p || !al16(p->page_table) || !al16(p->kv_len) || !al16(p->free_list) ||
        !al16(p->n_free) || !al16(p->n_held))
        return ST_EINVAL;
    return ST_OK;
}

inline int check_rope_cfg(const spec_rope_cfg* c, bool append) {
    if (!c) return ST_EINVAL;
    if (c->rows < 1 || c->Hq < 1 || c->Hkv < (append ? 1 : 0)) return ST_EINVAL;
    if ((int64_t)c->Hq + 2 * (int64_t)c->Hkv > (1 << 16)) return ST_EINVAL;
    if ((int64_t)c->rows * (c->Hq + 2 * c->Hkv) >= (1LL << 37)) return ST_EINVAL;
    if (c->D != 64 && c->D != 128) return ST_EINVAL;
    if (c->rot < 16 || c->rot > c->D || c->rot % 16 != 0) return ST_EINVAL;
    if (c->layout != SPEC_ROPE_HALF && c->layout != SPEC_ROPE_INTERLEAVED) return ST_EINVAL;
    if (c->inverse != 0 && c->inverse != 1) return ST_EINVAL;
    if (c->io_dtype != SPEC_IO_F32 && c->io_dtype != SPEC_IO_BF16) return ST_EUNSUPPORTED;
    const int vec = c->io_dtype == SPEC_IO_BF16 ? 8 : 4;
    const int64_t stride[3] = {c->q_stride, c->k_stride, c->v_stride};
    for (int i = 0; i < 3; ++i) {
        const int64_t least = (int64_t)(i ? c->Hkv : c->Hq) * c->D;
        if (stride[i] != 0 && (stride[i] < least || stride[i] % vec != 0 || stride[i] > (1LL << 31)))
            return ST_EINVAL;
    }
    return ST_OK;
}

inline int check_sample_cfg(const spec_sample_cfg* c) {
    if (!c) return ST_EINVAL;
    if (c->R < 1 || c->R > (1 << 20) || c->V < 1 || c->V > SPEC_MAX_SAMPLE_V || c->per < 1)
        return ST_EINVAL;
    if (c->io_dtype != SPEC_IO_F32 && c->io_dtype != SPEC_IO_BF16) return ST_EUNSUPPORTED;
    return ST_OK;
}

cudaError_t launch_pages_extend(const spec_paged_cfg& c, const spec_page_pool& p,
                                const int32_t* n_new, int64_t* slots, int32_t* n_ok, void* ws,
                                cudaStream_t st);
cudaError_t launch_pages_trim(const spec_paged_cfg& c, const spec_page_pool& p,
                              const int32_t* keep, void* ws, cudaStream_t st);
cudaError_t launch_rope(const spec_rope_cfg& c, const uint64_t* turns, float amp,
                        const int32_t* pos, const void* q, const void* k, void* q_out,
                        void* k_out, cudaStream_t st);
cudaError_t launch_rope_append(const spec_rope_cfg& c, const spec_paged_cfg& pc,
                               const spec_paged_kv& kv, const uint64_t* turns, float amp,
                               const int64_t* slots, const void* q, const void* k_new,
                               const void* v_new, void* q_out, void* ws, cudaStream_t st);
cudaError_t launch_token_sample(const spec_sample_cfg& c, const void* logits,
                                const spec_sample_params& p, const float* e,
                                const spec_sample_out& out, void* ws, cudaStream_t st);

}  // namespace spec
