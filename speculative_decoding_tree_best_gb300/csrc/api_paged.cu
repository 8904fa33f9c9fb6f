// api_paged.cu -- the extern "C" boundary of the paged-cache calls and the
// chain verification: argument checks, workspace sizing, launches.
#include <stdint.h>

#include "kernels.h"
#include "paged.cuh"

namespace {

using spec::al16;

int cuda_rc(cudaError_t e) {
    if (e == cudaSuccess) return ST_OK;
    if (e == cudaErrorInvalidConfiguration) return ST_EUNSUPPORTED;
    return ST_ECUDA;
}

}  // namespace

extern "C" {

size_t spec_paged_workspace_bytes(const spec_paged_cfg* cfg, int num_sms) {
    if (spec::check_paged_cfg(cfg) != ST_OK || num_sms < 0) return 0;
    if (num_sms == 0) num_sms = spec::device_sm_count();
    return num_sms < 1 ? 0 : spec::paged_ws_layout(*cfg, num_sms).total;
}

size_t spec_draft_workspace_bytes(const spec_draft_cfg* cfg, int num_sms) {
    if (spec::check_draft_cfg(cfg) != ST_OK || num_sms < 0) return 0;
    if (num_sms == 0) num_sms = spec::device_sm_count();
    return num_sms < 1 ? 0 : spec::draft_ws_layout(*cfg, num_sms).total;
}

int kv_page_append(const spec_paged_cfg* cfg, const spec_paged_kv* kv, const void* k_new,
                   const void* v_new, const int32_t* n_new, void* ws, void* stream) {
    int rc = spec::check_paged_cfg(cfg);
    if (rc) return rc;
    if ((rc = spec::check_paged_kv(*cfg, kv))) return rc;
    if (!al16(k_new) || !al16(v_new) || !al16(ws) || (n_new && !al16(n_new))) return ST_EINVAL;
    return cuda_rc(spec::launch_page_append(*cfg, *kv, k_new, v_new, n_new, ws,
                                            static_cast<cudaStream_t>(stream)));
}

int kv_page_read(const spec_paged_cfg* cfg, const spec_paged_kv* kv, int Lmax, void* k_out,
                 void* v_out, void* ws, void* stream) {
    int rc = spec::check_paged_cfg(cfg);
    if (rc) return rc;
    if ((rc = spec::check_paged_kv(*cfg, kv))) return rc;
    if (Lmax < 1 || Lmax > (1 << 30) || !al16(k_out) || !al16(v_out) || !al16(ws)) return ST_EINVAL;
    return cuda_rc(spec::launch_page_read(*cfg, *kv, Lmax, k_out, v_out, ws,
                                          static_cast<cudaStream_t>(stream)));
}

int attn_decode_paged(const spec_paged_cfg* cfg, const spec_paged_kv* kv, const void* q,
                      const int32_t* n_new, void* o, void* ws, void* stream) {
    int rc = spec::check_paged_cfg(cfg);
    if (rc) return rc;
    if ((rc = spec::check_paged_kv(*cfg, kv))) return rc;
    if (cfg->T > SPEC_MAX_ROWS || (int64_t)cfg->T * (cfg->Hq / cfg->Hkv) > 65536) return ST_EINVAL;
    // granules, each as often as a row group has tiles, are counted in 32 bits
    const int64_t per_req = ((int64_t)cfg->max_pages * cfg->page + 31) / 32 * 3;
    const int64_t segs = (int64_t)cfg->Hkv * spec::paged_row_tiles(*cfg).rtg;
    if (cfg->B * (per_req + 24) > 0x7fffffff / segs) return ST_EINVAL;
    if (!al16(q) || !al16(o) || !al16(ws) || (n_new && !al16(n_new))) return ST_EINVAL;
    return cuda_rc(spec::launch_attn_paged(*cfg, *kv, q, n_new, o, ws,
                                           static_cast<cudaStream_t>(stream)));
}

int draft_verify_sampled(const spec_draft_cfg* cfg, const int32_t* draft_tok,
                         const int32_t* n_draft, const float* draft_prob, const void* logits,
                         const float* u, const float* e, const spec_draft_out* out,
                         int32_t* kv_len, int32_t* root_tok, void* ws, void* stream) {
    int rc = spec::check_draft_cfg(cfg);
    if (rc) return rc;
    if (!out || !al16(out->accept_len) || !al16(out->out_tok)) return ST_EINVAL;
    if (!al16(logits) || !al16(e) || !al16(ws)) return ST_EINVAL;
    if (cfg->N > 0 && (!al16(draft_tok) || !al16(u) || !al16(out->target_prob))) return ST_EINVAL;
    if ((draft_prob && !al16(draft_prob)) || (n_draft && !al16(n_draft)) ||
        (kv_len && !al16(kv_len)) || (root_tok && !al16(root_tok)))
        return ST_EINVAL;
    return cuda_rc(spec::launch_draft_verify(*cfg, draft_tok, n_draft, draft_prob, logits, u, e,
                                             *out, kv_len, root_tok, ws,
                                             static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
