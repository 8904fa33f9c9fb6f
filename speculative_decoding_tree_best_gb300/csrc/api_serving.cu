// api_serving.cu -- the extern "C" boundary of the calls around a serving step:
// page tables, rotary positions, sampling.
#include <math.h>
#include <stdint.h>

#include "kernels.h"
#include "serving.cuh"

namespace {

using spec::al16;

int cuda_rc(cudaError_t e) {
    if (e == cudaSuccess) return ST_OK;
    if (e == cudaErrorInvalidConfiguration) return ST_EUNSUPPORTED;
    return ST_ECUDA;
}

bool al16_or_null(const void* p) { return !p || al16(p); }

bool is_finite(double x) { return x - x == 0.0; }

}  // namespace

extern "C" {

int page_tables_extend(const spec_paged_cfg* cfg, const spec_page_pool* pool,
                       const int32_t* n_new, int64_t* slots, int32_t* n_ok, void* ws,
                       void* stream) {
    int rc = spec::check_paged_cfg(cfg);
    if (rc) return rc;
    if ((rc = spec::check_pool(pool))) return rc;
    if (!al16(slots) || !al16(n_ok) || !al16(ws) || !al16_or_null(n_new)) return ST_EINVAL;
    return cuda_rc(spec::launch_pages_extend(*cfg, *pool, n_new, slots, n_ok, ws,
                                             static_cast<cudaStream_t>(stream)));
}

int page_tables_trim(const spec_paged_cfg* cfg, const spec_page_pool* pool, const int32_t* keep,
                     void* ws, void* stream) {
    int rc = spec::check_paged_cfg(cfg);
    if (rc) return rc;
    if ((rc = spec::check_pool(pool))) return rc;
    if (!al16(keep) || !al16(ws)) return ST_EINVAL;
    return cuda_rc(spec::launch_pages_trim(*cfg, *pool, keep, ws,
                                           static_cast<cudaStream_t>(stream)));
}

int spec_rope_turns(int rot, const spec_rope_scaling* s, uint64_t* turns, float* amp) {
    if (!s || !turns || !amp) return ST_EINVAL;
    if (rot < 16 || rot > 128 || rot % 16 != 0) return ST_EINVAL;
    if (s->kind < SPEC_ROPE_NONE || s->kind > SPEC_ROPE_YARN) return ST_EINVAL;
    if (!(s->base >= 1.0) || !is_finite(s->base)) return ST_EINVAL;
    const bool scaled = s->kind != SPEC_ROPE_NONE;
    if (scaled && (!(s->factor >= 1.0) || !is_finite(s->factor))) return ST_EINVAL;
    const bool yarn = s->kind == SPEC_ROPE_YARN;
    if (yarn && (s->orig_len < 1 || !(s->beta_slow >= 0.0) || !(s->beta_fast > s->beta_slow) ||
                 !is_finite(s->beta_fast)))
        return ST_EINVAL;
    double base = s->base;
    if (s->kind == SPEC_ROPE_NTK) base *= pow(s->factor, (double)rot / (rot - 2));
    if (!is_finite(base)) return ST_EINVAL;
    const double two_pi = 6.283185307179586476925;
    for (int j = 0; j < rot / 2; ++j) {
        double f = pow(base, -2.0 * j / rot);
        if (s->kind == SPEC_ROPE_LINEAR) f /= s->factor;
        if (yarn) {
            double g = (s->orig_len * f / two_pi - s->beta_slow) / (s->beta_fast - s->beta_slow);
            g = g < 0.0 ? 0.0 : (g > 1.0 ? 1.0 : g);
            f = (1.0 - g) * f / s->factor + g * f;
        }
        // f <= 1: under 0.16 turns a position
        turns[j] = (uint64_t)(f / two_pi * 18446744073709551616.0 + 0.5);
    }
    *amp = yarn ? (float)(0.1 * log(s->factor) + 1.0) : 1.0f;
    return ST_OK;
}

int rope_apply(const spec_rope_cfg* cfg, const uint64_t* turns, float amp, const int32_t* pos,
               const void* q, const void* k, void* q_out, void* k_out, void* stream) {
    const int rc = spec::check_rope_cfg(cfg, false);
    if (rc) return rc;
    if (!al16(turns) || !al16(pos) || !al16(q) || !al16(q_out) || !is_finite(amp)) return ST_EINVAL;
    if (cfg->Hkv > 0 && (!al16(k) || !al16(k_out))) return ST_EINVAL;
    return cuda_rc(spec::launch_rope(*cfg, turns, amp, pos, q, k, q_out, k_out,
                                     static_cast<cudaStream_t>(stream)));
}

int rope_page_append(const spec_rope_cfg* cfg, const spec_paged_cfg* pcfg,
                     const spec_paged_kv* kv, const uint64_t* turns, float amp,
                     const int64_t* slots, const void* q, const void* k_new, const void* v_new,
                     void* q_out, void* ws, void* stream) {
    int rc = spec::check_rope_cfg(cfg, true);
    if (rc) return rc;
    if ((rc = spec::check_paged_cfg(pcfg))) return rc;
    if ((rc = spec::check_paged_kv(*pcfg, kv))) return rc;
    if (cfg->Hq != pcfg->Hq || cfg->Hkv != pcfg->Hkv || cfg->D != pcfg->D ||
        cfg->io_dtype != pcfg->io_dtype || cfg->rows != (int64_t)pcfg->B * pcfg->T)
        return ST_EINVAL;
    if (!al16(turns) || !al16(slots) || !al16(q) || !al16(k_new) || !al16(v_new) ||
        !al16(q_out) || !al16(ws) || !is_finite(amp))
        return ST_EINVAL;
    return cuda_rc(spec::launch_rope_append(*cfg, *pcfg, *kv, turns, amp, slots, q, k_new, v_new,
                                            q_out, ws, static_cast<cudaStream_t>(stream)));
}

size_t spec_sample_workspace_bytes(const spec_sample_cfg* cfg, int num_sms) {
    if (spec::check_sample_cfg(cfg) != ST_OK || num_sms < 0) return 0;
    if (num_sms == 0) num_sms = spec::device_sm_count();
    return num_sms < 1 ? 0 : spec::ws_data_off(num_sms);
}

int token_sample(const spec_sample_cfg* cfg, const void* logits, const spec_sample_params* params,
                 const float* e, const spec_sample_out* out, void* ws, void* stream) {
    const int rc = spec::check_sample_cfg(cfg);
    if (rc) return rc;
    if (!params || !out || !al16(logits) || !al16(ws) || !al16_or_null(e)) return ST_EINVAL;
    if (!al16_or_null(params->temperature) || !al16_or_null(params->top_k) ||
        !al16_or_null(params->top_p) || !al16_or_null(params->min_p))
        return ST_EINVAL;
    if (!al16_or_null(out->tok) || !al16_or_null(out->tok_prob) || !al16_or_null(out->prob) ||
        !al16_or_null(out->logits))
        return ST_EINVAL;
    // a token needs its random numbers, and they a token
    if (!out->tok != !e || (out->tok_prob && !out->tok)) return ST_EINVAL;
    if (!out->tok && !out->prob && !out->logits) return ST_EINVAL;
    return cuda_rc(spec::launch_token_sample(*cfg, logits, *params, e, *out, ws,
                                             static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
