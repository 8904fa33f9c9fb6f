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

// ---- a rotation's frequencies, in pairs of doubles (the sum of both, some 100 bits).
// A table of 64-bit numbers needs more than a double's 53: at position 2^31 a relative
// error of 2^-53 is 2^-25 turns.

struct Two {
    double hi, lo;
};

Two joined(double a, double b) {                         // |a| >= |b|
    const double s = a + b;
    return Two{s, b - (s - a)};
}

Two add(Two a, Two b) {
    const double s = a.hi + b.hi, v = s - a.hi;
    return joined(s, (a.hi - (s - v)) + (b.hi - v) + (a.lo + b.lo));
}

Two mul(Two a, Two b) {
    volatile double p = a.hi * b.hi;                     // rounded by itself on every machine
    return joined(p, fma(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi));
}

Two neg(Two a) { return Two{-a.hi, -a.lo}; }

Two div(Two a, Two b) {
    const double x = a.hi / b.hi;
    Two r = add(a, neg(mul(Two{x, 0.0}, b)));
    const double y = r.hi / b.hi;
    r = add(r, neg(mul(Two{y, 0.0}, b)));
    return add(joined(x, y), Two{r.hi / b.hi, 0.0});
}

// base^(-j / n): a Newton step from the rounded power, whose n-th power times base^j is
// multiplied up in an order that stays near 1
Two root(double base, int j, int n) {
    const double f = pow(base, -(double)j / n);
    if (f == 0.0) return Two{0.0, 0.0};
    Two t{1.0, 0.0};
    for (int fs = n, bases = j; fs + bases > 0;) {
        const bool down = bases == 0 || (fs > 0 && t.hi >= 1.0);
        t = mul(t, Two{down ? f : base, 0.0});
        --(down ? fs : bases);
    }
    return joined(f, -f * ((t.hi - 1.0) + t.lo) / n);
}

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
    const int n = rot / 2;
    const bool ntk = s->kind == SPEC_ROPE_NTK;
    if (ntk && !is_finite(s->base * pow(s->factor, (double)n / (n - 1)))) return ST_EINVAL;
    const Two two_pi{6.283185307179586, 2.4492935982947064e-16}, factor{s->factor, 0.0};
    for (int j = 0; j < n; ++j) {
        Two f = root(s->base, j, n);
        if (ntk) f = mul(f, root(s->factor, j, n - 1));  // (factor^(n / (n - 1)))^(-j / n)
        if (s->kind == SPEC_ROPE_LINEAR) f = div(f, factor);
        if (yarn) {
            const Two slow{-s->beta_slow, 0.0};
            const Two over = div(mul(Two{(double)s->orig_len, 0.0}, f), two_pi);
            Two g = div(add(over, slow), add(Two{s->beta_fast, 0.0}, slow));
            if (g.hi <= 0.0) g = Two{0.0, 0.0};
            if (g.hi >= 1.0) g = Two{1.0, 0.0};
            f = add(div(mul(add(Two{1.0, 0.0}, neg(g)), f), factor), mul(g, f));
        }
        // f <= 1: under 0.16 turns a position
        const Two t = div(f, two_pi);
        const double hi = t.hi * 18446744073709551616.0, whole = floor(hi);
        const double rest = (hi - whole) + t.lo * 18446744073709551616.0;
        turns[j] = (uint64_t)whole + (uint64_t)(int64_t)floor(rest + 0.5);
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
        !al16_or_null(params->top_p) || !al16_or_null(params->min_p) ||
        !al16_or_null(params->last_row))
        return ST_EINVAL;
    if (params->idle != SPEC_IDLE_SKIP && params->idle != SPEC_IDLE_QUIET) return ST_EINVAL;
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
