// draft_verify.cu -- verification of a drafted chain from given random numbers
// (speculative-decoding tutorial (mlqm.cn), section 2.3: keep a draft x with
// probability min(1, p(x) / q(x)), else draw from max(0, p - q) renormalised).
//
// Mathematics.  u uniform: u q(x) < p(x) keeps x with that probability.  E_v
// independent standard exponentials: argmin_v E_v / w_v is v with probability
// w_v / sum w, so the draw is argmax_v w_v / e_v and needs neither the sum of
// max(0, p - q) nor a prefix sum over the vocabulary, whose fp32 rounding would
// move borders: a near-tie of two scores is the only place where a rounding
// can change the token.
//
// What bounds it: reading the logits rows once (2 V (n + 1) bytes a request in
// bf16), then one drafter row and the exponentials (8 V bytes a request).
// Two launches, the second under the first's tail:
//   1. row_mass: every needed logits row in `splits` segments, a CTA each:
//      (max, sum of 2^((x - max) k)), k = log2(e) / temperature, 16-byte loads,
//      eight in flight per thread.  Rows are V elements apart, so a row may
//      start inside a 16-byte group: the few elements beside its whole groups
//      are taken one by one.
//   2. race: each CTA decides its request's chain from the segments' masses
//      (a warp per row), then scans a slice of the vocabulary at the row where
//      the chain ended; the request's last CTA (a ticket) joins the slices and
//      writes the outputs.
// Measured (graph replays, V = 151936, bf16, a drafter's rows in fp32): one request
// of 8 drafts 9.2 us, two launches' latency; 24 requests of up to 8 drafts 20.9 us,
// 65 MB at 3.2 TB/s: each launch is a chain (loads, block reduction; masses,
// decision, loads, reduction, ticket) of which reading is about half.
#include <math.h>

#include "paged.cuh"

namespace spec {

namespace {

constexpr int NT = 256;
constexpr int NONE = 0x7fffffff;
constexpr float FOLD = 0x1p20f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// (m, s) += (om, os); a NaN sum stays.
__device__ __forceinline__ void merge(float& m, float& s, float om, float os, float k) {
    const float nm = fmaxf(m, om);
    s = (m == nm ? s : s * ex2((m - nm) * k)) + (om == nm ? os : os * ex2((om - nm) * k));
    m = nm;
}

// The warp's (m, s), in every lane.
__device__ __forceinline__ void warp_mass(float& m, float& s, float k) {
    float nm = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) nm = fmaxf(nm, __shfl_xor_sync(0xffffffffu, nm, o));
    if (m != nm) s *= ex2((m - nm) * k);
    m = nm;
    s = warp_sum(s);
}

struct Cand {
    float s;          // w / e of the best token, -inf when there is none
    int i;
};

__device__ __forceinline__ void take(Cand& a, float s, int i) {
    if (s > a.s || (s == a.s && i < a.i)) {
        a.s = s;
        a.i = i;
    }
}

// Best candidate of the block, in every thread.
__device__ __forceinline__ Cand block_best(Cand a, Cand* sh) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        take(a, __shfl_xor_sync(0xffffffffu, a.s, o), __shfl_xor_sync(0xffffffffu, a.i, o));
    __syncthreads();
    if (threadIdx.x % 32 == 0) sh[threadIdx.x / 32] = a;
    __syncthreads();
    a = sh[0];
#pragma unroll
    for (int w = 1; w < NT / 32; ++w) take(a, sh[w].s, sh[w].i);
    return a;
}

template <int IO> struct grp {
    static constexpr int VEC = 16 / sizeof(typename io_t<IO>::T);
    static __device__ __forceinline__ void unpack(const uint4& u, float (&x)[VEC]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (IO == SPEC_IO_F32) {
                x[i] = __uint_as_float(w[i]);
            } else {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    }
};

// Drafts of request b; -1 where there is no request.
__device__ __forceinline__ int drafts(const int32_t* n_draft, int b, int N, uint32_t& bits) {
    return n_draft && n_draft[b] == -1 ? -1 : new_rows(n_draft, b, N, bits);
}

template <int IO>
__global__ void __launch_bounds__(NT)
row_mass(spec_draft_cfg c, const int32_t* __restrict__ n_draft,
         const typename io_t<IO>::T* __restrict__ logits, float k, float2* part, int splits) {
    constexpr int VEC = grp<IO>::VEC, U = 8;
    __shared__ float sm[NT / 32], ss[NT / 32];
    const int row = blockIdx.x / splits, seg = blockIdx.x % splits;
    const int b = row / (c.N + 1), i = row % (c.N + 1);
    uint32_t ignore = 0;
    pdl_wait();
    // The second launch may start: it waits for this one's results.  It reads the
    // caller's inputs before, which is sound because this wait comes first in every
    // CTA: whatever wrote them has ended by then.
    pdl_trigger();
    if (i > drafts(n_draft, b, c.N, ignore)) return;
    // the row's own 16-byte groups [g0, g1), and the elements beside them
    const int64_t r0 = (int64_t)row * c.V, r1 = r0 + c.V;
    const int64_t g0 = (r0 + VEC - 1) / VEC, g1 = r1 / VEC;
    const int groups = g1 > g0 ? (int)(g1 - g0) : 0;
    const int per = (groups + splits - 1) / splits;
    const int lo = seg * per, hi = min(groups, lo + per), left = hi - lo;
    const uint4* src = reinterpret_cast<const uint4*>(logits) + g0;
    float m = -INFINITY, s = 0.0f;
    for (int at = 0; at < left; at += U * NT) {
        const int e0 = lo + at + threadIdx.x;
        uint4 u[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const uint32_t none = IO == SPEC_IO_F32 ? 0xff800000u : 0xff80ff80u;   // -inf
            u[j] = make_uint4(none, none, none, none);
            if (e0 + j * NT < hi) u[j] = __ldg(src + e0 + j * NT);
        }
        float nm = m;
        if constexpr (IO == SPEC_IO_F32) {
#pragma unroll
            for (int j = 0; j < U; ++j) {
                float x[VEC];
                grp<IO>::unpack(u[j], x);
#pragma unroll
                for (int v = 0; v < VEC; ++v) nm = fmaxf(nm, x[v]);
            }
        } else {
            __nv_bfloat162 h = *reinterpret_cast<const __nv_bfloat162*>(&u[0].x);
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&u[j]);
#pragma unroll
                for (int v = 0; v < 4; ++v) h = __hmax2(h, p[v]);
            }
            nm = fmaxf(nm, fmaxf(__low2float(h), __high2float(h)));   // a NaN is passed over
        }
        if (m != nm) s *= ex2((m - nm) * k);
        m = nm;
        // 2^((x - base) k) as 2^(x k - c), c = fl(base k): the sum of a product
        // and a constant is rounded once, and what c is off by, base k - c (a
        // fused multiply-add gives it exactly), is the same factor for all.  It
        // is at most FOLD 2^-25 there; beyond (a small temperature, or nothing
        // but masks of the type's lowest value) that factor, and base k itself,
        // leave fp32's range: there x - base comes first.
        const float base = m == -INFINITY ? 0.0f : m;      // a NaN beside -inf stays
        const float c0 = -base * k;
        float ps[4] = {};
        auto add = [&](auto&& term) {
#pragma unroll
            for (int j = 0; j < U; ++j) {
                if (at + j * NT >= left) break;            // the same for all threads
                float x[VEC];
                grp<IO>::unpack(u[j], x);
#pragma unroll
                for (int v = 0; v < VEC; ++v) ps[v % 4] += term(x[v]);
            }
        };
        float rest = 1.0f;
        if (fabsf(c0) <= FOLD) {
            add([&](float x) { return ex2(fmaf(x, k, c0)); });
            rest = ex2(-fmaf(base, k, c0));
        } else {
            add([&](float x) { return ex2((x - base) * k); });
        }
        s += ((ps[0] + ps[1]) + (ps[2] + ps[3])) * rest;
    }
    if (seg == 0) {
        // the elements of the row in groups that it shares with its neighbours
        const int64_t head = min(g0 * VEC, r1), tail = max(g1 * VEC, head);
        const int64_t at = threadIdx.x < head - r0 ? r0 + threadIdx.x
                                                   : tail + (threadIdx.x - (head - r0));
        if (at < r1 && (at < head || at >= tail)) {
            const float x = io_t<IO>::ld(logits, at);
            merge(m, s, x, x == -INFINITY ? 0.0f : x - x + 1.0f, k);   // NaN, +inf: NaN
        }
    }
    warp_mass(m, s, k);
    if (threadIdx.x % 32 == 0) {
        sm[threadIdx.x / 32] = m;
        ss[threadIdx.x / 32] = s;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        m = threadIdx.x < NT / 32 ? sm[threadIdx.x] : -INFINITY;
        s = threadIdx.x < NT / 32 ? ss[threadIdx.x] : 0.0f;
        warp_mass(m, s, k);
        if (threadIdx.x == 0) part[(size_t)row * splits + seg] = make_float2(m, s);
    }
}

struct RaceArgs {
    const int32_t* draft_tok;
    const int32_t* n_draft;
    const float* draft_prob;
    const void* logits;
    const float* u;
    const float* e;
    spec_draft_out out;
    int32_t* kv_len;
    int32_t* root_tok;
    void* ws;
    const float2* part;
    float2* cand;            // [B][slices]: (score, token)
    uint32_t* tickets;       // [B] where there is more than one slice
    int splits, slices, per; // per: tokens of a slice
    float k;                 // log2(e) / temperature
};

template <int IO>
__global__ void __launch_bounds__(NT)
race(spec_draft_cfg c, const __grid_constant__ RaceArgs a) {
    using T = typename io_t<IO>::T;
    // tokens per group, groups under way at once: 2 and 72 registers, so that
    // three CTAs share an SM (before the scores below, 24 requests 22.1 us; 1:
    // 23.4, 4 on two CTAs: 28)
    constexpr int VEC = 8, U = 2;
    __shared__ float row_m[SPEC_MAX_ROWS], row_s[SPEC_MAX_ROWS];
    __shared__ float tok_x[SPEC_MAX_ROWS], tok_q[SPEC_MAX_ROWS];
    __shared__ int keep[SPEC_MAX_ROWS], draft[SPEC_MAX_ROWS];
    __shared__ Cand sh[NT / 32];
    __shared__ int last_cta;
    const int b = blockIdx.y, N = c.N, V = c.V, tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const T* logits = static_cast<const T*>(a.logits);
    const int lo = blockIdx.x * a.per, hi = min(V, lo + a.per);
    const float* e = a.e + (size_t)b * V;
    // ---- what does not depend on the masses: this slice's first exponentials,
    // the drafts and what the target and the drafter say of them
    const bool vec = V % VEC == 0;
    float ev[U][VEC];
    auto load_e = [&](int v0) {
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int v = v0 + j * NT * VEC;
            if (v < hi) {
                *reinterpret_cast<float4*>(ev[j]) = __ldg(reinterpret_cast<const float4*>(e + v));
                *reinterpret_cast<float4*>(ev[j] + 4) =
                    __ldg(reinterpret_cast<const float4*>(e + v + 4));
            }
        }
    };
    const int first = lo + tid * VEC;
    if (vec) load_e(first);
    uint32_t bits = 0;
    const int n = drafts(a.n_draft, b, N, bits);
    if (tid < n) {
        const int x = a.draft_tok[(size_t)b * N + tid];
        const bool in = x >= 0 && x < V;
        if (!in) bits |= SPEC_DEV_BADTOK;
        draft[tid] = x;
        tok_x[tid] = in ? io_t<IO>::ld(logits, ((size_t)b * (N + 1) + tid) * V + x) : 0.0f;
        const float q = in && a.draft_prob ? a.draft_prob[((size_t)b * N + tid) * V + x] : 1.0f;
        tok_q[tid] = a.u[(size_t)b * N + tid] * q;
    }
    if (bits && blockIdx.x == 0) raise_status(a.ws, bits);
    pdl_wait();
    if (n < 0) {                                         // no request
        if (blockIdx.x > 0) return;
        if (tid <= N) a.out.out_tok[(size_t)b * (N + 1) + tid] = -1;
        if (tid < N) a.out.target_prob[(size_t)b * N + tid] = 0.0f;
        if (tid == 0) a.out.accept_len[b] = 0;
        return;
    }

    // ---- the rows' masses (a warp per row) and the chain
    for (int i = warp; i <= n; i += NT / 32) {
        const size_t row = (size_t)b * (N + 1) + i;
        float m = -INFINITY, s = 0.0f;
        for (int k = lane; k < a.splits; k += 32) {
            const float2 x = __ldcg(a.part + row * a.splits + k);
            merge(m, s, x.x, x.y, a.k);
        }
        warp_mass(m, s, a.k);
        if (lane == 0) {
            row_m[i] = m;
            row_s[i] = s > 0.0f && s <= 3.0e38f ? s : 0.0f;   // else NaN, +inf or no mass
        }
    }
    __syncthreads();
    if (tid < N) {
        float p = 0.0f;
        const bool in = tid < n && draft[tid] >= 0 && draft[tid] < V;
        if (in && row_s[tid] > 0.0f)
            p = expf((tok_x[tid] - row_m[tid]) / c.temperature) / row_s[tid];
        if (tid < n) keep[tid] = in && tok_q[tid] < p;
        if (blockIdx.x == 0) a.out.target_prob[(size_t)b * N + tid] = p;
    }
    __syncthreads();
    int kept = 0;
    while (kept < n && keep[kept]) ++kept;

    // ---- the race over this slice of the row where the chain ended
    const float m = row_m[kept], s = row_s[kept], inv = 1.0f / s;
    const T* lp = logits + ((size_t)b * (N + 1) + kept) * V;
    const float* qp =
        kept < n && a.draft_prob ? a.draft_prob + ((size_t)b * N + kept) * V : nullptr;
    const int point = kept < n && !a.draft_prob ? draft[kept] : -1;
    // Scores w / e by the approximate reciprocal; the thread keeps the weight and
    // exponential of its best, and where two scores are nearer than that
    // reciprocal tells apart, the quotients decide.  (A division per token made
    // the race 45 instructions a token.)
    // (top_lo is never 0: tokens without weight take no quotient.)  An exponential
    // below 2^-126 has an infinite approximate score, which makes top_hi infinite
    // for good: then the thread goes over its tokens again.  (Told apart here, it
    // made 24 requests 22.1 us instead of 20.9.)  One from 2^126 on has
    // none: if that is all there is, the request's last CTA sees to it.
    float top_lo = 0x1p-149f, top_hi = 0.0f, top_w = 0.0f, top_e = 1.0f;
    int top_i = NONE;
    auto score = [&](float x, float q, float ex, int v) {
        const float w = fmaf(ex2((x - m) * a.k), inv, -q);
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(ex));
        const float s = w * r;
        bool more = s > top_hi;
        if (!more && s >= top_lo) more = w / ex > top_w / top_e;     // seldom
        if (more) {
            top_lo = s * (1.0f - 0x1p-20f);
            top_hi = s * (1.0f + 0x1p-20f);
            top_w = w;
            top_e = ex;
            top_i = v;
        }
    };
    // a token by its quotient (res: by the residual, where there is one)
    auto take_quotient = [&](Cand& c, int v, bool res) {
        const float q = !res ? 0.0f : (qp ? qp[v] : (v == point ? 1.0f : 0.0f));
        const float w = fmaf(ex2((io_t<IO>::ld(lp, v) - m) * a.k), inv, -q);
        if (w > 0.0f) take(c, w / e[v], v);
    };
    if (s > 0.0f && vec) {
        for (int v0 = first; v0 < hi; v0 += U * NT * VEC) {
            if (v0 != first) load_e(v0);
            uint4 xu[U][IO == SPEC_IO_F32 ? 2 : 1];
            float q[U][VEC];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int v = v0 + j * NT * VEC;
#pragma unroll
                for (int i = 0; i < VEC; ++i) q[j][i] = v + i == point ? 1.0f : 0.0f;
                if (v >= hi) continue;
                const uint4* src = reinterpret_cast<const uint4*>(lp + v);
                xu[j][0] = __ldg(src);
                if constexpr (IO == SPEC_IO_F32) xu[j][1] = __ldg(src + 1);
                if (qp) {
                    *reinterpret_cast<float4*>(q[j]) =
                        __ldg(reinterpret_cast<const float4*>(qp + v));
                    *reinterpret_cast<float4*>(q[j] + 4) =
                        __ldg(reinterpret_cast<const float4*>(qp + v + 4));
                }
            }
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int v = v0 + j * NT * VEC;
                if (v >= hi) break;
                float x[VEC];
                grp<IO>::unpack(xu[j][0], reinterpret_cast<float(&)[grp<IO>::VEC]>(x[0]));
                if constexpr (IO == SPEC_IO_F32)
                    grp<IO>::unpack(xu[j][1], reinterpret_cast<float(&)[grp<IO>::VEC]>(x[4]));
#pragma unroll
                for (int i = 0; i < VEC; ++i) score(x[i], q[j][i], ev[j][i], v + i);
            }
        }
    } else if (s > 0.0f) {
#pragma unroll 4
        for (int v = lo + tid; v < hi; v += NT)
            score(io_t<IO>::ld(lp, v), qp ? qp[v] : (v == point ? 1.0f : 0.0f), e[v], v);
    }
    Cand best{top_i == NONE ? -INFINITY : top_w / top_e, top_i};
    if (!(top_hi < INFINITY)) {
        best = Cand{-INFINITY, NONE};
        const int len = vec ? VEC : 1;
        for (int v0 = lo + tid * len; v0 < hi; v0 += NT * len)
            for (int v = v0; v < v0 + len; ++v) take_quotient(best, v, true);
    }
    best = block_best(best, sh);
    if (a.slices > 1) {
        if (tid == 0) {
            __stcg(a.cand + (size_t)b * a.slices + blockIdx.x,
                   make_float2(best.s, __int_as_float(best.i)));
            asm volatile("fence.acq_rel.gpu;" ::: "memory");
            last_cta = atomicAdd(a.tickets + b, 1u) == (uint32_t)a.slices - 1;
            asm volatile("fence.acq_rel.gpu;" ::: "memory");
        }
        __syncthreads();
        if (!last_cta) return;
        best = Cand{-INFINITY, NONE};
        for (int k = tid; k < a.slices; k += NT) {
            const float2 x = __ldcg(a.cand + (size_t)b * a.slices + k);
            take(best, x.x, __float_as_int(x.y));
        }
        best = block_best(best, sh);
    }
    if (s > 0.0f && !(best.s >= 0x1p-100f)) {
        // No token, or scores where approximate ones lose bits or vanish: the
        // quotients of all.  Where p <= q everywhere in fp32 (a refusal at a
        // rounding's distance) p decides.
        for (int pass = 0; pass < 2; ++pass) {
            Cand again{-INFINITY, NONE};
            for (int v = tid; v < V; v += NT) take_quotient(again, v, pass == 0);
            best = block_best(again, sh);
            if (best.i != NONE) break;
        }
    }
    const int tok = best.i != NONE ? best.i : 0;
    for (int j = tid; j <= N; j += NT)
        a.out.out_tok[(size_t)b * (N + 1) + j] = j < kept ? draft[j] : (j == kept ? tok : -1);
    if (tid == 0) {
        if (a.slices > 1) a.tickets[b] = 0;              // for the next call
        a.out.accept_len[b] = kept + 1;
        if (a.kv_len) a.kv_len[b] += kept + 1;
        if (a.root_tok) a.root_tok[b] = tok;
        if (!(s > 0.0f)) raise_status(a.ws, SPEC_DEV_BADLOGIT);
    }
}

template <int IO>
cudaError_t verify_t(const spec_draft_cfg& c, const int32_t* n_draft, const void* logits,
                     RaceArgs a, const DraftWs& w, cudaStream_t st) {
    const int64_t ctas = (int64_t)c.B * (c.N + 1) * w.splits;
    if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
    cudaError_t e = launch_k(true, row_mass<IO>, dim3((unsigned)ctas), dim3(NT), 0, st, c,
                             n_draft, static_cast<const typename io_t<IO>::T*>(logits), a.k,
                             ws_ptr<float2>(a.ws, w.part_off), w.splits);
    if (e != cudaSuccess) return e;
    return launch_k(true, race<IO>, dim3(w.slices, c.B), dim3(NT), 0, st, c, a);
}

}  // namespace

cudaError_t launch_draft_verify(const spec_draft_cfg& c, const int32_t* draft_tok,
                                const int32_t* n_draft, const float* draft_prob,
                                const void* logits, const float* u, const float* e,
                                const spec_draft_out& out, int32_t* kv_len, int32_t* root_tok,
                                void* ws, cudaStream_t st) {
    const int sms = device_sm_count();
    if (sms < 1) return cudaErrorInvalidDevice;
    const DraftWs w = draft_ws_layout(c, sms);
    RaceArgs a{draft_tok, n_draft, draft_prob, logits, u, e, out, kv_len, root_tok, ws,
               ws_ptr<const float2>(ws, w.part_off), ws_ptr<float2>(ws, w.cand_off),
               ws_ptr<uint32_t>(ws, draft_ticket_off(sms)), w.splits, w.slices, w.per,
               fminf(1.4426950408889634f / c.temperature, 3.4028234663852886e38f)};
    return c.io_dtype == SPEC_IO_BF16 ? verify_t<SPEC_IO_BF16>(c, n_draft, logits, a, w, st)
                                      : verify_t<SPEC_IO_F32>(c, n_draft, logits, a, w, st);
}

}  // namespace spec
