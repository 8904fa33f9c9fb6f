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
//      four in flight per thread.  Rows are V elements apart, so a row may
//      start inside a 16-byte group: segments are cut at groups, and the
//      elements of a row's first and last group that are not its own count as
//      -inf.
//   2. race: each CTA decides its request's chain from the segments' masses
//      (a warp per row), then scans a slice of the vocabulary at the row where
//      the chain ended; the request's last CTA (a ticket) joins the slices and
//      writes the outputs.
#include <math.h>

#include "paged.cuh"

namespace spec {

namespace {

constexpr int NT = 256;
constexpr int NONE = 0x7fffffff;

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

template <int IO>
__global__ void __launch_bounds__(NT)
row_mass(spec_draft_cfg c, const int32_t* __restrict__ n_draft,
         const typename io_t<IO>::T* __restrict__ logits, float k, float2* part, int splits) {
    constexpr int VEC = grp<IO>::VEC, U = 4;
    __shared__ float sm[NT / 32], ss[NT / 32];
    const int row = blockIdx.x / splits, seg = blockIdx.x % splits;
    const int b = row / (c.N + 1), i = row % (c.N + 1);
    uint32_t ignore = 0;
    // the second launch may start: it waits for this one's results
    pdl_trigger();
    if (i > new_rows(n_draft, b, c.N, ignore)) return;
    const int64_t r0 = (int64_t)row * c.V, r1 = r0 + c.V;
    const int64_t total = (int64_t)c.B * (c.N + 1) * c.V;
    const int64_t g0 = r0 / VEC;
    const int groups = (int)((r1 + VEC - 1) / VEC - g0);
    const int per = (groups + splits - 1) / splits;
    const int lo = seg * per, hi = min(groups, lo + per);
    const uint4* src = reinterpret_cast<const uint4*>(logits) + g0;
    float m = -INFINITY, s = 0.0f;
    for (int e0 = lo + threadIdx.x; e0 < hi; e0 += U * NT) {
        float x[U][VEC];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int e = e0 + j * NT;
            const int64_t at = (g0 + e) * VEC;
            uint4 u = make_uint4(0, 0, 0, 0);
            if (e < hi && at + VEC <= total) u = __ldg(src + e);
            grp<IO>::unpack(u, x[j]);
            // the tensor's last elements, beyond its last whole group
            if (e < hi && at + VEC > total)
                for (int v = 0; v < VEC; ++v) x[j][v] = at + v < total ? io_t<IO>::ld(logits, at + v) : 0.0f;
            // a row's edges
            if (e >= hi || at < r0 || at + VEC > r1)
#pragma unroll
                for (int v = 0; v < VEC; ++v)
                    if (e >= hi || at + v < r0 || at + v >= r1) x[j][v] = -INFINITY;
        }
        float nm = m;
#pragma unroll
        for (int j = 0; j < U; ++j)
#pragma unroll
            for (int v = 0; v < VEC; ++v) nm = fmaxf(nm, x[j][v]);
        if (m != nm) s *= ex2((m - nm) * k);
        m = nm;
        const float base = m == -INFINITY ? 0.0f : m;      // a NaN beside -inf stays
        float part_s[U] = {};
#pragma unroll
        for (int v = 0; v < VEC; ++v)
#pragma unroll
            for (int j = 0; j < U; ++j) part_s[j] += ex2((x[j][v] - base) * k);
#pragma unroll
        for (int j = 0; j < U; ++j) s += part_s[j];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float om = __shfl_xor_sync(0xffffffffu, m, o);
        const float os = __shfl_xor_sync(0xffffffffu, s, o);
        merge(m, s, om, os, k);
    }
    if (threadIdx.x % 32 == 0) {
        sm[threadIdx.x / 32] = m;
        ss[threadIdx.x / 32] = s;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 1; w < NT / 32; ++w) merge(m, s, sm[w], ss[w], k);
        part[(size_t)row * splits + seg] = make_float2(m, s);
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
    float4* cand;            // [B][slices]: (score, token) of max(0, p - q) and of p
    uint32_t* tickets;       // [B]
    int splits, slices, per; // per: tokens of a slice
    float k;                 // log2(e) / temperature
};

template <int IO>
__global__ void __launch_bounds__(NT)
race(spec_draft_cfg c, const __grid_constant__ RaceArgs a) {
    using T = typename io_t<IO>::T;
    constexpr int VEC = 8;
    __shared__ float row_m[SPEC_MAX_ROWS], row_s[SPEC_MAX_ROWS];
    __shared__ int keep[SPEC_MAX_ROWS];
    __shared__ Cand sh[NT / 32];
    __shared__ int last_cta;
    const int b = blockIdx.y, N = c.N, V = c.V, tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const T* logits = static_cast<const T*>(a.logits);
    const int lo = blockIdx.x * a.per, hi = min(V, lo + a.per);
    const float* e = a.e + (size_t)b * V;
    // what does not depend on the decision: this slice's first exponentials
    const bool vec = V % VEC == 0;
    float ev[VEC];
    const int v0 = lo + tid * VEC;
    if (vec && v0 < hi) {
        *reinterpret_cast<float4*>(ev) = __ldg(reinterpret_cast<const float4*>(e + v0));
        *reinterpret_cast<float4*>(ev + 4) = __ldg(reinterpret_cast<const float4*>(e + v0 + 4));
    }
    uint32_t bits = 0;
    const int n = new_rows(a.n_draft, b, N, bits);
    pdl_wait();

    // ---- the chain: a warp per row
    for (int i = warp; i <= n; i += NT / 32) {
        const size_t row = (size_t)b * (N + 1) + i;
        float m = -INFINITY, s = 0.0f;
        for (int k = lane; k < a.splits; k += 32) {
            const float2 x = __ldcg(a.part + row * a.splits + k);
            merge(m, s, x.x, x.y, a.k);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float om = __shfl_xor_sync(0xffffffffu, m, o);
            const float os = __shfl_xor_sync(0xffffffffu, s, o);
            merge(m, s, om, os, a.k);
        }
        if (lane == 0) {
            const bool fine = s > 0.0f && s <= 3.0e38f;     // else NaN, +inf or no mass
            row_m[i] = m;
            row_s[i] = fine ? s : 0.0f;
            int ok = 0;
            if (i < n) {
                const int x = a.draft_tok[(size_t)b * N + i];
                const bool in = x >= 0 && x < V;
                float p = 0.0f;
                if (!in) bits |= SPEC_DEV_BADTOK;
                if (in && fine) {
                    p = expf((io_t<IO>::ld(logits, row * V + x) - m) / c.temperature) / s;
                    const float q = a.draft_prob ? a.draft_prob[((size_t)b * N + i) * V + x] : 1.0f;
                    ok = a.u[(size_t)b * N + i] * q < p;
                }
                if (blockIdx.x == 0) a.out.target_prob[(size_t)b * N + i] = p;
            }
            keep[i] = ok;
        }
    }
    if (blockIdx.x == 0) {
        for (int j = n + tid; j < N; j += NT) a.out.target_prob[(size_t)b * N + j] = 0.0f;
        if (bits) raise_status(a.ws, bits);
    }
    __syncthreads();
    int kept = 0;
    while (kept < n && keep[kept]) ++kept;

    // ---- the race over this slice of the row where the chain ended
    const size_t row = (size_t)b * (N + 1) + kept;
    const float m = row_m[kept], s = row_s[kept], inv = 1.0f / s;
    const T* lp = logits + row * V;
    const float* qp = kept < n && a.draft_prob ? a.draft_prob + ((size_t)b * N + kept) * V : nullptr;
    const int point = kept < n && !a.draft_prob ? a.draft_tok[(size_t)b * N + kept] : -1;
    Cand rest{-INFINITY, NONE}, all{-INFINITY, NONE};
    auto score = [&](float x, float q, float ex, int v) {
        const float p = ex2((x - m) * a.k) * inv;
        if (p > 0.0f) take(all, p / ex, v);
        const float w = p - q;
        if (w > 0.0f) take(rest, w / ex, v);
    };
    if (s > 0.0f) {
        if (vec) {
            for (int v = v0; v < hi; v += NT * VEC) {
                float x[VEC], q[VEC];
                if constexpr (IO == SPEC_IO_BF16) {
                    grp<IO>::unpack(__ldg(reinterpret_cast<const uint4*>(lp + v)), x);
                } else {
                    *reinterpret_cast<float4*>(x) = __ldg(reinterpret_cast<const float4*>(lp + v));
                    *reinterpret_cast<float4*>(x + 4) =
                        __ldg(reinterpret_cast<const float4*>(lp + v + 4));
                }
                if (qp) {
                    *reinterpret_cast<float4*>(q) = __ldg(reinterpret_cast<const float4*>(qp + v));
                    *reinterpret_cast<float4*>(q + 4) =
                        __ldg(reinterpret_cast<const float4*>(qp + v + 4));
                } else {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) q[j] = v + j == point ? 1.0f : 0.0f;
                }
                if (v != v0) {
                    *reinterpret_cast<float4*>(ev) = __ldg(reinterpret_cast<const float4*>(e + v));
                    *reinterpret_cast<float4*>(ev + 4) =
                        __ldg(reinterpret_cast<const float4*>(e + v + 4));
                }
#pragma unroll
                for (int j = 0; j < VEC; ++j) score(x[j], q[j], ev[j], v + j);
            }
        } else {
#pragma unroll 4
            for (int v = lo + tid; v < hi; v += NT)
                score(io_t<IO>::ld(lp, v), qp ? qp[v] : (v == point ? 1.0f : 0.0f), e[v], v);
        }
    }
    rest = block_best(rest, sh);
    all = block_best(all, sh);
    if (tid == 0) {
        __stcg(a.cand + (size_t)b * a.slices + blockIdx.x,
               make_float4(rest.s, __int_as_float(rest.i), all.s, __int_as_float(all.i)));
        __threadfence();
        last_cta = atomicAdd(a.tickets + b, 1u) == (uint32_t)a.slices - 1;
        __threadfence();
    }
    __syncthreads();
    if (!last_cta) return;
    rest = all = Cand{-INFINITY, NONE};
    for (int k = tid; k < a.slices; k += NT) {
        const float4 x = __ldcg(a.cand + (size_t)b * a.slices + k);
        take(rest, x.x, __float_as_int(x.y));
        take(all, x.z, __float_as_int(x.w));
    }
    rest = block_best(rest, sh);
    all = block_best(all, sh);
    const Cand best = kept < n && rest.i != NONE ? rest : all;
    const int tok = best.i != NONE ? best.i : 0;
    for (int j = tid; j <= N; j += NT)
        a.out.out_tok[(size_t)b * (N + 1) + j] =
            j < kept ? a.draft_tok[(size_t)b * N + j] : (j == kept ? tok : -1);
    if (tid == 0) {
        a.tickets[b] = 0;                                // for the next call
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
    cudaError_t e = launch_k(false, row_mass<IO>, dim3((unsigned)ctas), dim3(NT), 0, st, c, n_draft, static_cast<const typename io_t<IO>::T*>(logits), a.k,
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
               ws_ptr<const float2>(ws, w.part_off), ws_ptr<float4>(ws, w.cand_off),
               ws_ptr<uint32_t>(ws, w.ticket_off), w.splits, w.slices, w.per,
               1.4426950408889634f / c.temperature};
    return c.io_dtype == SPEC_IO_BF16 ? verify_t<SPEC_IO_BF16>(c, n_draft, logits, a, w, st)
                                      : verify_t<SPEC_IO_F32>(c, n_draft, logits, a, w, st);
}

}  // namespace spec
