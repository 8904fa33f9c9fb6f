// draft_verify.cu -- verification of a drafted chain from given random numbers
// (speculative-decoding tutorial (mlqm.cn), section 2.3).
//
// One CTA per request walks the chain: (max, sum of exp) of a row's logits,
// the row's decision, and at the row where the walk ends the race
// argmax_v w(v) / e(v) over the vocabulary.
#include <math.h>

#include "paged.cuh"

namespace spec {

namespace {

constexpr int NT = 512;

struct Cand {
    float s;          // w / e of the best token, -inf when none
    int i;
};

__device__ __forceinline__ void take(Cand& a, float s, int i) {
    if (s > a.s || (s == a.s && i < a.i)) {
        a.s = s;
        a.i = i;
    }
}

__device__ Cand block_best(Cand a, Cand* sh) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        take(a, __shfl_xor_sync(0xffffffffu, a.s, o), __shfl_xor_sync(0xffffffffu, a.i, o));
    __syncthreads();
    if (threadIdx.x % 32 == 0) sh[threadIdx.x / 32] = a;
    __syncthreads();
    a = sh[0];
    for (int w = 1; w < NT / 32; ++w) take(a, sh[w].s, sh[w].i);
    return a;
}

template <int IO>
__global__ void __launch_bounds__(NT)
verify_chain(spec_draft_cfg c, const int32_t* __restrict__ draft_tok,
             const int32_t* __restrict__ n_draft, const float* __restrict__ draft_prob,
             const typename io_t<IO>::T* __restrict__ logits, const float* __restrict__ u,
             const float* __restrict__ e, spec_draft_out out, int32_t* kv_len, int32_t* root_tok,
             void* ws) {
    __shared__ float red[2 * NT / 32];
    __shared__ Cand cands[NT / 32];
    const int b = blockIdx.x, N = c.N, V = c.V, tid = threadIdx.x;
    uint32_t bits = 0;
    const int n = new_rows(n_draft, b, N, bits);
    int kept = -1;
    for (int i = 0; i <= n; ++i) {
        const auto* row = logits + ((size_t)b * (N + 1) + i) * V;
        float m = -INFINITY;
        for (int v = tid; v < V; v += NT) m = fmaxf(m, io_t<IO>::ld(row, v));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        __syncthreads();
        if (tid % 32 == 0) red[tid / 32] = m;
        __syncthreads();
        for (int w = 0; w < NT / 32; ++w) m = fmaxf(m, red[w]);
        float sum = 0.0f;
        for (int v = tid; v < V; v += NT) sum += expf((io_t<IO>::ld(row, v) - m) / c.temperature);
        sum = warp_sum(sum);
        if (tid % 32 == 0) red[NT / 32 + tid / 32] = sum;
        __syncthreads();
        sum = 0.0f;
        for (int w = 0; w < NT / 32; ++w) sum += red[NT / 32 + w];
        const bool fine = sum > 0.0f && sum <= 3.0e38f;
        bool keep = false;
        int x = -1;
        const float* q = nullptr;
        if (i < n) {
            x = draft_tok[(size_t)b * N + i];
            const bool in = x >= 0 && x < V;
            if (!in) bits |= SPEC_DEV_BADTOK;
            q = draft_prob ? draft_prob + ((size_t)b * N + i) * V : nullptr;
            float p = 0.0f;
            if (in && fine) {
                p = expf((io_t<IO>::ld(row, x) - m) / c.temperature) / sum;
                keep = u[(size_t)b * N + i] * (q ? q[x] : 1.0f) < p;
            }
            if (tid == 0) out.target_prob[(size_t)b * N + i] = p;
        }
        if (kept >= 0 || keep) continue;
        kept = i;
        Cand rest{-INFINITY, 0x7fffffff}, all{-INFINITY, 0x7fffffff};
        if (fine) {
            for (int v = tid; v < V; v += NT) {
                const float p = expf((io_t<IO>::ld(row, v) - m) / c.temperature) / sum;
                const float ev = e[(size_t)b * V + v];
                if (p > 0.0f) take(all, p / ev, v);
                const float w = i < n ? p - (q ? q[v] : (v == x ? 1.0f : 0.0f)) : 0.0f;
                if (w > 0.0f) take(rest, w / ev, v);
            }
        } else {
            bits |= SPEC_DEV_BADLOGIT;
        }
        rest = block_best(rest, cands);
        all = block_best(all, cands);
        const Cand best = rest.i != 0x7fffffff ? rest : all;
        const int tok = best.i != 0x7fffffff ? best.i : 0;
        if (tid == 0) {
            for (int j = 0; j <= N; ++j)
                out.out_tok[(size_t)b * (N + 1) + j] =
                    j < kept ? draft_tok[(size_t)b * N + j] : (j == kept ? tok : -1);
            for (int j = n; j < N; ++j) out.target_prob[(size_t)b * N + j] = 0.0f;
            out.accept_len[b] = kept + 1;
            if (kv_len) kv_len[b] += kept + 1;
            if (root_tok) root_tok[b] = tok;
        }
    }
    if (bits && tid == 0) raise_status(ws, bits);
}

}  // namespace

cudaError_t launch_draft_verify(const spec_draft_cfg& c, const int32_t* draft_tok,
                                const int32_t* n_draft, const float* draft_prob,
                                const void* logits, const float* u, const float* e,
                                const spec_draft_out& out, int32_t* kv_len, int32_t* root_tok,
                                void* ws, cudaStream_t st) {
    if (c.io_dtype == SPEC_IO_BF16)
        return launch_k(false, verify_chain<SPEC_IO_BF16>, dim3(c.B), dim3(NT), 0, st, c, draft_tok,
                        n_draft, draft_prob, static_cast<const __nv_bfloat16*>(logits), u, e, out,
                        kv_len, root_tok, ws);
    return launch_k(false, verify_chain<SPEC_IO_F32>, dim3(c.B), dim3(NT), 0, st, c, draft_tok,
                    n_draft, draft_prob, static_cast<const float*>(logits), u, e, out, kv_len,
                    root_tok, ws);
}

}  // namespace spec
