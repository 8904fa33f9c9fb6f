// token_sample.cu -- sampling with temperature, min-p, top-k and top-p from given
// random numbers.
//
// Mathematics.  What stays is a prefix of the order (logit descending, index
// ascending), so it is {K >= t} of the key K = (logit's bits, made to order like
// the number; index, falling): one 52-bit integer, different for every token.
// min-p gives t directly.  top-k and top-p ask for the largest t with
// F(t) = sum of f over {K >= t} >= target: f = 1 and the count k, or f = the
// token's weight and top_p times the sum over what top-k left.  That is a radix
// selection: a histogram of f over the top bits of K - lo names the bin that the
// border is in, which becomes the next range.
//   Weights are integers, 2^-(62 - lg V) of the largest one, from an exponential
// of 2^-30 relative accuracy (a table of 2^(-j/64) and a cubic): sums of them are
// exact in 64 bits, so the border depends neither on the order of summation nor
// on fp32's rounding of long sums.
//   The draw: argmin e / w over independent exponentials e is token v with
// probability w_v / sum w.
//
// Data flow.  A cluster of CTAs owns a row.  It reads the row once, into shared
// memory (what does not fit is read again from L2), and each pass goes over that
// copy; histograms are added up in the cluster's first CTA, which finds the border
// bin and tells the others.
#include <cooperative_groups.h>
#include <math.h>

#include "serving.cuh"

namespace spec {

namespace {

namespace cg = cooperative_groups;

constexpr int NT = 512;
constexpr int NB = 2048;                 // bins of a pass
constexpr int IDX_BITS = 20;             // of a key: V <= 2^20
constexpr uint32_t IDX_MAX = (1u << IDX_BITS) - 1;
constexpr int MAX_CLUSTER = 16;
constexpr int NO_TOK = 0x7fffffff;
// weights below 2^-CUT of the largest are 0 in the sums
constexpr float CUT = 43.0f;

typedef unsigned long long u64;

struct SampleArgs {
    const void* logits;
    spec_sample_params p;
    const float* e;
    spec_sample_out out;
    void* ws;
    int R, V, per;
    int lg;                  // ceil(log2 V)
    int resident;            // 16-byte groups of a CTA's slice kept in shared memory
    u64 pow2[64];            // 2^(62 - j/64)
};

// What one CTA tells the others.
struct Border {
    u64 lo, hi;              // the next range
    u64 above;               // F over the keys past hi; where lo = hi, that key too
    u64 target;
    int found;               // 0: F never reaches the target
};

struct Cand {
    float s, x;
    int i;
};

__device__ __forceinline__ void take(Cand& a, const Cand& b) {
    if (b.s > a.s || (b.s == a.s && b.i < a.i)) a = b;
}

// A request's parameters, made by one thread (64-bit floating point is slow here).
struct Params {
    float c, c_lo, far;      // log2(e) / temperature; see Weights
    float min_p;
    double min_low;          // temperature ln(min_p)
    u64 top_p;               // in units of 2^-64; 0: off
    int top_k;               // 0: off
    float low;               // the least logit that min_p leaves
    uint32_t bits;
};

struct Shared {
    u64 mass[NB];
    uint32_t count[NB];
    u64 pow2[64];
    u64 part[NT / 32];
    Border border;
    float cta_max[MAX_CLUSTER];
    Cand cand[MAX_CLUSTER];
    Cand warp_cand[NT / 32];
    float warp_max[NT / 32];
    u64 cta_mass[MAX_CLUSTER];
    Params prm;
};

__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// bits that order like the number, -0 as 0
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

__device__ __forceinline__ u64 key_of(float x, int i) {
    return (u64)key_of(x) << IDX_BITS | (IDX_MAX - (uint32_t)i);
}

// The softmax's weights of a row: 2^-((m - x) c), c = log2(e) / temperature in two
// parts.
struct Weights {
    float m, c, c_lo, far;       // far: weights beyond it are 0 in the sums
    int lg;
    const u64* pow2;

    // the exponent's (m - x) c and what its rounding leaves
    template <int IO> __device__ __forceinline__ float exponent(float x, float& rest) const {
        const float d = fminf(m - x, 3.4028234663852886e38f), y = d * c;
        rest = fmaf(d, c_lo, fmaf(d, c, -y));
        // bf16 values lie on a coarse grid: their difference is exact where the
        // smaller is above 2^-16 of the larger, else 2^-24 of it off
        if constexpr (IO == SPEC_IO_F32) {
            const float b = d - m;
            rest = fmaf((m - (d - b)) - (x + b), c, rest);
        }
        return y;
    }
    // as an integer, of 2^(62 - lg) for the largest
    template <int IO> __device__ __forceinline__ u64 fixed(float x) const {
        if (!(fminf(m - x, 3.4028234663852886e38f) <= far)) return 0;
        float rest;
        const float y = exponent<IO>(x, rest);
        const float n = fmaf(y, 64.0f, 12582912.0f);           // rounded to an integer
        const int k = __float_as_int(n) - 0x4b400000;
        const float r = (fmaf(n - 12582912.0f, -0x1p-6f, y) + rest) * -0.6931471805599453f;
        const float p = r * fmaf(r, fmaf(r, 1.0f / 6.0f, 0.5f), 1.0f);      // e^r - 1, |r| < 0.0055
        const u64 t = pow2[k & 63];
        const u64 w = t + (((int64_t)__float2int_rn(p * 0x1p38f) * (int32_t)(t >> 32)) >> 6);
        const int s = (k >> 6) + lg;
        return (w + ((1ull << s) >> 1)) >> s;
    }
    // as a float (1 for the largest)
    template <int IO> __device__ __forceinline__ float value(float x) const {
        float rest;
        const float y = exponent<IO>(x, rest);
        if (!(y < 200.0f)) return 0.0f;
        return ex2(-y) * fmaf(rest, -0.6931471805599453f, 1.0f);
    }
};

template <int IO> struct Row {
    using T = typename io_t<IO>::T;
    static constexpr int VEC = 16 / sizeof(T);
    const T* logits;
    int64_t r0, r1, end;         // the row's elements, the tensor's end
    int64_t g0;                  // first 16-byte group with one of them
    int lo, hi;                  // this CTA's groups, from g0
    const uint4* smem;
    int resident;

    // group g from memory, with what is not the row's as -inf
    __device__ __forceinline__ uint4 load(int g) const {
        const int64_t e0 = (g0 + g) * VEC;
        const T low = IO == SPEC_IO_F32 ? (T)-INFINITY : (T)__uint_as_float(0xff800000u);
        if (e0 >= r0 && e0 + VEC <= r1) return reinterpret_cast<const uint4*>(logits)[g0 + g];
        alignas(16) T x[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) x[v] = e0 + v >= r0 && e0 + v < r1 ? logits[e0 + v] : low;
        return *reinterpret_cast<const uint4*>(x);
    }
    __device__ __forceinline__ uint4 get(int g) const {
        return g - lo < resident ? smem[g - lo] : load(g);
    }
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
    // f(x, index in the row) for all of this CTA's elements (-inf beside the row)
    template <typename F> __device__ __forceinline__ void each(F&& f) const {
        for (int g = lo + threadIdx.x; g < hi; g += NT) {
            float x[VEC];
            unpack(get(g), x);
            const int i = (int)((g0 + g) * VEC - r0);
#pragma unroll
            for (int v = 0; v < VEC; ++v) f(x[v], i + v);
        }
    }
};

__device__ __forceinline__ u64 block_sum(u64 x, u64* part) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    __syncthreads();
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = x;
    __syncthreads();
    x = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) x += part[w];
    return x;
}

// Exclusive prefix of x over the block.
__device__ __forceinline__ u64 block_prefix(u64 x, u64* part, u64& total) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    u64 s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    __syncthreads();
    if (lane == 31) part[warp] = s;
    __syncthreads();
    u64 before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) before += part[w];
        total += part[w];
    }
    return before + s - x;
}

// The largest t in [lo, hi] with F(t) >= target; `lo` where F never reaches it
// (no key is above hi).  MASS: f = weights, the target want 2^-64 of F(lo), and F(t)
// is left in `sum`; else f = 1 and the target `want`.
template <bool MASS, int IO>
__device__ u64 select(cg::cluster_group& cl, Shared& sh, const Row<IO>& row, const Weights& wt,
                      u64 lo, u64 hi, u64 want, u64& sum) {
    const int rank = cl.block_rank(), C = cl.num_blocks(), tid = threadIdx.x;
    const u64 first = lo;
    u64 above = 0, target = want;
    for (int pass = 0;; ++pass) {
        const u64 span = hi - lo;
        const int bits = 64 - __clzll((long long)span);
        const int shift = max(0, bits - 11);                   // span >> shift < NB
        row.each([&](float x, int i) {
            const u64 k = key_of(x, i);
            if (k < lo || k > hi || i < 0) return;
            const int bin = (int)((hi - k) >> shift);
            if (MASS) atomicAdd(&sh.mass[bin], wt.fixed<IO>(x));
            else atomicAdd(&sh.count[bin], 1u);
        });
        __syncthreads();
        if (rank != 0) {
            for (int b = tid; b < NB; b += NT) {
                if (MASS) {
                    if (sh.mass[b]) atomicAdd(cl.map_shared_rank(&sh.mass[b], 0), sh.mass[b]);
                    sh.mass[b] = 0;
                } else {
                    if (sh.count[b]) atomicAdd(cl.map_shared_rank(&sh.count[b], 0), sh.count[b]);
                    sh.count[b] = 0;
                }
            }
        }
        cl.sync();
        if (rank == 0) {
            constexpr int RUN = NB / NT;
            u64 f[RUN], s = 0, total;
#pragma unroll
            for (int j = 0; j < RUN; ++j) {
                f[j] = MASS ? sh.mass[tid * RUN + j] : sh.count[tid * RUN + j];
                s += f[j];
            }
            u64 before = block_prefix(s, sh.part, total) + above;
            total += above;
            if (MASS && pass == 0) {
                target = __umul64hi(total, want) + (total * want != 0);    // rounded up
                target = max(target, (u64)1);
            }
            if (tid == 0 && total < target) sh.border = Border{lo, hi, above, target, 0};
            if (before < target && target <= before + s) {     // one thread, or none
                int j = 0;
#pragma unroll
                for (int k = 0; k < RUN - 1; ++k)
                    if (j == k && before + f[k] < target) {
                        before += f[k];
                        ++j;
                    }
                const u64 top = hi - ((u64)(tid * RUN + j) << shift);
                const u64 width = 1ull << shift;
                const u64 low = top - lo < width ? lo : top - width + 1;
                sh.border = Border{low, top, low == top ? before + f[j] : before, target, 1};
            }
#pragma unroll
            for (int j = 0; j < RUN; ++j) {
                sh.mass[tid * RUN + j] = 0;
                sh.count[tid * RUN + j] = 0;
            }
            __syncthreads();
            if (tid > 0 && tid < C) *cl.map_shared_rank(&sh.border, tid) = sh.border;
        }
        cl.sync();
        const Border b = sh.border;
        if (!b.found) return first;
        above = b.above;
        target = b.target;
        lo = b.lo;
        hi = b.hi;
        if (lo == hi) {
            if (MASS) sum = above;
            return lo;
        }
    }
}

__device__ __forceinline__ Params params_of(const spec_sample_params& p, int req) {
    Params y{};
    float t = p.temperature ? p.temperature[req] : 1.0f;
    float top_p = p.top_p ? p.top_p[req] : 1.0f, min_p = p.min_p ? p.min_p[req] : 0.0f;
    const int top_k = p.top_k ? p.top_k[req] : 0;
    if (!(t >= 0.0f) || top_p != top_p || min_p != min_p) y.bits = SPEC_DEV_BADREQ;
    if (!(t >= 0.0f)) t = 0.0f;
    if (top_p != top_p) top_p = 1.0f;
    if (min_p != min_p) min_p = 0.0f;
    y.top_k = t == 0.0f ? 1 : max(top_k, 0);
    // at most 2^64 - 2^40; a top_p of 0 or below keeps one token, as the least does
    y.top_p = top_p >= 1.0f ? 0 : max((u64)(fmaxf(top_p, 0.0f) * 0x1p64f), (u64)1);
    y.min_p = min_p;
    if (min_p > 0.0f && min_p < 1.0f) y.min_low = (double)t * log((double)min_p);
    const double c = t > 0.0f ? fmin(1.4426950408889634 / (double)t, 1e38) : 0.0;
    y.c = (float)c;
    y.c_lo = (float)(c - (double)y.c);
    y.far = c > 0.0 ? (float)fmin((double)CUT / c, 3.0e38) : 3.4028234663852886e38f;
    return y;
}

template <int IO>
__global__ void __launch_bounds__(NT)
sample_rows(const __grid_constant__ SampleArgs a) {
    using T = typename io_t<IO>::T;
    constexpr int VEC = Row<IO>::VEC;
    extern __shared__ uint4 slice[];
    __shared__ Shared sh;
    cg::cluster_group cl = cg::this_cluster();
    const int rank = cl.block_rank(), C = cl.num_blocks(), tid = threadIdx.x;
    const int lane = tid % 32, warp = tid / 32;
    const int r = blockIdx.x / C, V = a.V;
    for (int b = tid; b < NB; b += NT) {
        sh.mass[b] = 0;
        sh.count[b] = 0;
    }
    if (tid < 64) sh.pow2[tid] = a.pow2[tid];
    Row<IO> row;
    row.logits = static_cast<const T*>(a.logits);
    row.r0 = (int64_t)r * V;
    row.r1 = row.r0 + V;
    row.g0 = row.r0 / VEC;
    const int groups = (int)((row.r1 + VEC - 1) / VEC - row.g0), share = (groups + C - 1) / C;
    row.lo = min(groups, rank * share);
    row.hi = min(groups, row.lo + share);
    row.smem = slice;
    row.resident = a.resident;
    pdl_wait();
    if (tid == 0) sh.prm = params_of(a.p, r / a.per);

    // ---- the row, and its maximum
    float m = -INFINITY;
#pragma unroll 4
    for (int g = row.lo + tid; g < row.hi; g += NT) {
        const uint4 u = row.load(g);
        if (g - row.lo < a.resident) slice[g - row.lo] = u;
        float x[VEC];
        Row<IO>::unpack(u, x);
#pragma unroll
        for (int v = 0; v < VEC; ++v) m = max_nan(m, x[v]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) sh.warp_max[warp] = m;
    __syncthreads();
    m = sh.warp_max[lane % (NT / 32)];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    cl.sync();                                           // everyone has started
    if (tid < C) *cl.map_shared_rank(&sh.cta_max[rank], tid) = m;
    cl.sync();
    m = -INFINITY;
    for (int c = 0; c < C; ++c) m = max_nan(m, sh.cta_max[c]);

    const Params& prm = sh.prm;
    const bool bad = !(fabsf(m) < INFINITY);
    if (tid == 0) {
        float low = -3.4028234663852886e38f;
        if (prm.min_p >= 1.0f) low = m;
        else if (prm.min_p > 0.0f) low = fmaxf(low, __double2float_ru((double)m + prm.min_low));
        sh.prm.low = low;
        const uint32_t bits = prm.bits | (bad ? SPEC_DEV_BADLOGIT : 0u);
        if (bits && rank == 0) raise_status(a.ws, bits);
    }
    __syncthreads();
    const Weights wt{m, prm.c, prm.c_lo, prm.far, a.lg, sh.pow2};

    // ---- the border
    u64 keep_from = ~0ull, sum = 0;
    if (!bad) {
        keep_from = (u64)key_of(prm.low) << IDX_BITS;
        const u64 most = (u64)key_of(m) << IDX_BITS | IDX_MAX;
        if (prm.top_k > 0 && prm.top_k < V)
            keep_from = select<false, IO>(cl, sh, row, wt, keep_from, most, prm.top_k, sum);
        if (prm.top_p != 0) {
            keep_from = select<true, IO>(cl, sh, row, wt, keep_from, most, prm.top_p, sum);
        } else if (a.out.tok_prob || a.out.prob) {
            row.each([&](float x, int i) {
                if (key_of(x, i) >= keep_from) sum += wt.fixed<IO>(x);
            });
            sum = block_sum(sum, sh.part);
            if (tid < C) *cl.map_shared_rank(&sh.cta_mass[rank], tid) = sum;
            cl.sync();
            sum = 0;
            for (int c = 0; c < C; ++c) sum += sh.cta_mass[c];
        }
    }

    // ---- what stays: the race and the outputs
    const float inv =
        bad || sum == 0 ? 0.0f : 1.0f / (__ull2float_rn(sum) * (1.0f / (float)(1ull << (62 - a.lg))));
    Cand best{-1.0f, 0.0f, NO_TOK};
    float* prob = a.out.prob;
    T* kept = static_cast<T*>(a.out.logits);
    for (int g = row.lo + tid; g < row.hi; g += NT) {
        const uint4 u = row.get(g);
        float x[VEC];
        Row<IO>::unpack(u, x);
        const int64_t e0 = (row.g0 + g) * VEC;
        const int i = (int)(e0 - row.r0);
        const bool whole = i >= 0 && i + VEC <= V;
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            if (!whole && (i + v < 0 || i + v >= V)) continue;
            const bool in = !bad && key_of(x[v], i + v) >= keep_from;
            const float w = in && (prob || a.e) ? wt.value<IO>(x[v]) : 0.0f;
            if (in && a.e) take(best, Cand{w / a.e[e0 + v], x[v], i + v});
            if (prob) prob[e0 + v] = w * inv;
            if (kept && (!in || kept != a.logits))
                kept[e0 + v] = in || bad ? (T)x[v] : (T)-INFINITY;
        }
    }
    if (!a.e) return;                                    // no CTA reads another's memory past here
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        take(best, Cand{__shfl_xor_sync(0xffffffffu, best.s, o),
                        __shfl_xor_sync(0xffffffffu, best.x, o),
                        __shfl_xor_sync(0xffffffffu, best.i, o)});
    if (lane == 0) sh.warp_cand[warp] = best;
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < NT / 32; ++w) take(best, sh.warp_cand[w]);
        *cl.map_shared_rank(&sh.cand[rank], 0) = best;
    }
    cl.sync();
    if (rank == 0 && tid == 0) {
        best = sh.cand[0];
        for (int c = 1; c < C; ++c) take(best, sh.cand[c]);
        const bool none = bad || best.i == NO_TOK;
        a.out.tok[r] = none ? 0 : best.i;
        if (a.out.tok_prob) a.out.tok_prob[r] = none ? 0.0f : wt.value<IO>(best.x) * inv;
    }
}

// CTAs per row: the more the fewer rows, and as many as hold the row in shared memory
// where 16 do.
template <int IO>
cudaError_t sample_t(const spec_sample_cfg& c, SampleArgs& a, cudaStream_t st) {
    constexpr int VEC = Row<IO>::VEC;
    const int most = 160 * 1024;
    const int64_t groups = ((int64_t)c.V + VEC - 1) / VEC + 1;
    int sms = device_sm_count();
    if (sms < 1) sms = 1;
    int C = 1;
    while (C < MAX_CLUSTER && ((int64_t)c.R * C * 2 <= sms || (groups + C - 1) / C * 16 > most) &&
           (groups / C) > 64)
        C *= 2;
    int64_t share = (groups + C - 1) / C;
    a.resident = (int)(share * 16 > most ? most / 16 : share);
    const size_t smem = (size_t)a.resident * 16;
    cudaError_t e = cudaFuncSetAttribute(sample_rows<IO>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(sample_rows<IO>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(c.R * C));
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, sample_rows<IO>, a);
}

}  // namespace

cudaError_t launch_token_sample(const spec_sample_cfg& c, const void* logits,
                                const spec_sample_params& p, const float* e,
                                const spec_sample_out& out, void* ws, cudaStream_t st) {
    static const struct Pow2 {
        u64 t[64];
        Pow2() {
            for (int j = 0; j < 64; ++j) t[j] = (u64)(exp2(-j / 64.0) * 4611686018427387904.0);
        }
    } pow2;
    SampleArgs a{};
    a.logits = logits;
    a.p = p;
    a.e = e;
    a.out = out;
    a.ws = ws;
    a.R = c.R;
    a.V = c.V;
    a.per = c.per;
    while ((1 << a.lg) < c.V) ++a.lg;
    for (int j = 0; j < 64; ++j) a.pow2[j] = pow2.t[j];
    return c.io_dtype == SPEC_IO_BF16 ? sample_t<SPEC_IO_BF16>(c, a, st)
                                      : sample_t<SPEC_IO_F32>(c, a, st);
}

}  // namespace spec
