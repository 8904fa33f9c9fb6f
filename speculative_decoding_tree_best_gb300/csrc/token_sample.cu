// token_sample.cu -- sampling with temperature, min-p, top-k and top-p from given
// random numbers.
//
// Mathematics.  What stays is a prefix of the order (logit descending, index
// ascending): all tokens above a border value and those at it up to a border index.
// min-p gives the value directly.  top-k and top-p ask for the shortest prefix with
// F >= target: F = its length and the count k, or F = the sum of its weights and
// top_p times that of what top-k left.
//   Weights are integers, 2^-(61 - lg V) of the largest one, from an exponential
// of 2^-29 relative accuracy (a table of 2^(-j/64) and a cubic): sums of them are
// exact in 64 bits, so the border depends neither on the order of summation nor
// on fp32's rounding of long sums.
//   The draw: argmin e / w over independent exponentials e is token v with
// probability w_v / sum w.
//
// The border, by what it takes:
//   top_k small   A lower bound of the k-th largest logit: the k-th of a pool of maxima
//                 of threads' shares, or (top_k above 3/4 of the pool) the least of the
//                 values that k / C of each CTA's threads reach.  The logits from there
//                 on, few more than k, are gathered in one CTA, sorted, and all filters
//                 and the draw decided on the sorted list.
//   else          A histogram over bins of 2^-7 of a value's binade, from the maximum
//                 down, names the bin that the border is in.  bf16 logits take one
//                 value in a bin: counts are all that masses need, a weight a bin, and
//                 the tokens at the border value stay from the first on.  fp32 logits'
//                 masses are added up themselves, and the bin's tokens gathered and
//                 sorted.  What lies below the bins counts in the totals.
//   and where that is not enough (a bin too full for the list, a border below the bins)
//                 a radix selection on the key K = (logit's bits, made to order like
//                 the number; index, falling), one 52-bit integer, different for
//                 every token: a histogram of F over the top bits of K names the
//                 bin that the border is in, which becomes the next range.
//
// Data flow.  A cluster of CTAs owns a row.  It reads the row once, into shared
// memory (what does not fit is read again from L2), and each pass goes over that
// copy.  Histograms are added up by parts: each CTA takes a part of the bins from
// all (reading the others' shared memory), and tells the others its total.
//
// What bounds it: reading the logits (2 or 4 bytes a token), the random numbers of what
// stays, writing what is asked for.  Measured (graph replays, V = 151936): one bf16 row
// 10.5 us, a chain of five exchanges and a sort; 24 fp32 rows with their probabilities
// 44 us, most of it the rows with a top_p alone (one such row 30.3 us; 73 instructions a
// token over all rows, and only their clusters' SMs at work at the end); 216 bf16 rows
// filtered and written back 76 us, 131 MB at 1.7 TB/s; 256 bf16 rows without a filter 90
// us, their nucleus 148.  The last three are bound by instructions (34, 46 and 66 warp
// instructions for 32 tokens) and by the CTAs of a cluster that wait for one another; 256
// rows are 3.4 rounds of the 76 clusters that fit.  Every instantiation spills at its 64
// registers: 120 to 176 bytes stored for clusters of one to four CTAs, 432 and 452 (bf16,
// fp32) for eight, 872 and 860 for sixteen, most of it border_bin's 16 bytes from each CTA.
#include <cooperative_groups.h>
#include <math.h>

#include <atomic>

#include "serving.cuh"

namespace spec {

namespace {

namespace cg = cooperative_groups;

// Two CTAs of 512 threads to an SM, 64 registers each.  (256 rows' nucleus, then in 149
// us: four of 256 threads and clusters twice as large 179, one of 1024 and half as
// large 160; one row 10.6, 11.7 and 12.8.)
constexpr int NT = 512;
constexpr int NBIN = 4096;               // bins of counts
constexpr int NMASS = NBIN / 2;          // bins of masses
constexpr int LIST = 2048;               // tokens that the sorted list holds
constexpr int ODD = 256;                 // tokens beside the bins that are noted down
constexpr int SOME = 64;                 // of a CTA, and
constexpr int POOL = 256;                // of a cluster: maxima that the k-th largest is bounded by
constexpr int IDX_BITS = 20;             // of a key: V <= 2^20
constexpr uint32_t IDX_MAX = (1u << IDX_BITS) - 1;
constexpr int MAX_CLUSTER = 16;
constexpr int NO_TOK = 0x7fffffff;
constexpr float LOWEST = -3.4028234663852886e38f;
// weights below 2^-CUT of the largest are 0 in the sums (CUT + lg <= 63)
constexpr float CUT = 42.0f;

typedef unsigned long long u64;

struct SampleArgs {
    const void* logits;
    spec_sample_params p;
    const float* e;
    spec_sample_out out;
    void* ws;
    int R, V, per;
    int lg;                  // ceil(log2 V) + 1: sums of weights are at most 2^61
    int resident;            // 16-byte groups of a CTA's slice kept in shared memory
    uint32_t pow2[64];       // 2^(29 - j/64)
};

// What a selection finds, told to all CTAs.
struct alignas(16) Border {
    u64 from;                // the border's key, or its bin
    u64 sum;                 // F up to there, the border's own included (a bin's: before it)
    u64 target;              // what F is to reach (a bin's: what is wanted of it)
    uint32_t tokens;         // of the bin
    int state;
};
enum { NOT_FOUND = 0, FOUND = 1, NARROWED = 2, BELOW = 3 };

struct Cand {
    float w, e, x;           // the score is w / e, w and e times the same power of two
    int i;
};

// e is brought to [1, 2) or near it, so that no product of take() leaves fp32's range
// where the scores are within it (the weights may go down to 2^-126, and e as far)
__device__ __forceinline__ Cand cand_of(float w, float e, float x, int i) {
    const float f = __uint_as_float((254u - min(__float_as_uint(e) >> 23, 253u)) << 23);
    return Cand{w * f, e * f, x, i};
}

// The better one: by cross products, lowest index on ties.
__device__ __forceinline__ void take(Cand& a, const Cand& b) {
    const float p = b.w * a.e, q = a.w * b.e;
    if (p > q || (p == q && b.i < a.i)) a = b;
}

// A request's parameters, made by one thread (64-bit floating point is slow here).
struct Params {
    float c, c_lo, far;      // 2 log2(e) / temperature; see Weights
    float min_p;
    double min_low;          // temperature ln(min_p)
    u64 top_p;               // in units of 2^-64; 0: off
    int top_k;               // 0: off
    float low;               // the least logit that min_p leaves
    uint32_t bits;
};

struct Shared {
    union alignas(16) {
        uint32_t count[NBIN + 32];       // the last ones take what belongs nowhere
        uint32_t mass[3][NMASS];         // three parts of 15 bits and more
        u64 list[LIST];
    };
    uint2 pow2[64];
    u64 part[NT / 32];
    u64 cta_sum[MAX_CLUSTER], cta_rest[MAX_CLUSTER];
    u64 near_0, rest;                    // F of what the bins do not hold: see bins()
    uint32_t odd_ones;
    float odd[ODD];
    Border border;
    Params prm;
    Cand cand[MAX_CLUSTER];
    Cand warp_cand[NT / 32];
    float2 cta_max[MAX_CLUSTER];         // and the value that enough of its threads reach
    float warp_max[NT / 32];
    float some[SOME], pool[NT], bound;   // for the bound on the top_k-th: see the kernel
    float cta_z[MAX_CLUSTER];
    uint32_t ties[MAX_CLUSTER];
    uint32_t listed[MAX_CLUSTER];        // tokens in the list, by the CTA they came from
    uint32_t my_listed;
    int border_index;
};

__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// The cluster's barrier, which the block enters as a whole.  The contract of arrive and
// wait asks for no barrier of the block here, and why it matters was not found: with
// warps that arrived by themselves, each converged, 33 of 1000 calls with 30 fp32 rows,
// L2 cold, left one token too many (which fits one key missing from the first CTA's
// list); with the block's barrier none of 2500 did, at 1 % of the time.  It was not seen
// again: copies of that kernel and of this one, without the block's barrier but with
// their path fixed and their indexes held in range, gave the same borders in 6000 such
// calls each.
__device__ __forceinline__ void cluster_arrive() {
    __syncthreads();
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
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

// added to a float under 2^22, leaves it rounded to an integer in the low bits
constexpr float MAGIC = 12582912.0f;
constexpr int MAGIC_BITS = 0x4b400000;

// The softmax's weights of a row: 2^-((m - x) / 2 c), c = 2 log2(e) / temperature in two
// parts.  (Halves, since m - x can leave fp32's range where m and x do not.)
struct Weights {
    float m, h, c, c_lo, far;    // h = m / 2; far: weights beyond it are 0 in the sums
    int lg;
    const uint2* pow2;           // (2^(29 - j/64) - MAGIC_BITS, 2^(29 - j/64) as a float)

    // (m - x) / 2
    __device__ __forceinline__ float below(float x) const { return fmaf(-0.5f, x, h); }
    // the exponent below(x) c and what the roundings of both leave (of bf16 values too: a
    // difference of numbers more than 2^16 apart is rounded)
    __device__ __forceinline__ float exponent(float x, float d, float& rest) const {
        const float y = d * c, b = d - h;
        rest = fmaf(d, c_lo, fmaf(d, c, -y));
        rest = fmaf((h - (d - b)) - fmaf(0.5f, x, b), c, rest);
        return y;
    }
    // as an integer, of 2^(62 - lg) for the largest, rounded down; without branches, so
    // that several are under way at once.  The exponent's multiple of 1/64 is looked up
    // (2^(29 - j/64), rounded) and the rest, under 0.0055, is a cubic whose product with
    // that is rounded by the magic number: 30 bits in all.  (A 62-bit product and a
    // rounded shift: 24 fp32 rows 48.5 us instead of 45.3.)
    __device__ __forceinline__ u64 fixed(float x) const {
        const float d = below(x);
        const bool some = d <= far;
        float rest;
        const float y = exponent(some ? x : m, some ? d : 0.0f, rest);
        const float n = fmaf(y, 64.0f, MAGIC);                 // rounded to an integer
        const float r = fmaf(n - MAGIC, -0x1p-6f, y) + rest;
        // 2^-r - 1
        const float q = r * fmaf(r, fmaf(r, -0.05550410866482158f, 0.2402265069591007f),
                                 -0.6931471805599453f);
        const uint2 t = pow2[__float_as_int(n) & 63];
        const uint32_t w = t.x + (uint32_t)__float_as_int(fmaf(q, __uint_as_float(t.y), MAGIC));
        const int s = (__float_as_int(n) >> 6) + (lg - (MAGIC_BITS >> 6));
        return some ? (u64)w << 33 >> s : 0;
    }
    // as a float (1 for the largest)
    __device__ __forceinline__ float value(float x) const {
        float rest;
        const float y = exponent(x, below(x), rest);
        if (!(y < 200.0f)) return 0.0f;
        return ex2(-y) * fmaf(rest, -0.6931471805599453f, 1.0f);
    }
};

template <int IO> struct Row {
    using T = typename io_t<IO>::T;
    static constexpr int VEC = 16 / sizeof(T);
    const T* logits;             // the row's first element, which may stand inside a
    const uint4* first;          // 16-byte group: the group
    int V, off;                  // and its place there
    int whole_lo, whole_n;       // groups of the row's elements only: [whole_lo, + whole_n)
    int64_t r0;                  // the row's first element in the tensor
    int lo, hi;                  // this CTA's groups, from `first`
    const uint4* smem;
    int resident;

    __device__ __forceinline__ Row(const T* tensor, int row, int vocab) : V(vocab) {
        r0 = (int64_t)row * vocab;
        logits = tensor + r0;
        off = (int)(r0 % VEC);
        first = reinterpret_cast<const uint4*>(logits - off);
        whole_lo = off != 0;
        whole_n = (off + V) / VEC - whole_lo;
    }
    __device__ __forceinline__ int groups() const { return (off + V + VEC - 1) / VEC; }
    __device__ __forceinline__ bool whole(int g) const {
        return (unsigned)(g - whole_lo) < (unsigned)whole_n;
    }
    // where in the row the group begins
    __device__ __forceinline__ int index(int g) const { return g * VEC - off; }
    // group g from memory, with what is not the row's as -inf
    __device__ __forceinline__ uint4 load(int g) const {
        if (whole(g)) return first[g];
        return load_edge(g);
    }
    __device__ __noinline__ uint4 load_edge(int g) const {
        const T low = IO == SPEC_IO_F32 ? (T)-INFINITY : (T)__uint_as_float(0xff800000u);
        alignas(16) T x[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const int i = index(g) + v;
            x[v] = i >= 0 && i < V ? logits[i] : low;
        }
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
    // the largest of a group, NaN where there is one
    static __device__ __forceinline__ float most(const uint4& u) {
        if constexpr (IO == SPEC_IO_F32) {
            return max_nan(max_nan(__uint_as_float(u.x), __uint_as_float(u.y)),
                           max_nan(__uint_as_float(u.z), __uint_as_float(u.w)));
        } else {
            const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
            const float2 y = __bfloat1622float2(
                __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3])));
            return max_nan(y.x, y.y);
        }
    }
    // f(x, index in the row) for the elements of groups [from, to), `step` apart (-inf
    // beside the row)
    template <typename F>
    __device__ __forceinline__ void range(int from, int to, F&& f, int step = 1) const {
        for (int g = from; g < to; g += step) {
            float x[VEC];
            unpack(get(g), x);
            const int i = index(g);
#pragma unroll
            for (int v = 0; v < VEC; ++v) f(x[v], i + v);
        }
    }
    // the same for all of this CTA's elements, a thread's own groups
    template <typename F> __device__ __forceinline__ void each(F&& f) const {
        range(lo + threadIdx.x, hi, f, NT);
    }
};

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

// What stays of a CTA's slice: logits above v, and those at v up to index `last`.
struct Kept {
    float v;
    int last;
    __device__ __forceinline__ bool has(float x, int i) const {
        return (x > v) | ((x == v) & (i <= last));       // without branches
    }
    // whether x alone says: all of the logits at v stay
    __device__ __forceinline__ bool by_value() const { return last == (int)IDX_MAX; }
};

__device__ __forceinline__ float value_of(u64 key) {
    const uint32_t k = (uint32_t)(key >> IDX_BITS);
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
// what stays when of those at v none do: the numbers above v
__device__ __forceinline__ Kept above_value(float v) {
    return Kept{value_of((u64)(key_of(v) + 1) << IDX_BITS), (int)IDX_MAX};
}
__device__ __forceinline__ int index_of(u64 key) { return IDX_MAX - ((uint32_t)key & IDX_MAX); }

// A group with -inf for what does not stay.  Two bf16 values at a time where the value
// alone says; the least bf16 value that stays is rounded up.
template <int IO> struct Filter {
    Kept kept;
    uint32_t v2;
    __device__ __forceinline__ Filter(const Kept& k) : kept(k), v2(0) {
        if (IO == SPEC_IO_BF16) {
            const __nv_bfloat162 h = __bfloat162bfloat162(__float2bfloat16_ru(k.v));
            v2 = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    __device__ __forceinline__ uint32_t two(uint32_t w, int i) const {
        uint32_t mask;
        if (kept.by_value()) {
            mask = __hge2_mask(*reinterpret_cast<const __nv_bfloat162*>(&w),
                               *reinterpret_cast<const __nv_bfloat162*>(&v2));
        } else {
            mask = (kept.has(__uint_as_float(w << 16), i) ? 0xffffu : 0u) |
                   (kept.has(__uint_as_float(w & 0xffff0000u), i + 1) ? 0xffff0000u : 0u);
        }
        return (w & mask) | (0xff80ff80u & ~mask);
    }
    __device__ __forceinline__ uint32_t one(uint32_t w, int i) const {
        return kept.has(__uint_as_float(w), i) ? w : 0xff800000u;
    }
    // u: the group, i: the index of its first
    __device__ __forceinline__ uint4 operator()(const uint4& u, int i) const {
        if constexpr (IO == SPEC_IO_BF16)
            return make_uint4(two(u.x, i), two(u.y, i + 2), two(u.z, i + 4), two(u.w, i + 6));
        else
            return make_uint4(one(u.x, i), one(u.y, i + 1), one(u.z, i + 2), one(u.w, i + 3));
    }
};

template <int C> struct Ctx {
    cg::cluster_group& cl;
    Shared& sh;
    int rank, tid;
    Weights wt;

    // the sum of the CTAs' x before this one, and of all; of their `rest`
    __device__ __forceinline__ void totals(u64 x, u64& before, u64& all, u64 mine_rest, u64& rest) {
        if (tid < C) {
            *cl.map_shared_rank(&sh.cta_sum[rank], tid) = x;
            *cl.map_shared_rank(&sh.cta_rest[rank], tid) = mine_rest;
        }
        cluster_sync();
        before = all = rest = 0;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const u64 y = sh.cta_sum[c];
            before += c < rank ? y : 0;
            all += y;
            rest += sh.cta_rest[c];
        }
    }
    __device__ __forceinline__ void tell(const Border& b, bool all = true) {
        if (!all) {                                      // this CTA alone
            sh.border = b;
            return;
        }
        const uint4* src = reinterpret_cast<const uint4*>(&b);
        const uint4 lo = src[0], hi = src[1];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            uint4* to = reinterpret_cast<uint4*>(cl.map_shared_rank(&sh.border, c));
            to[0] = lo;
            to[1] = hi;
        }
    }
};

// The target of a prefix's F: `want`, or that many 2^-64 of `all`, rounded up.
template <bool MASS> __device__ __forceinline__ u64 target_of(u64 want, u64 all) {
    if (!MASS) return want;
    return max(__umul64hi(all, want) + (all * want != 0), (u64)1);
}

// ---- bins: signed steps of 2^-7 of a binade from 0 (bf16's values), the smallest
// magnitudes as 0

constexpr int NEAR_0 = (127 - 12) << 7;                  // 2^-12
constexpr int FARTHEST = 0x7f80 - NEAR_0;                // infinity

__device__ __forceinline__ int step_of(float x) {
    const int i = __float_as_int(x) >> 16, sign = i >> 31;
    return (max((i & 0x7fff) - NEAR_0, 0) ^ sign) - sign;
}
__device__ __forceinline__ float step_value(int s) {
    const uint32_t b = (uint32_t)(abs(s) + NEAR_0) << 16;
    return s == 0 ? 0.0f : __uint_as_float(s < 0 ? b | 0x80000000u : b);
}
// the least fp32 number with that step
__device__ __forceinline__ float step_least(int s) {
    const uint32_t b = (uint32_t)(abs(s) + NEAR_0) << 16;
    return __uint_as_float(s > 0 ? b : b | 0x8000ffffu);
}

// What the bins hold: the tokens' number (top_k), the number at a bf16 value, which
// its weight makes a mass, or fp32 logits' masses, two steps to a bin.
enum { COUNTS, VALUES, MASSES };

template <int KIND> __device__ __forceinline__ int bin_of(int top, float x) {
    const int d = top - step_of(x);
    return KIND == MASSES ? d >> 1 : d;
}

// Adds to bin `b` of masses, in three parts of the weight (at most 2^61 / V): the first
// two of 15 bits, so that a CTA's 2^16 tokens do not overflow them, nor V tokens the
// third.  (64-bit atomics on shared memory are loops: 6 to 28 times as long as 32-bit
// ones, 1000 a thread of two CTAs an SM in 300 to 1380 us instead of 49.)
__device__ __forceinline__ void add_mass(Shared& sh, int b, u64 w) {
    atomicAdd(&sh.mass[0][b], (uint32_t)w & 0x7fffu);
    atomicAdd(&sh.mass[1][b], (uint32_t)(w >> 15) & 0x7fffu);
    atomicAdd(&sh.mass[2][b], (uint32_t)(w >> 30));
}

// This CTA's histogram of `kept`, bin 0 the maximum's (`top` its step).  Beside it
// sh.rest has F of what lies below the bins, and with VALUES sh.near_0 that of the
// bin of 0, whose count says nothing of its weights.
template <int KIND, int IO, int C>
__device__ __forceinline__ void bins(Ctx<C>& k, const Row<IO>& row, const Kept& kept, int top) {
    Shared& sh = k.sh;
    for (int b = k.tid; b < 3 * NMASS; b += NT) sh.mass[0][b] = 0;
    if (k.tid == 0) {
        sh.near_0 = sh.rest = 0;
        sh.odd_ones = 0;
    }
    __syncthreads();
    constexpr int END = KIND == MASSES ? NMASS : NBIN, VEC = Row<IO>::VEC;
    const float far = k.wt.far;
    // Odd ones, seldom there, are noted down for later: below the bins, or near 0
    // (where a bin holds more than one value).  Taken as they came, they made the pass
    // twice as long: the block waits for the warp with most of them.
    // (conditions of a token are joined without branches)
    auto beside = [&](int b) { return (b >= END) | (KIND == VALUES ? b == top : false); };
    // What does not stay is -inf, and below the bins; where what stays reaches there too
    // (deep), those found there are told apart later.
    const bool deep = bin_of<KIND>(top, kept.v) >= END;
    const Filter<IO> filter(kept);
    const int trash = (KIND == MASSES ? 0 : NBIN) + k.tid % 32;     // (nothing added to masses)
    for (int g = row.lo + k.tid; g < row.hi; g += NT) {
        const uint4 u = filter(row.get(g), row.index(g));
        float x[VEC];
        Row<IO>::unpack(u, x);
        bool odd = false;
        u64 w[VEC];
        if (KIND == MASSES)
#pragma unroll
            for (int v = 0; v < VEC; ++v) w[v] = k.wt.fixed(x[v]);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const int b = bin_of<KIND>(top, x[v]);
            odd |= KIND == VALUES ? b == top : false;
            if (deep) odd |= b >= END;
            // (a branch for each token costs more than an addition for nothing)
            if (KIND == MASSES) add_mass(sh, b < END ? b : trash, b < END ? w[v] : 0);
            else atomicAdd(&sh.count[b < END ? b : trash], 1u);
        }
        if (odd)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                if (!(x[v] > -INFINITY) || !beside(bin_of<KIND>(top, x[v]))) continue;
                if (KIND != COUNTS && !(k.wt.below(x[v]) <= far)) continue;      // weighs nothing
                const uint32_t at = atomicAdd(&sh.odd_ones, 1u);
                if (at < ODD) sh.odd[at] = x[v];
            }
    }
    u64 near = 0, rest = 0;
    auto look = [&](float x) {
        if (KIND == COUNTS) ++rest;
        else (bin_of<KIND>(top, x) < END ? near : rest) += k.wt.fixed(x);
    };
    __syncthreads();
    if (sh.odd_ones <= ODD) {
        for (int j = k.tid; j < (int)sh.odd_ones; j += NT) look(sh.odd[j]);
    } else {
        row.each([&](float x, int i) {
            if (beside(bin_of<KIND>(top, x)) && kept.has(x, i)) look(x);
        });
    }
    if (sh.odd_ones) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            near += __shfl_xor_sync(0xffffffffu, near, o);
            rest += __shfl_xor_sync(0xffffffffu, rest, o);
        }
        if (k.tid % 32 == 0) {
            if (near) atomicAdd(&sh.near_0, near);
            if (rest) atomicAdd(&sh.rest, rest);
        }
    }
}

// The border bin of all CTAs' histograms: tells them the bin and its tokens (but with
// MASSES), `sum` = F before it and `target` = what is wanted of it (BELOW: the border
// is below the bins).  The cluster has not synchronised since bins().
template <int KIND, int IO, int C>
__device__ __forceinline__ void border_bin(Ctx<C>& k, u64 want, int top) {
    Shared& sh = k.sh;
    cluster_sync();
    // bins [from, from + RUN) are this thread's: 16-byte pieces of four
    constexpr int N = KIND == MASSES ? NMASS : NBIN;
    constexpr int PART = N / C, RUN = PART / NT < 4 ? 4 : PART / NT;
    const bool mine = k.tid * RUN < PART;
    const int from = k.rank * PART + k.tid * RUN;
    uint32_t n[RUN];
    u64 f[RUN], s = 0;
#pragma unroll
    for (int j = 0; j < RUN; j += 4) {
        f[j] = f[j + 1] = f[j + 2] = f[j + 3] = 0;
#pragma unroll
        for (int part = 0; part < (KIND == MASSES ? 3 : 1); ++part) {
            uint4 x[C];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                x[c] = make_uint4(0, 0, 0, 0);
                if (mine)
                    x[c] = *reinterpret_cast<const uint4*>(k.cl.map_shared_rank(
                        &sh.mass[0][part * NMASS + from + j], (k.rank + c) % C));
            }
            n[j] = n[j + 1] = n[j + 2] = n[j + 3] = 0;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const uint32_t y[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (KIND == MASSES) f[j + i] += (u64)y[i] << (15 * part);
                    else n[j + i] += y[i];
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < RUN; ++j) {
        if (KIND != MASSES) f[j] = n[j];
        if (KIND == VALUES) {
            if (from + j == top) f[j] = 0;
            else if (n[j]) f[j] *= k.wt.fixed(step_value(top - from - j));
            if (mine && from + j == top)
                for (int c = 0; c < C; ++c) f[j] += *k.cl.map_shared_rank(&sh.near_0, c);
        }
        s += f[j];
    }
    u64 mine_all, before_me, all, rest;
    u64 at = block_prefix(s, sh.part, mine_all);
    k.totals(mine_all, before_me, all, sh.rest, rest);
    at += before_me;
    const u64 target = target_of<KIND != COUNTS>(want, all + rest);
    if (k.tid == 0 && k.rank == 0 && all < target)
        k.tell(Border{0, 0, 0, 0, all + rest < target ? NOT_FOUND : BELOW});
    if (at < target && target <= at + s) {               // one thread of the cluster, or none
        Border b{};
#pragma unroll
        for (int j = 0; j < RUN; ++j) {
            if (at < target && target <= at + f[j])
                b = Border{(u64)(from + j), at, target - at, n[j], NARROWED};
            at += f[j];
        }
        k.tell(b);
    }
    cluster_sync();
}

// Radix selection: the largest key t of `kept` such that F over its {K >= t} reaches
// the target; NOT_FOUND where it does not.
template <bool MASS, int IO, int C>
__device__ Border radix(Ctx<C>& k, const Row<IO>& row, const Kept& kept, u64 want) {
    Shared& sh = k.sh;
    const int tid = k.tid;
    // the range is the same in all CTAs (kept.v need not be: see first_ties)
    u64 lo = (u64)key_of(sh.prm.low) << IDX_BITS, hi = (u64)key_of(k.wt.m) << IDX_BITS | IDX_MAX;
    u64 above = 0, target = want;
    for (int pass = 0;; ++pass) {
        for (int b = tid; b < 3 * NMASS; b += NT) sh.mass[0][b] = 0;
        __syncthreads();
        const u64 span = hi - lo;
        const int shift = max(0, 64 - __clzll((long long)span) - 11);     // span >> shift < NMASS
        row.each([&](float x, int i) {
            const u64 key = key_of(x, i);
            if (key < lo || key > hi || !kept.has(x, i)) return;
            const int bin = (int)((hi - key) >> shift);
            if (MASS) add_mass(sh, bin, k.wt.fixed(x));
            else atomicAdd(&sh.count[bin], 1u);
        });
        cluster_sync();
        constexpr int PART = NMASS / C, RUN = PART / NT < 1 ? 1 : PART / NT;
        const int from = k.rank * PART + tid * RUN;
        u64 f[RUN], s = 0;
#pragma unroll
        for (int j = 0; j < RUN; ++j) {
            f[j] = 0;
            if (tid * RUN < PART) {
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    // (the counts lie where the first part does)
#pragma unroll
                    for (int part = 0; part < (MASS ? 3 : 1); ++part)
                        f[j] += (u64)*k.cl.map_shared_rank(&sh.mass[part][from + j], c)
                                << (15 * part);
                }
            }
            s += f[j];
        }
        u64 mine_all, before_me, all, rest;
        u64 at = block_prefix(s, sh.part, mine_all);
        k.totals(mine_all, before_me, all, 0, rest);
        at += before_me + above;
        if (pass == 0) target = target_of<MASS>(want, all);
        if (tid == 0 && k.rank == 0 && above + all < target)
            k.tell(Border{0, 0, 0, 0, NOT_FOUND});
        if (at < target && target <= at + s) {
            Border b{};
#pragma unroll
            for (int j = 0; j < RUN; ++j) {
                if (at < target && target <= at + f[j])
                    b = Border{(u64)(from + j), at, f[j], 0, NARROWED};
                at += f[j];
            }
            k.tell(b);
        }
        cluster_sync();
        Border b = sh.border;
        if (b.state == NOT_FOUND) return b;
        above = b.sum;
        hi -= b.from << shift;
        if (hi - lo >= 1ull << shift) lo = hi - (1ull << shift) + 1;
        if (lo == hi) return Border{lo, b.sum + b.target, 0, 0, FOUND};
    }
}

// What stays of this CTA's when of the tokens at value v the first `want` of all do.
// `mine`: the CTA's number of them.
template <int IO, int C>
__device__ __forceinline__ Kept first_ties(Ctx<C>& k, const Row<IO>& row, const Kept& in, float v,
                                           u64 want, uint32_t mine) {
    Shared& sh = k.sh;
    if (k.tid < C) *k.cl.map_shared_rank(&sh.ties[k.rank], k.tid) = mine;
    cluster_sync();
    u64 before = 0;
    for (int c = 0; c < k.rank; ++c) before += sh.ties[c];
    if (in.v > v) return in;                             // its ties left before
    if (want <= before) return above_value(v);
    if (want >= before + mine) return Kept{v, in.v == v ? in.last : (int)IDX_MAX};
    // the border is here: a run of groups a thread, in order
    const uint32_t left = (uint32_t)(want - before);
    const int n = row.hi - row.lo, run = (n + NT - 1) / NT;
    const int g0 = min(row.hi, row.lo + k.tid * run), g1 = min(row.hi, g0 + run);
    uint32_t count = 0;
    row.range(g0, g1, [&](float x, int i) { count += x == v && in.has(x, i); });
    u64 all;
    uint32_t at = (uint32_t)block_prefix(count, sh.part, all);
    if (at < left && left <= at + count)
        row.range(g0, g1, [&](float x, int i) {
            if (x == v && in.has(x, i) && ++at == left) sh.border_index = i;
        });
    __syncthreads();
    return Kept{v, sh.border_index};
}

// Sorts n keys (1 <= n <= LIST), the largest first, and returns where they are in `list`
// (which has room for the next power of two).  Up to RANKED keys by counting how many
// are larger, the threads shared out over the keys; more in a bitonic network.
constexpr int RANKED = NT;
static_assert(2 * RANKED <= LIST);

__device__ __forceinline__ u64* sort_list(u64* list, int n) {
    if (n <= RANKED) {
        int sh = 0;                                      // 2^sh threads to a key
        while (n << (sh + 1) <= NT && sh < 3) ++sh;
        const int at = threadIdx.x >> sh, part = threadIdx.x & ((1 << sh) - 1);
        const u64 x = at < n ? list[at] : 0;
        if (threadIdx.x == 0 && n % 2) list[n] = 0;      // keys are read in pairs
        __syncthreads();
        const ulonglong2* pairs = reinterpret_cast<const ulonglong2*>(list);
        int above = 0;
#pragma unroll 4
        for (int i = part; 2 * i < n; i += 1 << sh) {
            const ulonglong2 y = pairs[i];
            above += (y.x > x) + (y.y > x);
        }
        for (int o = 1; o < 1 << sh; o *= 2) above += __shfl_xor_sync(0xffffffffu, above, o);
        if (at < n && part == 0) list[RANKED + above] = x;
        __syncthreads();
        return list + RANKED;
    }
    int size = RANKED;
    while (size < n) size *= 2;
    for (int i = n + threadIdx.x; i < size; i += NT) list[i] = 0;
    __syncthreads();
    for (int k = 2; k <= size; k *= 2)
        for (int j = k / 2; j > 0; j /= 2) {
            for (int t = threadIdx.x; t < size / 2; t += NT) {
                const int a = 2 * t - (t & (j - 1)), b = a + j;
                const u64 x = list[a], y = list[b];
                if ((x < y) == ((a & k) == 0)) {
                    list[a] = y;
                    list[b] = x;
                }
            }
            __syncthreads();
        }
    return list;
}

__device__ __forceinline__ void take_across(Cand& best, int o) {
    take(best, Cand{__shfl_xor_sync(0xffffffffu, best.w, o),
                    __shfl_xor_sync(0xffffffffu, best.e, o),
                    __shfl_xor_sync(0xffffffffu, best.x, o),
                    __shfl_xor_sync(0xffffffffu, best.i, o)});
}

// The block's best candidate, in thread 0.
__device__ __forceinline__ void block_best(Cand& best, Shared& sh) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) take_across(best, o);
    if (threadIdx.x % 32 == 0) sh.warp_cand[threadIdx.x / 32] = best;
    __syncthreads();
    if (threadIdx.x == 0)
        for (int w = 1; w < NT / 32; ++w) take(best, sh.warp_cand[w]);
}

constexpr int SMALL_K = 1024;

// The least fp32 number that `want` of the n values in v reach, to the accuracy of a
// step (-inf where fewer are above -inf).  For one warp; n <= NT.
__device__ __forceinline__ float reached(const float* v, int n, int want) {
    const int lane = threadIdx.x % 32;
    int s[NT / 32];
    int lo = FARTHEST, hi = -FARTHEST;
#pragma unroll
    for (int j = 0; j < NT / 32; ++j) {
        s[j] = -FARTHEST - 1;
        if (lane + 32 * j < n) {
            s[j] = step_of(v[lane + 32 * j]);
            lo = min(lo, s[j]);
            hi = max(hi, s[j]);
        }
    }
    lo = __reduce_min_sync(0xffffffffu, lo);              // all of them reach lo
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (want > n) lo = hi = -FARTHEST;
    while (lo < hi) {
        const int mid = lo + (hi - lo + 1) / 2;
        unsigned count = 0;
#pragma unroll
        for (int j = 0; j < NT / 32; ++j) count += s[j] >= mid;
        if ((int)__reduce_add_sync(0xffffffffu, count) >= want) lo = mid;
        else hi = mid - 1;
    }
    return lo <= -FARTHEST ? -INFINITY : step_least(lo);
}

// n values in `v` (n a power of two, at most NT / 2), and which of them is how many below
// the largest: f(that number, value), once for each, in the threads that have it.
template <int N, typename P> __device__ __forceinline__ void ranked(const float* v, P&& f) {
    constexpr int PER = NT / N < 8 ? NT / N : 8;         // threads to a value
    const int at = threadIdx.x / PER, part = threadIdx.x % PER;
    if (threadIdx.x >= N * PER) return;
    const float x = v[at];
    int above = 0;
#pragma unroll
    for (int i = part; i < N; i += PER) above += (v[i] > x) | ((v[i] == x) & (i < at));
#pragma unroll
    for (int o = 1; o < PER; o *= 2) above += __shfl_xor_sync(0xffffffffu, above, o);
    if (part == 0) f(above, x);
}

// The logits x of the CTA's slice with f(x, i), all of them `least` or more, into its
// part of the first CTA's list, of LIST / C keys.  false: a part is too short for them
// (the same for all CTAs).
template <int IO, int C, typename P>
__device__ __forceinline__ bool gather(Ctx<C>& k, const Row<IO>& row, bool any, float least,
                                       P&& f) {
    Shared& sh = k.sh;
    if (any)
        for (int g = row.lo + k.tid; g < row.hi; g += NT) {
            const uint4 u = row.get(g);
            if (!(Row<IO>::most(u) >= least)) continue;
            float x[Row<IO>::VEC];
            Row<IO>::unpack(u, x);
            const int i = row.index(g);
#pragma unroll
            for (int v = 0; v < Row<IO>::VEC; ++v) {
                if (!f(x[v], i + v)) continue;
                const uint32_t at = atomicAdd(&sh.my_listed, 1u);
                if (at < LIST / C)
                    *k.cl.map_shared_rank(&sh.list[k.rank * (LIST / C) + at], 0) =
                        key_of(x[v], i + v);
            }
        }
    __syncthreads();
    const uint32_t mine = sh.my_listed;
    if (k.tid < C) *k.cl.map_shared_rank(&sh.listed[k.rank], k.tid) = mine;
    cluster_sync();
    if (k.tid == 0) sh.my_listed = 0;                    // (all have read it)
    bool fits = true;
#pragma unroll
    for (int c = 0; c < C; ++c) fits &= sh.listed[c] <= LIST / C;
    return fits;
}

// The border in the first CTA's list (its threads call this): the
// shortest prefix whose mass reaches `target` (0: top_p of that of the first `limit`),
// without both the first `limit`.  Tells all CTAs, or this one alone, the border with
// `above` added to its sum, and with e makes the draw.
template <int IO, int C>
__device__ __forceinline__ void solve_list(Ctx<C>& k, const Row<IO>& row, int limit, u64 top_p,
                                           u64 target, u64 above, bool all, const float* e,
                                           Cand& best) {
    Shared& sh = k.sh;
    const int tid = k.tid;
    // the parts moved together
    int n = 0;
    {
        constexpr int PART = LIST / C, PER = NT / C;     // threads to a part
        const int part = tid / PER;
        int to = 0;
        u64 key[PART / PER];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int y = (int)sh.listed[c];
            if (c < part) to += y;
            n += y;
        }
        const int mine = (int)sh.listed[part];
#pragma unroll
        for (int j = 0; j < PART / PER; ++j)
            if (tid % PER + j * PER < mine) key[j] = sh.list[part * PART + tid % PER + j * PER];
        __syncthreads();
#pragma unroll
        for (int j = 0; j < PART / PER; ++j)
            if (tid % PER + j * PER < mine) sh.list[to + tid % PER + j * PER] = key[j];
        __syncthreads();
    }
    limit = min(n, limit);
    if (n <= NT && n > 2 * limit) {
        // most are not among the first `limit`: those below the limit's step leave
        const u64 key = tid < n ? sh.list[tid] : 0;
        sh.pool[tid] = tid < n ? value_of(key) : -INFINITY;
        __syncthreads();
        if (tid < 32) {
            const float x = reached(sh.pool, n, limit);
            if (tid == 0) sh.bound = x;
        }
        __syncthreads();
        const bool stay = tid < n && value_of(key) >= sh.bound;
        const unsigned mask = __ballot_sync(0xffffffffu, stay);
        if (tid % 32 == 0) sh.part[tid / 32] = __popc(mask);
        __syncthreads();
        int at = __popc(mask & ((1u << (tid % 32)) - 1));
        n = 0;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) {
            if (w < tid / 32) at += (int)sh.part[w];
            n += (int)sh.part[w];
        }
        if (stay) sh.list[at] = key;
        __syncthreads();
    }
    const u64* list = sort_list(sh.list, n);
    // a run of keys a thread; their random numbers on their way meanwhile
    const int run = n <= NT ? 1 : LIST / NT;
    u64 w[LIST / NT], s = 0, total;
    float ex[LIST / NT], x[LIST / NT];
    int i[LIST / NT];
#pragma unroll
    for (int j = 0; j < LIST / NT; ++j) {
        const int at = tid * run + j;
        w[j] = 0;
        if (j >= run || at >= limit) continue;
        x[j] = value_of(list[at]);
        i[j] = index_of(list[at]);
        if (e) ex[j] = e[i[j]];
        w[j] = k.wt.fixed(x[j]);
        s += w[j];
    }
    u64 before = block_prefix(s, sh.part, total);
    const bool by_mass = target || top_p;
    if (top_p) target = target_of<true>(top_p, total);
#pragma unroll
    for (int j = 0; j < LIST / NT; ++j) {
        const int at = tid * run + j;
        if (j >= run || at >= limit) continue;
        const bool in = !by_mass || before < target;
        if (in && (by_mass ? target <= before + w[j] : at == limit - 1))
            k.tell(Border{list[at], above + before + w[j], 0, 0, FOUND}, all);
        if (in && e) take(best, cand_of(k.wt.value(x[j]), ex[j], x[j], i[j]));
        before += w[j];
    }
}

// Narrows `kept` to its shortest prefix whose F reaches the target; it stays as it is
// where F never does.  MASS leaves the sum of its weights in `sum`.
template <bool MASS, int IO, int C>
__device__ __forceinline__ void select(Ctx<C>& k, const Row<IO>& row, Kept& kept, u64 want,
                                       u64& sum) {
    constexpr int KIND = !MASS ? COUNTS : (IO == SPEC_IO_BF16 ? VALUES : MASSES);
    Shared& sh = k.sh;
    const int top = step_of(k.wt.m);
    Border b{0, 0, 0, 0, BELOW};
    if (top + FARTHEST >= NBIN) {                        // -inf is below the bins
        bins<KIND, IO>(k, row, kept, top);
        border_bin<KIND, IO>(k, want, top);
        b = sh.border;
        if (b.state == NOT_FOUND) return;
    }
    if (b.state == NARROWED) {
        const int bin = (int)b.from, s = top - bin;
        if (IO == SPEC_IO_BF16 && s != 0) {              // one value
            const float v = step_value(s);
            const u64 w = MASS ? k.wt.fixed(v) : 1;
            const u64 n = (b.target + w - 1) / w;
            if (MASS) sum = b.sum + n * w;
            if (n < b.tokens) kept = first_ties<IO>(k, row, kept, v, n, sh.count[bin]);
            else if (!(kept.v > v)) kept = Kept{v, kept.v == v ? kept.last : (int)IDX_MAX};
            return;                                      // (above v: its ties left before)
        }
        b.state = BELOW;
        if (gather<IO>(k, row, true, kept.v, [&](float x, int i) {
                return bin_of<KIND>(top, x) == bin && kept.has(x, i);
            })) {
            Cand none;
            if (k.rank == 0)
                solve_list<IO>(k, row, MASS ? LIST : (int)b.target, 0, MASS ? b.target : 0, b.sum,
                               true, nullptr, none);
            cluster_sync();
            b = sh.border;
        }
    }
    if (b.state != FOUND) b = radix<MASS, IO>(k, row, kept, want);
    if (b.state == NOT_FOUND) return;
    if (MASS) sum = b.sum;
    kept = Kept{value_of(b.from), index_of(b.from)};
}

// The race over what stays of this CTA's slice: `best` is the warp's best candidate
// in all its lanes.
//   A token is looked at where w / e can be above the best so far, that is
// log2 e < log2 w + log2(best.e / best.w); and bits(e) 2^-23 - 127 is at most log2 e
// (the chord is below the logarithm), which makes the test a multiply-add and an
// integer comparison, in units of 2^-7.  A group passes it seldom after the first.
// (256 rows without a filter: 103 us with two products and an exponential a token, 90
// with this test and the filter on two values at once, 56 million instructions.)
template <int IO, int C>
__device__ __forceinline__ void draw(const Ctx<C>& k, const Row<IO>& row, const Kept& kept,
                                     const float* e, Cand& best) {
    constexpr int VEC = Row<IO>::VEC;
    const float c = k.wt.c, c7 = fminf(c * 128.0f, 3.0e38f);
    const Filter<IO> filter(kept);
    float bar = 3.0e38f;                                 // everything passes
    // two units above, for the roundings of the test
    auto raise_bar = [&]() {
        bar = (best.w > 0.0f) & (best.e > 0.0f)
                  ? (__log2f(best.e) - __log2f(best.w) + 127.0f) * 128.0f + 2.0f + MAGIC : 3.0e38f;
    };
    // all the random numbers on their way into L2 at once (256 rows without a filter
    // 95 -> 88 us)
    for (int g = row.lo + k.tid; g < row.hi; g += NT)
        if (Row<IO>::most(row.get(g)) >= kept.v)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(e + max(row.index(g), 0)));
    bool shared_best = false;
    for (int g = row.lo + k.tid - k.tid % 32;; g += NT) {              // the same for the warp
        const int at = g + k.tid % 32, i = row.index(at);
        bool look = false;
        uint4 u;
        float ex[VEC];
        if (at < row.hi) {
            u = row.get(at);
            look = Row<IO>::most(u) >= kept.v;
        }
        if (look) {
            u = filter(u, i);
            if (row.whole(at)) {
#pragma unroll
                for (int v = 0; v < VEC; v += 4)
                    *reinterpret_cast<float4*>(&ex[v]) =
                        __ldg(reinterpret_cast<const float4*>(e + i + v));
            } else {
#pragma unroll
                for (int v = 0; v < VEC; ++v) ex[v] = i + v >= 0 && i + v < row.V ? e[i + v] : 1.0f;
            }
            float x[VEC];
            Row<IO>::unpack(u, x);
            look = false;
#pragma unroll
            for (int v = 0; v < VEC; ++v)
                look |= (__float_as_int(ex[v]) >> 16) + MAGIC_BITS <=
                        __float_as_int(fmaf(-k.wt.below(x[v]), c7, bar));
        }
        if (__any_sync(0xffffffffu, look)) {
            if (look) {
                float x[VEC];
                Row<IO>::unpack(u, x);
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    if (!(x[v] > -INFINITY)) continue;
                    take(best, cand_of(ex2(-k.wt.below(x[v]) * c), ex[v], x[v], i + v));
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) take_across(best, o);
            raise_bar();
        }
        if (!shared_best) {
            // the warps go on from the best of their first groups
            shared_best = true;
            if (k.tid % 32 == 0) k.sh.warp_cand[k.tid / 32] = best;
            __syncthreads();
            const Cand other = k.sh.warp_cand[k.tid % (NT / 32)];
            take(best, other);
#pragma unroll
            for (int o = NT / 64; o > 0; o >>= 1) take_across(best, o);
            raise_bar();
            __syncthreads();                             // (warp_cand is written again later)
        }
        if (g + NT >= row.hi) break;
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
    // 2 log2(e) / t to 2^-46: the quotient's remainder, divided again
    y.c = fminf(2.885390043258667f / t, 2e38f);
    y.c_lo = y.c < 2e38f && t < INFINITY
                 ? (fmaf(-y.c, t, 2.885390043258667f) + 3.851926067000022e-8f) / t : 0.0f;
    if (t == 0.0f) y.c = y.c_lo = 0.0f;
    y.far = y.c > 0.0f ? fminf(CUT / y.c, 3.4028234663852886e38f) : 3.4028234663852886e38f;
    return y;
}

template <int IO, int C>
__global__ void __launch_bounds__(NT, 2)
sample_rows(const __grid_constant__ SampleArgs a) {
    using T = typename io_t<IO>::T;
    constexpr int VEC = Row<IO>::VEC;
    extern __shared__ uint4 slice[];
    __shared__ Shared sh;
    cg::cluster_group cl = cg::this_cluster();
    const int rank = cl.block_rank(), tid = threadIdx.x;
    const int lane = tid % 32, warp = tid / 32;
    const int r = blockIdx.x / C, V = a.V;
    if (tid == 0) sh.my_listed = 0;
    if (tid < 64)
        sh.pow2[tid] = make_uint2(a.pow2[tid] - MAGIC_BITS, __float_as_uint((float)a.pow2[tid]));
    Row<IO> row(static_cast<const T*>(a.logits), r, V);
    const int groups = row.groups(), share = (groups + C - 1) / C;
    row.lo = min(groups, rank * share);
    row.hi = min(groups, row.lo + share);
    row.smem = slice;
    row.resident = a.resident;
    cluster_arrive();
    pdl_wait();
    bool idle = false;                                   // the same for the whole cluster
    if (a.p.last_row) {
        const int last = a.p.last_row[r / a.per];
        idle = last == -1 || r % a.per > max(last, 0);
        if (idle && a.p.idle == SPEC_IDLE_SKIP) {
            cluster_wait();
            return;
        }
    }

    // ---- the row, and its maximum; the last thread, while its loads are under way,
    // makes the request's parameters
    constexpr int U = 4;
    float m = -INFINITY;
    for (int g = row.lo + tid, first = true; first || g < row.hi; g += U * NT, first = false) {
        uint4 u[U];
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (g + j * NT < row.hi) u[j] = row.load(g + j * NT);
        if (first && tid == NT - 1) sh.prm = params_of(a.p, r / a.per);
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int at = g + j * NT - row.lo;
            if (g + j * NT >= row.hi) continue;
            if (at < a.resident) slice[at] = u[j];
            m = max_nan(m, Row<IO>::most(u[j]));
        }
    }
    const float thread_max = m;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        if (o == NT / SOME && lane % o == 0) sh.some[tid / o] = m;
        m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    if (lane == 0) sh.warp_max[warp] = m;
    __syncthreads();
    m = sh.warp_max[lane % (NT / 32)];
#pragma unroll
    for (int o = NT / 64; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    // A lower bound of the k-th largest logit: the k-th of a pool of maxima of threads'
    // shares, of each CTA its largest ones; or, where k is too large for that, the least
    // of what k / C of each CTA's threads reach.
    const int top_k = sh.prm.top_k < V ? sh.prm.top_k : 0;
    constexpr int EACH = POOL / C < SOME ? POOL / C : SOME;
    // (a share is 8 threads' groups; the last CTA's slice may be shorter)
    const int shares = min(EACH, share / (NT / SOME));
    const bool pooled = top_k > 0 && top_k <= shares * C * 3 / 4;
    const bool small_k = pooled || (top_k > 0 && top_k <= min(SMALL_K, C * NT / 2));
    float cut = INFINITY;
    if (small_k && !pooled) {
        sh.pool[tid] = thread_max;
        __syncthreads();
        if (tid < 32) cut = reached(sh.pool, NT, (top_k + C - 1) / C);
        __syncthreads();                                 // (the pool is written again below)
    }
    cluster_wait();                                      // everyone has started
    if (pooled)
        ranked<SOME>(sh.some, [&](int n, float x) {
            if (n < EACH)
#pragma unroll
                for (int c = 0; c < C; ++c) *cl.map_shared_rank(&sh.pool[rank * EACH + n], c) = x;
        });
    if (tid < C) *cl.map_shared_rank(&sh.cta_max[rank], tid) = make_float2(m, cut);
    cluster_sync();
#pragma unroll
    for (int c = 0; c < C; ++c) {
        m = max_nan(m, sh.cta_max[c].x);
        cut = fminf(cut, sh.cta_max[c].y);
    }
    if (pooled && tid < 32) {
        const float x = reached(sh.pool, EACH * C, top_k);
        if (tid == 0) sh.bound = x;
    }

    const Params& prm = sh.prm;
    const bool bad = !(fabsf(m) < INFINITY);
    if (tid == 0) {
        float low = LOWEST;
        if (prm.min_p >= 1.0f) low = m;
        else if (prm.min_p > 0.0f) low = fmaxf(low, __double2float_ru((double)m + prm.min_low));
        sh.prm.low = low;
        const uint32_t bits = prm.bits | (bad ? SPEC_DEV_BADLOGIT : 0u);
        if (bits && rank == 0 && !idle) raise_status(a.ws, bits);
    }
    __syncthreads();
    Ctx<C> k{cl, sh, rank, tid, Weights{m, 0.5f * m, prm.c, prm.c_lo, prm.far, a.lg, sh.pow2}};
    const Weights& wt = k.wt;

    // ---- the border
    const float* e = a.e ? a.e + row.r0 : nullptr;
    float* prob = a.out.prob ? a.out.prob + row.r0 : nullptr;
    T* out = a.out.logits ? static_cast<T*>(a.out.logits) + row.r0 : nullptr;
    Kept kept{prm.low, (int)IDX_MAX};
    u64 sum = 0;
    bool summed = false, drawn = false;
    Cand best{-1.0f, 1.0f, 0.0f, NO_TOK};
    if (bad) {
        kept.v = __int_as_float(0x7fffffff);             // NaN: nothing
    } else {
        if (small_k) {
            const float from = fmaxf(pooled ? sh.bound : cut, kept.v);
            if (gather<IO>(k, row, thread_max >= from, from,
                           [&](float x, int) { return x >= from; })) {
                // without more to write the first CTA ends it alone (all waiting, 256 rows' 10 to
                // 200 best 70 us instead of 62)
                const bool alone = !prob && !out;
                if (alone && rank != 0) return;
                if (rank == 0)
                    solve_list<IO>(k, row, top_k, prm.top_p, 0, 0, !alone, e, best);
                if (alone) __syncthreads();
                else cluster_sync();
                const Border b = sh.border;
                sum = b.sum;
                kept = Kept{value_of(b.from), index_of(b.from)};
                summed = drawn = true;
            }
        }
        if (!drawn) {
            if (top_k > 0) select<false, IO>(k, row, kept, top_k, sum);
            if (prm.top_p != 0) {
                select<true, IO>(k, row, kept, prm.top_p, sum);
                summed = true;
            }
        }
    }

    // ---- what stays: the draw and the outputs (other CTAs' memory is written up to the
    // next barrier, where there is one, and not read)
    const Filter<IO> filter(kept);
    // probabilities are w / z.  Where a border was found by mass, z is its sum; else it
    // only scales, and is summed up in fp32.
    float z = __ull2float_rn(sum) * (1.0f / (float)(1ull << (62 - a.lg)));
    if (!summed && !bad && (prob || a.out.tok_prob)) {
        z = 0.0f;
        for (int g = row.lo + tid; g < row.hi; g += NT) {
            float x[VEC];
            Row<IO>::unpack(filter(row.get(g), row.index(g)), x);
#pragma unroll
            for (int v = 0; v < VEC; ++v)
                z += x[v] > -INFINITY ? ex2(-wt.below(x[v]) * wt.c) : 0.0f;
        }
        z = warp_sum(z);
        __syncthreads();
        if (lane == 0) sh.warp_max[warp] = z;
        __syncthreads();
        z = 0.0f;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) z += sh.warp_max[w];
        if (tid < C) *cl.map_shared_rank(&sh.cta_z[rank], tid) = z;
        cluster_sync();
        z = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) z += sh.cta_z[c];
    }
    const float inv = z > 0.0f ? 1.0f / z : 0.0f;
    const bool race = e && !drawn && !bad;
    if (race) draw(k, row, kept, e, best);
    if (prob || out)
        for (int g = row.lo + tid; g < row.hi; g += NT) {
            const int i = row.index(g);
            const bool whole = row.whole(g);
            uint4 u = row.get(g);
            if (!bad) u = filter(u, i);
            if (out) {
                if (whole) {
                    *reinterpret_cast<uint4*>(out + i) = u;
                } else {
                    alignas(16) T y[VEC];
                    *reinterpret_cast<uint4*>(y) = u;
#pragma unroll
                    for (int v = 0; v < VEC; ++v)
                        if (i + v >= 0 && i + v < V) out[i + v] = y[v];
                }
            }
            if (prob) {
                float x[VEC], w[VEC];
                Row<IO>::unpack(u, x);
                const bool any = Row<IO>::most(u) >= kept.v;     // (never in a bad row)
#pragma unroll
                for (int v = 0; v < VEC; ++v) w[v] = 0.0f;
                if (any) {
#pragma unroll
                    for (int v = 0; v < VEC; ++v)
                        w[v] = x[v] > -INFINITY ? wt.value(x[v]) * inv : 0.0f;
                }
                if (whole) {
#pragma unroll
                    for (int v = 0; v < VEC; v += 4)
                        *reinterpret_cast<float4*>(prob + i + v) =
                            make_float4(w[v], w[v + 1], w[v + 2], w[v + 3]);
                } else {
#pragma unroll
                    for (int v = 0; v < VEC; ++v)
                        if (i + v >= 0 && i + v < V) prob[i + v] = w[v];
                }
            }
        }
    if (!e || (drawn && rank != 0)) return;
    block_best(best, sh);
    if (!drawn) {
        if (tid == 0) *cl.map_shared_rank(&sh.cand[rank], 0) = best;
        cluster_sync();
    }
    if (rank == 0 && tid == 0) {
        if (!drawn)
            for (int c = 0; c < C; ++c) take(best, sh.cand[c]);
        const bool none = best.i == NO_TOK;
        a.out.tok[r] = none ? 0 : best.i;
        if (a.out.tok_prob) a.out.tok_prob[r] = none ? 0.0f : wt.value(best.x) * inv;
    }
}

template <int IO, int C>
cudaError_t launch_c(const spec_sample_cfg& c, SampleArgs& a, int64_t groups, cudaStream_t st) {
    const int most = 180 * 1024;                         // a slice, with one CTA to an SM
    const int64_t share = (groups + C - 1) / C;
    a.resident = (int)(share * 16 > most ? most / 16 : share);
    // once per device and kernel
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(sample_rows<IO, C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 most);
        if (e == cudaSuccess && C > 8)
            e = cudaFuncSetAttribute(sample_rows<IO, C>,
                                     cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(c.R * C));
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = (size_t)a.resident * 16;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, sample_rows<IO, C>, a);
}

// CTAs per row: as many as it takes for two CTAs' slices to share an SM, and more
// while the rows leave SMs idle and a thread has a group (smaller slices give the
// bounds for top_k too few maxima: one row of 5000 tokens 18.6 us instead of 10.5).
//   Idle: with twice as many there were not more than 8/5 of the SMs' number, for
// clusters of 16 not more than that, since a GPC holds one of those at a CTA an SM.
// (Nucleus of 16 / 24 / 38 rows of 151936, up to twice the number: 37.3, 29.0, 42.1 us;
// up to once: 26.3, 29.6, 40.8; like this 26.3, 29.0, 40.8.)
template <int IO>
cudaError_t sample_t(const spec_sample_cfg& c, SampleArgs& a, cudaStream_t st) {
    constexpr int VEC = Row<IO>::VEC;
    const int two = 78 * 1024;                           // a slice, with two CTAs to an SM
    const int64_t groups = ((int64_t)c.V + VEC - 1) / VEC + 1;
    int sms = device_sm_count();
    if (sms < 1) sms = 1;
    int C = 1;
    while (C < MAX_CLUSTER && groups / C >= 2 * NT &&
           ((int64_t)c.R * 2 * C * 5 <= (2 * C == MAX_CLUSTER ? 5 : 8) * (int64_t)sms ||
            (groups + C - 1) / C * 16 > two))
        C *= 2;
    switch (C) {
        case 1: return launch_c<IO, 1>(c, a, groups, st);
        case 2: return launch_c<IO, 2>(c, a, groups, st);
        case 4: return launch_c<IO, 4>(c, a, groups, st);
        case 8: return launch_c<IO, 8>(c, a, groups, st);
        default: return launch_c<IO, 16>(c, a, groups, st);
    }
}

}  // namespace

cudaError_t launch_token_sample(const spec_sample_cfg& c, const void* logits,
                                const spec_sample_params& p, const float* e,
                                const spec_sample_out& out, void* ws, cudaStream_t st) {
    static const struct Pow2 {
        uint32_t t[64];
        Pow2() {
            for (int j = 0; j < 64; ++j) t[j] = (uint32_t)(exp2(29 - j / 64.0) + 0.5);
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
    while ((1 << a.lg) < 2 * c.V) ++a.lg;
    for (int j = 0; j < 64; ++j) a.pow2[j] = pow2.t[j];
    return c.io_dtype == SPEC_IO_BF16 ? sample_t<SPEC_IO_BF16>(c, a, st)
                                      : sample_t<SPEC_IO_F32>(c, a, st);
}

}  // namespace spec
