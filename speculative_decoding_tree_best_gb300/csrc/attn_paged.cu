// attn_paged.cu -- attention of a step's new tokens over the paged cache.
//
// Mathematics.  Row r = (new token i, q-head h of the kv-head's group) of a
// request sees keys [0, kv_len + i]:  o = sum_k w_k v_k / sum_k w_k with
// w_k = 2^(x_k - m), x_k = q.k log2(e) / sqrt(D), m the running maximum: one
// pass, kept per warp and joined at the end (the maxima, sums and outputs of
// two parts a, b join as m = max(m_a, m_b), o = o_a 2^(m_a - m) + o_b 2^(m_b - m)).
// In an 8-bit cache a value is code * scale per row: the key's scale multiplies
// the score, the value's the weight, w'_k = 2^(x_k - m) scale_k with m the maximum
// over x_k + log2 scale_k, scales below 2^LOW counting as that there (up to a factor of 2^SLACK, below), so that the weights that meet the codes are
// at most 2^(SLACK + LIFT) whatever the scales.
//
// What bounds it: reading the cache, 2 D values a key and kv-head against
// 4 D G T flops (G = Hq / Hkv), 2 G T flops a byte in bf16: far below the
// tensor cores' rate up to G T of about 100.  So the products run on
// mma.sync with the KEYS as the 16-row operand and the rows as its 8 columns
// (S^T = K Q^T, O^T = V^T W^T): a decode step's few rows then fill the
// instruction (4 rows of 8 at G = 4; tcgen05's smallest tile would hold 64 or
// 128 rows), the softmax's statistics stay with the thread that holds the
// column in both products, and W^T gets from the first product's layout to
// the second's by movmatrix alone.
//
// Data flow.  The cache is cut into granules of 32 or 64 rows.  The granules of
// all (request, kv-head, row group) segments are dealt out to one CTA per SM by
// their number, so lengths need not match; a segment cut between CTAs leaves
// parts in the workspace, and the CTA whose part is the last one (a ticket per
// segment) joins them, in their order.  In a CTA one warp issues TMA copies (up
// to 64 rows x 128 bytes, 128-byte swizzle) into a ring of granules, and W warps
// take them in turn.  A row's 16-byte chunks go to lanes so that the products
// need no transposition of K, and of V only byte permutes; the row order below
// keeps 128-bit shared loads free of bank conflicts under the swizzle.
//
// Rounding.  Scores, weights, sums and outputs are fp32.  What the tensor cores
// take is exact (cached values; bf16 q) or in parts: weights as two bf16 parts
// (2^-16) over a bf16 cache; over an 8-bit cache in fp16, times 2^LIFT: one part
// with bf16 outputs (2^-11, an eighth of the output's own rounding) unless a tile
// has weights below fp16's normal range (2^-25 of the largest so far), two parts
// there and with fp32 outputs (2^-22), the second REST times as large, so that what
// is left of a weight is at most 2^-48 of the largest; and an fp32 cache, q and
// weights as three bf16 parts each, without the products of parts beyond 2^-24.
// The tensor cores cut a sum off at its last bit, towards 0.  With bf16 outputs
// that is let be (131072 keys in one CTA: 1200 steps a warp, 2^-24 each on average,
// under a twentieth of the output's rounding).  With fp32 outputs each 16 keys' or
// elements' products start at 0 and are added to the rest in fp32: over 8192 keys
// 2.8e-7 of the output is lost instead of 6.9e-6 (all errors 5.2e-7 instead of
// 7.7e-6), for 2 to 3 % of the time, 10 to 17 % with more than eight rows.
//
// Measured (graph replays, bytes of K, V and scales over time): 8 x 131072 keys,
// 8 kv-heads, 8 bits 323-328 us, 6.8 TB/s, the rate of a plain copy; 24 requests of
// 1024-8192 keys bf16 72 us (6.2 TB/s), 8 bits 45 us (5.1 TB/s: two or three
// segments a CTA, whose ends the ring does not hide); one request of 4096 keys
// bf16 9.3 us, of which reading is 2.5: lengths, page ids and copies follow one
// another (3000 cycles), then parts are counted in (2700) and joined (5500).  8
// requests of 4096-8192 keys and 1-8 new tokens, 8 bits: 41 us (2.4 TB/s), by the
// conversions and products, done for each 16 rows; 16, 32, 128 new tokens each, 82,
// 181, 647 us: beyond 48 rows a kv-head the cache is read again for each 48.
#include <cuda.h>
#include <math.h>

#include <atomic>

#include "paged.cuh"
#include "tc_util.cuh"

namespace spec {

namespace {

using tc::mbar_wait;
using tc::smem_u32;

constexpr int SUB = 16;                // keys per product tile: the smallest page
constexpr int MAX_RTC = 3;             // row tiles per CTA, at most (paged_row_tiles)
// log2 of how far a weight may be above that of the maximum: few granules then
// change the maximum (8 instead of 0 gave 8 requests of drafts 40.6 -> 39.6 us)
constexpr float SLACK = 4.0f;
// fp16 weights: 2^LIFT times as large, up to 2^(SLACK + LIFT) = 2^15, so that fewer
// of them fall below fp16's normal range (with 8 and 7, drafts 40.8 us instead of
// 40.7, 8 x 131072 keys 336 instead of 328; without the second part for those that
// do, 39.6 and 327, but long flat tails are lost).  What a weight's fp16 part
// leaves goes times REST, against codes, or into outputs, that are scaled to match
// (exact: codes are multiples of 2^-9).
constexpr float LIFT = 11.0f, LIFT_INV = 0x1p-11f;
constexpr float REST = 0x1p12f;
// log2 of the least scale that the maximum goes by (the least that kv_page_append
// writes): a weight in the softmax's sum is at most 2^(SLACK - LOW), of which 2^23
// are within fp32's range, also where all values so far are zeros by a scale of 0
constexpr float LOW = -100.0f;
constexpr int MAX_SLOTS = 64;          // granules in a CTA's ring, at most

// ---- instruction wrappers -------------------------------------------------------------

__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 8x8 transpose of 16-bit elements across the warp
__device__ __forceinline__ uint32_t movm(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}
// four e4m3 codes as two f16x2 (codes 0, 1 and 2, 3): exact
__device__ __forceinline__ void e4m3x4(uint32_t x, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(x));
}
__device__ __forceinline__ void fence_gpu() { asm volatile("fence.acq_rel.gpu;" ::: "memory"); }
__device__ __forceinline__ void arrive_n(uint64_t* bar, int n) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n)
                 : "memory");
}
__device__ __forceinline__ float log2_scale(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t packh(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// both halves over REST
__device__ __forceinline__ uint32_t scale_f16(uint32_t x) {
    const __half2 f = __floats2half2_rn(1.0f / REST, 1.0f / REST);
    const __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&x), f);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t packb(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float lo_b(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi_b(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
// x = sum of three bf16 parts, by cutting off 8 bits at a time: exact for
// normal numbers; an infinity or NaN stays in the first part.  Parts come as
// fp32 bit patterns whose low half is zero.
__device__ __forceinline__ void split3(float x, uint32_t (&p)[3]) {
    p[0] = __float_as_uint(x) & 0xffff0000u;
    const float h = __uint_as_float(p[0]);
    const float r = h == x ? 0.0f : x - h;
    p[1] = __float_as_uint(r) & 0xffff0000u;
    p[2] = __float_as_uint(r - __uint_as_float(p[1]));     // its low half is never looked at
}
// the same parts of x and y as three bf16 pairs
__device__ __forceinline__ void split3x2(float x, float y, uint32_t& p0, uint32_t& p1,
                                         uint32_t& p2) {
    uint32_t a[3], b[3];
    split3(x, a);
    split3(y, b);
    p0 = __byte_perm(a[0], b[0], 0x7632);
    p1 = __byte_perm(a[1], b[1], 0x7632);
    p2 = __byte_perm(a[2], b[2], 0x7632);
}

// ---- layout of the operands -----------------------------------------------------------

template <int IO, int KV, int D, int NR> struct At {
    static constexpr bool Q8 = KV == SPEC_KV_E4M3;
    static constexpr bool F32 = !Q8 && IO == SPEC_IO_F32;
    static constexpr int EB = Q8 ? 1 : (IO == SPEC_IO_F32 ? 4 : 2);   // bytes of a cached value
    static constexpr int ROWB = D * EB;
    static constexpr int SW = ROWB < 128 ? ROWB : 128;  // bytes of a row in one swizzled block
    static constexpr int NB = ROWB / SW;                // blocks per row
    static constexpr int KCH = ROWB / 64;               // 16-byte chunks of a K row per lane
    static constexpr int EPC = 16 / EB;                 // values per chunk
    static constexpr int VL = ROWB / 8 < 16 ? 1 : ROWB / 128;   // V loads per row and lane
    static constexpr int RL = Q8 ? D / 8 : EPC;         // consecutive values of a lane in a row
    static constexpr int NT = D / 16;                   // 16-value tiles of O^T
    static constexpr int QT = F32 ? 3 : (Q8 && IO == SPEC_IO_F32 ? 2 : 1);  // parts of a Q value
    static constexpr int QR = EPC / 2;                  // Q registers per chunk and part
    static constexpr int PT = F32 ? 3 : (Q8 && IO == SPEC_IO_BF16 ? 1 : 2); // parts of a weight
    // Keys per granule.  With few rows memory is the bound: 64 keys in 8 bits, so
    // that issuing a granule's copies (four of them, see the producer) keeps
    // ahead of it.  With more rows the products are, and 32 keys spread better.
    static constexpr int GK = Q8 && NR == 1 ? 64 : 32;
    static constexpr int NSUB = GK / SUB;
    static constexpr int SLOT_KV = GK * ROWB;           // bytes of K (or V) of a granule
    static constexpr int SLOT = 2 * SLOT_KV;
};

// byte offset of 16-byte chunk c of key row r in a slot's K (or V) region
template <class A> __device__ __forceinline__ uint32_t chunk_off(int r, int c) {
    constexpr int CPB = A::SW / 16;
    const int blk = c / CPB, cc = c % CPB;
    const int x = A::SW == 128 ? (r & 7) : ((r >> 1) & 3);
    return (uint32_t)(blk * A::GK * A::SW + r * A::SW + ((cc ^ x) << 4));
}

struct AttnParams {
    PageMap pm;
    const void* q;
    const float* k_scale;
    const float* v_scale;
    const int32_t* n_new;
    void* o;
    void* ws;
    uint32_t* tickets;
    float4* part_o;
    float4* part_ml;
    int B, T, Hq, G;
    int rtc, rtg;            // row tiles per CTA, row groups per (request, kv-head)
    int slots;
    int gk_sh;               // log2 of a granule's keys
    int box;                 // rows per copy: a granule's, or a page's where that is less
    size_t table_lines, q_lines;   // 128-byte lines of the page table and of Q
    int min_sh;              // aligned: a CTA takes at least 2^min_sh granules
    unsigned long long g_mul;   // ceil(2^32 / G)
    float qk_scale;          // log2(e) / sqrt(D)
    // row / G, exact for the rows there can be (at most 2^16)
    __device__ __forceinline__ int tok(int r) const {
        return (int)(((unsigned long long)r * g_mul) >> 32);
    }
    __device__ __forceinline__ int hk(int seg) const { return rtg == 1 ? seg : seg / rtg; }
    __device__ __forceinline__ int rg(int seg) const { return rtg == 1 ? 0 : seg % rtg; }
    // a segment's row tiles that have rows, with n new tokens; at least one
    template <int NR> __device__ __forceinline__ int live(int n, int seg) const {
        if constexpr (NR == 1) return 1;
        const int rows = n * G - rg(seg) * rtc * 8 * NR;
        return min(max((rows + 8 * NR - 1) / (8 * NR), 1), rtc);
    }
    // what a granule of such a request costs, in granules of one row tile
    template <int NR> __device__ __forceinline__ int weight(int n) const {
        return rtg == 1 ? live<NR>(n, 0) : 1;
    }
};

// One request's lengths.
struct Req {
    int L, n, ng;            // committed rows, new rows, granules
};
__device__ __forceinline__ Req request(const AttnParams& p, int b, uint32_t& bits) {
    Req r;
    r.n = new_rows(p.n_new, b, p.T, bits);
    r.L = p.pm.kv_len[b];
    const int cap = p.pm.cap();
    if (r.L < 0 || r.L > cap - r.n) {
        bits |= SPEC_DEV_OVERFLOW;
        r.L = r.L < 0 ? 0 : min(r.L, cap);
    }
    const int end = r.n > 0 ? min(r.L + r.n, cap) : 0;
    r.ng = max(1, (end + (1 << p.gk_sh) - 1) >> p.gk_sh);
    return r;
}

// What a segment costs a CTA beside its granules (Q, the warps' wait for the last
// one, joining, a part), in units: each segment is dealt out as if it began
// with them.  Up to eight rows, 24 requests, 8-bit cache, 1, 4, 6, 8, 12: 51.7,
// 48.9, 47.3, 47.2, 47.4 us.  More rows, 8 requests of 4096-8192 keys, 8, 16, 20,
// 26, 32: 42.6, 41.4, 41.2, 40.2, 40.5 us; of 256-1024 keys 8, 16, 24: 21.1, 22.9,
// 24.8 us (segments are then cut to fewer CTAs), so that it goes by their length.
template <int NR> __device__ __forceinline__ int overhead(int units, int nseg) {
    return NR == 1 ? 8 : min(24, max(8, (int)((uint32_t)units / (4u * (uint32_t)nseg))));
}

// One pass over the segments of a CTA's share, in order.  A segment is ov units,
// then w for each granule; a granule is the share's that has its first unit.
template <int NR> struct Walk {
    int b, seg;              // request, segment in the request
    int at;                  // place in the segment, of its ov + w rq.ng
    int left;                // of the share
    int ov, w;
    Req rq;
    __device__ __forceinline__ int size() const { return NR == 1 ? ov + rq.ng : ov + w * rq.ng; }
    __device__ __forceinline__ int take() const { return min(size() - at, left); }
    __device__ __forceinline__ int granule(int unit) const {
        const int x = max(0, unit - ov);
        return NR == 1 || w == 1 ? x : (int)((uint32_t)(x + w - 1) / (uint32_t)w);
    }
    // the granules of this portion: [pos, pos + count)
    __device__ __forceinline__ int pos() const { return granule(at); }
    __device__ __forceinline__ int count() const { return granule(at + take()) - pos(); }
    __device__ __forceinline__ void next(const AttnParams& p, int hr) {
        const int c = take();
        left -= c;
        at += c;
        if (at < size() || left <= 0) return;
        at = 0;
        if (++seg == hr) {
            seg = 0;
            ++b;
            uint32_t bits = 0;
            rq = request(p, b, bits);
            w = p.template weight<NR>(rq.n);
        }
    }
};

// `units` (below 2^31) dealt to n CTAs: the first r get q + 1, the others q.
struct Deal {
    int q, r;
    Deal() = default;
    __device__ __forceinline__ Deal(int units, int n)
        : q((int)((uint32_t)units / (uint32_t)n)), r(units - q * n) {}
    __device__ __forceinline__ int start(int c) const { return c * q + min(c, r); }
    __device__ __forceinline__ int owner(int u) const {
        const int big = r * (q + 1);
        return u < big ? (int)((uint32_t)u / (uint32_t)(q + 1))
                       : r + (int)((uint32_t)(u - big) / (uint32_t)q);
    }
};

// CTAs to deal to: as many as there are, but a segment is not cut to less than
// twice its overhead.
__device__ __forceinline__ int cta_count(int units, int ov, int nseg, int most) {
    return min(most, max(nseg, (int)((uint32_t)units / (2u * (uint32_t)ov))));
}

// A segment that this CTA shares with others: what joining its parts needs.
struct Pend {
    int b, seg, n;           // request, segment in it, new rows
    int c0, c1, shift;       // its CTAs; 1: the part of c0 is that CTA's second
    int last;                // this CTA's part was the last one to be written
};

// NR column tiles of 8 rows per warp; W key warps times row tiles; QS: Q in shared
// memory instead of registers; NP producer warps
template <int IO, int KV, int D, int NR, int W, bool QS, int NP>
__global__ void __launch_bounds__(32 * (W + NP), 1)
attn_paged(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
           const __grid_constant__ AttnParams p) {
    using A = At<IO, KV, D, NR>;
    constexpr int NTH = 32 * (W + NP);
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[MAX_SLOTS], empty[MAX_SLOTS];
    __shared__ uint32_t flags[MAX_SLOTS];
    __shared__ int wsum[W + NP];
    __shared__ int first_off, first_b;
    __shared__ Req first_rq;
    __shared__ volatile int abort_flag;
    __shared__ Pend pend[2];

    constexpr int GK = A::GK, NS = 2;    // keys per granule, sub-tiles taken together
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int hr = p.pm.Hkv * p.rtg;
    uint8_t* ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    float* scales = reinterpret_cast<float*>(ring + (size_t)p.slots * A::SLOT);
    float4* buf = reinterpret_cast<float4*>(scales + (A::Q8 ? p.slots * 2 * A::GK : 0));

    // ---- this CTA's share of the granules
    if (tid == 0) {
        abort_flag = 0;
        pend[0].last = pend[1].last = 0;
    }
    if (warp == W && lane < 2) tc::tma_prefetch_desc(lane ? &mv : &mk);
    for (int s = tid; s < p.slots; s += NTH) {
        tc::mbar_init(&full[s], NP);
        tc::mbar_init(&empty[s], p.rtc);
        tc::fence_mbar_init();
    }
    // so far nothing that the launch before may have written (one request of 4096
    // keys 9.8 -> 9.1 us)
    pdl_wait();
    // what comes after the lengths: the page table and Q, on their way to L2
    // while the lengths are read (a line per thread of the grid, no more)
    const size_t line = (size_t)blockIdx.x * NTH + tid;
    if (line < p.table_lines + p.q_lines)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(
            line < p.table_lines
                ? reinterpret_cast<const char*>(p.pm.table) + line * 128
                : static_cast<const char*>(p.q) + (line - p.table_lines) * 128));
    // How the granules are dealt out.  Up to 32 requests every warp reads all
    // lengths, one per lane; beyond, the block does, some per thread.
    //   whole:   short segments (64 keys a warp at most), one to a
    //            CTA, when there are CTAs enough;
    //   aligned: few long segments: each gets CTAs of its own, by its length
    //            (no CTA then works, and joins, in two segments);
    //   else     the row of all segments, overheads included, is cut evenly.
    Walk<NR> wk;
    Deal deal;
    int g0 = 0, n_cta, units;
    int own_c0 = -1, own_c1 = -1;        // aligned: the segment's CTAs
    uint32_t bits = 0;
    const int nseg = p.B * hr, cta = blockIdx.x;
    if (p.B <= 32) {
        Req rq{0, 0, 0};
        if (lane < p.B) rq = request(p, lane, bits);
        const int cost = rq.ng * p.template weight<NR>(rq.n);
        const int granules = __reduce_add_sync(0xffffffffu, cost) * hr;
        const int longest = __reduce_max_sync(0xffffffffu, rq.ng);
        const bool whole = nseg <= (int)gridDim.x && longest <= 64 / GK * (W / p.rtc);
        n_cta = min((int)gridDim.x, (granules + (1 << p.min_sh) - 1) >> p.min_sh);
        const bool aligned = !whole && 4 * nseg <= n_cta && granules < (1 << 22);
        const int ov = overhead<NR>(granules, nseg);
        units = granules + nseg * ov;
        // CTAs per segment of the lane's request, or its segment's units
        int k = whole ? 1 : cost + ov;
        if (aligned)
            k = 1 + (n_cta - nseg) * cost / granules;
        else
            n_cta = whole ? nseg : cta_count(units, ov, nseg, gridDim.x);
        if (lane >= p.B) k = 0;
        int incl = k * hr;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        deal = Deal(units, n_cta);
        g0 = deal.start(cta);
        const int want = whole || aligned ? cta : g0;
        const uint32_t hit = __ballot_sync(0xffffffffu, want < incl);
        if (hit == 0 || cta >= n_cta) return;
        const int b = __ffs(hit) - 1;
        wk.b = b;
        wk.rq.L = __shfl_sync(0xffffffffu, rq.L, b);
        wk.rq.n = __shfl_sync(0xffffffffu, rq.n, b);
        wk.rq.ng = __shfl_sync(0xffffffffu, rq.ng, b);
        k = __shfl_sync(0xffffffffu, k, b);
        const int off = want - (__shfl_sync(0xffffffffu, incl, b) - k * hr);
        wk.seg = (int)((uint32_t)off / (uint32_t)k);
        const int rest = off - wk.seg * k;
        wk.ov = whole || aligned ? 0 : ov;
        wk.w = whole || aligned ? 1 : p.template weight<NR>(wk.rq.n);
        if (whole) {
            wk.at = 0;
            wk.left = wk.rq.ng;
        } else if (aligned) {
            const Deal d(wk.rq.ng, k);
            wk.at = d.start(rest);
            wk.left = d.start(rest + 1) - wk.at;
            own_c0 = cta - rest;
            own_c1 = own_c0 + k - 1;
        } else {
            wk.at = rest;
            wk.left = deal.start(cta + 1) - g0;
        }
        __syncthreads();
    } else {
        const int per = (p.B + NTH - 1) / NTH;
        int mine = 0;
        Req rq0{};
        for (int b = tid * per; b < min(p.B, (tid + 1) * per); ++b) {
            rq0 = request(p, b, bits);
            mine += rq0.ng * p.template weight<NR>(rq0.n) * hr;
        }
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) wsum[warp] = incl;
        __syncthreads();
        int before = 0;
        units = 0;
#pragma unroll
        for (int w = 0; w < W + NP; ++w) {
            const int x = wsum[w];
            if (w < warp) before += x;
            units += x;
        }
        const int ov = overhead<NR>(units, nseg);
        units += nseg * ov;
        n_cta = cta_count(units, ov, nseg, gridDim.x);
        if (cta >= n_cta) return;
        deal = Deal(units, n_cta);
        g0 = deal.start(cta);
        const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
        const int lo = before + incl - mine + b0 * hr * ov;
        mine += (b1 - b0) * hr * ov;
        if (g0 >= lo && g0 < lo + mine) {
            int at = lo;
            for (int b = tid * per;; ++b) {
                uint32_t ignore = 0;
                if (per > 1) rq0 = request(p, b, ignore);
                const int c = (rq0.ng * p.template weight<NR>(rq0.n) + ov) * hr;
                if (g0 < at + c) {
                    first_b = b;
                    first_off = g0 - at;
                    first_rq = rq0;
                    break;
                }
                at += c;
            }
        }
        __syncthreads();
        wk.b = first_b;
        wk.rq = first_rq;
        wk.left = deal.start(cta + 1) - g0;
        wk.ov = ov;
        wk.w = p.template weight<NR>(wk.rq.n);
        wk.seg = (int)((uint32_t)first_off / (uint32_t)wk.size());
        wk.at = first_off - wk.seg * wk.size();
    }
    if (bits && cta == 0) raise_status(p.ws, bits);
    const int rows_tile = 8 * NR;
    const int cap = p.pm.cap();

    if (warp >= W) {
        // ---- producer: one granule per lane, SB lanes at a time; the page ids of 32
        // granules are fetched at once.  Issuing costs this warp some 400 cycles
        // a group and 85 a copy; a large group waits for as many free slots.
        // (2.2 GB of 8-bit cache: 32 keys a granule, groups of 1, 2, 4, 8: 621,
        // 452, 366, 334 us; 64 keys, groups of 1, 2, 4: 391, 329, 342.  bf16, 24
        // requests, groups of 1, 2, 4, 8: 79, 77, 75.8, 78.8 us.)  Of two
        // producers one copies K, the other V.
        constexpr int SB = A::Q8 && A::GK == 64 ? 2 : 4;
        const bool do_k = NP == 1 || warp == W, do_v = NP == 1 || warp == W + 1;
        int slot0 = 0, use0 = 0;         // of the batch's first granule
        bool ok = true;
        uint32_t bad = 0;
        while (wk.left > 0 && ok) {
            const int hk = p.hk(wk.seg), rg = p.rg(wk.seg);
            const int r0 = rg * p.rtc * rows_tile;
            int end = 0;
            if (r0 < wk.rq.n * p.G) {
                const int last = min(r0 + p.rtc * rows_tile, wk.rq.n * p.G) - 1;
                end = min(wk.rq.L + p.tok(last) + 1, cap);
            }
            const int first = wk.pos(), cnt = wk.count();
            for (int base = 0; base < cnt && ok; base += 32) {
                const int gi = base + lane;
                const int key = (first + gi) * GK;
                int page[A::NSUB];
                uint32_t have = 0;           // sub-tiles whose rows are in the pool
#pragma unroll
                for (int h = 0; h < A::NSUB; ++h) {
                    const int at = key + h * SUB;
                    page[h] = -1;
                    // rows that come with an earlier copy of this granule
                    if (h > 0 && (h * SUB) % p.box != 0) {
                        page[h] = page[h - 1];
                    } else if (gi < cnt && at < end) {
                        page[h] = p.pm.table[(size_t)wk.b * p.pm.max_pages + (at >> p.pm.sh)];
                        if ((unsigned)page[h] >= (unsigned)p.pm.n_pages) {
                            bad = SPEC_DEV_BADPAGE;
                            page[h] = -1;
                        }
                    }
                    have |= (page[h] >= 0 ? 1u : 0u) << h;
                }
                int slot = slot0 + lane, use = use0;
                while (slot >= p.slots) {
                    slot -= p.slots;
                    ++use;
                }
                int n = 0;                   // granules of this batch under way
                for (; n < 32 && base + n < cnt; n += SB) {
                    const bool turn = lane / SB == n / SB && gi < cnt;
                    bool got = true;
                    if (turn) got = mbar_wait(&empty[slot], (use & 1) ^ 1, &abort_flag);
                    ok = __all_sync(0xffffffffu, got);
                    if (!ok) break;
                    if (turn) {
                        if (do_k) flags[slot] = have;
                        tc::mbar_arrive_expect_tx(
                            &full[slot],
                            __popc(have) * (A::SLOT / A::NSUB + (A::Q8 ? 8 * SUB : 0)) / NP);
#pragma unroll
                        for (int h = 0; h < A::NSUB; ++h) {
                            if (page[h] < 0 || (h * SUB) % p.box != 0) continue;
                            const int prow =
                                (hk << p.pm.sh) | ((key + h * SUB) & ((1 << p.pm.sh) - 1));
                            uint8_t* kd = ring + (size_t)slot * A::SLOT + h * SUB * A::SW;
#pragma unroll
                            for (int nb = 0; nb < A::NB; ++nb) {
                                if (do_k)
                                    tc::tma_load_3d(kd + nb * GK * A::SW, &mk, &full[slot],
                                                    nb * A::SW, prow, page[h]);
                                if (do_v)
                                    tc::tma_load_3d(kd + A::SLOT_KV + nb * GK * A::SW, &mv,
                                                    &full[slot], nb * A::SW, prow, page[h]);
                            }
                            if constexpr (A::Q8) {
                                const int64_t row =
                                    (((int64_t)page[h] * p.pm.Hkv) << p.pm.sh) + prow;
                                float* sd = scales + slot * 2 * GK + h * SUB;
#pragma unroll
                                for (int v = 0; v < 2; ++v) {
                                    if (!(v ? do_v : do_k)) continue;
                                    asm volatile(
                                        "cp.async.bulk.shared::cluster.global.mbarrier::"
                                        "complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                                            smem_u32(sd + v * GK)),
                                        "l"((v ? p.v_scale : p.k_scale) + row), "r"(4 * p.box),
                                        "r"(smem_u32(&full[slot]))
                                        : "memory");
                                }
                            }
                        }
                    }
                    __syncwarp();
                }
                if (!ok) {
                    // copies in flight land before the CTA's shared memory is
                    // released: each slot's last issued phase
                    if (lane < n) mbar_wait(&full[slot], use & 1, nullptr);
                    for (int k = lane; k < p.slots; k += 32) {
                        int s = slot0 + n + k, v = use0 - 1;   // the slots before them
                        while (s >= p.slots) {
                            s -= p.slots;
                            ++v;
                        }
                        if (v >= 0 && k < p.slots - n) mbar_wait(&full[s], v & 1, nullptr);
                    }
                    break;
                }
                slot0 += min(32, cnt - base);
                while (slot0 >= p.slots) {
                    slot0 -= p.slots;
                    ++use0;
                }
            }
            wk.next(p, hr);
        }
        if (__any_sync(0xffffffffu, bad != 0) && lane == 0) raise_status(p.ws, SPEC_DEV_BADPAGE);
        if (!ok) {
            abort_flag = 1;
            if (lane == 0) raise_status(p.ws, SPEC_DEV_TIMEOUT);
        }
        return;
    }

    // ---- consumers
    // Key warp kw of KW, row tile rt: the segment's `live` tiles with rows share the
    // warps.  Warps beyond KW live only keep the barriers.
    int live = 1, rt = 0, kw = warp, KW = W;
    auto roles = [&](int n, int seg) {
        if constexpr (NR > 1) {
            live = p.template live<NR>(n, seg);
            rt = live == 1 ? 0 : warp % live;
            kw = live == 1 ? warp : warp / live;
            KW = W / live;
        }
    };
    const int g = lane / 4, t = lane % 4;
    const int kr = g ^ ((g & 1) << 2);                       // key row of fragment row g
    const int va = 2 * t, vb = (2 * t + 1) ^ 4;              // of fragment columns 2t, 2t + 1
    int slot0 = 0, use0 = 0;             // of the segment portion's first granule

    float o[NR][A::NT][4];
    float m[NR][2], l[NR][2], rowf[NR][2] = {};  // rowf: not used with QS
    // Q^T, the first product's B operand: in registers, or (QS) in shared memory
    // as [rt][nr][chunk][pair][lane]
    static_assert(!QS || A::QT == 1, "Q in shared memory is in one part");
    uint32_t qf[NR][A::QT][A::KCH][A::QR] = {};  // not used with QS
    uint2* qs = reinterpret_cast<uint2*>(buf + W * NR * (A::NT + 1) * 32);
    float* qsf = reinterpret_cast<float*>(qs + (QS ? p.rtc * NR * A::KCH * (A::QR / 2) * 32 : 0));

    auto clear = [&]() {
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            m[nr][0] = m[nr][1] = -INFINITY;
            l[nr][0] = l[nr][1] = 0.0f;
#pragma unroll
            for (int i = 0; i < A::NT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nr][i][e] = 0.0f;
        }
    };
    auto bar = [&]() { asm volatile("bar.sync 1, %0;" ::"n"(32 * W) : "memory"); };
    constexpr int JW = NR * (A::NT + 1) * 32;            // float4 of a warp
    constexpr int TPR = NR * A::NT / 2;                  // pairs of tiles of a row tile
    constexpr int PO = NR * A::NT * 32, PM = NR * 32;    // float4 of a part's row tile
    // The end of a segment portion (or of the joining of parts): the key warps'
    // results meet in shared memory, (max, max, sum, sum) and the tiles of O^T in
    // register order; the tiles are shared out to the warps by twos, joined over
    // the key warps, and go to the output (whole) or to part `at` of the workspace.
    auto finish = [&](int b, int seg, int n, bool whole, size_t at) {
        bar();                                           // everyone is done with buf
        if (kw < KW) {
            float4* d = buf + warp * JW + lane;
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) {
                d[nr * (A::NT + 1) * 32] = make_float4(m[nr][0], m[nr][1], l[nr][0], l[nr][1]);
#pragma unroll
                for (int i = 0; i < A::NT; ++i)
                    d[(nr * (A::NT + 1) + 1 + i) * 32] =
                        make_float4(o[nr][i][0], o[nr][i][1], o[nr][i][2], o[nr][i][3]);
            }
        }
        bar();
#pragma unroll 1
        for (int task = warp; task < live * TPR; task += W) {
            const int rt2 = task / TPR, nr = task % TPR / (A::NT / 2);
            const int i = task % (A::NT / 2) * 2;
            const float4* s = buf + rt2 * JW + nr * (A::NT + 1) * 32 + lane;
            const int step = live * JW;
            float4 x[W];
            float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
#pragma unroll
            for (int k = 0; k < W; ++k) x[k] = s[min(k, KW - 1) * step];
#pragma unroll
            for (int k = 0; k < W; ++k) {
                m0 = fmaxf(m0, x[k].x);
                m1 = fmaxf(m1, x[k].y);
            }
            const float b0 = m0 == -INFINITY ? 0.0f : m0, b1 = m1 == -INFINITY ? 0.0f : m1;
            float4 y[2];
            y[0] = y[1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < W; ++k) {
                const float f0 = ex2(x[k].x - b0), f1 = ex2(x[k].y - b1);
                const float4 z0 = s[min(k, KW - 1) * step + (1 + i) * 32];
                const float4 z1 = s[min(k, KW - 1) * step + (2 + i) * 32];
                if (k >= KW) continue;
                l0 += x[k].z * f0;
                l1 += x[k].w * f1;
                y[0].x += z0.x * f0;
                y[0].y += z0.y * f1;
                y[0].z += z0.z * f0;
                y[0].w += z0.w * f1;
                y[1].x += z1.x * f0;
                y[1].y += z1.y * f1;
                y[1].z += z1.z * f0;
                y[1].w += z1.w * f1;
            }
            const int r0 = ((p.rg(seg) * p.rtc + rt2) * NR + nr) * 8 + 2 * t;
            if (!whole) {
                // lanes whose rows the step does not have write nothing
                if (r0 >= n * p.G) continue;
                const size_t pt = at * p.rtc + rt2;
                __stcg(p.part_o + pt * PO + (nr * A::NT + i) * 32 + lane, y[0]);
                __stcg(p.part_o + pt * PO + (nr * A::NT + i + 1) * 32 + lane, y[1]);
                if (i == 0)
                    __stcg(p.part_ml + pt * PM + nr * 32 + lane, make_float4(m0, m1, l0, l1));
                continue;
            }
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
                l0 += __shfl_xor_sync(0xffffffffu, l0, d);
                l1 += __shfl_xor_sync(0xffffffffu, l1, d);
            }
            using T = typename io_t<IO>::T;
            const int hk = p.hk(seg);
            bool bad = false;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int tok = p.tok(r0 + e);
                if (tok >= p.T) continue;
                const float sum = e ? l1 : l0;
                const bool real = tok < n && sum != 0.0f;
                const float inv = real ? (A::Q8 ? LIFT_INV : 1.0f) / sum : 0.0f;
                T* dst = static_cast<T*>(p.o) +
                         (((size_t)b * p.T + tok) * p.Hq + hk * p.G + r0 + e - tok * p.G) * D;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int d0 = ((i + k) / (A::RL / 2) * 8 + g) * A::RL +
                                   2 * ((i + k) % (A::RL / 2));
                    const float u = real ? (e ? y[k].y : y[k].x) * inv : 0.0f;
                    const float v = real ? (e ? y[k].w : y[k].z) * inv : 0.0f;
                    // from MOST on the output's type has no finite number
                    constexpr float MOST = IO == SPEC_IO_F32 ? INFINITY : 0x1.ffp127f;
                    bad |= !(fabsf(u) < MOST && fabsf(v) < MOST);
                    if constexpr (IO == SPEC_IO_F32)
                        *reinterpret_cast<float2*>(dst + d0) = make_float2(u, v);
                    else
                        *reinterpret_cast<uint32_t*>(dst + d0) = packb(u, v);
                }
            }
            if (bad) raise_status(p.ws, SPEC_DEV_RANGE);
        }
        if (NR > 1 && whole && live < p.rtc) {           // tiles without rows: zeros
            constexpr int CH = D * (IO == SPEC_IO_F32 ? 4 : 2) / 16;
            const int r0 = (p.rg(seg) * p.rtc + live) * rows_tile;
            for (int x = tid; x < (p.rtc - live) * rows_tile * CH; x += 32 * W) {
                const int r = r0 + x / CH, tok = p.tok(r);
                if (tok >= p.T) break;
                reinterpret_cast<uint4*>(p.o)[(((size_t)b * p.T + tok) * p.Hq + p.hk(seg) * p.G +
                                               r - tok * p.G) * CH + x % CH] =
                    make_uint4(0, 0, 0, 0);
            }
        }
    };

    // Keys that rows 2t, 2t + 1 of column tile nr see: [0, limit); rows that are
    // not the step's: all, and what comes of them is dropped.
    auto limit = [&](int nr, int e) {
        const int i = p.tok((p.rg(wk.seg) * p.rtc + rt) * rows_tile + nr * 8 + 2 * t + e);
        return i < wk.rq.n ? min(wk.rq.L + i + 1, cap) : 0x7fffffff;
    };
    auto row_factor = [&](int nr, int e) {
        if constexpr (QS)
            return qsf[(rt * NR + nr) * 8 + 2 * t + e];
        else
            return rowf[nr][e];
    };

    // NS sub-tiles of a granule, from its h0-th on: keys [kb + 16 h0, ..) in ring
    // slot `slot`; have: a bit per sub-tile that is in the pool
    auto products = [&](int kb, int h0, int slot, uint32_t have, int lim_min, int lim_max) {
        const uint32_t part = (have >> h0) & ((1u << NS) - 1u);
        if (part == 0 || kb + h0 * SUB >= lim_max) return;
        const uint32_t ks = smem_u32(ring + (size_t)slot * A::SLOT);
        const uint32_t vs = ks + A::SLOT_KV;
        float x[NR][NS][4];
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int h = 0; h < NS; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[nr][h][e] = 0.0f;
        // consecutive products go to different accumulators: the halves in turn
        auto q_of = [&](int nr, int q, int j, int i) {
            if constexpr (QS)
                return qs[(((rt * NR + nr) * A::KCH + j) * (A::QR / 2) + i) * 32 + lane];
            else
                return make_uint2(qf[nr][q][j][2 * i], qf[nr][q][j][2 * i + 1]);
        };
#pragma unroll
        for (int j = 0; j < A::KCH; ++j) {
            uint32_t w0[NS][4], w1[NS][4];
#pragma unroll
            for (int h = 0; h < NS; ++h) {
                const uint4 k0 = lds128(ks + chunk_off<A>((h0 + h) * SUB + kr, t + 4 * j));
                const uint4 k1 = lds128(ks + chunk_off<A>((h0 + h) * SUB + kr + 8, t + 4 * j));
                w0[h][0] = k0.x, w0[h][1] = k0.y, w0[h][2] = k0.z, w0[h][3] = k0.w;
                w1[h][0] = k1.x, w1[h][1] = k1.y, w1[h][2] = k1.z, w1[h][3] = k1.w;
            }
            if constexpr (A::Q8) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t a[NS][4];
#pragma unroll
                    for (int h = 0; h < NS; ++h) {
                        e4m3x4(w0[h][i], a[h][0], a[h][2]);
                        e4m3x4(w1[h][i], a[h][1], a[h][3]);
                    }
                    if constexpr (A::QT == 1) {
#pragma unroll
                        for (int nr = 0; nr < NR; ++nr) {
                            const uint2 b = q_of(nr, 0, j, i);
#pragma unroll
                            for (int h = 0; h < NS; ++h) mma_f16_16816(x[nr][h], a[h], b.x, b.y);
                        }
                    } else {
#pragma unroll
                        for (int h = 0; h < NS; ++h)
#pragma unroll
                            for (int nr = 0; nr < NR; ++nr) {
                                float y[4] = {};
#pragma unroll
                                for (int q = A::QT - 1; q >= 0; --q) {
                                    const uint2 b = q_of(nr, q, j, i);
                                    mma_f16_16816(y, a[h], b.x, b.y);
                                }
#pragma unroll
                                for (int e = 0; e < 4; ++e) x[nr][h][e] += y[e];
                            }
                    }
                }
            } else if constexpr (A::F32) {
#pragma unroll
                for (int h = 0; h < NS; ++h) {
                    uint32_t a[3][4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t* w = k % 2 ? w1[h] : w0[h];
                        split3x2(__uint_as_float(w[k / 2 * 2]), __uint_as_float(w[k / 2 * 2 + 1]),
                                 a[0][k], a[1][k], a[2][k]);
                    }
                    float y[NR][4] = {};
#pragma unroll
                    for (int q = 2; q >= 0; --q)              // parts i + q <= 2: 2^-24 is left
#pragma unroll
                        for (int i = 2 - q; i >= 0; --i)
#pragma unroll
                            for (int nr = 0; nr < NR; ++nr) {
                                const uint2 b = q_of(nr, q, j, 0);
                                mma_bf16_16816(y[nr], a[i], b.x, b.y);
                            }
#pragma unroll
                    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[nr][h][e] += y[nr][e];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int nr = 0; nr < NR; ++nr) {
                        const uint2 b = q_of(nr, 0, j, i);
#pragma unroll
                        for (int h = 0; h < NS; ++h) {
                            const uint32_t a[4] = {w0[h][2 * i], w1[h][2 * i], w0[h][2 * i + 1],
                                                   w1[h][2 * i + 1]};
                            mma_bf16_16816(x[nr][h], a, b.x, b.y);
                        }
                    }
            }
        }
        // scores in log2 units, -inf where the row does not see the key
        const bool masked = kb + (h0 + NS) * SUB > lim_min || part != (1u << NS) - 1u;
        float sv[NS][2];                                 // the values' scales
#pragma unroll
        for (int h = 0; h < NS; ++h) {
            float kf[2] = {1.0f, 1.0f};
            if constexpr (A::Q8) {
                const float* sc = scales + slot * 2 * GK + (h0 + h) * SUB + kr;
                kf[0] = sc[0];
                kf[1] = sc[8];
                sv[h][0] = sc[GK];
                sv[h][1] = sc[GK + 8];
            }
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[nr][h][e] *= A::Q8 ? row_factor(nr, e & 1) * kf[e >> 1] : p.qk_scale;
        }
        if (masked) {
#pragma unroll
            for (int h = 0; h < NS; ++h)
#pragma unroll
                for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (kb + (h0 + h) * SUB + kr + 8 * (e >> 1) >= limit(nr, e & 1) ||
                            !((have >> (h0 + h)) & 1u))
                            x[nr][h][e] = -INFINITY;
        }
        // The running maximum of what the V weights go by (fmaxf passes over a NaN).
        // It is brought up to date when a lane is above it by more than SLACK: the
        // weights are then at most 2^(SLACK + LIFT), which fp16 holds, and most granules do
        // without the shuffles.
        bool grow = false;
        float nm[NR][2], lv[NS][2];
        if constexpr (A::Q8) {
#pragma unroll
            for (int h = 0; h < NS; ++h)
#pragma unroll
                for (int k = 0; k < 2; ++k) lv[h][k] = fmaxf(log2_scale(sv[h][k]), LOW);
        }
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float y = -INFINITY;
#pragma unroll
                for (int h = 0; h < NS; ++h) {
                    if constexpr (A::Q8)
                        y = fmaxf(y, fmaxf(x[nr][h][e] + lv[h][0], x[nr][h][2 + e] + lv[h][1]));
                    else
                        y = fmaxf(y, fmaxf(x[nr][h][e], x[nr][h][2 + e]));
                }
                nm[nr][e] = fmaxf(m[nr][e], y);
                grow |= nm[nr][e] > m[nr][e] + SLACK;
            }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1)
                        nm[nr][e] = fmaxf(nm[nr][e], __shfl_xor_sync(0xffffffffu, nm[nr][e], d));
                    const float f = ex2(m[nr][e] - (nm[nr][e] == -INFINITY ? 0.0f : nm[nr][e]));
                    m[nr][e] = nm[nr][e];
                    l[nr][e] *= f;
#pragma unroll
                    for (int i = 0; i < A::NT; ++i) {
                        o[nr][i][e] *= f;
                        o[nr][i][2 + e] *= f;
                    }
                }
            }
        }
        // the weights, in place of the scores, and their sum
        uint32_t least = 0xffffffffu;                    // the least weight's bits
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            const float b0 = m[nr][0] == -INFINITY ? 0.0f : m[nr][0] - (A::Q8 ? LIFT : 0.0f);
            const float b1 = m[nr][1] == -INFINITY ? 0.0f : m[nr][1] - (A::Q8 ? LIFT : 0.0f);
#pragma unroll
            for (int h = 0; h < NS; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float d = x[nr][h][e] - ((e & 1) ? b1 : b0);
                    const float pl = ex2(d);
                    l[nr][e & 1] = A::Q8 ? fmaf(pl, LIFT_INV, l[nr][e & 1]) : l[nr][e & 1] + pl;
                    // the scale of a key that is not seen may be anything
                    if (A::Q8 && masked && x[nr][h][e] == -INFINITY)
                        x[nr][h][e] = 0.0f;
                    else
                        x[nr][h][e] = A::Q8 ? pl * sv[h][e >> 1] : pl;
                    least = min(least, __float_as_uint(x[nr][h][e]));
                }
        }
        // One fp16 part is not enough for weights below its normal range, 2^-14:
        // there may be more of them than the few large ones outweigh.
        bool rest = false;
        if constexpr (A::Q8 && A::PT == 1) {
            if (masked) {                                // but for the zeros
                least = 0xffffffffu;
#pragma unroll
                for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                    for (int h = 0; h < NS; ++h)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            least = min(least, __float_as_uint(x[nr][h][e]) - 1u);
            }
            rest = __any_sync(0xffffffffu, least < 0x38800000u - 1u);
        }
        // Keys that no row sees must not reach O (their weights are 0, but
        // 0 x inf is not): their V counts as zeros.  Of the keys that some rows
        // see and some do not, a value that is not finite must not reach the
        // latter: then the rows of each limit are taken by themselves.
        bool slow = false;
        if (masked && lim_min < lim_max) {
            bool bad = false;
#pragma unroll 1
            for (int c = lane; c < NS * SUB * (A::ROWB / 16); c += 32) {
                const int r = h0 * SUB + c % (NS * SUB);
                if (kb + r < lim_min || kb + r >= lim_max || !((have >> (r / SUB)) & 1u)) continue;
                const uint4 v = lds128(vs + chunk_off<A>(r, c / (NS * SUB)));
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (A::F32) {
                        bad |= (w[i] & 0x7f800000u) == 0x7f800000u;
                    } else if constexpr (A::Q8) {
#pragma unroll
                        for (int y = 0; y < 4; ++y) bad |= ((w[i] >> (8 * y)) & 0x7fu) == 0x7fu;
                    } else {
                        bad |= (w[i] & 0x7f80u) == 0x7f80u || (w[i] & 0x7f800000u) == 0x7f800000u;
                    }
                }
            }
            slow = __any_sync(0xffffffffu, bad);
        }
        int cut = slow ? lim_min : lim_max;
        bool again = false;                              // with what the first part left
#pragma unroll 1
        for (;;) {
            // volatile: in local memory, not in registers that the usual way needs
            volatile float keep[NR][A::NT][4];
            if (slow) {
#pragma unroll
                for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                    for (int i = 0; i < A::NT; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) keep[nr][i][e] = o[nr][i][e];
            }
#pragma unroll
            for (int h = 0; h < NS; ++h) {
                // the half's weights as the second product's B operand, in parts
                uint32_t wb[NR][A::PT][2];
#pragma unroll
                for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float u = x[nr][h][2 * k], v = x[nr][h][2 * k + 1];
                        if constexpr (A::F32) {
                            uint32_t c[3];
                            split3x2(u, v, c[0], c[1], c[2]);
#pragma unroll
                            for (int q = 0; q < 3; ++q) wb[nr][q][k] = movm(c[q]);
                        } else if constexpr (A::Q8) {
                            const uint32_t c = packh(u, v);
                            wb[nr][0][k] = movm(c);
                            if constexpr (A::PT == 2) {
                                const float2 b =
                                    __half22float2(*reinterpret_cast<const __half2*>(&c));
                                wb[nr][A::PT - 1][k] = movm(packh((u - b.x) * REST, (v - b.y) * REST));
                            }
                        } else {
                            const uint32_t c = packb(u, v);
                            wb[nr][0][k] = movm(c);
                            wb[nr][A::PT - 1][k] = movm(packb(u - lo_b(c), v - hi_b(c)));
                        }
                    }
                auto mma_o = [&](int nr, int i, const uint32_t (&a)[4], int part) {
                    if constexpr (A::Q8)
                        mma_f16_16816(o[nr][i], a, wb[nr][part][0], wb[nr][part][1]);
                    else
                        mma_bf16_16816(o[nr][i], a, wb[nr][part][0], wb[nr][part][1]);
                };
#pragma unroll
                for (int j = 0; j < A::VL; ++j) {
                    uint32_t v[4][4];
                    const int row[4] = {va, vb, va + 8, vb + 8};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int r = (h0 + h) * SUB + row[k];
                        if constexpr (A::ROWB == 64) {        // 8 bytes per lane and row
                            const uint2 u = lds64(vs + chunk_off<A>(r, g >> 1) + (g & 1) * 8);
                            v[k][0] = u.x;
                            v[k][1] = u.y;
                            v[k][2] = v[k][3] = 0;
                        } else {
                            const uint4 u = lds128(vs + chunk_off<A>(r, g + 8 * j));
                            v[k][0] = u.x;
                            v[k][1] = u.y;
                            v[k][2] = u.z;
                            v[k][3] = u.w;
                        }
                    }
                    if (masked) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (kb + (h0 + h) * SUB + row[k] >= cut || !((have >> (h0 + h)) & 1u))
                                v[k][0] = v[k][1] = v[k][2] = v[k][3] = 0;
                    }
                    // consecutive products go to different tiles
                    if constexpr (A::F32) {
                        uint32_t a[2][3][4];
#pragma unroll
                        for (int r = 0; r < 2; ++r)
#pragma unroll
                            for (int i = 0; i < 4; ++i)       // columns va, vb, then + 8
                                split3x2(__uint_as_float(v[i / 2 * 2][2 * r + i % 2]),
                                         __uint_as_float(v[i / 2 * 2 + 1][2 * r + i % 2]),
                                         a[r][0][i], a[r][1][i], a[r][2][i]);
                        float y[NR][2][4] = {};
#pragma unroll
                        for (int q = 2; q >= 0; --q)
#pragma unroll
                            for (int i = 2 - q; i >= 0; --i)
#pragma unroll
                                for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                                    for (int r = 0; r < 2; ++r)
                                        mma_bf16_16816(y[nr][r], a[r][i], wb[nr][q][0],
                                                       wb[nr][q][1]);
#pragma unroll
                        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                            for (int r = 0; r < 2; ++r)
#pragma unroll
                                for (int e = 0; e < 4; ++e) o[nr][j * 2 + r][e] += y[nr][r][e];
                    } else if constexpr (A::Q8) {
                        constexpr int NW = A::ROWB == 64 ? 2 : 4;
#pragma unroll
                        for (int i = 0; i < NW; ++i) {
                            uint32_t a[2][4];
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const uint32_t sel = y ? 0x7362 : 0x5140;
                                e4m3x4(__byte_perm(v[0][i], v[1][i], sel), a[y][0], a[y][1]);
                                e4m3x4(__byte_perm(v[2][i], v[3][i], sel), a[y][2], a[y][3]);
                            }
                            if constexpr (A::PT == 1) {
#pragma unroll
                                for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                                    for (int y = 0; y < 2; ++y) mma_o(nr, 2 * i + y, a[y], 0);
                            } else {
                                // (the small part last: the codes are scaled in place)
#pragma unroll
                                for (int y = 0; y < 2; ++y) {
                                    float z[NR][4] = {};
#pragma unroll
                                    for (int nr = 0; nr < NR; ++nr)
                                        mma_f16_16816(z[nr], a[y], wb[nr][0][0], wb[nr][0][1]);
#pragma unroll
                                    for (int k = 0; k < 4; ++k) a[y][k] = scale_f16(a[y][k]);
#pragma unroll
                                    for (int nr = 0; nr < NR; ++nr) {
                                        mma_f16_16816(z[nr], a[y], wb[nr][A::PT - 1][0],
                                                      wb[nr][A::PT - 1][1]);
#pragma unroll
                                        for (int e = 0; e < 4; ++e)
                                            o[nr][2 * i + y][e] += z[nr][e];
                                    }
                                }
                            }
                        }
                    } else {
                        uint32_t a[4][4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            a[i][0] = __byte_perm(v[0][i], v[1][i], 0x5410);
                            a[i][1] = __byte_perm(v[0][i], v[1][i], 0x7632);
                            a[i][2] = __byte_perm(v[2][i], v[3][i], 0x5410);
                            a[i][3] = __byte_perm(v[2][i], v[3][i], 0x7632);
                        }
#pragma unroll
                        for (int q = 0; q < A::PT; ++q)
#pragma unroll
                            for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                                for (int i = 0; i < 4; ++i) mma_o(nr, 4 * j + i, a[i], q);
                    }
                }
            }
            if (slow) {
#pragma unroll
                for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                    for (int i = 0; i < A::NT; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (limit(nr, e & 1) != cut) o[nr][i][e] = keep[nr][i][e];
                if (++cut <= lim_max) continue;
            }
            if (!rest) break;
            // once more with what the weights' fp16 part left, REST times as large,
            // into outputs as many times as large
            const float f = again ? 1.0f / REST : REST;
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                for (int i = 0; i < A::NT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[nr][i][e] *= f;
            if (again) break;
            again = true;
            cut = slow ? lim_min : lim_max;
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                for (int h = 0; h < NS; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float u = x[nr][h][e];
                        x[nr][h][e] = (u - __half2float(__float2half_rn(u))) * REST;
                    }
        }
    };

    // A column tile's Q rows (tile: in the CTA's row group) as they are in memory,
    // 16 bytes at a time (rows the step does not have: zeros)
    constexpr int QB = IO == SPEC_IO_F32 ? 4 : 2;
    constexpr int RAW = D * QB / 64;                     // 16-byte pieces of a row per lane
    auto load_q = [&](const Walk<NR>& w, int tile, uint4 (&raw)[RAW]) {
        const int r = (p.rg(w.seg) * p.rtc * NR + tile) * 8 + g, i = p.tok(r);
        const bool real = i < p.T;
        const uint4* qp = reinterpret_cast<const uint4*>(
            static_cast<const uint8_t*>(p.q) +
            (real ? (((size_t)w.b * p.T + i) * p.Hq + p.hk(w.seg) * p.G + r - i * p.G) * D * QB
                  : 0));
        constexpr int PC = RAW / A::KCH;                 // pieces per cache chunk
#pragma unroll
        for (int k = 0; k < RAW; ++k)
            raw[k] = real ? __ldg(qp + (t + 4 * (k / PC)) * PC + k % PC) : make_uint4(0, 0, 0, 0);
    };
    // and as the first product's operand
    auto make_q = [&](const uint4 (&raw)[RAW], uint32_t (&qr)[A::QT][A::KCH][A::QR], float& row) {
        row = p.qk_scale;
        if constexpr (!A::Q8 && !A::F32) {
#pragma unroll
            for (int j = 0; j < A::KCH; ++j) {
                qr[0][j][0] = raw[j].x;
                qr[0][j][1] = raw[j].y;
                qr[0][j][2] = raw[j].z;
                qr[0][j][3] = raw[j].w;
            }
        } else if constexpr (A::F32) {
#pragma unroll
            for (int j = 0; j < A::KCH; ++j) {
                const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    split3x2(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]), qr[0][j][k],
                             qr[1][j][k], qr[2][j][k]);
            }
        } else {
            // fp16 with the row scaled by a power of two so that its largest
            // value is in [2^14, 2^15): bf16 values down to 2^-28 of it keep
            // every bit, fp32 ones go in two parts
            float y[A::KCH][16], amax = 0.0f;
#pragma unroll
            for (int j = 0; j < A::KCH; ++j) {
                constexpr int PC = RAW / A::KCH;
#pragma unroll
                for (int c = 0; c < PC; ++c) {
                    const uint4 u = raw[j * PC + c];
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if constexpr (IO == SPEC_IO_BF16) {
                            y[j][8 * c + 2 * k] = lo_b(w[k]);
                            y[j][8 * c + 2 * k + 1] = hi_b(w[k]);
                        } else {
                            y[j][4 * c + k] = __uint_as_float(w[k]);
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < 16; ++k) amax = fmaxf(amax, fabsf(y[j][k]));
            }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // 2^(14 - exponent), within what fp32 holds (0 and inf: 1)
            int ex = (int)(__float_as_uint(amax) >> 23) - 127;
            if (!(amax > 0.0f) || ex == 128) ex = 14;
            ex = max(ex, -100);
            const float f = __uint_as_float((uint32_t)(127 + 14 - ex) << 23);
            row *= __uint_as_float((uint32_t)(127 - 14 + ex) << 23);
#pragma unroll
            for (int j = 0; j < A::KCH; ++j)
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float a = y[j][2 * k] * f, c = y[j][2 * k + 1] * f;
                    const uint32_t h = packh(a, c);
                    qr[0][j][k] = h;
                    if constexpr (A::QT == 2) {
                        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h));
                        qr[A::QT - 1][j][k] = packh(a - b.x, c - b.y);
                    }
                }
        }
    };

    int gpos = g0;                       // where this CTA is among all units
    uint4 raw[RAW];
    // one row tile: the next segment's Q rows are fetched during this one
    constexpr bool AHEAD = NR == 1 && IO == SPEC_IO_BF16;
    if (AHEAD) load_q(wk, rt, raw);
    for (;;) {
        int b, seg, n, c0 = 0, c1 = 0, which = 0;
        bool whole = true;
        size_t at = 0;
        clear();
        if (wk.left > 0) {
            roles(wk.rq.n, wk.seg);
            const int row0 = (p.rg(wk.seg) * p.rtc + rt) * rows_tile;
            const int first = wk.pos(), cnt = wk.count();
            if (cnt == 0) {                      // units that are no granule's first
                gpos += wk.take();
                wk.next(p, hr);
                if (AHEAD && wk.left > 0) load_q(wk, rt, raw);
                continue;
            }
            // ---- limits and Q of this warp's rows
            int lim_min = 0, lim_max = 0;
            if (row0 < wk.rq.n * p.G) {
                const int last = min(row0 + rows_tile, wk.rq.n * p.G) - 1;
                lim_min = min(wk.rq.L + p.tok(row0) + 1, cap);
                lim_max = min(wk.rq.L + p.tok(last) + 1, cap);
            }
            if constexpr (QS) {
                // the warps make a column tile each (they are past the last
                // segment's products: its joining had barriers)
                for (int tile = warp; tile < live * NR; tile += W) {
                    float row;
                    uint32_t qt[A::QT][A::KCH][A::QR];
                    load_q(wk, tile, raw);
                    make_q(raw, qt, row);
#pragma unroll
                    for (int j = 0; j < A::KCH; ++j)
#pragma unroll
                        for (int i = 0; i < A::QR / 2; ++i)
                            qs[((tile * A::KCH + j) * (A::QR / 2) + i) * 32 + lane] =
                                make_uint2(qt[0][j][2 * i], qt[0][j][2 * i + 1]);
                    if (t == 0) qsf[tile * 8 + g] = row;
                }
                bar();
            } else {
#pragma unroll
                for (int nr = 0; nr < NR; ++nr) {
                    float row;
                    if (!AHEAD) load_q(wk, rt * NR + nr, raw);
                    make_q(raw, qf[nr], row);
                    // lane (g, t) made row g; it needs rows 2t and 2t + 1
                    rowf[nr][0] = __shfl_sync(0xffffffffu, row, 8 * t);
                    rowf[nr][1] = __shfl_sync(0xffffffffu, row, 8 * t + 4);
                }
            }
            Walk<NR> nx = wk;
            nx.next(p, hr);
            if (AHEAD && nx.left > 0) load_q(nx, rt, raw);
            // ---- the granules: every KW-th one
            int slot = slot0 + kw, use = use0;
            for (int gi = kw; gi < cnt && kw < KW; gi += KW, slot += KW) {
                while (slot >= p.slots) {
                    slot -= p.slots;
                    ++use;
                }
                // The slot's granule before this one may be another warp's and may
                // land later than this warp's last one: a wait for this use's copy
                // is only good once that use is over, or its parity is the one
                // of two uses ago.
                bool got = use == 0 || mbar_wait(&empty[slot], (use - 1) & 1, &abort_flag);
                got = got && mbar_wait(&full[slot], use & 1, &abort_flag);
                if (!got) {
                    abort_flag = 1;
                    if (lane == 0) raise_status(p.ws, SPEC_DEV_TIMEOUT);
                }
                __syncwarp();
                const int kb = (first + gi) * GK;
                const uint32_t have = flags[slot];
#pragma unroll 1
                for (int h0 = 0; h0 < A::NSUB; h0 += NS)
                    products(kb, h0, slot, have, lim_min, lim_max);
                __syncwarp();
                // a slot is free after rtc arrivals, however many tiles are live
                if (lane == 0) arrive_n(&empty[slot], rt == 0 ? p.rtc - live + 1 : 1);
            }
            slot0 += cnt % p.slots;
            use0 += cnt / p.slots;
            if (slot0 >= p.slots) {
                slot0 -= p.slots;
                ++use0;
            }
            // ---- the segment's end
            b = wk.b;
            seg = wk.seg;
            n = wk.rq.n;
            whole = cnt == wk.rq.ng;
            if (!whole) {
                c0 = own_c0, c1 = own_c1;
                int shift = 0;
                if (c0 < 0) {
                    const int s0 = gpos - wk.at;
                    c0 = deal.owner(s0 + wk.ov);
                    c1 = deal.owner(s0 + wk.ov + (wk.rq.ng - 1) * (NR == 1 ? 1 : wk.w));
                    shift = s0 > deal.start(c0);
                }
                at = 2 * cta + (cta == c0 ? shift : 0);
                which = gpos != g0;
                if (tid == 0) {
                    Pend& pe = pend[which];
                    pe.b = b;
                    pe.seg = seg;
                    pe.n = n;
                    pe.c0 = c0;
                    pe.c1 = c1;
                    pe.shift = shift;
                }
            }
            gpos += wk.take();
            wk = nx;
        } else {
            // ---- out of granules: the segments whose last part was this CTA's
            bar();                                       // pend is there
            const int k = pend[0].last == 1 ? 0 : (pend[1].last == 1 ? 1 : 2);
            if (k == 2) break;
            const Pend pe = pend[k];
            bar();
            if (tid == 0) pend[k].last = 2;
            fence_gpu();
            b = pe.b;
            seg = pe.seg;
            n = pe.n;
            roles(n, seg);
            const int row0 = (p.rg(seg) * p.rtc + rt) * rows_tile;
            constexpr int STEP = NR == 1 ? 3 : 1;        // parts under way at once
#pragma unroll 1
            for (int c = pe.c0 + kw; c <= pe.c1 && kw < KW; c += KW * STEP) {
                float4 x[STEP][NR], z[STEP][NR][A::NT];
#pragma unroll
                for (int j = 0; j < STEP; ++j) {
                    const int cc = c + j * KW;
                    const size_t pt = (size_t)(2 * cc + (cc == pe.c0 ? pe.shift : 0)) * p.rtc + rt;
#pragma unroll
                    for (int nr = 0; nr < NR; ++nr) {
                        // lanes whose rows the step does not have read nothing
                        const bool in = cc <= pe.c1 && row0 + nr * 8 + 2 * t < n * p.G;
                        x[j][nr] = make_float4(-INFINITY, -INFINITY, 0.0f, 0.0f);
                        if (in) x[j][nr] = __ldcg(p.part_ml + pt * PM + nr * 32 + lane);
#pragma unroll
                        for (int i = 0; i < A::NT; ++i) {
                            z[j][nr][i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                            if (in)
                                z[j][nr][i] =
                                    __ldcg(p.part_o + pt * PO + (nr * A::NT + i) * 32 + lane);
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < STEP; ++j)
#pragma unroll
                    for (int nr = 0; nr < NR; ++nr) {
                        float f1[2], f2[2];
                        const float m2[2] = {x[j][nr].x, x[j][nr].y};
                        const float l2[2] = {x[j][nr].z, x[j][nr].w};
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float nm = fmaxf(m[nr][e], m2[e]);
                            const float base = nm == -INFINITY ? 0.0f : nm;
                            f1[e] = ex2(m[nr][e] - base);
                            f2[e] = ex2(m2[e] - base);
                            m[nr][e] = nm;
                            l[nr][e] = l[nr][e] * f1[e] + l2[e] * f2[e];
                        }
#pragma unroll
                        for (int i = 0; i < A::NT; ++i) {
                            const float4 y = z[j][nr][i];
                            o[nr][i][0] = o[nr][i][0] * f1[0] + y.x * f2[0];
                            o[nr][i][1] = o[nr][i][1] * f1[1] + y.y * f2[1];
                            o[nr][i][2] = o[nr][i][2] * f1[0] + y.z * f2[0];
                            o[nr][i][3] = o[nr][i][3] * f1[1] + y.w * f2[1];
                        }
                    }
            }
        }
        finish(b, seg, n, whole, at);
        if (!whole && warp < min(W, live * TPR)) {
            // each warp that wrote of the part counts itself in; the segment is
            // joined, when its CTA has no more granules, by who comes last.  (A
            // CTA's first part is counted in while it works on: the neighbour
            // then joins that segment, and no CTA is left with two.)
            fence_gpu();
            __syncwarp();
            if (lane == 0) {
                uint32_t* tk = p.tickets + c0;
                const uint32_t all = (uint32_t)(c1 - c0 + 1) * min(W, live * TPR);
                if (atomicAdd(tk, 1u) == all - 1) {
                    *tk = 0;                             // for the next call
                    pend[which].last = 1;
                }
            }
        }
    }
}

// ---- host ------------------------------------------------------------------------------

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static const EncodeTiledFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiledFn>(p);
    }();
    return fn;
}

// A pool as bytes [n_pages][Hkv page][row bytes], boxes of a granule's rows.
template <class A> bool pool_map(CUtensorMap* m, const spec_paged_cfg& c, const void* base) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t rows = (cuuint64_t)c.Hkv * c.page;
    const cuuint64_t dims[3] = {(cuuint64_t)A::ROWB, rows, (cuuint64_t)c.n_pages};
    const cuuint64_t str[2] = {(cuuint64_t)A::ROWB, rows * A::ROWB};
    const cuuint32_t box[3] = {(cuuint32_t)A::SW, (cuuint32_t)(c.page < A::GK ? c.page : A::GK), 1};
    const cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, str, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE,
               A::SW == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int SMEM_MAX = 225 * 1024;     // of 227 KB, beside the static variables

template <int IO, int KV, int D, int NR, int W, bool QS, int NP>
cudaError_t attn_launch(const spec_paged_cfg& c, const spec_paged_kv& kv, const void* q,
                        const int32_t* n_new, void* o, void* ws, cudaStream_t st) {
    using A = At<IO, KV, D, NR>;
    const int sms = device_sm_count();
    if (sms < 1) return cudaErrorInvalidDevice;
    const PagedWs w = paged_ws_layout(c, sms);
    CUtensorMap mk, mv;
    if (!pool_map<A>(&mk, c, kv.k_pages) || !pool_map<A>(&mv, c, kv.v_pages))
        return cudaErrorInvalidValue;
    AttnParams p{};
    p.pm = page_map(c, kv);
    p.q = q;
    p.k_scale = kv.k_scale;
    p.v_scale = kv.v_scale;
    p.n_new = n_new;
    p.o = o;
    p.ws = ws;
    p.tickets = ws_ptr<uint32_t>(ws, kTicketOff);
    p.part_o = ws_ptr<float4>(ws, w.part_o_off);
    p.part_ml = ws_ptr<float4>(ws, w.part_ml_off);
    p.B = c.B;
    p.T = c.T;
    p.Hq = c.Hq;
    p.G = c.Hq / c.Hkv;
    p.g_mul = ((1ull << 32) + p.G - 1) / p.G;
    p.rtc = w.rtc;
    p.rtg = w.rtg;
    p.gk_sh = A::GK == 64 ? 6 : 5;
    p.min_sh = 7 - p.gk_sh;              // 128 keys
    p.table_lines = ((size_t)c.B * c.max_pages * 4 + 127) / 128;
    p.q_lines = ((size_t)c.B * c.T * c.Hq * D * (IO == SPEC_IO_F32 ? 4 : 2) + 127) / 128;
    p.box = c.page < A::GK ? c.page : A::GK;
    p.qk_scale = 1.4426950408889634f / sqrtf((float)D);
    constexpr int fixed = 1024 + W * NR * (A::NT + 1) * 32 * 16 +
                          (QS ? MAX_RTC * NR * (A::KCH * A::QR * 128 + 32) : 0);
    constexpr int per_slot = A::SLOT + (A::Q8 ? 2 * A::GK * 4 : 0);
    constexpr int fit = (SMEM_MAX - fixed) / per_slot;
    static_assert(fit >= W && fit >= 4, "the ring's waits need a slot per key warp");
    p.slots = fit < MAX_SLOTS ? fit : MAX_SLOTS;
    const int smem = fixed + p.slots * per_slot;
    auto kern = attn_paged<IO, KV, D, NR, W, QS, NP>;
    // once per device and kernel (the size is a constant of the kernel)
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    // at most every granule of a full table
    const int64_t per_seg = ((int64_t)c.max_pages * c.page + A::GK - 1) / A::GK;
    const int64_t most = (int64_t)c.B * c.Hkv * w.rtg * per_seg;
    const int grid = (int)(most < sms ? most : sms);
    return launch_k(true, kern, dim3(grid), dim3(32 * (W + NP)), smem, st, mk, mv, p);
}

template <int IO, int KV, int D>
cudaError_t attn_t(const spec_paged_cfg& c, const spec_paged_kv& kv, const void* q,
                   const int32_t* n_new, void* o, void* ws, cudaStream_t st) {
    // Up to eight rows: seven key warps and the producer with up to 255 registers
    // each (eight leave 168: 24 requests, 8-bit cache, 48.4 us against 46.4).  More:
    // ten with 168, Q in shared memory (8 requests x 32 rows, 8-bit cache: 49.7
    // us; seven with 255: 59.9), and a second producer, which the warps' number
    // leaves registers for (43.8 -> 42.6 us).  In fp32 a granule at D = 128 is 32
    // KB, and the ring must have a slot per key warp; more than eight rows there take
    // 255 registers and spill 384 bytes (8 requests of 4096-8192 keys, 8 tokens: 315 us
    // over 57 of reading; fp32 over 8 bits spills 276 bytes: 83 us over 15).
    constexpr bool big = At<IO, KV, D, 1>::SLOT > 16384;
    if (paged_row_tiles(c).nr == 1)
        return attn_launch<IO, KV, D, 1, big ? 6 : 7, false, 1>(c, kv, q, n_new, o, ws, st);
    if constexpr (IO == SPEC_IO_BF16 && At<IO, KV, D, 2>::SLOT < 16384)
        return attn_launch<IO, KV, D, 2, 10, true, 2>(c, kv, q, n_new, o, ws, st);
    else
        return attn_launch<IO, KV, D, 2, big ? 5 : 7, IO == SPEC_IO_BF16, 1>(c, kv, q, n_new, o, ws,
                                                                            st);
}

}  // namespace

cudaError_t launch_attn_paged(const spec_paged_cfg& c, const spec_paged_kv& kv, const void* q,
                              const int32_t* n_new, void* o, void* ws, cudaStream_t st) {
    SPEC_PAGED_DISPATCH(attn_t, c, kv, q, n_new, o, ws, st);
}

}  // namespace spec
