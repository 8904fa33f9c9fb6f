// rope.cu -- rotary positions of queries and keys, alone or in one pass with the
// write of a step's new rows into the cache's pages.
//
// Mathematics.  The pair j of a head at position p turns by p f_j.  The angle is
// taken in turns, modulo one, in integers: the table holds f_j / 2 pi in whole units
// of 2^-64 turns, and p times that, modulo 2^64, is the fraction of a turn, at most
// 2^-34 off at the farthest position (half a unit times 2^31).  Its upper 32 bits are
// split into a quarter turn and a rest in [-pi/4, pi/4], whose sine and cosine are
// Taylor sums to x^9 and x^10 (the next terms: 1.8e-9, 1.1e-10).  No position needs
// more than fp32, and none loses accuracy to its size.
//
// Data flow.  A head's row belongs to D / 16 (bf16) or D / 8 (fp32) lanes; a lane
// holds two 16-byte pieces that are each other's partners (elements v and
// v + rot/2, or neighbours), so that a pair never leaves its thread.  A group of
// lanes makes the sines and cosines of its token once and goes over a share of
// the token's heads with them, two heads' loads under way at once.
//
// What bounds it: reading and writing each value once.  Measured (graph replays,
// D = 128, 32 q-heads, 8 kv-heads, bf16): 16383 tokens' q and k 52.3 us, 6.4 TB/s, 0.96
// of a plain copy's rate; 16376 tokens with the cache's rows in bf16 66 us, 6.1 TB/s; 4
// prompts of 4096 tokens into 8 bits 67.5 us, 5.5 TB/s (maxima, quotients and codes
// on top); 25 rows 1.8 us, 24 single tokens 2.5, a launch and two loads.
#include <math.h>

#include "cache_rows.cuh"
#include "serving.cuh"

namespace spec {

namespace {

// (Blocks of 256 threads at the same registers: prompts 54.5, 69.6 and 72.6 us instead
// of 52.3, 66 and 67.5 above, 25 rows 2.1.  One head at once: prompts 60.7, 76; four:
// 56, 73, 25 rows 2.8.  Two pairs by packed multiply-adds: 25 rows 2.0, 8 bits 73.)
constexpr int NT = 128;
constexpr int UNR = 2;

// sine and cosine of `turn` 2^-32 turns, times amp
__device__ __forceinline__ void sincos_turn(uint32_t turn, float amp, float& s, float& c) {
    const uint32_t quarter = (turn + 0x20000000u) >> 30;
    const float x = (float)(int32_t)(turn - (quarter << 30)) * 1.4629180792671596e-9f;  // 2 pi / 2^32
    const float z = x * x;
    float ps = fmaf(z, 1.0f / 362880.0f, -1.0f / 5040.0f);
    ps = fmaf(z, ps, 1.0f / 120.0f);
    ps = fmaf(z, ps, -1.0f / 6.0f);
    ps = fmaf(x * z, ps, x);
    float pc = fmaf(z, -1.0f / 3628800.0f, 1.0f / 40320.0f);
    pc = fmaf(z, pc, -1.0f / 720.0f);
    pc = fmaf(z, pc, 1.0f / 24.0f);
    pc = fmaf(z, pc, -0.5f);
    pc = fmaf(z, pc, 1.0f);
    const bool swap = quarter & 1;
    s = (swap ? pc : ps) * (quarter & 2 ? -amp : amp);
    c = (swap ? ps : pc) * ((quarter + 1) & 2 ? -amp : amp);
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

struct RopeArgs {
    const uint64_t* turns;
    const void *q, *k, *v;
    void *q_out, *k_out;
    int64_t q_stride, k_stride, v_stride;   // in 16-byte pieces
    int64_t groups;                         // rows * share
    int Hq, Hkv, items;                     // items: heads of a token
    int share, per;                         // groups per token, heads per group
    int pairs;                              // lanes of a group that rotate
    float amp;                              // negative sines: see inverse
    int inverse;
    const int32_t* pos;                     // rope_apply
    // rope_page_append
    const int64_t* slots;
    const int32_t* kv_len;
    void *k_pages, *v_pages;
    float *k_scale, *v_scale;
    int64_t n_slots;
    int T, sh;
    void* ws;
};

// A head's row, a lane's two pieces of it: where they are and whose.
struct Item {
    const uint4* src;
    uint4* dst;              // NULL: the cache
    int head, kind;          // kind 0 q, 1 k, 2 v, -1 none
};

template <int IO, int KV, int D, int LAYOUT, bool APPEND>
__global__ void __launch_bounds__(NT, 6)
rope_rows(const __grid_constant__ RopeArgs a) {
    constexpr int VEC = 16 / sizeof(typename io_t<IO>::T);
    constexpr int PPR = D / VEC, LPR = PPR / 2;        // pieces and lanes of a row
    const int64_t group = (int64_t)blockIdx.x * (NT / LPR) + threadIdx.x / LPR;
    const int lane = threadIdx.x % LPR;
    pdl_wait();
    bool live = group < a.groups;
    // (divisions in 32 bits where they do: all but launches of billions of groups)
    const bool small = a.groups >> 32 == 0;
    const int64_t row = !live ? 0 : (small ? (uint32_t)group / (uint32_t)a.share : group / a.share);
    const int first = live ? (int)(group - row * a.share) : 0;
    const bool turn = lane < a.pairs;
    const int v0 = LAYOUT == SPEC_ROPE_HALF && turn ? lane : 2 * lane;
    const int v1 = LAYOUT == SPEC_ROPE_HALF && turn ? lane + a.pairs : 2 * lane + 1;
    int pos = 0;
    int64_t slot = 0;
    if constexpr (APPEND) {
        if (live) {
            slot = a.slots[row];
            const int b = (int)((uint32_t)row / (uint32_t)a.T);       // rows < 2^31
            pos = a.kv_len[b] + (int)(row - (int64_t)b * a.T);
            live = slot >= 0;
            if (slot >= a.n_slots && lane == 0 && first == 0) raise_status(a.ws, SPEC_DEV_BADPAGE);
        }
    } else if (live) {
        pos = a.pos[row];
    }
    if (!__any_sync(0xffffffffu, live)) return;          // padding
    auto item = [&](int at) {
        Item x{nullptr, nullptr, 0, -1};
        if (!live || at >= a.items) return x;
        x.kind = at < a.Hq ? 0 : (at < a.Hq + a.Hkv ? 1 : 2);
        x.head = at - (x.kind > 0 ? a.Hq : 0) - (x.kind > 1 ? a.Hkv : 0);
        const void* base = x.kind == 0 ? a.q : (x.kind == 1 ? a.k : a.v);
        const int64_t stride = x.kind == 0 ? a.q_stride : (x.kind == 1 ? a.k_stride : a.v_stride);
        x.src = static_cast<const uint4*>(base) + row * stride + x.head * PPR;
        if (x.kind == 0)
            x.dst = static_cast<uint4*>(a.q_out) + (row * a.Hq + x.head) * PPR;
        else if (!APPEND)
            x.dst = static_cast<uint4*>(a.k_out) + (row * a.Hkv + x.head) * PPR;
        else if (slot >= a.n_slots)
            x.kind = -1;
        return x;
    };
    float sn[VEC], cs[VEC];
    for (int at = 0; at < a.per; at += UNR) {           // the same for all threads
        Item it[UNR];
        uint4 u[UNR][2];
#pragma unroll
        for (int j = 0; j < UNR; ++j) {
            it[j] = at + j < a.per ? item(first + (at + j) * a.share) : Item{nullptr, nullptr, 0, -1};
            u[j][0] = u[j][1] = make_uint4(0, 0, 0, 0);
            if (it[j].kind >= 0) {
                u[j][0] = it[j].src[v0];
                u[j][1] = it[j].src[v1];
            }
        }
        if (at == 0 && turn) {
            const uint32_t p = pos < 0 ? 0u - (uint32_t)pos : (uint32_t)pos;
            const float flip = (pos < 0) != (a.inverse != 0) ? -1.0f : 1.0f;
#pragma unroll
            for (int i = 0; i < VEC; i += 2) {
                const ulonglong2 t = *reinterpret_cast<const ulonglong2*>(a.turns + lane * VEC + i);
                sincos_turn((uint32_t)((p * t.x) >> 32), a.amp, sn[i], cs[i]);
                sincos_turn((uint32_t)((p * t.y) >> 32), a.amp, sn[i + 1], cs[i + 1]);
                sn[i] *= flip;
                sn[i + 1] *= flip;
            }
        }
#pragma unroll
        for (int j = 0; j < UNR; ++j) {
            float x[2][VEC];
            unpack<IO>(u[j][0], x[0]);
            unpack<IO>(u[j][1], x[1]);
            if (turn && it[j].kind < 2) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    float& p = LAYOUT == SPEC_ROPE_HALF ? x[0][i] : x[2 * i / VEC][2 * i % VEC];
                    float& q = LAYOUT == SPEC_ROPE_HALF ? x[1][i] : x[2 * i / VEC][2 * i % VEC + 1];
                    const float y = fmaf(p, cs[i], -(q * sn[i]));
                    q = fmaf(p, sn[i], q * cs[i]);
                    p = y;
                }
            }
            const bool cached = APPEND && it[j].kind > 0;
            int64_t dst = 0;
            if constexpr (APPEND)
                if (cached)
                    dst = ((((slot >> a.sh) * a.Hkv + it[j].head) << a.sh) |
                           (slot & ((1 << a.sh) - 1))) * PPR;
            if constexpr (APPEND && KV == SPEC_KV_E4M3) {
                if (__any_sync(0xffffffffu, cached)) {
                    float top = 0.0f;                    // NaN where there is one
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        top = max_nan(max_nan(top, fabsf(x[0][i])), fabsf(x[1][i]));
                    uint32_t most = __float_as_uint(top);
#pragma unroll
                    for (int o = 1; o < LPR; o <<= 1)
                        most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
                    if (cached) {
                        const float scale = row_scale(most), inv = __frcp_rn(scale);
                        void* pages = it[j].kind == 1 ? a.k_pages : a.v_pages;
                        if (lane == 0)
                            (it[j].kind == 1 ? a.k_scale : a.v_scale)[dst / PPR] = scale;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t c[VEC / 4];
#pragma unroll
                            for (int k = 0; k < VEC / 4; ++k)
                                c[k] = codes4(x[h][4 * k], x[h][4 * k + 1], x[h][4 * k + 2],
                                              x[h][4 * k + 3], scale, inv);
                            const int64_t to = dst + (h ? v1 : v0);
                            if constexpr (VEC == 8)
                                static_cast<uint2*>(pages)[to] = make_uint2(c[0], c[1]);
                            else
                                static_cast<uint32_t*>(pages)[to] = c[0];
                        }
                    }
                }
                if (cached) continue;
            }
            if (it[j].kind < 0) continue;
            uint4* to = cached ? static_cast<uint4*>(it[j].kind == 1 ? a.k_pages : a.v_pages) + dst
                               : it[j].dst;
            const bool same = it[j].kind == 2 || !turn;      // bits as they came
            to[v0] = same ? u[j][0] : pack<IO>(x[0]);
            to[v1] = same ? u[j][1] : pack<IO>(x[1]);
        }
    }
}

// How the heads of a token are shared out: every SM's threads are filled before a
// group takes a second head, at most MOST heads a group (the sines and cosines of
// eight pairs cost about as much as three heads; 8: prompts 1 us more, 16: 3).
constexpr int MOST = 12;

template <int IO, int KV, int D, int LAYOUT, bool APPEND>
cudaError_t launch_t(RopeArgs& a, int64_t rows, cudaStream_t st) {
    constexpr int LPR = D * (int)sizeof(typename io_t<IO>::T) / 32;
    int sms = device_sm_count();
    if (sms < 1) sms = 1;
    const int64_t room = (int64_t)sms * 2048 / LPR;
    int64_t per = rows * a.items / room;
    per = per < 1 ? 1 : (per > MOST ? MOST : per);
    a.share = (int)((a.items + per - 1) / per);
    a.per = (a.items + a.share - 1) / a.share;
    a.groups = rows * a.share;
    const int64_t ctas = (a.groups * LPR + NT - 1) / NT;
    if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
    return launch_k(true, rope_rows<IO, KV, D, LAYOUT, APPEND>, dim3((unsigned)ctas), dim3(NT), 0,
                    st, a);
}

RopeArgs rope_args(const spec_rope_cfg& c, const uint64_t* turns, float amp, const void* q,
                   const void* k, const void* v, void* q_out, void* k_out) {
    const int vec = c.io_dtype == SPEC_IO_BF16 ? 8 : 4;
    auto pieces = [&](int64_t stride, int heads) {
        return (stride ? stride : (int64_t)heads * c.D) / vec;
    };
    RopeArgs a{};
    a.turns = turns;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_out = q_out;
    a.k_out = k_out;
    a.q_stride = pieces(c.q_stride, c.Hq);
    a.k_stride = pieces(c.k_stride, c.Hkv);
    a.v_stride = pieces(c.v_stride, c.Hkv);
    a.Hq = c.Hq;
    a.Hkv = c.Hkv;
    a.items = c.Hq + (v ? 2 : 1) * c.Hkv;
    a.pairs = c.rot / (2 * vec);
    a.amp = amp;
    a.inverse = c.inverse;
    return a;
}

template <int IO, int D, int LAYOUT>
cudaError_t apply_t(RopeArgs& a, const spec_rope_cfg& c, cudaStream_t st) {
    return launch_t<IO, SPEC_KV_IO, D, LAYOUT, false>(a, c.rows, st);
}

template <int IO, int D, int LAYOUT>
cudaError_t append_t(RopeArgs& a, const spec_rope_cfg& c, int kv_dtype, cudaStream_t st) {
    return kv_dtype == SPEC_KV_E4M3 ? launch_t<IO, SPEC_KV_E4M3, D, LAYOUT, true>(a, c.rows, st)
                                    : launch_t<IO, SPEC_KV_IO, D, LAYOUT, true>(a, c.rows, st);
}

// fn<IO, D, LAYOUT>(...) for the configuration `c` in scope
#define SPEC_ROPE_DISPATCH(fn, ...)                                                       \
    do {                                                                                  \
        const bool d128 = c.D == 128, half = c.layout == SPEC_ROPE_HALF;                  \
        if (c.io_dtype == SPEC_IO_BF16) {                                                 \
            if (half)                                                                     \
                return d128 ? fn<SPEC_IO_BF16, 128, SPEC_ROPE_HALF>(__VA_ARGS__)          \
                            : fn<SPEC_IO_BF16, 64, SPEC_ROPE_HALF>(__VA_ARGS__);          \
            return d128 ? fn<SPEC_IO_BF16, 128, SPEC_ROPE_INTERLEAVED>(__VA_ARGS__)       \
                        : fn<SPEC_IO_BF16, 64, SPEC_ROPE_INTERLEAVED>(__VA_ARGS__);       \
        }                                                                                 \
        if (half)                                                                         \
            return d128 ? fn<SPEC_IO_F32, 128, SPEC_ROPE_HALF>(__VA_ARGS__)               \
                        : fn<SPEC_IO_F32, 64, SPEC_ROPE_HALF>(__VA_ARGS__);               \
        return d128 ? fn<SPEC_IO_F32, 128, SPEC_ROPE_INTERLEAVED>(__VA_ARGS__)            \
                    : fn<SPEC_IO_F32, 64, SPEC_ROPE_INTERLEAVED>(__VA_ARGS__);            \
    } while (0)

}  // namespace

cudaError_t launch_rope(const spec_rope_cfg& c, const uint64_t* turns, float amp,
                        const int32_t* pos, const void* q, const void* k, void* q_out,
                        void* k_out, cudaStream_t st) {
    RopeArgs a = rope_args(c, turns, amp, q, k, nullptr, q_out, k_out);
    a.pos = pos;
    SPEC_ROPE_DISPATCH(apply_t, a, c, st);
}

cudaError_t launch_rope_append(const spec_rope_cfg& c, const spec_paged_cfg& pc,
                               const spec_paged_kv& kv, const uint64_t* turns, float amp,
                               const int64_t* slots, const void* q, const void* k_new,
                               const void* v_new, void* q_out, void* ws, cudaStream_t st) {
    RopeArgs a = rope_args(c, turns, amp, q, k_new, v_new, q_out, nullptr);
    const PageMap pm = page_map(pc, kv);
    a.slots = slots;
    a.kv_len = kv.kv_len;
    a.k_pages = kv.k_pages;
    a.v_pages = kv.v_pages;
    a.k_scale = kv.k_scale;
    a.v_scale = kv.v_scale;
    a.n_slots = (int64_t)pc.n_pages << pm.sh;
    a.T = pc.T;
    a.sh = pm.sh;
    a.ws = ws;
    SPEC_ROPE_DISPATCH(append_t, a, c, pc.kv_dtype, st);
}

}  // namespace spec
