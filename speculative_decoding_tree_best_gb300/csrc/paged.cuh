// paged.cuh -- shapes, checks and addressing shared by the paged-cache kernels
// (paged_cache.cu, attn_paged.cu) and the chain verification (draft_verify.cu).
#pragma once

#include <cuda_fp8.h>

#include "checks.h"
#include "common.cuh"

namespace spec {

inline int check_paged_cfg(const spec_paged_cfg* c) {
    if (!c) return ST_EINVAL;
    if (c->B < 1 || c->B > SPEC_MAX_PAGED_B || c->T < 1 || c->T > (1 << 20)) return ST_EINVAL;
    if (c->Hq < 1 || c->Hkv < 1 || c->Hkv > SPEC_MAX_HKV || c->Hq % c->Hkv != 0) return ST_EINVAL;
    if ((int64_t)c->B * c->Hq > (1 << 24)) return ST_EINVAL;
    if (c->D != 64 && c->D != 128) return ST_EINVAL;
    if (c->page < SPEC_MIN_PAGE || c->page > SPEC_MAX_PAGE || (c->page & (c->page - 1)))
        return ST_EINVAL;
    if (c->n_pages < 1 || c->max_pages < 1 || (int64_t)c->max_pages * c->page > (1 << 30))
        return ST_EINVAL;
    if (c->io_dtype != SPEC_IO_F32 && c->io_dtype != SPEC_IO_BF16) return ST_EUNSUPPORTED;
    if (c->kv_dtype != SPEC_KV_IO && c->kv_dtype != SPEC_KV_E4M3) return ST_EUNSUPPORTED;
    return ST_OK;
}

inline int check_paged_kv(const spec_paged_cfg& c, const spec_paged_kv* kv) {
    if (!kv || !al16(kv->k_pages) || !al16(kv->v_pages) || !al16(kv->page_table) ||
        !al16(kv->kv_len))
        return ST_EINVAL;
    if (c.kv_dtype == SPEC_KV_E4M3 && (!al16(kv->k_scale) || !al16(kv->v_scale))) return ST_EINVAL;
    return ST_OK;
}

inline int check_draft_cfg(const spec_draft_cfg* c) {
    if (!c) return ST_EINVAL;
    if (c->B < 1 || c->B > 65535 || c->N < 0 || c->N + 1 > SPEC_MAX_ROWS)
        return ST_EINVAL;
    // the kernels step over a row in 32 bits, some thousands of tokens past its end
    if (c->V < 1 || c->V > SPEC_MAX_DRAFT_V) return ST_EINVAL;
    if (!(c->temperature > 0.0f && c->temperature <= 3.4028234663852886e38f) || c->reserved != 0u)
        return ST_EINVAL;
    if (c->io_dtype != SPEC_IO_F32 && c->io_dtype != SPEC_IO_BF16) return ST_EUNSUPPORTED;
    return ST_OK;
}

// How the decode attention's rows (T tokens x Hq/Hkv heads of a kv-head) are
// tiled: nr columns of 8 rows per warp, rtc row tiles per CTA, rtg row groups.
struct RowTiles {
    int nr, rtc, rtg;
};

inline RowTiles paged_row_tiles(const spec_paged_cfg& c) {
    const int64_t rows = (int64_t)c.T * (c.Hq / c.Hkv);
    RowTiles r{};
    r.nr = rows <= 8 ? 1 : 2;
    const int64_t tiles = (rows + 8 * r.nr - 1) / (8 * r.nr);
    r.rtg = (int)((tiles + 2) / 3);
    r.rtc = (int)((tiles + r.rtg - 1) / r.rtg);
    return r;
}

// The head of a workspace of the paged calls and of the chain verification:
// status word, then the tickets of both, which every call finds at zero and
// leaves at zero.  Their places and their number go by the SMs alone, so that no
// configuration has data where another has tickets, and one workspace serves any
// of them in turn.
//   attention      a ticket per CTA: a segment cut between CTAs counts in that of
//                  the CTA with its first granule (no two cut ones begin in a CTA)
//   verification   a ticket per request whose race is cut into slices: fewer
//                  requests than kRaceCtas per SM (draft_ws_layout)
constexpr int kRaceCtas = 3;
constexpr size_t kTicketOff = 256;
inline size_t draft_ticket_off(int num_sms) {
    return kTicketOff + sizeof(uint32_t) * (size_t)num_sms;
}
inline size_t ws_data_off(int num_sms) {
    return align_up(draft_ticket_off(num_sms) + sizeof(uint32_t) * kRaceCtas * (size_t)num_sms, 256);
}

// Attention: two parts per CTA (its first and last segment may be shared with its
// neighbours): fp32 outputs in the warps' register order, and (max, max, sum, sum)
// per lane.
struct PagedWs {
    size_t part_o_off, part_ml_off, total;
    int rtc, rtg;
};

inline PagedWs paged_ws_layout(const spec_paged_cfg& c, int num_sms) {
    PagedWs w{};
    w.total = ws_data_off(num_sms);
    if (c.T > SPEC_MAX_ROWS) return w;       // no attention with so many rows
    const RowTiles r = paged_row_tiles(c);
    w.rtc = r.rtc;
    w.rtg = r.rtg;
    const size_t tiles = (size_t)2 * num_sms * r.rtc * r.nr;
    w.part_o_off = w.total;
    w.part_ml_off = align_up(w.part_o_off + tiles * 8 * c.D * sizeof(float), 256);
    w.total = align_up(w.part_ml_off + tiles * 32 * 16, 256);
    return w;
}

// How the verification is split: `splits` segments per logits row, `slices` of
// `per` tokens for the race.  About eight CTAs per SM over all rows (five are
// resident at once: 1.7 waves), and kRaceCtas over the requests' races, but no segment under 4096 and no slice under 2048
// tokens (a load per thread).
struct DraftWs {
    size_t part_off, cand_off, total;
    int splits, slices, per;
};

inline DraftWs draft_ws_layout(const spec_draft_cfg& c, int num_sms) {
    DraftWs w{};
    const int64_t rows = (int64_t)c.B * (c.N + 1);
    auto clamp = [](int64_t want, int64_t most) {
        return (int)(want < 1 ? 1 : (want > most ? most : want));
    };
    w.splits = clamp((8LL * num_sms + rows - 1) / rows, ((int64_t)c.V + 4095) / 4096);
    w.slices = clamp(((int64_t)kRaceCtas * num_sms + c.B - 1) / c.B, ((int64_t)c.V + 2047) / 2048);
    w.per = (int)((((int64_t)c.V + w.slices - 1) / w.slices + 7) / 8 * 8);
    w.slices = (int)(((int64_t)c.V + w.per - 1) / w.per);
    w.part_off = ws_data_off(num_sms);
    w.cand_off = align_up(w.part_off + sizeof(float) * 2 * rows * w.splits, 256);
    w.total = align_up(w.cand_off + sizeof(float) * 2 * (size_t)c.B * w.slices, 256);
    return w;
}

cudaError_t launch_page_append(const spec_paged_cfg& c, const spec_paged_kv& kv, const void* k_new,
                               const void* v_new, const int32_t* n_new, void* ws, cudaStream_t st);
cudaError_t launch_page_read(const spec_paged_cfg& c, const spec_paged_kv& kv, int Lmax,
                             void* k_out, void* v_out, void* ws, cudaStream_t st);
cudaError_t launch_attn_paged(const spec_paged_cfg& c, const spec_paged_kv& kv, const void* q,
                              const int32_t* n_new, void* o, void* ws, cudaStream_t st);
cudaError_t launch_draft_verify(const spec_draft_cfg& c, const int32_t* draft_tok,
                                const int32_t* n_draft, const float* draft_prob,
                                const void* logits, const float* u, const float* e,
                                const spec_draft_out& out, int32_t* kv_len, int32_t* root_tok,
                                void* ws, cudaStream_t st);

// fn<IO, KV, D>(...) for the configuration `c` in scope
#define SPEC_PAGED_DISPATCH(fn, ...)                                                   \
    do {                                                                               \
        const bool d128 = c.D == 128, q8 = c.kv_dtype == SPEC_KV_E4M3;                 \
        if (c.io_dtype == SPEC_IO_BF16) {                                              \
            if (q8)                                                                    \
                return d128 ? fn<SPEC_IO_BF16, SPEC_KV_E4M3, 128>(__VA_ARGS__)         \
                            : fn<SPEC_IO_BF16, SPEC_KV_E4M3, 64>(__VA_ARGS__);         \
            return d128 ? fn<SPEC_IO_BF16, SPEC_KV_IO, 128>(__VA_ARGS__)               \
                        : fn<SPEC_IO_BF16, SPEC_KV_IO, 64>(__VA_ARGS__);               \
        }                                                                              \
        if (q8)                                                                        \
            return d128 ? fn<SPEC_IO_F32, SPEC_KV_E4M3, 128>(__VA_ARGS__)              \
                        : fn<SPEC_IO_F32, SPEC_KV_E4M3, 64>(__VA_ARGS__);              \
        return d128 ? fn<SPEC_IO_F32, SPEC_KV_IO, 128>(__VA_ARGS__)                    \
                    : fn<SPEC_IO_F32, SPEC_KV_IO, 64>(__VA_ARGS__);                    \
    } while (0)

// ---- device side ------------------------------------------------------------------

// What a paged kernel needs to find a row, by value.
struct PageMap {
    const int32_t* table;
    const int32_t* kv_len;
    int max_pages, n_pages, sh;          // page = 1 << sh
    int Hkv;
    __device__ __forceinline__ int cap() const { return max_pages << sh; }
    // index of (row, head) among the pool's rows, or -1 when the page is not in the pool
    __device__ __forceinline__ int64_t row(int b, int pos, int h) const {
        const int p = table[(size_t)b * max_pages + (pos >> sh)];
        if ((unsigned)p >= (unsigned)n_pages) return -1;
        return ((((int64_t)p * Hkv + h) << sh) | (pos & ((1 << sh) - 1)));
    }
};

inline PageMap page_map(const spec_paged_cfg& c, const spec_paged_kv& kv) {
    PageMap m{kv.page_table, kv.kv_len, c.max_pages, c.n_pages, 0, c.Hkv};
    while ((1 << m.sh) < c.page) ++m.sh;
    return m;
}

// New rows of request b: n_new[b] (NULL: T) clamped to [0, T]; raises
// SPEC_DEV_BADREQ through `bits`.
__device__ __forceinline__ int new_rows(const int32_t* n_new, int b, int T, uint32_t& bits) {
    if (!n_new) return T;
    const int n = n_new[b];
    if (n < 0 || n > T) bits |= SPEC_DEV_BADREQ;
    return n < 0 ? 0 : (n > T ? T : n);
}

}  // namespace spec
