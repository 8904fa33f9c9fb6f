// paged_cache.cu -- the paged key/value cache written and read back.
//
// A row (one token's key or value of one head, D values) belongs to 8, 16 or
// 32 lanes, 16 bytes of the I/O type each, so that its maximum is a few shuffles
// and its codes leave in one piece.
//
// Written with 8 bits: scale = max(amax / 448, 2^-100), code = e4m3(x / scale).
// 448 is e4m3's largest value, so the row's largest value keeps all three
// mantissa bits; a rounding is at most 2^-4 of a value (2^-10 scale below the
// normal range).  The floor keeps 1 / scale in fp32's range.  Rows of zeros
// take scale 1, rows with a non-finite value a NaN scale and NaN codes.
//
// What bounds it: reading or writing the flat tensors (2 bytes a value in bf16)
// and the codes (1).  Measured (graph replays, D = 128, 8 kv-heads, bf16 and
// 8-bit codes): 8 requests of 1024-8192 rows read back 33.9 us, 6.0 TB/s; 4
// prompts of 1-4000 tokens written 11.6 us, 4.4 TB/s, bound by instructions
// (exact quotients, maxima, packing); 24 single tokens 1.8 us, latency.
#include <math.h>

#include "cache_rows.cuh"
#include "paged.cuh"

namespace spec {

namespace {

constexpr int NT = 256;

// The rows of one request, (token, head) in memory order, are cut into blocks of
// RPC rows, one to a CTA; a thread has UNR rows of its block, of the keys and of
// the values, all under way at once, and looks a row's place up once for both.
// (Prompts written, 4 rows of one of them, 2 and 4 of both: 12.8, 11.6, 11.3 us;
// single tokens 1.78, 1.76, 2.1; read back, one request of 4095 rows in bf16 5.4,
// 5.2, 5.5, 8 requests in 8 bits 33.8, 33.9, 33.3, and with 1 of both 44.)
constexpr int UNR = 2;

template <int IO, int D> struct rows_of {
    static constexpr int PER = NT / geo<IO, D>::LPR;     // rows per pass of the block
    static constexpr int RPC = UNR * PER;
};

struct RowArgs {
    PageMap pm;
    int T;                   // tokens per request in the flat tensors
    int blocks;              // CTAs per request
    uint32_t h_mul;          // ceil(2^32 / Hkv), 0 for Hkv = 1
    // x / Hkv for x < Hkv + 2^12
    __device__ __forceinline__ int token(int x) const { return h_mul ? __umulhi(x, h_mul) : x; }
};

template <int IO, int KV, int D>
__global__ void __launch_bounds__(NT)
append_rows(const __grid_constant__ RowArgs a, const uint4* __restrict__ k_new,
            const uint4* __restrict__ v_new, const int32_t* __restrict__ n_new, void* k_pages,
            void* v_pages, float* k_scale, float* v_scale, void* ws) {
    using G = geo<IO, D>;
    using R = rows_of<IO, D>;
    const PageMap& pm = a.pm;
    pdl_wait();
    const int b = blockIdx.x / a.blocks, row0 = (blockIdx.x - b * a.blocks) * R::RPC;
    const int lane = threadIdx.x % G::LPR, mine = threadIdx.x / G::LPR;
    const int tok0 = row0 / pm.Hkv, h0 = row0 - tok0 * pm.Hkv;
    uint32_t bits = 0;
    const int n = new_rows(n_new, b, a.T, bits);
    const int L = pm.kv_len[b];
    if (L < 0 || L > pm.cap() - n) bits |= SPEC_DEV_OVERFLOW;
    if (bits && row0 == 0 && threadIdx.x == 0) raise_status(ws, bits);
    if ((bits & SPEC_DEV_OVERFLOW) || tok0 >= n) return;
    const size_t base = ((size_t)b * a.T * pm.Hkv + row0) * G::LPR + lane;
    uint4 u[2 * UNR];                                          // key and value of a row in turn
    int64_t dst[UNR];
#pragma unroll
    for (int j = 0; j < UNR; ++j) {
        const int r = j * R::PER + mine, dt = a.token(h0 + r);
        const int i = tok0 + dt, h = h0 + r - dt * pm.Hkv;
        dst[j] = -1;
        u[2 * j] = u[2 * j + 1] = make_uint4(0, 0, 0, 0);
        if (i < n) {
            u[2 * j] = __ldg(k_new + base + r * G::LPR);
            u[2 * j + 1] = __ldg(v_new + base + r * G::LPR);
            dst[j] = pm.row(b, L + i, h);
            if (dst[j] < 0 && lane == 0) raise_status(ws, SPEC_DEV_BADPAGE);
        }
    }
    if constexpr (KV == SPEC_KV_IO) {
#pragma unroll
        for (int j = 0; j < UNR; ++j)
            if (dst[j] >= 0) {
                reinterpret_cast<uint4*>(k_pages)[dst[j] * G::LPR + lane] = u[2 * j];
                reinterpret_cast<uint4*>(v_pages)[dst[j] * G::LPR + lane] = u[2 * j + 1];
            }
    } else {
        // the largest magnitudes as integers: bit patterns of magnitudes order
        // like the numbers, infinities and NaN on top
        uint32_t top[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t w[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
            if constexpr (IO == SPEC_IO_F32) {
                top[j] = max(max(w[0] & 0x7fffffffu, w[1] & 0x7fffffffu),
                             max(w[2] & 0x7fffffffu, w[3] & 0x7fffffffu));
            } else {
                const uint32_t y = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                                            __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
                top[j] = max(y << 16, y & 0xffff0000u);
            }
        }
        static_assert(UNR == 2);
        // The four are reduced together: lanes whose number ends in binary 00, 10,
        // 01, 11 keep 0 to 3, so that one exchange serves two of them and every
        // lane makes one scale instead of four.
        const bool o1 = lane & 1, o2 = lane & 2;
        uint32_t k0 = o1 ? top[2] : top[0], k1 = o1 ? top[3] : top[1];
        k0 = max(k0, __shfl_xor_sync(0xffffffffu, o1 ? top[0] : top[2], 1));
        k1 = max(k1, __shfl_xor_sync(0xffffffffu, o1 ? top[1] : top[3], 1));
        uint32_t most = max(o2 ? k1 : k0, __shfl_xor_sync(0xffffffffu, o2 ? k0 : k1, 2));
#pragma unroll
        for (int o = 4; o < G::LPR; o <<= 1)
            most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
        const float scale = row_scale(most);
        const int64_t at = o1 ? dst[1] : dst[0];
        if (lane < 4 && at >= 0) (o2 ? v_scale : k_scale)[at] = scale;
        const float inv = __frcp_rn(scale);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int from = 2 * (j & 1) + j / 2;
            const float sj = __shfl_sync(0xffffffffu, scale, from, G::LPR);
            const float rj = __shfl_sync(0xffffffffu, inv, from, G::LPR);
            float x[G::VEC];
            unpack<IO>(u[j], x);
            uint32_t c[G::VEC / 4];
#pragma unroll
            for (int k = 0; k < G::VEC / 4; ++k)
                c[k] = codes4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3], sj, rj);
            if (dst[j / 2] >= 0) {
                void* pages = j & 1 ? v_pages : k_pages;
                if constexpr (G::VEC == 8)
                    reinterpret_cast<uint2*>(pages)[dst[j / 2] * G::LPR + lane] =
                        make_uint2(c[0], c[1]);
                else
                    reinterpret_cast<uint32_t*>(pages)[dst[j / 2] * G::LPR + lane] = c[0];
            }
        }
    }
}

template <int IO, int KV, int D>
__global__ void __launch_bounds__(NT)
read_rows(const __grid_constant__ RowArgs a, const void* __restrict__ k_pages,
          const void* __restrict__ v_pages, const float* __restrict__ k_scale,
          const float* __restrict__ v_scale, uint4* __restrict__ k_out, uint4* __restrict__ v_out,
          void* ws) {
    using G = geo<IO, D>;
    using R = rows_of<IO, D>;
    const PageMap& pm = a.pm;
    pdl_wait();
    const int b = blockIdx.x / a.blocks, row0 = (blockIdx.x - b * a.blocks) * R::RPC;
    const int lane = threadIdx.x % G::LPR, mine = threadIdx.x / G::LPR;
    const int tok0 = row0 / pm.Hkv, h0 = row0 - tok0 * pm.Hkv;
    int L = pm.kv_len[b];
    const int most = min(a.T, pm.cap());
    if (L < 0 || L > most) {
        if (row0 == 0 && threadIdx.x == 0) raise_status(ws, SPEC_DEV_OVERFLOW);
        L = L < 0 ? 0 : most;
    }
    if (tok0 >= L) return;
    constexpr int NW = KV == SPEC_KV_E4M3 ? G::VEC / 4 : 4;   // 32-bit words of a lane's piece
    uint32_t w[2 * UNR][NW];                       // key and value of a row in turn
    float scale[2 * UNR];
    bool have[UNR];
#pragma unroll
    for (int j = 0; j < UNR; ++j) {
        const int r = j * R::PER + mine, dt = a.token(h0 + r);
        const int i = tok0 + dt, h = h0 + r - dt * pm.Hkv;
        have[j] = i < L;
        if (!have[j]) continue;
        const int64_t src = pm.row(b, i, h);
        have[j] = src >= 0;
        if (src < 0) {
            if (lane == 0) raise_status(ws, SPEC_DEV_BADPAGE);
            continue;
        }
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const void* pages = v ? v_pages : k_pages;
            uint32_t(&y)[NW] = w[2 * j + v];
            if constexpr (KV == SPEC_KV_E4M3) {
                scale[2 * j + v] = __ldg((v ? v_scale : k_scale) + src);
                if constexpr (NW == 2) {
                    const uint2 x =
                        __ldg(reinterpret_cast<const uint2*>(pages) + src * G::LPR + lane);
                    y[0] = x.x;
                    y[1] = x.y;
                } else {
                    y[0] = __ldg(reinterpret_cast<const uint32_t*>(pages) + src * G::LPR + lane);
                }
            } else {
                const uint4 x = __ldg(reinterpret_cast<const uint4*>(pages) + src * G::LPR + lane);
                y[0] = x.x;
                y[1] = x.y;
                y[NW - 2] = x.z;
                y[NW - 1] = x.w;
            }
        }
    }
    const size_t base = ((size_t)b * a.T * pm.Hkv + row0) * G::LPR + lane;
#pragma unroll
    for (int j = 0; j < 2 * UNR; ++j) {
        if (!have[j / 2]) continue;
        uint4 u;
        if constexpr (KV == SPEC_KV_IO) {
            u = make_uint4(w[j][0], w[j][1], w[j][NW - 2], w[j][NW - 1]);
        } else {
            float x[G::VEC];
#pragma unroll
            for (int k = 0; k < G::VEC / 2; ++k) {
                const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                    (__nv_fp8x2_storage_t)(w[j][k / 2] >> (16 * (k % 2))), __NV_E4M3);
                const float2 f = __half22float2(__half2(h));
                x[2 * k] = f.x * scale[j];
                x[2 * k + 1] = f.y * scale[j];
            }
            if constexpr (IO == SPEC_IO_F32)
                u = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                               __float_as_uint(x[3]));
            else
                u = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                               pack_bf16(x[G::VEC - 4], x[G::VEC - 3]),
                               pack_bf16(x[G::VEC - 2], x[G::VEC - 1]));
        }
        (j & 1 ? v_out : k_out)[base + (j / 2 * R::PER + mine) * G::LPR] = u;
    }
}

// The launches overlap the end of the one before (its last CTAs and the write-back;
// one token per request 2.06 -> 1.78 us, graph replays); pdl_wait() comes before
// any access to memory, and there is no early trigger, so that what follows needs
// no such care.
// cudaErrorInvalidConfiguration when the launch would need too many CTAs.
template <int IO, int D>
cudaError_t row_args(const spec_paged_cfg& c, const spec_paged_kv& kv, int64_t T, RowArgs& a) {
    const int64_t rows = T * c.Hkv;
    const int rpc = rows_of<IO, D>::RPC;
    const int64_t blocks = (rows + rpc - 1) / rpc;
    if (rows > 0x7fffffff - 4096 || blocks * c.B > 0x7fffffff) return cudaErrorInvalidConfiguration;
    a.pm = page_map(c, kv);
    a.T = (int)T;
    a.blocks = (int)blocks;
    a.h_mul = c.Hkv == 1 ? 0u : (uint32_t)(((1ull << 32) + c.Hkv - 1) / c.Hkv);
    return cudaSuccess;
}

template <int IO, int KV, int D>
cudaError_t append_t(const spec_paged_cfg& c, const spec_paged_kv& kv, const void* k_new,
                     const void* v_new, const int32_t* n_new, void* ws, cudaStream_t st) {
    RowArgs a;
    const cudaError_t e = row_args<IO, D>(c, kv, c.T, a);
    if (e != cudaSuccess) return e;
    return launch_k(true, append_rows<IO, KV, D>, dim3((unsigned)(a.blocks * c.B)), dim3(NT),
                    0, st, a, static_cast<const uint4*>(k_new), static_cast<const uint4*>(v_new),
                    n_new, kv.k_pages, kv.v_pages, kv.k_scale, kv.v_scale, ws);
}

template <int IO, int KV, int D>
cudaError_t read_t(const spec_paged_cfg& c, const spec_paged_kv& kv, int Lmax, void* k_out,
                   void* v_out, void* ws, cudaStream_t st) {
    RowArgs a;
    const cudaError_t e = row_args<IO, D>(c, kv, Lmax, a);
    if (e != cudaSuccess) return e;
    return launch_k(true, read_rows<IO, KV, D>, dim3((unsigned)(a.blocks * c.B)), dim3(NT), 0,
                    st, a, kv.k_pages, kv.v_pages, kv.k_scale, kv.v_scale,
                    static_cast<uint4*>(k_out), static_cast<uint4*>(v_out), ws);
}

}  // namespace


cudaError_t launch_page_append(const spec_paged_cfg& c, const spec_paged_kv& kv, const void* k_new,
                               const void* v_new, const int32_t* n_new, void* ws,
                               cudaStream_t st) {
    SPEC_PAGED_DISPATCH(append_t, c, kv, k_new, v_new, n_new, ws, st);
}

cudaError_t launch_page_read(const spec_paged_cfg& c, const spec_paged_kv& kv, int Lmax,
                             void* k_out, void* v_out, void* ws, cudaStream_t st) {
    SPEC_PAGED_DISPATCH(read_t, c, kv, Lmax, k_out, v_out, ws, st);
}

}  // namespace spec
