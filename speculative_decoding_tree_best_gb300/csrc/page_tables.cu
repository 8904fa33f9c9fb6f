// page_tables.cu -- page tables and slot maps from the requests' lengths, on the
// device: pages for the new tokens' rows (extend), pages given back (trim).
//
// Mathematics.  Which pages a request gets follows from the running total of
// what the requests before it lack: a prefix sum over at most 4096 requests.
// Totals grow, so the requests that the free list reaches are the first ones,
// and with G pages handed out in all, request b's begin at min(total before b, G)
// from the list's end.  Every CTA makes the whole sum for itself (a few loads a
// thread, from L2 after the first) instead of waiting for one that does; then the
// CTAs share out the slots and the table's new columns evenly, whatever the
// requests' lengths: a new page finds its request by a binary search over the
// totals.  What the sum is made from (n_held, n_free, kv_len) is brought up to
// date by the last CTA to have read it (a ticket), so nobody waits.
//
// What bounds it: the launch and the chain lengths - totals - table entry - slot;
// 8 bytes a slot written and 4 to 8 a page beyond that.  Measured (graph replays, both
// calls in turn): 256 requests of one token 7.8 us, 32 prompts of up to 8192 tokens,
// pages of 16, 10.1 us.
#include "serving.cuh"

namespace spec {

namespace {

constexpr int NT = 256;
// slots per CTA: four 16-byte stores a thread (512 threads: 11.9 us instead of 10.1 for prompts)
constexpr int SLOTS = NT * 8;

struct PoolArgs {
    spec_page_pool p;
    int B, T, max_pages, n_pages, sh;
};

// The requests in shared memory: rows held, pages held, new rows granted, and
// where their pages begin among those that change hands.
struct Req {
    int4* r;              // (kv_len, n_held, n, pages that change hands)
    int* first;
};

__device__ __forceinline__ Req req_smem(int B) {
    extern __shared__ int4 smem[];
    return Req{smem, reinterpret_cast<int*>(smem + B)};
}

// Exclusive prefix of x over the block, and the block's total.
__device__ __forceinline__ long long block_prefix(long long x, long long& total) {
    __shared__ long long part[NT / 32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    long long s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    if (lane == 31) part[warp] = s;
    __syncthreads();
    long long before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) before += part[w];
        total += part[w];
    }
    __syncthreads();
    return before + s - x;
}

__device__ __forceinline__ int free_pages(const PoolArgs& a, uint32_t& bits) {
    const int n = a.p.n_free[0];
    if (n < 0 || n > a.n_pages) bits |= SPEC_DEV_BADREQ;
    return n < 0 ? 0 : min(n, a.n_pages);
}

// The request whose pages hold number j of those that change hands.
__device__ __forceinline__ int owner(const Req& q, int B, long long j) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (q.first[mid] <= j) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Whether every CTA has read the pool: true in the last one to come here (all its
// threads), which finds the ticket at zero again.  The ticket is the attention's
// first, which is at zero between calls.
__device__ __forceinline__ bool all_have_read(void* ws) {
    __shared__ bool last;
    __syncthreads();
    if (threadIdx.x == 0) {
        last = true;
        if (gridDim.x > 1) {
            unsigned* t = ws_ptr<unsigned>(ws, kTicketOff);
            __threadfence();
            last = atomicAdd(t, 1u) == gridDim.x - 1;
            if (last) {
                __threadfence();
                *t = 0;
            }
        }
    }
    __syncthreads();
    return last;
}

__global__ void __launch_bounds__(NT)
extend_tables(const __grid_constant__ PoolArgs a, const int32_t* n_new, int64_t* slots,
              int32_t* n_ok, void* ws) {
    const Req q = req_smem(a.B);
    const int tid = threadIdx.x, B = a.B, page = 1 << a.sh;
    pdl_wait();
    uint32_t bits = 0;
    const int n_free = free_pages(a, bits);
    const long long cap = (long long)a.max_pages << a.sh;
    for (int b = tid; b < B; b += NT) {
        int n = new_rows(n_new, b, a.T, bits);
        const int L = a.p.kv_len[b], H = a.p.n_held[b];
        int grow = 0;
        if (L < 0 || L + (long long)n > cap) {
            bits |= SPEC_DEV_OVERFLOW;
            n = 0;
        } else if (H < 0 || H > a.max_pages) {
            bits |= SPEC_DEV_BADREQ;
            n = 0;
        } else if (n > 0) {
            grow = max(0, (int)((L + (long long)n + page - 1) >> a.sh) - H);
        }
        q.r[b] = make_int4(L, H, n, grow);
    }
    __syncthreads();
    // running totals: a run of requests per thread
    const int per = (B + NT - 1) / NT, b0 = min(B, tid * per), b1 = min(B, b0 + per);
    long long sum = 0, all;
    for (int b = b0; b < b1; ++b) sum += q.r[b].w;
    long long before = block_prefix(sum, all);
    long long given = 0;
    if (all > n_free) {                                  // not all of them, then
        long long t = before;
        for (int b = b0; b < b1; ++b) {
            t += q.r[b].w;
            if (t <= n_free) given = t;
        }
        __shared__ int most;
        if (tid == 0) most = 0;
        __syncthreads();
        atomicMax(&most, (int)given);
        __syncthreads();
        given = most;
    } else {
        given = all;
    }
    for (int b = b0; b < b1; ++b) {
        int4& r = q.r[b];
        q.first[b] = (int)min(before, given);
        before += r.w;
        if (r.w > 0 && before > n_free) {
            bits |= SPEC_DEV_NOPAGE;
            r.z = r.w = 0;
        }
    }
    if (bits && blockIdx.x == 0) raise_status(ws, bits);
    bits = 0;
    __syncthreads();
    // the new columns
    for (long long j = (long long)blockIdx.x * NT + tid; j < given; j += (long long)gridDim.x * NT) {
        const int b = owner(q, B, j);
        a.p.page_table[(size_t)b * a.max_pages + q.r[b].y + (j - q.first[b])] =
            a.p.free_list[n_free - 1 - j];
    }
    // the slots
    const int64_t c0 = (int64_t)blockIdx.x * SLOTS, end = (int64_t)B * a.T;
    const uint32_t r0 = (uint32_t)(c0 / a.T), off = (uint32_t)(c0 - (int64_t)r0 * a.T);
    auto slot = [&](uint32_t x) -> int64_t {
        const uint32_t db = x / (uint32_t)a.T;
        const int b = r0 + db, i = x - db * a.T;
        const int4 r = q.r[b];
        if (i >= r.z) return -1;
        const int pos = r.x + i, col = pos >> a.sh;
        const int p = col < r.y ? a.p.page_table[(size_t)b * a.max_pages + col]
                                : a.p.free_list[n_free - 1 - (q.first[b] + col - r.y)];
        if ((unsigned)p >= (unsigned)a.n_pages) {
            bits |= SPEC_DEV_BADPAGE;
            return -1;
        }
        return ((int64_t)p << a.sh) | (pos & (page - 1));
    };
#pragma unroll 2
    for (int at = 2 * tid; at < SLOTS; at += 2 * NT) {
        if (c0 + at >= end) break;
        longlong2 s;
        s.x = slot(off + at);
        if (c0 + at + 1 < end) {
            s.y = slot(off + at + 1);
            *reinterpret_cast<longlong2*>(slots + c0 + at) = s;
        } else {
            slots[c0 + at] = s.x;
        }
    }
    if (bits) raise_status(ws, bits);
    if (!all_have_read(ws)) return;
    for (int b = tid; b < B; b += NT) {
        const int4 r = q.r[b];
        n_ok[b] = r.z;
        if (r.w > 0) a.p.n_held[b] = r.y + r.w;
    }
    if (tid == 0) a.p.n_free[0] = n_free - (int)given;
}

__global__ void __launch_bounds__(NT)
trim_tables(const __grid_constant__ PoolArgs a, const int32_t* keep, void* ws) {
    const Req q = req_smem(a.B);
    const int tid = threadIdx.x, B = a.B, page = 1 << a.sh;
    pdl_wait();
    uint32_t bits = 0;
    const int n_free = free_pages(a, bits);
    for (int b = tid; b < B; b += NT) {
        const int L = a.p.kv_len[b], H = a.p.n_held[b];
        int k = keep[b];
        if (k < -1 || H < 0 || H > a.max_pages) {
            bits |= SPEC_DEV_BADREQ;
            k = -1;
        }
        const int left = k < 0 ? H : min(H, (int)((k + (long long)page - 1) >> a.sh));
        q.r[b] = make_int4(k < 0 ? L : min(L, k), left, k, H - left);
    }
    __syncthreads();
    const int per = (B + NT - 1) / NT, b0 = min(B, tid * per), b1 = min(B, b0 + per);
    long long sum = 0, all;
    for (int b = b0; b < b1; ++b) sum += q.r[b].w;
    long long before = block_prefix(sum, all);
    // (a pool whose tables name more than 2^31 pages names pages twice)
    for (int b = b0; b < b1; ++b) {
        q.first[b] = (int)min(before, 0x7fffffffLL);
        before += q.r[b].w;
    }
    if (n_free + all > a.n_pages) bits |= SPEC_DEV_BADREQ;
    __syncthreads();
    for (long long j = (long long)blockIdx.x * NT + tid; j < min(all, 0x7fffffffLL);
         j += (long long)gridDim.x * NT) {
        const int b = owner(q, B, j);
        int32_t* e = a.p.page_table + (size_t)b * a.max_pages + q.r[b].y + (j - q.first[b]);
        const int p = *e;
        *e = -1;
        if (n_free + j < a.n_pages) a.p.free_list[n_free + j] = p;
    }
    if (bits && blockIdx.x == 0) raise_status(ws, bits);
    if (!all_have_read(ws)) return;
    for (int b = tid; b < B; b += NT) {
        const int4 r = q.r[b];
        if (r.z < 0) continue;
        a.p.kv_len[b] = r.x;
        a.p.n_held[b] = r.y;
    }
    if (tid == 0) a.p.n_free[0] = (int)min(n_free + all, (long long)a.n_pages);
}

PoolArgs pool_args(const spec_paged_cfg& c, const spec_page_pool& p) {
    PoolArgs a{p, c.B, c.T, c.max_pages, c.n_pages, 0};
    while ((1 << a.sh) < c.page) ++a.sh;
    return a;
}

// Shared memory of a launch; past the 48 KB that need no leave (2457 requests) it
// is asked for.
template <typename K> cudaError_t req_bytes(K kernel, int B, size_t& bytes) {
    bytes = (size_t)B * (sizeof(int4) + sizeof(int));
    if (bytes <= 48 * 1024) return cudaSuccess;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

}  // namespace

cudaError_t launch_pages_extend(const spec_paged_cfg& c, const spec_page_pool& p,
                                const int32_t* n_new, int64_t* slots, int32_t* n_ok, void* ws,
                                cudaStream_t st) {
    size_t smem;
    const cudaError_t e = req_bytes(extend_tables, c.B, smem);
    if (e != cudaSuccess) return e;
    const int64_t ctas = ((int64_t)c.B * c.T + SLOTS - 1) / SLOTS;      // at most 2^20
    return launch_k(true, extend_tables, dim3((unsigned)ctas), dim3(NT), smem, st,
                    pool_args(c, p), n_new, slots, n_ok, ws);
}

cudaError_t launch_pages_trim(const spec_paged_cfg& c, const spec_page_pool& p,
                              const int32_t* keep, void* ws, cudaStream_t st) {
    size_t smem;
    const cudaError_t e = req_bytes(trim_tables, c.B, smem);
    if (e != cudaSuccess) return e;
    // no more pages change hands than there are: one a thread, a CTA an SM
    const int64_t most = c.n_pages < (int64_t)c.B * c.max_pages ? c.n_pages
                                                                : (int64_t)c.B * c.max_pages;
    int sms = device_sm_count();
    if (sms < 1) sms = 1;
    int64_t ctas = (most + NT - 1) / NT;
    if (ctas > sms) ctas = sms;
    return launch_k(true, trim_tables, dim3((unsigned)ctas), dim3(NT), smem, st, pool_args(c, p),
                    keep, ws);
}

}  // namespace spec
