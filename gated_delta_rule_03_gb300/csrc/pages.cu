// pages.cu -- pages of a paged cache: new tokens' pages, positions and slots from the requests'
// lengths, and pages given back.
//
// Integer work of a few kilobytes: bound by latency. One block scans the requests, 1024 at a
// time, and hands out their pages; the tokens' positions and slots follow in the same block up to
// kOneBlock of them, else in a second launch over as many blocks as they fill. 256 requests of a token each 5.4 us, 33
// prompts of 100 to 3000 tokens 6.9 us.
#include "internal.h"
#include "scan.cuh"
#include "spans.h"

namespace gdr {
namespace {

constexpr int kThreads = 1024;
// Tokens that one block places: 256 of them 5.2 us (7.1 with a second launch), 4000 6.5 (6.4), 8000 9.7 (7.3).
constexpr int64_t kOneBlock = 4096;

struct Plan {
    int64_t n, width, rows, pages;
    int log_page;
    const int32_t *q_lens, *kv_lens, *free_pages, *free_count;
    int32_t *table, *kv_out, *count_out, *cu, *start, *positions, *slots;
};

// Inclusive sum over the block; *total receives that of all threads.
__device__ int64_t block_scan(int64_t x, int64_t *sums, int64_t *total) {
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    x = warp_scan(x);
    __syncthreads();  // (sums of the last call have been read)
    if (lane == 31) sums[w] = x;
    __syncthreads();
    if (w == 0) sums[lane] = warp_scan(sums[lane]);
    __syncthreads();
    *total = sums[31];
    return x + (w ? sums[w - 1] : 0);
}
// First i in [0, n) with v[i] > x (n if there is none); v does not fall.
template <typename T> __device__ __forceinline__ int above(const T *v, int n, T x) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (v[mid] > x) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// Position and slot of token t, the i-th new one of request n that begins at `first` (< 0: refused).
__device__ __forceinline__ void place(const Plan &p, int64_t t, int64_t n, int64_t first, int64_t i) {
    int32_t pos = 0, slot = -1;
    if (first >= 0) {
        pos = (int32_t)(first + i);
        const int32_t page = p.table[n * p.width + (pos >> p.log_page)];
        if ((uint32_t)page <= (uint32_t)INT32_MAX >> p.log_page) slot = (page << p.log_page) + (pos & ((1 << p.log_page) - 1));
    }
    p.positions[t] = pos;
    p.slots[t] = slot;
}

template <bool kTokens> __global__ void __launch_bounds__(kThreads) plan_pages_kernel(Plan p) {
    __shared__ int64_t sums[32];
    __shared__ int64_t ends[kThreads];    // ends of the requests' new tokens
    __shared__ int32_t fresh[kThreads];   // ends of the pages they get, within this turn
    __shared__ int32_t firsts[kThreads];  // position of the first new token, -1 if refused
    __shared__ int32_t held[kThreads];    // pages they have
    __shared__ int64_t most;
    const int tid = threadIdx.x;
    const int64_t count = min((int64_t)*p.free_count, p.pages);
    int64_t tokens = 0, needs = 0;  // of the turns before
    if (tid == 0) most = 0;
    for (int64_t n0 = 0; n0 < p.n; n0 += kThreads) {
        const int64_t n = n0 + tid;
        const int here = (int)min((int64_t)kThreads, p.n - n0);
        int64_t q = 0, kv = 0;
        if (n < p.n) {
            q = max(p.q_lens ? p.q_lens[n] : 1, 0);
            kv = p.kv_lens[n];
        }
        int64_t total;
        const int64_t end = tokens + block_scan(q, sums, &total);
        const int64_t page = (int64_t)1 << p.log_page;
        const int64_t have = kv >= 0 ? (kv + page - 1) >> p.log_page : 0, all = (kv + q + page - 1) >> p.log_page;
        const bool fits = n < p.n && kv >= 0 && end <= p.rows && all <= p.width && kv + q <= INT32_MAX;
        const int64_t need = fits ? all - have : 0;
        int64_t total_need;
        const int64_t taken = needs + block_scan(need, sums, &total_need);
        const bool granted = fits && (need == 0 || taken <= count);
        const int get = granted ? (int)need : 0;
        int64_t got;
        const int64_t upto = block_scan(get, sums, &got);
        ends[tid] = end;
        fresh[tid] = (int32_t)upto;
        firsts[tid] = granted ? (int32_t)kv : -1;
        held[tid] = (int32_t)have;
        if (granted && need > 0) atomicMax((long long *)&most, (long long)taken);  // (any order gives the same)
        if (n < p.n) {
            if (n == 0) p.cu[0] = 0;
            p.cu[n + 1] = (int32_t)min(end, p.rows);
            p.start[n] = granted ? (int32_t)kv : -1;
            p.kv_out[n] = granted ? (int32_t)(kv + q) : (int32_t)kv;
        }
        __syncthreads();
        // the pages: those granted are the first `got` behind `needs`, as a refusal ends the list
        for (int64_t i = tid; i < got; i += kThreads) {
            const int r = above(fresh, here, (int32_t)i);
            const int j = (int)i - (r ? fresh[r - 1] : 0);
            p.table[(n0 + r) * p.width + held[r] + j] = p.free_pages[count - 1 - (needs + i)];
        }
        __syncthreads();
        if (kTokens) {
            const int64_t last = min(tokens + total, p.rows);
            for (int64_t t = tokens + tid; t < last; t += kThreads) {
                const int r = above(ends, here, t);
                place(p, t, n0 + r, firsts[r], t - (r ? ends[r - 1] : tokens));
            }
            __syncthreads();
        }
        tokens += total;
        needs += total_need;
    }
    if (kTokens)
        for (int64_t t = tokens + tid; t < p.rows; t += kThreads) {
            p.positions[t] = 0;
            p.slots[t] = -1;
        }
    __syncthreads();
    if (tid == 0) *p.count_out = (int32_t)(count - most);
}

__global__ void __launch_bounds__(256) place_tokens_kernel(Plan p) {
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= p.rows) return;
    const int n = above(p.cu + 1, (int)p.n, (int32_t)t);
    if (n < p.n)
        place(p, t, n, p.start[n], t - p.cu[n]);
    else {
        p.positions[t] = 0;
        p.slots[t] = -1;
    }
}

struct Release {
    int64_t n, width, pages;
    int log_page;
    const uint8_t *done;
    int32_t *kv_lens, *table, *free_pages, *free_count;
};

__global__ void __launch_bounds__(kThreads) release_pages_kernel(Release p) {
    __shared__ int64_t sums[32];
    __shared__ int32_t ends[kThreads];
    const int tid = threadIdx.x;
    int64_t count = max((int64_t)*p.free_count, (int64_t)0);
    __syncthreads();
    for (int64_t n0 = 0; n0 < p.n; n0 += kThreads) {
        const int64_t n = n0 + tid;
        const int here = (int)min((int64_t)kThreads, p.n - n0);
        int64_t give = 0;
        if (n < p.n && p.done[n]) {
            give = ((int64_t)max(p.kv_lens[n], 0) + (1 << p.log_page) - 1) >> p.log_page;
            give = min(give, p.width);
        }
        int64_t total;
        const int64_t upto = block_scan(give, sums, &total);
        // a request whose pages the list has no room for keeps them, and so do those behind it
        const int64_t room = max(p.pages - count, (int64_t)0);
        const bool fits = upto <= room;
        ends[tid] = fits ? (int32_t)upto : INT32_MAX;
        int64_t gone;
        block_scan(fits ? give : 0, sums, &gone);
        if (n < p.n && p.done[n] && fits) p.kv_lens[n] = 0;
        for (int64_t i = tid; i < gone; i += kThreads) {
            const int r = above(ends, here, (int32_t)i);
            int32_t *entry = p.table + (n0 + r) * p.width + (i - (r ? ends[r - 1] : 0));
            p.free_pages[count + i] = *entry;
            *entry = -1;
        }
        count += gone;
        __syncthreads();
        if (gone < total) break;
    }
    if (tid == 0) *p.free_count = (int32_t)count;
}

int check_shape(const gdr_page_shape *s, int *log_page) {
    if (!s || s->num_seqs < 1 || s->num_seqs > INT32_MAX / 2 || s->width < 1 || s->width > INT32_MAX) return GDR_ERR_INVALID_ARG;
    if (s->rows < 0 || s->rows > INT32_MAX || s->num_pages < 0) return GDR_ERR_INVALID_ARG;
    if (s->page != 16 && s->page != 32 && s->page != 64 && s->page != 128) return GDR_ERR_UNSUPPORTED;
    if (s->num_pages > INT32_MAX / s->page) return GDR_ERR_INVALID_ARG;
    *log_page = s->page == 16 ? 4 : s->page == 32 ? 5 : s->page == 64 ? 6 : 7;
    return GDR_OK;
}

}  // namespace
}  // namespace gdr

using namespace gdr;

extern "C" {

int gdr_page_plan(const gdr_page_shape *shape, const int32_t *q_lens, const int32_t *kv_lens,
                  const int32_t *free_pages, const int32_t *free_count, int32_t *block_table,
                  int32_t *kv_lens_out, int32_t *free_count_out, int32_t *cu_q, int32_t *start,
                  int32_t *positions, int32_t *slots, gdr_stream_t stream) {
    Plan p = {};
    const int st = check_shape(shape, &p.log_page);
    if (st != GDR_OK) return st;
    p.n = shape->num_seqs;
    p.width = shape->width;
    p.rows = shape->rows;
    p.pages = shape->num_pages;
    if (!kv_lens || !free_count || !block_table || !kv_lens_out || !free_count_out || !cu_q || !start) return GDR_ERR_INVALID_ARG;
    if ((p.rows > 0 && (!positions || !slots)) || (p.pages > 0 && !free_pages)) return GDR_ERR_INVALID_ARG;
    const void *all[] = {q_lens, kv_lens, free_pages, free_count, block_table, kv_lens_out, free_count_out, cu_q, start, positions, slots};
    for (const void *a : all)
        if (!aligned(a, 4)) return GDR_ERR_ALIGNMENT;
    const size_t n4 = (size_t)p.n * 4;
    const Bytes in[] = {{q_lens, n4}, {kv_lens_out == kv_lens ? nullptr : kv_lens, n4}, {free_pages, (size_t)p.pages * 4},
                        {free_count_out == free_count ? nullptr : free_count, 4}};
    const Bytes out[] = {{block_table, (size_t)(p.n * p.width) * 4}, {kv_lens_out, n4}, {free_count_out, 4}, {cu_q, n4 + 4},
                         {start, n4}, {positions, (size_t)p.rows * 4}, {slots, (size_t)p.rows * 4}};
    if (!outputs_apart(in, 4, out, 7)) return GDR_ERR_INVALID_ARG;
    p.q_lens = q_lens;
    p.kv_lens = kv_lens;
    p.free_pages = free_pages;
    p.free_count = free_count;
    p.table = block_table;
    p.kv_out = kv_lens_out;
    p.count_out = free_count_out;
    p.cu = cu_q;
    p.start = start;
    p.positions = positions;
    p.slots = slots;
    const cudaStream_t s = (cudaStream_t)stream;
    if (p.rows <= kOneBlock) {
        plan_pages_kernel<true><<<1, kThreads, 0, s>>>(p);
    } else {
        plan_pages_kernel<false><<<1, kThreads, 0, s>>>(p);
        place_tokens_kernel<<<(unsigned)((p.rows + 255) / 256), 256, 0, s>>>(p);
    }
    return cuda_status(cudaGetLastError());
}

int gdr_page_release(const gdr_page_shape *shape, const uint8_t *done, int32_t *kv_lens, int32_t *block_table,
                     int32_t *free_pages, int32_t *free_count, gdr_stream_t stream) {
    Release p = {};
    const int st = check_shape(shape, &p.log_page);
    if (st != GDR_OK) return st;
    p.n = shape->num_seqs;
    p.width = shape->width;
    p.pages = shape->num_pages;
    if (!done || !kv_lens || !block_table || !free_count || (p.pages > 0 && !free_pages)) return GDR_ERR_INVALID_ARG;
    const void *all[] = {kv_lens, block_table, free_pages, free_count};
    for (const void *a : all)
        if (!aligned(a, 4)) return GDR_ERR_ALIGNMENT;
    const Bytes in[] = {{done, (size_t)p.n}};
    const Bytes out[] = {{kv_lens, (size_t)p.n * 4}, {block_table, (size_t)(p.n * p.width) * 4}, {free_pages, (size_t)p.pages * 4}, {free_count, 4}};
    if (!outputs_apart(in, 1, out, 4)) return GDR_ERR_INVALID_ARG;
    p.done = done;
    p.kv_lens = kv_lens;
    p.table = block_table;
    p.free_pages = free_pages;
    p.free_count = free_count;
    release_pages_kernel<<<1, kThreads, 0, (cudaStream_t)stream>>>(p);
    return cuda_status(cudaGetLastError());
}

}  // extern "C"
