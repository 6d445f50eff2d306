// cache_append.cu -- new keys and values into the slots of a paged 8-bit cache.
//
// A run is a stretch of rows whose slots follow one another within a page. For each run, head and
// tensor: the largest size of the run's entries, the scale 2^k from it (with the page's scale
// where the run goes on behind older tokens), older codes rounded to a scale that grew, then the
// run's codes. Bound by memory: entries are read once (a run of up to kHold vectors per thread
// stays in registers between its two uses, the rest comes from L2 again), codes written once. 8 packed prompts of
// 512 to 8192 tokens, 4 heads of 128 in bf16, 123 MB in all: 31 us, 4.0 TB/s; 256 single tokens 5.8 us. A run's scale needs
// all its rows before the first code, so that a block waits for its loads, then for its warps, then writes: what it
// comes to is how many blocks an SM holds (6 of 80 registers a thread; fp32 4).
#include "codes.cuh"
#include "internal.h"
#include "spans.h"

namespace gdr {
namespace {

using namespace codes;

struct Append {
    const void *x[2];
    int64_t xs[2];
    uint8_t *cache[2];
    float *scale[2];
    const int32_t *slots;
    int64_t tokens, limit;  // limit: slots of the cache
    int heads, d, log_page, group;
};

constexpr int kWarps = 4;
constexpr int kHold = 4;

// 8 consecutive entries.
template <typename T> struct Eight;
template <> struct Eight<__nv_bfloat16> {
    uint4 w;
    __device__ __forceinline__ void load(const void *p) { w = __ldg((const uint4 *)p); }
    __device__ __forceinline__ uint32_t largest() const {  // bits of the largest size, as fp32
        uint32_t m = __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
        return max(m & 0xffffu, m >> 16) << 16;
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(a[i] << 16);
            v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
        }
    }
};
template <> struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const void *p) {
        a = __ldg((const float4 *)p);
        b = __ldg((const float4 *)p + 1);
    }
    __device__ __forceinline__ uint32_t largest() const {
        const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
        return m;
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
};

template <int kCode> __device__ __forceinline__ uint2 encode(const float (&v)[8], float inv) {
    uint2 r;
    r.x = from_f32x2<kCode>(v[0] * inv, v[1] * inv) | (from_f32x2<kCode>(v[2] * inv, v[3] * inv) << 16);
    r.y = from_f32x2<kCode>(v[4] * inv, v[5] * inv) | (from_f32x2<kCode>(v[6] * inv, v[7] * inv) << 16);
    return r;
}

// One run by kThreads threads (a warp, or the block with `shared` between its warps): rows t .. of the tensor into
// page `page` from place `off` on, at most `room` of them. A warp is told their number `len`; the block finds it while
// the first rows are on their way (a few too many at a run's end).
template <typename T, int kCode, int kThreads>
__device__ __forceinline__ void put_run(const Append &a, int which, int h, int64_t t, int32_t slot, int room, int len, uint32_t *shared) {
    const int tid = threadIdx.x & (kThreads - 1), lane = threadIdx.x & 31;
    const int64_t page = slot >> a.log_page;
    const int off = slot & ((1 << a.log_page) - 1);
    const int row_vecs = a.d >> 3, shift = 31 - __clz(row_vecs);  // of 8 entries
    const int64_t stride = which ? a.xs[1] : a.xs[0];
    const T *src = (const T *)(which ? a.x[1] : a.x[0]) + t * stride + (int64_t)h * a.d;
    auto from = [&](int i) { return src + (int64_t)(i >> shift) * stride + (i & (row_vecs - 1)) * 8; };
    float *const scale = (which ? a.scale[1] : a.scale[0]) + page * a.heads + h;
    uint8_t *const out = (which ? a.cache[1] : a.cache[0]) + (((page * a.heads + h) << a.log_page) + off) * a.d;
    const float before = off > 0 ? *scale : 0.f;

    int vecs = (kThreads > 32 ? room : len) << shift;
    Eight<T> held[kHold];
#pragma unroll
    for (int j = 0; j < kHold; ++j) {
        const int i = tid + j * kThreads;
        if (i < vecs) held[j].load(from(i));
    }
    if (kThreads > 32) {
        const bool follows = tid < room && __ldg(a.slots + t + tid) == slot + tid;
        const uint32_t some = __ballot_sync(~0u, follows);
        if (lane == 0) shared[threadIdx.x >> 5] = some;
        __syncthreads();
        len = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w)
            if (len == 32 * w) len += shared[w] == ~0u ? 32 : __ffs(~shared[w]) - 1;
        vecs = len << shift;
    }
    uint32_t most = 0;
#pragma unroll
    for (int j = 0; j < kHold; ++j)
        if (tid + j * kThreads < vecs) most = max(most, held[j].largest());
    for (int i = tid + kHold * kThreads; i < vecs; i += kThreads) {
        Eight<T> x;
        x.load(from(i));
        most = max(most, x.largest());
    }
    most = __reduce_max_sync(~0u, most);
    if (kThreads > 32) {
        uint32_t *const sums = shared + kThreads / 32;
        if (lane == 0) sums[threadIdx.x >> 5] = most;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) most = max(most, sums[i]);
    } else {
        __syncwarp();  // (every lane has read the page's scale)
    }
    float now = fmaxf(power_of_two(scale_exponent<kCode>(most)), before);
    const bool finite = most < 0x7f800000u && before == before;
    if (!finite) now = __int_as_float(0x7fffffff);
    if (tid == 0) *scale = now;
    const float inv = finite ? 1.f / now : 0.f;
    if (finite && before > 0.f && now > before) {
        uint2 *const old = (uint2 *)(out - (int64_t)off * a.d);
        const float ratio = before / now;
        for (int i = tid; i < off * row_vecs; i += kThreads) {
            const uint2 w = old[i];
            uint32_t p[4];
            to_f16x4<kCode>(w.x, p[0], p[1]);
            to_f16x4<kCode>(w.y, p[2], p[3]);
            float v[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 f = __half22float2(reinterpret_cast<const __half2 &>(p[e]));
                v[2 * e] = f.x;
                v[2 * e + 1] = f.y;
            }
            old[i] = encode<kCode>(v, ratio);
        }
    }
    auto put = [&](int i, const Eight<T> &x) {
        float v[8];
        x.get(v);
        if (!finite) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0.f;
        }
        ((uint2 *)out)[i] = encode<kCode>(v, inv);
    };
#pragma unroll
    for (int j = 0; j < kHold; ++j)
        if (tid + j * kThreads < vecs) put(tid + j * kThreads, held[j]);
    for (int i = tid + kHold * kThreads; i < vecs; i += kThreads) {
        Eight<T> x;
        x.load(from(i));
        put(i, x);
    }
    if (kThreads > 32) __syncthreads();  // (shared is used again by the next run)
}

// A block takes the runs that begin in its `group` rows, for one head of one tensor: by all its warps one after the other, or
// a warp each where they are short, 2048 entries on average (pages of 16, heads of 128: 35 us that way, 58 the
// other for 8 packed prompts of 512 to 8192 tokens; pages of 32: 40 and 33.5).
template <typename T, int kCode> __global__ void __launch_bounds__(kWarps * 32, sizeof(T) == 2 ? 6 : 4) append_kernel(Append a) {
    __shared__ uint32_t shared[2 * kWarps], starts[kWarps];
    __shared__ int least;  // entries of a run on average that are too many for a warp
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int64_t t0 = (int64_t)blockIdx.x * a.group;
    const int h = blockIdx.y, which = blockIdx.z;
    const int in_page = (1 << a.log_page) - 1;
    auto slot_of = [&](int64_t t) { return t < a.tokens ? __ldg(a.slots + t) : -1; };
    bool begins = false;
    if (tid < a.group) {
        const int64_t t = t0 + tid;
        const int32_t s = slot_of(t), last = t > 0 ? slot_of(t - 1) : -1;
        begins = s >= 0 && s < a.limit && (t == 0 || (s & in_page) == 0 || last != s - 1);
        // (few rows to a block: a run that goes on behind them may be long; 1000 tokens in pages of 128, heads of 256: 13 us, 30
        // by a warp)
        if (tid == a.group - 1) least = a.group < 32 && (slot_of(t + 1) & in_page) && slot_of(t + 1) == s + 1 ? a.group * a.d - 1 : 2048;
    }
    const uint32_t mine = __ballot_sync(~0u, begins);
    if (lane == 0) starts[w] = mine;
    __syncthreads();
    int runs = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) runs += __popc(starts[i]);
    const bool together = runs * least < a.group * a.d;
    int r = 0;
    for (int i = 0; i < kWarps; ++i) {
        for (uint32_t m = starts[i]; m; m &= m - 1, ++r) {
            if (!together && r % kWarps != w) continue;
            const int64_t t = t0 + 32 * i + __ffs(m) - 1;
            const int32_t s = slot_of(t);
            const int room = (int)min((int64_t)(in_page + 1 - (s & in_page)), a.tokens - t);
            if (together) {
                put_run<T, kCode, kWarps * 32>(a, which, h, t, s, room, 0, shared);
            } else {
                int len = 0;
                while (len < room) {  // 32 rows at a time, up to the first that does not follow
                    const int j = len + lane;
                    const uint32_t ok = __ballot_sync(~0u, j < room && slot_of(t + j) == s + j);
                    len += ok == ~0u ? 32 : __ffs(~ok) - 1;
                    if (ok != ~0u) break;
                }
                put_run<T, kCode, 32>(a, which, h, t, s, room, len, nullptr);
            }
        }
    }
}

template <typename T> void launch_append(const Append &a, int codes, cudaStream_t s) {
    const dim3 grid((unsigned)((a.tokens + a.group - 1) / a.group), a.heads, 2);
    if (codes == GDR_CODE_E4M3)
        append_kernel<T, GDR_CODE_E4M3><<<grid, kWarps * 32, 0, s>>>(a);
    else
        append_kernel<T, GDR_CODE_INT8><<<grid, kWarps * 32, 0, s>>>(a);
}

}  // namespace

int check_cache(const gdr_cache_shape *s, int *log_page) {
    if (!s || s->num_pages < 1 || s->kv_heads < 1 || s->kv_heads > 1 << 15) return GDR_ERR_INVALID_ARG;
    if (s->page != 16 && s->page != 32 && s->page != 64 && s->page != 128) return GDR_ERR_UNSUPPORTED;
    if (s->d != 64 && s->d != 128 && s->d != 256) return GDR_ERR_UNSUPPORTED;
    if (s->codes != GDR_CODE_E4M3 && s->codes != GDR_CODE_INT8) return GDR_ERR_UNSUPPORTED;
    if (s->dtype != GDR_F32 && s->dtype != GDR_BF16) return GDR_ERR_UNSUPPORTED;
    if (s->num_pages > INT32_MAX / s->page) return GDR_ERR_INVALID_ARG;
    *log_page = s->page == 16 ? 4 : s->page == 32 ? 5 : s->page == 64 ? 6 : 7;
    return GDR_OK;
}

}  // namespace gdr

using namespace gdr;

extern "C" int gdr_cache_append(const gdr_cache_shape *shape, int64_t tokens, const void *k, int64_t k_stride,
                                const void *v, int64_t v_stride, const int32_t *slots, void *k_cache,
                                void *v_cache, float *k_scale, float *v_scale, gdr_stream_t stream) {
    Append a = {};
    int st = check_cache(shape, &a.log_page);
    if (st != GDR_OK) return st;
    if (tokens < 0 || tokens > INT32_MAX) return GDR_ERR_INVALID_ARG;
    const size_t e = shape->dtype == GDR_F32 ? 4 : 2;
    const int64_t row = (int64_t)shape->kv_heads * shape->d;
    st = row_stride(k_stride, row, e, &a.xs[0]);
    if (st == GDR_OK) st = row_stride(v_stride, row, e, &a.xs[1]);
    if (st != GDR_OK) return st;
    if (!k_cache || !v_cache || !k_scale || !v_scale || (tokens > 0 && (!k || !v || !slots))) return GDR_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16)) return GDR_ERR_ALIGNMENT;
    if (!aligned(slots, 4) || !aligned(k_scale, 4) || !aligned(v_scale, 4)) return GDR_ERR_ALIGNMENT;
    const size_t cache = (size_t)shape->num_pages * row * shape->page, scales = (size_t)shape->num_pages * shape->kv_heads * 4;
    const Bytes in[] = {{k, reach(tokens, a.xs[0], row, e)}, {v, reach(tokens, a.xs[1], row, e)}, {slots, (size_t)tokens * 4}};
    const Bytes out[] = {{k_cache, cache}, {v_cache, cache}, {k_scale, scales}, {v_scale, scales}};
    if (!outputs_apart(in, 3, out, 4)) return GDR_ERR_INVALID_ARG;
    if (tokens == 0) return GDR_OK;
    a.x[0] = k, a.x[1] = v;
    a.cache[0] = (uint8_t *)k_cache, a.cache[1] = (uint8_t *)v_cache;
    a.scale[0] = k_scale, a.scale[1] = v_scale;
    a.slots = slots;
    a.tokens = tokens;
    a.limit = shape->num_pages * shape->page;
    a.heads = shape->kv_heads;
    a.d = shape->d;
    // Rows per block: single tokens of many requests are a run each, a warp's work; many rows are runs of
    // whole pages, and a block looks for one of 64 or 128, or for several. What the rows are is on the device, so their
    // number decides: 256 single tokens 3.8 us with 4 rows to a block (19.6 with 64), 2048 of them 13.6 (20.2), one prompt of 2048
    // 8.7 (5.3); 4096 single ones 24.7 (23.0), one prompt of 4096 13.8 (5.5); 4 heads of 128 in bf16.
    a.group = tokens <= 2048 ? kWarps : (shape->page < 64 ? 64 : shape->page);
    if (shape->dtype == GDR_F32)
        launch_append<float>(a, shape->codes, (cudaStream_t)stream);
    else
        launch_append<__nv_bfloat16>(a, shape->codes, (cudaStream_t)stream);
    return cuda_status(cudaGetLastError());
}
