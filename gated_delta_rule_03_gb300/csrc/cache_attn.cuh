// cache_attn.cuh -- shared parts of attention over a paged 8-bit cache.
//
// Weights. An entry of the cache is a code times the scale of its page and head, so with
// t_j = log2(e) s_j + log2(vs_j) (vs_j: the value scale of token j's page) a row's results are
//     o = sum_j w_j code_j / l,   w_j = 2^(t_j - ref),   l = sum_j w_j / vs_j,   lse = ln l + ref ln 2
// for any reference: the codes enter the second product as they are (exact in fp16), and a
// weight is relative to the largest contribution even where pages differ much in scale.
// A row's ref follows its maximum, kSpan below it, and moves only when a weight would pass
// 2^(kSpan + kSlack): moving it costs a pass over the row's outputs. Weights in fp16 keep their 11
// bits down to 2^-21 of the largest and are dropped below 2^-32. For bf16 results that is enough: their own rounding is 1.65e-3
// in norm, with such weights 1.67e-3; a second part, which fp32 results take, would double the second product.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <math.h>

#include <mutex>

#include "codes.cuh"
#include "internal.h"
#include "scan.cuh"

namespace gdr {
namespace cattn {

constexpr float kSpan = 7.f, kSlack = 8.f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNoRef = -3.4028234663852886e38f;  // of a row that has seen nothing: the lowest number

struct Attn {
    const void *q;
    const uint8_t *kc, *vc;
    const float *ks, *vs;
    const int32_t *table, *kv_lens, *cu;
    const float *slopes;
    void *o;
    float *lse;
    int32_t *status;
    int64_t num_seqs, tokens, max_q, width, qs, pages;
    int heads, kv_heads, group, log_page, causal;
    int group_shift;  // log2 of group, -1 if it is no power of two
    float scale, softcap;
};

// Token of row r of a head of the cache, and its head in the group.
__device__ __forceinline__ int token_of(const Attn &a, int r) { return a.group_shift >= 0 ? r >> a.group_shift : r / a.group; }

// New tokens of request n: the first row and their number.
__device__ __forceinline__ int2 rows_of(const Attn &a, int64_t n) {
    if (a.cu) {
        const int c = __ldg(a.cu + n);
        return make_int2(c, __ldg(a.cu + n + 1) - c);
    }
    const int64_t len = a.max_q;
    return make_int2((int)(n * len), (int)len);
}
__device__ __forceinline__ bool lengths_hold(const Attn &a, int64_t n) {
    const int len = __ldg(a.kv_lens + n);
    if (len < 0 || len > (a.width << a.log_page)) return false;
    if (!a.cu) return true;
    const int c = __ldg(a.cu + n), d = __ldg(a.cu + n + 1);
    return (n > 0 || c == 0) && d >= c && d <= a.tokens && d - c <= a.max_q;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// tanh(x) = 1 - 2 / (1 + e^2x) is off by some 2e-7 in all (held to 2^-21 by the tests), and the cap times that in the
// score. Near 0 two terms of its series are off by 2 x^5 / 15, relative 1e-7 where they are taken, so that a score far
// below its cap keeps its bits whatever the cap: 2^-16 relative in all, enough for bf16 results; fp32 ones take the
// library's. (Prompts in bf16 with caps up to 64 have a quicker form without the series, cache_attn_tc.cuh.)
__device__ __forceinline__ float reciprocal(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <bool kExact> __device__ __forceinline__ float cap_of(float x) {
    if (kExact) return tanhf(x);
    const float far = fmaf(-2.f, reciprocal(1.f + ex2(2.f * kLog2e * x)), 1.f), near = fmaf(x * x, x * (-1.f / 3.f), x);
    return fabsf(x) < 0.03f ? near : far;
}

// Two numbers as fp16, lo in the low half, and back.
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 unpack_f16(uint32_t r) { return __half22float2(reinterpret_cast<const __half2 &>(r)); }

// The score of a token from a product that is already scaled; away = |p - j|.
template <bool kExact> __device__ __forceinline__ float shaped(float z, float softcap, float inv_cap, float slope, float away) {
    if (softcap > 0.f) z = softcap * cap_of<kExact>(z * inv_cap);
    return fmaf(-slope, away, z);
}

// 2^n that brings a row with this largest size (bits of an fp32 number) to 2^14 .. 2^15, so that
// fp16 holds its entries (to 2^-39 of the largest, subnormal ones included); 0 for NaN and
// infinity, which stay what they are.
__device__ __forceinline__ int row_shift(uint32_t bits) {
    const int e = (int)(bits >> 23);
    return e == 255 ? 0 : min(14 - (e - 127), 126);
}
__device__ __forceinline__ float two_to(int n) { return __int_as_float((n + 127) << 23); }

// Sum over the block and inclusive sums, kThreads threads.
template <int kThreads> __device__ int64_t block_sums(int64_t x, int64_t *sums, int64_t *total) {
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    x = warp_scan(x);
    __syncthreads();
    if (lane == 31) sums[w] = x;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
        if (i < w) before += sums[i];
        all += sums[i];
    }
    *total = all;
    return x + before;
}

// Tensor map of boxes of up to `most` rows of one page and head of a cache, 128 bytes of each at most, swizzled by as
// many or not.
inline bool map_cache(CUtensorMap *map, const void *cache, const Attn &a, int D, int most, bool swizzled) {
    const int wide = D < 128 ? D : 128, page = 1 << a.log_page;
    static decltype(&cuTensorMapEncodeTiled) encode = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) == cudaSuccess &&
            found == cudaDriverEntryPointSuccess)
            encode = reinterpret_cast<decltype(encode)>(f);
    });
    if (!encode) return false;
    const cuuint64_t rows = (cuuint64_t)a.kv_heads << a.log_page;
    const cuuint64_t dims[3] = {(cuuint64_t)D, rows, (cuuint64_t)a.pages}, strides[2] = {(cuuint64_t)D, rows * D};
    const cuuint32_t box[3] = {(cuuint32_t)wide, (cuuint32_t)(page < most ? page : most), 1}, each[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(cache), dims, strides, box, each,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, !swizzled ? CU_TENSOR_MAP_SWIZZLE_NONE : wide == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A part of one item's keys, for a join of several: log2 of its sum, then its outputs (divided by it).
// kRows rows.
template <int kRows, int D> struct Part {
    float lse2[kRows];
    float o[kRows][D];
};

int launch_step64(const Attn &a, int codes, int dtype, void *ws, cudaStream_t s);
int launch_step128(const Attn &a, int codes, int dtype, void *ws, cudaStream_t s);
int launch_step256(const Attn &a, int codes, int dtype, void *ws, cudaStream_t s);
size_t step_bytes64();
size_t step_bytes128();
size_t step_bytes256();
int launch_tc64(const Attn &a, int codes, int dtype, void *ws, cudaStream_t s);
int launch_tc128(const Attn &a, int codes, int dtype, void *ws, cudaStream_t s);
int launch_tc256(const Attn &a, int codes, int dtype, void *ws, cudaStream_t s);
size_t tc_bytes64(const Attn &a, int dtype);
size_t tc_bytes128(const Attn &a, int dtype);
size_t tc_bytes256(const Attn &a, int dtype);

}  // namespace cattn
}  // namespace gdr
