// block_norm.cu -- the norms before and after a block, fused with the block's gate and the
// residual scale, and their gradients.
//
// For every row, with D entries, rms(a) = sqrt(mean a^2 + eps) and act the gate's function:
//   t  = y / rms(y) w_post   (or y),   x' = x + s act(g) t,   h = x' / rms(x') w_pre
// Backward, from dh and the gradient dx' that the stream after the block hands back, with
// rx = 1 / rms(x'), ry = 1 / rms(y):
//   dx = dx' + rx (dh w_pre) - rx^3 x' mean(dh w_pre x')        dw_pre  = sum dh x' rx
//   dz = s dx act(g),   dg = s dx t act'(g)                       dw_post = sum dz y ry
//   dy = ry (dz w_post) - ry^3 y mean(dz w_post y)                (or dz)
// The sums over rows: every block adds its own rows in order, a second kernel adds the
// blocks' sums in order, so that the result is the same every time.
//
// One row per TPR = blockDim.x threads, PER entries per thread in registers, so that every
// row is read once and written once; all arithmetic and every sum in fp32.
#include "internal.h"

namespace gdr {
namespace {

constexpr int kSms = 152;

// VEC consecutive entries (VEC divides D), read 16 bytes at a time where they are that many.
template <typename T, int VEC> struct alignas(sizeof(T) * VEC < 16 ? sizeof(T) * VEC : 16) Pack {
    T v[VEC];
};

template <typename T, int VEC, int PER>
__device__ __forceinline__ void load_row(const T *p, int D, float (&x)[PER]) {
#pragma unroll
    for (int j = 0; j < PER / VEC; ++j) {
        const int e = (threadIdx.x + blockDim.x * j) * VEC;
        if (e < D) {
            const Pack<T, VEC> a = *reinterpret_cast<const Pack<T, VEC> *>(p + e);
#pragma unroll
            for (int i = 0; i < VEC; ++i) x[j * VEC + i] = to_f32(a.v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) x[j * VEC + i] = 0.f;
        }
    }
}

template <typename T, int VEC, int PER>
__device__ __forceinline__ void store_row(T *p, int D, const float (&x)[PER]) {
#pragma unroll
    for (int j = 0; j < PER / VEC; ++j) {
        const int e = (threadIdx.x + blockDim.x * j) * VEC;
        if (e < D) {
            Pack<T, VEC> a;
#pragma unroll
            for (int i = 0; i < VEC; ++i) a.v[i] = from_f32<T>(x[j * VEC + i]);
            *reinterpret_cast<Pack<T, VEC> *>(p + e) = a;
        }
    }
}

template <int VEC, int PER>
__device__ __forceinline__ void load_weight(const float *w, int D, float (&x)[PER]) {
    if (w) {
        load_row<float, VEC>(w, D, x);
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) x[i] = 1.f;
    }
}

// Sums of K values over the blockDim.x threads of a row; `buf` has K floats per warp.
template <int K> __device__ __forceinline__ void row_sum(float (&s)[K], float *buf) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s[k] += __shfl_xor_sync(0xffffffffu, s[k], off);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return;
    const int warp = threadIdx.x >> 5;
    float *row = buf + threadIdx.y * warps * K;
    __syncthreads();  // the values of the sum before have been read
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) row[warp * K + k] = s[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float t = 0.f;
        for (int w = 0; w < warps; ++w) t += row[w * K + k];
        s[k] = t;
    }
}

__device__ __forceinline__ float sigmoid(float g) { return 1.f / (1.f + __expf(-g)); }

struct NormParams {
    int64_t rows;
    int D;
    int post, pre, act;
    int64_t gate_stride;  // 0: one row for all
    float s, eps;
    const float *w_post, *w_pre;
};

template <typename T, typename TX, int VEC, int PER>
__global__ void __launch_bounds__(512)
block_norm_fwd_kernel(const NormParams p, const TX *x, const T *y, const T *gate, TX *x_out, T *h) {
    __shared__ float buf[32];
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = row < p.rows;
    const int D = live ? p.D : 0;  // a row behind the last loads and stores nothing
    const int64_t at = row * p.D;
    float xv[PER], yv[PER], gv[PER];
    load_row<TX, VEC>(x + at, D, xv);
    if (y) {
        load_row<T, VEC>(y + at, D, yv);
        if (gate) load_row<T, VEC>(gate + row * p.gate_stride, D, gv);
        float w[PER];
        if (p.post) {
            float ss[1] = {0.f};
#pragma unroll
            for (int i = 0; i < PER; ++i) ss[0] = fmaf(yv[i], yv[i], ss[0]);
            row_sum(ss, buf);
            const float r = rsqrtf(ss[0] / p.D + p.eps);
            load_weight<VEC>(p.w_post, D, w);
#pragma unroll
            for (int i = 0; i < PER; ++i) yv[i] *= r * w[i];
        }
        if (gate) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const float a = p.act == GDR_GATE_IDENTITY ? gv[i] : sigmoid(gv[i]) * (p.act == GDR_GATE_SILU ? gv[i] : 1.f);
                yv[i] *= a;
            }
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) xv[i] = fmaf(p.s, yv[i], xv[i]);
        store_row<TX, VEC>(x_out + at, D, xv);
    }
    if (!h) return;
    float ss[1] = {0.f}, w[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) ss[0] = fmaf(xv[i], xv[i], ss[0]);
    row_sum(ss, buf);
    const float r = rsqrtf(ss[0] / p.D + p.eps);
    load_weight<VEC>(p.w_pre, D, w);
#pragma unroll
    for (int i = 0; i < PER; ++i) xv[i] *= r * w[i];
    store_row<T, VEC>(h + at, D, xv);
}

// Sums over this block's rows go to part[which][blockIdx.x * blockDim.y + threadIdx.y][D].
template <typename T, typename TX, int VEC, int PER>
__global__ void __launch_bounds__(512)
block_norm_bwd_kernel(const NormParams p, const TX *dx_out, const T *dh, const TX *x, const T *y,
                      const T *gate, TX *dx, T *dy, T *dgate, float *part_post, float *part_pre,
                      float *part_gate) {
    __shared__ float buf[96];
    float a_post[PER], a_pre[PER], a_gate[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) a_post[i] = a_pre[i] = a_gate[i] = 0.f;
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    const int64_t rounds = (p.rows + step - 1) / step;  // the same for every thread: barriers inside
    for (int64_t round = 0; round < rounds; ++round) {
        const int64_t row = round * step + (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
        const int D = row < p.rows ? p.D : 0;
        const int64_t at = row * p.D;
        float dv[PER], hv[PER], xv[PER], yv[PER], gv[PER], w[PER];
        if (dx_out) {
            load_row<TX, VEC>(dx_out + at, D, dv);
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i) dv[i] = 0.f;
        }
        if (dh) {
            load_row<T, VEC>(dh + at, D, hv);
            load_row<TX, VEC>(x + at, D, xv);
        }
        if (y) load_row<T, VEC>(y + at, D, yv);
        if (gate) load_row<T, VEC>(gate + row * p.gate_stride, D, gv);
        float sums[3] = {0.f, 0.f, 0.f};
        if (dh) {
            load_weight<VEC>(p.w_pre, D, w);
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                sums[0] = fmaf(xv[i], xv[i], sums[0]);
                sums[1] = fmaf(hv[i] * w[i], xv[i], sums[1]);
            }
        }
        if (p.post) {
#pragma unroll
            for (int i = 0; i < PER; ++i) sums[2] = fmaf(yv[i], yv[i], sums[2]);
        }
        if (dh || p.post) row_sum(sums, buf);
        if (dh) {
            const float r = rsqrtf(sums[0] / p.D + p.eps), m = r * r * (sums[1] / p.D);
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                a_pre[i] = fmaf(hv[i], xv[i] * r, a_pre[i]);
                dv[i] = fmaf(r, hv[i] * w[i] - xv[i] * m, dv[i]);
            }
        }
        store_row<TX, VEC>(dx + at, D, dv);
        if (!y) continue;
        const float r = p.post ? rsqrtf(sums[2] / p.D + p.eps) : 1.f;
        if (p.post) {
            load_weight<VEC>(p.w_post, D, w);
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i) w[i] = 1.f;
        }
        float dot[1] = {0.f};
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            float dz = p.s * dv[i];
            if (gate) {
                const float g = gv[i], sg = sigmoid(g);
                const float a = p.act == GDR_GATE_IDENTITY ? g : (p.act == GDR_GATE_SILU ? g * sg : sg);
                const float da = p.act == GDR_GATE_IDENTITY ? 1.f
                                 : (p.act == GDR_GATE_SILU ? sg * (1.f + g * (1.f - sg)) : sg * (1.f - sg));
                gv[i] = dz * (yv[i] * r * w[i]) * da;
                a_gate[i] += gv[i];
                dz *= a;
            }
            a_post[i] = fmaf(dz, yv[i] * r, a_post[i]);
            dz *= w[i];
            dot[0] = fmaf(dz, yv[i], dot[0]);
            dv[i] = dz;
        }
        if (gate && p.gate_stride && dgate) store_row<T, VEC>(dgate + at, D, gv);
        if (p.post) {
            row_sum(dot, buf);
            const float m = r * r * (dot[0] / p.D);
#pragma unroll
            for (int i = 0; i < PER; ++i) dv[i] = r * (dv[i] - yv[i] * m);
        }
        store_row<T, VEC>(dy + at, D, dv);
    }
    const int64_t mine = ((int64_t)blockIdx.x * blockDim.y + threadIdx.y) * p.D;
    if (part_post) store_row<float, VEC>(part_post + mine, p.D, a_post);
    if (part_pre) store_row<float, VEC>(part_pre + mine, p.D, a_pre);
    if (part_gate) store_row<float, VEC>(part_gate + mine, p.D, a_gate);
}

struct Sum {
    const float *part;
    void *out;
    int f32;  // out in fp32 (weights), else in the block's type (the gate's row)
};
struct Sums {
    Sum v[3];
};

// out[c] = sum over the parts of column c: 32 columns per block, 8 threads each take every
// eighth part, the eight added in order.
template <typename T>
__global__ void __launch_bounds__(256) column_sum_kernel(const Sums s, int parts, int D) {
    __shared__ float buf[8][33];
    const Sum &m = s.v[blockIdx.y];
    const int c = blockIdx.x * 32 + threadIdx.x;
    float t = 0.f;
    if (c < D)
        for (int r = threadIdx.y; r < parts; r += 8) t += m.part[(int64_t)r * D + c];
    buf[threadIdx.y][threadIdx.x] = t;
    __syncthreads();
    if (threadIdx.y == 0 && c < D) {
#pragma unroll
        for (int r = 1; r < 8; ++r) t += buf[r][threadIdx.x];
        if (m.f32) ((float *)m.out)[c] = t;
        else ((T *)m.out)[c] = from_f32<T>(t);
    }
}

// Threads per row, rows per block and (backward) blocks: a row's entries spread over whole
// warps, PER each; narrow rows share a block of up to 128 threads.
struct Shape2 {
    int per, vec;
    dim3 block;
};
Shape2 shape_of(int D) {
    Shape2 s;
    s.per = D <= 4096 ? 8 : 16;
    s.vec = D % 8 == 0 ? 8 : (D % 2 == 0 ? 2 : 1);
    const int tpr = ((D + s.per - 1) / s.per + 31) / 32 * 32;
    s.block = dim3((unsigned)tpr, (unsigned)(tpr >= 128 ? 1 : 128 / tpr));
    return s;
}
int bwd_blocks(int64_t rows, const Shape2 &s) {
    const int threads = (int)(s.block.x * s.block.y);
    const int64_t need = (rows + s.block.y - 1) / s.block.y;
    const int64_t most = (int64_t)kSms * (threads <= 512 ? 512 / threads : 1);
    return (int)(need < most ? need : most);
}

template <typename T, typename TX> struct Run {
    template <int VEC, int PER>
    static int fwd(const NormParams &p, const Shape2 &s, const void *x, const void *y, const void *gate,
                   void *x_out, void *h, cudaStream_t stream) {
        const int64_t blocks = (p.rows + s.block.y - 1) / s.block.y;
        block_norm_fwd_kernel<T, TX, VEC, PER><<<(unsigned)blocks, s.block, 0, stream>>>(
            p, (const TX *)x, (const T *)y, (const T *)gate, (TX *)x_out, (T *)h);
        return cuda_status(cudaGetLastError());
    }
    template <int VEC, int PER>
    static int bwd(const NormParams &p, const Shape2 &s, int blocks, const void *dx_out, const void *dh,
                   const void *x, const void *y, const void *gate, void *dx, void *dy, void *dgate,
                   float *pp, float *pn, float *pg, cudaStream_t stream) {
        block_norm_bwd_kernel<T, TX, VEC, PER><<<(unsigned)blocks, s.block, 0, stream>>>(
            p, (const TX *)dx_out, (const T *)dh, (const TX *)x, (const T *)y, (const T *)gate,
            (TX *)dx, (T *)dy, (T *)dgate, pp, pn, pg);
        return cuda_status(cudaGetLastError());
    }
};

#define GDR_NORM_BY_SHAPE(R, what, ...)                                        \
    do {                                                                       \
        if (s.per == 8) {                                                      \
            if (s.vec == 8) return R::template what<8, 8>(__VA_ARGS__);        \
            if (s.vec == 2) return R::template what<2, 8>(__VA_ARGS__);        \
            return R::template what<1, 8>(__VA_ARGS__);                        \
        }                                                                      \
        if (s.vec == 8) return R::template what<8, 16>(__VA_ARGS__);           \
        if (s.vec == 2) return R::template what<2, 16>(__VA_ARGS__);           \
        return R::template what<1, 16>(__VA_ARGS__);                           \
    } while (0)

template <typename T, typename TX>
int run_fwd(const NormParams &p, const Shape2 &s, const void *x, const void *y, const void *gate,
            void *x_out, void *h, cudaStream_t stream) {
    using R = Run<T, TX>;
    GDR_NORM_BY_SHAPE(R, fwd, p, s, x, y, gate, x_out, h, stream);
}
template <typename T, typename TX>
int run_bwd(const NormParams &p, const Shape2 &s, int blocks, const void *dx_out, const void *dh,
            const void *x, const void *y, const void *gate, void *dx, void *dy, void *dgate,
            float *pp, float *pn, float *pg, cudaStream_t stream) {
    using R = Run<T, TX>;
    GDR_NORM_BY_SHAPE(R, bwd, p, s, blocks, dx_out, dh, x, y, gate, dx, dy, dgate, pp, pn, pg, stream);
}

size_t elem(int dtype) { return dtype == GDR_F32 ? 4 : 2; }
bool apart(const void *a, size_t an, const void *b, size_t bn) {
    if (!a || !b || !an || !bn) return true;
    const char *pa = (const char *)a, *pb = (const char *)b;
    return pa + an <= pb || pb + bn <= pa;
}

int check_shape(const gdr_block_norm_shape *s, NormParams *p) {
    if (!s || s->rows < 0 || s->rows > INT32_MAX || s->D < 1) return GDR_ERR_INVALID_ARG;
    if (s->D > 8192) return GDR_ERR_UNSUPPORTED;
    if (s->dtype != GDR_F32 && s->dtype != GDR_BF16) return GDR_ERR_UNSUPPORTED;
    if (s->x_dtype != s->dtype && s->x_dtype != GDR_F32) return GDR_ERR_UNSUPPORTED;
    if (s->gate_act < GDR_GATE_IDENTITY || s->gate_act > GDR_GATE_SIGMOID) return GDR_ERR_UNSUPPORTED;
    if (s->gate_rows != 0 && s->gate_rows != 1 && s->gate_rows != s->rows) return GDR_ERR_INVALID_ARG;
    if (!(s->eps >= 0.f && s->eps < 3.0e38f)) return GDR_ERR_INVALID_ARG;
    if (!(s->res_scale > -3.0e38f && s->res_scale < 3.0e38f)) return GDR_ERR_INVALID_ARG;
    p->rows = s->rows;
    p->D = s->D;
    p->post = s->post_norm != 0;
    p->pre = s->pre_norm != 0;
    p->act = s->gate_act;
    // (with one row in all, the gate's gradient is a row's all the same)
    p->gate_stride = s->gate_rows > 1 || (s->gate_rows == 1 && s->rows == 1) ? s->D : 0;
    p->s = s->res_scale;
    p->eps = s->eps == 0.f ? 1e-6f : s->eps;
    return GDR_OK;
}

int aligned(const void *const *p, int n) {
    for (int i = 0; i < n; ++i)
        if ((uintptr_t)p[i] & 15u) return GDR_ERR_ALIGNMENT;
    return GDR_OK;
}

}  // namespace
}  // namespace gdr

using namespace gdr;

extern "C" {

int gdr_block_norm_fwd(const gdr_block_norm_shape *shape, const void *x, const void *y,
                       const void *gate, const float *w_post, const float *w_pre, void *x_out,
                       void *h, gdr_stream_t stream) {
    NormParams p;
    int st = check_shape(shape, &p);
    if (st != GDR_OK) return st;
    if ((w_post && !p.post) || (w_pre && !p.pre) || (h && !p.pre)) return GDR_ERR_INVALID_ARG;
    if (p.rows == 0) return GDR_OK;
    if (!y && (p.post || gate || x_out || !p.pre)) return GDR_ERR_INVALID_ARG;
    if ((gate != nullptr) != (shape->gate_rows != 0)) return GDR_ERR_INVALID_ARG;
    if (!x || (y && !x_out) || (p.pre && !h)) return GDR_ERR_INVALID_ARG;
    const void *all[] = {x, y, gate, w_post, w_pre, x_out, h};
    if ((st = aligned(all, 7)) != GDR_OK) return st;
    const size_t nx = (size_t)p.rows * p.D * elem(shape->x_dtype), nt = (size_t)p.rows * p.D * elem(shape->dtype);
    const size_t ng = (size_t)shape->gate_rows * p.D * elem(shape->dtype), nw = (size_t)p.D * 4;
    if (x_out != x && !apart(x_out, nx, x, nx)) return GDR_ERR_INVALID_ARG;
    if (!apart(x_out, nx, h, nt)) return GDR_ERR_INVALID_ARG;
    const struct { const void *p; size_t n; } in[] = {{y, nt}, {gate, ng}, {w_post, nw}, {w_pre, nw}};
    for (const auto &i : in)
        if (!apart(i.p, i.n, x_out, x_out ? nx : 0) || !apart(i.p, i.n, h, h ? nt : 0)) return GDR_ERR_INVALID_ARG;
    if (!apart(x, nx, h, nt)) return GDR_ERR_INVALID_ARG;
    p.w_post = w_post;
    p.w_pre = w_pre;
    const Shape2 s = shape_of(p.D);
    const cudaStream_t stm = (cudaStream_t)stream;
    if (shape->dtype == GDR_F32) return run_fwd<float, float>(p, s, x, y, gate, x_out, h, stm);
    if (shape->x_dtype == GDR_F32) return run_fwd<__nv_bfloat16, float>(p, s, x, y, gate, x_out, h, stm);
    return run_fwd<__nv_bfloat16, __nv_bfloat16>(p, s, x, y, gate, x_out, h, stm);
}

size_t gdr_block_norm_bwd_workspace_size(const gdr_block_norm_shape *shape) {
    NormParams p;
    if (check_shape(shape, &p) != GDR_OK) return 0;
    const Shape2 s = shape_of(p.D);
    const size_t parts = (size_t)bwd_blocks(p.rows, s) * s.block.y;
    return 256 + 3 * parts * ((size_t)(p.D + 3) / 4 * 4) * sizeof(float);
}

int gdr_block_norm_bwd(const gdr_block_norm_shape *shape, const void *dx_out, const void *dh,
                       const void *x_out, const void *y, const void *gate, const float *w_post,
                       const float *w_pre, void *dx, void *dy, void *dgate, float *dw_post,
                       float *dw_pre, void *workspace, size_t workspace_bytes, gdr_stream_t stream) {
    NormParams p;
    int st = check_shape(shape, &p);
    if (st != GDR_OK) return st;
    if (!y && (p.post || gate || dy) && p.rows > 0) return GDR_ERR_INVALID_ARG;
    if ((gate != nullptr) != (shape->gate_rows != 0) && p.rows > 0) return GDR_ERR_INVALID_ARG;
    if (((w_post || dw_post) && !p.post) || ((w_pre || dw_pre) && !p.pre) || (dgate && !shape->gate_rows))
        return GDR_ERR_INVALID_ARG;
    if (dh && !p.pre) return GDR_ERR_INVALID_ARG;
    if (p.rows > 0 && (!dx || (y && !dy) || (p.pre && (!dh || !x_out)) || (!p.pre && !dx_out)))
        return GDR_ERR_INVALID_ARG;
    const void *all[] = {dx_out, dh, x_out, y, gate, w_post, w_pre, dx, dy, dgate, dw_post, dw_pre, workspace};
    if ((st = aligned(all, 13)) != GDR_OK) return st;
    const size_t ws_need = gdr_block_norm_bwd_workspace_size(shape);
    const bool row_gate = gate && p.gate_stride == 0;
    if (dw_post || dw_pre || (row_gate && dgate))
        if (!workspace || workspace_bytes < ws_need) return GDR_ERR_WORKSPACE;
    const size_t nx = (size_t)p.rows * p.D * elem(shape->x_dtype), nt = (size_t)p.rows * p.D * elem(shape->dtype);
    const size_t ng = (size_t)shape->gate_rows * p.D * elem(shape->dtype), nw = (size_t)p.D * 4;
    const struct { const void *p; size_t n; } in[] = {{dx_out, nx}, {dh, nt}, {x_out, nx}, {y, nt},
                                                      {gate, ng}, {w_post, nw}, {w_pre, nw}};
    const struct { const void *p; size_t n; } out[] = {{dx, nx}, {dy, nt}, {dgate, ng}, {dw_post, nw},
                                                       {dw_pre, nw}, {workspace, workspace_bytes}};
    for (int i = 0; i < 6; ++i) {
        for (int j = 0; j < 7; ++j)
            if (!(i == 0 && j == 0 && dx == dx_out) && !apart(out[i].p, out[i].n, in[j].p, in[j].n))
                return GDR_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (!apart(out[i].p, out[i].n, out[j].p, out[j].n)) return GDR_ERR_INVALID_ARG;
    }
    p.w_post = w_post;
    p.w_pre = w_pre;
    const Shape2 s = shape_of(p.D);
    const cudaStream_t stm = (cudaStream_t)stream;
    const int blocks = bwd_blocks(p.rows, s);
    const int parts = blocks * (int)s.block.y;
    const size_t one = (size_t)parts * ((size_t)(p.D + 3) / 4 * 4);
    float *base = (float *)((char *)workspace + 256);
    float *pp = dw_post ? base : nullptr, *pn = dw_pre ? base + one : nullptr;
    float *pg = row_gate && dgate ? base + 2 * one : nullptr;
    if (blocks > 0) {
        if (shape->dtype == GDR_F32)
            st = run_bwd<float, float>(p, s, blocks, dx_out, dh, x_out, y, gate, dx, dy, dgate, pp, pn, pg, stm);
        else if (shape->x_dtype == GDR_F32)
            st = run_bwd<__nv_bfloat16, float>(p, s, blocks, dx_out, dh, x_out, y, gate, dx, dy, dgate, pp, pn, pg, stm);
        else
            st = run_bwd<__nv_bfloat16, __nv_bfloat16>(p, s, blocks, dx_out, dh, x_out, y, gate, dx, dy, dgate, pp, pn, pg, stm);
        if (st != GDR_OK) return st;
    }
    Sums sums = {};
    int n = 0;
    if (dw_post) sums.v[n++] = {pp, dw_post, 1};
    if (dw_pre) sums.v[n++] = {pn, dw_pre, 1};
    if (dgate && shape->gate_rows == 1 && p.gate_stride == 0) sums.v[n++] = {pg, dgate, shape->dtype == GDR_F32};
    if (n == 0) return GDR_OK;
    const dim3 grid((unsigned)((p.D + 31) / 32), (unsigned)n), block(32, 8);
    if (shape->dtype == GDR_F32) column_sum_kernel<float><<<grid, block, 0, stm>>>(sums, parts, p.D);
    else column_sum_kernel<__nv_bfloat16><<<grid, block, 0, stm>>>(sums, parts, p.D);
    return cuda_status(cudaGetLastError());
}

}  // extern "C"
