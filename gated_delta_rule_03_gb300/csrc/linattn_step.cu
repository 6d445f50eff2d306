// linattn_step.cu -- one token of linear attention with a constant decay per head, for
// every sequence of a batch: S <- lam S + k v^T, o = scale S^T q, the state read and written
// once.
//
// One CTA per (sequence, head, DVT columns of the state); every thread holds 16 rows x 4
// columns in registers, all 16 loads issued before any arithmetic. The columns of S are
// independent, so a small batch is split over more CTAs by narrower column tiles.
//
// Bound by the state's two passes: 256 sequences of 32 heads, 1.08 GB, in 156 us, 6.9 TB/s; a
// launch's latency below some hundred heads.
#include "linattn.cuh"

namespace gdr {
namespace linattn {
namespace {

template <typename T, int DK, int DVT>
__global__ void __launch_bounds__(DK / 16 * (DVT / 4))
linattn_step_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
                    const float *__restrict__ log_decay, float *__restrict__ S, T *__restrict__ o,
                    int H, int qg, int kg, int vg, int dv, float scale, int64_t qs, int64_t ks,
                    int64_t vs) {
    constexpr int RG = DK / 16, TPR = DVT / 4, NT = RG * TPR;
    __shared__ float sq[DK], sk[DK];
    __shared__ float4 part[RG][TPR];
    const int slices = dv / DVT;
    const int64_t nh = blockIdx.x / slices;
    const int64_t n = nh / H;
    const int h = (int)(nh % H), c0 = (int)(blockIdx.x % slices) * DVT;
    const int tid = threadIdx.x, cg = tid % TPR, rg = tid / TPR;
    float *Sp = S + nh * DK * dv + c0 + 4 * cg;
    float4 s[16];
#pragma unroll
    for (int m = 0; m < 16; ++m)
        s[m] = __ldcs(reinterpret_cast<const float4 *>(Sp + (int64_t)(rg + m * RG) * dv));
    const T *qp = q + n * qs + (h / qg) * DK, *kp = k + n * ks + (h / kg) * DK;
    for (int i = tid; i < DK; i += NT) {
        sq[i] = scale * to_f32(qp[i]);
        sk[i] = to_f32(kp[i]);
    }
    const T *vp = v + n * vs + (int64_t)(h / vg) * dv + c0 + 4 * cg;
    const float4 vv = make_float4(to_f32(vp[0]), to_f32(vp[1]), to_f32(vp[2]), to_f32(vp[3]));
    const float lam = expf(log_decay[h]);
    __syncthreads();
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int m = 0; m < 16; ++m) {
        const int r = rg + m * RG;
        const float kr = sk[r], qr = sq[r];
        float4 x;
        x.x = fmaf(lam, s[m].x, kr * vv.x);
        x.y = fmaf(lam, s[m].y, kr * vv.y);
        x.z = fmaf(lam, s[m].z, kr * vv.z);
        x.w = fmaf(lam, s[m].w, kr * vv.w);
        __stcs(reinterpret_cast<float4 *>(Sp + (int64_t)r * dv), x);
        acc.x = fmaf(qr, x.x, acc.x);
        acc.y = fmaf(qr, x.y, acc.y);
        acc.z = fmaf(qr, x.z, acc.z);
        acc.w = fmaf(qr, x.w, acc.w);
    }
    part[rg][cg] = acc;
    __syncthreads();
    if (rg == 0) {
        float4 sum = part[0][cg];
#pragma unroll
        for (int r = 1; r < RG; ++r) {
            const float4 x = part[r][cg];
            sum.x += x.x;
            sum.y += x.y;
            sum.z += x.z;
            sum.w += x.w;
        }
        T *op = o + nh * dv + c0 + 4 * cg;
        op[0] = from_f32<T>(sum.x);
        op[1] = from_f32<T>(sum.y);
        op[2] = from_f32<T>(sum.z);
        op[3] = from_f32<T>(sum.w);
    }
}

template <typename T, int DK, int DVT>
int launch_tile(const void *q, const void *k, const void *v, const float *ld, float *S, void *o,
                int64_t N, int H, int qg, int kg, int vg, int dv, float scale, int64_t qs,
                int64_t ks, int64_t vs, cudaStream_t stream) {
    linattn_step_kernel<T, DK, DVT>
        <<<(unsigned)(N * H * (dv / DVT)), DK / 16 * (DVT / 4), 0, stream>>>(
            (const T *)q, (const T *)k, (const T *)v, ld, S, (T *)o, H, qg, kg, vg, dv, scale, qs,
            ks, vs);
    return cuda_status(cudaGetLastError());
}

}  // namespace

int launch_step(const void *q, const void *k, const void *v, const float *log_decay, float *S,
                void *o, int64_t N, int H, int qg, int kg, int vg, int dk, int dv, int dtype,
                float scale, int64_t qs, int64_t ks, int64_t vs, cudaStream_t stream) {
    // Wide tiles once they alone give every SM work (152 SMs). d_k = d_v = 128, 32 and 128
    // columns: N H = 16 10.6 and 11.4 us, 64 10.4 and 11.8, 256 14.9 and 14.5, 1024 31.3 and 28.8.
    const bool wide = dv % 128 == 0 && N * H * (dv / 128) >= 152;
#define GDR_STEP(T, DK, DVT)                                                                        \
    return launch_tile<T, DK, DVT>(q, k, v, log_decay, S, o, N, H, qg, kg, vg, dv, scale, qs, ks, vs, stream)
#define GDR_STEP_T(T)                                                                               \
    if (dk == 128) {                                                                                \
        if (wide) GDR_STEP(T, 128, 128);                                                            \
        GDR_STEP(T, 128, 32);                                                                       \
    }                                                                                               \
    if (wide) GDR_STEP(T, 64, 128);                                                                 \
    GDR_STEP(T, 64, 32)
    if (dtype == GDR_BF16) {
        GDR_STEP_T(__nv_bfloat16);
    }
    GDR_STEP_T(float);
#undef GDR_STEP_T
#undef GDR_STEP
}

}  // namespace linattn
}  // namespace gdr
