// linattn_exact.cu -- the mix of linear attention (linattn.cuh) in fp32 arithmetic, for fp32
// inputs. A bf16 call without tokens comes here too: it only hands on its states, which are
// fp32, and no row of any type is read or written. And the sum of gradients of shared heads.
//
// One CTA per (segment, head, 64 columns of z) walks its segment in chunks of C tokens. The
// state lives in registers (thread (ty, tx): rows ty R .. + R - 1, columns 4 tx .. + 3) and
// is copied to shared memory once per chunk for the product x E.
//
// Bound by its fp32 multiply-adds and the shared-memory reads that feed them: a chunk of 64
// tokens with d_x = 128 is 3.7 MFLOP and takes 9 us.
#include "linattn.cuh"

namespace gdr {
namespace linattn {
namespace {

constexpr int NZ = 64, kThreads = 256;

template <int DX> struct Cfg {
    static constexpr int C = DX > 128 ? 32 : 64;   // tokens per chunk
    static constexpr int LX = DX + 4;              // row pitches in floats: 16-byte rows whose
    static constexpr int LZ = NZ + 4;              // float4 columns fall on different banks
    static constexpr int LP = C + 4;
    static constexpr size_t floats = 2 * C * LX + C * LZ + DX * LZ + C * LP + C + 1;
};

__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ void store4(float *p, float4 x) { *reinterpret_cast<float4 *>(p) = x; }
__device__ __forceinline__ void store4(__nv_bfloat16 *p, float4 x) {
    __nv_bfloat162 lo = __floats2bfloat162_rn(x.x, x.y), hi = __floats2bfloat162_rn(x.z, x.w);
    uint2 u;
    u.x = *reinterpret_cast<uint32_t *>(&lo);
    u.y = *reinterpret_cast<uint32_t *>(&hi);
    *reinterpret_cast<uint2 *>(p) = u;
}
__device__ __forceinline__ void fma4(float4 &a, float s, const float4 &b) {
    a.x = fmaf(s, b.x, a.x);
    a.y = fmaf(s, b.y, a.y);
    a.z = fmaf(s, b.z, a.z);
    a.w = fmaf(s, b.w, a.w);
}

// kOut: the mix itself; otherwise only the segment's own sum R.
template <int DX, bool kOut>
__global__ void __launch_bounds__(kThreads, 1) mix_exact_kernel(const Plan p, const Mix m) {
    constexpr int C = Cfg<DX>::C, LX = Cfg<DX>::LX, LZ = Cfg<DX>::LZ, LP = Cfg<DX>::LP;
    constexpr int R = DX / 16;          // state rows per thread
    constexpr int RT = C / 16;          // chunk rows per thread
    extern __shared__ __align__(16) float smem[];
    float *sX = smem, *sY = sX + C * LX, *sZ = sY + C * LX, *sE = sZ + C * LZ, *sP = sE + DX * LZ,
          *pw = sP + C * LP;  // pw[n] = lam^n, n <= C
    __shared__ Segment found;

    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int slices = m.dz / NZ;
    const int64_t block = blockIdx.x;
    const int slice = (int)(block % slices);
    const bool bad = !locate(p, block / slices, kOut ? 0 : 1 + m.backward, &found, (int *)smem);
    const Segment s = found;
    const int h = s.h;
    if (block == 0 && tid == 0 && p.first) p.status[0] = bad ? GDR_ERR_BAD_SEQLENS : GDR_OK;
    if (bad || s.seq < 0) return;

    const float l2 = log2_decay(p.log_decay[h]);
    for (int i = tid; i <= C; i += kThreads) pw[i] = decay_pow(l2, (float)i);

    float4 E[R];
#pragma unroll
    for (int a = 0; a < R; ++a) E[a] = make_float4(0.f, 0.f, 0.f, 0.f);
    const int z0 = slice * NZ + 4 * tx;  // this thread's first column of z
    const int64_t mat = (int64_t)m.dx * m.dz;
    auto add_state = [&](const float *S, float w) {
#pragma unroll
        for (int a = 0; a < R; ++a) {
            float4 v;
            if (m.turned)
                v = make_float4(S[state_at(m, ty * R + a, z0)], S[state_at(m, ty * R + a, z0 + 1)],
                                S[state_at(m, ty * R + a, z0 + 2)], S[state_at(m, ty * R + a, z0 + 3)]);
            else
                v = load4(S + state_at(m, ty * R + a, z0));
            fma4(E[a], w, v);
        }
    };
    if (kOut) {
        if (m.start) {
            const int64_t dist = m.backward ? s.behind : (int64_t)s.f * p.seg;
            add_state(m.start + ((int64_t)s.seq * p.H + h) * mat, decay_pow(l2, (float)dist));
        }
        for (int g = m.backward ? s.f : 0; m.R && g < (m.backward ? s.n - 1 : s.f); ++g) {
            const int apart = m.backward ? g - s.f : s.f - 1 - g;
            add_state(m.R + ((s.sum0 + g) * p.H + h) * mat, decay_pow(l2, (float)(apart * p.seg)));
        }
    }

    const float *x = (const float *)m.x + (int64_t)(h / m.xg) * m.dx;
    const float *y = (const float *)m.y + (int64_t)(h / m.yg) * m.dx;
    const float *z = (const float *)m.z + (int64_t)(h / m.zg) * m.dz + slice * NZ;
    const int chunks = (int)((s.tokens + C - 1) / C);
    for (int cc = 0; cc < chunks; ++cc) {
        const int c = m.backward ? chunks - 1 - cc : cc;
        const int64_t t0 = s.begin + (int64_t)c * C;
        const int64_t rest = s.begin + s.tokens - t0;
        const int n = (int)(rest < C ? rest : C);
        __syncthreads();  // the tiles of the chunk before have been used
        for (int e = tid; e < C * (DX / 4); e += kThreads) {
            const int r = e / (DX / 4), j = 4 * (e % (DX / 4));
            const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
            if (kOut) store4(sX + r * LX + j, r < n ? load4(x + (t0 + r) * m.xs + j) : zero);
            store4(sY + r * LX + j, r < n ? load4(y + (t0 + r) * m.ys + j) : zero);
        }
        for (int e = tid; e < C * (NZ / 4); e += kThreads) {
            const int r = e / (NZ / 4), j = 4 * (e % (NZ / 4));
            store4(sZ + r * LZ + j, r < n ? load4(z + (t0 + r) * m.zs + j) : make_float4(0.f, 0.f, 0.f, 0.f));
        }
        if (kOut) {
#pragma unroll
            for (int a = 0; a < R; ++a) store4(sE + (ty * R + a) * LZ + 4 * tx, E[a]);
            __syncthreads();
            // P_ri = s_intra M_ri lam^|r-i| x_r.y_i: rows ty + 16 a, columns tx + 16 b
            float acc[RT][RT];
#pragma unroll
            for (int a = 0; a < RT; ++a)
#pragma unroll
                for (int b = 0; b < RT; ++b) acc[a][b] = 0.f;
            for (int k = 0; k < DX; k += 4) {
                float4 xv[RT], yv[RT];
#pragma unroll
                for (int a = 0; a < RT; ++a) xv[a] = load4(sX + (ty + 16 * a) * LX + k);
#pragma unroll
                for (int b = 0; b < RT; ++b) yv[b] = load4(sY + (tx + 16 * b) * LX + k);
#pragma unroll
                for (int a = 0; a < RT; ++a)
#pragma unroll
                    for (int b = 0; b < RT; ++b) {
                        acc[a][b] = fmaf(xv[a].x, yv[b].x, acc[a][b]);
                        acc[a][b] = fmaf(xv[a].y, yv[b].y, acc[a][b]);
                        acc[a][b] = fmaf(xv[a].z, yv[b].z, acc[a][b]);
                        acc[a][b] = fmaf(xv[a].w, yv[b].w, acc[a][b]);
                    }
            }
#pragma unroll
            for (int a = 0; a < RT; ++a)
#pragma unroll
                for (int b = 0; b < RT; ++b) {
                    const int r = ty + 16 * a, i = tx + 16 * b;
                    const bool keep = m.backward ? i >= r && i < n : i <= r;
                    sP[r * LP + i] = keep ? m.s_intra * pw[m.backward ? i - r : r - i] * acc[a][b] : 0.f;
                }
            __syncthreads();
            // out rows ty + 16 a, columns 4 tx .. + 3
            float4 o[RT];
#pragma unroll
            for (int a = 0; a < RT; ++a) o[a] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = 0; k < DX; k += 4) {
                float4 ev[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) ev[j] = load4(sE + (k + j) * LZ + 4 * tx);
#pragma unroll
                for (int a = 0; a < RT; ++a) {
                    const float4 xv = load4(sX + (ty + 16 * a) * LX + k);
                    fma4(o[a], xv.x, ev[0]);
                    fma4(o[a], xv.y, ev[1]);
                    fma4(o[a], xv.z, ev[2]);
                    fma4(o[a], xv.w, ev[3]);
                }
            }
#pragma unroll
            for (int a = 0; a < RT; ++a) {
                const int r = ty + 16 * a;
                const float w = r < n ? m.s_inter * pw[m.backward ? n - 1 - r : r + 1] : 0.f;
                o[a] = make_float4(w * o[a].x, w * o[a].y, w * o[a].z, w * o[a].w);
            }
            for (int i = 0; i < C; i += 4) {
                float4 zv[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) zv[j] = load4(sZ + (i + j) * LZ + 4 * tx);
#pragma unroll
                for (int a = 0; a < RT; ++a) {
                    const float4 pv = load4(sP + (ty + 16 * a) * LP + i);
                    fma4(o[a], pv.x, zv[0]);
                    fma4(o[a], pv.y, zv[1]);
                    fma4(o[a], pv.z, zv[2]);
                    fma4(o[a], pv.w, zv[3]);
                }
            }
#pragma unroll
            for (int a = 0; a < RT; ++a) {
                const int r = ty + 16 * a;
                if (r >= n) continue;
                const int64_t at = ((t0 + r) * p.H + h) * m.dz + z0;
                store4((float *)m.out + at, o[a]);
            }
        } else {
            __syncthreads();
        }
        // E <- lam^n E + s_state sum_r w_upd(r) y_r z_r^T
        const float wn = pw[n];
#pragma unroll
        for (int a = 0; a < R; ++a) E[a] = make_float4(wn * E[a].x, wn * E[a].y, wn * E[a].z, wn * E[a].w);
        for (int r = 0; r < n; ++r) {
            const float w = m.s_state * pw[m.backward ? r + 1 : n - 1 - r];
            const float4 zv = load4(sZ + r * LZ + 4 * tx);
            const float4 zw = make_float4(w * zv.x, w * zv.y, w * zv.z, w * zv.w);
#pragma unroll
            for (int a = 0; a < R; a += 4) {
                const float4 yv = load4(sY + r * LX + ty * R + a);
                fma4(E[a], yv.x, zw);
                fma4(E[a + 1], yv.y, zw);
                fma4(E[a + 2], yv.z, zw);
                fma4(E[a + 3], yv.w, zw);
            }
        }
    }

    float *to = nullptr;
    if (!kOut) to = m.R_out + ((s.sum0 + s.f - m.backward) * p.H + h) * mat;
    else if (m.end && s.f == (m.backward ? 0 : s.n - 1)) to = m.end + ((int64_t)s.seq * p.H + h) * mat;
    if (!to) return;
#pragma unroll
    for (int a = 0; a < R; ++a) {
        if (m.turned) {
            to[state_at(m, ty * R + a, z0)] = E[a].x;
            to[state_at(m, ty * R + a, z0 + 1)] = E[a].y;
            to[state_at(m, ty * R + a, z0 + 2)] = E[a].z;
            to[state_at(m, ty * R + a, z0 + 3)] = E[a].w;
        } else {
            store4(to + state_at(m, ty * R + a, z0), E[a]);
        }
    }
}

template <int DX, bool kOut>
int launch_one(const Plan &p, const Mix &m, cudaStream_t stream) {
    constexpr size_t bytes = Cfg<DX>::floats * sizeof(float);
    static_assert(bytes <= 232448 - 512, "shared memory");
    if (cudaFuncSetAttribute(mix_exact_kernel<DX, kOut>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)bytes) != cudaSuccess)
        return GDR_ERR_CUDA;
    const int64_t blocks = (kOut ? p.units : p.handing) * (m.dz / NZ);
    mix_exact_kernel<DX, kOut><<<(unsigned)blocks, kThreads, bytes, stream>>>(p, m);
    return cuda_status(cudaGetLastError());
}

int launch_of(const Plan &p, const Mix &m, cudaStream_t stream) {
    const bool out = m.out != nullptr;
    switch (m.dx) {
        case 64: return out ? launch_one<64, true>(p, m, stream) : launch_one<64, false>(p, m, stream);
        case 128: return out ? launch_one<128, true>(p, m, stream) : launch_one<128, false>(p, m, stream);
        case 256: return launch_one<256, true>(p, m, stream);  // (sums have rows of d_k, 128 at most)
    }
    return GDR_ERR_UNSUPPORTED;
}

struct Shares {
    Share v[3];
};
// Bound by its reads: g fp32 per value written, 16 bytes at a time.
template <typename T> __global__ void __launch_bounds__(256) share_kernel(const Plan p, const Shares shares) {
    const Share &m = shares.v[blockIdx.y];
    if (p.status[0] != GDR_OK) return;
    const int64_t rows = p.cu_seqlens ? p.cu_seqlens[p.num_seqs] : p.total_tokens;
    const int shift = 29 - __clz(m.d);  // d / 4 quads, a power of two
    const int64_t total = rows * m.heads << shift;
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total; e += (int64_t)gridDim.x * 256) {
        const int j = (int)(e & ((1 << shift) - 1)) * 4;
        const int64_t rh = e >> shift;  // row * heads + head: its g parts are in[rh g ..]
        const float *in = m.in + rh * m.g * m.d + j;
        float4 sum = load4(in);
        for (int i = 1; i < m.g; ++i) fma4(sum, 1.f, load4(in + i * m.d));
        store4((T *)m.out + rh * m.d + j, sum);
    }
}

// Bound by reading the offsets once.
__global__ void __launch_bounds__(256) check_kernel(const Plan p) {
    for (int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x; n < p.num_seqs; n += (int64_t)gridDim.x * 256) {
        const int a = p.cu_seqlens[n], b = p.cu_seqlens[n + 1];
        if (b < a || a < 0 || b > p.total_tokens || (n == 0 && a != 0)) p.status[0] = GDR_ERR_BAD_SEQLENS;
    }
}

}  // namespace

int launch_check(const Plan &p, cudaStream_t stream) {
    static_assert(GDR_OK == 0, "");
    if (cudaMemsetAsync(p.status, 0, sizeof(int32_t), stream) != cudaSuccess) return GDR_ERR_CUDA;
    const int64_t blocks = (p.num_seqs + 255) / 256;
    check_kernel<<<(unsigned)(blocks < 152 * 8 ? blocks : 152 * 8), 256, 0, stream>>>(p);
    return cuda_status(cudaGetLastError());
}

int launch_mix_exact(const Plan &p, const Mix *mixes, int count, cudaStream_t stream) {
    for (int i = 0; i < count; ++i) {
        Plan pi = p;
        pi.first = p.first && i == 0;
        const int st = launch_of(pi, mixes[i], stream);
        if (st != GDR_OK) return st;
    }
    return GDR_OK;
}

int launch_share(const Plan &p, const Share *shares, int count, int dtype, cudaStream_t stream) {
    Shares all = {};
    int64_t quads = 0;
    for (int i = 0; i < count; ++i) {
        all.v[i] = shares[i];
        const int64_t q = p.total_tokens * shares[i].heads * (shares[i].d / 4);
        if (q > quads) quads = q;
    }
    const int64_t blocks = (quads + 255) / 256;
    const dim3 grid((unsigned)(blocks < 152 * 16 ? blocks : 152 * 16), (unsigned)count);
    if (dtype == GDR_BF16) share_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(p, all);
    else share_kernel<float><<<grid, 256, 0, stream>>>(p, all);
    return cuda_status(cudaGetLastError());
}

}  // namespace linattn
}  // namespace gdr
