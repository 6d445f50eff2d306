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
#include "f32x2.cuh"
#include "internal.h"

namespace gdr {
namespace {

constexpr int kSms = 152;

// VEC consecutive entries (VEC divides D) in 32-bit words, read 16 bytes at a time where they
// are that many; a bf16 unpacks by a shift or a mask, a pair packs in one conversion.
template <typename T, int VEC> struct alignas(sizeof(T) * VEC < 16 ? sizeof(T) * VEC : 16) Pack {
    uint32_t w[sizeof(T) * VEC / 4];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (uint32_t &x : w) x = 0;
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
    __device__ __forceinline__ void set(int i, float a, float b) {  // entries i, i + 1 (i even)
        if constexpr (sizeof(T) == 4) {
            w[i] = __float_as_uint(a);
            if (VEC > 1) w[i + 1 < VEC ? i + 1 : i] = __float_as_uint(VEC > 1 ? b : a);
        } else {
            const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
            w[i / 2] = reinterpret_cast<const uint32_t &>(v);
        }
    }
};
template <> struct Pack<__nv_bfloat16, 1> {  // (odd widths)
    __nv_bfloat16 v;
    __device__ __forceinline__ void zero() { v = __float2bfloat16_rn(0.f); }
    __device__ __forceinline__ float get(int) const { return __bfloat162float(v); }
    __device__ __forceinline__ void set(int, float a, float) { v = __float2bfloat16_rn(a); }
};
template <typename T, int VEC> __device__ __forceinline__ void pack_all(Pack<T, VEC> &p, const float *x) {
#pragma unroll
    for (int i = 0; i < VEC; i += 2) p.set(i, x[i], x[VEC > 1 ? i + 1 : i]);
}

// A thread's PER entries of a row as they are in memory: VEC at a time, blockDim.x VEC apart.
// Entries behind the row's end (and whole rows behind the last, D = 0) are zero.
template <typename T, int VEC, int PER> struct Raw {
    Pack<T, VEC> p[PER / VEC];
    __device__ __forceinline__ void load(const T *row, int D) {
#pragma unroll
        for (int j = 0; j < PER / VEC; ++j) {
            const int e = (threadIdx.x + blockDim.x * j) * VEC;
            if (e < D) p[j] = *reinterpret_cast<const Pack<T, VEC> *>(row + e);
            else p[j].zero();
        }
    }
    __device__ __forceinline__ float operator[](int i) const { return p[i / VEC].get(i % VEC); }
    __device__ __forceinline__ float2 two(int i) const { return make_float2((*this)[i], (*this)[i + 1]); }
};

template <typename T, int VEC, int PER>
__device__ __forceinline__ void store_row(T *row, int D, const float (&x)[PER]) {
#pragma unroll
    for (int j = 0; j < PER / VEC; ++j) {
        const int e = (threadIdx.x + blockDim.x * j) * VEC;
        Pack<T, VEC> a;
        pack_all(a, x + j * VEC);
        if (e < D) *reinterpret_cast<Pack<T, VEC> *>(row + e) = a;
    }
}

// A weight of a thread's entries, read where it is used (it stays in the first-level cache).
template <int VEC> struct Weight {
    float v[VEC];
};
template <int VEC> __device__ __forceinline__ Weight<VEC> weight_of(const float *w, int j, int D) {
    Weight<VEC> a;
    const int e = (threadIdx.x + blockDim.x * j) * VEC;
    Pack<float, VEC> p;
#pragma unroll
    for (int i = 0; i < VEC; ++i) p.w[i] = 0x3f800000u;
    if (w && e < D) p = *reinterpret_cast<const Pack<float, VEC> *>(w + e);
#pragma unroll
    for (int i = 0; i < VEC; ++i) a.v[i] = p.get(i);
    return a;
}

// Sums of K values (1 or 3) over the blockDim.x threads of a row: within the warp, then over the
// row's warps (at most 16) by every warp for itself. Of three values each half of the warp goes
// on with its own after an exchange: 6 shuffles instead of 15. `buf` has 2 x 16 x 3 floats. One
// barrier per sum is enough where every call takes the other half than the call before it, in a
// loop's next round too: a warp then comes back to a half only past the barrier of the sum between,
// which all warps reach after they have read that half. So the half is kept here, in `turn`, of
// which a block has one (0 at first) for all its sums.
constexpr int kBufBytes = 2 * 16 * 3 * (int)sizeof(float);
template <int K> __device__ __forceinline__ void row_sum(float (&s)[K], float *buf, int &turn) {
    static_assert(K == 1 || K == 3, "");
    const unsigned all = 0xffffffffu;
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    float v = s[0];
    if (K == 3) {  // lanes 0-7 go on with value 0, 16-23 with 1, the others with 2
        const bool high = lane & 16, last = lane & 8;
        const float x = (high ? s[1] : s[0]) + __shfl_xor_sync(all, high ? s[0] : s[1], 16);
        const float y = s[2] + __shfl_xor_sync(all, s[2], 16);
        v = (last ? y : x) + __shfl_xor_sync(all, last ? x : y, 8);
    }
#pragma unroll
    for (int off = K == 3 ? 4 : 16; off > 0; off >>= 1) v += __shfl_xor_sync(all, v, off);
    if (warps > 1) {
        float *row = buf + turn * 48 + threadIdx.y * warps * K;
        turn ^= 1;
        const int which = K == 3 ? (lane & 8 ? 2 : lane >> 4) : 0;
        if ((lane & (K == 3 ? 7 : 31)) == 0) row[which * warps + (threadIdx.x >> 5)] = v;
        __syncthreads();
        const int w = lane & 7;
        v = w < warps ? row[which * warps + w] : 0.f;
        if (w + 8 < warps) v += row[which * warps + w + 8];
#pragma unroll
        for (int off = 4; off > 0; off >>= 1) v += __shfl_xor_sync(all, v, off);
    }
    s[0] = K == 3 ? __shfl_sync(all, v, 0) : v;
    if (K == 3) {
        s[K / 2] = __shfl_sync(all, v, 16);
        s[K - 1] = __shfl_sync(all, v, 8);
    }
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// sigmoid by the hardware's exponential and reciprocal (a few units in the last place).
__device__ __forceinline__ float sigmoid(float g) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}
// The gate's function of N entries; one branch for all.
template <int N> __device__ __forceinline__ void gate_of(int act, const float (&g)[N], float (&a)[N]) {
    if (act == GDR_GATE_IDENTITY) {
#pragma unroll
        for (int e = 0; e < N; ++e) a[e] = g[e];
    } else if (act == GDR_GATE_SILU) {
#pragma unroll
        for (int e = 0; e < N; ++e) a[e] = g[e] * sigmoid(g[e]);
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) a[e] = sigmoid(g[e]);
    }
}
// The same of two entries with the derivative.
__device__ __forceinline__ void gate_both(int act, float2 g, float2 &a, float2 &da) {
    if (act == GDR_GATE_IDENTITY) {
        a = g;
        da = both(1.f);
        return;
    }
    const float2 s = make_float2(sigmoid(g.x), sigmoid(g.y)), rest = fma2(s, both(-1.f), both(1.f));
    if (act == GDR_GATE_SILU) {
        a = mul2(g, s);
        da = fma2(a, rest, s);
    } else {
        a = s;
        da = mul2(s, rest);
    }
}

struct NormParams {
    int64_t rows;
    int D;
    int post, pre, act;
    int64_t gate_stride;  // 0: one row for all
    float s, eps, inv_D;
    const float *w_post, *w_pre;
};

// One row per blockDim.x threads, 16 entries each where the row is wide enough: few threads
// with many loads in flight each, so that the two sums over a row cost little. Bound by memory:
// 16384 x 2048 bf16, 336 MB, in 55 us, 6.1 TB/s.
template <typename T, typename TX, int VEC, int PER>
__global__ void __launch_bounds__(512)
block_norm_fwd_kernel(const NormParams p, const TX *x, const T *y, const T *gate, TX *x_out, T *h) {
    __shared__ float buf[kBufBytes / sizeof(float)];
    int turn = 0;
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int D = row < p.rows ? p.D : 0;  // a row behind the last loads and stores nothing
    const int64_t at = row * p.D;
    Raw<TX, VEC, PER> xr;
    float v[PER];
    xr.load(x + at, D);
    if (y) {
        Raw<T, VEC, PER> yr, gr;
        yr.load(y + at, D);
        if (gate) gr.load(gate + row * p.gate_stride, D);
        float r = 1.f;
        if (p.post) {
            float ss[1] = {0.f};
#pragma unroll
            for (int i = 0; i < PER; ++i) ss[0] = fmaf(yr[i], yr[i], ss[0]);
            row_sum(ss, buf, turn);
            r = rsqrtf(ss[0] * p.inv_D + p.eps);
        }
        const float *w = p.post ? p.w_post : nullptr;
#pragma unroll
        for (int j = 0; j < PER / VEC; ++j) {
            const Weight<VEC> wj = weight_of<VEC>(w, j, D);
            float a[VEC], g[VEC];
            if (gate) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) g[e] = gr[j * VEC + e];
                gate_of(p.act, g, a);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) a[e] = 1.f;
            }
            const float rs = r * p.s;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int i = j * VEC + e;
                v[i] = fmaf(yr[i] * a[e], rs * wj.v[e], xr[i]);
            }
        }
        store_row<TX, VEC>(x_out + at, D, v);
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) v[i] = xr[i];
    }
    if (!h) return;
    float ss[1] = {0.f};
#pragma unroll
    for (int i = 0; i < PER; ++i) ss[0] = fmaf(v[i], v[i], ss[0]);
    row_sum(ss, buf, turn);
    const float r = rsqrtf(ss[0] * p.inv_D + p.eps);
#pragma unroll
    for (int j = 0; j < PER / VEC; ++j) {
        const Weight<VEC> wj = weight_of<VEC>(p.w_pre, j, D);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[j * VEC + e] *= r * wj.v[e];
    }
    store_row<T, VEC>(h + at, D, v);
}

__device__ __forceinline__ uint32_t smem_at(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

// A thread's 8 entries of a row on their way to shared memory, to slots that it alone uses (no
// barrier), 16 bytes of every thread side by side; zeros behind the row's end.
template <typename T> __device__ __forceinline__ void fetch8(uint32_t slot, const T *from, bool live, int threads) {
#pragma unroll
    for (int u = 0; u < (int)sizeof(T) / 2; ++u)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(slot + u * 16 * threads),
                     "l"((const char *)from + 16 * u), "r"(live ? 16 : 0)
                     : "memory");
}
template <typename T> __device__ __forceinline__ void read8(Pack<T, 8> &p, const char *slot, int threads) {
#pragma unroll
    for (int u = 0; u < (int)sizeof(T) / 2; ++u) {
        const uint4 x = *reinterpret_cast<const uint4 *>(slot + u * 16 * threads);
        p.w[4 * u] = x.x;
        p.w[4 * u + 1] = x.y;
        p.w[4 * u + 2] = x.z;
        p.w[4 * u + 3] = x.w;
    }
}

// What a block of the backward kernel keeps of its rows' inputs.
template <typename T, typename TX, int PER> __host__ __device__ constexpr int row_bytes() {
    return PER * (2 * (int)sizeof(TX) + 3 * (int)sizeof(T));
}
template <typename T, int VEC, int PER> __host__ __device__ constexpr bool fetches_ahead() { return PER == 8 && VEC == 8; }

// Sums over this block's rows go to part[which][blockIdx.x * blockDim.y + threadIdx.y][D]. The
// next row's inputs are on their way to shared memory while a row is worked on (in registers
// they would halve the warps, and the instructions, 89 per thread and entry, need the warps).
// 16384 x 2048 bf16, 537 MB, takes 127 us with the column sums, 4.2 TB/s, with two thirds of the
// issue slots and half of DRAM in use: the row's sums and the reads from shared memory leave
// gaps that 24 warps on an SM do not fill. With 80 registers 16 bytes are spilled (64 would take
// a fourth block and spill more: 151 us, 130 at that time). In fp32 shared memory
// holds 16 warps on an SM: 8192 x 2048, 537 MB, in 180 us, 3.0 TB/s.
// Rows wider than 4096 keep their columns' sums in shared memory instead. One gate row for all:
// with A = the sum over rows of s dx' n, dw_post is act(gate) A and dgate is act'(gate) w_post A.
template <typename T, typename TX, int VEC, int PER, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS > 256 ? 1 : (PER <= 8 ? 3 : 2))
block_norm_bwd_kernel(const NormParams p, const TX *dx_out, const T *dh, const TX *x, const T *y,
                      const T *gate, TX *dx, T *dy, T *dgate, float *part_post, float *part_pre,
                      float *part_gate) {
    constexpr bool kWide = PER > 8, kAhead = fetches_ahead<T, VEC, PER>();
    __shared__ float buf[kBufBytes / sizeof(float)];
    int turn = 0;
    extern __shared__ __align__(16) char dynamic[];
    float *wide = reinterpret_cast<float *>(dynamic);  // [2][D], each thread its own columns
    constexpr int kSums = kWide ? 1 : PER / 2;
    float2 a_post[kSums], a_pre[kSums];
#pragma unroll
    for (int i = 0; i < kSums; ++i) a_post[i] = a_pre[i] = both(0.f);
    if (kWide) {
        for (int e = threadIdx.x; e < 2 * p.D; e += blockDim.x) wide[e] = 0.f;
        __syncthreads();
    }
    auto column = [&](int i) { return (threadIdx.x + blockDim.x * (i / VEC)) * VEC + i % VEC; };
    auto add = [&](float2 (&a)[kSums], int which, int i, float2 x) {  // entries i, i + 1
        if (!kWide) {
            a[kWide ? 0 : i / 2] = fma2(x, both(1.f), a[kWide ? 0 : i / 2]);
        } else {
            if (column(i) < p.D) wide[which * p.D + column(i)] += x.x;
            if (column(i + 1) < p.D) wide[which * p.D + column(i + 1)] += x.y;
        }
    };
    const bool one_gate = gate && !p.gate_stride;
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    const int64_t rounds = (p.rows + step - 1) / step;  // the same for every thread: barriers inside
    int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int threads = blockDim.x * blockDim.y, id = threadIdx.y * blockDim.x + threadIdx.x;
    // a round's inputs, this thread's slots: dx_out, x, then dh, y, gate
    constexpr int kX = 8 * (int)sizeof(TX), kT = 8 * (int)sizeof(T), kRound = 2 * kX + 3 * kT;
    char *const mine_at = dynamic + 16 * id;
    const int e8 = threadIdx.x * 8;
    auto fetch = [&](int64_t round, int64_t at_row) {
        if constexpr (kAhead) {
            const bool live = at_row < p.rows && e8 < p.D;
            const int64_t at = live ? at_row * p.D + e8 : 0;
            const uint32_t to = smem_at(mine_at) + (round & 1 ? kRound * threads : 0);
            if (dx_out) fetch8(to, dx_out + at, live, threads);
            if (dh) {
                fetch8(to + kX * threads, x + at, live, threads);
                fetch8(to + 2 * kX * threads, dh + at, live, threads);
            }
            if (y) fetch8(to + (2 * kX + kT) * threads, y + at, live, threads);
            if (gate)
                fetch8(to + (2 * kX + 2 * kT) * threads, gate + (p.gate_stride ? at : (live ? e8 : 0)), live, threads);
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    };
    fetch(0, row);
    for (int64_t round = 0; round < rounds; ++round, row += step) {
        const int D = row < p.rows ? p.D : 0;
        const int64_t at = row * p.D;
        if (kAhead) {
            if (round + 1 < rounds) {
                fetch(round + 1, row + step);
                asm volatile("cp.async.wait_group 1;" ::: "memory");
            } else {
                asm volatile("cp.async.wait_group 0;" ::: "memory");
            }
        }
        const char *const here = mine_at + (round & 1 ? kRound * threads : 0);
        Raw<TX, VEC, PER> xr, dr;
        Raw<T, VEC, PER> hr, yr, gr;
        if constexpr (kAhead) {  // (dx_out and gate are read where they are used)
            if (dh) {
                read8(xr.p[0], here + kX * threads, threads);
                read8(hr.p[0], here + 2 * kX * threads, threads);
            }
            if (y) read8(yr.p[0], here + (2 * kX + kT) * threads, threads);
        } else {
            dr.load(dx_out + at, dx_out ? D : 0);
            xr.load(x + at, dh ? D : 0);
            hr.load(dh + at, dh ? D : 0);
            yr.load(y + at, y ? D : 0);
            gr.load(gate + row * p.gate_stride, gate ? D : 0);
        }
        // entries in pairs throughout
        float2 dv[PER / 2];
        float2 xx = both(0.f), hx = xx, yy = xx;
        if (dh) {
#pragma unroll
            for (int j = 0; j < PER / VEC; ++j) {
                const Weight<VEC> w = weight_of<VEC>(p.w_pre, j, D);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const int i = j * VEC + e;
                    (i & 1 ? dv[i / 2].y : dv[i / 2].x) = w.v[e];
                }
            }
#pragma unroll
            for (int i = 0; i < PER; i += 2) {
                const float2 xv = xr.two(i);
                dv[i / 2] = mul2(dv[i / 2], hr.two(i));
                xx = fma2(xv, xv, xx);
                hx = fma2(dv[i / 2], xv, hx);
            }
        }
        if (p.post) {
#pragma unroll
            for (int i = 0; i < PER; i += 2) yy = fma2(yr.two(i), yr.two(i), yy);
        }
        float sums[3] = {xx.x + xx.y, hx.x + hx.y, yy.x + yy.y};
        if (dh || p.post) row_sum(sums, buf, turn);
        if constexpr (kAhead)
            if (dx_out) read8(dr.p[0], here, threads);
        if (dh) {
            const float r = rsqrtf(sums[0] * p.inv_D + p.eps), m = r * r * (sums[1] * p.inv_D);
#pragma unroll
            for (int i = 0; i < PER; i += 2) {
                const float2 xv = xr.two(i);
                add(a_pre, 1, i, mul2(hr.two(i), mul2(xv, both(r))));
                dv[i / 2] = fma2(both(r), fma2(xv, both(-m), dv[i / 2]), dx_out ? dr.two(i) : both(0.f));
            }
        } else {
#pragma unroll
            for (int i = 0; i < PER; i += 2) dv[i / 2] = dr.two(i);
        }
        store_row<TX, VEC>(dx + at, D, reinterpret_cast<const float(&)[PER]>(dv));
        if (!y) continue;
        const float r = p.post ? rsqrtf(sums[2] * p.inv_D + p.eps) : 1.f;
        const float *w_post = p.post ? p.w_post : nullptr;
        float2 yd = both(0.f), wt[PER / 2];
        if constexpr (kAhead)
            if (gate) read8(gr.p[0], here + (2 * kX + 2 * kT) * threads, threads);
#pragma unroll
        for (int j = 0; j < PER / VEC; ++j) {
            const Weight<VEC> w = weight_of<VEC>(w_post, j, D);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int i = j * VEC + e;
                (i & 1 ? wt[i / 2].y : wt[i / 2].x) = w.v[e];
            }
        }
        if (gate) {
            float2 dg[PER / 2];
#pragma unroll
            for (int i = 0; i < PER; i += 2) {
                float2 a, da;
                gate_both(p.act, gr.two(i), a, da);
                const float2 dz = mul2(both(p.s), dv[i / 2]), n = mul2(yr.two(i), both(r));
                dg[i / 2] = mul2(mul2(dz, da), mul2(n, wt[i / 2]));
                dv[i / 2] = mul2(dz, a);
                add(a_post, 0, i, mul2(one_gate ? dz : dv[i / 2], n));
            }
            if (p.gate_stride && dgate) store_row<T, VEC>(dgate + at, D, reinterpret_cast<const float(&)[PER]>(dg));
        } else {
#pragma unroll
            for (int i = 0; i < PER; i += 2) {
                dv[i / 2] = mul2(both(p.s), dv[i / 2]);
                add(a_post, 0, i, mul2(dv[i / 2], mul2(yr.two(i), both(r))));
            }
        }
#pragma unroll
        for (int i = 0; i < PER; i += 2) {
            dv[i / 2] = mul2(dv[i / 2], wt[i / 2]);
            yd = fma2(dv[i / 2], yr.two(i), yd);
        }
        if (p.post) {
            float dot[1] = {yd.x + yd.y};
            row_sum(dot, buf, turn);
            const float m = r * r * (dot[0] * p.inv_D);
#pragma unroll
            for (int i = 0; i < PER; i += 2) dv[i / 2] = mul2(both(r), fma2(yr.two(i), both(-m), dv[i / 2]));
        }
        store_row<T, VEC>(dy + at, D, reinterpret_cast<const float(&)[PER]>(dv));
    }
    const int64_t mine = ((int64_t)blockIdx.x * blockDim.y + threadIdx.y) * p.D;
    const float *w_end = p.post ? p.w_post : nullptr;
    if constexpr (kWide) {
        __syncthreads();
        for (int e = threadIdx.x; e < p.D; e += blockDim.x) {
            float2 a = both(1.f), da = a;
            if (one_gate) gate_both(p.act, both((float)gate[e]), a, da);
            if (part_post) part_post[mine + e] = wide[e] * a.x;
            if (part_pre) part_pre[mine + e] = wide[p.D + e];
            if (part_gate) part_gate[mine + e] = wide[e] * (w_end ? w_end[e] : 1.f) * da.x;
        }
    } else {
        if (part_pre) store_row<float, VEC>(part_pre + mine, p.D, reinterpret_cast<const float(&)[PER]>(a_pre));
        if (one_gate) {
            Raw<T, VEC, PER> gr;
            gr.load(gate, p.D);
            float2 a_gate[kSums];
#pragma unroll
            for (int j = 0; j < PER / VEC; ++j) {
                const Weight<VEC> w = weight_of<VEC>(w_end, j, p.D);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const int i = j * VEC + e;
                    (i & 1 ? a_gate[i / 2].y : a_gate[i / 2].x) = w.v[e];
                }
            }
#pragma unroll
            for (int i = 0; i < PER; i += 2) {
                float2 a, da;
                gate_both(p.act, gr.two(i), a, da);
                a_gate[i / 2] = mul2(mul2(a_post[i / 2], a_gate[i / 2]), da);
                a_post[i / 2] = mul2(a_post[i / 2], a);
            }
            if (part_gate) store_row<float, VEC>(part_gate + mine, p.D, reinterpret_cast<const float(&)[PER]>(a_gate));
        }
        if (part_post) store_row<float, VEC>(part_post + mine, p.D, reinterpret_cast<const float(&)[PER]>(a_post));
    }
}

struct Sum {
    const float *part;
    void *out;
    int f32;  // out in fp32 (weights), else in the block's type (the gate's row)
};
struct Sums {
    Sum v[3];
};

// out[c] = sum over the parts of column c: 32 columns per block, 32 threads each take every
// 32nd part, the 32 added in order. Bound by the loads' latency, one behind the other.
constexpr int kSumRows = 32;
template <typename T>
__global__ void __launch_bounds__(32 * kSumRows) column_sum_kernel(const Sums s, int parts, int D) {
    __shared__ float buf[kSumRows][33];
    const Sum &m = s.v[blockIdx.y];
    const int c = blockIdx.x * 32 + threadIdx.x;
    float t = 0.f;
    if (c < D) {
#pragma unroll 8
        for (int r = threadIdx.y; r < parts; r += kSumRows) t += m.part[(int64_t)r * D + c];
    }
    buf[threadIdx.y][threadIdx.x] = t;
    __syncthreads();
    if (threadIdx.y == 0 && c < D) {
#pragma unroll
        for (int r = 1; r < kSumRows; ++r) t += buf[r][threadIdx.x];
        if (m.f32) ((float *)m.out)[c] = t;
        else ((T *)m.out)[c] = from_f32<T>(t);
    }
}

// Entries per thread, entries per access, threads per row and rows per block: a row's entries
// spread over whole warps, narrow rows share a block of up to 128 threads. Forward 16 entries
// per thread where 8 would take a second warp (16384 rows, 8 and 16: D = 512 26 and 23 us, 2048
// 74 and 60, 4096 145 and 113); backward 8, as a thread also holds the sums of its columns (D =
// 512 46 and 76 us, 2048 129 and 226, 4096 230 and 448), and 16 beyond D = 4096, where 8 would
// take more than 512 threads.
struct Shape2 {
    int per, vec;
    dim3 block;
};
Shape2 shape_of(int D, bool backward) {
    Shape2 s;
    s.per = D <= (backward ? 4096 : 256) ? 8 : 16;
    s.vec = D % 8 == 0 ? 8 : (D % 2 == 0 ? 2 : 1);
    const int tpr = ((D + s.per - 1) / s.per + 31) / 32 * 32;
    s.block = dim3((unsigned)tpr, (unsigned)(tpr >= 128 ? 1 : 128 / tpr));
    return s;
}
size_t elem(int dtype) { return dtype == GDR_F32 ? 4 : 2; }

// Blocks of a backward call: all of them are resident at once. Where a block has at most 256
// threads an SM takes 768 (registers: the kernel's bounds above) and what its 228 KB of shared memory
// hold (each block the rows that it fetches ahead, its buffer, and 1 KB of the system's), else one
// block. fp32 in widths of eights is where shared memory decides.
// With a third of the blocks left for a second round: 4099 x 1030 fp32 47 us, now 35; 8192 x 2048
// fp32 216 us, now 180.
int bwd_blocks(int64_t rows, const Shape2 &s, const gdr_block_norm_shape *shape) {
    const int threads = (int)(s.block.x * s.block.y);
    const int64_t need = (rows + s.block.y - 1) / s.block.y;
    int per_sm = threads <= 256 ? 768 / threads : 1;
    if (s.per == 8 && s.vec == 8) {  // fetches_ahead
        const int ahead = 2 * s.per * (int)(2 * elem(shape->x_dtype) + 3 * elem(shape->dtype)) * threads;
        const int fit = 228 * 1024 / (ahead + kBufBytes + 1024);
        if (fit < per_sm) per_sm = fit;
    }
    const int64_t most = (int64_t)kSms * per_sm;
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
        const int threads = (int)(s.block.x * s.block.y);
        const size_t bytes = PER > 8 ? 2 * (size_t)p.D * sizeof(float)
                             : (fetches_ahead<T, VEC, PER>() ? 2 * (size_t)row_bytes<T, TX, PER>() * threads : 0);
        auto kernel = PER > 8 || threads > 256 ? block_norm_bwd_kernel<T, TX, VEC, PER, 512>
                                               : block_norm_bwd_kernel<T, TX, VEC, PER, (PER > 8 ? 512 : 256)>;
        // (48 KB without asking, the kernel's own 384 bytes among them: D = 6144 has to ask)
        if (bytes + kBufBytes > 48 * 1024 &&
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess)
            return GDR_ERR_CUDA;
        kernel<<<(unsigned)blocks, s.block, bytes, stream>>>(
            p, (const TX *)dx_out, (const T *)dh, (const TX *)x, (const T *)y, (const T *)gate,
            (TX *)dx, (T *)dy, (T *)dgate, pp, pn, pg);
        return cuda_status(cudaGetLastError());
    }
};

#define GDR_NORM_BY_SHAPE(R, what, A, B, ...)                                   \
    do {                                                                       \
        if (s.per == A) {                                                      \
            if (s.vec == 8) return R::template what<8, A>(__VA_ARGS__);        \
            if (s.vec == 2) return R::template what<2, A>(__VA_ARGS__);        \
            return R::template what<1, A>(__VA_ARGS__);                        \
        }                                                                      \
        if (s.vec == 8) return R::template what<8, B>(__VA_ARGS__);            \
        if (s.vec == 2) return R::template what<2, B>(__VA_ARGS__);            \
        return R::template what<1, B>(__VA_ARGS__);                            \
    } while (0)

template <typename T, typename TX>
int run_fwd(const NormParams &p, const Shape2 &s, const void *x, const void *y, const void *gate,
            void *x_out, void *h, cudaStream_t stream) {
    using R = Run<T, TX>;
    GDR_NORM_BY_SHAPE(R, fwd, 8, 16, p, s, x, y, gate, x_out, h, stream);
}
template <typename T, typename TX>
int run_bwd(const NormParams &p, const Shape2 &s, int blocks, const void *dx_out, const void *dh,
            const void *x, const void *y, const void *gate, void *dx, void *dy, void *dgate,
            float *pp, float *pn, float *pg, cudaStream_t stream) {
    using R = Run<T, TX>;
    GDR_NORM_BY_SHAPE(R, bwd, 8, 16, p, s, blocks, dx_out, dh, x, y, gate, dx, dy, dgate, pp, pn, pg, stream);
}

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
    p->inv_D = 1.f / s->D;
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
    const Shape2 s = shape_of(p.D, false);
    const cudaStream_t stm = (cudaStream_t)stream;
    if (shape->dtype == GDR_F32) return run_fwd<float, float>(p, s, x, y, gate, x_out, h, stm);
    if (shape->x_dtype == GDR_F32) return run_fwd<__nv_bfloat16, float>(p, s, x, y, gate, x_out, h, stm);
    return run_fwd<__nv_bfloat16, __nv_bfloat16>(p, s, x, y, gate, x_out, h, stm);
}

size_t gdr_block_norm_bwd_workspace_size(const gdr_block_norm_shape *shape) {
    NormParams p;
    if (check_shape(shape, &p) != GDR_OK) return 0;
    const Shape2 s = shape_of(p.D, true);
    const size_t parts = (size_t)bwd_blocks(p.rows, s, shape) * s.block.y;
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
    const Shape2 s = shape_of(p.D, true);
    const cudaStream_t stm = (cudaStream_t)stream;
    const int blocks = bwd_blocks(p.rows, s, shape);
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
    const dim3 grid((unsigned)((p.D + 31) / 32), (unsigned)n), block(32, kSumRows);
    if (shape->dtype == GDR_F32) column_sum_kernel<float><<<grid, block, 0, stm>>>(sums, parts, p.D);
    else column_sum_kernel<__nv_bfloat16><<<grid, block, 0, stm>>>(sums, parts, p.D);
    return cuda_status(cudaGetLastError());
}

}  // extern "C"
