// rotary.cu -- rotary positions of queries and keys, and the turn back of their gradients.
//
// Pair i of a token at position p is turned by 2 pi (p rates[i] mod 2^64) / 2^64: the 64-bit
// product drops whole turns exactly, so a far position costs no precision, and no 64-bit
// floating arithmetic is needed (the card has little of it). A thread takes the pairs of two
// 16-byte vectors of a token and goes through several heads with one set of sines and cosines.
// Bound by memory: every value is read and written once. 16384 tokens of 20 bf16 heads, 168 MB: 33.7 us, 5.0 TB/s; 4099
// tokens of 10 fp32 heads of 256, 84 MB: 13.4 us. Two heads' loads are under way together, in 64 registers, so
// that four blocks share an SM: one head after the other took 47 us for the first.
#include <math.h>

#include "internal.h"
#include "spans.h"

namespace gdr {
namespace {

struct Rotary {
    const void *x[2];
    void *y[2];
    int64_t xs[2], ys[2];
    const int32_t *pos;
    const int64_t *rates;
    int64_t units;  // tokens * lanes
    int heads[2];
    int lanes, turning;  // vector pairs of a head, those of them that are turned
    int d, rot, step;    // step: heads of one thread
    bool neighbours, back;
    float amplitude;
};

template <typename T, int V> struct alignas(sizeof(T) * V) Vec {
    T v[V];
};

// V elements to a vector, two vectors to a thread: lane a < turning holds pairs a V .. a V + V - 1,
// the lanes behind copy what is not turned.
template <typename T, int V, bool kNeighbours> __global__ void __launch_bounds__(256, 4) rotary_kernel(Rotary r) {
    const int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (u >= r.units) return;
    const int64_t t = r.units < INT32_MAX ? (int64_t)((uint32_t)u / (uint32_t)r.lanes) : u / r.lanes;
    const int a = (int)(u - t * r.lanes);
    const bool turns = a < r.turning;
    int first, second;  // elements of the head where the two vectors begin
    if (turns) {
        first = kNeighbours ? 2 * a * V : a * V;
        second = kNeighbours ? first + V : first + r.rot / 2;
    } else {
        first = r.rot + 2 * (a - r.turning) * V;
        second = first + V;
    }
    const bool both = second < r.d;
    float c[V], s[V];
    if (turns) {
        const int64_t p = r.pos[t];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint64_t turn = (uint64_t)p * (uint64_t)r.rates[a * V + i];
            // to the nearest 2^-32 turn, and the nearest of both ways round: -1 <= half turns < 1. fp32 holds 24 bits of it; of
            // fp32 results the others, an angle below 2e-7, turn the sine and cosine on by their first derivatives (2.1e-8 in
            // norm, 2.7e-8 without; 1 % of the time, which bf16 results are spared).
            const int32_t nearest = (int32_t)((turn + 0x80000000u) >> 32);
            const float most = sizeof(T) == 4 ? __int2float_rz(nearest) : (float)nearest;
            sincospif(most * 4.656612873077393e-10f, &s[i], &c[i]);
            if (sizeof(T) == 4) {
                const float rest = (float)(nearest - (int32_t)most) * 1.4629180792671596e-9f;  // pi 2^-31
                const float s0 = s[i];
                s[i] = fmaf(c[i], rest, s0);
                c[i] = fmaf(-s0, rest, c[i]);
            }
            c[i] *= r.amplitude;
            s[i] *= r.back ? -r.amplitude : r.amplitude;
        }
    }
    using W = Vec<T, V>;
    const int all = r.heads[0] + r.heads[1];
    const int h0 = blockIdx.y * r.step, h1 = min(h0 + r.step, all);
    auto place = [&](int h, const T *&from, T *&to) {
        const bool k = h >= r.heads[0];
        const int at = k ? h - r.heads[0] : h;
        from = (const T *)(k ? r.x[1] : r.x[0]) + t * (k ? r.xs[1] : r.xs[0]) + (int64_t)at * r.d;
        to = (T *)(k ? r.y[1] : r.y[0]) + t * (k ? r.ys[1] : r.ys[0]) + (int64_t)at * r.d;
    };
    constexpr int kAhead = 2;  // heads whose loads are under way together
    for (int h = h0; h < h1; h += kAhead) {
        W x[kAhead], y[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (h + j < h1) {
                const T *from;
                T *to;
                place(h + j, from, to);
                x[j] = *(const W *)(from + first);
                if (both) y[j] = *(const W *)(from + second);
            }
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (h + j >= h1) break;
            const T *from;
            T *to;
            place(h + j, from, to);
            if (turns) {
                float e[2 * V];  // the two vectors
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    e[i] = to_f32<T>(x[j].v[i]);
                    e[V + i] = to_f32<T>(y[j].v[i]);
                }
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int m = kNeighbours ? 2 * i : i, n = kNeighbours ? 2 * i + 1 : V + i;
                    const float p = e[m], q = e[n];
                    e[m] = p * c[i] - q * s[i];
                    e[n] = p * s[i] + q * c[i];
                }
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    x[j].v[i] = from_f32<T>(e[i]);
                    y[j].v[i] = from_f32<T>(e[V + i]);
                }
            }
            *(W *)(to + first) = x[j];
            if (both) *(W *)(to + second) = y[j];
        }
    }
}

template <typename T, int V> int launch_rotary(Rotary r, int64_t tokens, bool in_place, cudaStream_t s) {
    r.turning = r.rot / (2 * V);
    const int rest = (r.d - r.rot + 2 * V - 1) / (2 * V);
    r.lanes = r.turning + (in_place ? 0 : rest);
    r.units = tokens * r.lanes;
    // Enough threads to fill the GPU (152 SMs of 2048 threads), each with as many heads as that
    // leaves: the sines of a pair are taken once for all of them.
    const int all = r.heads[0] + r.heads[1];
    const int64_t want = 152 * 2048;
    int64_t parts = (want + r.units - 1) / r.units;
    if (parts > all) parts = all;
    if (parts > 65535) parts = 65535;  // (of a grid)
    r.step = (int)((all + parts - 1) / parts);
    const dim3 grid((unsigned)((r.units + 255) / 256), (unsigned)((all + r.step - 1) / r.step));
    if (r.neighbours)
        rotary_kernel<T, V, true><<<grid, 256, 0, s>>>(r);
    else
        rotary_kernel<T, V, false><<<grid, 256, 0, s>>>(r);
    return cuda_status(cudaGetLastError());
}

// The widest vectors that the pairs allow: 16 bytes, else one element.
template <typename T> int pick_rotary(const Rotary &r, int64_t tokens, bool in_place, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    const int unit = r.neighbours ? r.rot : r.rot / 2;
    if (unit % (r.neighbours ? 2 * V : V) == 0) return launch_rotary<T, V>(r, tokens, in_place, s);
    return launch_rotary<T, 1>(r, tokens, in_place, s);
}

int rotary(const gdr_rotary_shape *sh, const void *q, const void *k, const int32_t *pos, const int64_t *rates,
           void *qo, void *ko, bool back, gdr_stream_t stream) {
    if (!sh || sh->tokens < 0 || sh->tokens > INT32_MAX) return GDR_ERR_INVALID_ARG;
    if (sh->q_heads < 1 || sh->k_heads < 0 || sh->q_heads > 1 << 16 || sh->k_heads > 1 << 16) return GDR_ERR_INVALID_ARG;
    if (sh->dtype != GDR_F32 && sh->dtype != GDR_BF16) return GDR_ERR_UNSUPPORTED;
    if (sh->d < 8 || sh->d > 256 || sh->d % 8 || sh->rot_dim < 2 || sh->rot_dim > sh->d || sh->rot_dim % 2)
        return GDR_ERR_UNSUPPORTED;
    if (!isfinite(sh->amplitude)) return GDR_ERR_INVALID_ARG;
    const size_t e = sh->dtype == GDR_F32 ? 4 : 2;
    Rotary r = {};
    r.heads[0] = sh->q_heads;
    r.heads[1] = sh->k_heads;
    r.x[0] = q, r.x[1] = k, r.y[0] = qo, r.y[1] = ko;
    const int64_t in[2] = {sh->q_stride, sh->k_stride}, out[2] = {sh->q_out_stride, sh->k_out_stride};
    Rows reads[4], writes[2];
    bool in_place = true;
    for (int i = 0; i < 2; ++i) {
        const int64_t row = (int64_t)r.heads[i] * sh->d;
        if (r.heads[i] == 0) {
            if (r.x[i] || r.y[i]) return GDR_ERR_INVALID_ARG;
            reads[i] = writes[i] = {nullptr, 0, 1, 0};
            continue;
        }
        int st = row_stride(in[i], row, e, &r.xs[i]);
        if (st == GDR_OK) st = row_stride(out[i], row, e, &r.ys[i]);
        if (st != GDR_OK) return st;
        if (sh->tokens > 0 && (!r.x[i] || !r.y[i])) return GDR_ERR_INVALID_ARG;
        if (!aligned(r.x[i], 16) || !aligned(r.y[i], 16)) return GDR_ERR_ALIGNMENT;
        const bool same = r.x[i] == r.y[i];
        if (same && r.xs[i] != r.ys[i]) return GDR_ERR_INVALID_ARG;
        if (!same) in_place = false;
        reads[i] = {same ? nullptr : r.x[i], sh->tokens, r.xs[i] * (int64_t)e, row * (int64_t)e};
        writes[i] = {r.y[i], sh->tokens, r.ys[i] * (int64_t)e, row * (int64_t)e};
    }
    if (sh->tokens > 0 && (!pos || !rates)) return GDR_ERR_INVALID_ARG;
    if (!aligned(pos, 4) || !aligned(rates, 8)) return GDR_ERR_ALIGNMENT;
    reads[2] = {pos, 1, 1, sh->tokens * 4};
    reads[3] = {rates, 1, 1, (int64_t)sh->rot_dim * 4};
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 4; ++j)
            if (sharing(writes[i], reads[j])) return GDR_ERR_INVALID_ARG;
    if (sharing(writes[0], writes[1])) return GDR_ERR_INVALID_ARG;
    if (sh->tokens == 0) return GDR_OK;
    r.pos = pos;
    r.rates = rates;
    r.d = sh->d;
    r.rot = sh->rot_dim;
    r.neighbours = sh->neighbours != 0;
    r.back = back;
    r.amplitude = sh->amplitude;
    const cudaStream_t s = (cudaStream_t)stream;
    return sh->dtype == GDR_F32 ? pick_rotary<float>(r, sh->tokens, in_place, s)
                                : pick_rotary<__nv_bfloat16>(r, sh->tokens, in_place, s);
}

}  // namespace
}  // namespace gdr

extern "C" {

int gdr_rotary_fwd(const gdr_rotary_shape *shape, const void *q, const void *k, const int32_t *positions,
                   const int64_t *rates, void *q_out, void *k_out, gdr_stream_t stream) {
    return gdr::rotary(shape, q, k, positions, rates, q_out, k_out, false, stream);
}

int gdr_rotary_bwd(const gdr_rotary_shape *shape, const void *dq_out, const void *dk_out, const int32_t *positions,
                   const int64_t *rates, void *dq, void *dk, gdr_stream_t stream) {
    return gdr::rotary(shape, dq_out, dk_out, positions, rates, dq, dk, true, stream);
}

}  // extern "C"
