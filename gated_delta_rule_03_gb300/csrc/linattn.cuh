// linattn.cuh -- what the kernels of linear attention with a constant decay per head share.
//
// With lam = exp(log_decay[h]), per sequence and head:
//   S_t = lam S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t.
// Backward, with D_t the gradient of S_t (D_T = dS_final for the last token T):
//   D_t = lam D_{t+1} + scale q_t do_t^T,   dq_t = scale S_t do_t,
//   dk_t = D_t v_t,   dv_t = D_t^T k_t,   dS0 = lam D_1.
//
// All four are one "mix" of rows x, y (d_x entries) and z (d_z entries) around a state
// E [d_x][d_z]. A chunk of n tokens (rows r = 0 .. n-1), entered with E, gives
//   out_r = s_intra sum_i M_ri lam^|r-i| (x_r.y_i) z_i + s_inter w_out(r) x_r E
//   E    <- lam^n E + s_state sum_r w_upd(r) y_r z_r^T
// with
//                 x    y    z    state    order    M_ri     w_out      w_upd
//   o             q    k    v    S        first    i <= r   lam^(r+1)  lam^(n-1-r)
//   dq            do   v    k    S^T      to last  i <= r   lam^(r+1)  lam^(n-1-r)
//   dv            k    q    do   E        last     i >= r   lam^(n-1-r) lam^(r+1)
//   dk            v    do   q    E^T      to first i >= r   lam^(n-1-r) lam^(r+1)
// where E = lam D_{t+1} is the state carried backwards (so that its start value is
// dS_final and its last value dS0), and s_intra = scale; s_inter, s_state = scale, 1 from
// first to last and 1, scale from last to first. Every power of lam has an exponent >= 0.
//
// Segments. Without a gate that depends on the tokens, the state after a run of tokens is
// lam^n times the state before it plus a sum that does not depend on that state. A sequence
// is cut into segments of `seg` tokens (the last one shorter). A first launch computes every
// segment's own sum R_f; in the second every segment starts from
//   first to last:  lam^(f seg) S0 + sum_{g<f} lam^((f-1-g) seg) R_g
//   last to first:  lam^(tokens behind f) dS_final + sum_{g>f} lam^((g-1-f) seg) R_g
// and all segments run at once. With one segment per sequence the first launch is left out.
// Where the sums alone would leave SMs idle, they are taken over parts of a segment. Of equal
// sequences only those may be cut that whole rounds of the SMs leave over.
#pragma once

#include "internal.h"

namespace gdr {
namespace linattn {

constexpr float kLog2e = 1.4426950408889634f;

// One mix of a launch.
struct Mix {
    const void *x, *y, *z;
    int64_t xs, ys, zs;     // elements from one token's rows to the next token's
    int xg, yg, zg;         // heads of the state that share one head of x, y, z
    void *out;              // [total_tokens, H, d_z], or null (state only)
    bool out_f32;           // out in fp32 whatever the input type (partial sums)
    int dx, dz;
    bool turned;            // the state in memory is [d_z][d_x] (S^T, E^T)
    bool backward;          // from the last token to the first
    float s_intra, s_inter, s_state;
    const float *start;     // S0 or dS_final, [num_seqs, H] matrices, or null
    float *end;             // S_final or dS0, or null
    const float *R;         // the segments' own sums (null: one segment)
    float *R_out;           // state only: where they go
};

// The sequences and segments of a call.
struct Plan {
    const int32_t *cu_seqlens;  // null: equal lengths
    int64_t num_seqs, total_tokens;
    int64_t seg;                // tokens per segment (a multiple of a block's chunk)
    int64_t seq_len;            // equal lengths
    int segs;                   // segments per sequence (equal lengths) ..
    int64_t whole;              // .. of all but the first `whole` (sequence, head) pairs: they stay whole
    int64_t sums;               // segments that hand a sum on, those of whole pairs too (packed: a bound)
    int64_t units, handing;     // (segment, head) pairs, and those that hand a sum on (packed: bounds)
    int split;                  // parts of a segment that are summed by themselves (each seg / split
                                // tokens): R has [sums, split, H] matrices
    int H;
    const float *log_decay;
    int32_t *status;            // the workspace's status word
    bool first;                 // the launch sets the status word (the call's first, unless `checked`)
    bool checked;               // launch_check has run: the status word says whether the offsets are ones
    bool fine;                  // a state goes out: its terms keep fp32's bits
};

struct Segment {
    int seq;        // -1: nothing to do
    int f, n;       // this segment's number and the sequence's count
    int64_t begin;  // first token of the segment
    int64_t tokens; // its tokens
    int64_t behind; // tokens of the sequence behind it
    int64_t sum0;   // its sequence's first sum in R: one per segment but the last (or the first)
    int h;          // head
};

// What unit `unit` of a launch is, a segment and a head: all of them, or (`handing` 1 or 2)
// those that hand a sum on, all of a sequence but its last (1) or its first (2). Equal
// lengths: first the pairs that stay whole, then the segments one after the other. Called
// by the whole block (a barrier inside). With cu_seqlens every block checks all of it (offsets
// from 0, not decreasing, at most total_tokens); where it is not so, no block does anything:
// false. Beyond kChecked sequences a launch ahead has done that (launch_check). Up to kOrdered
// sequences are taken longest first, so that short ones fill up the end of the launch (a
// sequence's place takes a look at every other, hence the limit). In this and in the order of
// memory: 8 of 1,611 to 7,848 tokens, shortest first, 32 heads 267 and 300 us; 31 of 900 and one of
// 6,000, 16 heads 173 and 215, backward with 32 heads 800 and 755. Of more, sequence n has the
// places from n + floor(cu[n] / seg) on (of those that hand a sum on: from floor(cu[n] / seg)): as
// many as it needs or one more, up to where the next one's begin and the last one's at the launch's
// end. So the pass that checks finds a place's sequence, and so does a search where there is no such
// pass, without counting places up (20,000 sequences of one token, two heads 2.1 ms, with places
// counted and offsets checked by every block 12.0; 1000 of 60, 16 heads 0.91 and 1.06).
// `scratch`: 2 kOrdered ints of shared memory.
constexpr int kOrdered = 64, kChecked = 2048;
__device__ __forceinline__ bool locate(const Plan &p, int64_t unit, int handing, Segment *shared, int *scratch) {
    const int skip = handing == 2;  // segments in front of the first item's
    const int less = handing != 0;
    auto fill = [&](int seq, int h, int f, int n, int64_t first, int64_t len, int64_t sum0) {
        Segment s;
        s.seq = seq;
        s.f = f;
        s.n = n;
        s.begin = first + (int64_t)f * p.seg;
        const int64_t rest = len - (int64_t)f * p.seg;
        s.tokens = n == 1 || rest < p.seg ? rest : p.seg;
        s.behind = rest - s.tokens;
        s.sum0 = sum0;
        s.h = h;
        *shared = s;
    };
    if (!p.cu_seqlens) {
        int64_t pair = unit;
        int f = 0, n = 1;
        if (less || unit >= p.whole) {
            const int64_t r = less ? unit : unit - p.whole, left = p.num_seqs * p.H - p.whole;
            pair = p.whole + r % left;
            f = (int)(r / left) + skip;
            n = p.segs;
        }
        const int64_t seq = pair / p.H;
        if (threadIdx.x == 0) fill((int)seq, (int)(pair % p.H), f, n, seq * p.seq_len, p.seq_len, seq * (p.segs - 1));
        __syncthreads();
        return true;
    }
    const int64_t item = unit / p.H;
    const int tid = threadIdx.x;
    if (tid == 0) shared->seq = -1;
    if (p.num_seqs > kOrdered) {
        int64_t n = -1;  // the sequence whose places `item` is among, in one thread
        if (p.checked) {
            if (__syncthreads_or(tid == 0 && *p.status != GDR_OK)) return false;
            // the last one whose places begin at `item` or before it: every thread looks at one of as
            // many, evenly apart, in each round
            int64_t from = 0, left = p.num_seqs;
            while (left > 1) {
                const int64_t apart = (left + blockDim.x - 1) / blockDim.x, at = from + tid * apart;
                bool begun = false;
                if (at < from + left) {
                    const int64_t place = item - (less ? 0 : at);  // floor(cu[at] / seg) <= place
                    begun = place >= 0 && p.cu_seqlens[at] < (place + 1) * p.seg;
                }
                const int64_t last = __syncthreads_count(begun) - 1;
                left = left - last * apart < apart ? left - last * apart : apart;
                from += last * apart;
            }
            if (tid == 0) n = from;
        } else {
            int wrong = 0;
#pragma unroll 4
            for (int64_t i = tid; i < p.num_seqs; i += blockDim.x) {
                const int64_t a = p.cu_seqlens[i], b = p.cu_seqlens[i + 1];
                if (b < a || a < 0 || b > p.total_tokens || (i == 0 && a != 0)) wrong = 1;
                // floor(a / seg) <= place < floor(b / seg), or one more for each sequence
                const int64_t place = item - (less ? 0 : i);
                if (place >= 0 && a < (place + 1) * p.seg && b >= (place + less) * p.seg) n = i;
            }
            if (__syncthreads_or(wrong)) return false;
        }
        if (n >= 0) {
            const int64_t a = p.cu_seqlens[n], len = (int64_t)p.cu_seqlens[n + 1] - a, first = a / p.seg;
            int64_t count = (len + p.seg - 1) / p.seg;
            if (count < 1) count = 1;  // an empty sequence still hands on its state
            const int64_t f = item - (less ? 0 : n) - first;
            if (f < count - less) fill((int)n, (int)(unit % p.H), (int)f + skip, (int)count, a, len, first);
        }
        __syncthreads();
        return true;
    }
    const int lane = tid & 31, warp = tid >> 5;
    __shared__ int64_t warp_sum[32];
    int *lens = scratch + kOrdered;
    const int mine = tid < p.num_seqs ? p.cu_seqlens[tid + 1] - p.cu_seqlens[tid] : 0;
    if (tid < p.num_seqs) lens[tid] = mine;
    __syncthreads();
    if (tid < p.num_seqs) {
        int rank = 0;
        for (int j = 0; j < (int)p.num_seqs; ++j) rank += lens[j] > mine || (lens[j] == mine && j < tid);
        scratch[rank] = tid;
    }
    __syncthreads();
    int wrong = 0;
    int64_t n = tid, a = 0, len = 0, count = 0;  // of place tid in the order
    if (tid < p.num_seqs) {
        n = scratch[tid];
        a = p.cu_seqlens[n];
        len = (int64_t)p.cu_seqlens[n + 1] - a;
        if (len < 0 || a < 0 || a + len > p.total_tokens || (n == 0 && a != 0)) {
            wrong = 1;
        } else {
            count = (len + p.seg - 1) / p.seg;
            if (count < 1) count = 1;
            count -= less;
        }
    }
    int64_t sum = count;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, sum, off);
        if (lane >= off) sum += up;
    }
    if (lane == 31) warp_sum[warp] = sum;
    __syncthreads();
    int64_t before = 0;
    for (int w = 0; w < warp; ++w) before += warp_sum[w];
    const int64_t first_item = before + sum - count;
    if (count > 0 && item >= first_item && item < first_item + count)
        fill((int)n, (int)(unit % p.H), (int)(item - first_item) + skip, (int)count + less, a, len, first_item - (less ? 0 : tid));
    return __syncthreads_or(wrong) == 0;
}

// log2 of the decay, held finite so that 0 * log2(lam) is 0 for lam = 0 (-inf); NaN stays.
__device__ __forceinline__ float log2_decay(float log_decay) {
    return log_decay < -1e30f ? -1e30f : log_decay * kLog2e;
}
// lam^n for n >= 0. The product's rounding shifts the result by |n log2 lam| 2^-24 of
// itself at most, where the power itself has shrunk to 2^-|n log2 lam|.
__device__ __forceinline__ float decay_pow(float l2, float n) { return exp2f(l2 * n); }

// Element (a, b) of a state matrix [d_x][d_z], or of its transpose in memory.
__device__ __forceinline__ int64_t state_at(const Mix &m, int a, int b) {
    return m.turned ? (int64_t)b * m.dx + a : (int64_t)a * m.dz + b;
}

// Sets the status word, by the offsets of cu_seqlens.
int launch_check(const Plan &p, cudaStream_t stream);
// (rows in fp32, or none)
int launch_mix_exact(const Plan &p, const Mix *mixes, int count, cudaStream_t stream);
// `sums`: the segments' own sums; `after_sums`: the launch ahead is theirs.
int launch_mix_tc(const Plan &p, const Mix *mixes, int count, int d_v, bool sums, bool after_sums, cudaStream_t stream);
// Sums the g parts of every head: in fp32 [rows, heads g, d] -> out [rows, heads, d]. Rows
// behind the last sequence are left as they are.
struct Share {
    const float *in;
    void *out;
    int heads, g, d;
};
int launch_share(const Plan &p, const Share *shares, int count, int dtype, cudaStream_t stream);
int launch_step(const void *q, const void *k, const void *v, const float *log_decay, float *S,
                void *o, int64_t N, int H, int qg, int kg, int vg, int dk, int dv, int dtype,
                float scale, int64_t qs, int64_t ks, int64_t vs, cudaStream_t stream);

}  // namespace linattn
}  // namespace gdr
