// cache_attn_step.cuh -- attention over a paged 8-bit cache for few rows: single tokens.
//
// Rows. The queries of one request that share a head of the cache (its group of heads, times its
// new tokens), up to kR of them: an item is (request, head of the cache).
//
// Products. Warp-level 16x8x16 MMAs in fp16 with fp32 sums, whose operands are registers, so that codes go from
// the copy in shared memory to an operand without a turn through it. Up to 8 rows (kR = 8) are the 8 columns and
// tokens and dims the 16 rows, half as many products and registers as with 16 rows against 8 tokens or
// dims (kR = 16, only for 9 rows and more). The order of the contraction is free: thread c of a quad takes 16 consecutive
// bytes of a key as the k indices of four steps (queries are laid out alike), and dims 16 g + u of a value as
// column g of step u, so that shared memory is read 16 bytes at a time.
// The tensor cores are far from busy (a tenth at 8 heads a group); the 5th-generation ones would need
// the codes converted through shared memory, rows filled up to 128, and the same bytes.
// The tensor cores cut sums instead of rounding them. fp32: the two products of a tile of 16 tokens, and of 16 dims of a
// score, begin at 0 and are added up by ordinary additions (otherwise outputs have a mean error of 4e-6 behind 8192 tokens and
// 2e-5 behind 32,768, and with heads of 256 7.8e-7 of scores alone, 3.0e-7 so; 1 to 3 % of the time). bf16 ones stay in the sums of the products: some 4e-8 of a sum for each tile of a warp, 3e-4 behind 500,000
// tokens, beside its own rounding's 2e-3 (added up outside, 256 requests of 512 to 8192 tokens take 414 us for 407).
//
// Bound by memory: each cached byte is read once. A warp streams tiles of 16 tokens
// through a ring of its own in shared memory (tensor copies, kStages deep: no barrier between warps until an
// item ends). 16-byte copies by threads stopped at 4.4 TB/s in the order that the products take them, 32 bytes
// of a line at a time, and at 5.3 TB/s by whole lines.
//
// Split. All items' keys, in units of kUnit tokens, are laid end to end and shared out equally
// among the resident blocks, whatever the requests' lengths (one token behind 2048, 8 heads: a unit to a block 9.1 us, four
// 12.3; behind 8192 14.5 and 13.5). A block that ends inside an item leaves its part in the workspace;
// join_parts_kernel adds them in order.
#pragma once

#include "cache_attn.cuh"
#include "sm100.cuh"

namespace gdr {
namespace cattn {

constexpr int kStepWarps = 4;
constexpr int kUnit = 16 * kStepWarps;  // tokens
constexpr int kSms = 152;
constexpr size_t kTaskBytes = kSms * 4 * 2 * sizeof(int4);  // (at most 4 blocks an SM)

template <int D, int kParts, int kR> struct StepConfig {
    static constexpr int kSteps = D / 16;                 // k steps of the first product
    // Tiles under way for each warp, and blocks of an SM. 64 requests of 512 to 8192 tokens, 32 heads over 8: heads of 128 in
    // bf16 116 us, with a block less an SM 115, a stage less 112; heads of 64 75, 78 and 74; of 256 222, 253 and 210; 12
    // heads a group 147, 153 and 146; fp32, heads of 128 124, 138 and 122.
    static constexpr int kStages = D == 64 ? 6 : D == 256 ? (kParts == 2 ? 2 : 3) : kR == 8 && kParts == 1 ? 3 : 4;
    static constexpr int kBlocks = D == 64 ? (kParts == 2 ? 3 : 4) : D == 256 ? 2 : kParts == 2 ? (kR == 8 ? 3 : 2) : kR == 8 ? 4 : 3;  // per SM
    static constexpr int kStage = 2 * 16 * D;             // bytes: keys, then values
    static constexpr int kRing = kStepWarps * kStages * kStage;
    static constexpr int kQ = kParts * kSteps * 32 * kR;
    // Queries stay in registers where there is room for them (fp32, heads of 128, up to 8 rows: 12 bytes of a thread would
    // spill, 132 us for 64 requests of 512 to 8192 tokens, 126 with queries from shared memory).
    static constexpr bool kInRegs = D * kParts * kR <= 2048 && !(kParts == 2 && D == 128);
    static constexpr int kSmem = kRing + kQ + 1024;
    static_assert(kStepWarps * kR * D * 4 <= kRing, "outputs of the warps meet in the ring");
};

// Where a row's 16-byte chunk lies among the 16 rows that a tensor copy brings, in blocks of 128 bytes a row
// (64 for D = 64) that are swizzled by the row: eight lanes read chunks c, c + 2, .. c + 6 of two neighbouring rows
// of keys, and two chunks of four even (or odd) rows of values, without a bank twice (D = 64: twice).
template <int D> __device__ __forceinline__ int place(int row, int chunk) {
    if (D == 64) return row * 64 + (chunk ^ ((row >> 1) & 3)) * 16;
    return (chunk >> 3) * 2048 + row * 128 + ((chunk ^ row) & 7) * 16;
}
// The chunk of a key that thread c of a quad takes as its j-th, for steps 4j .. 4j + 3 of the first product.
template <int D> __device__ __forceinline__ int key_chunk(int j, int c) { return D == 64 ? c : (j >> 1) * 8 + 2 * c + (j & 1); }

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

struct StepPlan {
    int4 *tasks;     // [blocks][2]: the items that begin in this block and that began before it and go on in it: request (-1: none), head, blocks of it, blocks of it before this one
    char *parts;     // [blocks][2] Part
    CUtensorMap maps[2];  // keys, values: 16 rows of one page and head at a time
};

// Where unit `u` lies: request n and the units before it.
struct Share {
    int64_t n, before, total;
    bool ok;
};
__device__ __forceinline__ int64_t units_of(const Attn &a, int64_t n) {
    return max((__ldg(a.kv_lens + n) + kUnit - 1) / kUnit, 1);
}
// The request of the first unit of this block's share, and the share itself.
__device__ inline Share find_share(const Attn &a, int64_t *sums, int64_t *found, int64_t *per) {
    constexpr int kThreads = kStepWarps * 32;
    const int tid = threadIdx.x;
    int64_t mine = 0;
    bool ok = true;
    auto weight = [&](int64_t n) { return rows_of(a, n).y > 0 ? (int64_t)a.kv_heads * units_of(a, n) : 0; };
    for (int64_t n = tid; n < a.num_seqs; n += kThreads) {
        if (lengths_hold(a, n)) mine += weight(n);
        else ok = false;
    }
    Share s;
    s.ok = __syncthreads_and(ok);
    if (!s.ok) return s;
    block_sums<kThreads>(mine, sums, &s.total);
    *per = max((s.total + gridDim.x - 1) / gridDim.x, (int64_t)1);
    const int64_t u = (int64_t)blockIdx.x * *per;
    s.n = s.before = 0;
    if (u >= s.total) return s;
    int64_t carry = 0;
    for (int64_t n0 = 0; n0 < a.num_seqs; n0 += kThreads) {
        const int64_t n = n0 + tid, w = n < a.num_seqs ? weight(n) : 0;
        int64_t total;
        const int64_t end = carry + block_sums<kThreads>(w, sums, &total);
        if (u >= end - w && u < end) {
            found[0] = n;
            found[1] = end - w;
        }
        carry += total;
        if (carry > u) break;
    }
    __syncthreads();
    s.n = found[0];
    s.before = found[1];
    return s;
}

template <typename T, int D, int kCode, int kParts, bool kShaped, int kR>
__global__ void __launch_bounds__(kStepWarps * 32, (StepConfig<D, kParts, kR>::kBlocks)) attn_step_kernel(const __grid_constant__ Attn a, const __grid_constant__ StepPlan plan) {
    using C = StepConfig<D, kParts, kR>;
    using P = Part<kR, D>;
    extern __shared__ char unaligned[];
    char *const smem = (char *)(((uintptr_t)unaligned + 1023) & ~(uintptr_t)1023);
    __shared__ int64_t sums[kStepWarps], found[2];
    __shared__ float2 scales[kStepWarps][C::kStages];
    __shared__ __align__(8) uint64_t bars[kStepWarps][C::kStages];
    __shared__ float row_factor[kR], row_slope[kR];
    __shared__ float warp_ref[kStepWarps][kR], warp_sum[kStepWarps][kR];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int R0 = kR == 16 ? g : 2 * c, R1 = kR == 16 ? g + 8 : 2 * c + 1;  // this thread's rows
    const int in_page = (1 << a.log_page) - 1;

    if (lane < C::kStages) sm100::mbar_init(sm100::smem_u32(&bars[warp][lane]), 1);
    sm100::fence_mbar_init();
    bool fine = true;

    int64_t per;
    const Share share = find_share(a, sums, found, &per);
    if (blockIdx.x == 0 && tid == 0) *a.status = share.ok ? GDR_OK : GDR_ERR_BAD_SEQLENS;
    if (plan.tasks && tid < 2) plan.tasks[2 * blockIdx.x + tid] = make_int4(-1, 0, 0, 0);
    sm100::griddep_launch_dependents();
    if (!share.ok) return;

    char *const ring = smem + warp * C::kStages * C::kStage;
    const uint32_t ring_s = sm100::smem_u32(ring);
    uint32_t *const qfrag = (uint32_t *)(smem + C::kRing);

    int fetched = 0, used = 0, turn = 0;  // places in the ring, and the parity of the turn round it
    int64_t u = (int64_t)blockIdx.x * per, n = share.n, before = share.before;
    const int64_t end_u = min(share.total, u + per);
    while (u < end_u) {
        const int2 rows = rows_of(a, n);
        const int len = __ldg(a.kv_lens + n);
        const int64_t units = units_of(a, n), weight = rows.y > 0 ? a.kv_heads * units : 0;
        if (u >= before + weight) {  // (also a request without new tokens)
            before += weight;
            ++n;
            continue;
        }
        const int64_t rel = u - before;
        const int head = (int)(rel / units), ua = (int)(rel - head * units), ub = (int)min(units, ua + (end_u - u));
        const int nrows = rows.y * a.group;  // at most kR: few_rows, and no request has more than max_q tokens
        // the tokens that the last row may see
        const int past = len - rows.y;  // position of the first new token
        const int far = a.causal ? max(0, min(len, past + rows.y)) : len;
        const int first = ua * kUnit, last = min(far, ub * kUnit);
        const int count = last > first && fine ? ((last - first + 15) / 16 - warp + kStepWarps - 1) / kStepWarps : 0;  // of this warp

        // ---- the stream of tiles: page and scales of 32 tiles at a time, one per lane
        int64_t page = 0;
        float ks = 0.f, vs = 0.f;
        auto look_up = [&](int i0) {
            const int tok = first + (warp + (i0 + lane) * kStepWarps) * 16;
            if (tok < last) {
                const int p = __ldg(a.table + n * a.width + (tok >> a.log_page));
                const bool good = p >= 0 && p < a.pages;
                page = good ? p : 0;
                ks = good ? __ldg(a.ks + page * a.kv_heads + head) : __int_as_float(0x7fffffff);
                vs = good ? __ldg(a.vs + page * a.kv_heads + head) : __int_as_float(0x7fffffff);
            }
        };
        auto fetch = [&](int i) {  // tile i of this warp
            if (i < count) {
                if ((i & 31) == 0) look_up(i);
                const int64_t pg = __shfl_sync(~0u, page, i & 31);
                const float k1 = __shfl_sync(~0u, ks, i & 31), v1 = __shfl_sync(~0u, vs, i & 31);
                const int tok = first + (warp + i * kStepWarps) * 16;
                if (lane == 0) {
                    scales[warp][fetched] = make_float2(k1, v1);
                    const uint32_t dst = ring_s + fetched * C::kStage, bar = sm100::smem_u32(&bars[warp][fetched]);
                    sm100::mbar_arrive_expect_tx(bar, C::kStage);
                    const int row = head * (in_page + 1) + (tok & in_page);
#pragma unroll
                    for (int x = 0; x < D; x += 128) {
                        sm100::tma_load_3d(dst + x * 16, &plan.maps[0], bar, x, row, (int)pg);
                        sm100::tma_load_3d(dst + 16 * D + x * 16, &plan.maps[1], bar, x, row, (int)pg);
                    }
                }
                if (++fetched == C::kStages) fetched = 0;
            }
        };
#pragma unroll
        for (int i = 0; i < C::kStages - 1; ++i) fetch(i);

        // ---- queries: fp16 with a power of two per row, in the order of the first product
        if (tid < 8 * kR) {
            const int r = tid >> 3, part = tid & 7;
            constexpr int kMine = D / 8;
            float v[kMine];
            uint32_t most = 0;
            if (r < nrows) {
                const int h = head * a.group + r % a.group;
                const T *src = (const T *)a.q + (int64_t)(rows.x + r / a.group) * a.qs + (int64_t)h * D + part * kMine;
                constexpr int kVec = 16 / sizeof(T);
#pragma unroll
                for (int i = 0; i < kMine; i += kVec) {
                    const uint4 w = __ldg((const uint4 *)(src + i));
                    const T *e = (const T *)&w;
#pragma unroll
                    for (int x = 0; x < kVec; ++x) v[i + x] = to_f32<T>(e[x]);
                }
#pragma unroll
                for (int i = 0; i < kMine; ++i) most = max(most, __float_as_uint(v[i]) & 0x7fffffffu);
                if (part == 0) row_slope[r] = kShaped && a.slopes ? __ldg(a.slopes + h) : 0.f;
            } else {
#pragma unroll
                for (int i = 0; i < kMine; ++i) v[i] = 0.f;
                if (part == 0) row_slope[r] = 0.f;
            }
#pragma unroll
            for (int d = 1; d < 8; d *= 2) most = max(most, __shfl_xor_sync(~0u, most, d));
            const int shift = row_shift(most);
            const float up = two_to(shift);
            if (part == 0) row_factor[r] = two_to(-shift) * a.scale;
#pragma unroll
            for (int i = 0; i < kMine; i += 2) {
                const int d = part * kMine + i;
                // chunk d / 16 is the j-th of thread cc
                const int chunk = d >> 4, j = D == 64 ? 0 : (chunk >> 3) * 2 + (chunk & 1), cc = D == 64 ? chunk : (chunk & 7) >> 1;
                const int step = j * 4 + ((d & 15) >> 2), pair = (d & 3) >> 1;
                uint32_t *const to = kR == 16 ? qfrag + (step * 32 + (r & 7) * 4 + cc) * 4 + (r >> 3) + 2 * pair : qfrag + (step * 32 + r * 4 + cc) * 2 + pair;
                const float x = v[i] * up, y = v[i + 1] * up;
                const uint32_t hi = pack_f16(x, y);
                *to = hi;
                if (kParts == 2) {
                    const float2 f = unpack_f16(hi);
                    to[C::kSteps * 8 * kR] = pack_f16(x - f.x, y - f.y);
                }
            }
        }
        __syncthreads();
        constexpr int kQRegs = kR / 4;  // of a step
        uint32_t qreg[C::kInRegs ? kParts * C::kSteps : 1][kQRegs];
        auto query = [&](int s, uint32_t (&q)[kQRegs]) {
            if constexpr (kR == 16) {
                const uint4 w = *(const uint4 *)(qfrag + (s * 32 + lane) * 4);
                q[0] = w.x, q[1] = w.y, q[2] = w.z, q[3] = w.w;
            } else {
                const uint2 w = *(const uint2 *)(qfrag + (s * 32 + lane) * 2);
                q[0] = w.x, q[1] = w.y;
            }
        };
        if (C::kInRegs) {
#pragma unroll
            for (int s = 0; s < kParts * C::kSteps; ++s) query(s, qreg[s]);
        }
        const float f0 = row_factor[R0], f1 = row_factor[R1], slope0 = row_slope[R0], slope1 = row_slope[R1];
        const int p0 = past + R0 / a.group, p1 = past + R1 / a.group;
        const int lim0 = a.causal ? min(len, p0 + 1) : len, lim1 = a.causal ? min(len, p1 + 1) : len;
        const int sure = a.causal ? min(len, past + 1) : len;  // seen by every row

        const float inv_cap = kShaped && a.softcap > 0.f ? 1.f / a.softcap : 0.f;
        float ref0 = kNoRef, ref1 = kNoRef, l0 = 0.f, l1 = 0.f;
        float acc[D * kR / 128][4];
#pragma unroll
        for (int i = 0; i < D * kR / 128; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;

        for (int i = 0; i < count; ++i) {
            __syncwarp();  // (the place in the ring has been read)
            fetch(i + C::kStages - 1);
            fine = __all_sync(~0u, sm100::mbar_wait(sm100::smem_u32(&bars[warp][used]), turn));
            if (!fine) break;
            const char *const at = ring + used * C::kStage;
            const float2 sc = scales[warp][used];
            if (++used == C::kStages) {
                used = 0;
                turn ^= 1;
            }
            const int tok = first + (warp + i * kStepWarps) * 16;
            // scores: kR = 16: [8 tokens][token, row]; kR = 8: sums of even and of odd steps, [token][row]
            float s[2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                uint4 k[2];
#pragma unroll
                for (int t = 0; t < 2; ++t) k[t] = *(const uint4 *)(at + place<D>(8 * t + g, key_chunk<D>(j, c)));
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int step = j * 4 + w;
                    uint32_t q[kParts][kQRegs];
#pragma unroll
                    for (int x = 0; x < kParts; ++x) {
                        if (C::kInRegs) {
#pragma unroll
                            for (int y = 0; y < kQRegs; ++y) q[x][y] = qreg[x * C::kSteps + step][y];
                        } else {
                            query(x * C::kSteps + step, q[x]);
                        }
                    }
                    uint32_t lo[2], hi[2];
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        codes::to_f16x4<kCode>(w == 0 ? k[t].x : w == 1 ? k[t].y : w == 2 ? k[t].z : k[t].w, lo[t], hi[t]);
                    float mine[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};  // of this step (kParts == 2)
#pragma unroll
                    for (int x = kParts - 1; x >= 0; --x) {
                        if constexpr (kR == 16) {
                            mma_f16(kParts == 2 ? mine[0] : s[0], q[x], lo[0], hi[0]);
                            mma_f16(kParts == 2 ? mine[1] : s[1], q[x], lo[1], hi[1]);
                        } else {
                            const uint32_t tokens[4] = {lo[0], lo[1], hi[0], hi[1]};
                            mma_f16(kParts == 2 ? mine[w & 1] : s[w & 1], tokens, q[x][0], q[x][1]);
                        }
                    }
                    if (kParts == 2) {
#pragma unroll
                        for (int t = 0; t < 2; ++t)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (kR == 16 || t == (w & 1)) s[t][e] += mine[t][e];
                    }
                }
            }
            if (kR == 8) {
#pragma unroll
                for (int e = 0; e < 4; ++e) s[0][e] += s[1][e];
            }
            // this thread's scores x: the token behind tok, and whether its row is R1
            constexpr int kMine = kR / 2;
            auto token = [&](int x) { return kR == 16 ? 8 * (x >> 2) + 2 * c + (x & 1) : g + 8 * (x >> 1); };
            auto second = [](int x) { return kR == 16 ? (x & 2) != 0 : (x & 1) != 0; };
            float w[kMine];
            // scores in powers of two, with the value scale's
            const float lv = lg2(sc.y), rv = sc.y == sc.y ? __fdividef(1.f, sc.y) : 1.f;  // (a weight there is NaN, or 0 if masked)
            const float m0 = f0 * sc.x * (kShaped ? 1.f : kLog2e), m1 = f1 * sc.x * (kShaped ? 1.f : kLog2e);
            const bool edge = tok + 16 > sure;
            float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll
            for (int x = 0; x < kMine; ++x) {
                const float z = s[x >> 2][x & 3];
                const int j = tok + token(x);
                if (kShaped)
                    w[x] = fmaf(shaped<kParts == 2>(z * (second(x) ? m1 : m0), a.softcap, inv_cap, second(x) ? slope1 : slope0,
                                                    fabsf((float)((second(x) ? p1 : p0) - j))), kLog2e, lv);
                else
                    w[x] = fmaf(z, second(x) ? m1 : m0, lv);
                if (edge && j >= (second(x) ? lim1 : lim0)) w[x] = -INFINITY;
                (second(x) ? top1 : top0) = fmaxf(second(x) ? top1 : top0, w[x]);
            }
            if (__any_sync(~0u, top0 > ref0 + (kSpan + kSlack) || top1 > ref1 + (kSpan + kSlack))) {
                float t0 = top0, t1 = top1;
#pragma unroll
                for (int d = kR == 16 ? 1 : 4; d < (kR == 16 ? 4 : 32); d *= 2) {  // the threads of the same rows
                    t0 = fmaxf(t0, __shfl_xor_sync(~0u, t0, d));
                    t1 = fmaxf(t1, __shfl_xor_sync(~0u, t1, d));
                }
                const float n0 = t0 > ref0 + (kSpan + kSlack) ? t0 - kSpan : ref0, n1 = t1 > ref1 + (kSpan + kSlack) ? t1 - kSpan : ref1;
                const float d0 = ex2(ref0 - n0), d1 = ex2(ref1 - n1);
                ref0 = n0;
                ref1 = n1;
                l0 *= d0;
                l1 *= d1;
#pragma unroll
                for (int x = 0; x < D * kR / 128; ++x)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[x][e] *= (kR == 16 ? e >= 2 : e & 1) ? d1 : d0;
            }
            float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
            for (int x = 0; x < kMine; ++x) {
                w[x] = ex2(w[x] - (second(x) ? ref1 : ref0));
                (second(x) ? sum1 : sum0) += w[x];
            }
            l0 = fmaf(sum0, rv, l0);
            l1 = fmaf(sum1, rv, l1);
            // weights as an operand: kR = 16 as they lie; kR = 8 turned, from tokens by rows to rows by tokens
            uint32_t p[kParts][kMine / 2];
#pragma unroll
            for (int y = 0; y < kMine / 2; ++y) {
                p[0][y] = pack_f16(w[2 * y], w[2 * y + 1]);
                if (kParts == 2) {
                    const float2 f = unpack_f16(p[0][y]);
                    p[kParts - 1][y] = pack_f16(w[2 * y] - f.x, w[2 * y + 1] - f.y);
                }
            }
            if (kR == 8) {
#pragma unroll
                for (int x = 0; x < kParts; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y) asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %0;" : "+r"(p[x][y]));
            }
            // bytes behind the last token, and those that stand in for a page that is none, may be anything
            const bool unsure = tok + 16 > len || sc.y != sc.y;
#pragma unroll
            for (int j = 0; j < (D + 127) / 128; ++j) {
                constexpr int kWords = D == 64 ? 2 : 4;
                uint32_t v[4][kWords];
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const int r = 2 * c + (t & 1) + 8 * (t >> 1);
                    if constexpr (D == 64) {
                        const uint2 z = *(const uint2 *)(at + 16 * D + place<D>(r, g >> 1) + (g & 1) * 8);
                        v[t][0] = z.x, v[t][1] = z.y;
                    } else {
                        const uint4 z = *(const uint4 *)(at + 16 * D + place<D>(r, 8 * j + g));
                        v[t][0] = z.x, v[t][1] = z.y, v[t][2] = z.z, v[t][3] = z.w;
                    }
                    if (unsure && (sc.y != sc.y || tok + r >= len)) {
#pragma unroll
                        for (int z = 0; z < kWords; ++z) v[t][z] = 0;
                    }
                }
#pragma unroll
                for (int z = 0; z < kWords; ++z) {
                    uint32_t b[2][4];  // [token pair][dim of the word]
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        codes::to_f16x4<kCode>(__byte_perm(v[2 * t][z], v[2 * t + 1][z], 0x5140), b[t][0], b[t][1]);
                        codes::to_f16x4<kCode>(__byte_perm(v[2 * t][z], v[2 * t + 1][z], 0x7362), b[t][2], b[t][3]);
                    }
                    const int u = j * 4 * kWords + z * 4;
#pragma unroll
                    for (int x = 0; x < 4; x += kR == 16 ? 1 : 2) {
                        float(&sum)[4] = acc[kR == 16 ? u + x : (u + x) / 2];
                        float mine[4] = {0.f, 0.f, 0.f, 0.f};  // of this tile (kParts == 2)
#pragma unroll
                        for (int y = kParts - 1; y >= 0; --y) {
                            float(&to)[4] = kParts == 2 ? mine : sum;
                            if constexpr (kR == 16) {
                                mma_f16(to, p[y], b[0][x], b[1][x]);
                            } else {
                                const uint32_t dims[4] = {b[0][x], b[0][x + 1], b[1][x], b[1][x + 1]};
                                mma_f16(to, dims, p[y][0], p[y][1]);
                            }
                        }
                        if (kParts == 2) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) sum[e] += mine[e];
                        }
                    }
                }
            }
        }
        if (!fine && count > 0) {  // a wait that ran out: the copies under way are waited for, again with a limit, before the ring is used
            do {
                sm100::mbar_wait(sm100::smem_u32(&bars[warp][used]), turn);
                if (++used == C::kStages) {
                    used = 0;
                    turn ^= 1;
                }
            } while (used != fetched);
        }
        // ---- the warps' parts meet
#pragma unroll
        for (int d = kR == 16 ? 1 : 4; d < (kR == 16 ? 4 : 32); d *= 2) {
            l0 += __shfl_xor_sync(~0u, l0, d);
            l1 += __shfl_xor_sync(~0u, l1, d);
        }
        if (kR == 16 ? c == 0 : g == 0) {
            warp_ref[warp][R0] = ref0;
            warp_ref[warp][R1] = ref1;
            warp_sum[warp][R0] = l0;
            warp_sum[warp][R1] = l1;
        }
        __syncthreads();
        float *const outs = (float *)smem;  // [warp][kR][D]
        constexpr int kU = D == 64 ? 8 : 16;  // dims of a thread in a row of 8 groups
#pragma unroll
        for (int x = 0; x < D / 8; ++x) {
            const int dim = (x / kU) * 128 + x % kU;
            if constexpr (kR == 16) {  // column n of 8 is dim + kU n
                float *const to = outs + (warp * 16 + g) * D + dim + kU * (2 * c);
                to[0] = acc[x][0];
                to[kU] = acc[x][1];
                to[8 * D] = acc[x][2];
                to[8 * D + kU] = acc[x][3];
            } else {  // row n of 8 is
                float *const to = outs + (warp * 8 + 2 * c) * D + dim + kU * g;
                to[0] = acc[x / 2][2 * (x & 1)];
                to[D] = acc[x / 2][2 * (x & 1) + 1];
            }
        }
        __syncthreads();
        const bool whole = ua == 0 && ub == units;
        P *const part = whole ? nullptr : (P *)plan.parts + (2 * (int64_t)blockIdx.x + (ua == 0));
        constexpr int kQuads = D / 4;
        for (int x = tid; x < kR * kQuads; x += kStepWarps * 32) {
            const int r = x / kQuads, d = (x % kQuads) * 4;
            if (r >= nrows) break;
            float top = kNoRef;
#pragma unroll
            for (int w = 0; w < kStepWarps; ++w) top = fmaxf(top, warp_ref[w][r]);
            float l = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kStepWarps; ++w) {
                const float f = ex2(warp_ref[w][r] - top);
                const float4 y = *(const float4 *)(outs + (w * kR + r) * D + d);
                l = fmaf(warp_sum[w][r], f, l);
                o.x = fmaf(y.x, f, o.x);
                o.y = fmaf(y.y, f, o.y);
                o.z = fmaf(y.z, f, o.z);
                o.w = fmaf(y.w, f, o.w);
            }
            const float inv = l == 0.f ? 0.f : 1.f / l, sum2 = l == 0.f ? -INFINITY : log2f(l) + top;
            o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
            if (part) {
                *(float4 *)&part->o[r][d] = o;
                if (d == 0) part->lse2[r] = sum2;
            } else {
                const int64_t row = (int64_t)(rows.x + r / a.group) * a.heads + head * a.group + r % a.group;
                T *const to = (T *)a.o + row * D + d;
                if constexpr (sizeof(T) == 4) {
                    *(float4 *)to = o;
                } else {
                    const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x, o.y), hi = __floats2bfloat162_rn(o.z, o.w);
                    *(uint2 *)to = make_uint2(reinterpret_cast<const uint32_t &>(lo), reinterpret_cast<const uint32_t &>(hi));
                }
                if (d == 0 && a.lse) a.lse[row] = sum2 * kLn2;
            }
        }
        if (!whole && tid == (ua == 0 ? 0 : 1)) {
            const int from = (int)((u - ua) / per), to = (int)((u - ua + units - 1) / per);  // blocks
            plan.tasks[2 * blockIdx.x + tid] = make_int4((int)n, head, to - from + 1, (int)blockIdx.x - from);
        }
        u += ub - ua;
        sm100::fence_async_smem();  // (before copies into the ring again)
        __syncthreads();
    }
    if (!fine) *a.status = GDR_ERR_DEVICE_TIMEOUT;
}

// Adds the parts of items that several blocks worked on, 64 columns of a row at a time. Bound by latency: a thread's loads
// are under way together. Up to kAtOnce parts are a warp's work, and the block that begins the item does it all
// (shared out, 64 requests took 6 us longer). More are shared out to all blocks that had a part, and the warps
// take the parts in turn and meet in shared memory (one token behind 131,072 has 8 items of 76 parts, which 8 blocks took
// 12 us to read). Every sum is in a fixed order.
template <typename T, int D, int kR> __global__ void __launch_bounds__(256) join_parts_kernel(const __grid_constant__ Attn a, const __grid_constant__ StepPlan plan) {
    using P = Part<kR, D>;
    constexpr int kCols = D / 64, kAtOnce = 8;
    __shared__ float tops[8], sums[8], outs[8][64];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    sm100::griddep_wait();
    const int4 tasks[2] = {plan.tasks[2 * blockIdx.x], plan.tasks[2 * blockIdx.x + 1]};
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        const int4 task = which ? tasks[1] : tasks[0];
        if (task.x < 0) continue;
        const int head = task.y, blocks = task.z, mine = task.w;
        const int2 rows = rows_of(a, task.x);
        const int units = rows.y * a.group * kCols;
        const bool many = blocks > kAtOnce;
        if (!many && mine > 0) continue;
        const int ways = many ? 8 : 1, abreast = 8 / ways, step = many ? blocks : abreast;  // warps for the parts of a unit; units at a time
        // the first block's part is its second one, that of the others their first
        const P *const parts = (const P *)plan.parts + 2 * ((int64_t)blockIdx.x - mine);
        for (int u0 = mine; u0 < units; u0 += step) {
            const int u = u0 + warp / ways, r = u / kCols, d = u % kCols * 64 + lane * 2;
            float top = -INFINITY, l = 0.f;
            float2 o = make_float2(0.f, 0.f);
#pragma unroll 1
            for (int i0 = warp % ways; u < units && i0 < blocks; i0 += ways * kAtOnce) {
                float lse[kAtOnce];
                float2 y[kAtOnce];
#pragma unroll
                for (int j = 0; j < kAtOnce; ++j) {
                    const int i = i0 + ways * j;
                    const P *const p = parts + 2 * i + (i == 0);
                    lse[j] = i < blocks ? p->lse2[r] : -INFINITY;
                    y[j] = i < blocks ? *(const float2 *)&p->o[r][d] : make_float2(0.f, 0.f);
                }
                float most = top;
#pragma unroll
                for (int j = 0; j < kAtOnce; ++j) most = fmaxf(most, lse[j]);
                const float base = most == -INFINITY ? 0.f : most, by = ex2(top - base);
                top = most;
                l *= by;
                o = make_float2(o.x * by, o.y * by);
#pragma unroll
                for (int j = 0; j < kAtOnce; ++j) {
                    const float f = ex2(lse[j] - base);
                    l += f;
                    o = make_float2(fmaf(y[j].x, f, o.x), fmaf(y[j].y, f, o.y));
                }
            }
            *(float2 *)&outs[warp][lane * 2] = o;
            if (lane == 0) {
                tops[warp] = top;
                sums[warp] = l;
            }
            __syncthreads();
            for (int x = threadIdx.x; x < abreast * 64 && u0 + x / 64 < units; x += 256) {
                const int first = x / 64 * ways, unit = u0 + x / 64;
                float most = -INFINITY, sum = 0.f, z = 0.f;
                for (int w = first; w < first + ways; ++w) most = fmaxf(most, tops[w]);
                const float base = most == -INFINITY ? 0.f : most;
                for (int w = first; w < first + ways; ++w) {
                    const float f = ex2(tops[w] - base);
                    sum = fmaf(sums[w], f, sum);
                    z = fmaf(outs[w][x % 64], f, z);
                }
                const int at = unit / kCols, dim = unit % kCols * 64 + x % 64;
                const int64_t row = (int64_t)(rows.x + at / a.group) * a.heads + head * a.group + at % a.group;
                ((T *)a.o)[row * D + dim] = from_f32<T>(sum == 0.f ? 0.f : z * (1.f / sum));
                if (dim == 0 && a.lse) a.lse[row] = (sum == 0.f ? -INFINITY : log2f(sum) + base) * kLn2;
            }
            __syncthreads();
        }
    }
}

template <typename T, int D, int kCode, int kParts, bool kShaped, int kR>
int launch_step_kernel(const Attn &a, const StepPlan &plan, bool join, cudaStream_t s) {
    using C = StepConfig<D, kParts, kR>;
    constexpr int kBlocks = kSms * C::kBlocks;
    const auto kernel = attn_step_kernel<T, D, kCode, kParts, kShaped, kR>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess) return GDR_ERR_CUDA;
    kernel<<<kBlocks, kStepWarps * 32, C::kSmem, s>>>(a, plan);
    if (cudaGetLastError() != cudaSuccess) return GDR_ERR_CUDA;
    if (!join) return GDR_OK;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kBlocks);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, join_parts_kernel<T, D, kR>, a, plan));
}

template <int D> int launch_step_d(const Attn &a, int codes, int dtype, void *ws, cudaStream_t s) {
    // (no request has more than one unit: no item is split)
    const bool join = ((a.width << a.log_page) + kUnit - 1) / kUnit > 1;
    StepPlan plan;
    plan.tasks = join ? (int4 *)ws : nullptr;
    plan.parts = (char *)ws + kTaskBytes;
    if (!map_cache(&plan.maps[0], a.kc, a, D, 16, true) || !map_cache(&plan.maps[1], a.vc, a, D, 16, true)) return GDR_ERR_CUDA;
    const bool shaped = a.softcap > 0.f || a.slopes;
    const bool e4m3 = codes == GDR_CODE_E4M3;
    const bool few = a.max_q * a.group <= 8;
#define GDR_STEP_ROWS(T, CODE, PARTS, ROWS) \
    (shaped ? launch_step_kernel<T, D, CODE, PARTS, true, ROWS>(a, plan, join, s) : launch_step_kernel<T, D, CODE, PARTS, false, ROWS>(a, plan, join, s))
#define GDR_STEP(T, CODE, PARTS) return few ? GDR_STEP_ROWS(T, CODE, PARTS, 8) : GDR_STEP_ROWS(T, CODE, PARTS, 16)
    if (dtype == GDR_F32) {
        if (e4m3) GDR_STEP(float, GDR_CODE_E4M3, 2);
        GDR_STEP(float, GDR_CODE_INT8, 2);
    }
    if (e4m3) GDR_STEP(__nv_bfloat16, GDR_CODE_E4M3, 1);
    GDR_STEP(__nv_bfloat16, GDR_CODE_INT8, 1);
#undef GDR_STEP
#undef GDR_STEP_ROWS
}

template <int D> size_t step_bytes_d() {
    return kTaskBytes + (size_t)kSms * 4 * 2 * sizeof(Part<16, D>);
}

}  // namespace cattn
}  // namespace gdr
