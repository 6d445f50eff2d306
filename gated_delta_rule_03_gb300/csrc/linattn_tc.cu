// linattn_tc.cu -- the mix of linear attention (linattn.cuh) on the 5th-generation tensor
// cores, for bf16 inputs with d_x, d_z of 64 or 128 per CTA.
//
// One CTA per (segment, head, 128 columns of d_v) walks its segment in chunks of C = 128
// tokens. Per chunk, with the decay weights of linattn.cuh:
//   P  = X Y^T            masked and weighted into bf16, kept in TMEM as an A operand
//   Oi = X E              E: the state entering the chunk, as bf16 in shared memory
//   Oa = P Z
//   U  = Yw^T Z           Yw: the rows of Y times w_upd
//   out = s_inter w_out Oi + Oa,   E <- lam^n E + U
// Nothing that the tensor cores compute for a chunk depends on the state but Oi: the state
// itself lives in fp32 registers, so that the sequential part of a chunk is one fused
// multiply-add per element and its copy to shared memory. Every weight is at most 1.
//
// Rounding. X, Y and Z are used as they are. P and the copy of E that Oi reads are rounded
// to bf16 once each, as a product's operand has to be; either costs an output element
// 2^-8 of the sum of its terms' sizes at most, like the output's own rounding. Yw is kept
// as two bf16 parts, 16 bits: a term of the state is off by 2^-16 at most, where one part
// would cost the outputs as much again as E's own rounding. U is summed chunk by chunk and
// added to E in fp32: a sum over a whole segment in the tensor cores would lose more.
//
// Shared memory: a ring of five 32 KB tiles for X, Y, Z (TMA, 128-byte swizzle), E in bf16,
// 32 KB for the lower part of Yw. The upper part overwrites Y once P has been taken.
//
// Warps 0-7: P into TMEM, then the output rows. Warps 8-15: Yw, the state (64 registers of a
// thread's 96 hold it). Warp 16: the loads. Warp 17: the MMAs, in the order P, Oi, U of the first 64 tokens, Oa, U of the
// others: each conversion runs behind products that do not need it.
#include "linattn.cuh"
#include "tc_common.cuh"

namespace gdr {
namespace linattn {
namespace {

using namespace sm100;
using tc::pack_bf16x2;

constexpr int C = 128;
constexpr uint32_t TILE = 32768, BLOCK = 16384;  // a tile: two blocks of 64 columns
constexpr int kSlots = 5;
constexpr uint32_t OFF_E = kSlots * TILE, OFF_LOW = OFF_E + TILE, OFF_END = OFF_LOW + TILE;
constexpr uint32_t kSmem = OFF_END + 1024;  // slack for the 1024-byte alignment
constexpr uint32_t TM_P = 0, TM_OA = 128, TM_OI = 256, TM_U = 384, TM_COLS = 512;
constexpr int kRowWarps = 8, kStateWarps = 8, kThreads = 32 * (kRowWarps + kStateWarps + 2);
constexpr int kRowThreads = 32 * kRowWarps, kStateThreads = 32 * kStateWarps;
constexpr int kLoadWarp = kRowWarps + kStateWarps;

struct TcMix {
    int mx, my, mz;              // maps
    int xg, yg, zg;              // heads sharing one
    int xstep, ystep, zstep;     // columns from one slice to the next
    int xb, zb;                  // blocks of 64 columns of x (and y), of z
    void *out;
    int64_t out_row, out_h, out_s;  // elements from one token, head, slice to the next
    bool out_f32, turned, backward;
    int astep, bstep;            // rows and columns of the state from one slice to the next
    float s_intra, s_inter, s_state;
    const float *start, *R;
    float *end, *R_out;
};
struct TcArgs {
    CUtensorMap maps[4];
    Plan p;
    TcMix mix[3];
    int count, slices;
    int pitch;     // d_v: columns of a state matrix in memory
    int64_t mat;   // its elements
    long long wait_cycles;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// mbarrier wait that sleeps in hardware until the phase ends, or about 0.1 ms.
__device__ __forceinline__ bool mbar_sleep(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(100000u)
        : "memory");
    return ok != 0;
}

// Two fp32 at a time.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<const uint64_t &>(a)), "l"(reinterpret_cast<const uint64_t &>(b)));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<const uint64_t &>(a)), "l"(reinterpret_cast<const uint64_t &>(b)),
          "l"(reinterpret_cast<const uint64_t &>(c)));
    return d;
}

// The weights of a chunk's rows, for n tokens, as two bf16 parts each (the larger in the
// low half); rows behind the last token get 0. By 256 threads, which meet at barrier 1.
__device__ __forceinline__ void row_weights(uint32_t *table, int n, bool backward, float l2, float s, int id) {
    asm volatile("bar.sync 1, 256;" ::: "memory");  // the table before has been used
    if (id < C) {
        const float x = id < n ? s * decay_pow(l2, (float)(backward ? id + 1 : n - 1 - id)) : 0.f;
        table[id] = pack_bf16x2(x, x - __bfloat162float(__float2bfloat16_rn(x)));
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");
}

// Rows [64 half, 64 half + 64) of the Y tile times their weights, as two bf16 parts: the
// larger in place, the other to `low` (the same places in a tile of its own). With the
// weight w = wh + wl (bf16 each), hi = round(y wh), lo = y wh - hi (exact: what is left of
// 16 bits) + y wl. `id` of 256 threads.
template <int HALF>
__device__ __forceinline__ void weigh_half(unsigned char *y, unsigned char *low, int blocks, int n,
                                           const uint32_t *table, int id) {
    const uint32_t at = (64 * HALF + (id >> 3)) * 128 + (id & 7) * 16;
#pragma unroll
    for (int it = 0; it < 2; ++it) {
        const int r = 64 * HALF + 32 * it + (id >> 3);
        const __nv_bfloat162 w = reinterpret_cast<const __nv_bfloat162 &>(table[r]);
        const __nv_bfloat162 wh = __low2bfloat162(w), wl = __high2bfloat162(w);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            if (b >= blocks) break;
            uint4 lo, in = *reinterpret_cast<const uint4 *>(y + b * BLOCK + at + it * 4096);
            if (r >= n) in = make_uint4(0, 0, 0, 0);  // (whatever lies behind the last token)
            uint32_t *pi = &in.x, *pl = &lo.x;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 k = reinterpret_cast<const __nv_bfloat162 &>(pi[e]);
                const __nv_bfloat162 h = __hmul2_rn(k, wh);
                const __nv_bfloat162 l = __hfma2(k, wl, __hfma2(k, wh, __hneg2(h)));
                pi[e] = reinterpret_cast<const uint32_t &>(h);
                pl[e] = reinterpret_cast<const uint32_t &>(l);
            }
            *reinterpret_cast<uint4 *>(y + b * BLOCK + at + it * 4096) = in;
            *reinterpret_cast<uint4 *>(low + b * BLOCK + at + it * 4096) = lo;
        }
    }
}

// Rows n .. 127 of a tile become zero.
__device__ __forceinline__ void clear_behind(unsigned char *tile, int blocks, int n, int id) {
    for (int e = id; e < (C - n) * 8 * blocks; e += kStateThreads) {
        const int b = e / ((C - n) * 8), r = n + e / 8 % (C - n);
        *reinterpret_cast<uint4 *>(tile + b * BLOCK + r * 128 + (e & 7) * 16) = make_uint4(0, 0, 0, 0);
    }
}

// Shared-memory descriptors (sm100.cuh's, with 1024 bytes between groups of 8 rows) by
// their lower words: the address moves there, the upper word is the same for all.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_k(uint32_t at) { return (at >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_mn(uint32_t at) { return (at >> 4) | ((BLOCK >> 4) << 16); }

// D (+)= A B, both in shared memory; the operands' places `a` and `b` bytes further on.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t da, uint32_t a, uint32_t db, uint32_t b,
                                       uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
        "r"(da + (a >> 4)), "r"(db + (b >> 4)), "r"(idesc), "r"((uint32_t)add), "r"(kDescHigh)
        : "memory");
}
// A in tensor memory.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t db, uint32_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(db + (b >> 4)), "r"(idesc), "r"((uint32_t)add), "r"(kDescHigh)
        : "memory");
}

// The MMAs of U over 64 tokens, the smaller part first. Descriptors of the whole tiles.
__device__ __forceinline__ void issue_update(uint32_t d, uint32_t y, uint32_t low, uint32_t z, int half,
                                             uint32_t idesc) {
#pragma unroll
    for (int i = 1; i >= 0; --i)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            const uint32_t at = (4 * half + kk) * 2048;
            mma_ss(d, i ? low : y, at, z, at, idesc, !(half == 0 && i == 1 && kk == 0));
        }
}

// E <- w E + 64 columns of this thread's TMEM lane.
__device__ __forceinline__ void add_update(float2 (&E)[32], float w, uint32_t taddr) {
    const float2 w2 = make_float2(w, w);
#pragma unroll
    for (int part = 0; part < 4; ++part) {  // (16 at a time: registers)
        float u[16];
        tmem_load16(taddr + 16 * part, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) E[8 * part + j] = fma2(w2, E[8 * part + j], make_float2(u[2 * j], u[2 * j + 1]));
    }
}

// Four lanes that hold 64 bytes each of a row of their own: afterwards bytes 16 i .. of lane
// q's registers are bytes 16 q .. of lane i's row.
__device__ __forceinline__ void turn_four(uint32_t (&p)[16], int lane) {
#pragma unroll
    for (int step = 1; step < 4; step *= 2) {
        const bool up = lane & step;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i & step) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                // the lower lane sends its part i + step, the upper one its part i
                const uint32_t mine = up ? p[4 * i + e] : p[4 * (i + step) + e];
                const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, step);
                if (up) p[4 * i + e] = other;
                else p[4 * (i + step) + e] = other;
            }
        }
    }
}

// A thread's 64 columns of state row a, from or to memory.
struct StateAt {
    int64_t first, step;  // element of column 0, elements from one column to the next
};
__device__ __forceinline__ StateAt state_row(const TcArgs &A, const TcMix &m, int slice, int a, int b) {
    const int64_t aa = a + m.astep * slice, bb = b + m.bstep * slice;
    return m.turned ? StateAt{bb * A.pitch + aa, A.pitch} : StateAt{aa * A.pitch + bb, 1};
}
__device__ __forceinline__ void read_state(float2 (&E)[32], const float *S, const StateAt &at, float w) {
    if (at.step == 1) {
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
            if (j % 8 == 0) asm volatile("" ::: "memory");  // (four loads at a time: registers)
            const float4 x = *reinterpret_cast<const float4 *>(S + at.first + 2 * j);
            E[j].x = fmaf(w, x.x, E[j].x);
            E[j].y = fmaf(w, x.y, E[j].y);
            E[j + 1].x = fmaf(w, x.z, E[j + 1].x);
            E[j + 1].y = fmaf(w, x.w, E[j + 1].y);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            if (j % 8 == 0) asm volatile("" ::: "memory");
            E[j].x = fmaf(w, S[at.first + 2 * j * at.step], E[j].x);
            E[j].y = fmaf(w, S[at.first + (2 * j + 1) * at.step], E[j].y);
        }
    }
}
__device__ __forceinline__ void write_state(const float2 (&E)[32], float *S, const StateAt &at) {
    if (at.step == 1) {
#pragma unroll
        for (int j = 0; j < 32; j += 2)
            *reinterpret_cast<float4 *>(S + at.first + 2 * j) = make_float4(E[j].x, E[j].y, E[j + 1].x, E[j + 1].y);
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            S[at.first + 2 * j * at.step] = E[j].x;
            S[at.first + (2 * j + 1) * at.step] = E[j].y;
        }
    }
}

// What a block of either kernel works on.
struct Work {
    Segment s;
    int role, slice, h, chunks;
    int64_t item;
};

enum { B_FULL = 0, B_EMPTY = kSlots, B_P = 2 * kSlots, B_PREADY, B_Y0, B_Y1, B_U, B_EREADY,
       B_O, B_OFREE, B_DRAIN, B_COUNT };

__global__ void __launch_bounds__(kThreads, 1) mix_tc_kernel(const __grid_constant__ TcArgs A) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t base = smem_u32(sm);
    __shared__ Segment found;
    __shared__ __align__(8) uint64_t bars[B_COUNT];
    __shared__ uint32_t tmem_slot;
    __shared__ int gave_up;
    __shared__ uint32_t row_w[C];
    __shared__ __align__(16) float step_pow[32];  // lam^(31-j), or lam^j from last to first
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    Work w;
    w.role = (int)(blockIdx.x % A.count);
    const int64_t rest = blockIdx.x / A.count;
    w.slice = (int)(rest % A.slices);
    w.h = (int)(rest / A.slices % A.p.H);
    w.item = rest / A.slices / A.p.H;
    bool bad;
    w.s = locate(A.p, w.item, &found, &bad);
    if (blockIdx.x == 0 && tid == 0 && A.p.first) A.p.status[0] = bad ? GDR_ERR_BAD_SEQLENS : GDR_OK;
    if (bad || w.s.seq < 0) return;
    const TcMix &m = A.mix[w.role];
    const float l2 = log2_decay(A.p.log_decay[w.h]);
    const int chunks = (int)((w.s.tokens + C - 1) / C);
    const bool ends = m.end && w.s.f == (m.backward ? 0 : w.s.n - 1);
    auto chunk_of = [&](int cc) { return m.backward ? chunks - 1 - cc : cc; };
    auto tokens_of = [&](int c) {
        const int64_t r = w.s.tokens - (int64_t)c * C;
        return (int)(r < C ? r : C);
    };
    auto slot = [&](int t) { return base + (uint32_t)(t % kSlots) * TILE; };
    auto slot_p = [&](int t) { return sm + (uint32_t)(t % kSlots) * TILE; };

    if (tid == 0) {
        for (int i = 0; i < 2 * kSlots; ++i) mbar_init(bar(i), 1);
        mbar_init(bar(B_P), 1);
        mbar_init(bar(B_PREADY), kRowThreads);
        mbar_init(bar(B_Y0), kStateThreads);
        mbar_init(bar(B_Y1), kStateThreads);
        mbar_init(bar(B_U), 1);
        mbar_init(bar(B_EREADY), kStateThreads);
        mbar_init(bar(B_O), 1);
        mbar_init(bar(B_OFREE), kRowThreads);
        mbar_init(bar(B_DRAIN), 1);
        fence_mbar_init();
        gave_up = 0;
        prefetch_tensormap(&A.maps[m.mx]);
        prefetch_tensormap(&A.maps[m.my]);
        prefetch_tensormap(&A.maps[m.mz]);
    }
    if (tid < 32) {
        step_pow[tid] = decay_pow(l2, (float)(m.backward ? tid : 31 - tid));
        tmem_alloc(smem_u32(&tmem_slot), TM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    // A bounded wait: the first that runs out ends the others too.
    volatile int *stop = &gave_up;
    auto wait = [&](int b, int phase) -> bool {
        if (mbar_sleep(bar(b), phase & 1)) return true;
        const long long t0 = clock64();
        while (!mbar_sleep(bar(b), phase & 1)) {
            if (*stop) return false;
            if (clock64() - t0 > A.wait_cycles) {
                *stop = 1;
                A.p.status[0] = GDR_ERR_DEVICE_TIMEOUT;
                return false;
            }
        }
        return true;
    };

    // by a whole warp: converged again, and of one mind
    auto warp_wait = [&](int b, int phase) -> bool { return __all_sync(0xffffffffu, wait(b, phase)); };

    if (warp < kRowWarps) {
        // ------------------------------------------------ P, then the output rows
        // two warps per lane quarter, each with half of the columns
        const int quarter = warp & 3, side = warp >> 2;
        const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16);
        const int t = 32 * quarter + lane;  // row of the chunk
        // lam^(t-i) = lam^(t - 32b - 31) lam^(31 - (i - 32b)): the first is at most 1 off the
        // diagonal block and at most lam^-31 on it, a float unless lam < 1/16 (`steep`)
        const bool steep = l2 < -4.f;
        float2 far[2];
#pragma unroll
        for (int bb = 0; bb < 2; ++bb) {
            const int b = 2 * side + bb;
            far[bb].x = far[bb].y = m.s_intra * ex2(l2 * (float)(m.backward ? 32 * b - t : t - 32 * b - 31));
        }
        for (int cc = 0; cc < chunks; ++cc) {
            const int c = chunk_of(cc), n = tokens_of(c);
            if (!warp_wait(B_P, cc)) break;
            tc_fence_after();
#pragma unroll
            for (int bb = 0; bb < 2; ++bb) {
                const int b = 2 * side + bb;
                uint32_t out[16];
                if (m.backward ? b < quarter : b > quarter) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) out[j] = 0;
                } else {
                    float v[32];
                    tmem_load32(lanes + TM_P + 32 * b, v);
                    if (steep && b == quarter) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            v[j] *= m.s_intra * ex2(l2 * (float)(m.backward ? j - lane : lane - j));
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            const float4 g = *reinterpret_cast<const float4 *>(&step_pow[j]);
                            const float2 x = mul2(make_float2(v[j], v[j + 1]), mul2(far[bb], make_float2(g.x, g.y)));
                            const float2 z = mul2(make_float2(v[j + 2], v[j + 3]), mul2(far[bb], make_float2(g.z, g.w)));
                            v[j] = x.x;
                            v[j + 1] = x.y;
                            v[j + 2] = z.x;
                            v[j + 3] = z.y;
                        }
                    }
                    // columns beyond the diagonal; from last to first, columns behind the last token
                    const int first = m.backward ? t - 32 * b : 0, last = m.backward ? n - 1 - 32 * b : t - 32 * b;
                    if (b == quarter || (m.backward && 32 * b + 32 > n)) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = j >= first && j <= last ? v[j] : 0.f;
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j) out[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
                }
                // the bf16 copy of a block overwrites the first half of its own columns
                tmem_store16(lanes + TM_P + 32 * b, out);
            }
            tc_fence_before();
            mbar_arrive(bar(B_PREADY));
            if (!warp_wait(B_O, cc)) break;
            tc_fence_after();
            const float wo = m.s_inter * decay_pow(l2, (float)(m.backward ? (t < n ? n - 1 - t : 0) : t + 1));
            const float2 wo2 = make_float2(wo, wo);
            // rows leave four at a time, 16 bytes of a row per lane
            const int r0 = 32 * quarter + (lane & ~3);
            const int64_t at = (w.s.begin + (int64_t)c * C + r0) * m.out_row + w.h * m.out_h + w.slice * m.out_s;
#pragma unroll 1
            for (int b = m.zb * side; b < m.zb * side + m.zb; ++b) {
                float oi[32], oa[32];
                tmem_load32(lanes + TM_OA + 32 * b, oa);
                tmem_load32(lanes + TM_OI + 32 * b, oi);
                if (b == m.zb * side + m.zb - 1) {
                    tc_fence_before();
                    mbar_arrive(bar(B_OFREE));
                }
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    const float2 x = fma2(wo2, make_float2(oi[j], oi[j + 1]), make_float2(oa[j], oa[j + 1]));
                    oa[j] = x.x;
                    oa[j + 1] = x.y;
                }
                if (m.out_f32) {
                    float *o = (float *)m.out + at + 32 * b;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t p[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) p[j] = __float_as_uint(oa[16 * half + j]);
                        turn_four(p, lane);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (r0 + i < n)
                                *reinterpret_cast<uint4 *>(o + i * m.out_row + 16 * half + 4 * (lane & 3)) =
                                    make_uint4(p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3]);
                    }
                } else {
                    uint32_t p[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) p[j] = pack_bf16x2(oa[2 * j], oa[2 * j + 1]);
                    turn_four(p, lane);
                    __nv_bfloat16 *o = (__nv_bfloat16 *)m.out + at + 32 * b;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (r0 + i < n)
                            *reinterpret_cast<uint4 *>(o + i * m.out_row + 8 * (lane & 3)) =
                                make_uint4(p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3]);
                }
                __syncwarp();
            }
        }
    } else if (warp < kLoadWarp) {
        // ------------------------------------------------ Yw and the state
        const int id = tid - kRowThreads;
        const int a = 32 * (warp & 3) + lane, b0 = 64 * (id / 128);  // this thread's row and columns
        const bool mine = a < 64 * m.xb && b0 < 64 * m.zb;
        const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const StateAt st = state_row(A, m, w.slice, a, b0);
        float2 E[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) E[j] = make_float2(0.f, 0.f);
        if (mine) {
            if (m.start) {
                const int64_t dist = m.backward ? w.s.behind : (int64_t)w.s.f * A.p.seg;
                read_state(E, m.start + ((int64_t)w.s.seq * A.p.H + w.h) * A.mat, st, decay_pow(l2, (float)dist));
            }
            for (int g = m.backward ? w.s.f + 1 : 0; m.R && g < (m.backward ? w.s.n : w.s.f); ++g) {
                const int apart = m.backward ? g - 1 - w.s.f : w.s.f - 1 - g;
                read_state(E, m.R + ((w.s.item0 + g) * A.p.H + w.h) * A.mat, st, decay_pow(l2, (float)(apart * A.p.seg)));
            }
        }
        // rows a of E as the K rows of a B operand: columns b0 .. b0 + 63, one swizzled block
        auto publish = [&]() {
            if (b0 < 64 * m.zb) {
                unsigned char *row = sm + OFF_E + (b0 / 64) * BLOCK + a * 128;
#pragma unroll
                for (int j = 0; j < 32; j += 4)
                    *reinterpret_cast<uint4 *>(row + ((((j >> 2) ^ a) & 7) << 4)) =
                        make_uint4(pack_bf16x2(E[j].x, E[j].y), pack_bf16x2(E[j + 1].x, E[j + 1].y),
                                   pack_bf16x2(E[j + 2].x, E[j + 2].y), pack_bf16x2(E[j + 3].x, E[j + 3].y));
            }
            fence_async_smem();
            mbar_arrive(bar(B_EREADY));
        };
        if (chunks > 0) publish();
        int weighed = 0;  // the length that the weights are for
        unsigned char *low = sm + OFF_LOW;
        for (int cc = 0; cc < chunks; ++cc) {
            const int c = chunk_of(cc), n = tokens_of(c);
            const bool need = cc + 1 < chunks || ends;
            if (!warp_wait(B_P, cc)) break;  // P has been taken: Y may be overwritten
            if (!warp_wait(B_FULL + (3 * cc + 1) % kSlots, (3 * cc + 1) / kSlots)) break;
            if (n < C) {
                if (!warp_wait(B_FULL + (3 * cc + 2) % kSlots, (3 * cc + 2) / kSlots)) break;
                clear_behind(slot_p(3 * cc + 2), m.zb, n, id);
            }
            unsigned char *y = slot_p(3 * cc + 1);
            if (n != weighed) row_weights(row_w, weighed = n, m.backward, l2, m.s_state, id);
            if (need) weigh_half<0>(y, low, m.xb, n, row_w, id);
            fence_async_smem();
            mbar_arrive(bar(B_Y0));
            if (!need) continue;  // (the last chunk)
            weigh_half<1>(y, low, m.xb, n, row_w, id);
            fence_async_smem();
            mbar_arrive(bar(B_Y1));
            if (!warp_wait(B_U, cc)) break;
            tc_fence_after();
            if (b0 < 64 * m.zb) add_update(E, decay_pow(l2, (float)n), lanes + TM_U + b0);
            tc_fence_before();
            if (cc + 1 < chunks) publish();
        }
        if (ends && mine && !*stop)
            write_state(E, m.end + ((int64_t)w.s.seq * A.p.H + w.h) * A.mat, st);
    } else if (warp == kLoadWarp) {
        // ------------------------------------------------ the loads
        if (lane == 0) {
            int issued = 0;
            for (int cc = 0; cc < chunks; ++cc) {
                const int t0 = (int)(w.s.begin + (int64_t)chunk_of(cc) * C);
                bool ok = true;
                for (int i = 0; i < 3 && ok; ++i) {
                    const int t = 3 * cc + i;
                    if (t >= kSlots && !(ok = wait(B_EMPTY + t % kSlots, t / kSlots - 1))) break;
                    const CUtensorMap *map = &A.maps[i == 0 ? m.mx : (i == 1 ? m.my : m.mz)];
                    const int col = w.slice * (i == 0 ? m.xstep : (i == 1 ? m.ystep : m.zstep));
                    const int head = w.h / (i == 0 ? m.xg : (i == 1 ? m.yg : m.zg));
                    const int blocks = i == 2 ? m.zb : m.xb;
                    const uint32_t full = bar(B_FULL + t % kSlots);
                    mbar_arrive_expect_tx(full, blocks * BLOCK);
                    for (int b = 0; b < blocks; ++b)
                        tma_load_3d(slot(t) + b * BLOCK, map, full, col + 64 * b, head, t0);
                    ++issued;
                }
                if (!ok) break;
            }
            // after a wait gave up: every load issued has landed before the block ends
            for (int t = issued > kSlots ? issued - kSlots : 0; *stop && t < issued; ++t)
                mbar_wait_for(bar(B_FULL + t % kSlots), (t / kSlots) & 1, A.wait_cycles);
        }
    } else if (lane == 0) {
        // ------------------------------------------------ the MMAs
        const uint32_t id_pp = idesc_bf16(128, 128, 0, 0);           // A and B K-major
        const uint32_t id_o = idesc_bf16(128, 64 * m.zb, 0, 1);      // B with rows of z along K
        const uint32_t id_u = idesc_bf16(128, 64 * m.zb, 1, 1);      // A turned: rows of y along K
        const bool wide = m.xb == 2;
        for (int cc = 0; cc < chunks; ++cc) {
            const bool need = cc + 1 < chunks || ends;
            const int tx = 3 * cc, ty = tx + 1, tz = tx + 2;
            uint32_t x = desc_k(slot(tx)), y = desc_k(slot(ty)), yt = desc_mn(slot(ty)), z = desc_mn(slot(tz));
            uint32_t E = desc_mn(base + OFF_E), low = desc_mn(base + OFF_LOW);
            // (kept from being added up ahead of the loop: registers)
            asm volatile("" : "+r"(x), "+r"(y), "+r"(yt), "+r"(z), "+r"(E), "+r"(low));
            if (!wait(B_FULL + tx % kSlots, tx / kSlots) || !wait(B_FULL + ty % kSlots, ty / kSlots)) break;
            if (cc > 0 && !wait(B_O, cc - 1)) break;  // P's columns have been read
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
                const uint32_t at = (kk >> 2) * BLOCK + (kk & 3) * 32;
                if (kk < 4 || wide) mma_ss(tmem + TM_P, x, at, y, at, id_pp, kk > 0);
            }
            mma_commit(bar(B_P));
            if (!wait(B_EREADY, cc) || (cc > 0 && !wait(B_OFREE, cc - 1))) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
                if (kk < 4 || wide)
                    mma_ss(tmem + TM_OI, x, (kk >> 2) * BLOCK + (kk & 3) * 32, E, kk * 2048, id_o, kk > 0);
            mma_commit(bar(B_EMPTY + tx % kSlots));
            if (!wait(B_FULL + tz % kSlots, tz / kSlots) || !wait(B_Y0, cc)) break;
            tc_fence_after();
            if (need) issue_update(tmem + TM_U, yt, low, z, 0, id_u);
            if (!wait(B_PREADY, cc)) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
                mma_ts(tmem + TM_OA, tmem + TM_P + 32 * (kk >> 1) + 8 * (kk & 1), z, kk * 2048, id_o, kk > 0);
            mma_commit(bar(B_O));
            if (need) {
                if (!wait(B_Y1, cc)) break;
                tc_fence_after();
                issue_update(tmem + TM_U, yt, low, z, 1, id_u);
                mma_commit(bar(B_U));
            }
            mma_commit(bar(B_EMPTY + ty % kSlots));
            mma_commit(bar(B_EMPTY + tz % kSlots));
        }
        mma_commit(bar(B_DRAIN));
        mbar_wait_for(bar(B_DRAIN), 0, A.wait_cycles);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, TM_COLS);
}

// ---------------------------------------------------------------- the segments' own sums

constexpr int kSumWeighWarps = 8, kSumStateWarps = 8, kSumThreads = 32 * (kSumWeighWarps + kSumStateWarps + 2);
constexpr int kSumLoadWarp = kSumWeighWarps + kSumStateWarps;
constexpr uint32_t OFF_STAGE = kSlots * TILE, kSumSmem = OFF_STAGE + 2 * TILE + 1024;
constexpr uint32_t kSumCols = 256;
enum { S_FULL = 0, S_EMPTY = kSlots, S_READY = 2 * kSlots, S_U = S_READY + 2,
       S_UFREE = S_U + 2, S_DRAIN = S_UFREE + 2, S_COUNT };

// R_f of every segment but the last from the side that the state comes from: U chunk by
// chunk as in the mix, with two accumulators and two tiles for Yw's lower part, so that weighing, products and sums of neighbouring chunks run at once. Bound by
// reading Y and Z.
__global__ void __launch_bounds__(kSumThreads, 1) sum_tc_kernel(const __grid_constant__ TcArgs A) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t base = smem_u32(sm);
    __shared__ Segment found;
    __shared__ __align__(8) uint64_t bars[S_COUNT];
    __shared__ uint32_t tmem_slot;
    __shared__ int gave_up;
    __shared__ uint32_t row_w[C];
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Work w;
    w.role = (int)(blockIdx.x % A.count);
    const int64_t rest = blockIdx.x / A.count;
    w.slice = (int)(rest % A.slices);
    w.h = (int)(rest / A.slices % A.p.H);
    w.item = rest / A.slices / A.p.H;
    bool bad;
    w.s = locate(A.p, w.item, &found, &bad);
    if (blockIdx.x == 0 && tid == 0 && A.p.first) A.p.status[0] = bad ? GDR_ERR_BAD_SEQLENS : GDR_OK;
    if (bad || w.s.seq < 0) return;
    const TcMix &m = A.mix[w.role];
    if (w.s.f == (m.backward ? 0 : w.s.n - 1)) return;  // hands nothing on
    const float l2 = log2_decay(A.p.log_decay[w.h]);
    const int chunks = (int)((w.s.tokens + C - 1) / C);
    auto chunk_of = [&](int cc) { return m.backward ? chunks - 1 - cc : cc; };
    auto tokens_of = [&](int c) {
        const int64_t r = w.s.tokens - (int64_t)c * C;
        return (int)(r < C ? r : C);
    };
    if (tid == 0) {
        for (int i = 0; i < 2 * kSlots; ++i) mbar_init(bar(i), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(S_READY + i), kStateThreads);
            mbar_init(bar(S_U + i), 1);
            mbar_init(bar(S_UFREE + i), kStateThreads);
        }
        mbar_init(bar(S_DRAIN), 1);
        fence_mbar_init();
        gave_up = 0;
    }
    if (tid < 32) {
        tmem_alloc(smem_u32(&tmem_slot), kSumCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    volatile int *stop = &gave_up;
    auto wait = [&](int b, int phase) -> bool {
        if (mbar_sleep(bar(b), phase & 1)) return true;
        const long long t0 = clock64();
        while (!mbar_sleep(bar(b), phase & 1)) {
            if (*stop) return false;
            if (clock64() - t0 > A.wait_cycles) {
                *stop = 1;
                A.p.status[0] = GDR_ERR_DEVICE_TIMEOUT;
                return false;
            }
        }
        return true;
    };
    auto warp_wait = [&](int b, int phase) -> bool { return __all_sync(0xffffffffu, wait(b, phase)); };
    auto slot = [&](int t) { return (uint32_t)(t % kSlots) * TILE; };
    auto stage = [&](int i) { return OFF_STAGE + (uint32_t)(i & 1) * TILE; };

    if (warp < kSumWeighWarps) {
        int weighed = 0;
        for (int cc = 0; cc < chunks; ++cc) {
            const int n = tokens_of(chunk_of(cc)), ty = 2 * cc, tz = ty + 1;
            bool ok = warp_wait(S_FULL + ty % kSlots, ty / kSlots);
            if (ok && n < C) {
                ok = warp_wait(S_FULL + tz % kSlots, tz / kSlots);
                if (ok) clear_behind(sm + slot(tz), m.zb, n, tid);
            }
            if (ok && cc >= 2) ok = warp_wait(S_U + (cc & 1), (cc >> 1) - 1);  // the tile is free
            if (!ok) break;
            if (n != weighed) row_weights(row_w, weighed = n, m.backward, l2, m.s_state, tid);
            weigh_half<0>(sm + slot(ty), sm + stage(cc), m.xb, n, row_w, tid);
            weigh_half<1>(sm + slot(ty), sm + stage(cc), m.xb, n, row_w, tid);
            fence_async_smem();
            mbar_arrive(bar(S_READY + (cc & 1)));
        }
    } else if (warp < kSumLoadWarp) {
        const int id = tid - 32 * kSumWeighWarps;
        const int a = 32 * (warp & 3) + lane, b0 = 64 * (id / 128);
        const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        float2 E[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) E[j] = make_float2(0.f, 0.f);
        for (int cc = 0; cc < chunks; ++cc) {
            if (!warp_wait(S_U + (cc & 1), cc >> 1)) break;
            tc_fence_after();
            if (b0 < 64 * m.zb) add_update(E, decay_pow(l2, (float)tokens_of(chunk_of(cc))), lanes + 128 * (cc & 1) + b0);
            tc_fence_before();
            mbar_arrive(bar(S_UFREE + (cc & 1)));
        }
        if (a < 64 * m.xb && b0 < 64 * m.zb && !*stop)
            write_state(E, m.R_out + (w.item * A.p.H + w.h) * A.mat, state_row(A, m, w.slice, a, b0));
    } else if (warp == kSumLoadWarp) {
        if (lane == 0) {
            int issued = 0;
            for (int cc = 0; cc < chunks; ++cc) {
                const int t0 = (int)(w.s.begin + (int64_t)chunk_of(cc) * C);
                bool ok = true;
                for (int i = 0; i < 2 && ok; ++i) {
                    const int t = 2 * cc + i;
                    if (t >= kSlots && !(ok = wait(S_EMPTY + t % kSlots, t / kSlots - 1))) break;
                    const int blocks = i ? m.zb : m.xb;
                    const uint32_t full = bar(S_FULL + t % kSlots);
                    mbar_arrive_expect_tx(full, blocks * BLOCK);
                    for (int b = 0; b < blocks; ++b)
                        tma_load_3d(base + slot(t) + b * BLOCK, &A.maps[i ? m.mz : m.my], full,
                                    w.slice * (i ? m.zstep : m.ystep) + 64 * b, w.h / (i ? m.zg : m.yg), t0);
                    ++issued;
                }
                if (!ok) break;
            }
            for (int t = issued > kSlots ? issued - kSlots : 0; *stop && t < issued; ++t)
                mbar_wait_for(bar(S_FULL + t % kSlots), (t / kSlots) & 1, A.wait_cycles);
        }
    } else if (lane == 0) {
        const uint32_t id_u = idesc_bf16(128, 64 * m.zb, 1, 1);
        bool ok = true;
        for (int cc = 0; cc < chunks && ok; ++cc) {
            const int ty = 2 * cc, tz = ty + 1;
            if (!(ok = wait(S_FULL + tz % kSlots, tz / kSlots))) break;
            if (cc >= 2 && !(ok = wait(S_UFREE + (cc & 1), (cc >> 1) - 1))) break;
            if (!(ok = wait(S_READY + (cc & 1), cc >> 1))) break;
            tc_fence_after();
            for (int half = 0; half < 2; ++half)
                issue_update(tmem + 128 * (cc & 1), desc_mn(base + slot(ty)), desc_mn(base + stage(cc)),
                             desc_mn(base + slot(tz)), half, id_u);
            mma_commit(bar(S_U + (cc & 1)));
            mma_commit(bar(S_EMPTY + ty % kSlots));
            mma_commit(bar(S_EMPTY + tz % kSlots));
        }
        mma_commit(bar(S_DRAIN));
        mbar_wait_for(bar(S_DRAIN), 0, A.wait_cycles);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, kSumCols);
}

template <typename K> int run(K kernel, const TcArgs &A, int threads, uint32_t smem, cudaStream_t stream) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return GDR_ERR_CUDA;
    const int64_t blocks = A.p.items * A.p.H * A.slices * A.count;
    kernel<<<(unsigned)blocks, threads, smem, stream>>>(A);
    return cuda_status(cudaGetLastError());
}

}  // namespace

// Every mix of one launch has the same slices; `sums`: the segments' own sums.
int launch_mix_tc(const Plan &p, const Mix *mixes, int count, int d_v, bool sums, cudaStream_t stream) {
    TcArgs A = {};
    A.p = p;
    A.count = count;
    A.slices = d_v == 256 ? 2 : 1;
    A.pitch = d_v;
    A.wait_cycles = kWaitCycles;
    // the tensors among the mixes' inputs, each mapped once
    struct {
        const void *base;
        int64_t stride;
        int group, d;
    } have[4];
    int n = 0;
    auto map_of = [&](const void *base, int64_t stride, int group, int d, int *at) -> bool {
        for (int i = 0; i < n; ++i)
            if (have[i].base == base && have[i].stride == stride && have[i].group == group && have[i].d == d) {
                *at = i;
                return true;
            }
        if (n == 4) return false;
        *at = n;
        have[n] = {base, stride, group, d};
        return tc::make_map_rows(&A.maps[n++], base, d, p.H / group, stride, p.total_tokens);
    };
    for (int i = 0; i < count; ++i) {
        const Mix &s = mixes[i];
        TcMix &m = A.mix[i];
        if (!sums && !map_of(s.x, s.xs, s.xg, s.dx, &m.mx)) return GDR_ERR_CUDA;
        if (!map_of(s.y, s.ys, s.yg, s.dx, &m.my) || !map_of(s.z, s.zs, s.zg, s.dz, &m.mz)) return GDR_ERR_CUDA;
        A.mat = (int64_t)s.dx * s.dz;
        m.xg = s.xg; m.yg = s.yg; m.zg = s.zg;
        const int dx = s.dx > 128 ? 128 : s.dx, dz = s.dz > 128 ? 128 : s.dz;
        m.xb = dx / 64;
        m.zb = dz / 64;
        m.xstep = m.ystep = m.astep = s.dx > 128 ? 128 : 0;
        m.zstep = m.bstep = s.dz > 128 ? 128 : 0;
        m.out = s.out;
        m.out_f32 = s.out_f32;
        // slices of z lie side by side; of x they are sums of their own
        const int parts = s.dx > 128 ? A.slices : 1;
        m.out_s = s.dz > 128 ? 128 : (parts > 1 ? s.dz : 0);
        m.out_h = (int64_t)s.dz * parts;
        m.out_row = (int64_t)p.H * m.out_h;
        m.turned = s.turned;
        m.backward = s.backward;
        m.s_intra = s.s_intra; m.s_inter = s.s_inter; m.s_state = s.s_state;
        m.start = s.start; m.end = s.end; m.R = s.R; m.R_out = s.R_out;
    }
    if (sums) return run(sum_tc_kernel, A, kSumThreads, kSumSmem, stream);
    return run(mix_tc_kernel, A, kThreads, kSmem, stream);
}

}  // namespace linattn
}  // namespace gdr
