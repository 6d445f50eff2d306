// linattn_tc.cu -- the mix of linear attention (linattn.cuh) on the 5th-generation tensor
// cores, for bf16 inputs with d_x, d_z of 64 or 128 per CTA.
//
// One CTA per (segment, head, 128 columns of d_v) walks its segment in chunks of C = 128
// tokens. Per chunk, with the decay weights of linattn.cuh:
//   P  = X Y^T           masked and weighted into bf16, kept in TMEM as an A operand
//   O  = P Z + X E       E: the state entering the chunk, as bf16 in shared memory
//   U  = Yw^T Z          Yw: the rows of Y times w_upd, turned into TMEM as an A operand
//   out_r = s_inter f_r O_r,   E <- lam^n E + U
// Nothing that the tensor cores compute for a chunk depends on the state but X E: the
// state itself lives in fp32 registers, so that the sequential part of a chunk is one fused
// multiply-add per element and its copy to shared memory.
//
// One accumulator for both halves of O: a row's factor f_r = max(w_out(r), 2^-60) is taken
// out of it, so P's weights are lam^|r-i| / f_r. Where w_out is below 2^-60 the state's
// part of that row counts for 2^-60 of its size instead of less: nothing, next to P Z in fp32.
//
// Rounding. X, Y and Z are used as they are. P and the copy of E are rounded to bf16 once
// each, as a product's operand has to be; either costs an output element 2^-8 of the sum
// of its terms' sizes at most, like the output's own rounding. Yw is rounded to fp32 and kept
// as three bf16 parts, which hold that exactly, so that a state that goes out (S_final, dS0) is
// off by 1 to 5e-7 in norm, like a sum in fp32. Where none goes out, two parts, 16 bits: a term
// of the state is then off by 2^-16 at most, and only bf16 outputs see it (one part would cost
// them as much again as E's own rounding). The third part's products take 7 to 22 us of 91 to 302
// (figures below): 4 x 4096 tokens 84 us with two parts, eight packed prompts 177, 65536 tokens 270.
// U is summed chunk by chunk and added to E in fp32: a sum over a whole segment in the tensor
// cores would lose more.
//
// What bounds it: a product of two operands in shared memory reads them at all of shared
// memory's bandwidth (128 x 128 x 16: 8 KB in 64 cycles), and loads, conversions and copies
// use the same. So P and Yw are A operands in TMEM (512 columns: P, O, U, Yw of 128 each; Yw's
// third part in columns of O and U that the chunk leaves free), and Yw goes there straight from
// Y (ldmatrix turns it) instead of through shared memory.
//
// Shared memory: X, Y and Z tiles of two chunks (TMA, 128-byte swizzle), E in bf16.
// Warp 17 issues the MMAs in the order P Z, X E, P of the next chunk, U. Warps 0-15 all do
// the same work on a sixteenth each (a lane quarter by 32 columns or tokens), in the order
// in which the products end: the output rows, P's weights of the next chunk, the state, Yw of
// the next chunk. Warp 16: the loads. With 96 registers a thread next to nothing may spill (shared
// memory leaves no first-level cache to spill to): hence 16 columns at a time, and
// what would be worked out ahead of the loop made opaque. (8 bytes do.)
//
// Measured: 4 sequences of 4096 tokens, 16 heads, d_k = d_v = 128 (273 MB, two segments each)
// in 91 us with the sums, 3.0 TB/s: a chunk takes 2.8 us (2.5 with two parts), the chain of its
// products and what lies between them, with neither the tensor cores nor the schedulers busy half
// of the time. Where all 152 SMs run and every tile comes from DRAM (128 KB a chunk) it takes 3.1.
#include <mutex>

#include "f32x2.cuh"
#include "linattn.cuh"
#include "tc_common.cuh"

namespace gdr {
namespace linattn {
namespace {

using namespace sm100;
using tc::pack_bf16x2;

constexpr int C = 128;
constexpr uint32_t TILE = 32768, BLOCK = 16384;  // a tile: two blocks of 64 columns
constexpr int kSlots = 6;
constexpr uint32_t OFF_E = kSlots * TILE, kSmem = OFF_E + TILE;
constexpr uint32_t TM_P = 0, TM_O = 128, TM_U = 256, TM_Y = 384, TM_COLS = 512;
constexpr int kWorkers = 16, kWorkThreads = 32 * kWorkers, kLoadWarp = kWorkers;
constexpr int kThreads = kWorkThreads + 64;

struct TcMix {
    int mx, my, mz;              // maps
    int xg, yg, zg;              // heads sharing one
    int xstep, ystep, zstep;     // columns from one slice to the next
    int xb, zb;                  // blocks of 64 columns of x (and y), of z
    void *out;
    int64_t out_row, out_h, out_s;  // elements from one token, head, slice to the next
    bool out_f32, turned, backward;
    int astep, bstep;            // rows and columns of the state from one slice to the next
    float s_intra, s_inter, s_state;  // (s_intra: relative to s_inter)
    const float *start, *R;
    float *end, *R_out;
};
struct TcArgs {
    CUtensorMap maps[4];  // q, k, v, do
    CUtensorMap outs[3];  // the mixes' outputs (bf16)
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

// The weights of the 32 tokens that a warp weighs, of a chunk of n: table[i] holds those of tokens
// 32 sub + 2i and the one after, in fp32 (kFine) or as two bf16 parts, the larger ones of both
// tokens, then the smaller ones. Each warp has a table of its own.
template <bool kFine>
__device__ __forceinline__ void row_weights(uint2 *table, int n, bool backward, float l2, float s, int sub, int lane) {
    __syncwarp();
    const int r = 32 * sub + 2 * (lane & 15);
    const float x = s * decay_pow(l2, (float)(backward ? r + 1 : max(n - 1 - r, 0)));
    const float y = s * decay_pow(l2, (float)(backward ? r + 2 : max(n - 2 - r, 0)));
    const float hx = __bfloat162float(__float2bfloat16_rn(x)), hy = __bfloat162float(__float2bfloat16_rn(y));
    if (lane < 16)
        table[lane] = kFine ? make_uint2(__float_as_uint(x), __float_as_uint(y))
                            : make_uint2(pack_bf16x2(hx, hy), pack_bf16x2(x - hx, y - hy));
    __syncwarp();
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
// 16 TMEM lanes x 8 columns: register 2j + e of thread t is lane 8e + t/4, column 4j + t%4.
__device__ __forceinline__ void tmem_store_16x128b_x2(uint32_t taddr, const uint32_t (&r)[4]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}
// 16 columns of this thread's TMEM lane on their way; tmem_arrived names them, so that no use
// comes before it. (It waits for every load of the thread.)
__device__ __forceinline__ void tmem_fetch16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_arrived(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15])::"memory");
}
__device__ __forceinline__ void tmem_store8_nowait(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two bf16 minus two fp32.
__device__ __forceinline__ float2 minus(uint32_t a, float2 x) {
    float2 d;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "sub.rn.f32.bf16 %0, l, %3;\n\tsub.rn.f32.bf16 %1, h, %4;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "r"(a), "f"(x.x), "f"(x.y));
    return d;
}
// Two fp32 cut to their upper halves, bf16.
__device__ __forceinline__ uint32_t cut_bf16x2(float2 x) {
    return __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632);
}

// Yw of 32 tokens into TMEM: lane = column of Y, TMEM column = two tokens, the larger parts
// at `taddr`, the smaller ones 64 columns on. With a weight w = wh + wl (bf16 each),
// hi = round(y wh), lo = y wh - hi (exact: what is left of 16 bits) + y wl. kFine: y w, rounded
// to fp32, is cut into three parts of 8 bits each that hold it exactly: hi, minus lo, and the
// rest at `third`. (The mixed-precision subtractions keep the ALU free for the cuts; with masks
// instead, eight packed prompts took 211 us, not 200.) A warp takes the 32 columns of its lane
// quarter and the tokens 32 sub ..; ldmatrix hands each thread two tokens of one column, as the
// store wants them.
template <bool kFine>
__device__ __forceinline__ void weigh(uint32_t y, uint32_t taddr, int quarter, int sub, int n,
                                      const uint2 *table, int lane, uint32_t third) {
    const int mat = lane >> 3;
    const int token = 32 * sub + (mat >> 1) * 8 + (lane & 7);
    uint2 w[4];  // of two tokens each
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = table[4 * i + (lane & 3)];
#pragma unroll 1
    for (int mb = 0; mb < 2; ++mb) {
        const int m0 = 32 * quarter + 16 * mb, chunk = ((m0 & 63) >> 3) + (mat & 1);
        const uint32_t at = y + (m0 >> 6) * BLOCK + token * 128 + (((chunk ^ lane) & 7) << 4);
        const uint32_t to = taddr + ((uint32_t)m0 << 16) + 16 * sub;
        uint32_t r[2][4];
        ldmatrix_x4_trans(r[0], at);
        ldmatrix_x4_trans(r[1], at + 2048);  // 16 tokens further on
        if (n < C) {  // whatever lies behind the last token
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 32 * sub + 8 * i + 2 * (lane & 3);
                const uint32_t keep = t + 1 < n ? 0xffffffffu : (t < n ? 0xffffu : 0u);
                r[i >> 1][2 * (i & 1)] &= keep;
                r[i >> 1][2 * (i & 1) + 1] &= keep;
            }
        }
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {
            uint32_t hi[4], lo[4];
            if constexpr (kFine) {
                uint32_t rest[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint2 we = w[2 * jj + (e >> 1)];
                    float2 x = make_float2(__uint_as_float(r[jj][e] << 16), __uint_as_float(r[jj][e] & 0xffff0000u));
                    x = mul2(x, make_float2(__uint_as_float(we.x), __uint_as_float(we.y)));
                    hi[e] = cut_bf16x2(x);
                    x = minus(hi[e], x);  // minus what is left ..
                    lo[e] = cut_bf16x2(x);
                    x = minus(lo[e], x);  // .. and what is left after that
                    rest[e] = cut_bf16x2(x);
                }
                tmem_store_16x128b_x2(third + ((uint32_t)m0 << 16) + 8 * jj, rest);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const __nv_bfloat162 v = reinterpret_cast<const __nv_bfloat162 &>(r[jj][e]);
                    const __nv_bfloat162 wh = reinterpret_cast<const __nv_bfloat162 &>(w[2 * jj + (e >> 1)].x);
                    const __nv_bfloat162 wl = reinterpret_cast<const __nv_bfloat162 &>(w[2 * jj + (e >> 1)].y);
                    const __nv_bfloat162 h = __hmul2_rn(v, wh);
                    const __nv_bfloat162 l = __hfma2(v, wl, __hfma2(v, wh, __hneg2(h)));
                    hi[e] = reinterpret_cast<const uint32_t &>(h);
                    lo[e] = reinterpret_cast<const uint32_t &>(l);
                }
            }
            tmem_store_16x128b_x2(to + 8 * jj, hi);
            tmem_store_16x128b_x2(to + 64 + 8 * jj, lo);
        }
    }
}

// Rows n .. 127 of a tile become zero.
__device__ __forceinline__ void clear_behind(unsigned char *tile, int blocks, int n, int id) {
    for (int e = id; e < (C - n) * 8 * blocks; e += kWorkThreads) {
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

// The MMAs of U: the smaller parts first. kFine: three parts, the smallest at `third`, in 16 columns
// of every kApart, and minus the middle one (kNegateA, in the instruction's descriptor).
constexpr uint32_t kNegateA = 1u << 13;
template <bool kFine, int kApart>
__device__ __forceinline__ void issue_update(uint32_t d, uint32_t y, uint32_t z, uint32_t idesc, uint32_t third) {
    if (kFine) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) mma_ts(d, third + kApart * (kk >> 1) + 8 * (kk & 1), z, kk * 2048, idesc, kk > 0);
    }
#pragma unroll
    for (int i = 1; i >= 0; --i)
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
            mma_ts(d, y + 64 * i + 8 * kk, z, kk * 2048, kFine && i == 1 ? idesc | kNegateA : idesc, kFine || i == 0 || kk > 0);
}

// lam^n for n tokens that a state is carried over, rounded once where it is near 1: the hardware's
// exponential is off by 2^-22, the same way every time, which adds up over the chunks of a long
// sequence (65536 tokens: states off by 1.4e-6 with it).
__device__ __forceinline__ float carried(float l2, int n) {
    const float x = l2 * (float)n;
    return x > -0.5f ? 1.f + expm1f(x * 0.69314718056f) : exp2f(x);
}

// E <- w E + 32 columns of this thread's TMEM lane.
__device__ __forceinline__ void add_update(float2 (&E)[16], float w, uint32_t taddr) {
    const float2 w2 = make_float2(w, w);
    uint32_t u[2][16];
    tmem_fetch16(taddr, u[0]);
    tmem_fetch16(taddr + 16, u[1]);
    tmem_arrived(u[0]);
    tmem_arrived(u[1]);
#pragma unroll
    for (int j = 0; j < 16; ++j)
        E[j] = fma2(w2, E[j], make_float2(__uint_as_float(u[j >> 3][2 * j & 15]), __uint_as_float(u[j >> 3][(2 * j & 15) + 1])));
}

// Four lanes that hold 16 words each of a row of their own (4 words per part): afterwards part
// i of lane q is part q of lane i's row.
__device__ __forceinline__ void turn_four(float (&p)[16], int lane) {
#pragma unroll
    for (int step = 1; step < 4; step *= 2) {
        const bool up = lane & step;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i & step) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                // the lower lane sends its part i + step, the upper one its part i
                const float mine = up ? p[4 * i + e] : p[4 * (i + step) + e];
                const float other = __shfl_xor_sync(0xffffffffu, mine, step);
                if (up) p[4 * i + e] = other;
                else p[4 * (i + step) + e] = other;
            }
        }
    }
}

// A thread's 32 columns of state row a, from or to memory.
struct StateAt {
    int64_t first;  // element of column 0
    int step;       // elements from one column to the next
};
__device__ __forceinline__ StateAt state_row(const TcArgs &A, const TcMix &m, int slice, int a, int b) {
    const int64_t aa = a + m.astep * slice, bb = b + m.bstep * slice;
    return m.turned ? StateAt{bb * A.pitch + aa, A.pitch} : StateAt{aa * A.pitch + bb, 1};
}
// E += w times them. (Pointers are opaque after some steps: 32 places worked out ahead would
// take 64 registers.)
__device__ __forceinline__ void read_state(float2 (&E)[16], const float *S, const StateAt &at, float w) {
    const float *p = S + at.first;
    const float2 w2 = make_float2(w, w);
    if (at.step == 1) {
        float4 x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = reinterpret_cast<const float4 *>(p)[j];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            E[2 * j] = fma2(w2, make_float2(x[j].x, x[j].y), E[2 * j]);
            E[2 * j + 1] = fma2(w2, make_float2(x[j].z, x[j].w), E[2 * j + 1]);
        }
    } else {
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            float x[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                x[j] = *p;
                p += at.step;
                if (j % 4 == 3) asm volatile("" : "+l"(p));
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) E[8 * part + j] = fma2(w2, make_float2(x[2 * j], x[2 * j + 1]), E[8 * part + j]);
        }
    }
}
__device__ __forceinline__ void write_state(const float2 (&E)[16], float *p, int step) {
    if (step == 1) {
#pragma unroll
        for (int j = 0; j < 16; j += 2)
            *reinterpret_cast<float4 *>(p + 2 * j) = make_float4(E[j].x, E[j].y, E[j + 1].x, E[j + 1].y);
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            p[0] = E[j].x;
            p[step] = E[j].y;
            p += 2 * step;
            asm volatile("" : "+l"(p));
        }
    }
}

enum { B_FULL = 0, B_EMPTY = kSlots, B_P = 2 * kSlots, B_PREADY, B_A, B_YREADY, B_U, B_EREADY,
       B_O, B_OFREE, B_STAGED, B_DRAIN, B_COUNT };

// One body for both directions, its loops kept rolled where they can be: the warps of a
// block run far apart in the code, and a copy of it per direction or role costs more in
// instruction fetches than the selects do (gradients: 2.5 times the time with three copies). kFine:
// a state goes out, Yw has three parts. Two loops in one kernel, the second with three parts for the
// chunks near the end alone, were slower than three parts throughout (prompts of 4 x 4096 120 us,
// 91), and so was a choice chunk by chunk (97).
template <bool kFine> __global__ void __launch_bounds__(kThreads, 1) mix_tc_kernel(const __grid_constant__ TcArgs A) {
    extern __shared__ __align__(1024) unsigned char sm[];
    const uint32_t base = smem_u32(sm);
    __shared__ Segment found;
    __shared__ __align__(8) uint64_t bars[B_COUNT];
    __shared__ uint32_t tmem_slot;
    __shared__ int gave_up;
    __shared__ int kept_slice;  // (for the end, in no register meanwhile)
    __shared__ float shrink[2];  // kFine: lam^n over a whole chunk and the last one
    __shared__ uint2 weights[kWorkers][16];
    __shared__ __align__(16) float step_of[32];  // lam^(31-j), or lam^j from last to first
    __shared__ float pow_of[63];                  // lam^(i-31), 0 for i < 31
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const int role = (int)(blockIdx.x % A.count);
    const int64_t rest = blockIdx.x / A.count;
    const int slice = (int)(rest % A.slices);
    const bool bad = !locate(A.p, rest / A.slices, 0, &found, (int *)weights);
    if (blockIdx.x == 0 && tid == 0 && A.p.first) A.p.status[0] = bad ? GDR_ERR_BAD_SEQLENS : GDR_OK;
    if (bad || found.seq < 0) {
        griddep_wait();  // no launch ends before the one ahead of it
        return;
    }
    const TcMix &m = A.mix[role];
    const bool back = m.backward;
    const float l2_of_head = log2_decay(A.p.log_decay[found.h]);
    const int chunks = (int)((found.tokens + C - 1) / C);
    const bool ends = m.end && found.f == (back ? 0 : found.n - 1);
    auto chunk_of = [&](int cc) { return back ? chunks - 1 - cc : cc; };
    const int tail = (int)(found.tokens - (int64_t)(chunks - 1) * C);  // tokens of the last chunk
    auto tokens_of = [&](int c) { return c == chunks - 1 ? tail : C; };
    // tile i (X, Y, Z) of chunk cc: its slot, and the phase of the slot's barriers
    auto slot = [&](int cc, int i) { return 3 * (cc & 1) + i; };
    auto phase = [&](int cc) { return cc >> 1; };

    if (tid == 0) {
        // (X, Y, Z, X, Y, Z: Y is freed by the warps that weigh it, X by the output that has
        // left it)
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(bar(B_FULL + i), 1);
            mbar_init(bar(B_EMPTY + i), i % 3 == 1 ? kWorkers : 1);
        }
        mbar_init(bar(B_P), 1);
        mbar_init(bar(B_PREADY), kWorkers);
        mbar_init(bar(B_A), 1);
        mbar_init(bar(B_YREADY), kWorkers);
        mbar_init(bar(B_U), 1);
        mbar_init(bar(B_EREADY), kWorkers);
        mbar_init(bar(B_O), 1);
        mbar_init(bar(B_OFREE), kWorkers);
        mbar_init(bar(B_STAGED), kWorkers);
        mbar_init(bar(B_DRAIN), 1);
        fence_mbar_init();
        gave_up = 0;
        kept_slice = slice;
        prefetch_tensormap(&A.maps[m.mx]);
        prefetch_tensormap(&A.maps[m.my]);
        prefetch_tensormap(&A.maps[m.mz]);
    }
    if (tid < 32) {
        step_of[tid] = decay_pow(l2_of_head, (float)(back ? tid : 31 - tid));
        pow_of[31 + tid] = decay_pow(l2_of_head, (float)tid);
        if (kFine && tid < 2) shrink[tid] = carried(l2_of_head, tid ? tail : C);
        if (tid < 31) pow_of[tid] = 0.f;
        __syncwarp();
        tmem_alloc(smem_u32(&tmem_slot), TM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    // kFine: O and U of a chunk share columns, in turn the two halves of TM_O and TM_U: U starts when
    // O has been read. The half of the other chunks is free then, and holds Yw's smallest part.
    auto o_at = [](int cc) -> uint32_t { return kFine ? TM_O + 128 * (cc & 1) : TM_O; };
    auto u_at = [&](int cc) -> uint32_t { return kFine ? o_at(cc) : TM_U; };
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

    if (warp < kWorkers) {
        int quarter = warp & 3, sub = warp >> 2;
        int lane = tid & 31;
        float l2 = l2_of_head;
        uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16);
        int t = 32 * quarter + lane;  // row of the chunk, and of the state
        int col = 32 * sub;          // this warp's columns of P, O and the state
        const bool has_z = col < 64 * m.zb;
        // an arrival for the warp, after what its lanes have written
        auto arrive = [&](int b) {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(b));
        };

        // ---- the state: row t, columns col ..
        const StateAt st = state_row(A, m, slice, t, col);
        const bool mine = t < 64 * m.xb && has_z;
        float2 E[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) E[j] = make_float2(0.f, 0.f);
        if (found.n > 1) griddep_wait();  // the segments' sums are there (the loads began before)
        if (mine) {
            if (m.start)
                read_state(E, m.start + ((int64_t)found.seq * A.p.H + found.h) * A.mat, st,
                           decay_pow(l2, (float)(back ? found.behind : (int64_t)found.f * A.p.seg)));
            if (m.R) {
                const int part = (int)(A.p.seg / A.p.split);
                const float *R = m.R + (found.sum0 * A.p.split * A.p.H + found.h) * A.mat;
                const int first = back ? found.f * A.p.split : 0, end = (back ? found.n - 1 : found.f) * A.p.split;
#pragma unroll 1
                for (int i = first; i < end; ++i) {
                    const int apart = back ? i - first : end - 1 - i;
                    read_state(E, R + (int64_t)i * A.p.H * A.mat, st, decay_pow(l2, (float)apart * (float)part));
                }
            }
        }
        // rows of E as the K rows of a B operand
        auto publish = [&]() {
            if (has_z) {
                unsigned char *row = sm + OFF_E + (sub >> 1) * BLOCK + t * 128;
#pragma unroll
                for (int j = 0; j < 16; j += 4)
                    *reinterpret_cast<uint4 *>(row + ((((4 * sub + (j >> 2)) ^ t) & 7) << 4)) =
                        make_uint4(pack_bf16x2(E[j].x, E[j].y), pack_bf16x2(E[j + 1].x, E[j + 1].y),
                                   pack_bf16x2(E[j + 2].x, E[j + 2].y), pack_bf16x2(E[j + 3].x, E[j + 3].y));
            }
            fence_async_smem();
            arrive(B_EREADY);
        };

        // ---- Yw
        int weighed = 0;  // the length that the weights are for
        auto weigh_chunk = [&](int cc) -> bool {
            const int n = tokens_of(chunk_of(cc)), sy = slot(cc, 1);
            if (n != weighed) row_weights<kFine>(weights[warp], weighed = n, back, l2, m.s_state, sub, lane);
            if (!warp_wait(B_FULL + sy, phase(cc))) return false;
            // (the smallest part: into this warp's own block of U of the chunk before, which it has read)
            if (quarter < 2 * m.xb)
                weigh<kFine>(base + sy * TILE, tmem + TM_Y, quarter, sub, n, weights[warp], lane, tmem + o_at(cc + 1) + col);
            tmem_store_wait();
            tc_fence_before();
            arrive(B_EMPTY + sy);
            if (lane == 0) mbar_arrive(bar(B_YREADY));
            return true;
        };

        // ---- P's weights lam^|t-i| / f_t: 2^60 at most
        auto row_factor = [&](int n) {  // log2 f_t
            return fmaxf(l2 * (float)(back ? max(n - 1 - t, 0) : t + 1), -60.f);
        };
        auto weigh_scores = [&](int cc) -> bool {
            const int n = tokens_of(chunk_of(cc)), sz = slot(cc, 2);
            if (n < C) {  // Z's rows behind the last token meet P's zeros
                if (!warp_wait(B_FULL + sz, phase(cc))) return false;
                clear_behind(sm + sz * TILE, m.zb, n, tid);
                fence_async_smem();
            }
            if (!warp_wait(B_P, cc)) return false;
            tc_fence_after();
            const float f = row_factor(n);
            // 16 columns at a time, the next ones on their way meanwhile
            const bool diagonal = sub == quarter;
            if (back ? sub < quarter : sub > quarter) {
                const uint32_t none[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                tmem_store8_nowait(lanes + TM_P + col, none);
                tmem_store8_nowait(lanes + TM_P + col + 8, none);
            } else {
                uint32_t ahead[16];
                tmem_fetch16(lanes + TM_P + col, ahead);
                // off the diagonal: the way to the block's near column, times the way on to column
                // j; on it each distance by itself, 0 beyond it
                const float far = m.s_intra * ex2(diagonal ? -f : fmaf(l2, (float)(back ? col - t : t - col - 31), -f));
                const float2 far2 = make_float2(far, far);
                const float *g = pow_of + (back ? 31 - lane : 31 + lane);
                const int lo = back && diagonal ? lane : 0, hi = back ? n - 1 - col : (diagonal ? lane : 31);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    tmem_arrived(ahead);
                    float2 v[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = make_float2(__uint_as_float(ahead[2 * j]), __uint_as_float(ahead[2 * j + 1]));
                    if (half == 0) tmem_fetch16(lanes + TM_P + col + 16, ahead);
                    if (diagonal) {
                        const float *gh = back ? g + 16 * half : g - 16 * half;
                        if (back) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) v[j] = mul2(v[j], make_float2(gh[2 * j], gh[2 * j + 1]));
                        } else {
#pragma unroll
                            for (int j = 0; j < 8; ++j) v[j] = mul2(v[j], make_float2(gh[-2 * j], gh[-2 * j - 1]));
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; j += 2) {
                            const float4 w4 = *reinterpret_cast<const float4 *>(&step_of[16 * half + 2 * j]);
                            v[j] = mul2(v[j], make_float2(w4.x, w4.y));
                            v[j + 1] = mul2(v[j + 1], make_float2(w4.z, w4.w));
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = mul2(v[j], far2);
                    if (n < C) {  // what lies behind the last token may be anything
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int i = 16 * half + 2 * j;
                            v[j].x = i >= lo && i <= hi ? v[j].x : 0.f;
                            v[j].y = i + 1 >= lo && i + 1 <= hi ? v[j].y : 0.f;
                        }
                    }
                    uint32_t out[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) out[j] = pack_bf16x2(v[j].x, v[j].y);
                    // the bf16 copy goes to the first half of the block's own columns: those of
                    // the second half's copy have been read by now
                    tmem_store8_nowait(lanes + TM_P + col + 8 * half, out);
                }
            }
            tmem_store_wait();
            tc_fence_before();
            arrive(B_PREADY);
            return true;
        };

        // ---- the output rows, 32 columns of row t: by way of the chunk's X tile, which has been
        // used, and TMA (by rows of their own the stores would take the load/store unit 2000
        // cycles a chunk); what is not a whole tile of bf16, straight to its place
        int pitch = (int)m.out_row * (m.out_f32 ? 4 : 2);
        char *out0 = (char *)m.out + ((found.begin + t) * m.out_row + found.h * m.out_h + slice * m.out_s + col) * (m.out_f32 ? 4 : 2);
        auto store_rows = [&](int cc) -> bool {
            const int c = chunk_of(cc), n = tokens_of(c);
            if (!warp_wait(B_O, cc)) return false;
            tc_fence_after();
            uint32_t o[2][16];
            tmem_fetch16(lanes + o_at(cc) + col, o[0]);
            tmem_fetch16(lanes + o_at(cc) + col + 16, o[1]);
            tmem_arrived(o[0]);
            tmem_arrived(o[1]);
            tc_fence_before();
            arrive(B_OFREE);
            const float wo = m.s_inter * ex2(row_factor(n));
            const float2 wo2 = make_float2(wo, wo);
            const bool tile = n == C && !m.out_f32;
            unsigned char *row = sm + slot(cc, 0) * TILE + (sub >> 1) * BLOCK + t * 128;
            char *to = out0 + (int64_t)c * C * pitch;
            if (m.out_f32) {
                // four rows at a time, 16 bytes of one per lane: whole sectors of 32
                const int live = has_z ? n - (t & ~3) : 0;  // rows of the four to be written
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    float p[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) p[j] = wo * __uint_as_float(o[half][j]);
                    turn_four(p, lane);
                    char *at = to + (16 - pitch) * (lane & 3) + 64 * half;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (i < live)
                            *reinterpret_cast<float4 *>(at) = make_float4(p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3]);
                        at += pitch;
                    }
                }
            } else {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t p[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 x = mul2(wo2, make_float2(__uint_as_float(o[half][2 * j]), __uint_as_float(o[half][2 * j + 1])));
                        p[j] = pack_bf16x2(x.x, x.y);
                    }
                    if (!has_z) {
                    } else if (tile) {
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            *reinterpret_cast<uint4 *>(row + (((4 * sub + 2 * half + i) ^ t) & 7) * 16) =
                                make_uint4(p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3]);
                    } else if (t < n) {
                        *reinterpret_cast<uint4 *>(to + 32 * half) = make_uint4(p[0], p[1], p[2], p[3]);
                        *reinterpret_cast<uint4 *>(to + 32 * half + 16) = make_uint4(p[4], p[5], p[6], p[7]);
                    }
                }
            }
            fence_async_smem();
            arrive(B_STAGED);
            return true;
        };
        // (nothing needs the state behind the last chunk unless it goes out)
        auto need = [&](int cc) { return cc + 1 < chunks || ends; };
        // (one place for each step, the first chunk's included: the code is fetched as it runs)
        bool ok = true;
        for (int cc = -1; cc < chunks; ++cc) {
            // opaque in every round: what follows from them, worked out ahead of the loop,
            // would take more registers than there are
            asm volatile("" : "+r"(pitch), "+l"(out0), "+r"(lane), "+r"(t), "+f"(l2), "+r"(quarter), "+r"(sub), "+r"(col), "+r"(lanes));
            const bool more = cc + 1 < chunks;
            if (cc >= 0 && !(ok = store_rows(cc))) break;
            if (more && !(ok = weigh_scores(cc + 1))) break;
            if (cc >= 0 && need(cc)) {
                if (!(ok = warp_wait(B_U, cc))) break;
                tc_fence_after();
                const int n = tokens_of(chunk_of(cc));
                if (has_z) add_update(E, kFine ? shrink[n < C] : ex2(l2 * (float)n), lanes + u_at(cc) + col);
                tc_fence_before();
            }
            if (!more) break;
            publish();
            if (need(cc + 1) && !(ok = weigh_chunk(cc + 1))) break;
        }
        if (ends && ok && t < 64 * m.xb && has_z) {
            const StateAt to = state_row(A, m, kept_slice, t, col);
            write_state(E, m.end + ((int64_t)found.seq * A.p.H + found.h) * A.mat + to.first, to.step);
        }
    } else if (warp == kLoadWarp) {
        // ------------------------------------------------ the loads, and the outputs' stores
        if (lane == 0) {
            int issued[3] = {0, 0, 0};
            const int h = found.h;
            const int64_t begin = found.begin;
            auto load = [&](int cc, int i) {
                const int to = slot(cc, i);
                const CUtensorMap *map = &A.maps[i == 0 ? m.mx : (i == 1 ? m.my : m.mz)];
                const int at = slice * (i == 0 ? m.xstep : (i == 1 ? m.ystep : m.zstep));
                const int head = h / (i == 0 ? m.xg : (i == 1 ? m.yg : m.zg));
                const int blocks = i == 2 ? m.zb : m.xb, t0 = (int)(begin + (int64_t)chunk_of(cc) * C);
                const uint32_t full = bar(B_FULL + to);
                mbar_arrive_expect_tx(full, blocks * BLOCK);
                for (int b = 0; b < blocks; ++b) tma_load_3d(base + to * TILE + b * BLOCK, map, full, at + 64 * b, head, t0);
                ++issued[i];
            };
            for (int cc = 0; cc < 2 && cc < chunks; ++cc)
                for (int i = 0; i < 3; ++i) load(cc, i);
            const CUtensorMap *out = &A.outs[role];
            const int out_col = m.out_s ? slice * (int)m.out_s : 0;
            for (int cc = 0; cc < chunks; ++cc) {
                const bool more = cc + 2 < chunks;
                if (more) {
                    if (!wait(B_EMPTY + slot(cc, 1), phase(cc))) break;
                    load(cc + 2, 1);
                }
                if (!wait(B_STAGED, cc)) break;
                if (tokens_of(chunk_of(cc)) == C && !m.out_f32) {
                    for (int b = 0; b < m.zb; ++b)
                        tma_store_3d(out, base + slot(cc, 0) * TILE + b * BLOCK, out_col + 64 * b, h,
                                     (int)(begin + (int64_t)chunk_of(cc) * C));
                    bulk_commit_group();
                    bulk_wait_group_read<0>();
                }
                if (more) {
                    load(cc + 2, 0);
                    if (!wait(B_EMPTY + slot(cc, 2), phase(cc))) break;
                    load(cc + 2, 2);
                }
            }
            bulk_wait_group_all();
            // after a wait gave up: every load issued has landed before the block ends
            for (int i = 0; *stop && i < 3; ++i)
                for (int cc = issued[i] > 2 ? issued[i] - 2 : 0; cc < issued[i]; ++cc)
                    mbar_wait_for(bar(B_FULL + slot(cc, i)), phase(cc) & 1, A.wait_cycles);
        }
    } else if (lane == 0) {
        // ------------------------------------------------ the MMAs
        const uint32_t id_pp = idesc_bf16(128, 128, 0, 0);           // A and B K-major
        const uint32_t id_o = idesc_bf16(128, 64 * m.zb, 0, 1);      // B with rows of z along K
        const uint32_t id_u = id_o;                                  // A in TMEM as for O
        const bool wide = m.xb == 2;
        const uint32_t E = desc_mn(base + OFF_E);
        auto scores = [&](int cc) -> bool {  // P of chunk cc
            const int sx = slot(cc, 0), sy = slot(cc, 1);
            if (!wait(B_FULL + sx, phase(cc)) || !wait(B_FULL + sy, phase(cc))) return false;
            if (cc > 0 && !wait(B_A, cc - 1)) return false;  // P's columns have been used
            tc_fence_after();
            const uint32_t x = desc_k(base + sx * TILE), y = desc_k(base + sy * TILE);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
                const uint32_t at = (kk >> 2) * BLOCK + (kk & 3) * 32;
                if (kk < 4 || wide) mma_ss(tmem + TM_P, x, at, y, at, id_pp, kk > 0);
            }
            mma_commit(bar(B_P));
            return true;
        };
        bool ok = chunks == 0 || scores(0);
        for (int cc = 0; ok && cc < chunks; ++cc) {
            const bool need = cc + 1 < chunks || ends;
            const int sx = slot(cc, 0), sz = slot(cc, 2);
            const uint32_t x = desc_k(base + sx * TILE), z = desc_mn(base + sz * TILE);
            // (the accumulator is free: O of the chunk before has been read, or (kFine) U of the chunk
            // before, whose smallest part lay there, is complete)
            ok = wait(B_FULL + sz, phase(cc)) && wait(B_PREADY, cc) && (cc == 0 || wait(kFine ? B_U : B_OFREE, cc - 1));
            if (!ok) break;
            const uint32_t o = tmem + o_at(cc);
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
                mma_ts(o, tmem + TM_P + 32 * (kk >> 1) + 8 * (kk & 1), z, kk * 2048, id_o, kk > 0);
            mma_commit(bar(B_A));
            if (!(ok = wait(B_EREADY, cc))) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
                if (kk < 4 || wide) mma_ss(o, x, (kk >> 2) * BLOCK + (kk & 3) * 32, E, kk * 2048, id_o, true);
            mma_commit(bar(B_O));
            if (cc + 1 < chunks && !(ok = scores(cc + 1))) break;
            if (need) {
                if (!(ok = wait(B_YREADY, cc) && (!kFine || wait(B_OFREE, cc)))) break;
                tc_fence_after();
                issue_update<kFine, 32>(tmem + u_at(cc), tmem + TM_Y, z, id_u, tmem + o_at(cc + 1));
                mma_commit(bar(B_U));
            }
            mma_commit(bar(B_EMPTY + sz));
        }
        mma_commit(bar(B_DRAIN));
        mbar_wait_for(bar(B_DRAIN), 0, A.wait_cycles);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_wait();  // no launch ends before the one ahead of it
    if (warp == 0) tmem_dealloc(tmem, TM_COLS);
}

// ---------------------------------------------------------------- the segments' own sums

constexpr int kSumThreads = kWorkThreads + 64;
constexpr uint32_t kSumSmem = kSlots * TILE;
enum { S_FULL = 0, S_EMPTY = kSlots, S_READY = 2 * kSlots, S_U = S_READY + 2,
       S_UFREE = S_U + 2, S_DRAIN = S_UFREE + 2, S_COUNT };

// R_f of every segment but the last from the side that the state comes from: U chunk by
// chunk as in the mix, with two buffers of Yw, so that a chunk is weighed while the products of
// the one before it run, and two of U. With three parts of Yw (kFine) there are columns for one U:
// its products wait until the one before has been read. 1.2 us a chunk: bound by reading Y and Z,
// 64 KB, where all SMs run; with three parts 1.6.
template <bool kFine> __global__ void __launch_bounds__(kSumThreads, 1) sum_tc_kernel(const __grid_constant__ TcArgs A) {
    extern __shared__ __align__(1024) unsigned char sm[];
    const uint32_t base = smem_u32(sm);
    __shared__ Segment found;
    __shared__ __align__(8) uint64_t bars[S_COUNT];
    __shared__ uint32_t tmem_slot;
    __shared__ int gave_up;
    __shared__ uint2 weights[kWorkers][16];
    __shared__ float shrink[2];
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int role = (int)(blockIdx.x % A.count);
    const int64_t rest = blockIdx.x / A.count;
    const int slice = (int)(rest % A.slices);
    const int part = (int)(rest / A.slices / A.p.handing);
    griddep_launch_dependents();
    const bool bad = !locate(A.p, rest / A.slices % A.p.handing, 1 + A.mix[role].backward, &found, (int *)weights);
    Segment s = found;
    const int h = s.h;
    if (blockIdx.x == 0 && tid == 0 && A.p.first) A.p.status[0] = bad ? GDR_ERR_BAD_SEQLENS : GDR_OK;
    if (bad || s.seq < 0) return;
    const TcMix &m = A.mix[role];
    const int64_t part_len = A.p.seg / A.p.split;
    s.begin += part * part_len;
    s.tokens = max((int64_t)0, min(part_len, s.tokens - part * part_len));  // (none: a sum of zero)
    const int64_t sum = (s.sum0 + s.f - m.backward) * A.p.split + part;
    const float l2 = log2_decay(A.p.log_decay[h]);
    const int chunks = (int)((s.tokens + C - 1) / C);
    auto u_at = [&](int cc) -> uint32_t { return kFine ? 0 : 128 * (cc & 1); };
    auto y_at = [&](int cc) -> uint32_t { return kFine ? 128 + 192 * (cc & 1) : 256 + 128 * (cc & 1); };
    auto chunk_of = [&](int cc) { return m.backward ? chunks - 1 - cc : cc; };
    auto tokens_of = [&](int c) {
        const int64_t r = s.tokens - (int64_t)c * C;
        return (int)(r < C ? r : C);
    };
    if (tid == 0) {
        // (Y in the even slots: freed by the threads that weigh it)
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(bar(S_FULL + i), 1);
            mbar_init(bar(S_EMPTY + i), i % 2 == 0 ? kWorkers : 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(S_READY + i), kWorkers);
            mbar_init(bar(S_U + i), 1);
            mbar_init(bar(S_UFREE + i), kWorkers);
        }
        mbar_init(bar(S_DRAIN), 1);
        fence_mbar_init();
        gave_up = 0;
    }
    if (tid < 32) {
        if (kFine && tid < 2) shrink[tid] = carried(l2, tid ? tokens_of(chunks - 1) : C);
        __syncwarp();
        tmem_alloc(smem_u32(&tmem_slot), TM_COLS);
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

    if (warp < kWorkers) {
        const int quarter = warp & 3, sub = warp >> 2;
        const int t = 32 * quarter + lane, col = 32 * sub;  // row and columns of the state
        const bool has_z = col < 64 * m.zb;
        const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16);
        auto arrive = [&](int b) {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(b));
        };
        float2 E[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) E[j] = make_float2(0.f, 0.f);
        int weighed = 0;
        bool ok = true;
        for (int cc = 0; ok && cc <= chunks; ++cc) {
            if (cc < chunks) {
                const int n = tokens_of(chunk_of(cc)), ty = 2 * cc, tz = ty + 1;
                if (n != weighed) row_weights<kFine>(weights[warp], weighed = n, m.backward, l2, m.s_state, sub, lane);
                if (!(ok = warp_wait(S_FULL + ty % kSlots, ty / kSlots))) break;
                if (n < C) {
                    if (!(ok = warp_wait(S_FULL + tz % kSlots, tz / kSlots))) break;
                    clear_behind(sm + slot(tz), m.zb, n, tid);
                    fence_async_smem();
                }
                // (the buffer is free: U of chunk cc - 2 has been read below)
                if (quarter < 2 * m.xb)
                    weigh<kFine>(base + slot(ty), tmem + y_at(cc), quarter, sub, n, weights[warp], lane,
                                 tmem + y_at(cc) + 128 + 16 * sub);
                tmem_store_wait();
                tc_fence_before();
                arrive(S_EMPTY + ty % kSlots);
                if (lane == 0) mbar_arrive(bar(S_READY + (cc & 1)));
            }
            if (cc == 0) continue;
            const int b = cc - 1;  // the chunk before: its U
            if (!(ok = warp_wait(S_U + (b & 1), b >> 1))) break;
            tc_fence_after();
            const int n = tokens_of(chunk_of(b));
            if (has_z) add_update(E, kFine ? shrink[n < C] : decay_pow(l2, (float)n), lanes + u_at(b) + col);
            tc_fence_before();
            arrive(S_UFREE + (b & 1));
        }
        if (ok && t < 64 * m.xb && has_z) {
            const StateAt st = state_row(A, m, slice, t, col);
            write_state(E, m.R_out + (sum * A.p.H + h) * A.mat + st.first, st.step);
        }
    } else if (warp == kLoadWarp) {
        if (lane == 0) {
            int issued = 0;
            for (int cc = 0; cc < chunks; ++cc) {
                const int t0 = (int)(s.begin + (int64_t)chunk_of(cc) * C);
                bool ok = true;
                for (int i = 0; i < 2 && ok; ++i) {
                    const int t = 2 * cc + i;
                    if (t >= kSlots && !(ok = wait(S_EMPTY + t % kSlots, t / kSlots - 1))) break;
                    const int blocks = i ? m.zb : m.xb;
                    const uint32_t full = bar(S_FULL + t % kSlots);
                    mbar_arrive_expect_tx(full, blocks * BLOCK);
                    for (int b = 0; b < blocks; ++b)
                        tma_load_3d(base + slot(t) + b * BLOCK, &A.maps[i ? m.mz : m.my], full,
                                    slice * (i ? m.zstep : m.ystep) + 64 * b, h / (i ? m.zg : m.yg), t0);
                    ++issued;
                }
                if (!ok) break;
            }
            for (int t = issued > kSlots ? issued - kSlots : 0; *stop && t < issued; ++t)
                mbar_wait_for(bar(S_FULL + t % kSlots), (t / kSlots) & 1, A.wait_cycles);
        }
    } else if (lane == 0) {
        const uint32_t id_u = idesc_bf16(128, 64 * m.zb, 0, 1);
        for (int cc = 0; cc < chunks; ++cc) {
            const int tz = 2 * cc + 1;
            if (!wait(S_FULL + tz % kSlots, tz / kSlots)) break;
            const int reader = cc - (kFine ? 1 : 2);  // the chunk whose U has to have been read
            if (reader >= 0 && !wait(S_UFREE + (reader & 1), reader >> 1)) break;
            if (!wait(S_READY + (cc & 1), cc >> 1)) break;
            tc_fence_after();
            issue_update<kFine, 16>(tmem + u_at(cc), tmem + y_at(cc), desc_mn(base + slot(tz)), id_u, tmem + y_at(cc) + 128);
            mma_commit(bar(S_U + (cc & 1)));
            mma_commit(bar(S_EMPTY + tz % kSlots));
        }
        mma_commit(bar(S_DRAIN));
        mbar_wait_for(bar(S_DRAIN), 0, A.wait_cycles);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, TM_COLS);
}

// Tensor map over a [T, heads, d] bf16 tensor whose tokens are `stride` elements apart, with
// 64 (features) x 1 (head) x 128 (tokens) boxes, 128-byte swizzle; 256 bytes of L2 at a time.
bool make_map_rows(CUtensorMap *map, const void *base, int d, int heads, int64_t stride, int64_t T) {
    static decltype(&cuTensorMapEncodeTiled) encode = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        cudaDriverEntryPointQueryResult found;
        void *f = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) == cudaSuccess &&
            found == cudaDriverEntryPointSuccess)
            encode = reinterpret_cast<decltype(encode)>(f);
    });
    if (!encode) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)T};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, 1, 128}, each[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, each,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// `after_sums`: may start while the sums' launch ahead of it ends (it waits for it before it
// reads them).
template <typename K>
int run(K kernel, const TcArgs &A, int64_t units, int threads, uint32_t smem, bool after_sums, cudaStream_t stream) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return GDR_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * A.slices * A.count));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = after_sums ? 1 : 0;
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, A));
}

}  // namespace

// Every mix of one launch has the same slices.
int launch_mix_tc(const Plan &p, const Mix *mixes, int count, int d_v, bool sums, bool after_sums, cudaStream_t stream) {
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
        return make_map_rows(&A.maps[n++], base, d, p.H / group, stride, p.total_tokens);
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
        if (!sums && !s.out_f32 && !make_map_rows(&A.outs[i], s.out, s.dz, p.H, (int64_t)p.H * s.dz, p.total_tokens))
            return GDR_ERR_CUDA;
        // slices of z lie side by side; of x they are sums of their own
        const int parts = s.dx > 128 ? A.slices : 1;
        m.out_s = s.dz > 128 ? 128 : (parts > 1 ? s.dz : 0);
        m.out_h = (int64_t)s.dz * parts;
        m.out_row = (int64_t)p.H * m.out_h;
        m.turned = s.turned;
        m.backward = s.backward;
        // from first to last both are the scale, from last to first s_inter is 1
        m.s_intra = s.backward ? s.s_intra : 1.f;
        m.s_inter = s.s_inter;
        m.s_state = s.s_state;
        m.start = s.start; m.end = s.end; m.R = s.R; m.R_out = s.R_out;
    }
    if (sums)
        return run(p.fine ? sum_tc_kernel<true> : sum_tc_kernel<false>, A, p.handing * p.split, kSumThreads, kSumSmem, false, stream);
    return run(p.fine ? mix_tc_kernel<true> : mix_tc_kernel<false>, A, p.units, kThreads, kSmem, after_sums, stream);
}

}  // namespace linattn
}  // namespace gdr
