// cache_attn_tc.cuh -- attention over a paged 8-bit cache for many rows: prompts and pieces of them.
//
// Rows. As in cache_attn_step.cuh the rows of an item are the queries that share a head of the
// cache, token by token; a block takes 128 kTiles of them and goes through the keys that the last of them
// sees, kKeys at a time.
//
// Products on the 5th-generation tensor cores in fp16 with fp32 sums in TMEM: scores = Q K^T from shared
// memory, outputs += W codes with the weights W read from TMEM, where they take their scores' place.
// Codes come into shared memory by tensor copies, up to 64 keys of a page at a time, and converter warps turn them
// into fp16 tiles in the 128-byte-swizzled layout: a tile's row is a token, which is K-major for the first product
// and MN-major for the second, so that both are written alike. (Codes loaded into the converters' registers a tile
// ahead: 330 us for 4 x 4096 tokens of 16 heads, of which 70 were waits for them.)
//
// Roles (480 threads): kTiles groups of 128 threads for the softmax, a row to a thread; the rest of
// 384 convert; a thread of a warp for each row tile issues its products; a warp issues the copies. Scores have two buffers, so that the next
// tile's are there when a tile's weights are done. A block stays and goes from item to item: the next
// item's queries and first keys are on their way while the outputs of the last leave. (A block for each
// item took 32 thousand cycles more per item, as much as six tiles of 128 keys.)
//
// fp32: queries and weights as two fp16 parts, hi + lo, whose products are added in the same TMEM sums.
#pragma once

#include <atomic>
#include <type_traits>

#include "cache_attn.cuh"
#include "f32x2.cuh"
#include "sm100.cuh"

namespace gdr {
namespace cattn {

using namespace sm100;

constexpr int kTcThreads = 480, kTcRegs = 128;
constexpr int kRing = 8;   // tiles of scales
constexpr int kAll = 16 | 16 << 5 | 16 << 10 | 16 << 15;  // rows of a whole tile
// Tiles of keys whose outputs are added up in TMEM. The tensor cores cut these sums instead of rounding them, up to 2^-23 of
// them per step of 16 keys and always towards zero. fp32 outputs leave TMEM every kFlush tiles (256 rows behind 32,768
// tokens off by 3.1e-7 in norm and 2 x 4096 tokens 553 us; every 2 tiles 1.6e-7 and 843, every 16 1.9e-6 and 338). Of bf16 ones an
// item has kMost tiles (2^-11 at most, 2.6e-4 measured; without an end 2e-3 behind 300,000 tokens and 6e-3 behind a million); longer
// ones are several items of a block in turn, which meet in the workspace. That takes registers of the softmax (kLong: 4 x 4096
// tokens 262 us, 249 without; as a test within the loop over tiles 280), so tables that hold less go without.
constexpr int kFlush = 4, kMost = 1024;

template <int D, int kParts> struct TcConfig {
    static constexpr int kTiles = kParts == 1 && D <= 128 ? 2 : 1;
    // Two row tiles leave TMEM for scores of 4 x 64 keys. (128 keys and one buffer for each: every softmax waits
    // for its products, 376 us for 4 x 4096 tokens, 16 heads.)
    static constexpr int kKeys = 64;
    static constexpr int kRows = 128 * kTiles;
    static constexpr int kSoft = 128 * kTiles;         // threads
    static constexpr int kConv = 384 - kSoft;
    // Registers of a thread: 15 warps are launched with kTcRegs each; what the converters give up the softmax
    // gets (kSoft kSoftRegs + kConv kConvRegs = 384 x kTcRegs).
    static constexpr int kConvRegs = kTiles == 2 ? 80 : 96, kSoftRegs = kTiles == 2 ? 152 : 192;
    static_assert(kSoft * kSoftRegs + kConv * kConvRegs <= 384 * kTcRegs, "registers of the launch");
    static constexpr int kQ = 128 * D * 2;             // bytes of a part of a row tile
    static constexpr int kKv = kKeys * D * 2;          // of a tile of keys or values
    static constexpr int kStages = D == 256 ? (kParts == 2 ? 1 : 2) : 3;
    static constexpr int kRaw = D == 256 ? 1 : 3;      // tiles of codes
    static constexpr int kStage = D == 256 ? 0 : kSoft / 32 * 2048;  // 64 bytes of every row on their way out (D = 256: no room)
    static constexpr int kSmem = kTiles * kParts * kQ + 2 * kStages * kKv + kRaw * kKv + kStage + 1024;
    // TMEM columns: scores of two slots per row tile (weights in their place), low parts of weights, outputs
    static constexpr uint32_t kLow = 128, kLowStep = kKeys / 2, kO = 256;
    static_assert(kSmem <= 232448 - 2000, "shared memory");
    static_assert(kO + kTiles * D <= 512 && kTiles * 2 * kKeys + (kParts == 2 ? 2 * kLowStep : 0) <= kO, "TMEM");
};

struct TcPlan {
    char *parts;   // fp32 outputs and sums of the splits: [tile][head][split] Part
    char *pieces;  // [block][row] TcPiece, of tables that hold more than kMost tiles of keys for a split (bf16)
    int64_t tiles; // row tiles, empty ones among them, for each head of the cache
    int splits;    // of each item's keys
};
// A row's outputs and sum of weights of the pieces so far, times 2^-ref (l = 0: of none).
template <int D> struct alignas(16) TcPiece {
    float o[D], ref, l;
};

__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int b_mn) {
    return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Low words of shared-memory descriptors of 128-byte-swizzled tiles (sw128_desc), to which places within a
// tile are added: K-major, and MN-major with `apart` bytes between 64-wide blocks. The high word is one for all.
__device__ __forceinline__ uint32_t desc_k(uint32_t at) { return (at >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_mn(uint32_t at, uint32_t apart) { return (at >> 4) | ((apart >> 4) << 16); }
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add), "r"(kDescHigh)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add), "r"(kDescHigh)
        : "memory");
}

// Row tiles are numbered request by request; packed ones from floor(first row / kRows) + n on, a bound that needs
// no sum over the requests and leaves a tile empty here and there.
template <int kRows> __device__ __forceinline__ int64_t first_tile(const Attn &a, int64_t n) {
    if (!a.cu) return n * ((a.max_q * a.group + kRows - 1) / kRows);
    return (int64_t)__ldg(a.cu + n) * a.group / kRows + n;
}

struct TcItem {
    int n, first, len, past;   // request: its first row of q, tokens in the cache, those before the new ones
    int row0, rows;            // of the tile
    int head, j0, count;       // head of the cache; tiles of keys
    int64_t part;
    bool later, more;          // kLong: pieces of the same rows come before, behind
};

// Where a block is among its items.
struct TcTurn {
    int64_t k = 0;
    int piece = 0;
};

// The next item of this block, false behind the last. Those that see the most keys come first, and the blocks take
// them to and fro. An empty one has rows = 0.
template <int kRows, int kKeys, bool kLong> __device__ __forceinline__ bool get_item(const Attn &a, const TcPlan &plan, TcTurn &turn, TcItem &t) {
    const int64_t k = turn.k;
    const int64_t each = (int64_t)a.kv_heads * plan.splits;
    const int64_t idx = k * gridDim.x + (k & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    if (idx >= plan.tiles * each) return false;
    const int64_t y = idx / each;
    const int rest = (int)(idx - y * each), split = rest / a.kv_heads;
    t.head = rest - split * a.kv_heads;
    int64_t x, tile;
    if (!a.cu) {
        const int64_t per = plan.tiles / a.num_seqs;
        t.n = (int)(y % a.num_seqs);
        tile = per - 1 - y / a.num_seqs;
        x = t.n * per + tile;
    } else {
        x = plan.tiles - 1 - y;
        int64_t lo = 0, hi = a.num_seqs - 1;  // the last request whose tiles begin at x or before
        while (lo < hi) {
            const int64_t mid = (lo + hi + 1) / 2;
            if (first_tile<kRows>(a, mid) <= x) lo = mid;
            else hi = mid - 1;
        }
        t.n = (int)lo;
        tile = x - first_tile<kRows>(a, lo);
    }
    const int2 r = rows_of(a, t.n);
    t.first = r.x;
    t.len = __ldg(a.kv_lens + t.n);
    t.past = t.len - r.y;
    const int64_t left = (int64_t)r.y * a.group - tile * kRows;
    t.row0 = (int)(tile * kRows);
    t.rows = left <= 0 ? 0 : (int)(left < kRows ? left : kRows);
    // keys that the last row sees, and this split's tiles of them
    const int far = a.causal ? max(0, min(t.len, t.past + token_of(a, t.row0 + t.rows - 1) + 1)) : t.len;
    const int all = t.rows ? (far + kKeys - 1) / kKeys : 0, per = (all + plan.splits - 1) / plan.splits;
    t.j0 = min(all, split * per);
    t.count = min(all, t.j0 + per) - t.j0;
    t.part = (x * a.kv_heads + t.head) * plan.splits + split;
    t.later = t.more = false;
    if (kLong) {
        const int before = turn.piece * kMost;
        t.later = turn.piece > 0;
        t.more = t.count - before > kMost;
        t.j0 += before;
        t.count = t.more ? kMost : t.count - before;
    }
    turn.piece = t.more ? turn.piece + 1 : 0;
    turn.k = t.more ? k : k + 1;
    return true;
}

// 16 columns of this thread's TMEM lane, the wait apart; the wait names every register, so that no use
// comes before it.
__device__ __forceinline__ void tmem_fetch16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_arrive16(uint32_t (&r)[16]) {
#pragma unroll
    for (int i = 0; i < 16; i += 8)
        asm volatile("tcgen05.wait::ld.sync.aligned;"
                     : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]), "+r"(r[i + 6]),
                       "+r"(r[i + 7])::"memory");
}
// 16 columns stored, the wait apart (tmem_stored).
__device__ __forceinline__ void tmem_put16(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// What becomes of scores: nothing more, a cap, or a bias by distance with or without a cap. bf16: the quick form of a cap is
// off by up to 2^-21 of it whatever the score, 3e-5 of caps up to kCaps (a usual one is 30 or 50; lse off by 1.4e-6 at
// 64, 2.2e-5 at 1000). Higher ones go the third way, where 1000 rows of heads of 256 behind 32,768 tokens take 1066 us for 643.
constexpr float kCaps = 64.f;
enum { kPlain = 0, kCapped = 1, kBiased = 2 };

// Exponents of 16 keys' weights from products with their codes: m scales a product (log2(e) in it if
// kPlain), off: log2 of the value scale less the row's reference, away: p - j of the first key.
// tanh(x) = 1 - 2 / (1 + e^2x) as in cache_attn.cuh; of a capped score the rest folds into one multiply-add.
template <int kMode, bool kExact> struct Shape {
    float m, off, cap, slope, away, k;
    __device__ __forceinline__ Shape(float m_, float off_, float cap_, float inv_cap, float slope_, float away_)
        : m(m_), off(off_), cap(cap_), slope(slope_), away(away_), k(0.f) {
        if (kMode == kCapped && !kExact) {
            m = m_ * inv_cap * (2.f * kLog2e);
            off = fmaf(cap_, kLog2e, off_);
            k = -2.f * kLog2e * cap_;
        } else if (kMode != kPlain && cap_ > 0.f) {
            k = inv_cap;
        }
    }
    __device__ __forceinline__ float one(float z, int e) const {
        z *= m;
        if (cap > 0.f) z = cap * cap_of<kExact>(z * k);
        if (kMode == kBiased) z = fmaf(-slope, fabsf(away - (float)e), z);
        return fmaf(z, kLog2e, off);
    }
    // Keys e .. e + 3.
    __device__ __forceinline__ void operator()(const uint32_t *bits, int e, float2 &t0, float2 &t1) const {
        const float2 z0 = make_float2(__uint_as_float(bits[0]), __uint_as_float(bits[1]));
        const float2 z1 = make_float2(__uint_as_float(bits[2]), __uint_as_float(bits[3]));
        if (kMode == kPlain) {
            t0 = fma2(z0, make_float2(m, m), make_float2(off, off));
            t1 = fma2(z1, make_float2(m, m), make_float2(off, off));
        } else if (kMode == kCapped && !kExact) {
            // four reciprocals from one (the special functions bound capped scores: 12 cycles of theirs a key with one
            // each, 6 so): exponents are held below 30, where tanh is 1, so that no product overflows
            const float2 x0 = mul2(z0, make_float2(m, m)), x1 = mul2(z1, make_float2(m, m));
            const float2 a = add2(make_float2(ex2(below(x0.x)), ex2(below(x1.x))), make_float2(1.f, 1.f));
            const float2 b = add2(make_float2(ex2(below(x0.y)), ex2(below(x1.y))), make_float2(1.f, 1.f));
            const float2 ab = mul2(a, b);
            const float r = reciprocal(ab.x * ab.y);
            const float2 q = mul2(make_float2(r, r), make_float2(ab.y, ab.x));  // reciprocals of ab
            t0 = fma2(mul2(make_float2(q.x, q.x), make_float2(b.x, a.x)), make_float2(k, k), make_float2(off, off));
            t1 = fma2(mul2(make_float2(q.y, q.y), make_float2(b.y, a.y)), make_float2(k, k), make_float2(off, off));
        } else {
            t0 = make_float2(one(z0.x, e), one(z0.y, e + 1));
            t1 = make_float2(one(z1.x, e + 2), one(z1.y, e + 3));
        }
    }
    static __device__ __forceinline__ float below(float x) {  // (NaN stays NaN)
        float y;
        asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(30.f));
        return y;
    }
};

__device__ __forceinline__ uint4 load16(uint32_t saddr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(saddr) : "memory");
    return v;
}
// Issued where it stands: a load that the compiler may move ends up next to its use.
__device__ __forceinline__ uint4 ld_nc(const void *p) {
    uint4 v;
    asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ void store16(uint32_t saddr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(saddr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

__device__ __forceinline__ void store8(uint32_t saddr, uint32_t x, uint32_t y) {
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(saddr), "r"(x), "r"(y) : "memory");
}

__device__ __forceinline__ bool elect() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}
template <int kRegs> __device__ __forceinline__ void set_registers_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs)); }
template <int kRegs> __device__ __forceinline__ void set_registers_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs)); }

template <typename T, int D, int kParts, int kMode, int kCode, bool kLong>
__global__ void __launch_bounds__(kTcThreads, 1) attn_tc_kernel(const __grid_constant__ Attn a, const __grid_constant__ TcPlan plan, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
    using C = TcConfig<D, kParts>;
    extern __shared__ unsigned char sm[];
    const uint32_t base = (smem_u32(sm) + 1023u) & ~1023u;
    const uint32_t sq = base, sk = base + C::kTiles * kParts * C::kQ, sv = sk + C::kStages * C::kKv, sr = sv + C::kStages * C::kKv;
    __shared__ float4 scales[kRing][4];  // of 16 keys: key scale, log2 and reciprocal of the value scale
    __shared__ uint32_t tmem_slot;
    __shared__ int gave_up, copied;  // whether a wait ran out; tiles that have been asked for, of keys and values in turn
    __shared__ int held[kRing];  // 5 bits for each 16 keys: the rows that there are
    // Of the stages of keys and values, and of their codes (R); of the scores' slots (2 tile + parity of the key tile); per row tile
    enum { K_FULL = 0, K_FREE = 4, V_FULL = 8, V_FREE = 12, S_FULL = 16, W_FULL = 20, O_DONE = 24, Q_FULL = 28, O_FREE = 30, O_LAST = 32, RK_FULL = 34, RK_FREE = 37, RV_FULL = 40, RV_FREE = 43, BARS = 46 };
    __shared__ __align__(8) uint64_t bars[BARS];
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        gave_up = copied = 0;
        for (int s = 0; s < 4; ++s) {
            mbar_init(bar(K_FULL + s), C::kConv);
            mbar_init(bar(V_FULL + s), C::kConv);
            mbar_init(bar(K_FREE + s), C::kTiles);
            mbar_init(bar(V_FREE + s), C::kTiles);
            mbar_init(bar(S_FULL + s), 1);
            mbar_init(bar(W_FULL + s), 128);
            mbar_init(bar(O_DONE + s), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(Q_FULL + s), 128);
            mbar_init(bar(O_FREE + s), 128);
            mbar_init(bar(O_LAST + s), 1);
        }
        for (int s = 0; s < 3; ++s) {
            mbar_init(bar(RK_FULL + s), 1);
            mbar_init(bar(RV_FULL + s), 1);
            mbar_init(bar(RK_FREE + s), C::kConv / 32);
            mbar_init(bar(RV_FREE + s), C::kConv / 32);
        }
        fence_mbar_init();
    }
    bool good = true;
    for (int64_t n = tid; n < a.num_seqs; n += kTcThreads) good = good && lengths_hold(a, n);
    const bool ok = __syncthreads_and(good);
    if (tid == 0 && blockIdx.x == 0) *a.status = ok ? GDR_OK : GDR_ERR_BAD_SEQLENS;
    if (!ok) return;
    if (warp == 12) {
        tmem_alloc(smem_u32(&tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    bool fine = true;
    TcItem item;
    TcTurn turn;
    int gi0 = 0;       // tiles of keys before this item

    if (warp < C::kSoft / 32) {
        // ---------------------------------------------------------------- softmax
        set_registers_up<C::kSoftRegs>();
        const int tile = warp >> 2;  // row tile
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const uint32_t out = tmem + lanes + C::kO + tile * D;
        const float cap = kMode == kPlain ? 0.f : a.softcap, inv_cap = cap > 0.f ? 1.f / cap : 0.f;
        using P = Part<C::kRows, D>;
        auto row_of = [&](const TcItem &t) {
            const int at = t.row0 + tid, token = token_of(a, at);
            return (int64_t)(t.first + token) * a.heads + t.head * a.group + at - token * a.group;
        };
        auto query_of = [&](const TcItem &t) {
            const int at = t.row0 + tid, token = token_of(a, at);
            return (const T *)a.q + (int64_t)(t.first + token) * a.qs + (int64_t)(t.head * a.group + at - token * a.group) * D;
        };
        // The next item that has keys to look at; those before it that have none get their zeros.
        auto next_item = [&](TcItem &t) {
            while (get_item<C::kRows, C::kKeys, kLong>(a, plan, turn, t)) {
                if (t.count) return true;
                if (tid >= t.rows) continue;
                P *const part = (P *)plan.parts + t.part;
                const int64_t row = row_of(t);
                if (plan.splits > 1) part->lse2[tid] = -INFINITY;
                else if (a.lse) a.lse[row] = -INFINITY;
                uint4 *const to = plan.splits > 1 ? (uint4 *)part->o[tid] : (uint4 *)((T *)a.o + row * D);
                const int vecs = (plan.splits > 1 ? 4 : (int)sizeof(T)) * D / 16;
                for (int e = 0; e < vecs; ++e) to[e] = make_uint4(0, 0, 0, 0);
            }
            return false;
        };
        // This warp's 32 rows of queries in fp16 with a power of two each, its sign that of the scale; returns what products
        // with this thread's are to be multiplied by. Lanes share a row, so that a load takes whole lines of few rows (a row
        // to a thread: 32 lines a load, 4096 cycles of them for an item of two row tiles).
        auto put_queries = [&](const TcItem &t) {
            constexpr int kVecs = D * (int)sizeof(T) / 16, kLanes = kVecs < 32 ? kVecs : 32, kPieces = kVecs / kLanes;
            constexpr int kAtOnce = 32 / kLanes, kBatch = 16 / kPieces < kLanes ? 16 / kPieces : kLanes;  // rows of a load; loads under way
            const uint64_t mine = (uint64_t)query_of(t);
            const uint32_t alive = __ballot_sync(~0u, tid < t.rows);
            const uint32_t to = sq + tile * kParts * C::kQ;
            const int sub = lane % kLanes;
            int my_shift = 0;
#pragma unroll 1
            for (int j0 = 0; j0 < kLanes; j0 += kBatch) {
                uint4 w[kBatch][kPieces];
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    const int r = (j0 + j) * kAtOnce + lane / kLanes;
                    const char *const src = (const char *)__shfl_sync(~0u, mine, r);
#pragma unroll
                    for (int x = 0; x < kPieces; ++x) w[j][x] = alive >> r & 1 ? ld_nc(src + (x * 32 + sub) * 16) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    const int r = (j0 + j) * kAtOnce + lane / kLanes;
                    uint32_t most = 0;
#pragma unroll
                    for (int x = 0; x < kPieces; ++x) {
                        const uint4 &q = w[j][x];
                        if constexpr (sizeof(T) == 2) {
                            most = __vmaxu2(__vmaxu2(q.x & 0x7fff7fffu, q.y & 0x7fff7fffu), __vmaxu2(q.z & 0x7fff7fffu, q.w & 0x7fff7fffu));
                            most = max(most & 0xffffu, most >> 16) << 16;
                        } else {
                            most = max(most, max(max(q.x & 0x7fffffffu, q.y & 0x7fffffffu), max(q.z & 0x7fffffffu, q.w & 0x7fffffffu)));
                        }
                    }
#pragma unroll
                    for (int d = 1; d < kLanes; d *= 2) most = max(most, __shfl_xor_sync(~0u, most, d));
                    const int shift = row_shift(most), its = __shfl_sync(~0u, shift, lane % kAtOnce * kLanes);
                    if (lane / kAtOnce == j0 + j) my_shift = its;
                    const float up = a.scale < 0.f ? -two_to(shift) : two_to(shift);
                    const float2 up_pair = make_float2(up, up);
#pragma unroll
                    for (int x = 0; x < kPieces; ++x) {
                        const uint32_t in[4] = {w[j][x].x, w[j][x].y, w[j][x].z, w[j][x].w};
                        constexpr int kPairs = 8 / (int)sizeof(T);
                        uint32_t hi[kPairs], lo[kPairs];
#pragma unroll
                        for (int i = 0; i < kPairs; ++i) {
                            float2 z;
                            if constexpr (sizeof(T) == 2) z = make_float2(__uint_as_float(in[i] << 16), __uint_as_float(in[i] & 0xffff0000u));
                            else z = make_float2(__uint_as_float(in[2 * i]), __uint_as_float(in[2 * i + 1]));
                            z = mul2(z, up_pair);
                            hi[i] = pack_f16(z.x, z.y);
                            if (kParts == 2) {
                                const float2 f = unpack_f16(hi[i]);
                                lo[i] = pack_f16(z.x - f.x, z.y - f.y);
                            }
                        }
                        const int d = (x * 32 + sub) * (16 / (int)sizeof(T));
                        const uint32_t dst = to + (d >> 6) * 16384 + sw128_offset((warp & 3) * 32 + r, d & 63);
                        if constexpr (sizeof(T) == 2) {
                            store16(dst, hi[0], hi[1], hi[2], hi[3]);
                        } else {
                            store8(dst, hi[0], hi[1]);
                            store8(dst + C::kQ, lo[0], lo[1]);
                        }
                    }
                }
            }
            fence_async_smem();
            mbar_arrive(bar(Q_FULL + tile));
            return two_to(-my_shift) * fabsf(a.scale);
        };

        bool have = next_item(item);
        float row_up = have ? put_queries(item) : 0.f;
        for (int done = 0; have && fine; ++done) {
            const int at = item.row0 + tid;
            const int p = item.past + token_of(a, at), lim = a.causal ? min(item.len, p + 1) : item.len;
            const int sure = a.causal ? min(item.len, item.past + token_of(a, item.row0 + tile * 128) + 1) : item.len;
            const bool live = tid < item.rows;
            const int64_t row = row_of(item);
            P *const part = (P *)plan.parts + item.part;
            float *const row_out = plan.splits > 1 ? part->o[tid] : (float *)a.o + row * D;  // (fp32 only without splits)
            const float slope = kMode == kBiased && a.slopes && live ? __ldg(a.slopes + item.head * a.group + at - token_of(a, at) * a.group) : 0.f;
            const float up2 = row_up * (kMode == kPlain ? kLog2e : 1.f);
            float ref = 0.f, l = 0.f;
            float sum_ref = 0.f, sum_l = 0.f;  // kParts == 2: of what has left TMEM
            const int count = item.count, j0 = item.j0;
            TcItem then;
            have = next_item(then);
            if (have && tid < then.rows)
                for (int e = 0; e < D * (int)sizeof(T); e += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"((const char *)query_of(then) + e));

            // fp32: the outputs of kFlush tiles leave TMEM and are added up in memory.
            auto flush = [&] {
                const bool some = sum_l != 0.f;
                const float by = some ? ex2(sum_ref - ref) : 0.f;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float v[32];
                    __syncwarp();  // (a warp reads its lanes together)
                    tmem_load32(out + c, v);
                    if (!live) continue;
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        float4 o = some ? *(const float4 *)(row_out + c + e) : make_float4(0.f, 0.f, 0.f, 0.f);
                        o = make_float4(fmaf(o.x, by, v[e]), fmaf(o.y, by, v[e + 1]), fmaf(o.z, by, v[e + 2]), fmaf(o.w, by, v[e + 3]));
                        *(float4 *)(row_out + c + e) = o;
                    }
                }
                sum_l = fmaf(sum_l, by, l);
                sum_ref = ref;
                l = 0.f;
            };

#pragma unroll 1
            for (int i = 0; i < count && fine; ++i) {
                const int gi = gi0 + i, slot = 2 * tile + (gi & 1);
                const uint32_t s_at = tmem + lanes + slot * C::kKeys;
                if (!mbar_wait(bar(S_FULL + slot), (gi >> 1) & 1)) {
                    fine = false;
                    break;
                }
                // The outputs of the tiles before: the scores' barrier says that those of the last but one are there,
                // and those of the last have a barrier that even and odd tiles share in turn.
                auto outputs_done = [&] {
                    if (!mbar_wait(bar(O_DONE + 2 * tile + ((gi - 1) & 1)), ((gi - 1) >> 1) & 1)) fine = false;
                    __syncwarp();
                    tc_fence_after();
                };
                __syncwarp();
                tc_fence_after();
                const bool anew = kParts == 2 && i % kFlush == 0;  // (this tile's product begins the outputs)
                if (anew && i > 0) {
                    outputs_done();
                    if (!__all_sync(~0u, fine)) break;
                    flush();
                }
                const int tok = (j0 + i) * C::kKeys;
                const float4 *const sc = scales[gi % kRing];
                const bool edge = tok + C::kKeys > sure;

                // Exponents of all weights first, relative to the row's reference: the first tile, or one that is too large,
                // moves the reference, and the outputs so far with it. (A row that sees no key of the first tile sees
                // no later ones.)
                float2 t[C::kKeys / 2];
#pragma unroll 1
                for (bool again = i > 0;;) {
                    {
                        uint32_t x[C::kKeys / 16][16];
#pragma unroll
                        for (int g = 0; g < C::kKeys / 16; ++g) tmem_fetch16(s_at + 16 * g, x[g]);
#pragma unroll
                        for (int g = 0; g < C::kKeys / 16; ++g) {
                            tmem_arrive16(x[g]);
                            const float4 f = sc[g];
                            const Shape<kMode, kParts == 2> shape(f.x * up2, f.y - ref, cap, inv_cap, slope, (float)(p - tok - 16 * g));
#pragma unroll
                            for (int e = 0; e < 16; e += 4) shape(x[g] + e, e, t[8 * g + e / 2], t[8 * g + e / 2 + 1]);
                        }
                    }
                    if (edge) {
#pragma unroll
                        for (int e = 0; e < C::kKeys; e += 2) {
                            if (tok + e >= lim) t[e / 2].x = -INFINITY;
                            if (tok + e + 1 >= lim) t[e / 2].y = -INFINITY;
                        }
                    }
                    float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int e = 0; e < C::kKeys / 2; ++e) tops[e & 3] = fmaxf(tops[e & 3], fmaxf(t[e].x, t[e].y));
                    const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                    const bool move = i == 0 ? top > -INFINITY : top > kSpan + kSlack;
                    if (!__any_sync(~0u, move)) break;
                    // (a whole number: references below 2^24 move without a rounding)
                    const float up = move ? rintf(top) - kSpan : 0.f;
                    ref += up;
                    if (i > 0) {
                        const float by = ex2(-up);
                        l *= by;
                        if (!anew) {
                            outputs_done();
                            // (32 columns a time: 4 x 4096 tokens 250 us, by 16 260)
#pragma unroll 1
                            for (int c = 0; c < D; c += 32) {
                                float v[32];
                                tmem_load32(out + c, v);
                                uint32_t u[32];
#pragma unroll
                                for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(v[e] * by);
                                tmem_put16(out + c, u);
                                tmem_put16(out + c + 16, u + 16);
                            }
                            tmem_stored();
                        }
                    }
                    // An exponent far above the old reference (a bias by distance lifts it so from tile to tile) has lost bits to
                    // rounding, 2^-25 of its height: beyond 2^-15 of a weight (fp32: 2^-20) all are taken anew.
                    if (again && __any_sync(~0u, up > (kParts == 2 ? 32.f : 1024.f))) {
                        again = false;
                        continue;
                    }
#pragma unroll
                    for (int e = 0; e < C::kKeys / 2; ++e) t[e] = add2(t[e], make_float2(-up, -up));
                    break;
                }
                // the weights, in the scores' place
#pragma unroll
                for (int c = 0; c < C::kKeys / 2; c += 16) {
                    uint32_t hi[16], lo[kParts == 2 ? 16 : 1];
                    float2 some[2];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float2 w = make_float2(ex2(t[c + e].x), ex2(t[c + e].y));
                        some[e / 8] = e % 8 ? add2(some[e / 8], w) : w;
                        hi[e] = pack_f16(w.x, w.y);
                        if (kParts == 2) {
                            const float2 v = unpack_f16(hi[e]);
                            lo[e] = pack_f16(w.x - v.x, w.y - v.y);
                        }
                    }
                    tmem_put16(s_at + c, hi);
                    if constexpr (kParts == 2) tmem_put16(tmem + lanes + C::kLow + (gi & 1) * C::kLowStep + c, lo);
                    l = fmaf(some[0].x + some[0].y, sc[c / 8].z, l);
                    l = fmaf(some[1].x + some[1].y, sc[c / 8 + 1].z, l);
                }
                tmem_stored();
                tc_fence_before();
                mbar_arrive(bar(W_FULL + slot));
            }
            gi0 += count;
            // ---- the next item's queries (the scores of the last tile are there, and were the last to need these), then the
            // results. A warp reads its lanes together, whichever rows are live.
            if (!__all_sync(~0u, fine)) break;
            if (have) row_up = put_queries(then);
            fine = mbar_wait(bar(O_LAST + tile), done & 1);
            if (!__all_sync(~0u, fine)) {
                fine = false;
                break;
            }
            tc_fence_after();
            // Outputs from before, if there are `older` ones, stand at `from` and are to be multiplied by `by`, these by `now`.
            float by = kParts == 2 ? ex2(sum_ref - ref) : 0.f, now = 1.f;
            static_assert(!kLong || kParts == 1, "fp32 outputs leave TMEM anyway");
            bool older = kParts == 2 && sum_l != 0.f;
            TcPiece<D> *const piece = (TcPiece<D> *)plan.pieces + (int64_t)blockIdx.x * C::kRows + tid;
            const float *const from = kLong ? piece->o : row_out;
            if (kLong && item.later && live) {
                sum_ref = piece->ref;
                sum_l = piece->l;
                older = sum_l != 0.f;
                const float most = older ? fmaxf(sum_ref, l != 0.f ? ref : sum_ref) : ref;
                by = ex2(sum_ref - most);
                now = l != 0.f ? ex2(ref - most) : 0.f;
                ref = most;
                l *= now;
            }
            if (older) l = fmaf(sum_l, by, l);
            const bool some = l != 0.f;
            const bool more = kLong && item.more;
            const float inv = more ? 1.f : some ? 1.f / l : 0.f;
            if (more && live) {
                piece->ref = ref;
                piece->l = l;
            }
            if (live && !more) {
                const float sum2 = some ? log2f(l) + ref : -INFINITY;
                if (plan.splits > 1) part->lse2[tid] = sum2;
                else if (a.lse) a.lse[row] = sum2 * kLn2;
            }
            // 64 bytes of every row: through shared memory, four lanes to a row (a row to a thread: 32 lines a store)
            char *const mine = more ? (char *)piece->o : plan.splits > 1 ? (char *)part->o[tid] : (char *)((T *)a.o + row * D);
            const uint32_t alive = __ballot_sync(~0u, live);
            auto hand_out = [&](const uint32_t *w, int at) {
                if constexpr (C::kStage == 0) {
                    if (live) {
#pragma unroll
                        for (int x = 0; x < 4; ++x) *(uint4 *)(mine + at + 16 * x) = make_uint4(w[4 * x], w[4 * x + 1], w[4 * x + 2], w[4 * x + 3]);
                    }
                    __syncwarp();
                } else {
                    const uint32_t stage = sr + C::kRaw * C::kKv + warp * 2048;
#pragma unroll
                    for (int x = 0; x < 4; ++x) store16(stage + lane * 64 + ((x ^ (lane >> 1)) & 3) * 16, w[4 * x], w[4 * x + 1], w[4 * x + 2], w[4 * x + 3]);
                    __syncwarp();
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int r = x * 8 + (lane >> 2);
                        const uint4 y = load16(stage + r * 64 + ((lane ^ (r >> 1)) & 3) * 16);
                        char *const to = (char *)__shfl_sync(~0u, (uint64_t)mine, r);
                        if (alive >> r & 1) *(uint4 *)(to + at + (lane & 3) * 16) = y;
                    }
                    __syncwarp();
                }
            };
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                float v[32];
                if (kParts == 2 || kLong) __syncwarp();
                tmem_load32(out + c, v);
                if (older && live) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const float4 o = *(const float4 *)(from + c + e);
                        v[e] = fmaf(o.x, by, v[e] * now);
                        v[e + 1] = fmaf(o.y, by, v[e + 1] * now);
                        v[e + 2] = fmaf(o.z, by, v[e + 2] * now);
                        v[e + 3] = fmaf(o.w, by, v[e + 3] * now);
                    }
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] *= inv;
                if (more || plan.splits > 1 || sizeof(T) == 4) {
#pragma unroll
                    for (int e = 0; e < 32; e += 16) {
                        uint32_t w[16];
#pragma unroll
                        for (int x = 0; x < 16; ++x) w[x] = __float_as_uint(v[e + x]);
                        hand_out(w, (c + e) * 4);
                    }
                } else {
                    uint32_t w[16];
#pragma unroll
                    for (int x = 0; x < 16; ++x) {
                        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * x], v[2 * x + 1]);
                        w[x] = reinterpret_cast<const uint32_t &>(b);
                    }
                    hand_out(w, c * 2);
                }
            }
            tc_fence_before();
            mbar_arrive(bar(O_FREE + tile));
            item = then;
        }
    } else if (warp < 12) {
        // ---------------------------------------------------------------- codes to fp16
        set_registers_down<C::kConvRegs>();
        const int ct = tid - C::kSoft, cw = ct >> 5;
        constexpr int kBlocks = D / 64;                     // 64 dims to a swizzled block of rows
        constexpr int kWarpRows = 8 / kBlocks;              // rows of a warp's pass of 512 bytes
        constexpr int kPass = kWarpRows * (C::kConv / 32);  // rows of a pass
        constexpr int kPasses = C::kKeys / kPass;
        // Eight lanes in turn read chunks x of codes and write chunks 2x and 2x + 1 of two rows. In 128-byte-swizzled
        // rows r and r ^ 5 no two of them meet in a bank, either way; D = 64, whose codes lie in plain rows of 64 bytes,
        // takes r and r + 1.
        const int x = lane & 3, blk = (lane >> 3) & (kBlocks - 1), odd = (lane >> 2) & 1;
        const int pair = kBlocks == 4 ? cw & 3 : (cw & 1) * 2 + (lane >> 4);
        const int row = kBlocks == 1 ? cw * 8 + odd + 2 * (lane >> 3) : cw / (kBlocks == 4 ? 4 : 2) * 8 + (odd ? pair ^ 5 : pair);
        const uint32_t chunk0 = (uint32_t)((2 * x) ^ (row & 7)) << 4;  // its first 16-byte chunk; the second is one bit away
        const uint32_t to0 = blk * (C::kKeys * 128) + row * 128, 
                       from0 = kBlocks == 1 ? row * 64 + x * 16 : (blk >> 1) * (C::kKeys * 128) + row * 128 + (((blk & 1) * 4 + x) ^ (row & 7)) * 16;
        while (fine && get_item<C::kRows, C::kKeys, kLong>(a, plan, turn, item)) {
            const int count = item.count;
#pragma unroll 1
            for (int t = 0; t < 2 * count; ++t) {  // keys and values in turn
                const int gi = gi0 + (t >> 1), is_v = t & 1, st = gi % C::kStages, raw = gi % C::kRaw;
                if (!mbar_wait(bar((is_v ? RV_FULL : RK_FULL) + raw), (gi / C::kRaw) & 1) ||
                    !mbar_wait(bar((is_v ? V_FREE : K_FREE) + st), ((gi / C::kStages) & 1) ^ 1)) {
                    fine = false;
                    break;
                }
                const uint32_t from = sr + raw * C::kKv + is_v * (C::kKv / 2) + from0, to = (is_v ? sv : sk) + st * C::kKv + to0;
                uint4 w[kPasses];
#pragma unroll
                for (int ps = 0; ps < kPasses; ++ps) w[ps] = load16(from + ps * kPass * (kBlocks == 1 ? 64 : 128));
                const int rows = held[gi % kRing];
                if (rows != kAll) {  // places of no token, or of a page that is none
#pragma unroll
                    for (int ps = 0; ps < kPasses; ++ps) {
                        const int r = ps * kPass + row;
                        if ((r & 15) >= ((rows >> (r / 16 * 5)) & 31)) w[ps] = make_uint4(0, 0, 0, 0);
                    }
                }
#pragma unroll
                for (int ps = 0; ps < kPasses; ++ps) {
                    uint32_t f[8];
                    codes::to_f16x4<kCode>(w[ps].x, f[0], f[1]);
                    codes::to_f16x4<kCode>(w[ps].y, f[2], f[3]);
                    codes::to_f16x4<kCode>(w[ps].z, f[4], f[5]);
                    codes::to_f16x4<kCode>(w[ps].w, f[6], f[7]);
                    // (kPass is a multiple of 8: a thread's rows have one place in the swizzle)
                    store16(to + ps * kPass * 128 + chunk0, f[0], f[1], f[2], f[3]);
                    store16(to + ps * kPass * 128 + (chunk0 ^ 16), f[4], f[5], f[6], f[7]);
                }
                fence_async_smem();
                mbar_arrive(bar((is_v ? V_FULL : K_FULL) + st));
                __syncwarp();
                if (lane == 0) mbar_arrive(bar((is_v ? RV_FREE : RK_FREE) + raw));
            }
            gi0 += count;
        }
    } else if (warp < 12 + C::kTiles) {
        // ---------------------------------------------------------------- products
        const int tile = warp - 12;  // row tile
        const uint32_t id_s = idesc_f16(128, C::kKeys, 0), id_o = idesc_f16(128, D, 1);
        // (the low parts first: a sum is cut while it is small)
        auto scores = [&](int gi) {
            const int slot = 2 * tile + (gi & 1);
            const uint32_t kt = desc_k(sk + (gi % C::kStages) * C::kKv), qt = desc_k(sq + tile * kParts * C::kQ);
            if (elect()) {
#pragma unroll
            for (int x = kParts - 1; x >= 0; --x)
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_ss(tmem + slot * C::kKeys, qt + ((x * C::kQ + (kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                           kt + (((kk >> 2) * (C::kKeys * 128) + (kk & 3) * 32) >> 4), id_s, x < kParts - 1 || kk > 0);
            mma_commit(bar(S_FULL + slot));
            }
            __syncwarp();
        };
        auto outputs = [&](int gi, int i) {
            const int slot = 2 * tile + (gi & 1);
            const uint32_t vt = desc_mn(sv + (gi % C::kStages) * C::kKv, C::kKeys * 128);
            const bool add = (kParts == 2 ? i % kFlush : i) > 0;
            if (elect()) {
#pragma unroll
            for (int x = kParts - 1; x >= 0; --x)
#pragma unroll
                for (int kk = 0; kk < C::kKeys / 16; ++kk)
                    mma_ts(tmem + C::kO + tile * D, (x == 0 ? tmem + slot * C::kKeys : tmem + C::kLow + (gi & 1) * C::kLowStep) + 8 * kk,
                           vt + ((kk * 2048) >> 4), id_o, add || x < kParts - 1 || kk > 0);
            mma_commit(bar(O_DONE + slot));
            }
            __syncwarp();
        };
        auto wait = [&](int b, uint32_t parity) {
            if (fine) fine = mbar_wait(bar(b), parity & 1);
            if (b >= W_FULL) tc_fence_after();
            return fine;
        };
        int done = 0;
        while (fine && get_item<C::kRows, C::kKeys, kLong>(a, plan, turn, item)) {
            const int count = item.count;
            if (!count) continue;
            wait(Q_FULL + tile, done);
            // (each product is written once: warps far apart in the code cost instruction fetches)
#pragma unroll 1
            for (int i = -1; i < count && fine; ++i) {
                const int gi = gi0 + i;
                if (i + 1 < count) {
                    const int st = (gi + 1) % C::kStages;
                    if (!wait(K_FULL + st, (gi + 1) / C::kStages)) break;
                    scores(gi + 1);
                    if (elect()) mma_commit(bar(K_FREE + st));
                }
                if (i >= 0) {
                    const int st = gi % C::kStages;
                    if (!wait(V_FULL + st, gi / C::kStages)) break;
                    if (!wait(W_FULL + 2 * tile + (gi & 1), gi >> 1)) break;
                    if (i == 0 && done > 0 && !wait(O_FREE + tile, done - 1)) break;
                    outputs(gi, i);
                    if (elect()) mma_commit(bar(V_FREE + st));
                }
            }
            if (elect()) mma_commit(bar(O_LAST + tile));
            gi0 += count;
            ++done;
        }
        // (also after a wait that ran out: what was issued ends before the TMEM goes)
        if (!fine) mbar_wait(bar(O_LAST + tile), (done - 1) & 1);
    } else if (warp == 12 + C::kTiles) {
        // ---------------------------------------------------------------- copies
        const int in_page = (1 << a.log_page) - 1, box = min(C::kKeys, in_page + 1);
        while (fine && get_item<C::kRows, C::kKeys, kLong>(a, plan, turn, item)) {
            const int count = item.count, j0 = item.j0, len = item.len;
            const int32_t *const table = a.table + (int64_t)item.n * a.width;
            // Lane g < 4 sees to 16 keys of a tile. Their page: -1 behind the last token, -2 outside the cache.
            auto page_of = [&](int i) {
                const int tok = (j0 + i) * C::kKeys + lane * 16;
                if (i >= count || lane >= 4 || tok >= len) return -1;
                const int pg = __ldg(table + (tok >> a.log_page));
                return pg >= 0 && pg < a.pages ? pg : -2;
            };
            auto scale_of = [&](int pg) {
                if (pg < 0) return make_float2(pg == -1 ? 1.f : __int_as_float(0x7fffffff), pg == -1 ? 1.f : __int_as_float(0x7fffffff));
                const int64_t at = (int64_t)pg * a.kv_heads + item.head;
                return make_float2(__ldg(a.ks + at), __ldg(a.vs + at));
            };
            int page = page_of(0), next = page_of(1);
            float2 scale = scale_of(page);
#pragma unroll 1
            for (int i = 0; i < count && fine; ++i) {
                const int gi = gi0 + i, raw = gi % C::kRaw, tok = (j0 + i) * C::kKeys + lane * 16;
                const float2 coming = scale_of(next);
                const int later = page_of(i + 2);
                const int rows = page >= 0 ? min(16, len - tok) : 0;
                const int all = __shfl_sync(~0u, rows, 0) | __shfl_sync(~0u, rows, 1) << 5 | __shfl_sync(~0u, rows, 2) << 10 | __shfl_sync(~0u, rows, 3) << 15;
                // a copy brings as many rows as a page and a tile have in common, all of one page
                const bool copies = rows > 0 && lane * 16 % box == 0;
                const int boxes = __popc(__ballot_sync(~0u, copies));
                if (lane < 4)
                    scales[gi % kRing][lane] = make_float4(scale.x, lg2(scale.y), scale.y == scale.y ? __fdividef(1.f, scale.y) : 1.f, 0.f);
                if (lane == 0) held[gi % kRing] = all;
                __syncwarp();
#pragma unroll 1
                for (int is_v = 0; is_v < 2; ++is_v) {
                    const uint32_t full = bar((is_v ? RV_FULL : RK_FULL) + raw);
                    if (!mbar_wait(bar((is_v ? RV_FREE : RK_FREE) + raw), ((gi / C::kRaw) & 1) ^ 1)) fine = false;
                    fine = __all_sync(~0u, fine);
                    if (!fine) {
                        if (lane == 0) copied = 2 * gi + is_v;
                        break;
                    }
                    if (lane == 0) mbar_arrive_expect_tx(full, boxes * box * D);
                    __syncwarp();
                    if (copies) {
                        const int at = item.head * (in_page + 1) + (tok & in_page);
                        const uint32_t to = sr + raw * C::kKv + is_v * (C::kKv / 2) + lane * 16 * (D < 128 ? D : 128);
#pragma unroll
                        for (int x = 0; x < D; x += 128) tma_load_3d(to + x * C::kKeys, is_v ? &v_map : &k_map, full, x, at, page);
                    }
                }
                page = next;
                next = later;
                scale = coming;
            }
            gi0 += count;
            if (fine && lane == 0) copied = 2 * gi0;
        }
    }
    if (!fine) gave_up = 1;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 12) tmem_dealloc(tmem, 512);
    if (tid == 0 && gave_up) {  // no copy outlives the block: the last ones are waited for, again with a limit
        for (int is_v = 0; is_v < 2; ++is_v) {
            const int n = (copied + 1 - is_v) / 2;
            for (int i = max(0, n - C::kRaw); i < n; ++i) mbar_wait(bar((is_v ? RV_FULL : RK_FULL) + i % C::kRaw), (i / C::kRaw) & 1);
        }
        *a.status = GDR_ERR_DEVICE_TIMEOUT;
    }
}

// Adds the splits of an item in order: a warp to a row.
template <typename T, int D, int kParts> __global__ void __launch_bounds__(256) join_splits_kernel(const __grid_constant__ Attn a, const TcPlan plan) {
    using C = TcConfig<D, kParts>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (*(volatile int32_t *)a.status != GDR_OK) return;
    const int64_t row = (int64_t)blockIdx.x * 8 + warp;  // of o
    const int64_t t = row / a.heads;
    if (t >= a.tokens) return;
    const int h = (int)(row - t * a.heads), head = h / a.group;
    int64_t n = a.cu ? 0 : t / a.max_q;
    if (a.cu) {
        if (t >= __ldg(a.cu + a.num_seqs)) return;
        int64_t hi = a.num_seqs - 1;  // the first request that ends behind t
        while (n < hi) {
            const int64_t mid = (n + hi) / 2;
            if (__ldg(a.cu + mid + 1) > t) hi = mid;
            else n = mid + 1;
        }
    }
    const int64_t r = (t - rows_of(a, n).x) * a.group + h % a.group, tile = r / C::kRows;
    const Part<C::kRows, D> *const parts =
        (const Part<C::kRows, D> *)plan.parts + ((first_tile<C::kRows>(a, n) + tile) * a.kv_heads + head) * plan.splits;
    const int at = (int)(r - tile * C::kRows);
    float top = -INFINITY;
    for (int i = 0; i < plan.splits; ++i) top = fmaxf(top, parts[i].lse2[at]);
    const float base = top == -INFINITY ? 0.f : top;
    float l = 0.f, o[D / 32];
#pragma unroll
    for (int e = 0; e < D / 32; ++e) o[e] = 0.f;
    for (int i = 0; i < plan.splits; ++i) {
        const float f = ex2(parts[i].lse2[at] - base);
        l += f;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) o[e] = fmaf(parts[i].o[at][e * 32 + lane], f, o[e]);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) ((T *)a.o)[row * D + e * 32 + lane] = from_f32<T>(o[e] * inv);
    if (lane == 0 && a.lse) a.lse[row] = (l == 0.f ? -INFINITY : log2f(l) + base) * kLn2;
}

// Row tiles of a grid and the splits of their keys. With fewer items than SMs, or a last round of blocks
// that is far from full, an item's keys are split so that the rounds (152 blocks of one per SM, each
// with about three tiles' time to begin and end) take least.
template <int D, int kParts> TcPlan tc_plan(const Attn &a, bool packed) {
    using C = TcConfig<D, kParts>;
    const int64_t rows = a.max_q * a.group;
    const int64_t tiles = packed ? a.tokens * a.group / C::kRows + a.num_seqs : a.num_seqs * ((rows + C::kRows - 1) / C::kRows);
    TcPlan p = {nullptr, nullptr, tiles, 1};
    const int64_t items = tiles * a.kv_heads, keys = ((a.width << a.log_page) + C::kKeys - 1) / C::kKeys;
    double best = 1e300;
    for (int s = 1; s <= 64 && (s == 1 || (items * s <= 8 * 152 && keys >= 4 * s)); ++s) {
        const double cost = (double)((items * s + 151) / 152) * ((double)((keys + s - 1) / s) + 3 + (s > 1 ? 1 : 0));
        if (cost < best * 0.97) {
            best = cost;
            p.splits = s;
        }
    }
    return p;
}
inline int64_t tc_blocks(const Attn &a, const TcPlan &p) {
    const int64_t items = p.tiles * a.kv_heads * p.splits;
    return items < 152 ? items : 152;
}
template <int D, int kParts> size_t tc_parts_bytes(const Attn &a, const TcPlan &p) {
    return p.splits == 1 ? 0 : (size_t)p.tiles * a.kv_heads * p.splits * sizeof(Part<TcConfig<D, kParts>::kRows, D>);
}
template <int D, int kParts> bool tc_long(const Attn &a, const TcPlan &p) {
    const int64_t keys = ((a.width << a.log_page) + TcConfig<D, kParts>::kKeys - 1) / TcConfig<D, kParts>::kKeys;
    return kParts == 1 && (keys + p.splits - 1) / p.splits > kMost;
}
template <int D, int kParts> size_t tc_pieces_bytes(const Attn &a, const TcPlan &p) {
    return tc_long<D, kParts>(a, p) ? (size_t)tc_blocks(a, p) * TcConfig<D, kParts>::kRows * sizeof(TcPiece<D>) : 0;
}
template <int D, int kParts> size_t tc_bytes_for(const Attn &a, bool packed) {
    const TcPlan p = tc_plan<D, kParts>(a, packed);
    return tc_parts_bytes<D, kParts>(a, p) + tc_pieces_bytes<D, kParts>(a, p);
}
template <int D> size_t tc_bytes_d(const Attn &a, int dtype) {
    Attn b = a;
    size_t most = dtype == GDR_F32 ? tc_bytes_for<D, 2>(b, true) : tc_bytes_for<D, 1>(b, true);
    if (a.tokens % a.num_seqs == 0) {  // (equal lengths without offsets)
        b.max_q = a.tokens / a.num_seqs;
        const size_t equal = dtype == GDR_F32 ? tc_bytes_for<D, 2>(b, false) : tc_bytes_for<D, 1>(b, false);
        if (equal > most) most = equal;
    }
    return most;
}

template <typename K> int registers_of(K kernel) {
    cudaFuncAttributes attr;
    if (cudaFuncGetAttributes(&attr, kernel) == cudaSuccess) return attr.numRegs;
    (void)cudaGetLastError();
    return -1;
}

template <typename T, int D, int kParts, int kMode, int kCode, bool kLong> int launch_tc_kernel(const Attn &a, const TcPlan &plan, cudaStream_t s) {
    using C = TcConfig<D, kParts>;
    const auto kernel = attn_tc_kernel<T, D, kParts, kMode, kCode, kLong>;
    // The roles' shares of registers add up to what the block is launched with, if the compiler gave it that many: the
    // build refuses another number, and so does the call (asked until there is an answer, 2 us a call).
    static std::atomic<int> registers{-1};
    int has = registers.load(std::memory_order_relaxed);
    if (has < 0) registers.store(has = registers_of(kernel), std::memory_order_relaxed);
    if (has != kTcRegs) return GDR_ERR_CUDA;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess) return GDR_ERR_CUDA;
    CUtensorMap maps[2];
    if (!map_cache(&maps[0], a.kc, a, D, C::kKeys, D >= 128) || !map_cache(&maps[1], a.vc, a, D, C::kKeys, D >= 128)) return GDR_ERR_CUDA;
    kernel<<<(unsigned)tc_blocks(a, plan), kTcThreads, C::kSmem, s>>>(a, plan, maps[0], maps[1]);
    if (cudaGetLastError() != cudaSuccess) return GDR_ERR_CUDA;
    if (plan.splits > 1)
        join_splits_kernel<T, D, kParts><<<(unsigned)((a.tokens * a.heads + 7) / 8), 256, 0, s>>>(a, plan);
    return cuda_status(cudaGetLastError());
}

template <typename T, int D, int kParts, int kMode, bool kLong> int launch_tc_code(const Attn &a, const TcPlan &plan, int code, cudaStream_t s) {
    return code == GDR_CODE_E4M3 ? launch_tc_kernel<T, D, kParts, kMode, GDR_CODE_E4M3, kLong>(a, plan, s)
                                 : launch_tc_kernel<T, D, kParts, kMode, GDR_CODE_INT8, kLong>(a, plan, s);
}
template <typename T, int D, int kParts, bool kLong> int launch_tc_mode(const Attn &a, const TcPlan &plan, int mode, int code, cudaStream_t s) {
    return mode == kPlain    ? launch_tc_code<T, D, kParts, kPlain, kLong>(a, plan, code, s)
           : mode == kCapped ? launch_tc_code<T, D, kParts, kCapped, kLong>(a, plan, code, s)
                             : launch_tc_code<T, D, kParts, kBiased, kLong>(a, plan, code, s);
}
template <int D, int kParts> TcPlan tc_plan_in(const Attn &a, void *ws) {
    TcPlan plan = tc_plan<D, kParts>(a, a.cu != nullptr);
    plan.parts = (char *)ws;
    plan.pieces = (char *)ws + tc_parts_bytes<D, kParts>(a, plan);
    return plan;
}

template <int D> int launch_tc_d(const Attn &a, int code, int dtype, void *ws, cudaStream_t s) {
    const int mode = a.slopes || (dtype == GDR_BF16 && a.softcap > kCaps) ? kBiased : a.softcap > 0.f ? kCapped : kPlain;
    if (dtype == GDR_F32) return launch_tc_mode<float, D, 2, false>(a, tc_plan_in<D, 2>(a, ws), mode, code, s);
    const TcPlan plan = tc_plan_in<D, 1>(a, ws);
    return tc_long<D, 1>(a, plan) ? launch_tc_mode<__nv_bfloat16, D, 1, true>(a, plan, mode, code, s)
                                  : launch_tc_mode<__nv_bfloat16, D, 1, false>(a, plan, mode, code, s);
}

}  // namespace cattn
}  // namespace gdr
