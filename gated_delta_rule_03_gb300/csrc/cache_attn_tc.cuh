// cache_attn_tc.cuh -- attention over a paged 8-bit cache for many rows: prompts and pieces of them.
//
// Rows. As in cache_attn_step.cuh the rows of an item are the queries that share a head of the
// cache, token by token; a block takes 128 kTiles of them and goes through the keys that the last of them
// sees, kKeys at a time.
//
// Products on the 5th-generation tensor cores in fp16 with fp32 sums in TMEM: scores = Q K^T from shared
// memory, outputs += W codes with the weights W read from TMEM, where they take their scores' place.
// Converter warps turn codes into fp16 tiles in the 128-byte-swizzled layout: a tile's row is a token,
// which is K-major for the first product and MN-major for the second, so that both are written alike.
// Loads of codes go to registers a tile ahead, as they have to pass through them.
//
// Roles (416 threads): kTiles groups of 128 threads for the softmax, a row to a thread; the rest of
// 384 convert; one thread of the last warp issues the products. With two row tiles one's softmax runs
// under the other's products; with one (wide heads, fp32) the scores have two buffers and the next
// tile's product runs under the softmax.
//
// fp32: queries and weights as two fp16 parts, hi + lo, whose products are added in the same TMEM sums.
#pragma once

#include <type_traits>

#include "cache_attn.cuh"
#include "f32x2.cuh"
#include "sm100.cuh"

namespace gdr {
namespace cattn {

using namespace sm100;

constexpr int kTcThreads = 416;
constexpr int kRing = 4;   // tiles of scales
constexpr int kFlush = 4;  // tiles whose outputs are added up in TMEM (fp32)

template <int D, int kParts> struct TcConfig {
    static constexpr int kTiles = kParts == 1 && D <= 128 ? 2 : 1;
    static constexpr int kKeys = kParts == 2 ? 64 : 128;
    static constexpr int kRows = 128 * kTiles;
    static constexpr int kSoft = 128 * kTiles;         // threads
    static constexpr int kConv = 384 - kSoft;
    static constexpr int kQ = 128 * D * 2;             // bytes of a part of a row tile
    static constexpr int kKv = kKeys * D * 2;          // of a tile of keys or values
    static constexpr int kStages = D == 256 ? 1 : 2;
    static constexpr int kSmem = kTiles * kParts * kQ + 2 * kStages * kKv + 1024;
    // TMEM columns: scores of two slots (weights in their place), outputs, low parts of weights
    static constexpr uint32_t kS = kKeys, kO = 256;
    static constexpr uint32_t kLow = 128, kLowStep = kKeys / 2;
    static_assert(kSmem <= 232448 - 1024, "shared memory");
    static_assert(kO + kTiles * D <= 512 && 2 * kKeys + (kParts == 2 ? 2 * kLowStep : 0) <= kO, "TMEM");
};

struct TcPlan {
    char *parts;   // fp32 outputs and sums of the splits: [item][split] TcPart
    int tiles;     // row tiles that the grid has per head of the cache
    int splits;    // of each item's keys
};
template <int kRows, int D> struct TcPart {
    float lse2[kRows];
    float o[kRows][D];
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

// Where a block's rows are: request n, its rows from row0 on.
struct TcItem {
    int n, row0, first, len, nq;  // first: the request's first token; nq: its new tokens
};

// Finds tile `x` (the last ones first: they see the most keys). Every thread of the block; false if there
// is no such tile, *ok whether the lengths hold.
template <int kRows> __device__ inline bool find_tile(const Attn &a, int64_t x, int64_t *sums, TcItem *found, bool *ok) {
    const int tid = threadIdx.x;
    auto tiles = [&](int64_t n) { return ((int64_t)rows_of(a, n).y * a.group + kRows - 1) / kRows; };
    bool good = true;
    int64_t mine = 0;
    for (int64_t n = tid; n < a.num_seqs; n += kTcThreads) {
        if (lengths_hold(a, n)) mine += tiles(n);
        else good = false;
    }
    *ok = __syncthreads_and(good);
    if (!*ok) return false;
    if (!a.cu) {  // equal lengths: the last tiles of all requests first
        const int64_t each = tiles(0);
        if (x >= each * a.num_seqs) return false;
        if (tid == 0) {
            found->n = (int)(x % a.num_seqs);
            found->row0 = (int)((each - 1 - x / a.num_seqs) * kRows);
        }
    } else {
        int64_t total;
        block_sums<kTcThreads>(mine, sums, &total);
        if (x >= total) return false;
        const int64_t want = total - 1 - x;
        int64_t carry = 0;
        for (int64_t n0 = 0; n0 < a.num_seqs; n0 += kTcThreads) {
            const int64_t n = n0 + tid, w = n < a.num_seqs ? tiles(n) : 0;
            int64_t all;
            const int64_t end = carry + block_sums<kTcThreads>(w, sums, &all);
            if (want >= end - w && want < end) {
                found->n = (int)n;
                found->row0 = (int)((want - (end - w)) * kRows);
            }
            carry += all;
            if (carry > want) break;
        }
    }
    __syncthreads();
    if (tid == 0) {
        const int2 r = rows_of(a, found->n);
        found->first = r.x;
        found->nq = r.y;
        found->len = __ldg(a.kv_lens + found->n);
    }
    __syncthreads();
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

// What becomes of scores: nothing more, a cap, or a bias by distance with or without a cap.
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
    static __device__ __forceinline__ float rcp(float x) {
        float y;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
        return y;
    }
    __device__ __forceinline__ float one(float z, int e) const {
        z *= m;
        if (cap > 0.f) z = cap * (kExact ? tanhf(z * k) : fmaf(-2.f, rcp(1.f + ex2(z * k * (2.f * kLog2e))), 1.f));
        if (kMode == kBiased) z = fmaf(-slope, fabsf(away - (float)e), z);
        return fmaf(z, kLog2e, off);
    }
    __device__ __forceinline__ float2 operator()(float2 z, int e) const {
        if (kMode == kPlain) return fma2(z, make_float2(m, m), make_float2(off, off));
        if (kMode == kCapped && !kExact) {
            float2 x = mul2(z, make_float2(m, m));
            x = add2(make_float2(ex2(x.x), ex2(x.y)), make_float2(1.f, 1.f));
            return fma2(make_float2(rcp(x.x), rcp(x.y)), make_float2(k, k), make_float2(off, off));
        }
        return make_float2(one(z.x, e), one(z.y, e + 1));
    }
};

__device__ __forceinline__ uint32_t f16_pair(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 f16_values(uint32_t r) { return __half22float2(reinterpret_cast<const __half2 &>(r)); }
// Issued where it stands: a load that the compiler may move ends up next to its use.
__device__ __forceinline__ uint4 ld_nc(const void *p) {
    uint4 v;
    asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ void store16(uint32_t saddr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(saddr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

template <typename T, int D, int kParts, int kMode>
__global__ void __launch_bounds__(kTcThreads, 1) attn_tc_kernel(const __grid_constant__ Attn a, const TcPlan plan, const int code) {
    using C = TcConfig<D, kParts>;
    extern __shared__ unsigned char sm[];
    const uint32_t base = (smem_u32(sm) + 1023u) & ~1023u;
    const uint32_t sq = base, sk = base + C::kTiles * kParts * C::kQ, sv = sk + C::kStages * C::kKv;
    __shared__ int64_t sums[kTcThreads / 32];
    __shared__ TcItem item;
    __shared__ float4 scales[kRing][8];  // of 16 keys: score factor, log2 and reciprocal of the value scale
    __shared__ uint32_t tmem_slot;
    __shared__ int gave_up;
    enum { K_FULL = 0, K_FREE = 2, V_FULL = 4, V_FREE = 6, S_FULL = 8, W_FULL = 10, O_DONE = 12, O_LAST = 14, BARS = 15 };
    __shared__ __align__(8) uint64_t bars[BARS];
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    bool ok;
    const int split = blockIdx.z, head = blockIdx.y;
    const bool mine = find_tile<C::kRows>(a, blockIdx.x, sums, &item, &ok);
    if (tid == 0 && blockIdx.x == 0 && head == 0 && split == 0) *a.status = ok ? GDR_OK : GDR_ERR_BAD_SEQLENS;
    if (!mine) return;

    const int n = item.n, row0 = item.row0, len = item.len, past = len - item.nq;
    const int nrows = min(C::kRows, (int)min((int64_t)item.nq * a.group - row0, (int64_t)C::kRows));
    // keys that the last row sees, and this split's tiles of them
    const int far = a.causal ? max(0, min(len, past + (row0 + nrows - 1) / a.group + 1)) : len;
    const int all_tiles = (far + C::kKeys - 1) / C::kKeys;
    const int each = (all_tiles + plan.splits - 1) / plan.splits;
    const int j0 = min(all_tiles, split * each), j1 = min(all_tiles, j0 + each), count = j1 - j0;

    if (tid == 0) {
        gave_up = 0;
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(K_FULL + s), C::kConv);
            mbar_init(bar(V_FULL + s), C::kConv);
            mbar_init(bar(K_FREE + s), 1);
            mbar_init(bar(V_FREE + s), 1);
            mbar_init(bar(S_FULL + s), 1);
            mbar_init(bar(W_FULL + s), 128);
            mbar_init(bar(O_DONE + s), 1);
        }
        mbar_init(bar(O_LAST), 1);
        fence_mbar_init();
    }
    if (warp == 12) {
        tmem_alloc(smem_u32(&tmem_slot), 512);
        tmem_relinquish();
    }
    float row_up = 1.f;
    if (warp < C::kSoft / 32) {
        // ---- queries: this thread's row in fp16 with a power of two, its sign that of the scale
        const int r = tid, at = row0 + r;
        const uint32_t to = sq + (r >> 7) * kParts * C::kQ;
        const bool live = r < nrows;
        const T *src = live ? (const T *)a.q + (int64_t)(item.first + at / a.group) * a.qs + (int64_t)(head * a.group + at % a.group) * D : nullptr;
        // 256 bytes of the row at a time in registers, all of them under way together; longer rows come twice
        constexpr int kPiece = 256 / sizeof(T), kPieces = (D + kPiece - 1) / kPiece, kVecs = (D < kPiece ? D : kPiece) * sizeof(T) / 16;
        constexpr int kVec = 16 / sizeof(T);
        uint4 w[kVecs];
        auto fetch = [&](int piece) {
#pragma unroll
            for (int i = 0; i < kVecs; ++i) w[i] = live ? ld_nc(src + piece * kPiece + i * kVec) : make_uint4(0, 0, 0, 0);
        };
        uint32_t most = 0;
#pragma unroll 1
        for (int piece = kPieces - 1; piece >= 0; --piece) {
            fetch(piece);
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const T *e = (const T *)&w[i];
#pragma unroll
                for (int x = 0; x < kVec; ++x) most = max(most, __float_as_uint(to_f32<T>(e[x])) & 0x7fffffffu);
            }
        }
        const int shift = row_shift(most);
        const float up = a.scale < 0.f ? -two_to(shift) : two_to(shift);
        row_up = two_to(-shift) * fabsf(a.scale);
#pragma unroll 1
        for (int piece = 0; piece < kPieces; ++piece) {
            if (piece > 0) fetch(piece);
#pragma unroll
            for (int c = 0; c < kVecs * kVec; c += 8) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int e = c + 2 * i;
                    const float x = to_f32<T>(((const T *)&w[e / kVec])[e % kVec]) * up, y = to_f32<T>(((const T *)&w[(e + 1) / kVec])[(e + 1) % kVec]) * up;
                    hi[i] = f16_pair(x, y);
                    const float2 f = f16_values(hi[i]);
                    lo[i] = f16_pair(x - f.x, y - f.y);
                }
                const int d = piece * kPiece + c;
                const uint32_t dst = to + (d >> 6) * 16384 + sw128_offset(r & 127, d & 63);
                store16(dst, hi[0], hi[1], hi[2], hi[3]);
                if (kParts == 2) store16(dst + C::kQ, lo[0], lo[1], lo[2], lo[3]);
            }
        }
        fence_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    bool fine = true;

    if (warp < C::kSoft / 32) {
        // ---------------------------------------------------------------- softmax
        const int tile = warp >> 2;  // row tile
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const int at = row0 + tid;
        const int p = past + at / a.group, lim = a.causal ? min(len, p + 1) : len;
        const int sure = a.causal ? min(len, past + (row0 + tile * 128) / a.group + 1) : len;
        const uint32_t out = tmem + lanes + C::kO + tile * D;
        const bool live = tid < nrows;
        const int64_t row = (int64_t)(item.first + at / a.group) * a.heads + head * a.group + at % a.group;
        TcPart<C::kRows, D> *const part = (TcPart<C::kRows, D> *)plan.parts + (((int64_t)head * plan.tiles + blockIdx.x) * plan.splits + split);
        float *const row_out = plan.splits > 1 ? part->o[tid] : (float *)a.o + row * D;  // (fp32 only without splits)
        const float slope = kMode == kBiased && a.slopes && live ? __ldg(a.slopes + head * a.group + at % a.group) : 0.f;
        const float cap = kMode == kPlain ? 0.f : a.softcap, inv_cap = cap > 0.f ? 1.f / cap : 0.f;
        const float up2 = row_up * (kMode == kPlain ? kLog2e : 1.f);
        float ref = 0.f, l = 0.f;
        float sum_ref = 0.f, sum_l = 0.f;  // kParts == 2: of what has left TMEM

        // The tensor cores cut the sums in TMEM instead of rounding them, some 2^-24 of them per step and always
        // towards zero: fp32 results take the outputs of kFlush tiles at a time out and add them up in memory.
        auto flush = [&] {
            const bool some = sum_l != 0.f;
            const float by = some ? ex2(sum_ref - ref) : 0.f;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                float v[32];
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

        for (int i = 0; i < count && fine; ++i) {
            const int slot = C::kTiles == 2 ? tile : i & 1, use = C::kTiles == 2 ? i : i >> 1;
            const uint32_t s_at = tmem + lanes + slot * C::kS;
            if (!mbar_wait(bar(S_FULL + slot), use & 1)) {
                fine = false;
                break;
            }
            // The outputs of the tiles before. With two row tiles the scores' barrier says that they are there; with
            // one it does so of the last but one tile, and the last has a barrier that even and odd tiles share in turn.
            auto outputs_done = [&] {
                if (C::kTiles == 1 && !mbar_wait(bar(O_DONE + ((i - 1) & 1)), ((i - 1) >> 1) & 1)) fine = false;
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
            const float4 *const sc = scales[(j0 + i) % kRing];
            const bool edge = tok + C::kKeys > sure;

            // Weights with the row's reference as it is, 16 keys at a time, and the largest exponent. The first tile
            // (a row that sees none of its keys sees no later ones), or an exponent that is too large, moves the
            // reference, and the outputs so far with it; then the weights are taken again.
            uint32_t hi[C::kKeys / 2], lo[kParts == 2 ? C::kKeys / 2 : 1];
            float sum = 0.f, top = -INFINITY;
            auto weigh = [&](auto at_edge) {
                constexpr bool kEdge = decltype(at_edge)::value;
                float2 all = make_float2(0.f, 0.f);
                top = -INFINITY;
                uint32_t x[2][16];
                tmem_fetch16(s_at, x[0]);
#pragma unroll
                for (int g = 0; g < C::kKeys / 16; ++g) {
                    uint32_t(&y)[16] = x[g & 1];
                    tmem_arrive16(y);
                    if (g + 1 < C::kKeys / 16) tmem_fetch16(s_at + 16 * (g + 1), x[(g + 1) & 1]);
                    const float4 f = sc[g];
                    const Shape<kMode, kParts == 2> shape(f.x * up2, f.y - ref, cap, inv_cap, slope, (float)(p - tok - 16 * g));
                    float2 some = make_float2(0.f, 0.f);
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        float2 w = shape(make_float2(__uint_as_float(y[e]), __uint_as_float(y[e + 1])), e);
                        if (kEdge) {
                            const int j = tok + 16 * g + e;
                            if (j >= lim) w.x = -INFINITY;
                            if (j + 1 >= lim) w.y = -INFINITY;
                        }
                        top = fmaxf(top, fmaxf(w.x, w.y));
                        w.x = ex2(w.x);
                        w.y = ex2(w.y);
                        some = add2(some, w);
                        const int q = 8 * g + e / 2;
                        hi[q] = f16_pair(w.x, w.y);
                        if (kParts == 2) {
                            const float2 v = f16_values(hi[q]);
                            lo[q] = f16_pair(w.x - v.x, w.y - v.y);
                        }
                    }
                    all = fma2(some, make_float2(f.z, f.z), all);
                }
                sum = all.x + all.y;
            };
            for (bool settled = false;; settled = true) {
                if (edge) weigh(std::true_type{});
                else weigh(std::false_type{});
                if (settled || (i > 0 && !__any_sync(~0u, top > kSpan + kSlack))) break;
                const bool move = i == 0 ? top > -INFINITY : top > kSpan + kSlack;
                if (move) ref += top - kSpan;
                if (i > 0) {
                    const float by = move ? ex2(kSpan - top) : 1.f;
                    l *= by;
                    if (!anew) {
                        outputs_done();
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            float v[32];
                            tmem_load32(out + c, v);
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] *= by;
                            tmem_store32(out + c, v);
                        }
                    }
                }
            }
            l += sum;
#pragma unroll
            for (int c = 0; c < C::kKeys / 2; c += 16) {
                tmem_put16(s_at + c, hi + c);
                if constexpr (kParts == 2) tmem_put16(tmem + lanes + C::kLow + slot * C::kLowStep + c, lo + c);
            }
            tmem_stored();
            tc_fence_before();
            mbar_arrive(bar(W_FULL + slot));
        }
        // ---- results
        if (count > 0 && fine) {
            fine = mbar_wait(bar(O_LAST), 0);
            __syncwarp();
            tc_fence_after();
        }
        // (a warp reads its lanes together, whichever rows are live)
        if (__all_sync(~0u, fine)) {
            const float by = kParts == 2 ? ex2(sum_ref - ref) : 0.f;
            const bool older = kParts == 2 && sum_l != 0.f;
            if (older) l = fmaf(sum_l, by, l);
            const bool some = l != 0.f;
            const float inv = some ? 1.f / l : 0.f;
            if (live) {
                const float sum2 = some ? log2f(l) + ref : -INFINITY;
                if (plan.splits > 1) part->lse2[tid] = sum2;
                else if (a.lse) a.lse[row] = sum2 * kLn2;
            }
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                float v[32];
                if (count > 0) {
                    tmem_load32(out + c, v);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = 0.f;
                }
                if (!live) continue;
                if (older) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const float4 o = *(const float4 *)(row_out + c + e);
                        v[e] = fmaf(o.x, by, v[e]);
                        v[e + 1] = fmaf(o.y, by, v[e + 1]);
                        v[e + 2] = fmaf(o.z, by, v[e + 2]);
                        v[e + 3] = fmaf(o.w, by, v[e + 3]);
                    }
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = some ? v[e] * inv : 0.f;
                if (plan.splits > 1 || sizeof(T) == 4) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4) *(float4 *)(row_out + c + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                } else {
                    __nv_bfloat16 *const to = (__nv_bfloat16 *)a.o + row * D + c;
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        uint32_t w[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const __nv_bfloat162 b = __floats2bfloat162_rn(v[e + 2 * x], v[e + 2 * x + 1]);
                            w[x] = reinterpret_cast<const uint32_t &>(b);
                        }
                        *(uint4 *)(to + e) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
        }
    } else if (warp < 12) {
        // ---------------------------------------------------------------- codes to fp16
        const int ct = tid - C::kSoft, cw = ct >> 5;
        constexpr int kBlocks = D / 64;                     // 64 dims to a swizzled block of rows
        constexpr int kWarpRows = 8 / kBlocks;              // rows of a warp's pass of 512 bytes
        constexpr int kPass = kWarpRows * (C::kConv / 32);  // rows of a pass
        constexpr int kPasses = C::kKeys / kPass;
        // Eight lanes in turn write 16-byte chunks 2x of two rows, one even and one odd: no two in the same banks.
        const int x = lane & 3, blk = (lane >> 3) & (kBlocks - 1), row_lo = (lane >> 2) & 1;
        const int row = cw * kWarpRows + row_lo + 2 * (lane >> (3 + (kBlocks == 4 ? 2 : kBlocks == 2 ? 1 : 0)));
        const int in_page = (1 << a.log_page) - 1, lane_off = (row & 15) * D + blk * 64 + x * 16;
        // Lane g < 8 knows 16 keys of a tile: their page (-1 behind the last token, -2 outside the cache), and
        // where their codes begin.
        struct Keys {
            int page;
            int64_t at;
        };
        auto keys_of = [&](int i) {
            const int tok = (j0 + i) * C::kKeys + (lane & 7) * 16;
            if (i >= count || (lane & 7) * 16 >= C::kKeys || tok >= len) return Keys{-1, 0};
            int pg = __ldg(a.table + (int64_t)n * a.width + (tok >> a.log_page));
            if (pg < 0 || pg >= a.pages) pg = -2;
            return Keys{pg, (((int64_t)pg * a.kv_heads + head) * (in_page + 1) + (tok & in_page)) * D};
        };
        auto load = [&](const uint8_t *cache, int i, const Keys &keys, uint4 (&v)[kPasses]) {
            const bool full = (j0 + i + 1) * C::kKeys <= len && __all_sync(~0u, keys.page >= 0 || (lane & 7) * 16 >= C::kKeys);
#pragma unroll
            for (int ps = 0; ps < kPasses; ++ps) {
                const int g = (ps * kPass + cw * kWarpRows) >> 4;  // (a warp's rows of a pass lie in one of the 16s)
                const uint8_t *const from = cache + (__shfl_sync(~0u, keys.at, g) + lane_off);
                if (full) {
                    v[ps] = ld_nc(from);
                } else {
                    const int pg = __shfl_sync(~0u, keys.page, g);
                    v[ps] = make_uint4(0, 0, 0, 0);
                    if (pg >= 0 && (j0 + i) * C::kKeys + ps * kPass + row < len) v[ps] = ld_nc(from);
                }
            }
        };
        auto put = [&](uint32_t to, const uint4 (&v)[kPasses]) {
#pragma unroll
            for (int ps = 0; ps < kPasses; ++ps) {
                const int r = ps * kPass + row;
                const uint32_t w[4] = {v[ps].x, v[ps].y, v[ps].z, v[ps].w};
                uint32_t h[8];
                if (code == GDR_CODE_E4M3) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) codes::to_f16x4<GDR_CODE_E4M3>(w[e], h[2 * e], h[2 * e + 1]);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) codes::to_f16x4<GDR_CODE_INT8>(w[e], h[2 * e], h[2 * e + 1]);
                }
                const uint32_t at = to + blk * (C::kKeys * 128) + r * 128;
                store16(at + (((2 * x) ^ (r & 7)) << 4), h[0], h[1], h[2], h[3]);
                store16(at + (((2 * x + 1) ^ (r & 7)) << 4), h[4], h[5], h[6], h[7]);
            }
            fence_async_smem();
        };
        Keys keys = keys_of(0), next = keys_of(1);
        uint4 k[kPasses], v[kPasses];
        load(a.kc, 0, keys, k);
        for (int i = 0; i < count; ++i) {
            const int st = i % C::kStages, turn = (i / C::kStages) & 1;
            load(a.vc, i, keys, v);
            if (cw == 0 && lane < C::kKeys / 16) {
                float4 f = make_float4(0.f, 0.f, 1.f, 0.f);  // (behind the last token: masked)
                if (keys.page != -1) {
                    const float bad = __int_as_float(0x7fffffff);
                    const float ks = keys.page < 0 ? bad : __ldg(a.ks + (int64_t)keys.page * a.kv_heads + head);
                    const float vs = keys.page < 0 ? bad : __ldg(a.vs + (int64_t)keys.page * a.kv_heads + head);
                    f = make_float4(ks, lg2(vs), vs == vs ? __fdividef(1.f, vs) : 1.f, 0.f);
                }
                scales[(j0 + i) % kRing][lane] = f;
            }
            if (!mbar_wait(bar(K_FREE + st), turn ^ 1)) {
                fine = false;
                break;
            }
            put(sk + st * C::kKv, k);
            mbar_arrive(bar(K_FULL + st));
            keys = next;
            next = keys_of(i + 2);
            load(a.kc, i + 1, keys, k);
            if (!mbar_wait(bar(V_FREE + st), turn ^ 1)) {
                fine = false;
                break;
            }
            put(sv + st * C::kKv, v);
            mbar_arrive(bar(V_FULL + st));
        }
    } else if (lane == 0) {
        // ---------------------------------------------------------------- products
        const uint32_t id_s = idesc_f16(128, C::kKeys, 0), id_o = idesc_f16(128, D, 1);
        // (the low parts first: a sum is cut while it is small)
        auto scores = [&](int i, int tile, int slot) {
            const uint32_t kt = desc_k(sk + (i % C::kStages) * C::kKv), qt = desc_k(sq + tile * kParts * C::kQ);
#pragma unroll
            for (int x = kParts - 1; x >= 0; --x)
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_ss(tmem + slot * C::kS, qt + ((x * C::kQ + (kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                           kt + (((kk >> 2) * (C::kKeys * 128) + (kk & 3) * 32) >> 4), id_s, x < kParts - 1 || kk > 0);
            mma_commit(bar(S_FULL + slot));
        };
        auto outputs = [&](int i, int tile, int slot) {
            const uint32_t vt = desc_mn(sv + (i % C::kStages) * C::kKv, C::kKeys * 128);
            const bool add = (kParts == 2 ? i % kFlush : i) > 0;
#pragma unroll
            for (int x = kParts - 1; x >= 0; --x)
#pragma unroll
                for (int kk = 0; kk < C::kKeys / 16; ++kk)
                    mma_ts(tmem + C::kO + tile * D, (x == 0 ? tmem + slot * C::kS : tmem + C::kLow + slot * C::kLowStep) + 8 * kk,
                           vt + ((kk * 2048) >> 4), id_o, add || x < kParts - 1 || kk > 0);
        };
        auto turn = [&](int i) { return (uint32_t)(i / C::kStages) & 1u; };
        auto wait = [&](int b, uint32_t parity) {
            if (fine) fine = mbar_wait(bar(b), parity);
            tc_fence_after();
            return fine;
        };
        if (C::kTiles == 2) {
            if (count > 0 && wait(K_FULL, 0)) {
                scores(0, 0, 0);
                scores(0, 1, 1);
                mma_commit(bar(K_FREE));
            }
            for (int i = 0; i < count && fine; ++i) {
                const int st = i % C::kStages, st1 = (i + 1) % C::kStages;
                if (!wait(V_FULL + st, turn(i))) break;
#pragma unroll 1
                for (int tile = 0; tile < 2; ++tile) {
                    if (!wait(W_FULL + tile, i & 1)) break;
                    outputs(i, tile, tile);
                    if (tile == 1) mma_commit(bar(V_FREE + st));
                    if (i + 1 < count) {
                        if (tile == 0 && !wait(K_FULL + st1, turn(i + 1))) break;
                        scores(i + 1, tile, tile);
                        if (tile == 1) mma_commit(bar(K_FREE + st1));
                    }
                }
            }
        } else {
            if (count > 0 && wait(K_FULL, 0)) {
                scores(0, 0, 0);
                mma_commit(bar(K_FREE));
            }
            for (int i = 0; i < count && fine; ++i) {
                const int st = i % C::kStages, st1 = (i + 1) % C::kStages;
                if (i + 1 < count) {
                    if (!wait(K_FULL + st1, turn(i + 1))) break;
                    scores(i + 1, 0, (i + 1) & 1);
                    mma_commit(bar(K_FREE + st1));
                }
                if (!wait(V_FULL + st, turn(i)) || !wait(W_FULL + (i & 1), (i >> 1) & 1)) break;
                outputs(i, 0, i & 1);
                mma_commit(bar(V_FREE + st));
                mma_commit(bar(O_DONE + (i & 1)));
            }
        }
        // (also after a wait that ran out: what was issued ends before the TMEM goes)
        if (count > 0) {
            mma_commit(bar(O_LAST));
            if (!fine) mbar_wait(bar(O_LAST), 0);
        }
    }
    if (!fine) gave_up = 1;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 12) tmem_dealloc(tmem, 512);
    if (tid == 0 && gave_up) *a.status = GDR_ERR_DEVICE_TIMEOUT;
}

// Adds the splits of an item in order: a warp to a row.
template <typename T, int D, int kParts> __global__ void __launch_bounds__(256) join_splits_kernel(const __grid_constant__ Attn a, const TcPlan plan) {
    using C = TcConfig<D, kParts>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (*(volatile int32_t *)a.status == GDR_ERR_BAD_SEQLENS) return;
    // a row of q and its head: the block of the item that it belongs to
    const int64_t row = (int64_t)blockIdx.x * 8 + warp;
    const int64_t t = row / a.heads;
    if (t >= a.tokens) return;
    const int h = (int)(row - t * a.heads), head = h / a.group;
    int64_t n, first, tiles_before = 0, total = 0;
    if (!a.cu) {
        n = t / a.max_q;
        first = n * a.max_q;
    } else {
        if (t >= __ldg(a.cu + a.num_seqs)) return;
        int64_t lo = 0, hi = a.num_seqs - 1;  // the last request that begins at t or before and has t
        while (lo < hi) {
            const int64_t mid = (lo + hi) / 2;
            if (__ldg(a.cu + mid + 1) > t) hi = mid;
            else lo = mid + 1;
        }
        n = lo;
        first = __ldg(a.cu + n);
        for (int64_t m = lane; m < a.num_seqs; m += 32) {
            const int64_t k = ((int64_t)rows_of(a, m).y * a.group + C::kRows - 1) / C::kRows;
            total += k;
            if (m < n) tiles_before += k;
        }
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            total += __shfl_xor_sync(~0u, total, d);
            tiles_before += __shfl_xor_sync(~0u, tiles_before, d);
        }
    }
    const int64_t r = (t - first) * a.group + h % a.group, tile = r / C::kRows;
    int64_t x;
    if (!a.cu) {
        const int64_t each = (a.max_q * a.group + C::kRows - 1) / C::kRows;
        x = (each - 1 - tile) * a.num_seqs + n;
    } else {
        x = total - 1 - (tiles_before + tile);
    }
    const TcPart<C::kRows, D> *const parts = (const TcPart<C::kRows, D> *)plan.parts + ((int64_t)head * plan.tiles + x) * plan.splits;
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
    int64_t tiles = a.num_seqs * ((rows + C::kRows - 1) / C::kRows);
    if (packed) {
        const int64_t most = a.tokens * a.group / C::kRows + a.num_seqs;
        if (most < tiles) tiles = most;
    }
    TcPlan p = {nullptr, (int)tiles, 1};
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
template <int D, int kParts> size_t tc_bytes_for(const Attn &a, bool packed) {
    const TcPlan p = tc_plan<D, kParts>(a, packed);
    return p.splits == 1 ? 0 : (size_t)p.tiles * a.kv_heads * p.splits * sizeof(TcPart<TcConfig<D, kParts>::kRows, D>);
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

template <typename T, int D, int kParts, int kMode> int launch_tc_kernel(const Attn &a, int code, void *ws, cudaStream_t s) {
    using C = TcConfig<D, kParts>;
    TcPlan plan = tc_plan<D, kParts>(a, a.cu != nullptr);
    plan.parts = (char *)ws;
    const auto kernel = attn_tc_kernel<T, D, kParts, kMode>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess) return GDR_ERR_CUDA;
    kernel<<<dim3((unsigned)plan.tiles, (unsigned)a.kv_heads, (unsigned)plan.splits), kTcThreads, C::kSmem, s>>>(a, plan, code);
    if (cudaGetLastError() != cudaSuccess) return GDR_ERR_CUDA;
    if (plan.splits > 1)
        join_splits_kernel<T, D, kParts><<<(unsigned)((a.tokens * a.heads + 7) / 8), 256, 0, s>>>(a, plan);
    return cuda_status(cudaGetLastError());
}

template <int D> int launch_tc_d(const Attn &a, int code, int dtype, void *ws, cudaStream_t s) {
    const int mode = a.slopes ? kBiased : a.softcap > 0.f ? kCapped : kPlain;
    if (dtype == GDR_F32)
        return mode == kPlain    ? launch_tc_kernel<float, D, 2, kPlain>(a, code, ws, s)
               : mode == kCapped ? launch_tc_kernel<float, D, 2, kCapped>(a, code, ws, s)
                                 : launch_tc_kernel<float, D, 2, kBiased>(a, code, ws, s);
    return mode == kPlain    ? launch_tc_kernel<__nv_bfloat16, D, 1, kPlain>(a, code, ws, s)
           : mode == kCapped ? launch_tc_kernel<__nv_bfloat16, D, 1, kCapped>(a, code, ws, s)
                             : launch_tc_kernel<__nv_bfloat16, D, 1, kBiased>(a, code, ws, s);
}

}  // namespace cattn
}  // namespace gdr
