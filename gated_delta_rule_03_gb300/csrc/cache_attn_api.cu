// cache_attn_api.cu -- C ABI of attention over a paged 8-bit cache: checks of the arguments, the
// workspace and the choice of the kernel.
#include <math.h>

#include "cache_attn.cuh"
#include "spans.h"

namespace gdr {
int check_cache(const gdr_cache_shape *s, int *log_page);

namespace cattn {
namespace {

struct Call {
    Attn a;
    int d, codes, dtype;
    size_t e;
};

constexpr int kBeyond = 4096;  // places behind a request's last that the kernels look ahead, as 32-bit numbers

int64_t most_rows(const Attn &a) { return (INT32_MAX - 256) / a.group; }  // new tokens of a request (rows are 32-bit numbers)

int check_shape(const gdr_cache_attn_shape *s, Call *c) {
    if (!s) return GDR_ERR_INVALID_ARG;
    Attn &a = c->a;
    a = {};
    int st = check_cache(&s->cache, &a.log_page);
    if (st != GDR_OK) return st;
    if (s->num_seqs < 1 || s->num_seqs > INT32_MAX / 2 || s->total_tokens < 0 || s->total_tokens > INT32_MAX) return GDR_ERR_INVALID_ARG;
    if (s->max_q < 0 || s->max_q > INT32_MAX || s->width < 1 || s->width > (INT32_MAX - kBeyond) / s->cache.page) return GDR_ERR_INVALID_ARG;
    if (s->heads < 1 || s->heads > 1 << 16 || s->heads % s->cache.kv_heads) return GDR_ERR_INVALID_ARG;
    if (!isfinite(s->scale) || !isfinite(s->softcap) || s->softcap < 0.f) return GDR_ERR_INVALID_ARG;
    if (s->softcap > 0.f && s->softcap < 1e-18f) return GDR_ERR_INVALID_ARG;  // (its reciprocal is used)
    c->d = s->cache.d;
    c->codes = s->cache.codes;
    c->dtype = s->cache.dtype;
    c->e = c->dtype == GDR_F32 ? 4 : 2;
    if ((st = row_stride(s->q_stride, (int64_t)s->heads * c->d, c->e, &a.qs)) != GDR_OK) return st;
    a.num_seqs = s->num_seqs;
    a.tokens = s->total_tokens;
    a.max_q = s->max_q < s->total_tokens ? s->max_q : s->total_tokens;
    a.width = s->width;
    a.pages = s->cache.num_pages;
    a.heads = s->heads;
    a.kv_heads = s->cache.kv_heads;
    a.group = s->heads / s->cache.kv_heads;
    a.causal = s->causal != 0;
    a.group_shift = -1;
    for (int i = 0; i < 17; ++i)
        if (a.group == 1 << i) a.group_shift = i;
    if (a.max_q > most_rows(a)) return GDR_ERR_INVALID_ARG;
    a.scale = s->scale;
    a.softcap = s->softcap;
    return GDR_OK;
}

constexpr size_t kHead = 256;  // the status word

// Few rows share a head of the cache: at most a tile of the warp-level products, 16, so that its keys are read once. Single
// tokens are (up to 16 heads a group). 64 requests of some 4000 tokens, 8 heads of the cache of 128, with tiles of 16 rows
// one after the other against the many-row kernel: 32 rows 125 us either way, 64 rows 217 and 128; of two such
// requests 32 rows 39 and 27. fp32 would gain up to 32 rows (154 us for 232) by a tile more, which the few-row kernel
// does not have.
bool few_rows(const Attn &a) { return a.max_q * a.group <= 16; }

size_t workspace_bytes(const Call &c) {
    // (equal lengths without offsets may be shorter than max_q)
    const size_t step = c.d == 64 ? step_bytes64() : c.d == 128 ? step_bytes128() : step_bytes256();
    if (few_rows(c.a)) return kHead + step;
    const size_t tc = c.d == 64 ? tc_bytes64(c.a, c.dtype) : c.d == 128 ? tc_bytes128(c.a, c.dtype) : tc_bytes256(c.a, c.dtype);
    return kHead + (tc > step ? tc : step);
}

}  // namespace
}  // namespace cattn
}  // namespace gdr

using namespace gdr;
using namespace gdr::cattn;

extern "C" {

size_t gdr_cache_attn_workspace_size(const gdr_cache_attn_shape *shape) {
    Call c;
    return check_shape(shape, &c) == GDR_OK ? workspace_bytes(c) : 0;
}

int gdr_cache_attn(const gdr_cache_attn_shape *shape, const void *q, const void *k_cache, const void *v_cache,
                   const float *k_scale, const float *v_scale, const int32_t *block_table, const int32_t *kv_lens,
                   const int32_t *cu_q, const float *slopes, void *o, float *lse, void *workspace,
                   size_t workspace_bytes_given, gdr_stream_t stream) {
    Call c;
    int st = check_shape(shape, &c);
    if (st != GDR_OK) return st;
    Attn &a = c.a;
    if (!cu_q && a.tokens % a.num_seqs) return GDR_ERR_INVALID_ARG;
    if (!cu_q) a.max_q = a.tokens / a.num_seqs;
    if (a.max_q > most_rows(a)) return GDR_ERR_INVALID_ARG;
    if (!workspace) return GDR_ERR_WORKSPACE;
    const size_t need = workspace_bytes(c);
    if (workspace_bytes_given < need) return GDR_ERR_WORKSPACE;
    if (!k_cache || !v_cache || !k_scale || !v_scale || !block_table || !kv_lens) return GDR_ERR_INVALID_ARG;
    if (a.tokens > 0 && (!q || !o)) return GDR_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(o, 16) || !aligned(workspace, 16))
        return GDR_ERR_ALIGNMENT;
    const void *small[] = {k_scale, v_scale, block_table, kv_lens, cu_q, slopes, lse};
    for (const void *p : small)
        if (!aligned(p, 4)) return GDR_ERR_ALIGNMENT;
    const int64_t row = (int64_t)a.heads * c.d, cached = (int64_t)a.kv_heads * c.d << a.log_page;
    const Bytes in[] = {{q, reach(a.tokens, a.qs, row, c.e)},
                        {k_cache, (size_t)(a.pages * cached)},
                        {v_cache, (size_t)(a.pages * cached)},
                        {k_scale, (size_t)(a.pages * a.kv_heads) * 4},
                        {v_scale, (size_t)(a.pages * a.kv_heads) * 4},
                        {block_table, (size_t)(a.num_seqs * a.width) * 4},
                        {kv_lens, (size_t)a.num_seqs * 4},
                        {cu_q, (size_t)(a.num_seqs + 1) * 4},
                        {slopes, (size_t)a.heads * 4}};
    const Bytes out[] = {{o, (size_t)(a.tokens * row) * c.e}, {lse, (size_t)(a.tokens * a.heads) * 4}, {workspace, need}};
    if (!outputs_apart(in, 9, out, 3)) return GDR_ERR_INVALID_ARG;
    a.q = q;
    a.kc = (const uint8_t *)k_cache;
    a.vc = (const uint8_t *)v_cache;
    a.ks = k_scale;
    a.vs = v_scale;
    a.table = block_table;
    a.kv_lens = kv_lens;
    a.cu = cu_q;
    a.slopes = slopes;
    a.o = o;
    a.lse = lse;
    a.status = (int32_t *)workspace;
    void *const ws = (char *)workspace + kHead;
    const cudaStream_t s = (cudaStream_t)stream;
    if (few_rows(a))
        return c.d == 64 ? launch_step64(a, c.codes, c.dtype, ws, s)
                         : c.d == 128 ? launch_step128(a, c.codes, c.dtype, ws, s) : launch_step256(a, c.codes, c.dtype, ws, s);
    return c.d == 64 ? launch_tc64(a, c.codes, c.dtype, ws, s)
                     : c.d == 128 ? launch_tc128(a, c.codes, c.dtype, ws, s) : launch_tc256(a, c.codes, c.dtype, ws, s);
}

}  // extern "C"
