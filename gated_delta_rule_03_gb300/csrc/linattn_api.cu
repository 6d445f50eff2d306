// linattn_api.cu -- C ABI of linear attention with a constant decay per head: checks of the
// arguments, the segments of a call, the workspace and the launches.
#include <math.h>
#include <string.h>

#include "linattn.cuh"

namespace gdr {
namespace linattn {
namespace {

size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

struct Call {
    int64_t N, T;
    int H, qh, kh, vh, dk, dv, dtype;
    float scale;
    int64_t qs, ks, vs;
    size_t e;  // bytes per element
    size_t state() const { return (size_t)N * H * dk * dv * sizeof(float); }
};

int check_stride(int64_t given, int heads, int d, size_t e, int64_t *out) {
    const int64_t dense = (int64_t)heads * d;
    *out = given == 0 ? dense : given;
    if (*out < dense || *out > INT32_MAX) return GDR_ERR_INVALID_ARG;
    return (*out * (int64_t)e) % 16 == 0 ? GDR_OK : GDR_ERR_ALIGNMENT;
}

int check_shape(const gdr_linattn_shape *s, Call *c) {
    if (!s || s->num_seqs < 1 || s->total_tokens < 0 || s->H < 1) return GDR_ERR_INVALID_ARG;
    if (s->H > 1 << 16) return GDR_ERR_INVALID_ARG;  // a row of outputs stays below 2^31 bytes
    if (s->total_tokens > INT32_MAX || s->num_seqs > INT32_MAX / 2) return GDR_ERR_INVALID_ARG;
    if (s->q_heads < 1 || s->k_heads < 1 || s->v_heads < 1) return GDR_ERR_INVALID_ARG;
    if (s->H % s->q_heads || s->H % s->k_heads || s->H % s->v_heads) return GDR_ERR_INVALID_ARG;
    if (s->dtype != GDR_F32 && s->dtype != GDR_BF16) return GDR_ERR_UNSUPPORTED;
    if ((s->d_k != 64 && s->d_k != 128) || (s->d_v != 64 && s->d_v != 128 && s->d_v != 256))
        return GDR_ERR_UNSUPPORTED;
    if (!isfinite(s->scale)) return GDR_ERR_INVALID_ARG;
    c->N = s->num_seqs;
    c->T = s->total_tokens;
    c->H = s->H;
    c->qh = s->q_heads;
    c->kh = s->k_heads;
    c->vh = s->v_heads;
    c->dk = s->d_k;
    c->dv = s->d_v;
    c->dtype = s->dtype;
    c->scale = s->scale;
    c->e = s->dtype == GDR_F32 ? 4 : 2;
    // blocks of a launch: at most (tiles of 64 + sequences) x heads x slices (4) or parts (4) x mixes (3)
    if ((c->T / 64 + c->N) > (int64_t)(INT32_MAX / 16) / c->H) return GDR_ERR_INVALID_ARG;
    int st = check_stride(s->q_stride, c->qh, c->dk, c->e, &c->qs);
    if (st == GDR_OK) st = check_stride(s->k_stride, c->kh, c->dk, c->e, &c->ks);
    if (st == GDR_OK) st = check_stride(s->v_stride, c->vh, c->dv, c->e, &c->vs);
    return st;
}

// bf16 goes to the tensor cores (a call without tokens has nothing for them).
bool on_tensor_cores(const Call &c) { return c.dtype == GDR_BF16 && c.T > 0; }
// Slices of d_v: a tensor-core block takes 128 of its columns.
int slices(const Call &c) { return on_tensor_cores(c) && c.dv > 128 ? c.dv / 128 : 1; }
int columns(const Call &c, bool backward) {
    if (on_tensor_cores(c)) return (backward ? 3 : 1) * slices(c);
    return backward ? c.dk / 64 : c.dv / 64;
}

// How sequences are cut, by a model of the time in microseconds: a launch takes rounds of 152
// blocks. Tensor cores: a tile of 128 tokens takes 2.5 us in a mix and 1.2 in a sum, a block 8 to
// start and end, and reads a sum in 1; the second launch costs 4. (Where a state goes out both
// take 0.3 longer; the choice is the same.) fp32 arithmetic: tiles of 64
// tokens, 9 and 4 us, 3 to start, 2 a sum. Blocks of different lengths filling up an SM take
// 1.2 times their sum, and half a block's time is lost at the end. Measured, with the state:
//   4 x 4096 x 16 heads: 1, 2, 3, 4 segments 104, 90, 114, 121 us (without it 89, 80, 100, 107)
//   65536 x 16 chains: 5, 7, 9, 10 segments 477, 360, 301, 428 us (414, 317, 267, 376)
//   192 chains of 4096 (a backward call): all whole 180 us, 150 of them whole and 42 in three 150
//   eight packed sequences, 40,000 tokens, 16 heads, segments of 24 and of 72 tiles: all equal 208
//   and 145 us, the longest 1.6 times the mean 210 and 206, twice 256 and 284, 4 times 210 and
//   285; with 4 heads 11 tiles 76 us, 72 tiles 129
struct Cost {
    int tile;
    double mix, sum, start, read;
};
Cost cost_of(const Call &c) {
    if (on_tensor_cores(c)) return {128, 2.5, 1.2, 8, 1};
    return {64, 9, 4, 3, 2};
}
struct Cut {
    int64_t seg;    // tokens per segment
    int split;      // parts of one that are summed by themselves
    int64_t whole;  // (sequence, head) pairs that are not cut
};
Cut cut(const Call &c, bool packed, bool backward) {
    const Cost k = cost_of(c);
    const bool tc = on_tensor_cores(c);
    const int cols = columns(c, backward), sum_cols = tc && backward ? cols / 3 * 2 : cols;
    const int64_t tiles = (c.T + k.tile - 1) / k.tile;
    const int64_t mean = (c.T / c.N + k.tile - 1) / k.tile;
    // The longest sequence. Of packed ones the host knows no lengths, and takes 7/4 of the mean
    // (to a multiple of 4); a longer one is cut there, with its sums in up to four parts.
    int64_t m = mean;
    if (packed) {
        m = ((7 * mean + 3) / 4 + 3) / 4 * 4;
        if (c.N == 1 || m > tiles) m = tiles;
    }
    if (m <= 1) return {k.tile, 1, 0};
    const double sms = 152;
    const int64_t pairs = c.N * c.H;
    // blocks one after the other on every SM: equal ones in rounds, others filling up
    auto time = [&](double blocks, double longest, double total) {
        if (blocks <= sms) return longest + k.start;
        if (!packed) return ceil(blocks / sms) * (longest + k.start);
        return 1.2 * (total + blocks * k.start) / sms + 0.5 * (longest + k.start);
    };
    Cut best = {m, 1, 0};
    double best_cost = 1e300;
    // Pairs of equal lengths that fill whole rounds may stay whole, and only the rest is cut.
    const int64_t full = packed || pairs * cols < sms ? 0 : (int64_t)sms * (pairs * cols / (int64_t)sms) / cols;
    // Segments per sequence: each count up to 16, then in steps of an eighth, and those that
    // fill one to four rounds.
    auto consider = [&](int64_t n) {
        const int64_t len = (m + n - 1) / n, segs = (m + len - 1) / len;
        for (int64_t whole : {(int64_t)0, full}) {
            if (whole && (n == 1 || whole == pairs)) break;
            const int64_t cuts = pairs - whole;
            double items = (double)(cuts * segs);
            if (packed) items = fmax(((double)tiles / len + 0.5 * c.N) * c.H, (double)pairs);
            const double all = (double)(packed ? tiles * c.H : cuts * m);  // tiles of a mix
            const double handing = (items - cuts) / items;
            // (the sums in 1, 2 or 4 parts of a segment, on the tensor cores)
            for (int parts = 1; parts <= (n > 1 && tc ? 4 : 1); parts *= 2) {
                if (len % parts) break;
                double cost = time(items * cols, len * k.mix, all * cols * k.mix);
                if (whole) cost += time((double)(whole * cols), m * k.mix, 0);
                if (n > 1)
                    cost += 4 + time(items * handing * sum_cols * parts, (double)len / parts * k.sum, all * handing * sum_cols * k.sum) +
                            (double)(n - 1) * parts * k.read;
                if (cost < best_cost) {
                    best_cost = cost;
                    best = {len, parts, whole};
                }
            }
        }
    };
    for (int64_t n = 1; n <= m && n <= 256; n += n < 16 ? 1 : n / 8) consider(n);
    for (int64_t r = 1; r <= 4; ++r) {
        const int64_t n = r * (int64_t)sms / (pairs * cols);
        if (n > 16 && n <= m && n <= 256) consider(n);
    }
    best.seg *= k.tile;
    // (parts where the sums' blocks, most of them with nothing to do, still are one round: four
    // parts always, and so: 8 sequences of 1,611 to 7,848 tokens, 32 heads 267 and 258 us; 33 of
    // 300 to 2,200, 32 heads 338 and 310)
    if (packed && best.seg == m * k.tile && m < tiles && tc)
        for (best.split = 4; best.split > 1 && c.T / best.seg * c.H * sum_cols * best.split > sms;) best.split /= 2;
    return best;
}

Plan make_plan(const Call &c, const float *log_decay, const int32_t *cu, bool backward, void *ws) {
    Plan p = {};
    p.cu_seqlens = cu;
    p.num_seqs = c.N;
    p.total_tokens = c.T;
    p.H = c.H;
    p.log_decay = log_decay;
    p.status = (int32_t *)ws;
    const Cut at = cut(c, cu != nullptr, backward);
    p.seg = at.seg;
    p.split = at.split;
    if (cu) {
        p.sums = c.T / p.seg;
        p.handing = p.sums * c.H;
        p.units = p.handing + c.N * c.H;
    } else {
        p.seq_len = c.T / c.N;
        p.segs = (int)((p.seq_len + p.seg - 1) / p.seg);
        if (p.segs < 1) p.segs = 1;
        p.whole = p.segs > 1 ? at.whole : 0;
        p.sums = c.N * (p.segs - 1);
        p.handing = (c.N * c.H - p.whole) * (p.segs - 1);
        p.units = c.N * c.H + p.handing;
    }
    return p;
}
bool segmented(const Plan &p) { return p.cu_seqlens ? p.total_tokens > p.seg : p.segs > 1; }

// Workspace: status word; a copy of S0 where S_final is to be written over it; the
// segments' own sums (backward: those of both directions, and fp32 gradients of heads that
// share one).
struct Layout {
    size_t copy, R, R2, part[3], total;
    int parts[3];  // heads and slices whose gradients add up to one head's of dq, dk, dv
};
// `sums_each`: matrices of the segments' own sums per head and direction.
Layout layout(const Call &c, int64_t sums_each, bool backward) {
    Layout L = {};
    size_t off = 256;
    const size_t sums = (size_t)sums_each * c.H * c.dk * c.dv * sizeof(float);
    L.copy = off;
    if (!backward) off = align_up(off + c.state());
    L.R = off;
    off = align_up(off + sums);
    L.R2 = off;
    if (backward) {
        off = align_up(off + sums);
        const int heads[3] = {c.qh, c.kh, c.vh}, d[3] = {c.dk, c.dk, c.dv};
        for (int i = 0; i < 3; ++i) {
            L.part[i] = off;
            L.parts[i] = c.H / heads[i] * (i < 2 ? slices(c) : 1);
            if (L.parts[i] > 1) off = align_up(off + (size_t)c.T * heads[i] * L.parts[i] * d[i] * sizeof(float));
        }
    }
    L.total = off;
    return L;
}
int64_t sums_of(const Plan &p) { return segmented(p) ? p.sums * p.split : 0; }
// What a call needs, the larger of what equal and packed lengths take; its plan in *p.
size_t plan_call(const Call &c, bool backward, const float *log_decay, const int32_t *cu, void *ws, Plan *p) {
    static const int32_t some = 0;
    *p = make_plan(c, log_decay, cu, backward, ws);
    int64_t sums = sums_of(*p);
    if (!cu || c.T % c.N == 0) {
        const int64_t other = sums_of(make_plan(c, log_decay, cu ? nullptr : &some, backward, ws));
        if (other > sums) sums = other;
    }
    return layout(c, sums, backward).total;
}
size_t workspace_bytes_for(const Call &c, bool backward) {
    static const int32_t some = 0;
    Plan p;
    return plan_call(c, backward, nullptr, &some, nullptr, &p);
}

struct Span {
    const void *p;
    size_t n;
};
Span rows(const void *p, const Call &c, int64_t stride, int heads, int d) {
    return {p, c.T == 0 ? 0 : ((size_t)(c.T - 1) * stride + (size_t)heads * d) * c.e};
}
bool overlap(const Span &a, const Span &b) {
    if (!a.p || !b.p || !a.n || !b.n) return false;
    const char *x = (const char *)a.p, *y = (const char *)b.p;
    return x < y + b.n && y < x + a.n;
}
int check_spans(const Span *in, int ni, const Span *out, int no) {
    for (int i = 0; i < ni; ++i)
        if ((uintptr_t)in[i].p & 15u) return GDR_ERR_ALIGNMENT;
    for (int i = 0; i < no; ++i) {
        if ((uintptr_t)out[i].p & 15u) return GDR_ERR_ALIGNMENT;
        for (int j = 0; j < ni; ++j)
            if (overlap(out[i], in[j])) return GDR_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return GDR_ERR_INVALID_ARG;
    }
    return GDR_OK;
}

Mix mix_of(const Call &c, const void *x, int64_t xs, int xh, const void *y, int64_t ys, int yh,
           const void *z, int64_t zs, int zh, int dx, int dz) {
    Mix m = {};
    m.x = x; m.y = y; m.z = z;
    m.xs = xs; m.ys = ys; m.zs = zs;
    m.xg = c.H / xh; m.yg = c.H / yh; m.zg = c.H / zh;
    m.dx = dx; m.dz = dz;
    m.s_intra = m.s_inter = c.scale;
    m.s_state = 1.f;
    return m;
}

int launch(const Call &c, const Plan &p, const Mix *mixes, int count, bool sums, cudaStream_t s) {
    if (!on_tensor_cores(c)) return launch_mix_exact(p, mixes, count, s);
    return launch_mix_tc(p, mixes, count, c.dv, sums, !sums && segmented(p), s);
}
// Ahead of the first launch: it sets the status word, or a check of the offsets does.
int begin(Plan *p, cudaStream_t s) {
    p->checked = p->cu_seqlens && p->num_seqs > kChecked;
    p->first = !p->checked;
    return p->checked ? launch_check(*p, s) : GDR_OK;
}

}  // namespace
}  // namespace linattn
}  // namespace gdr

using namespace gdr;
using namespace gdr::linattn;

extern "C" {

size_t gdr_linattn_fwd_workspace_size(const gdr_linattn_shape *shape) {
    Call c;
    return check_shape(shape, &c) == GDR_OK ? workspace_bytes_for(c, false) : 0;
}

size_t gdr_linattn_bwd_workspace_size(const gdr_linattn_shape *shape) {
    Call c;
    return check_shape(shape, &c) == GDR_OK ? workspace_bytes_for(c, true) : 0;
}

int gdr_linattn_fwd(const gdr_linattn_shape *shape, const void *q, const void *k, const void *v,
                    const float *log_decay, const float *S0, const int32_t *cu_seqlens, void *o,
                    float *S_final, void *workspace, size_t workspace_bytes, gdr_stream_t stream) {
    Call c;
    int st = check_shape(shape, &c);
    if (st != GDR_OK) return st;
    if (!cu_seqlens && c.T % c.N != 0) return GDR_ERR_INVALID_ARG;
    if (!workspace) return GDR_ERR_WORKSPACE;
    if (!log_decay || (c.T > 0 && (!q || !k || !v || !o))) return GDR_ERR_INVALID_ARG;
    if (((uintptr_t)log_decay | (uintptr_t)cu_seqlens) & 3u) return GDR_ERR_ALIGNMENT;
    Plan p;
    const size_t need = plan_call(c, false, log_decay, cu_seqlens, workspace, &p);
    if (workspace_bytes < need) return GDR_ERR_WORKSPACE;
    const Span in[] = {rows(q, c, c.qs, c.qh, c.dk), rows(k, c, c.ks, c.kh, c.dk),
                       rows(v, c, c.vs, c.vh, c.dv), {S0 == S_final ? nullptr : S0, c.state()}};
    const Span out[] = {rows(o, c, (int64_t)c.H * c.dv, c.H, c.dv), {S_final, c.state()}, {workspace, need}};
    if ((st = check_spans(in, 4, out, 3)) != GDR_OK) return st;
    const Span small[] = {{log_decay, (size_t)c.H * 4}, {cu_seqlens, (size_t)(c.N + 1) * 4}};
    for (const Span &s : out)
        if (overlap(s, small[0]) || overlap(s, small[1])) return GDR_ERR_INVALID_ARG;

    const Layout L = layout(c, sums_of(p), false);
    char *ws = (char *)workspace;
    const cudaStream_t s = (cudaStream_t)stream;
    Mix m = mix_of(c, q, c.qs, c.qh, k, c.ks, c.kh, v, c.vs, c.vh, c.dk, c.dv);
    if ((st = begin(&p, s)) != GDR_OK) return st;
    p.fine = S_final != nullptr;
    if (segmented(p)) {
        // (the first segment of a sequence reads S0 while its last one may write S_final)
        if (S0 && S0 == S_final) {
            if (cudaMemcpyAsync(ws + L.copy, S0, c.state(), cudaMemcpyDeviceToDevice, s) != cudaSuccess)
                return GDR_ERR_CUDA;
            S0 = (const float *)(ws + L.copy);
        }
        Mix sums = m;
        sums.R_out = (float *)(ws + L.R);
        if ((st = launch(c, p, &sums, 1, true, s)) != GDR_OK) return st;
        m.R = sums.R_out;
        p.first = false;
    }
    m.start = S0;
    m.end = S_final;
    m.out = c.T > 0 ? o : (void *)workspace;  // (no rows: nothing is written to it)
    return launch(c, p, &m, 1, false, s);
}

int gdr_linattn_bwd(const gdr_linattn_shape *shape, const void *d_o, const void *q, const void *k,
                    const void *v, const float *log_decay, const float *S0, const float *dS_final,
                    const int32_t *cu_seqlens, void *dq, void *dk, void *dv, float *dS0,
                    void *workspace, size_t workspace_bytes, gdr_stream_t stream) {
    Call c;
    int st = check_shape(shape, &c);
    if (st != GDR_OK) return st;
    if (!cu_seqlens && c.T % c.N != 0) return GDR_ERR_INVALID_ARG;
    if (!workspace) return GDR_ERR_WORKSPACE;
    if (!log_decay || (c.T > 0 && (!d_o || !q || !k || !v || !dq || !dk || !dv))) return GDR_ERR_INVALID_ARG;
    if (((uintptr_t)log_decay | (uintptr_t)cu_seqlens) & 3u) return GDR_ERR_ALIGNMENT;
    Plan p;
    const size_t need = plan_call(c, true, log_decay, cu_seqlens, workspace, &p);
    if (workspace_bytes < need) return GDR_ERR_WORKSPACE;
    const int64_t os = (int64_t)c.H * c.dv;
    const Span in[] = {rows(q, c, c.qs, c.qh, c.dk), rows(k, c, c.ks, c.kh, c.dk), rows(v, c, c.vs, c.vh, c.dv),
                       rows(d_o, c, os, c.H, c.dv), {S0, c.state()}, {dS_final, c.state()}};
    const Span out[] = {rows(dq, c, (int64_t)c.qh * c.dk, c.qh, c.dk), rows(dk, c, (int64_t)c.kh * c.dk, c.kh, c.dk),
                        rows(dv, c, (int64_t)c.vh * c.dv, c.vh, c.dv), {dS0, c.state()}, {workspace, need}};
    if ((st = check_spans(in, 6, out, 5)) != GDR_OK) return st;
    const Span small[] = {{log_decay, (size_t)c.H * 4}, {cu_seqlens, (size_t)(c.N + 1) * 4}};
    for (const Span &s : out)
        if (overlap(s, small[0]) || overlap(s, small[1])) return GDR_ERR_INVALID_ARG;

    const Layout L = layout(c, sums_of(p), true);
    char *ws = (char *)workspace;
    const cudaStream_t s = (cudaStream_t)stream;
    Mix q_, k_, v_;  // dq, dk, dv
    q_ = mix_of(c, d_o, os, c.H, v, c.vs, c.vh, k, c.ks, c.kh, c.dv, c.dk);
    q_.turned = true;
    k_ = mix_of(c, v, c.vs, c.vh, d_o, os, c.H, q, c.qs, c.qh, c.dv, c.dk);
    k_.turned = true;
    v_ = mix_of(c, k, c.ks, c.kh, q, c.qs, c.qh, d_o, os, c.H, c.dk, c.dv);
    k_.backward = v_.backward = true;
    k_.s_inter = v_.s_inter = 1.f;
    k_.s_state = v_.s_state = c.scale;
    if ((st = begin(&p, s)) != GDR_OK) return st;
    p.fine = dS0 != nullptr;
    if (segmented(p)) {
        Mix sums[2];
        sums[0] = mix_of(c, nullptr, 0, c.H, k, c.ks, c.kh, v, c.vs, c.vh, c.dk, c.dv);
        sums[0].R_out = (float *)(ws + L.R);
        sums[1] = v_;
        sums[1].R_out = (float *)(ws + L.R2);
        if ((st = launch(c, p, sums, 2, true, s)) != GDR_OK) return st;
        q_.R = sums[0].R_out;
        k_.R = v_.R = sums[1].R_out;
        p.first = false;
    }
    q_.start = S0;
    k_.start = v_.start = dS_final;
    v_.end = dS0;
    Mix all[3] = {q_, k_, v_};
    void *to[3] = {dq, dk, dv};
    const int heads[3] = {c.qh, c.kh, c.vh};
    for (int i = 0; i < 3; ++i) {
        all[i].out_f32 = L.parts[i] > 1;
        all[i].out = all[i].out_f32 ? (void *)(ws + L.part[i]) : to[i];
        if (c.T == 0) all[i].out = workspace;  // (no rows: nothing is written to it)
    }
    if ((st = launch(c, p, all, 3, false, s)) != GDR_OK) return st;
    Share shares[3];
    int n = 0;
    for (int i = 0; i < 3 && c.T > 0; ++i)
        if (all[i].out_f32) shares[n++] = {(const float *)all[i].out, to[i], heads[i], L.parts[i], i == 2 ? c.dv : c.dk};
    if (n > 0) return launch_share(p, shares, n, c.dtype, s);
    return GDR_OK;
}

int gdr_linattn_step(const gdr_linattn_shape *shape, const void *q, const void *k, const void *v,
                     const float *log_decay, float *S, void *o, gdr_stream_t stream) {
    if (shape && shape->num_seqs == 0 && shape->total_tokens == 0) {
        gdr_linattn_shape one = *shape;
        one.num_seqs = 1;
        Call c;
        return check_shape(&one, &c);
    }
    Call c;
    int st = check_shape(shape, &c);
    if (st != GDR_OK) return st;
    if (c.T != c.N || c.N > INT32_MAX / 8 / c.H) return GDR_ERR_INVALID_ARG;
    if (!q || !k || !v || !log_decay || !S || !o) return GDR_ERR_INVALID_ARG;
    if ((uintptr_t)log_decay & 3u) return GDR_ERR_ALIGNMENT;
    const Span in[] = {rows(q, c, c.qs, c.qh, c.dk), rows(k, c, c.ks, c.kh, c.dk), rows(v, c, c.vs, c.vh, c.dv)};
    const Span out[] = {rows(o, c, (int64_t)c.H * c.dv, c.H, c.dv), {S, c.state()}};
    if ((st = check_spans(in, 3, out, 2)) != GDR_OK) return st;
    const Span decay = {log_decay, (size_t)c.H * 4};
    if (overlap(out[0], decay) || overlap(out[1], decay)) return GDR_ERR_INVALID_ARG;
    return launch_step(q, k, v, log_decay, S, o, c.N, c.H, c.H / c.qh, c.H / c.kh, c.H / c.vh, c.dk,
                       c.dv, c.dtype, c.scale, c.qs, c.ks, c.vs, (cudaStream_t)stream);
}

}  // extern "C"
