"""Attention over a paged 8-bit cache against 64 bits: prompts, pieces of prompts and single tokens.
Pages that no request has, and places behind a request's last token, hold codes and scales
that are no numbers."""
import ctypes
import itertools
import math

import numpy as np
import pytest
import torch

from tests import cache_ref as ref
from tests.helpers import check_guards, poisoned

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
E4M3, INT8 = torch.float8_e4m3fn, torch.int8


def make(new, held, H, Hkv, d, page, dtype, codes, seed=0, behind=0, fused=False, size=1.0, spread=2):
    """new, held: new tokens and tokens in the cache (the new ones among them) of every request."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = len(new)
    need = [-(-x // page) for x in held]
    width, pages = max(1, max(need)) + 1, sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((n, width), -7, dtype=torch.int32, device="cuda")
    junk = 0x7f if codes == E4M3 else 0x80
    c = dict(new=new, held=held, H=H, Hkv=Hkv, d=d, page=page, dtype=dtype, codes=codes, table=table)
    for x in "kv":
        codes_ = torch.full((pages, Hkv, page, d), junk, dtype=torch.uint8, device="cuda")
        scale = torch.full((pages, Hkv), math.nan, device="cuda")
        at = 0
        for i in range(n):
            mine = order[at:at + need[i]].long()
            at += need[i]
            table[i, :need[i]] = mine.int()
            if not need[i]:
                continue
            z = torch.randn(need[i], Hkv, page, d, generator=g, device="cuda") * (100 if codes == E4M3 else 40)
            z = (z.clamp(-448, 448).to(codes) if codes == E4M3 else z.round().clamp(-127, 127).to(codes)).view(torch.uint8)
            place = torch.arange(need[i] * page, device="cuda").view(need[i], 1, page, 1)
            codes_[mine] = torch.where(place < held[i], z, junk)
            scale[mine] = torch.exp2((-6.5 if codes == E4M3 else -5) + spread * torch.randn(need[i], Hkv, generator=g, device="cuda")).clamp(2.0 ** -16, 1)
        c[x + "c"], c[x + "s"] = codes_.view(codes), scale
    T = sum(new) + behind
    w = (size * torch.randn(T, (H + 2) * d, generator=g, device="cuda")).to(dtype)
    c["q"] = w[:, :H * d].view(T, H, d) if fused else w[:, :H * d].reshape(T, H, d).contiguous()
    c["kv"] = torch.tensor(held, dtype=torch.int32, device="cuda")
    c["cu_list"] = [0] + list(np.cumsum(new))
    c["cu"] = torch.tensor(c["cu_list"], dtype=torch.int32, device="cuda")
    c["T"] = T
    return c


def run(c, cu=True, **kw):
    from gated_delta_rule_03_gb300 import cache_attn
    (o, g0), (lse, g1) = poisoned(c["q"].shape, c["dtype"], "cuda"), poisoned(c["q"].shape[:2], F32, "cuda")
    kw = dict(dict(cu_q=c["cu"] if cu else None, max_q=max(max(c["new"]), 1)), **kw)
    cache_attn(c["q"], c["kc"], c["vc"], c["ks"], c["vs"], c["table"], c["kv"], return_lse=True, o=o, lse=lse, **kw)
    check_guards([g0, g1])
    return o, lse


def compare(c, o, lse, scale=None, softcap=0.0, slopes=None, causal=True, **_):
    rows = sum(c["new"])
    want = ref.attend(c["q"][:rows], c["kc"], c["vc"], c["ks"], c["vs"], c["table"], c["held"], c["cu_list"],
                      c["d"] ** -0.5 if scale is None else scale, softcap, slopes, causal)
    bo, bl = ref.attend_bounds(want, c["dtype"], c["d"], max(c["held"]), softcap)
    ref.check("lse", lse[:rows], want["lse"], bl)
    ref.check("o", o[:rows], want["o"], bo)
    assert bool(o[rows:].isnan().all()) and bool(lse[rows:].isnan().all()), "rows behind the last request were written"


def check(c, cu=True, **kw):
    compare(c, *run(c, cu, **kw), **{k: v for k, v in kw.items() if k != "max_q"})


# new tokens, tokens in the cache, heads, heads of the cache, d, page
CASES = [
    ([1], [1], 1, 1, 64, 16),
    ([1], [16], 4, 1, 128, 16),
    ([1, 1, 1], [65, 1, 130], 8, 2, 64, 32),
    ([1] * 5, [0, 7, 300, 64, 1], 6, 2, 128, 16),
    ([1, 0, 1], [4000, 50, 9], 8, 1, 128, 64),
    ([1], [9001], 16, 1, 256, 128),
    ([1] * 3, [700, 40, 1500], 40, 2, 64, 16),
    ([3, 0, 5, 1], [3, 0, 200, 77], 4, 2, 128, 16),
    ([17], [17], 2, 2, 64, 16),
    ([130, 1], [130, 300], 3, 1, 128, 32),
    ([65, 128, 9], [200, 128, 1000], 4, 4, 64, 64),
    ([300], [2000], 2, 1, 256, 64),
    ([257, 40], [257, 500], 8, 2, 128, 128),
    ([9], [4], 2, 1, 64, 16),
    ([200, 31], [60, 31], 4, 2, 128, 16),
    ([600], [600], 1, 1, 128, 64),
]


@gpu
@pytest.mark.parametrize("codes", [E4M3, INT8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_against_64_bits(case, dtype, codes):
    c = make(*case, dtype, codes, behind=3, fused=True)
    check(c)
    check(c, causal=False)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", [2, 4, 9, 10, 11, 13, 14], ids=str)
def test_capped_scores_and_a_bias_by_distance(case, dtype):
    new, held, H, Hkv, d, page = CASES[case]
    c = make(new, held, H, Hkv, d, page, dtype, E4M3, seed=1, size=4.0)
    slopes = torch.exp2(-8 * (torch.arange(H, device="cuda") + 1.0) / H)
    for kw in (dict(softcap=5.0), dict(slopes=slopes), dict(softcap=20.0, slopes=slopes, scale=0.3), dict(slopes=slopes, causal=False),
               dict(slopes=-0.01 * slopes, scale=-0.2)):
        check(c, **kw)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_equal_lengths_without_offsets(dtype):
    for new, held in ((1, [5, 100, 64, 0]), (40, [40, 100, 64, 41]), (130, [130, 300])):
        c = make([new] * len(held), held, 4, 2, 128, 32, dtype, E4M3, seed=2)
        check(c, cu=False, max_q=None)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("new", [1, 70])
def test_scores_and_pages_of_very_different_size(dtype, new):
    """Peaked rows, maxima that move late, pages whose scales differ by 2^15, queries of size 2^-120 to 2^100."""
    c = make([new, new], [900, 333], 2, 1, 64, 16, dtype, E4M3, seed=3, size=30.0, spread=5)
    check(c)
    q = c["q"].clone()
    c["q"] = q * 2.0 ** 100
    check(c, scale=2.0 ** -100 / 8)
    c["q"] = q * 2.0 ** -120
    check(c, scale=2.0 ** 100)
    c["q"] = q * torch.exp2(torch.arange(64, device="cuda") - 40.0).to(dtype)
    check(c, scale=2.0 ** -24)


@gpu
def test_more_requests_than_a_block_has_threads():
    r = np.random.RandomState(4)
    held = r.randint(0, 200, 1200).tolist()
    c = make([1 if i % 7 else 0 for i in range(1200)], held, 2, 1, 64, 16, BF16, INT8, seed=4)
    check(c)
    new = [int(min(h, x)) for h, x in zip(held, r.randint(0, 20, 1200))]
    check(make(new, held, 2, 1, 64, 16, BF16, E4M3, seed=5, behind=2))


@gpu
@pytest.mark.parametrize("new", [1, 60])
def test_a_long_cache(new):
    c = make([new], [70001], 4, 1, 128, 64, BF16, E4M3, seed=6)
    check(c)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_keys_of_few_rows_are_shared_out(d, dtype):
    """A long cache that many blocks work on for one request, a short one beside it, one without new tokens and one
    without cached ones; for a few rows and for many."""
    for new in ([1, 1, 0, 1], [40, 3, 0, 2]):
        c = make(new, [9000, 70, 500, 0], 6, 2, d, 128, dtype, INT8, seed=11, behind=1)
        check(c)
        check(c, softcap=3.0, slopes=torch.full((6,), 0.01, device="cuda"))


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_more_items_than_the_gpu_has_blocks(d, dtype):
    """Blocks go from item to item: of several tiles of rows, of few and of none."""
    c = make([300, 0, 17, 1, 129], [350, 40, 17, 900, 200], 64, 32, d, 16, dtype, E4M3, seed=12, behind=2)
    check(c)
    c = make([3, 1, 2] * 20, [50, 0, 300] * 20, 32, 32, d, 32, dtype, E4M3, seed=13)
    check(c)


@gpu
def test_calls_without_rows():
    from gated_delta_rule_03_gb300 import cache_attn
    c = make([0, 0], [30, 0], 4, 2, 64, 16, BF16, E4M3)
    for cu in (c["cu"], None):
        o, lse = cache_attn(c["q"], c["kc"], c["vc"], c["ks"], c["vs"], c["table"], c["kv"], cu_q=cu, return_lse=True)
        torch.cuda.synchronize()
        assert o.shape == (0, 4, 64) and lse.shape == (0, 4)


@gpu
@pytest.mark.parametrize("new", [1, 90])
def test_a_cache_behind_two_to_the_31_bytes(new):
    from gated_delta_rule_03_gb300 import cache_attn
    c = make([new, new], [150, 260], 4, 2, 256, 128, BF16, E4M3, seed=7)
    want = run(c)
    pages = 2 ** 31 // (2 * 128 * 256) + 20
    far = torch.randperm(16, device="cuda").int()[:int((c["table"] >= 0).sum())] + pages - 16
    at = c["table"] >= 0
    big = {}
    for x in ("kc", "vc"):
        big[x] = torch.zeros(pages, 2, 128, 256, dtype=torch.uint8, device="cuda")
        big[x][far.long()] = c[x].view(torch.uint8)[c["table"][at].long()]
    for x in ("ks", "vs"):
        big[x] = torch.zeros(pages, 2, device="cuda")
        big[x][far.long()] = c[x][c["table"][at].long()]
    table = c["table"].clone()
    table[at] = far
    got = cache_attn(c["q"], big["kc"].view(E4M3), big["vc"].view(E4M3), big["ks"], big["vs"], table, c["kv"], cu_q=c["cu"], max_q=new, return_lse=True)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("new", [1, 5, 64])
def test_a_page_without_a_scale_reaches_only_who_looks_at_it(new, dtype):
    c = make([new, new], [100, 90], 2, 2, 64, 16, dtype, E4M3, seed=8)
    clean = run(c)
    page = int(c["table"][0, 5])  # tokens 80 .. 95 of the first request
    for x in ("ks", "vs"):
        keep = c[x].clone()
        c[x][page, 1] = math.nan
        o, lse = run(c)
        c[x].copy_(keep)
        sees = torch.zeros(2 * new, 2, dtype=torch.bool, device="cuda")
        for i in range(new):
            sees[i, 1] = 100 - new + i >= 80
        assert torch.equal(o.isnan().all(-1), sees) and torch.equal(o.isnan().any(-1), sees)
        assert torch.equal(lse.isnan(), sees)
        assert torch.equal(o[~sees], clean[0][~sees]) and torch.equal(lse[~sees], clean[1][~sees])
    # an entry outside the cache, of either sign
    for bad in (-1, c["kc"].shape[0], 2 ** 31 - 1):
        table = c["table"].clone()
        c["table"][0, 5] = bad
        o, lse = run(c)
        c["table"].copy_(table)
        sees[:, 0] = sees[:, 1]
        assert torch.equal(o.isnan().all(-1), sees) and torch.equal(lse.isnan(), sees) and torch.equal(o[~sees], clean[0][~sees])


@gpu
@pytest.mark.parametrize("new", [1, 40])
def test_a_query_that_is_not_finite_stays_in_its_row(new):
    c = make([new, new], [100, 90], 4, 2, 64, 16, BF16, E4M3, seed=9)
    clean = run(c)
    for bad in (math.nan, math.inf):
        keep = c["q"].clone()
        c["q"][new - 1, 2, 5] = bad
        o, lse = run(c)
        c["q"].copy_(keep)
        hit = torch.zeros(2 * new, 4, dtype=torch.bool, device="cuda")
        hit[new - 1, 2] = True
        assert bool(o[hit].isnan().all()) and torch.equal(o[~hit], clean[0][~hit]) and torch.equal(lse[~hit], clean[1][~hit])


@gpu
@pytest.mark.parametrize("new", [1, 3, 50])
def test_lengths_that_do_not_hold_are_found_on_the_device(new):
    from gated_delta_rule_03_gb300 import cache_attn, ops
    c = make([new, new], [100, 90], 4, 2, 64, 16, BF16, E4M3, seed=10)
    ws = torch.empty(1 << 27, dtype=torch.uint8, device="cuda")
    width = c["table"].shape[1]

    def status(cu=None, kv=None, max_q=new):
        o = torch.full_like(c["q"], math.nan)
        cache_attn(c["q"], c["kc"], c["vc"], c["ks"], c["vs"], c["table"], c["kv"] if kv is None else torch.tensor(kv, dtype=torch.int32, device="cuda"),
                   cu_q=c["cu"] if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda"), max_q=max_q, o=o, workspace=ws)
        st = ops.read_device_status(ws)
        assert bool(o.isnan().all()) == (st != 0)
        return st

    assert status() == 0
    for cu in ([1, new, 2 * new], [0, new, 2 * new + 1], [0, new + 1, new], [0, -1, new], [0, 2 ** 31 - 1, 2 * new]):
        assert status(cu=cu) == -7, cu
    for kv in ([-1, 5], [5, width * 16 + 1], [2 ** 31 - 1, 0]):
        assert status(kv=kv) == -7, kv
    assert status(max_q=new - 1) == -7
    assert status() == 0


@gpu
@pytest.mark.parametrize("new,H", [(1, 8), (33, 4)])
def test_two_calls_at_once_a_graph_and_the_same_bits(new, H):
    from gated_delta_rule_03_gb300 import cache_attn
    cs = [make([new, new, 1], [3000, 40, 777], H, 2, 128, 64, BF16, E4M3, seed=20 + i) for i in range(2)]
    call = lambda c, **kw: cache_attn(c["q"], c["kc"], c["vc"], c["ks"], c["vs"], c["table"], c["kv"], cu_q=c["cu"], max_q=new, return_lse=True, **kw)  # noqa: E731
    want = [call(c) for c in cs]
    sides = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [call(c, stream=s) for c, s in zip(cs, sides)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for w, g in zip(want, got) for a, b in zip(w, g))
    ws = torch.empty(1 << 27, dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for c in cs:  # two graphs that share a workspace, in order on one stream
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(c, workspace=ws))
        graphs.append(g)
    for i in (0, 1, 1, 0, 1):
        ws.fill_(255)
        for t in outs[i]:
            t.fill_(math.nan)
        graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want[i], outs[i]))
    # a replay takes the lengths it finds
    c = cs[0]
    c["kv"].copy_(torch.tensor([2000, 40, 1], dtype=torch.int32))
    c["held"] = [2000, 40, 1]
    graphs[0].replay()
    torch.cuda.synchronize()
    compare(c, *[torch.cat([t, torch.full_like(t[:1], math.nan)]) for t in outs[0]])


def shape(**kw):
    from gated_delta_rule_03_gb300.cache import CacheAttnShape, CacheShape
    cache = dict(num_pages=10, kv_heads=2, page=16, d=64, codes=0, dtype=1)
    rest = dict(num_seqs=2, total_tokens=8, max_q=8, width=5, q_stride=0, heads=4, causal=1, scale=0.125, softcap=0.0)
    for k, v in kw.items():
        (cache if k in cache else rest)[k] = v
    return ctypes.byref(CacheAttnShape(CacheShape(**cache), **rest))


def test_refusals_on_the_host():
    from gated_delta_rule_03_gb300 import ops
    lib = ops._load()
    A = [0x100000000 * (i + 1) for i in range(12)]
    size = lib.gdr_cache_attn_workspace_size
    assert size(shape()) > 0

    def call(ws_bytes=None, **kw):
        names = ("q", "kc", "vc", "ks", "vs", "table", "kv", "cu", "slopes", "o", "lse", "ws")
        args = [kw.pop(n, a) for n, a in zip(names, A)]
        s = shape(**kw)
        return lib.gdr_cache_attn(s, *args, size(s) if ws_bytes is None else ws_bytes, None)

    for kw in (dict(num_pages=0), dict(kv_heads=0), dict(heads=5), dict(heads=0), dict(num_seqs=0), dict(total_tokens=-1), dict(max_q=-1), dict(width=0),
               dict(scale=math.inf), dict(softcap=-1.0), dict(softcap=1e-20), dict(softcap=math.nan), dict(q_stride=128)):
        assert size(shape(**kw)) == 0 and call(1 << 40, **kw) == -1, kw
    for kw in (dict(page=8), dict(d=96), dict(codes=2), dict(dtype=5)):
        assert size(shape(**kw)) == 0 and call(1 << 40, **kw) == -2, kw
    for n in ("q", "kc", "vc", "ks", "vs", "table", "kv", "o"):
        assert call(**{n: None}) == -1, n
    for n, by in (("q", 8), ("kc", 8), ("vc", 4), ("o", 2), ("ws", 8), ("ks", 2), ("table", 2), ("kv", 1), ("cu", 2), ("slopes", 2), ("lse", 2)):
        at = A[("q", "kc", "vc", "ks", "vs", "table", "kv", "cu", "slopes", "o", "lse", "ws").index(n)] + by
        assert call(**{n: at}) == -3, n
    assert call(q_stride=260) == -3
    assert call(ws=None) == -4 and call(ws_bytes=size(shape()) - 1) == -4
    assert call(cu=None, num_seqs=3) == -1
    for a, b in itertools.product(("o", "lse", "ws"), ("q", "kc", "vs", "table", "kv", "cu", "slopes")):
        names = ("q", "kc", "vc", "ks", "vs", "table", "kv", "cu", "slopes", "o", "lse", "ws")
        assert call(**{a: A[names.index(b)]}) == -1, (a, b)
    assert call(lse=A[9]) == -1 and call(ws=A[9]) == -1
    assert lib.gdr_cache_attn(None, *A, 1 << 40, None) == -1


@gpu
def test_refusals_of_tensors():
    from gated_delta_rule_03_gb300 import cache_attn
    c = make([1, 1], [20, 30], 4, 2, 64, 16, BF16, E4M3)
    good = dict(q=c["q"], k_cache=c["kc"], v_cache=c["vc"], k_scale=c["ks"], v_scale=c["vs"], block_table=c["table"], kv_lens=c["kv"])
    cache_attn(**good)
    for kw, err in ((dict(q=c["q"].half()), TypeError), (dict(q=c["q"][0]), TypeError), (dict(k_cache=c["kc"].view(torch.uint8)), TypeError),
                    (dict(v_cache=c["vc"].view(INT8)), TypeError), (dict(v_scale=c["vs"][:1]), ValueError), (dict(block_table=c["table"].long()), TypeError),
                    (dict(block_table=c["table"][0]), ValueError), (dict(kv_lens=c["kv"][:1]), ValueError), (dict(kv_lens=c["kv"].cpu()), ValueError),
                    (dict(cu_q=c["cu"][:2]), ValueError), (dict(slopes=torch.ones(3, device="cuda")), ValueError),
                    (dict(q=torch.zeros(2, 4, 128, device="cuda", dtype=BF16)), ValueError), (dict(o=torch.zeros(2, 4, 64, device="cuda")), TypeError),
                    (dict(lse=torch.zeros(2, 3, device="cuda")), ValueError), (dict(q=c["q"][..., ::2]), ValueError)):
        with pytest.raises(err):
            cache_attn(**dict(good, **kw))


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("new", [1, 200])
def test_a_bias_by_distance_far_behind_a_row(new, dtype):
    """Of the scores only those near a row's own place weigh anything, and those are small: how far the others
    fall may not count in the error. So the size of a score in the bound is that of tokens with 2^-30 of the
    largest weight or more: those behind them have less than 2^-24 together (the slopes fall by 2^-30 within
    1100 tokens), and 2^-24 times their scores' errors is nothing beside the rest."""
    H = 6
    slopes = torch.tensor([0.02, 0.5, 1.0, 37.0, 1000.0, 30000.0], device="cuda")
    c = make([new], [20000], H, 2, 128, 64, dtype, E4M3, seed=5)
    o, lse = run(c, slopes=slopes)
    want = ref.attend(c["q"], c["kc"], c["vc"], c["ks"], c["vs"], c["table"], c["held"], c["cu_list"], c["d"] ** -0.5, 0.0, slopes)
    # such a token's bias is at most 30 ln 2 and the products' difference, 2 dots; its |s| one more
    want["most"] = 3 * want["dots"] + 30 * math.log(2)
    bo, bl = ref.attend_bounds(want, dtype, 128, 20000)
    ref.check("lse", lse, want["lse"], bl)
    ref.check("o", o, want["o"], bo)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("new", [1, 20])
def test_a_score_of_any_size_is_a_score(new, dtype):
    """The last token sees one key, at a score of some 1e33 of either sign: it takes its value."""
    c = make([new], [1], 4, 2, 128, 16, dtype, E4M3, seed=12)
    for scale in (1e32, -1e32):
        o, lse = run(c, scale=scale)
        want = ref.attend(c["q"], c["kc"], c["vc"], c["ks"], c["vs"], c["table"], c["held"], c["cu_list"], scale)
        assert float(want["lse"][-1].abs().min()) > 1e31 and bool((o[:-1] == 0).all()) and bool((lse[:-1] == -math.inf).all())
        # o: a weight over itself, and the value scale's logarithm lost beside the score, twice ...
        ref.check("o", o[-1:], want["o"][-1:], (2 * ref.HALF_STEP[dtype] + 2.0 ** -10) * want["o"][-1:].abs())
        # ... lse: scores of 128 products, with roundings of 2^-23 of their sizes, queries of 22 bits
        ref.check("lse", lse[-1:], want["lse"][-1:], 256 * 2.0 ** -23 * want["dots"][-1:] + 2.0 ** -20 * want["lse"][-1:].abs())


@gpu
@pytest.mark.parametrize("new", [1, 6, 70])
@pytest.mark.parametrize("cap", [2000.0, 1e5, 1e9])
def test_caps_far_above_the_scores(new, cap):
    """A score far below its cap is off by 2^-16 of itself, not of the cap."""
    for size in (1.0, 6.0):
        c = make([new], [900], 8, 4, 128, 32, BF16, INT8, seed=13, size=size)
        slopes = torch.exp2(-torch.arange(1.0, 9.0, device="cuda"))
        for kw in (dict(), dict(slopes=slopes)):
            o, lse = run(c, softcap=cap, **kw)
            want = ref.attend(c["q"], c["kc"], c["vc"], c["ks"], c["vs"], c["table"], c["held"], c["cu_list"], 128 ** -0.5, cap, kw.get("slopes"))
            bo, bl = ref.attend_bounds(want, BF16, 128, 900)
            capped = 2.0 ** -16 * want["dots"]  # |s| before a bias is below this sum of sizes
            ref.check("lse", lse, want["lse"], bl + capped)
            ref.check("o", o, want["o"], bo + 2 * capped[..., None] * want["size"])


@gpu
@pytest.mark.parametrize("new", [4, 70])
@pytest.mark.parametrize("cap", [65.0, 200.0, 1000.0, 1024.0, 1e4])
def test_a_capped_score_keeps_its_bits(new, cap):
    """Rows that see one key have that score for lse. Queries and keys of one entry, a bf16 number and 1: the product is
    exact, the cap off by 2^-16 of the score, the rest by a few roundings of the score, 2^-24 each, and of the
    logarithms of the value scale (7 of either sign)."""
    from gated_delta_rule_03_gb300 import cache_attn
    g = torch.Generator(device="cuda").manual_seed(3)
    c = make([new], [1], 2, 1, 128, 16, BF16, INT8)
    q = torch.zeros(new, 2, 128, device="cuda", dtype=BF16)
    q[..., 0] = torch.exp2(9 * torch.rand(new, 2, generator=g, device="cuda") - 6) * torch.sign(torch.randn(new, 2, generator=g, device="cuda"))
    page = c["table"][0, 0].long()
    c["kc"][page], c["ks"][page], c["vs"][page] = 0, 2.0 ** -6, 2.0 ** -7
    c["kc"][page, 0, 0, 0] = 64
    o, lse = cache_attn(q, c["kc"], c["vc"], c["ks"], c["vs"], c["table"], c["kv"], scale=1.0, softcap=cap, causal=False, return_lse=True)
    s = q[..., 0].double()
    want = cap * torch.tanh(s / cap)
    ref.check("lse", lse, want, 2.0 ** -16 * s.abs() + 8 * 2.0 ** -24 * (s.abs() + 14))
    value = c["vc"][page, 0, 0].double() * 2.0 ** -7
    ref.check("o", o, value.expand(new, 2, 128), 3 * ref.HALF_STEP[BF16] * value.abs().expand(new, 2, 128))


def test_tables_whose_tokens_pass_32_bits_are_refused():
    from gated_delta_rule_03_gb300 import ops
    size = ops._load().gdr_cache_attn_workspace_size
    most = (2 ** 31 - 4097) // 16
    assert size(shape(width=most)) > 0 and size(shape(width=most + 1)) == 0 and size(shape(width=(2 ** 31 - 1) // 16)) == 0


def test_rows_that_pass_32_bits_are_refused():
    """With offsets by max_q, without them by the tokens of each request, whatever max_q says."""
    from gated_delta_rule_03_gb300 import ops
    lib = ops._load()
    A = [2 ** 52 * (i + 1) for i in range(12)]
    names = ("q", "kc", "vc", "ks", "vs", "table", "kv", "cu", "slopes", "o", "lse", "ws")
    for cu, kw in ((A[7], dict(max_q=2 ** 21)), (None, dict(max_q=2 ** 21)), (None, dict(max_q=1))):
        args = [cu if n == "cu" else a for n, a in zip(names, A)]
        assert lib.gdr_cache_attn(shape(num_seqs=1, total_tokens=2 ** 21, heads=2048, kv_heads=1, **kw), *args, 2 ** 51, None) == -1, kw
