"""New keys and values in a paged 8-bit cache, run by run against 64 bits, and refusals. Scales are
powers of two, so every step but one rounding to a code is exact: codes and scales are equal."""
import ctypes
import math

import numpy as np
import pytest
import torch

from tests import cache_ref as ref

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
E4M3, INT8 = torch.float8_e4m3fn, torch.int8


def cache_of(pages, heads, page, d, codes, seed=0):
    g = torch.Generator().manual_seed(seed)
    make = lambda: (40 * torch.randn(pages, heads, page, d, generator=g)).clamp(-127, 127).round().to(codes)  # noqa: E731
    scale = lambda: torch.exp2(torch.randint(-9, -3, (pages, heads), generator=g).float())  # noqa: E731
    return [make(), make(), scale(), scale()]


def bits(t):
    return t.view(torch.uint8) if t.dtype == E4M3 else t


def check(k, v, slots, cache, but=()):
    """Appends on the GPU and in the reference; `cache` (CPU) is left as the reference has it. `but`: pages
    of which nothing is said."""
    from gated_delta_rule_03_gb300 import cache_append
    on = [t.cuda() for t in cache]
    cache_append(k, v, slots.cuda(), *on)
    ref.append(k, slots, cache[0], cache[2])
    ref.append(v, slots, cache[1], cache[3])
    for name, got, want in zip(("k_scale", "v_scale", "k_cache", "v_cache"), on[2:] + on[:2], cache[2:] + cache[:2]):
        got, want = got.cpu(), want.clone()
        for p in but:
            got[p] = want[p]
        if got.dtype == F32:
            assert torch.equal(got.nan_to_num(-1.0), want.nan_to_num(-1.0)), name
        else:
            assert torch.equal(bits(got), bits(want)), name
    return on


def rows_of(T, heads, d, dtype, seed, size=1.0, fused=False):
    g = torch.Generator().manual_seed(seed)
    w = (size * torch.randn(T, 2 * heads * d + 16, generator=g) * torch.exp(torch.randn(T, 1, generator=g))).to(dtype).cuda()
    k, v = w[:, :heads * d].view(T, heads, d), w[:, heads * d:2 * heads * d].view(T, heads, d)
    return (k, v) if fused else (k.contiguous(), v.contiguous())


# (place in a page, length) of the runs: (page, off, n); heads, page, d
CASES = [
    ([(2, 0, 1)], 1, 16, 64),
    ([(0, 15, 1), (3, 0, 16), (1, 5, 7)], 3, 16, 128),
    ([(5, 0, 64), (4, 0, 64), (0, 0, 3), (1, 63, 1), (2, 10, 54)], 2, 64, 128),
    ([(1, 100, 28), (0, 0, 128), (3, 1, 127)], 2, 128, 256),
    ([(i, (7 * i) % 32, 1) for i in range(40)], 8, 32, 128),
    ([(i, 0, 128) for i in range(20)], 1, 128, 64),
]


@gpu
@pytest.mark.parametrize("codes", [E4M3, INT8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_runs(case, dtype, codes):
    runs, heads, page, d = case
    pages = max(p for p, _, _ in runs) + 2
    slots = torch.tensor([p * page + off + i for p, off, n in runs for i in range(n)], dtype=torch.int32)
    for seed, size in ((0, 1.0), (1, 1e-4), (2, 300.0)):  # scales that stay, fall behind, grow
        k, v = rows_of(len(slots), heads, d, dtype, seed, size, fused=seed == 1)
        check(k, v, slots, cache_of(pages, heads, page, d, codes, seed))


@gpu
@pytest.mark.parametrize("codes", [E4M3, INT8], ids=["e4m3", "int8"])
def test_many_rows_with_padding(codes):
    """More than 2,048 rows: runs of whole pages and single tokens among them, slots outside the cache.
    Rows of no slot cut the run of page 42 in two: that page is unspecified, all others are not."""
    page, heads, d = 32, 2, 64
    runs = [(2 * i, 0, 32) for i in range(60)] + [(2 * i + 1, 4, 1) for i in range(60)] + [(120 + i, 8, 20) for i in range(8)]
    slots = [p * page + off + i for p, off, n in runs for i in range(n)]
    slots = [-1, -5] + slots[:700] + [-1] * 33 + slots[700:] + [2 ** 30, 129 * page, -(2 ** 31)] + [-1] * 100
    k, v = rows_of(len(slots), heads, d, BF16, 3)
    check(k, v, torch.tensor(slots, dtype=torch.int32), cache_of(129, heads, page, d, codes), but=[42])


@gpu
@pytest.mark.parametrize("codes", [E4M3, INT8], ids=["e4m3", "int8"])
def test_extreme_entries(codes):
    """Zeros, the smallest numbers, more than the largest scale holds, the exact top of a scale and one step
    above, ties between codes."""
    top = ref.TOP[codes]
    rows = torch.zeros(16, 1, 64)
    rows[1, 0, 0] = 1e-40
    rows[2, 0, 3] = 3e38
    rows[3, 0, 3], rows[3, 0, 4] = top * 2.0 ** -5, 5 * 2.0 ** -6
    rows[4, 0, 3] = top * 2.0 ** -5 * (1 + 2.0 ** -23)
    rows[5] = torch.arange(64) * top / 63
    rows[6] = torch.arange(64) + 0.5
    rows[7] = -rows[6]
    rows[8, 0, 0], rows[8, 0, 1] = top * 2.0 ** 60, 2.0 ** 50
    rows[9, 0, 0] = top * 2.0 ** -60
    k = rows.cuda()
    slots = torch.arange(16, dtype=torch.int32) * 16
    check(k, -k, slots, cache_of(16, 1, 16, 64, codes))


@gpu
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_entries_that_are_not_finite(bad):
    """They take the scale of their page and head; the page recovers when it is begun anew."""
    cache = cache_of(4, 2, 16, 64, E4M3)
    k, v = rows_of(20, 2, 64, BF16, 5)
    k[3, 1, 7] = bad
    slots = torch.tensor([16 + i for i in range(16)] + [32 + i for i in range(4)], dtype=torch.int32)
    check(k, v, slots, cache)
    assert cache[2][1].isnan().tolist() == [False, True] and not bool(cache[2][2].isnan().any()) and not bool(cache[3].isnan().any())
    k2, v2 = rows_of(1, 2, 64, BF16, 6)
    check(k2, v2, torch.tensor([16 + 9], dtype=torch.int32), cache)
    assert cache[2][1].isnan().tolist() == [False, True]
    check(k2, v2, torch.tensor([16], dtype=torch.int32), cache)
    assert not bool(cache[2].isnan().any())


@gpu
@pytest.mark.parametrize("codes", [E4M3, INT8], ids=["e4m3", "int8"])
def test_token_by_token_and_from_a_graph(codes):
    """A page filled by single tokens that grow: rescaled again and again."""
    from gated_delta_rule_03_gb300 import cache_append
    cache = cache_of(3, 2, 16, 64, codes)
    on = [t.cuda() for t in cache]
    k, v = rows_of(2, 2, 64, BF16, 7)
    slots = torch.zeros(2, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    cache_append(k, v, torch.full_like(slots, -1), *on)
    with torch.cuda.graph(graph):
        cache_append(k, v, slots, *on)
    for i in range(16):
        k2, v2 = rows_of(2, 2, 64, BF16, 10 + i, size=1.5 ** i)
        k.copy_(k2)
        v.copy_(v2)
        at = torch.tensor([i, 32 + i], dtype=torch.int32)
        slots.copy_(at)
        graph.replay()
        ref.append(k, at, cache[0], cache[2])
        ref.append(v, at, cache[1], cache[3])
        assert torch.equal(on[2].cpu(), cache[2]) and torch.equal(on[3].cpu(), cache[3])
        assert torch.equal(bits(on[0].cpu()), bits(cache[0])) and torch.equal(bits(on[1].cpu()), bits(cache[1]))


def test_refusals_on_the_host():
    from gated_delta_rule_03_gb300 import ops
    from gated_delta_rule_03_gb300.cache import CacheShape
    lib = ops._load()
    A = [0x100000000 * (i + 1) for i in range(7)]
    base = dict(num_pages=10, kv_heads=2, page=16, d=64, codes=0, dtype=1)

    def call(T=8, k=A[0], ks=0, v=A[1], vs=0, slots=A[2], kc=A[3], vc=A[4], ksc=A[5], vsc=A[6], **kw):
        return lib.gdr_cache_append(ctypes.byref(CacheShape(**dict(base, **kw))), T, k, ks, v, vs, slots, kc, vc, ksc, vsc, None)

    for kw in (dict(num_pages=0), dict(kv_heads=0), dict(num_pages=2 ** 28), dict(T=-1), dict(k=None), dict(slots=None), dict(kc=None),
               dict(vsc=None), dict(ks=64), dict(kc=A[4]), dict(ksc=A[6]), dict(kc=A[0]), dict(ksc=A[2])):
        assert call(**kw) == -1, kw
    for kw in (dict(page=8), dict(page=24), dict(d=96), dict(d=32), dict(codes=2), dict(dtype=3)):
        assert call(**kw) == -2, kw
    for kw in (dict(k=A[0] + 8), dict(vc=A[4] + 4), dict(slots=A[2] + 1), dict(vsc=A[6] + 2), dict(vs=132)):
        assert call(**kw) == -3, kw
    assert call(T=0) == 0 and lib.gdr_cache_append(None, 8, A[0], 0, A[1], 0, *A[2:], None) == -1


@gpu
def test_refusals_of_tensors():
    from gated_delta_rule_03_gb300 import cache_append
    cache = [t.cuda() for t in cache_of(4, 2, 16, 64, E4M3)]
    k, v = rows_of(3, 2, 64, BF16, 1)
    slots = torch.zeros(3, dtype=torch.int32, device="cuda")
    for args, err in (((k.half(), v, slots, *cache), TypeError), ((k, v.float(), slots, *cache), TypeError),
                      ((k[:, :1], v, slots, *cache), ValueError), ((k, v, slots[:2], *cache), ValueError),
                      ((k, v, slots.long(), *cache), TypeError), ((k, v, slots, cache[0].view(torch.uint8), *cache[1:]), TypeError),
                      ((k, v, slots, cache[0], cache[1][:3], *cache[2:]), ValueError), ((k, v, slots, *cache[:2], cache[2].T, cache[3]), ValueError),
                      ((k.cpu(), v, slots, *cache), ValueError), ((k[..., ::2], v, slots, *cache), ValueError)):
        with pytest.raises(err):
            cache_append(*args)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("page,d", [(16, 64), (16, 128), (16, 256), (32, 64), (32, 128), (64, 64), (128, 64)])
def test_many_packed_rows(page, d, dtype):
    """More rows than a warp per few: whole pages, then stretches of short runs, single rows and padding, so that
    blocks with long runs, with short ones and with none stand side by side."""
    rng = np.random.default_rng(page + d)
    order = list(rng.permutation(1400))
    slots = []
    for piece in range(4):
        for _ in range(640 // page):
            first = int(order.pop()) * page
            slots += range(first, first + page)
        for _ in range(40):
            n = int(rng.integers(1, min(page, 12) + 1))
            off = int(rng.integers(0, page - n + 1))
            first = int(order.pop()) * page + off
            slots += range(first, first + n)
        slots += [-1] * 90
    assert len(slots) > 2048
    k, v = rows_of(len(slots), 1, d, dtype, 3, fused=True)
    check(k, v, torch.tensor(slots, dtype=torch.int32), cache_of(1400, 1, page, d, E4M3 if d != 64 else INT8, 4))


@gpu
@pytest.mark.parametrize("page,d", [(16, 64), (64, 128), (128, 256)])
def test_a_few_rows_that_are_long_runs(page, d):
    """Up to 2048 rows: a prompt's pages, a run that ends behind a block's rows, singles between, the rows' end."""
    slots = list(range(3, 3 * page)) + [5 * page + 1] + list(range(6 * page + 2, 7 * page)) + [-1, -1, 9 * page] + list(range(10 * page, 11 * page + 5))
    for cut in (len(slots), len(slots) - 1, 5):
        k, v = rows_of(cut, 2, d, BF16, cut)
        check(k, v, torch.tensor(slots[:cut], dtype=torch.int32), cache_of(12, 2, page, d, INT8, 6))
