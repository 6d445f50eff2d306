"""Attention over a paged 8-bit cache: the error of long sums. Values of one sign, so that sums that are cut at every
step instead of rounded show as a mean error that grows with the length."""
import pytest
import torch

from gated_delta_rule_03_gb300 import cache_attn
from tests import cache_ref as ref

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
E4M3 = torch.float8_e4m3fn


def one_sign(n, new, held, H, Hkv, d, dtype, page=64, shared=False):
    """n requests of `held` tokens each, in pages of their own or the same ones; values of 50 to 400 times 2^-7, unlike by
    column; queries of size 1."""
    g = torch.Generator(device="cuda").manual_seed(1)
    per = -(-held // page)
    pages = per if shared else n * per
    kc, vc = (torch.empty(pages, Hkv, page, d, dtype=E4M3, device="cuda") for _ in "kv")
    size = 0.25 + 0.75 * torch.rand(d, generator=g, device="cuda")
    for a in range(0, pages, 4096):
        shape = kc[a:a + 4096].shape
        kc[a:a + 4096] = (90 * torch.randn(shape, generator=g, device="cuda")).clamp(-448, 448).to(E4M3)
        vc[a:a + 4096] = ((200 + 200 * torch.rand(shape, generator=g, device="cuda")) * size).to(E4M3)
    scale = torch.full((pages, Hkv), 2.0 ** -7, device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(-1, per).expand(n, per).contiguous()
    return dict(q=torch.randn(n * new, H, d, generator=g, device="cuda").to(dtype), k_cache=kc, v_cache=vc, k_scale=scale,
                v_scale=scale.clone(), block_table=table,
                kv_lens=torch.full((n,), held, dtype=torch.int32, device="cuda"))


def errors(c, o, requests, rows, heads):
    """(norm of the error, mean of the relative error) of the first rows and heads of some requests, in 64 bits."""
    T, H, d = c["q"].shape
    pages, Hkv, page, _ = c["k_cache"].shape
    n, per = c["block_table"].shape
    held, new = int(c["kv_lens"][0]), T // n
    got, want = [], []
    for i in requests:
        for h in heads:
            first = int(c["block_table"][i, 0])
            k, v = (c[x][first:first + per, h * Hkv // H].reshape(-1, d)[:held] for x in ("k_cache", "v_cache"))
            x, top, out = c["q"][i * new:i * new + rows, h].double(), 0.0, 0.0
            pos = torch.arange(held - new, held - new + rows, device="cuda")[:, None]
            for a in range(0, held, 65536):  # (scores are a few units: no maximum needed in 64 bits)
                w = torch.exp(x @ k[a:a + 65536].double().T * 2.0 ** -7 * d ** -0.5)
                w = torch.where(torch.arange(a, a + w.shape[1], device="cuda") <= pos, w, 0.0)
                top, out = top + w.sum(-1, keepdim=True), out + w @ v[a:a + 65536].double() * 2.0 ** -7
            want.append(out / top)
            got.append(o[i * new:i * new + rows, h].double())
    got, want = torch.stack(got), torch.stack(want)
    return float((got - want).norm() / want.norm()), float(((got - want) / want).mean())


@gpu
@pytest.mark.parametrize("H,Hkv,d,n,held", [(8, 8, 128, 80, 16384), (8, 8, 64, 160, 8192), (96, 8, 256, 40, 8192), (16, 1, 128, 8, 131)])
def test_fp32_single_tokens_behind_many_each(H, Hkv, d, n, held):
    """Weights in two fp16 parts are off by 2^-21 of themselves, the two products of a tile of 16 tokens may be cut by
    2^-23 of its sum each, and the sum of tiles is rounded to nearest, either way: the mean does not grow with the length.
    A score is off by (d / 16) 2 steps of 2^-23 of a size of a few units, of either sign, and so are weights: 2^-20 in norm."""
    c = one_sign(n, 1, held, H, Hkv, d, F32)
    norm, mean = errors(c, cache_attn(**c), (0, n // 2, n - 1), 1, range(min(H, 8)))
    assert abs(mean) < 2.0 ** -21 + 3 * 2.0 ** -23 and norm < 2.0 ** -20 + 2.0 ** -21 + 3 * 2.0 ** -23, (norm, mean)


@gpu
@pytest.mark.parametrize("H,d", [(8, 64), (8, 128), (8, 256), (96, 256)])
def test_fp32_scores_of_single_tokens(H, d):
    """Queries and keys of one sign, scores of some 50: a sum over d whose steps were all cut would be too small by d / 8 cuts of
    half a 2^-23. Cut are the two products of a step of 16 by 2^-23 of their sum each, 2^-22 of the score; the steps' sum,
    queries in 22 bits and what comes after are rounded either way, which leaves the mean over 200 rows and 300 keys."""
    c = one_sign(200, 1, 300, H, 8, d, F32)
    c["q"] = c["q"].abs()
    c["k_cache"] = (c["k_cache"].view(torch.uint8) & 0x7f).view(E4M3)
    scale = 128 / d
    lse = cache_attn(**c, scale=scale, return_lse=True)[1]
    k = c["k_cache"].view(200, -1, 8, 64, d).double().transpose(1, 2).reshape(200, 8, -1, d)[:, :, :300] * 2.0 ** -7
    s = torch.einsum("nhd,nhjd->nhj", c["q"].double(), k.repeat_interleave(H // 8, 1)) * scale
    want = torch.logsumexp(s, -1)
    assert 20 < float(want.mean()) < 200
    mean = float(((lse.double() - want) / want).mean())
    assert abs(mean) < 2.0 ** -22 + 2.0 ** -23, mean


@gpu
@pytest.mark.parametrize("d,n,new,held", [(128, 152, 256, 1000000), (128, 152, 300, 300001), (128, 60, 256, 500000), (64, 155, 200, 400000),
                                          (256, 152, 128, 300000), (128, 1, 40, 66000)])
def test_bf16_prompts_behind_very_many_tokens(d, n, new, held):
    """Sums that stay in the tensor cores are cut by 2^-23 at most per step of 16 tokens, of 65,536 tokens at most: 2^-11. The
    outputs of a column are nearly the same for all rows; rounded to bf16 they are off by 2^-8 at most, 2^-8 / sqrt 3
    in the root mean square, so the mean over d columns by four times 2^-8 / sqrt(3 d) but once in 10,000 inputs."""
    c = one_sign(n, new, held, 1, 1, d, BF16, shared=True)
    norm, mean = errors(c, cache_attn(**c), (0, n // 2, n - 1), 4, range(1))
    assert abs(mean) < 2.0 ** -11 + 4 * 2.0 ** -8 / (3 * d) ** 0.5 and norm < 2.0 ** -8, (norm, mean)


@gpu
@pytest.mark.parametrize("n", [1, 38, 152])
@pytest.mark.parametrize("kw", [dict(slopes=0.002), dict(slopes=-0.002), dict(slopes=0.5), dict(causal=False), dict(softcap=4.0), dict(scale=1e-3, new=300)], ids=str)
def test_rows_whose_keys_are_seen_in_pieces(n, kw):
    """References that move between the pieces or fall, rows that see nothing of the last piece, heads that share keys, short
    requests beside long ones, with lse. Scores near a row's place count (see the test of biases in test_cache_attn.py)."""
    kw = dict(kw)
    new, held, H = kw.pop("new", 130), [131072 + 64 - 2, 140000, 33, 65536, 196700], 2
    c = one_sign(n, new, held[-1], H, 1, 64, BF16, page=128, shared=True)
    lens = [held[i % 5] for i in range(n - 1)] + [held[-1]]
    c["kv_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if "slopes" in kw:
        kw["slopes"] = torch.tensor([kw["slopes"], 0.3 * kw["slopes"]], device="cuda")
    o, lse = cache_attn(**c, return_lse=True, **kw)
    for i in sorted({0, 1 % n, 2 % n, 3 % n, n - 1}):
        rows = slice(i * new, (i + 1) * new)
        args = dict(dict(scale=64 ** -0.5), **kw)
        want = ref.attend(c["q"][rows], c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"], c["block_table"][i:i + 1], [lens[i]],
                          [0, new], **args)
        if "slopes" in kw and float(kw["slopes"][0]) > 0:
            want["most"] = 3 * want["dots"] + 30 * 0.7
        bo, bl = ref.attend_bounds(want, BF16, 64, lens[i], kw.get("softcap", 0.0))
        ref.check("lse", lse[rows], want["lse"], bl)
        ref.check("o", o[rows], want["o"], bo)


@gpu
def test_pieces_with_a_page_without_a_scale():
    """It reaches the rows that see it, whichever piece it stands in, and no others."""
    new, held, n = 130, 140000, 152
    c = one_sign(n, new, held, 1, 1, 64, BF16, page=128, shared=True)
    clean = cache_attn(**c, return_lse=True)
    spare = c["k_cache"].shape[0]
    for x in ("k_cache", "v_cache"):
        c[x] = torch.cat([c[x].view(torch.uint8), c[x][:1].view(torch.uint8)]).view(E4M3)
    for where in (3, 600, 1093):
        for x in ("k_scale", "v_scale"):
            scales = {y: torch.cat([c[y], c[y][:1]]) for y in ("k_scale", "v_scale")}
            scales[x][spare] = float("nan")
            table = c["block_table"].clone()
            table[5, where] = spare
            o, lse = cache_attn(**dict(c, block_table=table, **scales), return_lse=True)
            sees = torch.zeros(n * new, 1, dtype=torch.bool, device="cuda")
            sees[5 * new:6 * new, 0] = torch.arange(held - new, held, device="cuda") >= where * 128
            assert torch.equal(o.isnan().all(-1), sees) and torch.equal(o.isnan().any(-1), sees) and torch.equal(lse.isnan(), sees)
            assert torch.equal(o[~sees], clean[0][~sees]) and torch.equal(lse[~sees], clean[1][~sees])


@gpu
def test_more_new_tokens_than_cached_ones_in_pieces():
    """70,100 new tokens of 70,000: the first 100 rows see nothing; the next see one key after the other."""
    new, held = 70100, 70000
    c = one_sign(1, new, held, 1, 1, 64, BF16)
    o, lse = cache_attn(**c, return_lse=True)
    assert not bool(o[:100].any()) and bool((lse[:100] == -float("inf")).all())
    k, v = (c[x].reshape(-1, 64)[:held].double() * 2.0 ** -7 for x in ("k_cache", "v_cache"))
    for row in (100, 101, 164, 357, 65635, 65636, 65700, 70098, 70099):
        s = (c["q"][row, 0].double() @ k[:row - 99].T) / 8
        want = torch.softmax(s, 0) @ v[:row - 99]
        # bf16's half step, fp16 weights and 2^-11 of sums that are cut; a score is off by 2^-16 of a few units at most
        assert float(((o[row, 0].double() - want) / want).abs().max()) < 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -11 + 2.0 ** -12
        assert abs(float(lse[row, 0]) - float(torch.logsumexp(s, 0))) < 2.0 ** -14
