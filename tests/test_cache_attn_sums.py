"""Attention over a paged 8-bit cache: the error of long sums. Values of one sign, so that sums that are cut at every
step instead of rounded show as a mean error that grows with the length."""
import pytest
import torch

from gated_delta_rule_03_gb300 import cache_attn

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
E4M3 = torch.float8_e4m3fn


def one_sign(n, new, held, H, Hkv, d, dtype, page=64):
    """n requests of `held` tokens each, values of 50 to 400 times 2^-7, unlike by column; queries of size 1."""
    g = torch.Generator(device="cuda").manual_seed(1)
    per = -(-held // page)
    kc, vc = (torch.empty(n * per, Hkv, page, d, dtype=E4M3, device="cuda") for _ in "kv")
    size = 0.25 + 0.75 * torch.rand(d, generator=g, device="cuda")
    for a in range(0, n * per, 4096):
        shape = kc[a:a + 4096].shape
        kc[a:a + 4096] = (90 * torch.randn(shape, generator=g, device="cuda")).clamp(-448, 448).to(E4M3)
        vc[a:a + 4096] = ((200 + 200 * torch.rand(shape, generator=g, device="cuda")) * size).to(E4M3)
    scale = torch.full((n * per, Hkv), 2.0 ** -7, device="cuda")
    return dict(q=torch.randn(n * new, H, d, generator=g, device="cuda").to(dtype), k_cache=kc, v_cache=vc, k_scale=scale,
                v_scale=scale.clone(), block_table=torch.arange(n * per, dtype=torch.int32, device="cuda").view(n, per),
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
            k, v = (c[x][i * per:(i + 1) * per, h * Hkv // H].reshape(-1, d)[:held] for x in ("k_cache", "v_cache"))
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
