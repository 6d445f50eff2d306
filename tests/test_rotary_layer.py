"""A layer that is trained with rotary positions: one projection's views turned to their positions, linear attention
over packed sequences, and back through both, against the definitions in 64 bits and against differences."""
import numpy as np
import pytest
import torch

from tests import cache_ref as ref
from tests import linattn_ref as lin

gpu = pytest.mark.gpu
LENS, H, HK, D, ROT = [70, 1, 129], 4, 2, 64, 32


def layer(w, pos, rates, decay, cu, neighbours, amplitude):
    from gated_delta_rule_03_gb300 import linattn_fwd, rotary_fwd
    q, k, v = (t.unflatten(1, (-1, D)) for t in w.split([H * D, HK * D, HK * D], 1))
    q, k = rotary_fwd(q, k, pos, rates, neighbours=neighbours, amplitude=amplitude)
    o, _ = linattn_fwd(q, k, v, decay, cu_seqlens=cu, scale=D ** -0.5, final_state=False)
    return q, k, v, o


def pair_sums(x, neighbours):
    """|x| + |y| for the entries of a pair (CPU, 64 bits)."""
    y = torch.as_tensor(x).abs().clone()
    a, b = (slice(0, ROT, 2), slice(1, ROT, 2)) if neighbours else (slice(0, ROT // 2), slice(ROT // 2, ROT))
    both = y[..., a] + y[..., b]
    y[..., a], y[..., b] = both, both
    return y


@gpu
@pytest.mark.parametrize("neighbours", [False, True])
def test_gradients_of_a_layer(neighbours):
    from gated_delta_rule_03_gb300 import linattn_bwd, rotary_bwd, rotary_rates
    g = torch.Generator().manual_seed(5)
    T, amplitude = sum(LENS), 1.2
    w = torch.randn(T, (H + 2 * HK) * D, generator=g).cuda()
    do = torch.randn(T, H, D, generator=g).cuda()
    pos = torch.cat([torch.arange(n) for n in LENS]).int().cuda()
    cu = torch.tensor([0, *np.cumsum(LENS)], dtype=torch.int32, device="cuda")
    rates, decay = rotary_rates(ROT), -torch.tensor([0.0, 0.01, 0.1, 1.0], device="cuda")
    args = (pos, rates, decay, cu, neighbours, amplitude)
    q, k, v, o = layer(w, *args)
    dq, dk, dv, _ = linattn_bwd(do, q, k, v, decay, cu_seqlens=cu, scale=D ** -0.5)
    dq, dk = rotary_bwd(dq, dk, pos, rates, neighbours=neighbours, amplitude=amplitude, dq=dq, dk=dk)

    x = [t.cpu().double().unflatten(1, (-1, D)) for t in w.split([H * D, HK * D, HK * D], 1)]
    ld, g64 = decay.cpu().double().numpy(), do.cpu().double().numpy()
    turned = [ref.rotary(t, pos, rates.cpu(), neighbours, amplitude).numpy() for t in x[:2]] + [x[2].numpy()]
    want = lin.backward(g64, *turned, ld, LENS, scale=D ** -0.5)
    # An entry turned is off by e of its pair's size: sine and cosine by 2^-21 (see test_rotary.py), amplitude, products
    # and a sum 2^-24 each. Linear attention takes sums of at most L + 2 D terms, a rounding of each and of the sum so far, and
    # powers of the decay, 2^-20; sums over the pairs' sizes bound both.
    e = amplitude * (2.0 ** -21 + 4 * 2.0 ** -24)
    sums = (max(LENS) + 2 * D) * 2.0 ** -23 + 2.0 ** -20 + 4 * e
    sizes = [amplitude * pair_sums(t, neighbours).numpy() for t in x[:2]] + [x[2].abs().numpy()]
    most = lin.backward(np.abs(g64), *sizes, ld, LENS, scale=D ** -0.5)
    for name, got in (("dq", dq), ("dk", dk), ("dv", dv)):
        exact, bound = torch.from_numpy(want[name][0]), torch.from_numpy(sums * most[name][0])
        if name != "dv":
            bound = amplitude * pair_sums(bound, neighbours) + e * pair_sums(exact, neighbours)
            exact = ref.rotary(exact, pos, rates.cpu(), neighbours, amplitude, True)
        ref.check(name, got.cpu(), exact, bound + 2.0 ** -24 * exact.abs())
        assert float((got.cpu().double() - exact).norm() / exact.norm()) < 1e-5  # (errors of 100 terms and more of either sign)

    # differences of sum(o do) along a direction: the sum is linear in each of the three
    def total(u):
        return float((layer(u, *args)[3].double() * do.double()).sum())

    grad = torch.cat([t.flatten(1) for t in (dq, dk, dv)], 1).double()
    for a, b in ((0, H * D), (H * D, (H + HK) * D), ((H + HK) * D, w.shape[1])):
        step = torch.zeros_like(w)
        step[:, a:b] = torch.randn(T, b - a, generator=g).cuda()
        along = float((grad * step.double()).sum())
        # (each total is a sum of T H D outputs times do, off by 1e-5 in norm)
        tol = 1e-5 * 2 * float(layer(w + step, *args)[3].norm() * do.norm())
        assert abs((total(w + step) - total(w - step)) / 2 - along) < tol
