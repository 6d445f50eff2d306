"""Rotary positions against pairs turned in 64 bits, their gradients, and refusals."""
import ctypes
import math

import numpy as np
import pytest
import torch

from tests import cache_ref as ref
from tests.helpers import check_guards, poisoned

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def bound(x, dtype, amplitude):
    """An entry's terms are at most |amplitude| times its pair's size r = |x| + |y|: sine and cosine
    off by 2^-22 (the turn to fp32 half a step of its at most 2 radians-fold, the functions 2 units),
    amplitude, two products and a sum 2^-24 each; then the result's own rounding."""
    return lambda want, size: ref.HALF_STEP[dtype] * want.abs() + abs(amplitude) * size * (2.0 ** -21 + 4 * 2.0 ** -24) + 1e-44


def sizes(x, rot, neighbours):
    y = x.detach().cpu().double().abs()
    out = y.clone()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if neighbours else (slice(0, rot // 2), slice(rot // 2, rot))
    out[..., a] = out[..., b] = y[..., a] + y[..., b]
    out[..., rot:] = 0
    return out


def make(T, Hq, Hk, d, dtype, seed=0, far=5000, fused=False):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(T, (Hq + Hk + 1) * d, generator=g).to(dtype).cuda()
    q, k = w[:, :Hq * d].view(T, Hq, d), w[:, Hq * d:(Hq + Hk) * d].view(T, Hk, d)
    if not fused:
        q, k = q.contiguous(), k.contiguous()
    return q, k if Hk else None, torch.randint(0, far, (T,), generator=g, dtype=torch.int32).cuda()


CASES = [  # T, q heads, k heads, d, rot, neighbours, amplitude, fused
    (1, 1, 1, 64, 64, False, 1.0, False),
    (257, 5, 2, 128, 128, False, 1.0, True),
    (33, 16, 16, 128, 32, True, 1.2, True),
    (700, 3, 1, 256, 64, False, 0.5, False),
    (19, 4, 4, 96, 96, True, 1.0, False),
    (41, 7, 0, 40, 10, False, 1.0, False),
    (64, 2, 2, 72, 66, True, 1.0, True),
    (5, 32, 8, 8, 2, False, 1.0, False),
    (130, 9, 3, 128, 122, False, 1.0, True),
]


@gpu
@pytest.mark.parametrize("back", [False, True], ids=["fwd", "bwd"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_against_64_bits(case, dtype, back):
    from gated_delta_rule_03_gb300 import rotary_bwd, rotary_fwd, rotary_rates
    T, Hq, Hk, d, rot, neighbours, amplitude, fused = case
    q, k, pos = make(T, Hq, Hk, d, dtype, fused=fused)
    rates = rotary_rates(rot)
    outs = {n: poisoned(t.shape, dtype, "cuda") for n, t in (("q", q), ("k", k)) if t is not None}
    names = ("dq", "dk") if back else ("q_out", "k_out")
    (rotary_bwd if back else rotary_fwd)(q, k, pos, rates, neighbours=neighbours, amplitude=amplitude,
                                         **{o: outs[n][0] for o, n in zip(names, "qk") if n in outs})
    check_guards([g for _, g in outs.values()])
    for n, t in (("q", q), ("k", k)):
        if t is None:
            continue
        want = ref.rotary(t, pos, rates.cpu(), neighbours, amplitude, back)
        ref.check(n, outs[n][0].cpu(), want, bound(t, dtype, amplitude)(want, sizes(t, rot, neighbours)))
        assert torch.equal(outs[n][0][..., rot:], t[..., rot:]), "entries behind the pairs changed"


@gpu
@pytest.mark.parametrize("neighbours", [False, True])
def test_in_place_views_keep_their_neighbours(neighbours):
    from gated_delta_rule_03_gb300 import rotary_fwd, rotary_rates
    T, Hq, Hk, d = 50, 4, 2, 128
    w = torch.randn(T, (Hq + 2 * Hk) * d, device="cuda").bfloat16()
    before = w.clone()
    q, k = w[:, :Hq * d].view(T, Hq, d), w[:, Hq * d:(Hq + Hk) * d].view(T, Hk, d)
    pos, rates = torch.arange(T, dtype=torch.int32, device="cuda"), rotary_rates(64)
    want = rotary_fwd(q.clone(), k.clone(), pos, rates, neighbours=neighbours)
    got = rotary_fwd(q, k, pos, rates, neighbours=neighbours, q_out=q, k_out=k)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(w[:, (Hq + Hk) * d:], before[:, (Hq + Hk) * d:])
    # into the same places of another buffer
    u = torch.zeros_like(before)
    rotary_fwd(before[:, :Hq * d].view(T, Hq, d), before[:, Hq * d:(Hq + Hk) * d].view(T, Hk, d), pos, rates,
               neighbours=neighbours, q_out=u[:, :Hq * d].view(T, Hq, d), k_out=u[:, Hq * d:(Hq + Hk) * d].view(T, Hk, d))
    assert torch.equal(u[:, :(Hq + Hk) * d], w[:, :(Hq + Hk) * d]) and not bool(u[:, (Hq + Hk) * d:].any())


@gpu
def test_far_and_negative_positions():
    """fp32 angles would be off by whole radians here."""
    from gated_delta_rule_03_gb300 import rotary_fwd, rotary_rates
    pos = torch.tensor([0, 1, 2 ** 20 + 1, 2 ** 24 + 3, 2 ** 31 - 1, -1, -(2 ** 31), -77777], dtype=torch.int32, device="cuda")
    q = torch.randn(len(pos), 2, 128, device="cuda")
    rates = rotary_rates(128, base=500000.0)
    got, none = rotary_fwd(q, None, pos, rates)
    assert none is None
    want = ref.rotary(q, pos, rates.cpu(), False, 1.0)
    ref.check("q", got.cpu(), want, bound(q, F32, 1.0)(want, sizes(q, 128, False)))


@gpu
def test_small_angles_are_rounded_either_way():
    """The sine of a turn of a few 2^-32 shows how the turn was rounded: to the nearest, half of that step at most."""
    from gated_delta_rule_03_gb300 import rotary_fwd
    rates = torch.tensor([2 ** 33 - 1, 2 ** 32 - 1, 2 ** 33 + 1, 3 * 2 ** 32 - 1, 2 ** 31 - 1, 2 ** 31 + 1, -(2 ** 32) - 1, -1, 1, 12345678901], device="cuda")
    q = torch.zeros(2, 1, 24, device="cuda")
    q[..., :10] = 1
    got, _ = rotary_fwd(q, None, torch.tensor([1, -1], dtype=torch.int32, device="cuda"), rates)
    for sign, y in zip((1, -1), got[:, 0, 10:20].double().cpu()):
        turns = torch.tensor([sign * int(r) / 2.0 ** 64 for r in rates.tolist()], dtype=torch.float64)
        assert bool(((y / (2 * math.pi) - turns).abs() <= 2.0 ** -33 + 2.0 ** -22 * turns.abs()).all())


@gpu
def test_sines_and_cosines_of_fp32_outputs():
    """Pairs (1, 0) become (cos, sin). Those are off by 2 units of CUDA's functions and half of one of the step behind them,
    2^-23 of their size each, and by what the angle is: 2^-33 turns, the square of 2e-7 beside it."""
    from gated_delta_rule_03_gb300 import rotary_fwd
    g = torch.Generator().manual_seed(2)
    rates = torch.randint(-2 ** 63, 2 ** 63 - 1, (100,), generator=g, dtype=torch.int64)
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (300,), generator=g, dtype=torch.int32)
    # and angles around quarter turns, where sine or cosine is small
    rates[:8] = torch.tensor([2 ** 62, 2 ** 62 + 2 ** 35, -(2 ** 62) + 2 ** 36, 2 ** 63 - 2 ** 33, -(2 ** 63), 2 ** 61, 77 * 2 ** 32, -(2 ** 63) + 2 ** 34])
    pos[:3] = torch.tensor([1, -1, 3])
    q = torch.zeros(300, 1, 200)
    q[..., :100] = 1
    got, _ = rotary_fwd(q.cuda(), None, pos.cuda(), rates.cuda())
    want = ref.rotary(q, pos, rates, False, 1.0)
    ref.check("cos, sin", got.cpu(), want, 2.5 * 2.0 ** -23 * want.abs() + 2.0 ** -33 * 2 * math.pi + 2.0 ** -44)


@gpu
def test_the_turn_back_is_the_gradient():
    """Differences of a weighted sum of outputs, which is linear in each input."""
    from gated_delta_rule_03_gb300 import rotary_bwd, rotary_fwd, rotary_rates
    q, k, pos = make(6, 2, 1, 16, F32)
    rates, dq, dk = rotary_rates(12), torch.randn_like(q), torch.randn_like(k)
    gq, gk = rotary_bwd(dq, dk, pos, rates, amplitude=1.3)

    def total(q, k):
        a, b = rotary_fwd(q, k, pos, rates, amplitude=1.3)
        return float((a.double() * dq.double()).sum() + (b.double() * dk.double()).sum())

    for x, g, f in ((q, gq, lambda t: total(t, k)), (k, gk, lambda t: total(q, t))):
        for i in (0, 5, 13, x.numel() - 1):
            up, down = x.clone(), x.clone()
            up.view(-1)[i] += 1
            down.view(-1)[i] -= 1
            assert abs((f(up) - f(down)) / 2 - float(g.view(-1)[i])) < 1e-4  # (200 terms of 2^-22 each, no curvature)


@gpu
def test_another_stream_and_a_graph():
    from gated_delta_rule_03_gb300 import rotary_fwd, rotary_rates
    q, k, pos = make(300, 8, 2, 128, BF16)
    rates = rotary_rates(128)
    want = rotary_fwd(q, k, pos, rates)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = rotary_fwd(q, k, pos, rates, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = rotary_fwd(q, k, pos, rates)
    pos.add_(1)
    graph.replay()
    later = rotary_fwd(q, k, pos, rates)
    for a, b, c, e in zip(want, got, again, later):
        assert torch.equal(a, b) and torch.equal(c, e) and not torch.equal(a, c)


def test_rates_of_stretched_contexts():
    from gated_delta_rule_03_gb300 import rotary_amplitude, rotary_rates
    turns = lambda r: [x % 2 ** 64 / 2.0 ** 64 for x in r.tolist()]  # noqa: E731
    plain = turns(rotary_rates(128, device="cpu"))
    for i, t in enumerate(plain):
        assert math.isclose(t * 2 * math.pi, 10000.0 ** (-i / 64), rel_tol=1e-12)
    assert all(math.isclose(a, b / 4, rel_tol=1e-9) for a, b in zip(turns(rotary_rates(128, factor=4.0, device="cpu")), plain))
    parts = turns(rotary_rates(128, factor=4.0, trained_length=4096, device="cpu"))
    for a, b in zip(parts, plain):
        turned = 4096 * b
        assert math.isclose(a, b, rel_tol=1e-9) if turned >= 32 else math.isclose(a, b / 4, rel_tol=1e-9) if turned <= 1 else b / 4 < a < b
    assert rotary_amplitude(1.0) == 1.0 and math.isclose(rotary_amplitude(8.0), 0.1 * math.log(8) + 1)
    for bad in (dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=4, base=0.0), dict(rot_dim=4, factor=0.0),
                dict(rot_dim=4, trained_length=10, fast_turns=1.0, slow_turns=1.0)):
        with pytest.raises(ValueError):
            rotary_rates(device="cpu", **bad)


def test_rates_are_the_nearest_there_are():
    """By logarithms and a sum of arctangents in 90 decimals: no rate is off by more than half of 2^-64 turns."""
    import decimal
    from gated_delta_rule_03_gb300 import rotary_rates
    with decimal.localcontext(decimal.Context(prec=90)):
        D = decimal.Decimal

        def arctan_of_inverse(n):  # sum of (-1)^k / ((2k + 1) n^(2k + 1))
            return sum(D((-1) ** k) / ((2 * k + 1) * D(n) ** (2 * k + 1)) for k in range(130))

        pi = 16 * arctan_of_inverse(5) - 4 * arctan_of_inverse(239)
        for rot, base, factor in ((128, 10000.0, 1.0), (256, 500000.0, 1.0), (34, 1234.5, 1.0), (64, 1e6, 3.7)):
            for i, r in enumerate(rotary_rates(rot, base=base, factor=factor, device="cpu").tolist()):
                want = (D(base).ln() * D(-2 * i) / rot).exp() / D(factor) / (2 * pi) * 2 ** 64
                assert abs((D(r) - want + 2 ** 63) % 2 ** 64 - 2 ** 63) <= D("0.5000001"), (rot, base, i)
        assert torch.equal(rotary_rates(np.int64(128), base=np.float32(10000), factor=np.float32(4), trained_length=np.int32(4096), device="cpu"),
                           rotary_rates(128, factor=4.0, trained_length=4096.0, device="cpu"))
        for i, r in enumerate(rotary_rates(128, factor=4.0, trained_length=4096, device="cpu").tolist()):
            turns = (D(10000).ln() * D(-2 * i) / 128).exp() / (2 * pi)
            keep = min(D(1), max(D(0), (4096 * turns - 1) / 31))
            want = (turns * keep + turns / 4 * (1 - keep)) * 2 ** 64
            assert abs((D(r) - want + 2 ** 63) % 2 ** 64 - 2 ** 63) <= D("0.5000001"), i


def test_refusals_on_the_host():
    from gated_delta_rule_03_gb300 import ops
    from gated_delta_rule_03_gb300.rotary import RotaryShape
    lib = ops._load()
    A = [0x10000000 * (i + 1) for i in range(6)]
    base = dict(tokens=8, q_heads=4, k_heads=2, d=64, rot_dim=64, dtype=1, neighbours=0, amplitude=1.0,
                q_stride=0, k_stride=0, q_out_stride=0, k_out_stride=0)

    def call(f=lib.gdr_rotary_fwd, q=A[0], k=A[1], pos=A[2], rates=A[3], qo=A[4], ko=A[5], **kw):
        return f(ctypes.byref(RotaryShape(**dict(base, **kw))), q, k, pos, rates, qo, ko, None)

    for f in (lib.gdr_rotary_fwd, lib.gdr_rotary_bwd):
        assert f(None, *A, None) == -1
        for kw in (dict(tokens=-1), dict(q_heads=0), dict(k_heads=-1), dict(amplitude=math.inf), dict(amplitude=math.nan),
                   dict(q=None), dict(ko=None), dict(pos=None), dict(rates=None), dict(q_stride=128), dict(k_heads=0),
                   dict(qo=A[5]), dict(qo=A[1]), dict(ko=A[0]), dict(qo=A[0] + 16), dict(qo=A[2]), dict(ko=A[3]),
                   dict(qo=A[0], q_stride=512), dict(tokens=2 ** 31)):
            assert call(f, **kw) == -1, kw
        for kw in (dict(d=12), dict(d=264), dict(rot_dim=3), dict(rot_dim=66), dict(rot_dim=0), dict(dtype=2)):
            assert call(f, **kw) == -2, kw
        for kw in (dict(q=A[0] + 8), dict(ko=A[5] + 2), dict(pos=A[2] + 2), dict(rates=A[3] + 4), dict(q_stride=260)):
            assert call(f, **kw) == -3, kw
        # views of one buffer: the same stride, and places of a row that meet
        row = dict(q_stride=1024, k_stride=1024, q_out_stride=1024, k_out_stride=1024)
        assert call(f, k=A[0] + 4 * 64 * 2 - 16, qo=A[0], ko=A[5], **row) == -1
        assert call(f, tokens=0) == 0


@gpu
def test_more_heads_than_a_grid_is_high():
    from gated_delta_rule_03_gb300 import rotary_fwd, rotary_rates
    q, k, pos = make(1, 65536, 65536, 16, BF16)
    rates = rotary_rates(16)
    for t, y in zip((q, k), rotary_fwd(q, k, pos, rates)):
        want = ref.rotary(t, pos, rates.cpu(), False, 1.0)
        ref.check("heads", y.cpu(), want, bound(t, BF16, 1.0)(want, sizes(t, 16, False)))
