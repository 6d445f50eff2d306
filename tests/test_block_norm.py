"""The norms before and after a block with gate and residual scale, against 64 bits."""
import ctypes
import math

import numpy as np
import pytest
import torch

from tests.helpers import check_guards, poisoned

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
U = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
EPS = 1e-6


def act(kind, g):
    sig = 1 / (1 + np.exp(-g))
    if kind == "identity":
        return g, np.ones_like(g)
    return (sig, sig * (1 - sig)) if kind == "sigmoid" else (g * sig, sig * (1 + g * (1 - sig)))


def rstd(a, eps=EPS):
    return 1 / np.sqrt((a * a).mean(-1, keepdims=True) + eps)


def forward(x, y, g, wp, wn, post, pre, kind, s, eps=EPS):
    """(x', h) in float64 numpy; h None without the second norm."""
    if y is not None:
        t = y * rstd(y, eps) * (1 if wp is None else wp) if post else y
        if g is not None:
            t = t * act(kind, g)[0]
        x = x + s * t
    return x, (x * rstd(x, eps) * (1 if wn is None else wn) if pre else None)


def backward(dx_out, dh, x, y, g, wp, wn, post, pre, kind, s, eps=EPS):
    """{name: (gradient, sum of the absolute values of its terms)}."""
    a, out = np.abs, {}
    dx, dxa = (0 * x, 0 * x) if dx_out is None else (dx_out, a(dx_out))
    if pre:
        r = rstd(x, eps)
        n, m = x * r, dh * (1 if wn is None else wn)
        out["dw_pre"] = ((dh * n).sum(0), a(dh * n).sum(0))
        dx = dx + r * (m - n * (m * n).mean(-1, keepdims=True))
        dxa = dxa + r * (a(m) + a(n) * a(m * n).mean(-1, keepdims=True))
    out["dx"] = (dx, dxa)
    if y is None:
        return out
    dz, dza = s * dx, abs(s) * dxa
    r = rstd(y, eps) if post else np.ones((len(y), 1))
    n, w = y * r, (1 if wp is None or not post else wp)
    if g is not None:
        f, df = act(kind, g)
        out["dgate"] = (dz * n * w * df, dza * a(n * w * df))
        dz, dza = dz * f, dza * a(f)
    if not post:
        out["dy"] = (dz, dza)
        return out
    out["dw_post"] = ((dz * n).sum(0), (dza * a(n)).sum(0))
    m, ma = dz * w, dza * a(w)
    out["dy"] = (r * (m - n * (m * n).mean(-1, keepdims=True)), r * (ma + a(n) * (ma * a(n)).mean(-1, keepdims=True)))
    return out


def f64(t):
    return None if t is None else t.detach().to("cpu", torch.float64).numpy()


def terms(D, rows=0):
    """Roundings of 2^-24 that a term meets at most: a mean of D entries (twice, one norm
    feeding the other), the sum over rows, the gate's exponential and quotient (16), the
    products (16)."""
    return 2 * D + rows + 32


def check(name, got, want, Abs, dtype, n):
    got = f64(got)
    assert got.shape == want.shape, name
    assert np.isfinite(got).all(), f"{name}: not finite"
    # the result's own rounding, and the fp32 roundings of its terms
    may = U[dtype] * np.abs(want) * (1 + 1e-3) + n * U[F32] * Abs + 1e-30
    worst = float((np.abs(got - want) / may).max()) if got.size else 0.0
    assert worst <= 1.0, f"{name}: {worst:.3g} of what is allowed"


def make(rows, D, dtype, x_dtype, gate, post, pre, seed=0, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    new = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    c = dict(x=new(rows, D).to(x_dtype), y=new(rows, D).to(dtype), dx_out=new(rows, D).to(x_dtype),
             dh=new(rows, D).to(dtype) if pre != "no" else None,
             gate=None if gate == "none" else new(*((rows, D) if gate == "rows" else (D,))).to(dtype),
             w_post=1 + 0.2 * new(D) if post == "weight" else None,
             w_pre=1 + 0.2 * new(D) if pre == "weight" else None)
    return {k: None if t is None else t.to(device) for k, t in c.items()}


# rows, D, type, stream's type, gate, act, norm after, norm before, scale
CASES = [
    (1, 1, F32, F32, "rows", "silu", "weight", "weight", 1.0),
    (1, 128, BF16, BF16, "rows", "silu", "weight", "weight", 1.0),
    (3, 7, BF16, BF16, "one", "sigmoid", "weight", "weight", 0.5),
    (5, 2048, BF16, BF16, "rows", "silu", "weight", "weight", 1.0),
    (700, 2048, BF16, F32, "one", "identity", "ones", "ones", 0.22),
    (33, 1030, F32, F32, "one", "identity", "weight", "weight", 0.25),
    (40, 4096, BF16, BF16, "rows", "sigmoid", "weight", "weight", 0.5),
    (9, 4104, BF16, F32, "rows", "silu", "weight", "weight", -1.0),
    (17, 8191, F32, F32, "rows", "sigmoid", "weight", "weight", 1.0),
    (300, 8192, BF16, BF16, "one", "silu", "weight", "weight", 1.0),
    (6, 514, BF16, BF16, "none", "silu", "weight", "no", 1.0),
    (1000, 96, BF16, BF16, "rows", "silu", "no", "weight", 1.0),
    (257, 255, F32, F32, "none", "silu", "no", "no", 0.5),
    (2, 8, BF16, BF16, "one", "sigmoid", "no", "ones", 0.0),
]
IDS = [str(i) for i in range(len(CASES))]


@gpu
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(case):
    from gated_delta_rule_03_gb300 import block_norm_fwd
    rows, D, dt, xdt, gate, kind, post, pre, s = case
    c = make(rows, D, dt, xdt, gate, post, pre, seed=1)
    x_out, g1 = poisoned((rows, D), xdt, "cuda")
    h, g2 = poisoned((rows, D), dt, "cuda")
    block_norm_fwd(c["x"], c["y"], gate=c["gate"], act=kind, w_post=c["w_post"], w_pre=c["w_pre"],
                   post_norm=post != "no", pre_norm=pre != "no", res_scale=s, eps=EPS, x_out=x_out,
                   h=None if pre == "no" else h)
    check_guards([g1, g2])
    x, y, g, wp, wn = (f64(c[n]) for n in ("x", "y", "gate", "w_post", "w_pre"))
    want_x, want_h = forward(x, y, g, wp, wn, post != "no", pre != "no", kind, s)
    size = np.abs(x) + np.abs(want_x - x)
    check("x", x_out, want_x, size, xdt, terms(D))
    if pre != "no":
        w = 1 if wn is None else np.abs(wn)
        check("h", h, want_h, size * rstd(want_x) * w + np.abs(want_h), dt, terms(D))
    else:
        assert bool(torch.isnan(h).all())


@gpu
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(case):
    from gated_delta_rule_03_gb300 import block_norm_bwd
    rows, D, dt, xdt, gate, kind, post, pre, s = case
    c = make(rows, D, dt, xdt, gate, post, pre, seed=2)
    outs = dict(dx=poisoned((rows, D), xdt, "cuda"), dy=poisoned((rows, D), dt, "cuda"))
    if c["gate"] is not None:
        outs["dgate"] = poisoned(tuple(c["gate"].shape), dt, "cuda")
    for n in ("w_post", "w_pre"):
        if c[n] is not None:
            outs["d" + n] = poisoned((D,), F32, "cuda")
    kw = dict(gate=c["gate"], act=kind, w_post=c["w_post"], w_pre=c["w_pre"], post_norm=post != "no",
              pre_norm=pre != "no", res_scale=s, eps=EPS)
    block_norm_bwd(c["dx_out"], c["dh"], c["x"], c["y"], **kw, **{n: t for n, (t, _) in outs.items()})
    check_guards([g for _, g in outs.values()])
    want = backward(*(f64(c[n]) for n in ("dx_out", "dh", "x", "y", "gate", "w_post", "w_pre")),
                    post != "no", pre != "no", kind, s)
    for name, (t, _) in outs.items():
        w, size = want[name]
        if name == "dgate" and gate == "one":
            w, size = w.sum(0), size.sum(0)
        dtype = F32 if name.startswith("dw") else xdt if name == "dx" else dt
        check(name, t, w, size, dtype, terms(D, rows))
    again = block_norm_bwd(c["dx_out"], c["dh"], c["x"], c["y"], **kw)
    for name, t in zip(("dx", "dy", "dgate", "dw_post", "dw_pre"), again):
        if t is not None:
            assert torch.equal(t, outs[name][0]), f"{name}: other bits the second time"


@gpu
def test_the_first_block_has_only_the_norm_before_it():
    from gated_delta_rule_03_gb300 import block_norm_bwd, block_norm_fwd
    c = make(19, 1000, BF16, F32, "none", "no", "weight", seed=3)
    x_same, h = block_norm_fwd(c["x"], w_pre=c["w_pre"], dtype=BF16)
    assert x_same is c["x"] and h.dtype == BF16
    x, wn = f64(c["x"]), f64(c["w_pre"])
    want = forward(x, None, None, None, wn, False, True, "silu", 1.0)[1]
    check("h", h, want, 2 * np.abs(want), BF16, terms(1000))
    for d in (c["dx_out"], None):
        dx, dy, dg, dwp, dwn = block_norm_bwd(d, c["dh"], c["x"], w_pre=c["w_pre"])
        assert dy is None and dg is None and dwp is None
        ref = backward(f64(d), f64(c["dh"]), x, None, None, None, wn, False, True, "silu", 1.0)
        check("dx", dx, *ref["dx"], F32, terms(1000))
        check("dw_pre", dwn, *ref["dw_pre"], F32, terms(1000, 19))


@gpu
def test_in_place_zero_rows_and_rows_of_zeros():
    from gated_delta_rule_03_gb300 import block_norm_bwd, block_norm_fwd
    c = make(50, 768, BF16, BF16, "one", "weight", "weight", seed=4)
    want = block_norm_fwd(c["x"], c["y"], gate=c["gate"], w_post=c["w_post"], w_pre=c["w_pre"])
    x = c["x"].clone()
    got = block_norm_fwd(x, c["y"], gate=c["gate"], w_post=c["w_post"], w_pre=c["w_pre"], x_out=x)
    assert got[0] is x and torch.equal(x, want[0]) and torch.equal(got[1], want[1])
    args = (c["dh"], want[0], c["y"], c["gate"], "silu", c["w_post"], c["w_pre"])
    ref = block_norm_bwd(c["dx_out"], *args)
    d = c["dx_out"].clone()
    out = block_norm_bwd(d, *args, dx=d)
    assert out[0] is d and all(torch.equal(a, b) for a, b in zip(out, ref))
    # no rows: the sums over rows are zero
    e = c["x"][:0]
    assert block_norm_fwd(e, e, gate=c["gate"], w_post=c["w_post"], w_pre=c["w_pre"])[1].shape == (0, 768)
    _, _, dg, dwp, dwn = block_norm_bwd(e, e, e, e, c["gate"], "silu", c["w_post"], c["w_pre"])
    assert not dg.any() and not dwp.any() and not dwn.any()
    # rows of zeros: eps alone under the root
    z = torch.zeros(4, 768, dtype=BF16, device="cuda")
    x2, h2 = block_norm_fwd(z, z, w_post=c["w_post"], w_pre=c["w_pre"])
    assert not x2.any() and not h2.any()


@gpu
def test_a_row_that_is_not_finite_stays_alone():
    from gated_delta_rule_03_gb300 import block_norm_fwd
    c = make(12, 512, BF16, BF16, "rows", "weight", "weight", seed=5)
    clean = block_norm_fwd(c["x"], c["y"], gate=c["gate"], w_post=c["w_post"], w_pre=c["w_pre"])
    c["y"][5, 3], c["x"][7, 0], c["gate"][9, 1] = math.nan, math.inf, math.nan
    out = block_norm_fwd(c["x"], c["y"], gate=c["gate"], w_post=c["w_post"], w_pre=c["w_pre"])
    keep = [i for i in range(12) if i not in (5, 7, 9)]
    for a, b in zip(clean, out):
        assert torch.equal(a[keep], b[keep])
    assert bool(torch.isnan(out[1][[5, 9]]).all())


@gpu
def test_captured_and_replayed_and_on_another_stream():
    from gated_delta_rule_03_gb300 import block_norm_bwd, block_norm_fwd
    c = make(333, 1030, BF16, F32, "one", "weight", "weight", seed=6)
    kw = dict(gate=c["gate"], w_post=c["w_post"], w_pre=c["w_pre"])
    f = lambda: [*block_norm_fwd(c["x"], c["y"], **kw), *block_norm_bwd(c["dx_out"], c["dh"], c["x"], c["y"], **kw)]  # noqa: E731
    first = f()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = f()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        third = f()
    for t in third:
        t.fill_(math.nan)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, d) for a, b, d in zip(first, second, third))


# ------------------------------------------------------------------ without a GPU

def test_the_gradients_are_differences():
    rng = np.random.default_rng(0)
    rows, D = 2, 5
    x, y, g, dx_out, dh = rng.standard_normal((5, rows, D))
    wp, wn = 1 + 0.1 * rng.standard_normal((2, D))
    for kind in ("identity", "silu", "sigmoid"):
        for post, pre in ((True, True), (False, True), (True, False)):
            def loss(x, y, g, wp, wn):
                a, h = forward(x, y, g, wp, wn, post, pre, kind, 0.7)
                return (a * dx_out).sum() + ((h * dh).sum() if pre else 0.0)
            total = forward(x, y, g, wp, wn, post, pre, kind, 0.7)[0]
            grads = backward(dx_out, dh, total, y, g, wp, wn, post, pre, kind, 0.7)
            point = [x, y, g, wp, wn]
            for i, name in enumerate(("dx", "dy", "dgate", "dw_post", "dw_pre")):
                if name not in grads:
                    continue
                for at in np.ndindex(point[i].shape):
                    lo, hi = [[p.copy() for p in point] for _ in range(2)]
                    lo[i][at] -= 1e-5
                    hi[i][at] += 1e-5
                    diff = (loss(*hi) - loss(*lo)) / 2e-5
                    assert abs(diff - grads[name][0][at]) < 1e-7, (kind, name)


@pytest.fixture(scope="module")
def lib():
    import os
    from gated_delta_rule_03_gb300 import build, ops
    if not os.path.exists(ops.library_path()):
        build.build()
    return ops._load()


def shape(**kw):
    from gated_delta_rule_03_gb300.block_norm import BlockNormShape
    base = dict(rows=16, D=256, dtype=1, x_dtype=1, post_norm=1, pre_norm=1, gate_act=1, gate_rows=16,
                res_scale=1.0, eps=0.0)
    return ctypes.byref(BlockNormShape(**dict(base, **kw)))


def fake(i):
    return 0x10000 + i * 0x100000000


BAD = [(dict(rows=-1), -1), (dict(D=0), -1), (dict(D=8193), -2), (dict(dtype=3), -2), (dict(x_dtype=2), -2),
       (dict(dtype=0), -2), (dict(gate_act=3), -2), (dict(gate_act=-1), -2), (dict(gate_rows=2), -1),
       (dict(eps=-1.0), -1), (dict(eps=math.nan), -1), (dict(res_scale=math.inf), -1), (dict(gate_rows=0), -1)]


@pytest.mark.parametrize("kw,status", BAD)
def test_bad_shapes_are_refused(lib, kw, status):
    s = shape(**kw)
    assert lib.gdr_block_norm_fwd(s, *(fake(i) for i in range(7)), None) == status
    assert lib.gdr_block_norm_bwd(s, *(fake(i) for i in range(13)), 1 << 30, None) == status
    if kw != dict(gate_rows=0):
        assert lib.gdr_block_norm_bwd_workspace_size(s) == 0


@pytest.mark.parametrize("kw,i,p,status", [
    ({}, 0, None, -1), ({}, 1, None, -1), ({}, 2, None, -1), ({}, 5, None, -1), ({}, 6, None, -1),
    (dict(post_norm=0), 0, fake(0), -1), (dict(pre_norm=0), 0, fake(0), -1), ({}, 5, fake(6), -1),
    ({}, 5, fake(0) + 16, -1), ({}, 6, fake(0), -1), ({}, 6, fake(1), -1), ({}, 5, fake(2), -1),
    ({}, 5, fake(3), -1), ({}, 0, fake(0) + 8, -3), ({}, 4, fake(4) + 4, -3)])
def test_bad_arguments_of_the_forward_call_are_refused(lib, kw, i, p, status):
    a = [fake(j) for j in range(7)]
    a[i] = p
    assert lib.gdr_block_norm_fwd(shape(**kw), *a, None) == status


@pytest.mark.parametrize("kw,i,p,status", [
    ({}, 1, None, -1), ({}, 2, None, -1), ({}, 3, None, -1), ({}, 4, None, -1), ({}, 7, None, -1), ({}, 8, None, -1),
    (dict(post_norm=0), 0, fake(0), -1), (dict(pre_norm=0), 0, fake(0), -1), ({}, 12, None, -4),
    ({}, 7, fake(1), -1), ({}, 7, fake(0) + 32, -1), ({}, 8, fake(3), -1), ({}, 9, fake(8), -1), ({}, 10, fake(5), -1),
    ({}, 11, fake(10), -1), ({}, 12, fake(9), -1), ({}, 11, fake(11) + 4, -3)])
def test_bad_arguments_of_the_backward_call_are_refused(lib, kw, i, p, status):
    a = [fake(j) for j in range(13)]
    a[i] = p
    assert lib.gdr_block_norm_bwd(shape(**kw), *a, 1 << 30, None) == status
    small = lib.gdr_block_norm_bwd_workspace_size(shape()) - 1
    assert lib.gdr_block_norm_bwd(shape(), *(fake(j) for j in range(13)), small, None) == -4


@gpu
def test_the_binding_checks_shapes_and_types():
    from gated_delta_rule_03_gb300 import block_norm_bwd, block_norm_fwd
    c = make(4, 64, BF16, BF16, "rows", "weight", "weight")
    x, y, g = c["x"], c["y"], c["gate"]
    for kw in (dict(act="relu"), dict(gate=g[:2]), dict(w_post=c["w_post"][:32]), dict(post_norm=False, w_post=c["w_post"]),
               dict(x_out=x[:2]), dict(pre_norm=False, h=torch.empty_like(x))):
        with pytest.raises(ValueError):
            block_norm_fwd(x, y, **kw)
    with pytest.raises(ValueError):
        block_norm_fwd(x.t(), y.t())
    with pytest.raises(TypeError):
        block_norm_fwd(x, y, gate=g.float())
    with pytest.raises(TypeError):
        block_norm_fwd(x, y, w_post=c["w_post"].double())
    with pytest.raises(ValueError):
        block_norm_bwd(c["dx_out"], None, x, y)
    with pytest.raises(ValueError):
        block_norm_bwd(c["dx_out"], c["dh"], x, y, dgate=torch.empty_like(g))
    # leading shapes of any rank
    a = block_norm_fwd(x, y, gate=g)
    b = block_norm_fwd(x.view(2, 2, 64), y.view(2, 2, 64), gate=g.view(2, 2, 64))
    assert all(torch.equal(u, v.view(4, 64)) for u, v in zip(a, b))
