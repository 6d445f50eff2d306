"""The gradients of the block norms where a block takes many rows one after the other, and
bounds that count the additions as the kernels make them.

Roundings (units of u = 2^-24, first order; ROOM covers the products of two of them):
  ROW   a sum over a row: at most 16 entries per thread in order, 5 steps within the warp, 4
        over the warps
  RS    1 / rms: half of a mean's ROW + 3 (1 / D, the product, eps) and rsqrtf's 2 units in the
        last place, 4 u
  GATE  sigmoid for |g| <= 6: the exponent 12, the exponential 4, 1 + e 1, the quotient 2, and
        the product with g 1
  DGATE its derivative, relative to a sum of absolute values (gate_sizes): twice GATE, 1
A sum over rows adds one row per round in a block, then parts / 32 blocks' sums, then 32. A call
has at least min(rows, 152) rows at work at once, and at most 3648 parts.
"""
import numpy as np
import pytest
import torch

from tests.test_block_norm import BF16, EPS, F32, U, backward, f64, forward, lib, make, rstd, shape  # noqa: F401

gpu = pytest.mark.gpu
u = 2.0 ** -24
ROOM = 1.001
ROW = 16 + 5 + 4
RS = (ROW + 3) / 2 + 4
GATE = 20
DGATE = 2 * GATE + 1


def sum_depth(rows):
    return rows / 152 + 1 + min(rows + 3, 3648) / 32 + 1 + 32


# dx: the mean of dh w x' (ROW + 1, 1 / D and its product 2), r twice and the products (2 RS + 2);
# its two multiply-adds and the weight's product 3, r RS
KX = ROW + 5 + 2 * RS + 3 + RS
# the gradient of t: dx, the scale, the gate and its product
KZ = KX + 1 + GATE + 1
KN = RS + 1  # y / rms(y)


def gate_sizes(kind, g):
    """The absolute terms of act'(g)."""
    s = 1 / (1 + np.exp(-g))
    return np.abs(g * s) + s if kind == "silu" else s if kind == "sigmoid" else np.ones_like(g)


def bounds(want, c, rows, post, kind, gate):
    """{name: what its fp32 arithmetic may be off by}, from `backward`'s sums of absolutes."""
    x, y, g, wp = (f64(c[n]) for n in ("x", "y", "gate", "w_post"))
    s = sum_depth(rows)
    out = {"dx": KX * u * want["dx"][1]}
    if "dw_pre" in want:
        out["dw_pre"] = (KN + 1 + s) * u * want["dw_pre"][1]
    if y is None:
        return out
    if not post:
        out["dy"] = KZ * u * want["dy"][1]
    else:
        # the mean's path again, behind that of dz
        out["dy"] = (KZ + 1 + KX) * u * want["dy"][1]
        out["dw_post"] = (KZ + KN + 1 + s) * u * want["dw_post"][1]
    if g is not None:
        size = want["dx"][1] * abs(c["s"]) * np.abs(y * (rstd(y) if post else 1) * (1 if wp is None else wp)) * gate_sizes(kind, g)
        if gate == "one":
            out["dgate"] = (KX + 1 + KN + 3 + DGATE + s) * u * size.sum(0)
        else:
            out["dgate"] = (KX + 1 + KN + 3 + DGATE) * u * size
    return out


def check_forward(rows, D, dt, xdt, gate, kind, post, pre, s, seed=12):
    from gated_delta_rule_03_gb300 import block_norm_fwd
    c = make(rows, D, dt, xdt, gate, post, pre, seed=seed)
    got_x, got_h = block_norm_fwd(c["x"], c["y"], gate=c["gate"], act=kind, w_post=c["w_post"], w_pre=c["w_pre"],
                                  post_norm=post != "no", pre_norm=pre != "no", res_scale=s, eps=EPS)
    x, y, g, wp, wn = (f64(c[n]) for n in ("x", "y", "gate", "w_post", "w_pre"))
    want_x, want_h = forward(x, y, g, wp, wn, post != "no", pre != "no", kind, s)
    # x + (y act) (r s) w: the gate, r, three products; the addition
    may = u * ((GATE + RS + 3) * np.abs(want_x - x) + np.abs(want_x))
    compare("x", got_x, want_x, may, xdt)
    if pre == "no":
        assert got_h is None
        return
    # x' w r: what x' is off by, itself and in its mean square; r and two products
    r = rstd(want_x)
    shift = np.sqrt((may * may).mean(-1, keepdims=True)) * r
    may = may * r * (1 if wn is None else np.abs(wn)) + np.abs(want_h) * (shift + (RS + 2) * u)
    compare("h", got_h, want_h, may, dt)


def compare(name, got, want, may, dtype):
    got = f64(got)
    assert got.shape == want.shape, name
    assert np.isfinite(got).all(), f"{name}: not finite"
    may = ROOM * (U[dtype] * (np.abs(want) + may) + may) + 1e-30
    worst = float((np.abs(got - want) / may).max())
    assert worst <= 1.0, f"{name}: {worst:.3g} of what is allowed"


def check_backward(rows, D, dt, xdt, gate, kind, post, pre, s, repeats, first=False, seed=11):
    from gated_delta_rule_03_gb300 import block_norm_bwd
    c = make(rows, D, dt, xdt, gate, post, pre, seed=seed)
    c["s"] = s
    if first:
        c["y"] = c["gate"] = None
    kw = dict(gate=c["gate"], act=kind, w_post=c["w_post"], w_pre=c["w_pre"], post_norm=post != "no",
              pre_norm=pre != "no", res_scale=s, eps=EPS)
    names = ("dx", "dy", "dgate", "dw_post", "dw_pre")
    call = lambda: dict(zip(names, block_norm_bwd(c["dx_out"], c["dh"], c["x"], c["y"], **kw)))  # noqa: E731
    got = call()
    for _ in range(repeats):
        again = call()
        for n in names:
            assert got[n] is None or torch.equal(got[n], again[n]), f"{n}: other bits another time"
    want = backward(*(f64(c[n]) for n in ("dx_out", "dh", "x", "y", "gate", "w_post", "w_pre")),
                    post != "no", pre != "no", kind, s)
    may = bounds(want, c, rows, post != "no", kind, gate)
    for n in names:
        if got[n] is None:
            continue
        w = want[n][0].sum(0) if n == "dgate" and gate == "one" else want[n][0]
        compare(n, got[n], w, may[n], F32 if n.startswith("dw") else xdt if n == "dx" else dt)


# several rows per block and more than one warp per row: the sums of consecutive rows of a
# block meet in the same shared memory
ROUNDS = [(514, 5000), (1030, 3100), (2048, 2300), (4096, 900), (8192, 900)]
TYPES = [(F32, F32), (BF16, BF16), (BF16, F32)]
TYPE_IDS = ["fp32", "bf16", "bf16 on fp32"]


@gpu
@pytest.mark.parametrize("dt,xdt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("D,rows", ROUNDS)
def test_many_rows_without_the_norm_after_the_block(D, rows, dt, xdt):
    check_backward(rows, D, dt, xdt, "rows", "silu", "no", "weight", 0.5, repeats=20)


@gpu
@pytest.mark.parametrize("dt,xdt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("D,rows", ROUNDS)
def test_many_rows_of_the_first_block(D, rows, dt, xdt):
    check_backward(rows, D, dt, xdt, "none", "silu", "no", "weight", 1.0, repeats=20, first=True)


@gpu
@pytest.mark.parametrize("dt,xdt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("D", [6096, 6097, 6120, 6143, 6144, 6145])
def test_widths_whose_column_sums_take_just_48_kb(D, dt, xdt):
    # (what a kernel has without asking for more, its own buffer among it)
    check_backward(155, D, dt, xdt, "one", "silu", "weight", "weight", 1.0, repeats=1)


# rows, D, type, stream's type, gate, act, norm after, norm before, scale: wide rows, each access
# width (eights, pairs, single entries) below and above the 4096 columns where the forms change
WIDE = [
    (700, 8192, F32, F32, "rows", "silu", "weight", "weight", 1.0),
    (330, 8190, F32, F32, "one", "sigmoid", "weight", "weight", 0.5),
    (160, 8191, F32, F32, "one", "silu", "weight", "ones", 1.0),
    (400, 5120, BF16, F32, "rows", "silu", "weight", "weight", -1.0),
    (170, 7168, BF16, BF16, "one", "silu", "ones", "weight", 1.0),
    (200, 4100, BF16, F32, "none", "silu", "weight", "no", 1.0),
    (333, 6143, BF16, BF16, "rows", "identity", "no", "weight", 0.25),
    (1100, 4096, F32, F32, "one", "silu", "weight", "weight", 0.5),
    (900, 2048, F32, F32, "rows", "silu", "weight", "weight", 1.0),
    (1500, 1536, F32, F32, "rows", "sigmoid", "weight", "weight", 1.0),
    (2000, 1024, BF16, F32, "one", "identity", "weight", "weight", 1.0),
    (1300, 1030, F32, F32, "rows", "silu", "weight", "weight", 0.25),
    (900, 1999, F32, F32, "none", "silu", "weight", "weight", 1.0),
    (5000, 136, F32, F32, "one", "silu", "weight", "weight", 1.0),
]


@gpu
@pytest.mark.parametrize("case", WIDE, ids=[f"{c[0]}x{c[1]}" for c in WIDE])
def test_forward_rounds_as_often_as_its_sums_are_deep(case):
    check_forward(*case)


@gpu
@pytest.mark.parametrize("case", WIDE, ids=[f"{c[0]}x{c[1]}" for c in WIDE])
def test_gradients_round_as_often_as_their_sums_are_deep(case):
    check_backward(*case, repeats=2)


# ------------------------------------------------------------------ without a GPU

@pytest.mark.parametrize("D", [8, 104, 256, 512, 768, 1024, 1280, 1536, 1792, 2048, 2056, 4096])
@pytest.mark.parametrize("dtype,x_dtype", [(0, 0), (1, 1), (1, 0)], ids=TYPE_IDS)
def test_the_blocks_of_a_backward_call_fit_the_gpu_at_once(lib, dtype, x_dtype, D):  # noqa: F811
    # widths in eights up to 4096: two rows' five inputs in shared memory, 8 entries a thread
    threads = (D + 255) // 256 * 32
    rows_at_once = 1 if threads >= 128 else 128 // threads
    threads *= rows_at_once
    size = {0: 4, 1: 2}
    block = 2 * 8 * (2 * size[x_dtype] + 3 * size[dtype]) * threads + 96 * 4 + 1024  # (1 KB each is the system's)
    held = lib.gdr_block_norm_bwd_workspace_size(shape(rows=1 << 20, D=D, dtype=dtype, x_dtype=x_dtype, gate_rows=0)) - 256
    blocks, left = divmod(held, 3 * D * 4 * rows_at_once)
    assert left == 0 and blocks % 152 == 0
    per_sm = blocks // 152
    assert per_sm * block <= 228 * 1024 and per_sm * threads <= 768
    # and as many as fit: one block more would be too much for either
    assert (per_sm + 1) * block > 228 * 1024 or (per_sm + 1) * threads > 768 or threads > 256
