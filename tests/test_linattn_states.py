"""The fp32 states that linear attention hands out from bf16 inputs are as exact as fp32 arithmetic.

In norm a state may be off by 2^-20 of itself, 16 roundings of 2^-24: a term k_t v_t^T meets its
weight (|n ln lam| + 4 of them where the weight is e^(n ln lam): 4 at most) and its product with it
(1), the sums of a chunk in the tensor cores and one addition per chunk, at random signs. Terms of
16 bits, 2^-17 each, would leave it off by 4e-6.
"""
import numpy as np
import pytest
import torch

from tests import linattn_ref as ref
from tests.test_linattn import BF16, make

gpu = pytest.mark.gpu
MAY = 2.0 ** -20


def decayed_sums(x, z, ld, spans, start, scale, backward):
    """Per sequence and head the last state of S <- lam S + scale x z^T from `start`, from the first
    token to the last, or (backward) of D <- lam (D + scale x z^T) from the last to the first."""
    H = len(ld)
    out = np.zeros((len(spans), H, x.shape[2], z.shape[2]))
    for n, (a, b) in enumerate(spans):
        for h in range(H):
            t = np.arange(b - a)
            w = ref.powers(ld[h], t + 1 if backward else b - a - 1 - t)[:, None]
            out[n, h] = scale * (w * x[a:b, h * x.shape[1] // H]).T @ z[a:b, h * z.shape[1] // H]
            if start is not None:
                out[n, h] += ref.powers(ld[h], b - a) * start[n, h]
    return out


def check(name, got, want):
    off = np.linalg.norm(ref.f64(got) - want, axis=(2, 3))
    size = np.linalg.norm(want, axis=(2, 3))
    worst = float((off / np.maximum(size, 1e-30)).max())
    assert worst <= MAY, f"{name}: off by {worst:.3g} in norm"


# lens, H, q heads, k heads, v heads, dk, dv, decay, states given, equal lengths: one chunk and its
# parts, whole sequences, cut ones with sums in parts, both numbers of columns
CASES = [
    ([1], 2, 2, 2, 2, 128, 128, "retention", True, True),
    ([128], 2, 2, 2, 2, 128, 128, "retention", False, True),
    ([129, 255, 0, 64], 4, 4, 2, 2, 64, 64, "slopes", True, False),
    ([1000, 1000], 8, 8, 8, 8, 128, 256, "retention", False, True),
    ([4096] * 4, 16, 16, 16, 16, 128, 128, "retention", False, True),
    ([9000], 2, 1, 2, 2, 64, 128, "none", True, True),
    ([9000], 2, 2, 2, 2, 128, 64, "strong", True, True),
    ([30000], 3, 3, 3, 3, 128, 128, "retention", True, True),
    ([5000, 300, 77, 2000], 8, 8, 4, 4, 128, 128, "slopes", True, False),
    ([300, 900], 4, 4, 4, 4, 128, 128, "ends", False, False),
    ([1, 17, 3, 129], 4, 4, 4, 4, 128, 128, "strong", True, False),
]


@gpu
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_states_from_bf16_inputs(case):
    from gated_delta_rule_03_gb300 import linattn_bwd, linattn_fwd
    lens, H, qh, kh, vh, dk, dv, kind, given, equal = case
    c = make(lens, H, qh, kh, vh, dk, dv, BF16, kind, s0=given, seed=21)
    c["scale"] = dk ** -0.5
    kw = dict(num_seqs=len(lens)) if equal else dict(cu_seqlens=c["cu"])
    args = (c["q"], c["k"], c["v"], c["ld"])
    S = linattn_fwd(*args, S0=c["S0"], scale=c["scale"], **kw)[1]
    q, k, v, do, ld, S0, dS = (ref.f64(c[n]) for n in ("q", "k", "v", "do", "ld", "S0", "dS"))
    spans = ref.spans(lens)
    check("S_final", S, decayed_sums(k, v, ld, spans, S0, 1.0, False))
    dS0 = torch.empty_like(S)
    linattn_bwd(c["do"], *args, S0=c["S0"], dS_final=c["dS"], scale=c["scale"], dS0=dS0, **kw)
    check("dS0", dS0, decayed_sums(q, do, ld, spans, dS, c["scale"], True))


@gpu
def test_outputs_do_not_depend_on_whether_the_state_goes_out():
    """Both forms of the kernel, with and without the state, within the rounding of bf16 outputs."""
    from gated_delta_rule_03_gb300 import linattn_bwd, linattn_fwd
    c = make([2500, 100, 900], 4, 4, 2, 2, 128, 128, BF16, "slopes", s0=True, seed=22)
    args = (c["q"], c["k"], c["v"], c["ld"])
    with_state, _ = linattn_fwd(*args, S0=c["S0"], cu_seqlens=c["cu"])
    without, none = linattn_fwd(*args, S0=c["S0"], cu_seqlens=c["cu"], final_state=False)
    assert none is None
    q, k, v, S0, ld = (ref.f64(c[n]) for n in ("q", "k", "v", "S0", "ld"))
    want, _, size, _ = ref.forward(q, k, v, ld, c["lens"], S0)
    for o in (with_state, without):
        ref.check("o", o, want, size, BF16, ref.f32_terms(2500, 128, 128))
    grads = linattn_bwd(c["do"], *args, dS_final=c["dS"], cu_seqlens=c["cu"])
    want = ref.backward(ref.f64(c["do"]), q, k, v, ld, c["lens"], None, ref.f64(c["dS"]))
    assert grads[3] is None
    for name, g in zip(("dq", "dk", "dv"), grads):
        ref.check(name, g, *want[name], BF16, ref.f32_terms(2500, 128, 128, 4))


def test_the_sums_of_this_file_are_the_definition():
    c = make([7, 0, 5], 2, 2, 1, 2, 64, 64, BF16, "slopes", s0=True, device="cpu")
    q, k, v, do, ld, S0, dS = (ref.f64(c[n]) for n in ("q", "k", "v", "do", "ld", "S0", "dS"))
    spans = ref.spans(c["lens"])
    S = ref.forward(q, k, v, ld, c["lens"], S0, 0.5)[1]
    assert np.allclose(decayed_sums(k, v, ld, spans, S0, 1.0, False), S, atol=1e-12)
    dS0 = ref.backward(do, q, k, v, ld, c["lens"], S0, dS, 0.5)["dS0"][0]
    assert np.allclose(decayed_sums(q, do, ld, spans, dS, 0.5, True), dS0, atol=1e-12)
