"""Linear attention with a constant decay per head against its definition in 64 bits."""
import ctypes
import math

import numpy as np
import pytest
import torch

from tests import linattn_ref as ref
from tests.helpers import check_guards, poisoned

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def decays(H, kind):
    h = np.arange(H)
    ld = {"retention": np.log1p(-2.0 ** -(5 + 7 * h / max(1, H - 1))),
          "slopes": -2.0 ** (-8 * (h + 1) / H),
          "none": np.zeros(H),
          "strong": -3.0 * (h + 1),
          "ends": np.where(h % 2 == 0, -np.inf, 0.0)}[kind]
    return torch.tensor(ld, dtype=F32)


def make(lens, H, qh, kh, vh, dk, dv, dtype, kind="retention", s0=False, fused=False, behind=0,
         seed=0, device="cuda"):
    """Inputs of a call; `behind` rows of NaN follow the last sequence."""
    g = torch.Generator().manual_seed(seed)
    T = sum(lens) + behind
    rows = lambda heads, d: torch.randn(T, heads, d, generator=g)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True).clamp_min(1e-9)  # noqa: E731
    q, k, v = unit(rows(qh, dk)), unit(rows(kh, dk)), rows(vh, dv)
    do = rows(H, dv)
    if behind:
        for t in (q, k, v, do):
            t[sum(lens):] = math.nan
    q, k, v, do = (t.to(dtype).to(device) for t in (q, k, v, do))
    if fused:
        w = torch.cat([q.flatten(1), k.flatten(1), v.flatten(1)], 1).contiguous()
        a, b = qh * dk, (qh + kh) * dk
        q, k, v = w[:, :a].view(T, qh, dk), w[:, a:b].view(T, kh, dk), w[:, b:].view(T, vh, dv)
    state = lambda: (0.5 * torch.randn(len(lens), H, dk, dv, generator=g)).to(device)  # noqa: E731
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=device)
    return dict(q=q, k=k, v=v, do=do, ld=decays(H, kind).to(device), S0=state() if s0 else None,
                dS=state() if s0 else None, cu=cu, lens=lens, H=H, dk=dk, dv=dv, dtype=dtype,
                scale=dk ** -0.5 if fused else 1.0)


def run_fwd(c, cu="packed", **kw):
    from gated_delta_rule_03_gb300 import linattn_fwd
    n = len(c["lens"])
    o, g1 = poisoned((c["q"].shape[0], c["H"], c["dv"]), c["dtype"], "cuda")
    S, g2 = poisoned((n, c["H"], c["dk"], c["dv"]), F32, "cuda")
    linattn_fwd(c["q"], c["k"], c["v"], c["ld"], S0=c["S0"], cu_seqlens=c["cu"] if cu == "packed" else None,
                num_seqs=n, scale=c["scale"], o=o, S_final=S, **kw)
    check_guards([g1, g2])
    return o, S


def check_fwd(c, o, S):
    T = sum(c["lens"])
    q, k, v, S0 = (ref.f64(c[n]) for n in ("q", "k", "v", "S0"))
    ld = ref.f64(c["ld"])
    want_o, want_S, abs_o, abs_S = ref.forward(q[:T], k[:T], v[:T], ld, c["lens"], S0, c["scale"])
    terms = ref.f32_terms(max(c["lens"]), c["dk"], c["dv"])
    ref.check("o", o[:T], want_o, abs_o, c["dtype"], terms)
    ref.check("S_final", S, want_S, abs_S, F32, terms)
    assert bool(torch.isnan(o[T:]).all()), "rows behind the last sequence were written"


# lens, H, q heads, k heads, v heads, dk, dv, decay, S0, fused views, rows behind
CASES = [
    ([1], 1, 1, 1, 1, 128, 128, "retention", False, False, 0),
    ([0], 2, 2, 2, 2, 128, 128, "retention", True, False, 0),
    ([0, 5, 0, 0], 2, 2, 2, 2, 64, 64, "retention", True, False, 3),
    ([127, 1, 0, 128, 129], 4, 4, 2, 1, 128, 128, "slopes", True, True, 7),
    ([63, 64, 65], 6, 2, 3, 6, 64, 128, "slopes", False, True, 1),
    ([257], 3, 3, 1, 1, 128, 256, "retention", True, False, 0),
    ([700], 1, 1, 1, 1, 128, 128, "none", False, False, 0),
    ([1500], 2, 1, 2, 1, 128, 128, "retention", True, True, 70),
    ([900, 3, 1100], 2, 2, 2, 2, 64, 64, "none", True, False, 0),
    ([300, 200], 4, 4, 4, 4, 128, 128, "ends", True, False, 0),
    ([300, 131], 4, 4, 4, 4, 128, 64, "strong", True, False, 5),
    ([40] * 30, 8, 8, 8, 8, 128, 128, "slopes", False, False, 0),
    ([1, 2, 3, 4, 5, 6, 7, 8], 32, 32, 8, 8, 64, 256, "slopes", True, True, 0),
]


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_forward(case, dtype):
    lens, H, qh, kh, vh, dk, dv, kind, s0, fused, behind = case
    c = make(lens, H, qh, kh, vh, dk, dv, dtype, kind, s0, fused, behind, seed=1)
    check_fwd(c, *run_fwd(c))


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("n,T", [(3, 130), (1, 1000), (7, 64), (2, 1)])
def test_forward_equal_lengths_are_the_packed_ones(n, T, dtype):
    c = make([T] * n, 4, 4, 4, 4, 128, 128, dtype, "slopes", True)
    o, S = run_fwd(c, cu=None)
    check_fwd(c, o, S)


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_backward(case, dtype):
    from gated_delta_rule_03_gb300 import linattn_bwd
    lens, H, qh, kh, vh, dk, dv, kind, s0, fused, behind = case
    c = make(lens, H, qh, kh, vh, dk, dv, dtype, kind, s0, fused, behind, seed=2)
    outs = {n: poisoned(t.shape, dtype, "cuda") for n, t in (("dq", c["q"]), ("dk", c["k"]), ("dv", c["v"]))}
    outs["dS0"] = poisoned((len(lens), H, dk, dv), F32, "cuda")
    linattn_bwd(c["do"], c["q"], c["k"], c["v"], c["ld"], S0=c["S0"], dS_final=c["dS"],
                cu_seqlens=c["cu"], scale=c["scale"], **{n: t for n, (t, _) in outs.items()})
    check_guards([g for _, g in outs.values()])
    T = sum(lens)
    do, q, k, v = (ref.f64(c[n])[:T] for n in ("do", "q", "k", "v"))
    want = ref.backward(do, q, k, v, ref.f64(c["ld"]), lens, ref.f64(c["S0"]), ref.f64(c["dS"]), c["scale"])
    for name, (t, _) in outs.items():
        terms = ref.f32_terms(max(lens), dk, dv, H)
        got = t if name == "dS0" else t[:T]
        ref.check(name, got, *want[name], F32 if name == "dS0" else dtype, terms)
        if name != "dS0":
            assert bool(torch.isnan(t[T:]).all()), "rows behind the last sequence were written"


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N,H,qh,kh,vh,dk,dv,kind", [
    (1, 1, 1, 1, 1, 64, 64, "retention"), (3, 4, 2, 4, 1, 128, 128, "slopes"),
    (5, 6, 6, 3, 2, 64, 256, "ends"), (80, 8, 8, 8, 8, 128, 256, "strong"),
    (160, 2, 2, 2, 2, 64, 128, "none"), (33, 32, 32, 8, 8, 128, 64, "slopes")])
def test_step(N, H, qh, kh, vh, dk, dv, kind, dtype):
    from gated_delta_rule_03_gb300 import linattn_step
    c = make([1] * N, H, qh, kh, vh, dk, dv, dtype, kind, True, True, seed=3)
    S, g1 = poisoned(tuple(c["S0"].shape), F32, "cuda", fill=c["S0"])
    o, g2 = poisoned((N, H, dv), dtype, "cuda")
    linattn_step(c["q"], c["k"], c["v"], c["ld"], S, scale=c["scale"], o=o)
    check_guards([g1, g2])
    q, k, v, S0 = (ref.f64(c[n]) for n in ("q", "k", "v", "S0"))
    want_o, want_S, abs_o, abs_S = ref.forward(q, k, v, ref.f64(c["ld"]), c["lens"], S0, c["scale"])
    terms = ref.f32_terms(1, dk, dv)
    ref.check("o", o, want_o, abs_o, dtype, terms)
    ref.check("S", S, want_S, abs_S, F32, terms)


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_prompt_in_pieces_then_steps_is_the_whole(dtype):
    """130 + 70 tokens and three single steps, the state handed on in place, against 203."""
    from gated_delta_rule_03_gb300 import linattn_fwd, linattn_step
    c = make([203], 4, 4, 2, 2, 128, 128, dtype, "slopes", True, seed=4)
    q, k, v, ld = c["q"], c["k"], c["v"], c["ld"]
    S = c["S0"].clone()
    outs = []
    for a, b in ((0, 130), (130, 200)):
        outs.append(linattn_fwd(q[a:b], k[a:b], v[a:b], ld, S0=S, S_final=S)[0])
    for t in range(200, 203):
        outs.append(linattn_step(q[t:t + 1], k[t:t + 1], v[t:t + 1], ld, S))
    check_fwd(c, torch.cat(outs), S)


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_state_in_place_over_several_segments(dtype):
    from gated_delta_rule_03_gb300 import linattn_fwd
    c = make([5000], 1, 1, 1, 1, 128, 128, dtype, "retention", True, seed=5)
    S = c["S0"].clone()
    o, _ = linattn_fwd(c["q"], c["k"], c["v"], c["ld"], S0=S, S_final=S)
    o2, S2 = run_fwd(c)
    assert torch.equal(o, o2) and torch.equal(S, S2)
    assert linattn_fwd(c["q"], c["k"], c["v"], c["ld"], S0=c["S0"], final_state=False)[1] is None


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_values_that_are_not_finite_stay_in_their_sequence_and_head(dtype):
    lens = [100, 130, 60]
    c = make(lens, 2, 2, 2, 2, 128, 128, dtype, "retention", seed=6)
    clean_o, clean_S = run_fwd(c)
    for name in ("q", "k", "v"):
        c[name][100 + 40:100 + 60, 1] = math.nan if name != "k" else math.inf
    o, S = run_fwd_raw(c)
    other = [slice(0, 100), slice(230, 290)]
    for r in other:
        assert torch.equal(o[r], clean_o[r])
    assert torch.equal(o[:, 0], clean_o[:, 0]) and torch.equal(S[:, 0], clean_S[:, 0])
    assert torch.equal(S[0], clean_S[0]) and torch.equal(S[2], clean_S[2])
    assert bool(torch.isnan(o[100 + 60:230, 1]).all()) and bool(torch.isnan(S[1, 1]).any())


def run_fwd_raw(c):
    from gated_delta_rule_03_gb300 import linattn_fwd
    return linattn_fwd(c["q"], c["k"], c["v"], c["ld"], S0=c["S0"], cu_seqlens=c["cu"], scale=c["scale"])


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_same_bits_again_on_another_stream_and_from_a_graph(dtype):
    from gated_delta_rule_03_gb300 import linattn_bwd, linattn_fwd
    c = make([700, 0, 333], 4, 4, 2, 2, 128, 128, dtype, "slopes", True, seed=7)
    args = (c["q"], c["k"], c["v"], c["ld"])
    fwd = lambda: linattn_fwd(*args, S0=c["S0"], cu_seqlens=c["cu"])  # noqa: E731
    bwd = lambda: linattn_bwd(c["do"], *args, S0=c["S0"], dS_final=c["dS"], cu_seqlens=c["cu"])  # noqa: E731
    first = [*fwd(), *bwd()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = [*fwd(), *bwd()]
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for f in (fwd, bwd):  # each graph with a workspace of its own (from its pool)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(f())
        graphs.append(g)
    for _ in range(2):
        for g, out in zip(graphs, outs):
            for t in out:
                t.fill_(math.nan)
            g.replay()
    torch.cuda.synchronize()
    for a, b, d in zip(first, second, [*outs[0], *outs[1]]):
        assert torch.equal(a, b) and torch.equal(a, d)


@gpu
@pytest.mark.parametrize("cu", [[0, 5, 3, 10], [1, 5, 8, 10], [0, 5, 8, 11], [0, -1, 8, 10]])
def test_bad_offsets_are_reported_and_nothing_is_written(cu):
    from gated_delta_rule_03_gb300 import (linattn_bwd, linattn_bwd_workspace_size, linattn_fwd,
                                           linattn_fwd_workspace_size, read_device_status)
    for dtype in (F32, BF16):
        c = make([5, 3, 2], 2, 2, 1, 1, 128, 128, dtype)
        bad = torch.tensor(cu, dtype=torch.int32, device="cuda")
        sizes = (3, 10, 2, 128, 128, dtype)
        ws = torch.zeros(linattn_fwd_workspace_size(*sizes, k_heads=1, v_heads=1), dtype=torch.uint8, device="cuda")
        o = torch.full((10, 2, 128), math.nan, dtype=dtype, device="cuda")
        S = torch.full((3, 2, 128, 128), math.nan, device="cuda")
        linattn_fwd(c["q"], c["k"], c["v"], c["ld"], cu_seqlens=bad, o=o, S_final=S, workspace=ws)
        assert read_device_status(ws) == -7
        assert bool(torch.isnan(o).all()) and bool(torch.isnan(S).all())
        wb = torch.zeros(linattn_bwd_workspace_size(*sizes, k_heads=1, v_heads=1), dtype=torch.uint8, device="cuda")
        d = [torch.full_like(c[n], math.nan) for n in ("q", "k", "v")]
        linattn_bwd(c["do"], c["q"], c["k"], c["v"], c["ld"], cu_seqlens=bad, dq=d[0], dk=d[1], dv=d[2], workspace=wb)
        assert read_device_status(wb) == -7
        assert all(bool(torch.isnan(t).all()) for t in d)
        linattn_fwd(c["q"], c["k"], c["v"], c["ld"], cu_seqlens=c["cu"], o=o, S_final=S, workspace=ws)
        assert read_device_status(ws) == 0 and bool(torch.isfinite(o).all())


# ------------------------------------------------------------------ without a GPU

def test_the_definition_is_the_recurrence_and_its_gradients_are_differences():
    rng = np.random.default_rng(0)
    lens, H, dk, dv, scale = [5, 0, 3], 2, 3, 2, 0.7
    ld = np.array([-0.3, -np.inf])
    q, k, v = (rng.standard_normal((8, h, d)) for h, d in ((2, dk), (1, dk), (1, dv)))
    S0, dS = rng.standard_normal((2, 3, H, dk, dv))
    do = rng.standard_normal((8, H, dv))
    o, S, _, _ = ref.forward(q, k, v, ld, lens, S0, scale)
    lam = np.exp(ld)
    for n, (a, b) in enumerate(ref.spans(lens)):
        for h in range(H):
            s = S0[n, h].copy()
            for t in range(a, b):
                s = lam[h] * s + np.outer(k[t, 0], v[t, 0])
                assert np.allclose(o[t, h], scale * s.T @ q[t, h], atol=1e-12)
            assert np.allclose(S[n, h], s, atol=1e-12)
    loss = lambda q, k, v, S0: (lambda o, S: (o * do).sum() + (S * dS).sum())(  # noqa: E731
        *ref.forward(q, k, v, ld, lens, S0, scale)[:2])
    grads = ref.backward(do, q, k, v, ld, lens, S0, dS, scale)
    point = [q, k, v, S0]
    for i, name in enumerate(("dq", "dk", "dv", "dS0")):
        for at in np.ndindex(point[i].shape):
            lo, hi = [[x.copy() for x in point] for _ in range(2)]
            lo[i][at] -= 0.5
            hi[i][at] += 0.5
            # (the loss is linear in each argument by itself: the difference is exact)
            assert abs(loss(*hi) - loss(*lo) - grads[name][0][at]) < 1e-11


@pytest.fixture(scope="module")
def lib():
    import os
    from gated_delta_rule_03_gb300 import build, ops
    if not os.path.exists(ops.library_path()):
        build.build()
    return ops._load()


def shape(**kw):
    from gated_delta_rule_03_gb300.linattn import LinattnShape
    base = dict(num_seqs=2, total_tokens=128, H=4, q_heads=4, k_heads=2, v_heads=1, d_k=128, d_v=128,
                dtype=1, scale=1.0, q_stride=0, k_stride=0, v_stride=0)
    return LinattnShape(**dict(base, **kw))


BAD_SHAPES = [
    (dict(num_seqs=0), -1), (dict(total_tokens=-1), -1), (dict(H=0), -1), (dict(q_heads=3), -1),
    (dict(k_heads=0), -1), (dict(v_heads=8), -1), (dict(d_k=96), -2), (dict(d_k=256), -2),
    (dict(d_v=32), -2), (dict(dtype=2), -2), (dict(scale=math.nan), -1), (dict(scale=math.inf), -1),
    (dict(q_stride=100), -1), (dict(q_stride=4 * 128 + 4), -3), (dict(k_stride=-256), -1),
    (dict(total_tokens=2 ** 31), -1), (dict(num_seqs=2 ** 31), -1),
    (dict(H=2 ** 20, q_heads=1, k_heads=1, v_heads=1, total_tokens=2 ** 20, num_seqs=1), -1),
    (dict(total_tokens=129), -1),
]


def fake(i):  # aligned addresses far apart, never dereferenced: the call is refused before
    return 0x10000 + i * 0x100000000


@pytest.mark.parametrize("kw,status", BAD_SHAPES)
def test_bad_shapes_are_refused(lib, kw, status):
    s = ctypes.byref(shape(**kw))
    if kw != dict(total_tokens=129):  # (not a multiple of the sequences: the call's to refuse)
        assert lib.gdr_linattn_fwd_workspace_size(s) == 0
        assert lib.gdr_linattn_bwd_workspace_size(s) == 0
    big = 1 << 40
    assert lib.gdr_linattn_fwd(s, *(fake(i) for i in range(4)), None, None, fake(5), fake(6), fake(7), big, None) == status
    assert lib.gdr_linattn_bwd(s, *(fake(i) for i in range(5)), None, None, None, fake(6), fake(7), fake(8),
                               None, fake(9), big, None) == status
    if kw != dict(total_tokens=129):
        assert lib.gdr_linattn_step(s, *(fake(i) for i in range(6)), None) in (status, -1)


def fwd_call(lib, **kw):
    a = dict(q=fake(0), k=fake(1), v=fake(2), ld=fake(3), S0=None, cu=None, o=fake(4), S=fake(5), ws=fake(6), n=1 << 40)
    a.update(kw)
    return lib.gdr_linattn_fwd(ctypes.byref(shape()), a["q"], a["k"], a["v"], a["ld"], a["S0"], a["cu"],
                               a["o"], a["S"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(ld=None), -1), (dict(o=None), -1),
    (dict(ws=None), -4), (dict(n=255), -4), (dict(q=fake(0) + 8), -3), (dict(S=fake(5) + 4), -3),
    (dict(ld=fake(3) + 2), -3), (dict(cu=fake(8) + 1), -3), (dict(o=fake(0)), -1), (dict(o=fake(2) + 256), -1),
    (dict(S=fake(4)), -1), (dict(ws=fake(4)), -1), (dict(S0=fake(5) + 16), -1), (dict(ld=fake(4)), -1),
    (dict(cu=fake(6) + 64), -1)])
def test_bad_arguments_of_the_forward_call_are_refused(lib, kw, status):
    assert fwd_call(lib, **kw) == status


@pytest.mark.parametrize("i,p,status", [
    (0, None, -1), (1, None, -1), (4, None, -1), (8, None, -1), (9, None, -1), (10, None, -1), (12, None, -4),
    (8, fake(9), -1), (8, fake(1), -1), (11, fake(5), -1), (11, fake(6), -1), (12, fake(10), -1), (0, fake(0) + 2, -3)])
def test_bad_arguments_of_the_backward_call_are_refused(lib, i, p, status):
    a = [fake(0), fake(1), fake(2), fake(3), fake(4), fake(5), fake(6), None, fake(8), fake(9), fake(10), fake(11), fake(12)]
    a[i] = p
    assert lib.gdr_linattn_bwd(ctypes.byref(shape()), *a, 1 << 40, None) == status


@pytest.mark.parametrize("i,p,status", [(0, None, -1), (4, None, -1), (5, None, -1), (5, fake(4), -1),
                                        (5, fake(0), -1), (3, fake(4), -1), (4, fake(4) + 8, -3)])
def test_bad_arguments_of_a_step_are_refused(lib, i, p, status):
    a = [fake(j) for j in range(6)]
    a[i] = p
    assert lib.gdr_linattn_step(ctypes.byref(shape(num_seqs=128)), *a, None) == status


def test_a_step_wants_one_token_per_sequence_and_takes_none(lib):
    a = [fake(j) for j in range(6)]
    assert lib.gdr_linattn_step(ctypes.byref(shape()), *a, None) == -1
    assert lib.gdr_linattn_step(ctypes.byref(shape(num_seqs=0, total_tokens=0)), *([None] * 6), None) == 0
    assert lib.gdr_linattn_step(ctypes.byref(shape(num_seqs=0, total_tokens=0, d_k=7)), *([None] * 6), None) == -2


def test_the_binding_refuses_what_it_cannot_pass_on():
    from gated_delta_rule_03_gb300 import linattn_bwd, linattn_fwd, linattn_step
    q = torch.zeros(4, 2, 128)
    for f in (lambda: linattn_fwd(q, q, q, torch.zeros(2)), lambda: linattn_step(q, q, q, torch.zeros(2), q),
              lambda: linattn_bwd(q, q, q, q, torch.zeros(2))):
        with pytest.raises(ValueError, match="CUDA"):
            f()


@gpu
def test_the_binding_checks_shapes_types_and_strides():
    from gated_delta_rule_03_gb300 import GdrError, linattn_bwd, linattn_fwd, linattn_step
    c = make([8], 2, 2, 2, 2, 128, 128, BF16)
    q, k, v, ld = c["q"], c["k"], c["v"], c["ld"]
    S = torch.zeros(1, 2, 128, 128, device="cuda")
    turned = q.transpose(0, 1).contiguous().transpose(0, 1)  # heads outermost in memory
    with pytest.raises(ValueError, match="contiguous"):
        linattn_fwd(turned, k, v, ld)
    with pytest.raises(ValueError, match="stride"):
        linattn_fwd(q[:1].expand(8, 2, 128), k, v, ld)
    for bad in (dict(S0=S[:, :1]), dict(o=c["do"][:4]), dict(S_final=S[0]), dict(num_seqs=3, cu_seqlens=c["cu"])):
        with pytest.raises(ValueError):
            linattn_fwd(q, k, v, ld, **bad)
    with pytest.raises(TypeError):
        linattn_fwd(q, k.float(), v, ld)
    with pytest.raises(TypeError):
        linattn_fwd(q, k, v, ld.double())
    with pytest.raises(ValueError):
        linattn_fwd(q, k[:4], v, ld)
    with pytest.raises(ValueError):
        linattn_bwd(c["do"][:, :1], q, k, v, ld)
    with pytest.raises(ValueError):
        linattn_step(q, k, v, ld, S)
    with pytest.raises(GdrError):
        linattn_fwd(q, k, v, ld, num_seqs=3)
    with pytest.raises(GdrError):
        linattn_fwd(q, k, v, ld, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(GdrError):
        linattn_fwd(q, k, v, ld, o=v)
