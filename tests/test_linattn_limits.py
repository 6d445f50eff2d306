"""Linear attention and the block norms where calls go wrong first: sequences that are cut into
segments in every way, tensors behind 2^31 elements, values shared by arguments, other streams."""
import ctypes
import math

import pytest
import torch

from tests import linattn_ref as ref
from tests.helpers import check_guards, poisoned
from tests.test_linattn import check_fwd, fake, make, run_fwd, run_fwd_raw, shape

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def check_bwd(c, cu="packed"):
    from gated_delta_rule_03_gb300 import linattn_bwd
    n, T, dtype = len(c["lens"]), sum(c["lens"]), c["dtype"]
    outs = {name: poisoned(c[t].shape, dtype, "cuda") for name, t in (("dq", "q"), ("dk", "k"), ("dv", "v"))}
    outs["dS0"] = poisoned((n, c["H"], c["dk"], c["dv"]), F32, "cuda")
    linattn_bwd(c["do"], c["q"], c["k"], c["v"], c["ld"], S0=c["S0"], dS_final=c["dS"],
                cu_seqlens=c["cu"] if cu == "packed" else None, num_seqs=n, scale=c["scale"],
                **{name: t for name, (t, _) in outs.items()})
    check_guards([g for _, g in outs.values()])
    do, q, k, v = (ref.f64(c[name])[:T] for name in ("do", "q", "k", "v"))
    want = ref.backward(do, q, k, v, ref.f64(c["ld"]), c["lens"], ref.f64(c["S0"]), ref.f64(c["dS"]), c["scale"])
    terms = ref.f32_terms(max(c["lens"]), c["dk"], c["dv"], c["H"])
    for name, (t, _) in outs.items():
        ref.check(name, t if name == "dS0" else t[:T], *want[name], F32 if name == "dS0" else dtype, terms)
        if name != "dS0":
            assert bool(torch.isnan(t[T:]).all()), "rows behind the last sequence were written"


# lens, H, q heads, k heads, v heads, d_k, d_v, decay, rows behind: one long sequence, equal long
# ones, a long one among short ones (cut), a tail of one token behind a segment
CUT = [
    ([2900], 1, 1, 1, 1, 64, 256, "retention", 0),
    ([2561], 2, 1, 2, 1, 128, 256, "none", 40),
    ([1800, 1800], 2, 2, 1, 2, 64, 128, "retention", 0),
    ([1, 2600, 0, 130, 5, 127, 1, 90], 2, 2, 2, 1, 128, 128, "retention", 9),
    ([2305, 1, 1, 1, 1, 1, 1, 1, 1, 1], 3, 3, 3, 3, 128, 64, "slopes", 0),
]


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", CUT, ids=[str(i) for i in range(len(CUT))])
def test_cut_sequences(case, dtype):
    lens, H, qh, kh, vh, dk, dv, kind, behind = case
    c = make(lens, H, qh, kh, vh, dk, dv, dtype, kind, s0=True, behind=behind, seed=3)
    check_fwd(c, *run_fwd(c))
    check_bwd(c)


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_more_sequences_than_a_block_has_threads(dtype):
    """The offsets are scanned a block's width at a time; one sequence behind the first
    width is cut."""
    c = make([1, 0, 2] * 230 + [2100] + [3, 1] * 60, 1, 1, 1, 1, 64, 64, dtype, "retention", s0=True, behind=3, seed=11)
    assert len(c["lens"]) > 576
    check_fwd(c, *run_fwd(c))
    check_bwd(c)


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("n,T,H", [(2, 1700, 1), (3, 640, 2), (1, 2177, 2)])
def test_equal_lengths_forward_and_backward(n, T, H, dtype):
    c = make([T] * n, H, H, H, H, 128, 128, dtype, "retention", s0=True, seed=4)
    check_fwd(c, *run_fwd(c, cu=None))
    check_bwd(c, cu=None)


@gpu
@pytest.mark.parametrize("N,T,H,dtype", [(9, 2560, 17, BF16), (3, 2500, 18, BF16), (7, 650, 11, F32)],
                         ids=["forward-bf16", "backward-bf16", "f32"])
def test_some_pairs_whole_and_the_rest_cut(N, T, H, dtype):
    """A few chains more than the GPU has SMs (153, 162 and 154 of them): most (sequence, head)
    pairs stay whole, the last ones are cut. Corners against the definition, all pairs written."""
    from gated_delta_rule_03_gb300 import linattn_bwd
    c = make([T] * N, H, H, H, H, 128, 128, dtype, "retention", s0=True, seed=12)
    o, S = run_fwd(c, cu=None)
    outs = [torch.full_like(c[n], math.nan) for n in ("q", "k", "v", "S0")]
    linattn_bwd(c["do"], c["q"], c["k"], c["v"], c["ld"], S0=c["S0"], dS_final=c["dS"], num_seqs=N,
                scale=c["scale"], dq=outs[0], dk=outs[1], dv=outs[2], dS0=outs[3])
    assert all(bool(torch.isfinite(t).all()) for t in (o, S, *outs))
    terms = ref.f32_terms(T, 128, 128, 1)
    for n, h in [(0, 0), (N - 2, H - 1), (N - 1, 0), (N - 1, H - 2), (N - 1, H - 1)]:
        rows = slice(n * T, (n + 1) * T)
        q, k, v, do = (ref.f64(c[x][rows, h:h + 1]) for x in ("q", "k", "v", "do"))
        ld, S0, dS = ref.f64(c["ld"][h:h + 1]), ref.f64(c["S0"][n:n + 1, h:h + 1]), ref.f64(c["dS"][n:n + 1, h:h + 1])
        want_o, want_S, abs_o, abs_S = ref.forward(q, k, v, ld, [T], S0, c["scale"])
        ref.check("o", o[rows, h:h + 1], want_o, abs_o, dtype, terms)
        ref.check("S_final", S[n:n + 1, h:h + 1], want_S, abs_S, F32, terms)
        want = ref.backward(do, q, k, v, ld, [T], S0, dS, c["scale"])
        for name, t in zip(("dq", "dk", "dv"), outs):
            ref.check(name, t[rows, h:h + 1], *want[name], dtype, terms)
        ref.check("dS0", outs[3][n:n + 1, h:h + 1], *want["dS0"], F32, terms)


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_one_tensor_as_query_key_and_value(dtype):
    c = make([500, 77], 2, 2, 2, 2, 128, 128, dtype, "retention", s0=True, seed=5)
    c["k"] = c["v"] = c["q"]
    check_fwd(c, *run_fwd(c))
    check_bwd(c)


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_a_decay_that_is_not_a_number_stays_in_its_head(dtype):
    from gated_delta_rule_03_gb300 import linattn_bwd
    c = make([1500, 40], 3, 3, 3, 3, 128, 128, dtype, "retention", seed=6)
    args = (c["q"], c["k"], c["v"])
    o, S = run_fwd_raw(c)
    d = linattn_bwd(c["do"], *args, c["ld"], cu_seqlens=c["cu"])[:3]
    c["ld"][1] = math.nan
    o2, S2 = run_fwd_raw(c)
    d2 = linattn_bwd(c["do"], *args, c["ld"], cu_seqlens=c["cu"])[:3]
    keep = [0, 2]
    assert torch.equal(S[:, keep], S2[:, keep]) and bool(torch.isnan(S2[:, 1]).all())
    for a, b in zip([o, *d], [o2, *d2]):
        assert torch.equal(a[:, keep], b[:, keep])
        assert bool(torch.isnan(b[:, 1]).any())


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("cu", [[0, 2000, 1000, 4000], [0, 2000, 3000, 4001], [0, -5, 3000, 4000]])
def test_bad_offsets_of_long_calls_write_nothing(cu, dtype):
    from gated_delta_rule_03_gb300 import (linattn_bwd, linattn_bwd_workspace_size, linattn_fwd,
                                           linattn_fwd_workspace_size, read_device_status)
    c = make([2000, 1000, 1000], 2, 2, 1, 2, 128, 128, dtype, s0=True)
    bad = torch.tensor(cu, dtype=torch.int32, device="cuda")
    nan = lambda t: torch.full_like(t, math.nan)  # noqa: E731
    sizes = (3, 4000, 2, 128, 128, dtype)
    ws = torch.zeros(linattn_fwd_workspace_size(*sizes, k_heads=1), dtype=torch.uint8, device="cuda")
    o, S = nan(c["v"]), nan(c["S0"])
    linattn_fwd(c["q"], c["k"], c["v"], c["ld"], S0=c["S0"], cu_seqlens=bad, o=o, S_final=S, workspace=ws)
    assert read_device_status(ws) == -7
    wb = torch.zeros(linattn_bwd_workspace_size(*sizes, k_heads=1), dtype=torch.uint8, device="cuda")
    d = [nan(c[n]) for n in ("q", "k", "v", "S0")]
    linattn_bwd(c["do"], c["q"], c["k"], c["v"], c["ld"], S0=c["S0"], dS_final=c["dS"], cu_seqlens=bad,
                dq=d[0], dk=d[1], dv=d[2], dS0=d[3], workspace=wb)
    assert read_device_status(wb) == -7
    assert all(bool(torch.isnan(t).all()) for t in (o, S, *d))


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_two_calls_at_once_and_two_graphs_that_share_a_workspace(dtype):
    from gated_delta_rule_03_gb300 import linattn_fwd, linattn_fwd_workspace_size
    cs = [make([2000, 300], 4, 4, 4, 4, 128, 128, dtype, "retention", s0=True, seed=s) for s in (8, 9)]
    want = [run_fwd_raw(c) for c in cs]
    call = lambda c, **kw: linattn_fwd(c["q"], c["k"], c["v"], c["ld"], S0=c["S0"],  # noqa: E731
                                       cu_seqlens=c["cu"], **kw)
    sides = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    got = [call(c, stream=s) for _ in range(5) for c, s in zip(cs, sides)]
    torch.cuda.synchronize()
    for i, (o, S) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(S, want[i % 2][1])
    ws = torch.empty(linattn_fwd_workspace_size(2, 2300, 4, 128, 128, dtype), dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for c in cs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(c, workspace=ws))
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 0, 1)):
        for o, S in outs:
            o.fill_(math.nan), S.fill_(math.nan)
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for (o, S), (o1, S1) in zip(outs, want):
            assert torch.equal(o, o1) and torch.equal(S, S1)


@gpu
def test_new_results_on_another_stream_are_memory_of_that_stream():
    """The current stream still has to write memory that it has given back: a call on another
    stream, which does not wait for that, must not get it."""
    from gated_delta_rule_03_gb300 import block_norm_bwd, block_norm_fwd, linattn_bwd, linattn_fwd, linattn_step
    c = make([1200, 200], 2, 2, 2, 2, 128, 128, BF16, "retention", s0=True, seed=10)
    args = (c["q"], c["k"], c["v"], c["ld"])
    S = c["S0"].clone()
    x = torch.randn(1400, 512, device="cuda").bfloat16()
    y, w = torch.randn_like(x), torch.randn(512, device="cuda")
    tok = [t[:2].contiguous() for t in args[:3]]
    calls = [lambda s: linattn_fwd(*args, S0=c["S0"], cu_seqlens=c["cu"], stream=s),
             lambda s: linattn_bwd(c["do"], *args, S0=c["S0"], dS_final=c["dS"], cu_seqlens=c["cu"], stream=s),
             lambda s: [linattn_step(*tok, c["ld"], S, stream=s)],
             lambda s: block_norm_fwd(x, y, w_post=w, w_pre=w, stream=s),
             lambda s: [t for t in block_norm_bwd(x, y, x, y, w_post=w, w_pre=w, stream=s) if t is not None]]
    side = torch.cuda.Stream()
    for call in calls:
        S.copy_(c["S0"])
        want = [t.clone() for t in call(None)]
        S.copy_(c["S0"])
        torch.cuda.synchronize()
        held = [torch.empty_like(t) for t in want for _ in range(2)]
        held += [torch.empty(1 << n, dtype=torch.uint8, device="cuda") for n in range(9, 26)]
        torch.cuda._sleep(30_000_000)
        for t in held:
            t.fill_(255 if t.dtype is torch.uint8 else math.nan)
        del held, t
        got = call(side)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@gpu
def test_rows_behind_2_to_the_31_elements():
    """The last of two sequences lies behind element 2^31 of every tensor."""
    from gated_delta_rule_03_gb300 import linattn_bwd, linattn_fwd
    H, d, T, last, heads = 128, 128, 140_000, 200, [0, 127]
    assert (T - last) * H * d > 2 ** 31
    q, k, v, do = (torch.empty(T, H, d, dtype=BF16, device="cuda").normal_().mul_(0.1) for _ in range(4))
    ld = torch.full((H,), -0.01, device="cuda")
    cu = torch.tensor([0, T - last, T], dtype=torch.int32, device="cuda")
    c = [t[-last:, heads].cpu().double().numpy() for t in (q, k, v, do)]
    ldh, terms = ref.f64(ld[heads]), ref.f32_terms(last, d, d, 1)
    o, S = linattn_fwd(q, k, v, ld, cu_seqlens=cu)
    want_o, want_S, abs_o, abs_S = ref.forward(*c[:3], ldh, [last])
    ref.check("o", o[-last:, heads], want_o, abs_o, BF16, terms)
    ref.check("S_final", S[1:, heads], want_S, abs_S, F32, terms)
    del o
    grads = linattn_bwd(do, q, k, v, ld, cu_seqlens=cu)
    want = ref.backward(c[3], *c[:3], ldh, [last], None, None, 1.0)
    for name, got in zip(("dq", "dk", "dv"), grads):
        ref.check(name, got[-last:, heads], *want[name], BF16, terms)


@gpu
def test_block_norm_rows_behind_2_to_the_31_elements():
    from gated_delta_rule_03_gb300 import block_norm_bwd, block_norm_fwd
    D, rows, last = 4096, 530_000, 64
    assert (rows - last) * D > 2 ** 31
    x, y, g = (torch.empty(rows, D, dtype=BF16, device="cuda").normal_() for _ in range(3))
    w = torch.randn(D, device="cuda")
    few = [t[-last:].clone() for t in (x, y, g)]
    x2, h = block_norm_fwd(x, y, g, w_post=w, w_pre=w)
    a = block_norm_fwd(*few, w_post=w, w_pre=w)
    assert torch.equal(x2[-last:], a[0]) and torch.equal(h[-last:], a[1])
    got = block_norm_bwd(x, h, x2, y, g, w_post=w, w_pre=w)
    b = block_norm_bwd(few[0], a[1], a[0], few[1], few[2], w_post=w, w_pre=w)
    for s, t in zip(got[:3], b[:3]):
        assert torch.equal(s[-last:], t)


# ------------------------------------------------------------------ without a GPU


def test_more_heads_than_a_row_can_have_are_refused():
    from gated_delta_rule_03_gb300 import ops
    lib = ops._load()
    s = ctypes.byref(shape(H=1 << 17, q_heads=1, k_heads=1, v_heads=1))
    assert lib.gdr_linattn_fwd_workspace_size(s) == 0 and lib.gdr_linattn_bwd_workspace_size(s) == 0
    assert lib.gdr_linattn_step(s, *(fake(i) for i in range(6)), None) == -1


def test_the_workspace_size_holds_for_packed_and_for_equal_lengths():
    from gated_delta_rule_03_gb300 import ops
    lib = ops._load()
    for n, T in [(1, 1), (1, 65536), (4, 16384), (8, 40000), (64, 6400), (3, 5000)]:
        for dtype in (0, 1):
            s = ctypes.byref(shape(num_seqs=n, total_tokens=T, dtype=dtype, k_heads=4, v_heads=4))
            fwd, bwd = lib.gdr_linattn_fwd_workspace_size(s), lib.gdr_linattn_bwd_workspace_size(s)
            assert fwd > 0 and bwd > 0
            for cu in (None, fake(11)):
                if cu is None and T % n:
                    continue
                # one byte less is refused before any launch
                assert lib.gdr_linattn_fwd(s, *(fake(i) for i in range(4)), None, cu, fake(5), fake(6), fake(7), fwd - 1, None) == -4
                assert lib.gdr_linattn_bwd(s, *(fake(i) for i in range(5)), None, None, cu, fake(6), fake(7), fake(8),
                                           None, fake(9), bwd - 1, None) == -4


def test_the_workspace_does_not_grow_with_short_sequences():
    """A sum is kept for a segment that hands one on: at most T / 128 of them, in four parts."""
    from gated_delta_rule_03_gb300 import ops
    lib = ops._load()
    matrix = 4 * 128 * 128 * 4  # heads, d_k, d_v, bytes
    for n, T in [(64, 6400), (4096, 40960), (1000, 1000)]:
        s = ctypes.byref(shape(num_seqs=n, total_tokens=T, k_heads=4, v_heads=4))
        sums = 4 * (T // 128) * matrix
        assert lib.gdr_linattn_fwd_workspace_size(s) <= n * matrix + sums + 1024
        assert lib.gdr_linattn_bwd_workspace_size(s) <= 2 * sums + 1024
