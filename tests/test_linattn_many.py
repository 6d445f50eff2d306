"""Linear attention over more packed sequences than are taken longest first (64)."""
import math

import numpy as np
import pytest
import torch

from tests.test_linattn import BF16, F32, check_fwd, make, run_fwd
from tests.test_linattn_limits import check_bwd

gpu = pytest.mark.gpu


def lengths(n, longest, seed):
    """n sequences: empty ones, single tokens, a few tokens, whole segments (multiples of 128
    tokens begin and end on their border), some longer than the rest together."""
    rng = np.random.default_rng(seed)
    lens = rng.choice([0, 0, 1, 1, 2, 3, 64, 128, 256], size=n, p=[.2, .2, .2, .1, .1, .1, .04, .03, .03])
    lens[rng.integers(0, n, 2)] = longest
    lens[0] = lens[0] if seed % 2 else 0
    lens[-1] = lens[-1] if seed % 3 else 0
    return [int(x) for x in lens]


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("n,longest,H,behind", [(65, 2000, 2, 0), (577, 1500, 1, 5), (3000, 1100, 1, 0)])
def test_many_packed_sequences(n, longest, H, behind, dtype):
    lens = lengths(n, longest, n)
    c = make(lens, H, H, 1, H, 64, 64, dtype, "slopes", s0=True, behind=behind, seed=n)
    check_fwd(c, *run_fwd(c))
    check_bwd(c)


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_nothing_but_empty_sequences_and_one(dtype):
    for at in (0, 99, 149):
        lens = [0] * 150
        lens[at] = 700
        c = make(lens, 2, 2, 2, 2, 64, 128, dtype, "retention", s0=True, seed=at)
        check_fwd(c, *run_fwd(c))
        check_bwd(c)


# below and above the number from which a launch ahead checks the offsets
@gpu
@pytest.mark.parametrize("n", [1500, 2500])
@pytest.mark.parametrize("at,value", [(0, 1), (700, 3), (1400, 10 ** 6), (1, -1), (-1, 10 ** 4)])
def test_bad_offsets_among_many_write_nothing(at, value, n):
    from gated_delta_rule_03_gb300 import linattn_bwd, linattn_bwd_workspace_size, linattn_fwd, read_device_status
    for dtype in (F32, BF16):
        c = make([2] * n, 1, 1, 1, 1, 64, 64, dtype)
        bad = c["cu"].clone()
        bad[at] = value
        o = torch.full((2 * n, 1, 64), math.nan, dtype=dtype, device="cuda")
        S = torch.full((n, 1, 64, 64), math.nan, device="cuda")
        ws = torch.zeros(linattn_bwd_workspace_size(n, 2 * n, 1, 64, 64, dtype) + (64 << 20), dtype=torch.uint8, device="cuda")
        linattn_fwd(c["q"], c["k"], c["v"], c["ld"], cu_seqlens=bad, o=o, S_final=S, workspace=ws)
        assert read_device_status(ws) == -7
        d = [torch.full_like(c[t], math.nan) for t in ("q", "k", "v")]
        linattn_bwd(c["do"], c["q"], c["k"], c["v"], c["ld"], cu_seqlens=bad, dq=d[0], dk=d[1], dv=d[2], workspace=ws)
        assert read_device_status(ws) == -7
        assert all(bool(torch.isnan(t).all()) for t in (o, S, *d))


@gpu
def test_a_captured_call_of_many_sequences_takes_the_offsets_of_each_replay():
    from gated_delta_rule_03_gb300 import linattn_fwd, linattn_fwd_workspace_size, read_device_status
    lens = lengths(2600, 900, 5)
    c = make(lens, 2, 2, 2, 2, 64, 64, BF16, "slopes", s0=True, seed=6)
    T, cu = sum(lens), c["cu"].clone()
    ws = torch.zeros(linattn_fwd_workspace_size(2600, T, 2, 64, 64), dtype=torch.uint8, device="cuda")
    o, S = torch.empty((T, 2, 64), dtype=BF16, device="cuda"), torch.empty_like(c["S0"])
    call = lambda: linattn_fwd(c["q"], c["k"], c["v"], c["ld"], S0=c["S0"], cu_seqlens=cu, o=o, S_final=S, workspace=ws)  # noqa: E731
    call()
    want = o.clone(), S.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for good in (True, False, True):
        cu.copy_(c["cu"])
        if not good:
            cu[1000] = T + 1
        o.fill_(math.nan)
        S.fill_(math.nan)
        g.replay()
        assert read_device_status(ws) == (0 if good else -7)
        if good:
            assert torch.equal(o, want[0]) and torch.equal(S, want[1])
        else:
            assert bool(torch.isnan(o).all()) and bool(torch.isnan(S).all())


# ------------------------------------------------------------------ without a GPU

def places(cu, total, seg, hand_on):
    """{place: (sequence, segment)} by the rule of the kernels: sequence n has the places from
    floor(cu[n] / seg) on, and one more for each sequence before it unless only segments that
    hand a sum on are meant."""
    found = {}
    for n in range(len(cu) - 1):
        count = max(1, -(-(cu[n + 1] - cu[n]) // seg)) - hand_on
        first = cu[n] // seg + (0 if hand_on else n)
        for f in range(count):
            assert first + f not in found
            found[first + f] = (n, f)
            assert first + f < cu[n + 1] // seg + (0 if hand_on else n + 1)
    assert all(0 <= p < total // seg + (0 if hand_on else len(cu) - 1) for p in found)
    return found


def test_places_by_offsets_are_apart_and_within_the_launch():
    rng = np.random.default_rng(3)
    for _ in range(2000):
        n, seg = int(rng.integers(1, 9)), int(rng.choice([1, 2, 3, 7, 128]))
        lens = rng.choice([0, 0, 1, 2, seg - 1, seg, seg + 1, 2 * seg, 5 * seg + 1], size=n)
        cu = [0, *np.cumsum(lens).tolist()]
        total = cu[-1] + int(rng.choice([0, 1, seg]))
        assert len(places(cu, total, seg, 0)) == sum(max(1, -(-x // seg)) for x in lens.tolist())
        places(cu, total, seg, 1)
