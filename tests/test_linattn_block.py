"""Linear attention and the block norms as a network uses them: two layers forward and
backward over packed sequences, and a prompt continued by single tokens, against the same
network in 64 bits.

How far the results may be off is taken from the network itself: in 64 bits, every tensor
that an operator hands on (forward and backward) is moved by one rounding of the type, up or
down at random, and the results' shift is measured. In bf16 an operator rounds at most two
intermediate values as often as the one it hands on, so three such shifts, and a fourth for the
choice of the signs. In fp32 a sum over n terms adds up to n roundings: n + 1 shifts.
"""
import numpy as np
import pytest
import torch

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
U = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
H, DK, DV, D, SCALE, RES, EPS = 2, 128, 128, 256, 128 ** -0.5, 0.5, 1e-6
LENS = [37, 300, 1, 129]
LONGEST_SUM = 300
ACTS = ["silu", "sigmoid"]


class Moved(torch.autograd.Function):
    """x and its gradient, every value moved by the relative size u."""
    @staticmethod
    def forward(ctx, x, u, gen):
        ctx.u, ctx.gen = u, gen
        return x * (1 + u * (2.0 * torch.randint(2, x.shape, generator=gen) - 1))

    @staticmethod
    def backward(ctx, g):
        return g * (1 + ctx.u * (2.0 * torch.randint(2, g.shape, generator=ctx.gen) - 1)), None, None


class Plain:
    """The operators by their formulas in 64 bits."""
    def __init__(self, u=0.0, seed=0):
        self.u, self.gen = u, torch.Generator().manual_seed(seed)

    def hand(self, x):
        return Moved.apply(x, self.u, self.gen) if self.u else x

    def linattn(self, q, k, v, ld, S0, lens):
        o, S, a = [], [], 0
        for n, length in enumerate(lens):
            t = torch.arange(length, dtype=torch.float64)
            W = torch.exp(ld[:, None, None] * (t[:, None] - t[None, :]).clamp(min=0)).tril()
            qs, ks, vs = (x[a:a + length].transpose(0, 1) for x in (q, k, v))
            P = qs @ ks.transpose(1, 2) * W
            w = torch.exp(ld[:, None] * (t + 1))[..., None]
            o.append(SCALE * (P @ vs + w * (qs @ S0[n])).transpose(0, 1))
            w = torch.exp(ld[:, None] * (length - 1 - t))[..., None]
            S.append(torch.exp(ld * length)[:, None, None] * S0[n] + (w * ks).transpose(1, 2) @ vs)
            a += length
        return self.hand(torch.cat(o)), self.hand(torch.stack(S))

    def norm(self, x, y, gate, act, w_post, w_pre):
        rms = lambda a: a * torch.rsqrt((a * a).mean(-1, keepdim=True) + EPS)
        if y is not None:
            x = x + RES * getattr(torch.nn.functional, act)(gate) * rms(y) * w_post
        return self.hand(x), self.hand(rms(x) * w_pre)

    def matmul(self, a, w):
        return self.hand(a @ w)


class Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, ld, S0, cu):
        import gated_delta_rule_03_gb300 as g
        ctx.save_for_backward(q, k, v, ld, S0, cu)
        return g.linattn_fwd(q, k, v, ld, S0=S0, cu_seqlens=cu, scale=SCALE)

    @staticmethod
    def backward(ctx, do, dS):
        import gated_delta_rule_03_gb300 as g
        q, k, v, ld, S0, cu = ctx.saved_tensors
        dq, dk, dv, dS0 = g.linattn_bwd(do.contiguous(), q, k, v, ld, S0=S0, dS_final=dS.contiguous(),
                                        cu_seqlens=cu, scale=SCALE)
        return dq, dk, dv, None, dS0, None


class Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, y, gate, act, w_post, w_pre, dtype):
        import gated_delta_rule_03_gb300 as g
        x_out, h = g.block_norm_fwd(x, y, gate, act, w_post, w_pre, res_scale=RES, eps=EPS, dtype=dtype)
        ctx.save_for_backward(x_out, y, gate, w_post, w_pre)
        ctx.act = act
        return (x_out.view_as(x_out) if y is None else x_out), h

    @staticmethod
    def backward(ctx, dx_out, dh):
        import gated_delta_rule_03_gb300 as g
        x_out, y, gate, w_post, w_pre = ctx.saved_tensors
        dx, dy, dgate, dw_post, dw_pre = g.block_norm_bwd(
            dx_out.contiguous(), dh.contiguous(), x_out, y, gate, ctx.act, w_post, w_pre, res_scale=RES, eps=EPS)
        return dx, dy, dgate, None, dw_post, dw_pre, None


class Ours:
    def __init__(self, dtype):
        self.dtype = dtype

    def linattn(self, q, k, v, ld, S0, lens):
        cu = torch.tensor([0, *np.cumsum(lens)], dtype=torch.int32, device="cuda")
        return Attention.apply(q, k, v, ld, S0, cu)

    def norm(self, x, y, gate, act, w_post, w_pre):
        return Norm.apply(x, y, gate, act, w_post, w_pre, self.dtype)

    def matmul(self, a, w):
        return a @ w


class Steps(Ours):
    """One token per sequence; the states are updated in place."""
    def linattn(self, q, k, v, ld, S0, lens):
        import gated_delta_rule_03_gb300 as g
        return g.linattn_step(q, k, v, ld, S0, scale=SCALE), S0


def network(ops, p, x, states, lens):
    """(x, h, [S of each layer])."""
    x, h = ops.norm(x, None, None, "silu", None, p["w0"])
    new = []
    for i, act in enumerate(ACTS):
        q, k, v = (ops.matmul(h, p[f"{n}{i}"]).view(len(h), H, -1) for n in "qkv")
        gate = ops.matmul(h, p[f"g{i}"])
        o, S = ops.linattn(q, k, v, p[f"ld{i}"], states[i], lens)
        y = ops.matmul(o.reshape(len(h), H * DV), p[f"o{i}"])
        x, h = ops.norm(x, y, gate, act, p[f"post{i}"], p[f"pre{i}"])
        new.append(S)
    return x, h, new


def make(dtype, seed=0):
    """Parameters and inputs, values of the type, in 64 bits; which of them are fp32."""
    g = torch.Generator().manual_seed(seed)
    p, small = {"w0": 1 + 0.1 * torch.randn(D, generator=g)}, {"w0"}
    for i in range(len(ACTS)):
        for n, shape in (("q", (D, H * DK)), ("k", (D, H * DK)), ("v", (D, H * DV)), ("g", (D, D)), ("o", (H * DV, D))):
            p[f"{n}{i}"] = torch.randn(shape, generator=g).mul(shape[0] ** -0.5).to(dtype)
        p[f"post{i}"], p[f"pre{i}"] = (1 + 0.1 * torch.randn(D, generator=g) for _ in range(2))
        p[f"ld{i}"] = torch.tensor([-0.02, -0.3 - 0.2 * i])
        small |= {f"post{i}", f"pre{i}", f"ld{i}"}
    x = torch.randn(sum(LENS), D, generator=g)
    states = [0.3 * torch.randn(len(LENS), H, DK, DV, generator=g) for _ in ACTS]
    return {n: t.double() for n, t in p.items()}, small, x.double(), [s.double() for s in states]


def shift(a, b):
    return (a.double().cpu() - b.double()).norm().item()


def compare(dtype, got, exact, moved):
    few = 4 if dtype is BF16 else LONGEST_SUM + 1
    for name in exact:
        allowed = few * max(shift(m[name], exact[name]) for m in moved)
        assert allowed > 0, name
        off = shift(got[name], exact[name])
        assert off <= allowed, f"{name}: {off:.3e} off, {allowed:.3e} allowed"


def train(ops, p, x, states, cot):
    """The results and every gradient, by name."""
    leaves = {n: t.detach().clone().requires_grad_() for n, t in p.items() if not n.startswith("ld")}
    every = {**p, **leaves}
    leaves["x_in"] = x = x.detach().clone().requires_grad_()
    states = [s.detach().clone().requires_grad_() for s in states]
    leaves.update({f"S_in{i}": s for i, s in enumerate(states)})
    x, h, new = network(ops, every, x, states, LENS)
    out = {"x": x, "h": h, **{f"S{i}": s for i, s in enumerate(new)}}
    torch.autograd.backward(list(out.values()), [cot[n] for n in out])
    return {**{n: t.detach() for n, t in out.items()}, **{"d " + n: t.grad for n, t in leaves.items()}}


def on_gpu(dtype, p, small, x, states):
    p = {n: t.to("cuda", F32 if n in small else dtype) for n, t in p.items()}
    return p, x.to("cuda", F32), [s.to("cuda", F32) for s in states]


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_two_layers_and_their_gradients(dtype):
    p, small, x, states = make(dtype)
    g = torch.Generator().manual_seed(7)
    cot = {"x": torch.randn(x.shape, generator=g), "h": torch.randn(x.shape, generator=g).to(dtype),
           **{f"S{i}": 0.1 * torch.randn(s.shape, generator=g) for i, s in enumerate(states)}}
    exact = train(Plain(), p, x, states, {n: t.double() for n, t in cot.items()})
    moved = [train(Plain(U[dtype], seed), p, x, states, {n: t.double() for n, t in cot.items()}) for seed in (1, 2)]
    got = train(Ours(dtype), *on_gpu(dtype, p, small, x, states), {n: t.cuda() for n, t in cot.items()})
    compare(dtype, got, exact, moved)


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_two_layers_prompt_then_single_tokens(dtype):
    tail = 5
    p, small, _, states = make(dtype)
    lens = [n + tail for n in LENS]
    x = torch.randn(sum(lens), D, generator=torch.Generator().manual_seed(8)).double()

    def whole(ops):
        x2, h2, new = network(ops, p, x, states, lens)
        return {"x": x2, "h": h2, **{f"S{i}": s for i, s in enumerate(new)}}
    exact, moved = whole(Plain()), [whole(Plain(U[dtype], seed)) for seed in (1, 2)]

    pg, xg, sg = on_gpu(dtype, p, small, x, states)
    begin = [0, *np.cumsum(lens)]
    rows = [torch.arange(begin[i], begin[i] + n) for i, n in enumerate(LENS)]
    px, ph, now = network(Ours(dtype), pg, xg[torch.cat(rows)], sg, LENS)
    ox, oh = torch.empty_like(xg), torch.empty(xg.shape, dtype=dtype, device="cuda")
    ox[torch.cat(rows)], oh[torch.cat(rows)] = px, ph
    for t in range(tail):
        at = torch.tensor([begin[i] + n + t for i, n in enumerate(LENS)])
        ox[at], oh[at], now = network(Steps(dtype), pg, xg[at], now, None)
    compare(dtype, {"x": ox, "h": oh, **{f"S{i}": s for i, s in enumerate(now)}}, exact, moved)


def test_the_network_in_64_bits_has_the_gradients_of_its_differences():
    """Along one direction through all leaves: the gradient against a central difference."""
    p, _, x, states = make(F32)
    g = torch.Generator().manual_seed(9)
    cot = {"x": torch.randn(x.shape, generator=g).double(), "h": torch.randn(x.shape, generator=g).double(),
           **{f"S{i}": torch.randn(s.shape, generator=g).double() for i, s in enumerate(states)}}
    res = train(Plain(), p, x, states, cot)
    step = {n[2:]: 1e-6 * torch.randn(t.shape, generator=g).double() for n, t in res.items() if n.startswith("d ")}
    slope = sum((res["d " + n] * s).sum() for n, s in step.items())

    def value(sign):
        q = {n: t + sign * step[n] if n in step else t for n, t in p.items()}
        x2, h2, new = network(Plain(), q, x + sign * step["x_in"],
                              [s + sign * step[f"S_in{i}"] for i, s in enumerate(states)], LENS)
        return (x2 * cot["x"]).sum() + (h2 * cot["h"]).sum() + sum((s * cot[f"S{i}"]).sum() for i, s in enumerate(new))
    # third derivatives over steps of 1e-6, and 2^-53 of sums of about 1e4
    assert abs((value(1) - value(-1)) / 2 - slope) <= 1e-5 * abs(slope)
