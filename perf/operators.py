"""Measured calls of the linear-attention and block-norm operators.

Operators
  linattn_fwd    linear attention with one constant decay per head over prompts (equal or
                 packed lengths): S_t = lam S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t
  linattn_step   the same recurrence for a single token of every sequence, state in place
  linattn_bwd    the gradients of linattn_fwd
  block_norm_fwd the norms before and after a block, fused with the block's gate and the
                 residual scale: x' = x + s act(g) rmsnorm(y) w_post, h = rmsnorm(x') w_pre
  block_norm_bwd its gradients

`own` false: the plain form (elementary torch operations in 32 bits, decay tables in 64).
`own` true: the calls of gated_delta_rule_03_gb300.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
PLAIN_CHUNK = 128


# ------------------------------------------------------------------ the cases

def listed():
    fwd = dict(op="linattn_fwd", N=1, T=0, lo=0, hi=0, lens=0, H=16, Hq=16, Hk=16, Hv=16, dk=128,
               dv=128, dtype="bf16", s0=False, fused=False, scale=1.0, decay="retention")
    bwd = dict(fwd, op="linattn_bwd", ds=False)
    step = dict(op="linattn_step", N=1, H=32, Hq=32, Hk=32, Hv=32, dk=128, dv=128, dtype="bf16",
                scale=1.0, decay="retention")
    norm = dict(op="block_norm_fwd", rows=1, D=2048, dtype="bf16", x_dtype="bf16", act="silu",
                gate="rows", post=True, pre=True, res_scale=1.0)
    nbwd = dict(norm, op="block_norm_bwd")
    return [
        # a short fp32 prompt of a small model: latency and the fp32 arithmetic
        dict(fwd, name="fwd_tiny_fp32", N=1, T=256, H=2, Hq=2, Hk=2, Hv=2, dk=64, dv=64, dtype="f32"),
        # a batch of four prompts of 4,096 tokens
        dict(fwd, name="fwd_prefill_bf16", N=4, T=4096),
        # eight packed prompts of odd lengths, keys and values shared by groups of four
        # heads, views of one fused projection, continuing from states
        dict(fwd, name="fwd_packed_shared_bf16", N=8, lo=512, hi=8192, lens=2, Hk=4, Hv=4, s0=True,
             fused=True, scale=128 ** -0.5, decay="slopes"),
        # one long document
        dict(fwd, name="fwd_long_bf16", N=1, T=65536, H=8, Hq=8, Hk=8, Hv=8, dv=256),
        # one sequence's next token
        dict(step, name="step_one_bf16", N=1),
        # the next token of a full serving batch
        dict(step, name="step_batch_bf16", N=256),
        # a training step's layer: four sequences of 4,096 tokens
        dict(bwd, name="bwd_train_bf16", N=4, T=4096),
        # packed training sequences of odd lengths, keys and values shared by two heads,
        # carried states with their gradients
        dict(bwd, name="bwd_packed_shared_bf16", N=5, lo=100, hi=3000, lens=3, H=8, Hq=8, Hk=4, Hv=4,
             s0=True, ds=True, fused=True, scale=128 ** -0.5, decay="slopes"),
        # the residual stream of a prompt batch, gate per token
        dict(norm, name="norm_fwd_prefill_bf16", rows=16384),
        # the residual stream of a decode batch: 32 heads of 128
        dict(norm, name="norm_fwd_decode_bf16", rows=256, D=4096, act="sigmoid", res_scale=0.5),
        # a training step's layer
        dict(nbwd, name="norm_bwd_train_bf16", rows=16384),
        # an odd width in fp32, one learned gate row for all tokens
        dict(nbwd, name="norm_bwd_odd_fp32", rows=4099, D=1030, dtype="f32", x_dtype="f32",
             act="identity", gate="one", res_scale=0.25),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _divisor(rng, H):
    return rng.choice([d for d in range(1, H + 1) if H % d == 0 and H // d <= 8])


def draw(rng):
    op = rng.choice(["linattn_fwd", "linattn_fwd", "linattn_step", "linattn_bwd", "linattn_bwd",
                     "block_norm_fwd", "block_norm_bwd"])
    if op.startswith("block_norm"):
        D = _log_int(rng, 96, 8192)
        rows = _log_int(rng, 1, max(2, (1 << 25) // D))
        dtype = rng.choice(["bf16", "bf16", "f32"])
        return dict(op=op, rows=rows, D=D, dtype=dtype, x_dtype=rng.choice([dtype, "f32"]),
                    act=rng.choice(["silu", "sigmoid", "identity"]),
                    gate=rng.choice(["rows", "rows", "one", "none"]), post=rng.random() < 0.8,
                    pre=rng.random() < 0.8, res_scale=rng.choice([1.0, 0.5, 0.22]))
    dtype = rng.choice(["bf16", "bf16", "f32"])
    H = _log_int(rng, 1, 32)
    dk, dv = rng.choice([(128, 128), (128, 128), (128, 256), (64, 128), (64, 64)])
    if op == "linattn_bwd" and dv == 256 and dtype == "f32":
        dv = 128
    heads = dict(H=H, Hq=_divisor(rng, H), Hk=_divisor(rng, H), Hv=_divisor(rng, H), dk=dk, dv=dv,
                 dtype=dtype, scale=rng.choice([1.0, dk ** -0.5]),
                 decay=rng.choice(["retention", "slopes", "none"]))
    if op == "linattn_step":
        return dict(op=op, N=_log_int(rng, 1, max(1, 8192 * 128 // (H * dv))), **heads)
    budget = (1 << 18) if dtype == "bf16" else (1 << 16)  # token-heads
    most = budget // H * 128 // dv
    case = dict(op=op, T=0, lo=0, hi=0, lens=0, s0=rng.random() < 0.5, fused=rng.random() < 0.5, **heads)
    if op == "linattn_bwd":
        case["ds"] = rng.random() < 0.5
        most //= 2
    if rng.random() < 0.4:
        case["T"] = _log_int(rng, 1, most)
        case["N"] = _log_int(rng, 1, min(64, max(1, most // case["T"])))
    else:
        case["N"] = _log_int(rng, 1, min(64, max(1, most // 64)))
        case["hi"] = _log_int(rng, 8, max(9, most // case["N"]))
        case["lo"] = rng.randrange(0, case["hi"])
        case["lens"] = rng.randrange(1, 1 << 20)
    return case


def _lens(case):
    """Tokens of every sequence."""
    if case["T"]:
        return [case["T"]] * case["N"]
    return [int(n) for n in np.random.RandomState(case["lens"]).randint(case["lo"], case["hi"] + 1, case["N"])]


# ------------------------------------------------------------------ inputs

def _normal(gen, shape, dtype, unit=False):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    if unit:
        x /= x.norm(dim=-1, keepdim=True).clamp_min(1e-12)
    return x.to(dtype)


def _decays(case):
    """log of the decay of each head, fp32: slow to fast over the heads."""
    H = case["H"]
    h = np.arange(H, dtype=np.float64)
    if case["decay"] == "retention":    # lam = 1 - 2^-5 .. 1 - 2^-12
        ld = np.log1p(-2.0 ** -(5 + 7 * h / max(1, H - 1)))
    elif case["decay"] == "slopes":     # lam = exp(-2^(-8 (h + 1) / H))
        ld = -2.0 ** (-8 * (h + 1) / H)
    else:
        ld = np.zeros(H)
    return torch.tensor(ld, dtype=torch.float32, device="cuda")


def _qkv(case, gen, rows):
    dt, dk, dv = DTYPES[case["dtype"]], case["dk"], case["dv"]
    q = _normal(gen, (rows, case["Hq"], dk), dt, True)
    k = _normal(gen, (rows, case["Hk"], dk), dt, True)
    v = _normal(gen, (rows, case["Hv"], dv), dt)
    if case.get("fused"):  # views of one projection's rows
        w = torch.cat([q.flatten(1), k.flatten(1), v.flatten(1)], 1)
        a, b = case["Hq"] * dk, (case["Hq"] + case["Hk"]) * dk
        q, k, v = (w[:, :a].view(rows, -1, dk), w[:, a:b].view(rows, -1, dk), w[:, b:].view(rows, -1, dv))
    return q, k, v


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case=case, op=case["op"])
    if case["op"].startswith("block_norm"):
        dt, xdt, n, D = DTYPES[case["dtype"]], DTYPES[case["x_dtype"]], case["rows"], case["D"]
        s["y"] = _normal(gen, (n, D), dt)
        s["gate"] = None if case["gate"] == "none" else _normal(gen, (n if case["gate"] == "rows" else 1, D), dt)
        s["w_post"] = 1 + 0.1 * _normal(gen, (D,), torch.float32) if case["post"] else None
        s["w_pre"] = 1 + 0.1 * _normal(gen, (D,), torch.float32) if case["pre"] else None
        s["x"] = _normal(gen, (n, D), xdt)
        if case["op"] == "block_norm_bwd":  # x holds the sum that the forward call wrote
            s["dx_out"] = _normal(gen, (n, D), xdt)
            s["dh"] = _normal(gen, (n, D), dt) if case["pre"] else None
        return s
    s["log_decay"] = _decays(case)
    N, H, dk, dv = case["N"], case["H"], case["dk"], case["dv"]
    if case["op"] == "linattn_step":
        s["q"], s["k"], s["v"] = _qkv(case, gen, N)
        s["S"] = 0.5 * _normal(gen, (N, H, dk, dv), torch.float32)
        return s
    lens = _lens(case)
    rows = sum(lens)
    s["q"], s["k"], s["v"] = _qkv(case, gen, rows)
    s["S0"] = 0.5 * _normal(gen, (N, H, dk, dv), torch.float32) if case["s0"] else None
    s["cu"] = None if case["T"] else torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    s["longest"] = max(1, max(lens))
    if case["op"] == "linattn_bwd":
        s["do"] = _normal(gen, (rows, H, dv), DTYPES[case["dtype"]])
        s["dS"] = 0.5 * _normal(gen, (N, H, dk, dv), torch.float32) if case["ds"] else None
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return {"linattn_fwd": _fwd, "linattn_step": _step, "linattn_bwd": _bwd,
            "block_norm_fwd": _norm_fwd, "block_norm_bwd": _norm_bwd}[s["op"]](s)


def _rows(s):
    """For packed rows as [N, longest]: the row of every place, and whether it is one."""
    c = s["case"]
    at = torch.arange(s["longest"], device="cuda")
    if s["cu"] is None:
        row = torch.arange(c["N"], device="cuda")[:, None] * c["T"] + at
        return row, torch.ones_like(row, dtype=torch.bool)
    cu = s["cu"].long()
    live = at < (cu[1:] - cu[:-1])[:, None]
    return torch.where(live, cu[:-1, None] + at, 0), live


def _padded(x, row, live, H):
    """[rows, Hx, d] as fp32 [N, H, longest, d]: zero behind each sequence's last row."""
    y = x.float()[row] * live[..., None, None]
    return y.repeat_interleave(H // x.shape[1], 2).transpose(1, 2)


def _mix(x, y, z, log_decay, length, start):
    """For every head, with lam its decay, n its tokens:
    out_t = sum_{i<=t} lam^(t-i) (x_t.y_i) z_i + lam^(t+1) x_t start, and the end state
    sum_i lam^(n-1-i) y_i z_i^T + lam^n start. Chunks side by side, the states between them
    by one product over the chunks."""
    N, H, T, _ = x.shape
    C = PLAIN_CHUNK
    nc = (T + C - 1) // C
    x, y, z = (torch.nn.functional.pad(a, (0, 0, 0, nc * C - T)).reshape(N, H, nc, C, a.shape[-1]) for a in (x, y, z))
    ld = log_decay.double()[:, None, None]
    i = torch.arange(C, device="cuda", dtype=torch.float64)
    c = torch.arange(nc, device="cuda", dtype=torch.float64)
    lower = lambda n: torch.where(n[:, None] >= n, n[:, None] - n, math.inf)  # noqa: E731
    power = lambda n: torch.where(torch.isinf(n), 0.0, torch.exp(ld * torch.where(torch.isinf(n), 0.0, n)))  # noqa: E731
    inside = power(lower(i)).float()                                                      # [H, C, C]
    after = torch.exp(ld[:, 0] * (C - 1 - i)).float()                                     # [H, C]
    scores = x @ y.transpose(-1, -2) * inside[:, None]
    out = scores @ z
    own_state = (y * after[:, None, :, None]).transpose(-1, -2) @ z                       # [N, H, nc, dx, dz]
    between = power(lower(c - 1) * C - C).float().tril(-1)                                # lam^(C (c - c' - 1))
    flat = own_state.flatten(-2)
    entering = between @ flat
    if start is not None:
        entering = entering + torch.exp(ld[:, 0] * (c * C)).float()[..., None] * start.flatten(-2)[:, :, None]
    entering = entering.reshape(own_state.shape)
    out = out + torch.exp(ld[:, 0] * (i + 1)).float()[:, None, :, None] * (x @ entering)
    # the end state: every place's decay to its sequence's last token
    to_end = length.double()[:, None, None] - 1 - torch.arange(nc * C, device="cuda", dtype=torch.float64)  # [N, 1, nc C]
    w = torch.where(to_end >= 0, torch.exp(ld[:, 0] * to_end.clamp_min(0)), 0.0).float()
    end = (y.reshape(N, H, nc * C, -1) * w[..., None]).transpose(-1, -2) @ z.reshape(N, H, nc * C, -1)
    if start is not None:
        end = end + torch.exp(ld * length.double()[:, None, None, None]).float() * start
    return out.reshape(N, H, nc * C, -1)[:, :, :T], end


def _unpad(x, s, row, live, heads, dtype):
    """fp32 [N, H, longest, d] back to packed rows; heads that share one are summed."""
    x = x.transpose(1, 2)[live]
    return x.reshape(x.shape[0], heads, -1, x.shape[-1]).sum(2).to(dtype)


def _lengths(s):
    c = s["case"]
    if s["cu"] is None:
        return torch.full((c["N"],), c["T"], device="cuda")
    return s["cu"][1:] - s["cu"][:-1]


def _fwd(s):
    c = s["case"]
    if own:
        from gated_delta_rule_03_gb300 import linattn_fwd
        o, S = linattn_fwd(s["q"], s["k"], s["v"], s["log_decay"], S0=s["S0"], cu_seqlens=s["cu"],
                           num_seqs=c["N"], scale=c["scale"])
        return {"o": o, "S": S}
    row, live = _rows(s)
    q, k, v = (_padded(s[n], row, live, c["H"]) for n in "qkv")
    o, S = _mix(q, k, v, s["log_decay"], _lengths(s), s["S0"])
    return {"o": _unpad(o * c["scale"], s, row, live, c["H"], s["q"].dtype), "S": S}


def _step(s):
    c = s["case"]
    if own:
        from gated_delta_rule_03_gb300 import linattn_step
        return {"o": linattn_step(s["q"], s["k"], s["v"], s["log_decay"], s["S"], scale=c["scale"]), "S": s["S"]}
    q, k, v = (s[n].float().repeat_interleave(c["H"] // s[n].shape[1], 1) for n in "qkv")
    S = s["S"]
    S.mul_(torch.exp(s["log_decay"])[:, None, None]).add_(k[..., None] * v[..., None, :])
    o = (q[..., None, :] @ S)[..., 0, :] * c["scale"]
    return {"o": o.to(s["q"].dtype), "S": S}


def _bwd(s):
    c = s["case"]
    if own:
        from gated_delta_rule_03_gb300 import linattn_bwd
        dq, dk, dv, dS0 = linattn_bwd(s["do"], s["q"], s["k"], s["v"], s["log_decay"], S0=s["S0"],
                                      dS_final=s["dS"], cu_seqlens=s["cu"], num_seqs=c["N"], scale=c["scale"])
        return {"dq": dq, "dk": dk, "dv": dv, **({} if dS0 is None else {"dS0": dS0})}
    row, live = _rows(s)
    q, k, v = (_padded(s[n], row, live, c["H"]) for n in "qkv")
    do = _padded(s["do"], row, live, c["H"]) * c["scale"]
    ld, n = s["log_decay"], _lengths(s)
    turned = lambda a: None if a is None else a.transpose(-1, -2)  # noqa: E731
    dq, _ = _mix(do, v, k, ld, n, turned(s["S0"]))
    # the other two run from the last token to the first: every sequence's rows turned round
    at = torch.arange(s["longest"], device="cuda")
    back = torch.where(live, n[:, None].long() - 1 - at, at)[:, None, :, None]
    flip = lambda a: torch.gather(a, 2, back.expand(a.shape))  # noqa: E731
    q, k, v, do = flip(q), flip(k), flip(v), flip(do)
    # lam^t instead of lam^(t+1) for the state that enters: what dS weighs in is kept apart
    dv, A = _mix(k, q, do, ld, n, None)
    dk, _ = _mix(v, do, q, ld, n, None)
    lam = torch.exp(ld.double())[:, None, None]
    dS0 = (lam * A).float()
    if s["dS"] is not None:
        w = torch.exp(ld.double()[:, None] * at).float()[..., None]
        dv = dv + w * (k @ s["dS"])
        dk = dk + w * (v @ turned(s["dS"]))
        dS0 = dS0 + torch.exp(ld.double()[:, None, None] * n.double()[:, None, None, None]).float() * s["dS"]
    dk, dv = flip(dk), flip(dv)
    dt = s["q"].dtype
    out = {"dq": _unpad(dq, s, row, live, c["Hq"], dt), "dk": _unpad(dk, s, row, live, c["Hk"], dt),
           "dv": _unpad(dv, s, row, live, c["Hv"], dt)}
    return {**out, "dS0": dS0} if s["S0"] is not None else out


EPS = 1e-6


def _act(kind, g):
    """The gate's value and its derivative."""
    if kind == "identity":
        return g, torch.ones_like(g)
    sig = torch.sigmoid(g)
    return (sig, sig * (1 - sig)) if kind == "sigmoid" else (g * sig, sig * (1 + g * (1 - sig)))


def _norm_fwd(s):
    c = s["case"]
    if own:
        from gated_delta_rule_03_gb300 import block_norm_fwd
        x_out, h = block_norm_fwd(s["x"], s["y"], gate=s["gate"], act=c["act"], w_post=s["w_post"],
                                  w_pre=s["w_pre"], post_norm=c["post"], pre_norm=c["pre"],
                                  res_scale=c["res_scale"], eps=EPS)
        return {"x": x_out, **({} if h is None else {"h": h})}
    r = s["y"].float()
    if c["post"]:
        r = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS) * s["w_post"]
    if s["gate"] is not None:
        r = r * _act(c["act"], s["gate"].float())[0]
    x = s["x"].float() + c["res_scale"] * r
    out = {"x": x.to(s["x"].dtype)}
    if c["pre"]:
        out["h"] = (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["w_pre"]).to(s["y"].dtype)
    return out


def _norm_bwd(s):
    c = s["case"]
    if own:
        from gated_delta_rule_03_gb300 import block_norm_bwd
        g = block_norm_bwd(s["dx_out"], s["dh"], s["x"], s["y"], gate=s["gate"], act=c["act"],
                           w_post=s["w_post"], w_pre=s["w_pre"], post_norm=c["post"],
                           pre_norm=c["pre"], res_scale=c["res_scale"], eps=EPS)
        return {n: t for n, t in zip(("dx", "dy", "dgate", "dw_post", "dw_pre"), g) if t is not None}
    out, dx = {}, s["dx_out"].float()
    if c["pre"]:
        x, dh = s["x"].float(), s["dh"].float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        n, m = x * r, dh * s["w_pre"]
        out["dw_pre"] = (dh * n).sum(0)
        dx = dx + r * (m - n * (m * n).mean(-1, keepdim=True))
    out["dx"] = dx.to(s["x"].dtype)
    y, dz = s["y"].float(), c["res_scale"] * dx
    if c["post"]:
        r = torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)
        n = y * r
        t = n * s["w_post"]
    else:
        t = y
    if s["gate"] is not None:
        a, da = _act(c["act"], s["gate"].float())
        dg = dz * t * da
        out["dgate"] = (dg if c["gate"] == "rows" else dg.sum(0, keepdim=True)).to(s["gate"].dtype)
        dz = dz * a
    if c["post"]:
        out["dw_post"] = (dz * n).sum(0)
        m = dz * s["w_post"]
        dz = r * (m - n * (m * n).mean(-1, keepdim=True))
    out["dy"] = dz.to(s["y"].dtype)
    return out


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"].startswith("block_norm"):
        n, D = case["rows"], case["D"]
        e, xe = (2 if case[t] == "bf16" else 4 for t in ("dtype", "x_dtype"))
        gate = {"rows": n, "one": 1, "none": 0}[case["gate"]]
        w = 4 * D * (case["post"] + case["pre"])
        if case["op"] == "block_norm_fwd":
            return {"bytes": n * D * (e + 2 * xe + (e if case["pre"] else 0)) + gate * D * e + w, "flops": 14 * n * D}
        # reads y, dx_out, with the pre-norm x and dh, the gate; writes dx, dy, the gate's
        return {"bytes": n * D * (2 * e + 2 * xe + ((e + xe) if case["pre"] else 0)) + 2 * gate * D * e + 2 * w,
                "flops": 30 * n * D}
    H, dk, dv, N = case["H"], case["dk"], case["dv"], case["N"]
    e = 2 if case["dtype"] == "bf16" else 4
    qkv = (case["Hq"] + case["Hk"]) * dk + case["Hv"] * dv
    state = 4 * N * H * dk * dv
    if case["op"] == "linattn_step":
        return {"bytes": 2 * state + N * e * (qkv + H * dv) + 4 * H, "flops": 5 * N * H * dk * dv}
    T = sum(_lens(case))
    if case["op"] == "linattn_fwd":  # the recurrence: write k v^T, decay, read q
        return {"bytes": T * e * (qkv + H * dv) + state * (1 + case["s0"]) + 4 * H, "flops": 5 * T * H * dk * dv}
    # the state again, dq, the adjoint state, dk, dv
    return {"bytes": T * e * (2 * qkv + H * dv) + state * (2 * case["s0"] + case["ds"]) + 4 * H,
            "flops": 12 * T * H * dk * dv}


# ------------------------------------------------------------------ 64 bits, token by token

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("block_norm"):
        return _exact_norm(case, s)
    H = case["H"]
    lam = s["log_decay"].double().exp()[:, None, None]
    wide = lambda a: a.double().repeat_interleave(H // a.shape[1], 1)  # noqa: E731
    if case["op"] == "linattn_step":
        S = s["S"].double() * lam + torch.einsum("nhk,nhv->nhkv", wide(s["k"]), wide(s["v"]))
        return {"o": torch.einsum("nhkv,nhk->nhv", S, wide(s["q"])) * case["scale"], "S": S}
    lens = _lens(case)
    if sum(lens) == 0:
        return None
    ends = np.cumsum(lens)
    starts = ends - lens
    # sequences in order of length, so that the ones with a token t are the first of them
    order = np.argsort(-np.asarray(lens), kind="stable")
    sizes = np.asarray(lens)[order]
    first = torch.tensor(starts[order], device="cuda")
    turn = torch.tensor(order, device="cuda")
    q, k, v = wide(s["q"]), wide(s["k"]), wide(s["v"])
    alive = [int((sizes > t).sum()) for t in range(int(sizes[0]))]
    S = torch.zeros(case["N"], H, case["dk"], case["dv"], dtype=torch.float64, device="cuda")
    if s["S0"] is not None:
        S += s["S0"].double()[turn]
    if case["op"] == "linattn_fwd":
        o = torch.zeros(sum(lens), H, case["dv"], dtype=torch.float64, device="cuda")
        for t, n in enumerate(alive):
            r, P = first[:n] + t, S[:n]
            P.mul_(lam).addcmul_(k[r][..., None], v[r][..., None, :])
            o[r] = (q[r][..., None, :] @ P)[..., 0, :]
        back = torch.empty_like(S)
        back[turn] = S
        return {"o": o * case["scale"], "S": back}
    do = s["do"].double() * case["scale"]
    dq, dk, dv = (torch.zeros_like(a) for a in (q, k, v))
    for t, n in enumerate(alive):
        r, P = first[:n] + t, S[:n]
        P.mul_(lam).addcmul_(k[r][..., None], v[r][..., None, :])
        dq[r] = (P @ do[r][..., None])[..., 0]
    D = torch.zeros_like(S)
    if s["dS"] is not None:
        D += s["dS"].double()[turn]
    for t in range(len(alive) - 1, -1, -1):  # D: the gradient of the state after token t
        n = alive[t]
        r, P = first[:n] + t, D[:n]
        P.addcmul_(q[r][..., None], do[r][..., None, :])
        dk[r] = (P @ v[r][..., None])[..., 0]
        dv[r] = (k[r][..., None, :] @ P)[..., 0, :]
        P.mul_(lam)
    share = lambda a, heads: a.reshape(a.shape[0], heads, -1, a.shape[-1]).sum(2)  # noqa: E731
    out = {"dq": share(dq, case["Hq"]), "dk": share(dk, case["Hk"]), "dv": share(dv, case["Hv"])}
    if s["S0"] is not None:
        out["dS0"] = torch.empty_like(D)
        out["dS0"][turn] = D
    return out


def _exact_norm(case, s):
    """The forward sum in 64 bits; its gradients by torch's own differentiation of it."""
    leaf = lambda a: None if a is None else a.double().requires_grad_()  # noqa: E731
    x, y, g, wp, wn = (leaf(s[n]) for n in ("x", "y", "gate", "w_post", "w_pre"))
    rms = lambda a: a / (a.square().mean(-1, keepdim=True) + EPS).sqrt()  # noqa: E731
    act = {"identity": lambda a: a, "sigmoid": lambda a: 1 / (1 + (-a).exp()),
           "silu": lambda a: a / (1 + (-a).exp())}[case["act"]]
    r = y if wp is None else rms(y) * wp
    r = r if g is None else r * act(g)
    if case["op"] == "block_norm_fwd":
        total = x + case["res_scale"] * r
        return {"x": total.detach(), **({} if wn is None else {"h": (rms(total) * wn).detach()})}
    # x is the sum already: the gradient of it from the norm, then on to the block's parts
    grads = {}
    dx = s["dx_out"].double()
    if wn is not None:
        gx, grads["dw_pre"] = torch.autograd.grad(rms(x) * wn, (x, wn), s["dh"].double())
        dx = dx + gx
    grads["dx"] = dx
    names = [(n, a) for n, a in (("dy", y), ("dgate", g), ("dw_post", wp)) if a is not None]
    for (n, _), d in zip(names, torch.autograd.grad(r, [a for _, a in names], case["res_scale"] * dx)):
        grads[n] = d
    return grads
