"""Linear attention with a constant decay per head in 64 bits, and how far a kernel may be off.

`forward` and `backward` are the definition summed directly: every pair of tokens by its
own power of the decay. They share nothing with the kernels' chunks, segments or states.
Every result comes with `Abs`, the same sum over the absolute values of all its terms: a
rounding of relative size u anywhere in the sum moves the result by u Abs at most.
"""
import numpy as np
import torch

U_BF16, U_F32 = 2.0 ** -8, 2.0 ** -24


def f64(t):
    return None if t is None else t.detach().to("cpu", torch.float64).numpy()


def powers(ld, n):
    """lam^n for an array n >= 0 (lam = 0 for ld = -inf, with lam^0 = 1)."""
    n = np.asarray(n, dtype=np.float64)
    if np.isneginf(ld):
        return (n == 0).astype(np.float64)
    return np.exp(ld * n)


def _pairs(x, y, z, W):
    """sum_i W_ti (x_t.y_i) z_i and the same over absolute values."""
    a = np.abs
    return (W * (x @ y.T)) @ z, (W * (a(x) @ a(y).T)) @ a(z)


def _lower(ld, n):
    d = np.arange(n)[:, None] - np.arange(n)[None, :]
    return np.where(d >= 0, powers(ld, np.maximum(d, 0)), 0.0)


def spans(lens):
    ends = np.cumsum(lens)
    return [(int(e - n), int(e)) for n, e in zip(lens, ends)]


def forward(q, k, v, ld, lens, S0=None, scale=1.0):
    """(o, S, Abs of o, Abs of S); q, k, v [T, heads, d] float64 numpy, ld [H]."""
    H, dk, dv = len(ld), q.shape[2], v.shape[2]
    o, oa = np.zeros((q.shape[0], H, dv)), np.zeros((q.shape[0], H, dv))
    S, Sa = np.zeros((len(lens), H, dk, dv)), np.zeros((len(lens), H, dk, dv))
    for n, (a, b) in enumerate(spans(lens)):
        for h in range(H):
            qq, kk, vv = (t[a:b, h * t.shape[1] // H] for t in (q, k, v))
            L = b - a
            o[a:b, h], oa[a:b, h] = _pairs(qq, kk, vv, _lower(ld[h], L))
            w = powers(ld[h], L - 1 - np.arange(L))[:, None]
            S[n, h], Sa[n, h] = (w * kk).T @ vv, (w * np.abs(kk)).T @ np.abs(vv)
            if S0 is not None:
                wo = powers(ld[h], np.arange(L) + 1)[:, None]
                o[a:b, h] += wo * (qq @ S0[n, h])
                oa[a:b, h] += wo * (np.abs(qq) @ np.abs(S0[n, h]))
                S[n, h] += powers(ld[h], L) * S0[n, h]
                Sa[n, h] += powers(ld[h], L) * np.abs(S0[n, h])
    return o * scale, S, oa * abs(scale), Sa


def backward(do, q, k, v, ld, lens, S0=None, dS=None, scale=1.0):
    """{name: (gradient, Abs)} for dq, dk, dv, dS0."""
    H, dk, dv = len(ld), q.shape[2], v.shape[2]
    out = {n: (np.zeros(t.shape), np.zeros(t.shape)) for n, t in (("dq", q), ("dk", k), ("dv", v))}
    out["dS0"] = (np.zeros((len(lens), H, dk, dv)), np.zeros((len(lens), H, dk, dv)))
    a_ = np.abs

    def add(name, rows, h, value, size):
        at = (rows, h * out[name][0].shape[1] // H)
        out[name][0][at] += value
        out[name][1][at] += size

    for n, (a, b) in enumerate(spans(lens)):
        r = slice(a, b)
        for h in range(H):
            qq, kk, vv = (t[r, h * t.shape[1] // H] for t in (q, k, v))
            g, L = do[r, h] * scale, b - a
            W = _lower(ld[h], L)
            add("dq", r, h, *_pairs(g, vv, kk, W))
            add("dk", r, h, *_pairs(vv, g, qq, W.T))
            add("dv", r, h, *_pairs(kk, qq, g, W.T))
            w1 = powers(ld[h], np.arange(L) + 1)[:, None]
            add("dS0", n, h, (w1 * qq).T @ g, (w1 * a_(qq)).T @ a_(g))
            if S0 is not None:
                add("dq", r, h, w1 * (g @ S0[n, h].T), w1 * (a_(g) @ a_(S0[n, h]).T))
            if dS is not None:
                w = powers(ld[h], L - 1 - np.arange(L))[:, None]
                add("dk", r, h, w * (vv @ dS[n, h].T), w * (a_(vv) @ a_(dS[n, h]).T))
                add("dv", r, h, w * (kk @ dS[n, h]), w * (a_(kk) @ a_(dS[n, h])))
                add("dS0", n, h, powers(ld[h], L) * dS[n, h], powers(ld[h], L) * a_(dS[n, h]))
    return out


def f32_terms(T, dk, dv, group=1):
    """Roundings of 2^-24 that one term of a result meets at most in fp32 arithmetic: the
    scores (d_k or d_v products), the sum over the chunk's tokens and over the state's rows,
    the state's own sum over all tokens, the group's sum; a power of the decay is off by
    |n ln lam| + 4 of them, and below e^-100 it is nothing; a state, a scale, a weight."""
    return 2 * max(dk, dv) + 128 + T + group + 104 + 16


def allowed(want, Abs, dtype, terms):
    """How far an output may be off. bf16: its own rounding; besides, the tensor-core kernel
    rounds the scores and the state's copy to bf16, each once, and a term goes through one of
    the two: u Abs together. (The state's sum from two bf16 halves is off by u^2 Abs, the
    rounding of what is off already by u^2: 2 % of u covers both, and the fp32 roundings are
    counted.)"""
    f32 = terms * U_F32 * Abs + 1e-30
    if dtype == torch.float32:
        return f32 + U_F32 * np.abs(want)
    return 1.02 * U_BF16 * (np.abs(want) + Abs) + f32


def check(name, got, want, Abs, dtype, terms):
    got = f64(got)
    assert got.shape == want.shape, name
    assert np.isfinite(got).all(), f"{name}: not finite"
    off, may = np.abs(got - want), allowed(want, Abs, dtype, terms)
    worst = float((off / may).max()) if off.size else 0.0
    assert worst <= 1.0, f"{name}: {worst:.3g} of what is allowed"
