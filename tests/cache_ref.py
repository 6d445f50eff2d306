"""The operators around a paged 8-bit cache, from their definitions in 64 bits, and what their
arithmetic may be off by."""
import math

import torch

F64 = torch.float64
TOP = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def f64(t):
    return None if t is None else t.detach().to(F64)


# ------------------------------------------------------------------ rotary positions

def rotary(x, positions, rates, neighbours, amplitude, back=False):
    """x [T, heads, d] in 64 bits: pairs turned by exact fractions of a turn."""
    rot = 2 * rates.numel()
    turns = [[(int(p) * int(r)) % 2 ** 64 / 2.0 ** 64 for r in rates.tolist()] for p in positions.tolist()]
    angle = 2 * math.pi * torch.tensor(turns, dtype=F64).reshape(len(turns), 1, rot // 2) * (-1 if back else 1)
    cos, sin = amplitude * angle.cos(), amplitude * angle.sin()
    y = x.detach().cpu().to(F64).clone()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if neighbours else (slice(0, rot // 2), slice(rot // 2, rot))
    p, q = y[..., a].clone(), y[..., b].clone()
    y[..., a], y[..., b] = p * cos - q * sin, p * sin + q * cos
    return y


# ------------------------------------------------------------------ pages

def plan(table, kv_lens, free, count, page, q_lens, rows):
    """The plan of lists, request by request; the table is a list of rows, changed in place."""
    n, width = len(table), len(table[0])
    kv, start, cu, positions, slots = list(kv_lens), [], [0], [0] * rows, [-1] * rows
    end = asked = used = 0
    for i in range(n):
        q = max(0, q_lens[i])
        at, end = end, end + q
        have = -(-kv[i] // page) if kv[i] >= 0 else 0
        need = -(-(kv[i] + q) // page) - have
        fits = kv[i] >= 0 and end <= rows and have + need <= width
        if fits:
            asked += need
        granted = fits and (need == 0 or asked <= count)
        if granted:
            for j in range(need):
                table[i][have + j] = free[count - 1 - used - j]
            used += need
            for j in range(q):
                positions[at + j] = kv[i] + j
                slots[at + j] = table[i][(kv[i] + j) // page] * page + (kv[i] + j) % page
        start.append(kv[i] if granted else -1)
        kv[i] += q if granted else 0
        cu.append(min(end, rows))
    return dict(table=table, kv_lens=kv, free_count=[count - used], cu_q=cu, start=start, positions=positions, slots=slots)


# ------------------------------------------------------------------ the cache

def least_scale(amax, top):
    k = -60
    while k < 60 and amax > top * 2.0 ** k:
        k += 1
    return 2.0 ** k


def encode(x, codes):
    """Codes of scaled entries, by torch's own rounding to nearest even."""
    x = x.clamp(-TOP[codes], TOP[codes])
    return x.round().to(torch.int8) if codes == torch.int8 else x.to(torch.float32).to(codes)


def append(x, slots, cache, scale):
    """One tensor's rows x [T, heads, d] into cache and scale (CPU), run by run."""
    pages, heads, page, d = cache.shape
    x, slots = x.detach().cpu().to(F64), slots.tolist()
    t = 0
    while t < len(slots):
        s = slots[t]
        if not 0 <= s < pages * page:
            t += 1
            continue
        n = 1
        while t + n < len(slots) and slots[t + n] == s + n and (s + n) % page:
            n += 1
        p, off = s // page, s % page
        for h in range(heads):
            run = x[t:t + n, h]
            old = float(scale[p, h]) if off else 0.0
            if not bool(torch.isfinite(run).all()) or old != old:
                scale[p, h] = math.nan
                cache[p, h, off:off + n] = encode(torch.zeros_like(run), cache.dtype)
                continue
            new = max(least_scale(float(run.abs().max()), TOP[cache.dtype]), old)
            if off and 0 < old < new:
                cache[p, h, :off] = encode(cache[p, h, :off].to(F64) * (old / new), cache.dtype)
            scale[p, h] = new
            cache[p, h, off:off + n] = encode(run / new, cache.dtype)
        t += n


# ------------------------------------------------------------------ attention

def attend(q, k_cache, v_cache, k_scale, v_scale, table, kv_lens, cu, scale, softcap=0.0, slopes=None, causal=True):
    """Per row: outputs, lse, sum_j p_j |v_j| (the size that a weight's relative error counts with), `step`: the
    largest p_j vs_j times sum_j |code_j| (what an equal error of all weights relative to the largest counts
    with), the largest scale sum |q_i k_i| of a token it sees and the largest |s|."""
    T, H, d = q.shape
    pages, Hkv, page, _ = k_cache.shape
    dev = q.device
    o, size, step = (torch.zeros(T, H, d, dtype=F64, device=dev) for _ in range(3))
    lse = torch.full((T, H), -math.inf, dtype=F64, device=dev)
    dots, most = torch.zeros(T, H, dtype=F64, device=dev), torch.zeros(T, H, dtype=F64, device=dev)
    as_numbers = lambda c: c.view(torch.uint8)  # noqa: E731
    for n in range(len(kv_lens)):
        r0, r1, L = cu[n], cu[n + 1], kv_lens[n]
        if r1 == r0 or L == 0:
            continue
        at = table[n, :-(-L // page)].long()

        def whole(codes, sc):
            x = as_numbers(codes)[at].view(codes.dtype).to(F64) * sc[at].to(F64)[..., None, None]
            return x.transpose(0, 1).reshape(Hkv, -1, d)[:, :L].repeat_interleave(H // Hkv, 0)

        k, v = whole(k_cache, k_scale), whole(v_cache, v_scale)
        x = q[r0:r1].to(F64).transpose(0, 1)
        s = scale * x @ k.transpose(1, 2)
        sizes = abs(scale) * x.abs() @ k.abs().transpose(1, 2)
        if softcap:
            s = softcap * torch.tanh(s / softcap)
        away = torch.arange(L - (r1 - r0), L, device=dev)[:, None] - torch.arange(L, device=dev)
        if slopes is not None:
            s = s - slopes.to(F64)[:, None, None] * away.abs()
        seen = (away >= 0) if causal else torch.ones_like(away, dtype=torch.bool)
        live = seen.any(1)
        if not bool(live.any()):
            continue
        s = torch.where(seen, s, -math.inf)
        p = torch.where(seen, torch.exp(s - torch.where(live[:, None], s, 0.0).amax(-1, keepdim=True)), 0.0)
        total = p.sum(-1, keepdim=True)
        p = torch.where(total > 0, p / total, 0.0)
        o[r0:r1] = (p @ torch.where(torch.isnan(v), 0.0, v)).transpose(0, 1)
        size[r0:r1] = (p @ torch.where(torch.isnan(v), 0.0, v).abs()).transpose(0, 1)
        lse[r0:r1] = torch.where(live[:, None], torch.logsumexp(torch.where(live[:, None], s, 0.0), -1).T, -math.inf)
        vs = v_scale[at].to(F64).T.repeat_interleave(page, 1)[:, :L].repeat_interleave(H // Hkv, 0).nan_to_num(0.0)
        code = torch.where(vs[..., None] > 0, v / vs[..., None], 0.0).abs()
        step[r0:r1] = ((p * vs[:, None]).amax(-1, keepdim=True) * (seen.to(F64) @ code)).transpose(0, 1)
        dots[r0:r1] = torch.where(seen, sizes, 0.0).amax(-1).T
        most[r0:r1] = torch.where(seen, s.abs(), 0.0).amax(-1).T
    return dict(o=o, lse=lse, size=size, step=step, dots=dots, most=most)


def attend_bounds(want, dtype, d, longest, softcap=0.0):
    """(bound of o, bound of lse). Scores: d fp32 products and sums, each off by at most 2^-23 of
    the terms' size (a tensor core may cut instead of round), a few more roundings of the score itself, one
    of its sum with log2 of the page's scale (2^-16 and up: at most 16 2^-24); fp32: queries as two fp16
    parts, 2^-22 of each. The cap's tanh is off by 2^-21 of the cap at most. A score's error moves weights
    by as much, each way. Weights: 2^-11 in fp16, 2^-21 in two parts, and not below fp16's
    smallest step, 2^-24: half of it, 2^-25, where the largest is 2^7 at least (it is that when the row's reference
    was last set, and the reference stays), so 2^-32 of the largest. Sums over the tokens in fp32: one rounding for each 16
    tokens and a few for joining parts."""
    fp32 = dtype == torch.float32
    score = (d + 8) * 2.0 ** -23 * want["dots"] + 8 * 2.0 ** -23 * want["most"] + softcap * 2.0 ** -21 + 2.0 ** -20
    if fp32:
        score = score + 2.0 ** -21 * want["dots"]
    sums = (longest / 16 + 64) * 2.0 ** -23
    weight = 2.0 ** -21 if fp32 else 2.0 ** -11
    o = HALF_STEP[dtype] * want["o"].abs() + (weight + sums + 2 * score)[..., None] * want["size"] + 2.0 ** -32 * want["step"]
    lse = score + sums + 2.0 ** -22 * (1 + want["lse"].abs().nan_to_num(posinf=0.0, neginf=0.0))
    return o, lse


def check(name, got, want, bound):
    """Same places that are not finite, the others within the bound."""
    got = got.detach().to(F64)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fine) and torch.equal(got[~fine].nan_to_num(7.0), want[~fine].nan_to_num(7.0)), f"{name}: other places are not finite"
    off = ((got - want).abs() / bound.clamp_min(1e-300))[fine]
    if off.numel():
        assert float(off.max()) <= 1, f"{name}: {float(off.max()):.3g} times the bound"
