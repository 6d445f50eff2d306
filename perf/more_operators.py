"""Measured calls of the operators around a paged cache of 8-bit keys and values.

Operators
  rotary_fwd    rotary positions of queries and keys: halves or neighbours as pairs, part of
                the head, frequencies and amplitude scaled for long contexts
  rotary_bwd    its gradients (the turn back)
  page_plan     pages for the new tokens of every request: block table, token offsets, each
                token's position and slot in the cache
  cache_append  keys and values put into their slots, held in 8 bits with one scale (a power
                of two) for each page and head; a page that was begun is rescaled if needed
  cache_attn    softmax attention of prompts, pieces of prompts and single tokens over that
                cache, with an optional cap of the scores and a bias by distance

`own` false: the plain form (elementary torch operations in 32 bits, angles in 64).
`own` true: the calls of gated_delta_rule_03_gb300.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
TOP = {"e4m3": 448.0, "int8": 127.0}
LEAST, MOST = -60, 60   # exponents of the scales
BASE = 10000.0


# ------------------------------------------------------------------ the cases

def listed():
    rot = dict(op="rotary_fwd", T=1, Hq=16, Hk=4, d=128, rot=128, neighbours=False, far=4096, factor=1.0,
               dtype="bf16", fused=False)
    plan = dict(op="page_plan", N=1, lo=1, hi=1, lens=1, past=1, page=64, rows=0)
    app = dict(op="cache_append", N=1, lo=1, hi=1, lens=1, past=0, page=64, Hkv=8, d=128, dtype="bf16", codes="e4m3")
    att = dict(op="cache_attn", N=1, T=1, lo=0, hi=0, lens=1, past_lo=0, past_hi=0, page=64, H=16, Hkv=4, d=128,
               dtype="bf16", codes="e4m3", cap=0.0, slopes=False, causal=True)
    return [
        # the next token of a full serving batch
        dict(rot, name="rotary_step_bf16", T=256, Hq=32, Hk=8, far=8192),
        # a batch of four prompts of 4,096 tokens, views of one projection, frequencies of a
        # context stretched by eight
        dict(rot, name="rotary_prompts_bf16", T=16384, far=131072, factor=8.0, fused=True),
        # gradients of a training step, a quarter of wide fp32 heads, neighbours as pairs, an odd length
        dict(rot, name="rotary_bwd_part_fp32", op="rotary_bwd", T=4099, Hq=8, Hk=2, d=256, rot=64,
             neighbours=True, dtype="f32"),
        # slots for the next token of a full serving batch, short pages
        dict(plan, name="plan_step", N=256, past=8192, page=16),
        # slots for packed prompts of odd lengths
        dict(plan, name="plan_prompts", N=33, lo=100, hi=3000, lens=3, past=2000),
        # the next token of that batch goes into pages of 16, some of them rescaled
        dict(app, name="append_step_int8", N=256, past=8192, page=16, codes="int8"),
        # eight packed prompts of odd lengths
        dict(app, name="append_prompts_e4m3", N=8, lo=512, hi=8192, lens=2, past=100, Hkv=4),
        # one sequence's next token behind a long document
        dict(att, name="attn_step_long", past_lo=131071, past_hi=131071, H=32, Hkv=8),
        # the next token of a full serving batch, odd lengths
        dict(att, name="attn_step_batch", N=256, past_lo=511, past_hi=8191, page=16, H=32, Hkv=8),
        # a batch of four prompts of 4,096 tokens
        dict(att, name="attn_prompts", N=4, T=4096),
        # a piece of a prompt behind a long cache: wide heads, capped scores, int8
        dict(att, name="attn_piece_capped_int8", T=1000, past_lo=32768, past_hi=32768, H=16, Hkv=2, d=256,
             codes="int8", cap=50.0),
        # a small fp32 model with a bias by distance: short prompts of odd lengths, latency
        dict(att, name="attn_small_fp32", N=3, T=0, lo=1, hi=60, lens=4, past_lo=0, past_hi=300, page=16,
             H=4, Hkv=4, d=64, dtype="f32", slopes=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary_fwd", "rotary_bwd", "page_plan", "cache_append", "cache_append", "cache_attn",
                     "cache_attn", "cache_attn", "cache_attn"])
    page = rng.choice([16, 32, 64, 128])
    if op.startswith("rotary"):
        dtype = rng.choice(["bf16", "bf16", "f32"])
        Hk, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 96, 128, 256])
        Hq = Hk * rng.choice([1, 2, 3, 4, 8])
        return dict(op=op, T=_log_int(rng, 1, max(2, (1 << 25) // (Hq * d))), Hq=Hq, Hk=Hk, d=d,
                    rot=rng.choice([d, d, d // 2, d // 4, d - 6]), neighbours=rng.random() < 0.5,
                    far=_log_int(rng, 100, 1 << 20), factor=rng.choice([1.0, 1.0, 4.0, 16.0]), dtype=dtype,
                    fused=rng.random() < 0.5)
    if op == "page_plan":
        N = _log_int(rng, 1, 1024)
        hi = _log_int(rng, 1, (1 << 16) // N)
        return dict(op=op, N=N, lo=rng.randrange(0, hi + 1), hi=hi, lens=rng.randrange(1, 1 << 20),
                    past=_log_int(rng, 1, 16384), page=page, rows=rng.choice([0, 0, 7, 1000]))
    if op == "cache_append":
        Hkv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256])
        most = (1 << 24) // (Hkv * d)
        N = _log_int(rng, 1, min(256, most))
        hi = _log_int(rng, 1, max(1, most // N))
        return dict(op=op, N=N, lo=rng.randrange(0, hi + 1), hi=hi, lens=rng.randrange(1, 1 << 20),
                    past=_log_int(rng, 1, 4096), page=page, Hkv=Hkv, d=d, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    codes=rng.choice(["e4m3", "int8"]))
    Hkv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 256])
    H = Hkv * rng.choice([1, 2, 3, 4, 8, 16])
    case = dict(op=op, T=1, lo=0, hi=0, lens=rng.randrange(1, 1 << 20), page=page, H=H, Hkv=Hkv, d=d,
                dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]), codes=rng.choice(["e4m3", "int8"]),
                cap=rng.choice([0.0, 0.0, 30.0]), slopes=rng.random() < 0.3, causal=rng.random() < 0.8)
    if rng.random() < 0.5:  # single tokens: the cache's bytes are the cost
        most = (1 << 29) // (Hkv * d)
        case["N"] = _log_int(rng, 1, min(256, most // 16))
        far = _log_int(rng, 1, min(131072, most // case["N"]))
    else:                   # prompts or pieces of them: pairs of a query and a key are
        pairs = (1 << 28) // (H * d // 64)
        case["T"] = _log_int(rng, 2, min(4096, int(math.sqrt(pairs))))
        case["N"] = _log_int(rng, 1, max(1, min(64, pairs // case["T"] ** 2)))
        far = _log_int(rng, 1, max(1, min(65536, pairs // (case["T"] * case["N"]) - case["T"])))
        if rng.random() < 0.5:  # odd lengths
            case.update(T=0, hi=case["T"], lo=rng.randrange(0, case["T"] + 1))
    case["past_hi"] = far if rng.random() < 0.7 else 0
    case["past_lo"] = rng.randrange(0, case["past_hi"] + 1)
    return case


def _between(seed, lo, hi, n):
    return np.random.RandomState(seed).randint(lo, hi + 1, n).astype(np.int64)


def _new(case):
    """New tokens of every request."""
    if case.get("T"):
        return np.full(case["N"], case["T"], dtype=np.int64)
    lens = _between(case["lens"], case["lo"], case["hi"], case["N"])
    lens[0] += lens.sum() == 0
    return lens


def _past(case):
    """Tokens that every request has in the cache before."""
    if case["op"] == "cache_attn":
        return _between(case["lens"] + 1, case["past_lo"], case["past_hi"], case["N"])
    return _between(case["lens"] + 1, 0, case["past"], case["N"])


# ------------------------------------------------------------------ inputs

def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _ints(a, dtype=torch.int32):
    return torch.tensor(a, dtype=dtype, device="cuda")


def _offsets(lens):
    return _ints(np.concatenate([[0], np.cumsum(lens)]))


def _frequencies(case):
    """Radians per position of every pair, in 64 bits. A context stretched by `factor`: pairs
    that turn less than once over 4,096 tokens are slowed by it, those that turn more than 32
    times are left, a ramp between; the amplitude grows with its logarithm."""
    rot, factor = case["rot"], case["factor"]
    f = BASE ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    keep = np.clip((4096 * f / (2 * math.pi) - 1) / (32 - 1), 0, 1)
    return f * keep + f / factor * (1 - keep), (1.0 if factor == 1 else 0.1 * math.log(factor) + 1.0)


def _turns(f):
    """Turns per position in steps of 2^-64, as 64-bit integers."""
    whole = [round(x / (2 * math.pi) * 2 ** 64) % 2 ** 64 for x in f.tolist()]
    return _ints([x - 2 ** 64 if x >= 2 ** 63 else x for x in whole], torch.int64)


def _table(gen, pages, N, width, spare):
    """A block table whose first pages[n] entries of row n are pages of the cache in random
    order, -1 behind them; the pages that are left."""
    total = int(pages.sum()) + spare
    order = torch.randperm(total, generator=gen, device="cuda").int()
    table = torch.full((N, width), -1, dtype=torch.int32, device="cuda")
    col = torch.arange(width, device="cuda")[None]
    held = _ints(pages, torch.int64)[:, None]
    at = (torch.cumsum(held, 0) - held) + col
    table = torch.where(col < held, order[at.clamp(max=total - 1)], table)
    return table, order[int(pages.sum()):].contiguous(), total


def _cache(gen, case, pages):
    """Codes and scales of a cache in use, for keys or values."""
    shape = (pages, case["Hkv"], case["page"], case["d"])
    if case["codes"] == "int8":
        c = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0, 32, generator=gen)
        c = c.round_().clamp_(-127, 127).to(torch.int8)
        mid = -5
    else:
        c = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0, 90, generator=gen)
        c = c.clamp_(-448, 448).to(torch.float8_e4m3fn)
        mid = -6.5
    return c, torch.exp2(torch.round(mid + 0.6 * _normal(gen, shape[:2], torch.float32)))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case=case, op=case["op"])
    if case["op"].startswith("rotary"):
        T, Hq, Hk, d, dt = case["T"], case["Hq"], case["Hk"], case["d"], DTYPES[case["dtype"]]
        s["q"], s["k"] = _normal(gen, (T, Hq, d), dt), _normal(gen, (T, Hk, d), dt)
        if case["fused"]:  # views of one projection's rows: queries, keys, values
            w = torch.cat([s["q"].flatten(1), s["k"].flatten(1), s["k"].flatten(1)], 1)
            s["q"], s["k"] = w[:, :Hq * d].view(T, Hq, d), w[:, Hq * d:(Hq + Hk) * d].view(T, Hk, d)
        s["pos"] = torch.randint(0, case["far"], (T,), generator=gen, device="cuda", dtype=torch.int32)
        f, s["amplitude"] = _frequencies(case)
        s["freq"], s["rates"] = torch.tensor(f, device="cuda"), _turns(f)
        return s
    N, page = case["N"], case["page"]
    new, past = _new(case), _past(case)
    s["rows"] = int(new.sum()) + case.get("rows", 0)
    old_pages, all_pages = -(-past // page), -(-(past + new) // page)
    width = max(1, int(all_pages.max()))
    if case["op"] == "page_plan":
        s["q_lens"], s["kv_lens"] = _ints(new), _ints(past)
        s["table"], s["free"], _ = _table(gen, old_pages, N, width, int((all_pages - old_pages).sum()) + 5)
        s["count"] = _ints([s["free"].numel()])
        return s
    s["table"], left, pages = _table(gen, all_pages, N, width, 3)
    s["spare"] = left[-1].long()  # a page of no request
    s["cu"] = _offsets(new)
    s["k_cache"], s["k_scale"] = _cache(gen, case, pages)
    s["v_cache"], s["v_scale"] = _cache(gen, case, pages)
    dt, d = DTYPES[case["dtype"]], case["d"]
    if case["op"] == "cache_append":
        # channels of unlike size, now and then a large token: pages differ in scale
        s["k"], s["v"] = ((_normal(gen, (s["rows"], case["Hkv"], d), torch.float32)
                           * torch.exp(0.5 * _normal(gen, (d,), torch.float32))
                           * torch.exp(0.3 * _normal(gen, (s["rows"], 1, 1), torch.float32))).to(dt) for _ in "kv")
        s["start"] = _ints(past)
        of = np.repeat(np.arange(N), new)
        pos = _ints(np.arange(s["rows"]) - np.repeat(np.cumsum(new) - new, new) + past[of], torch.int64)
        s["slots"] = (s["table"][_ints(of, torch.int64), pos // page] * page + pos % page).int()
        return s
    s["kv_lens"] = _ints(past + new)
    s["q"] = 1.5 * _normal(gen, (s["rows"], case["H"], d), torch.float32)
    s["q"] = s["q"].to(dt)
    s["max_q"], s["scale"] = max(1, int(new.max())), d ** -0.5
    H = case["H"]
    s["slopes"] = None
    if case["slopes"]:
        s["slopes"] = torch.exp2(-8 * (torch.arange(H, device="cuda", dtype=torch.float32) + 1) / H)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return {"rotary_fwd": _rotary, "rotary_bwd": _rotary, "page_plan": _plan, "cache_append": _append,
            "cache_attn": _attn}[s["op"]](s)


def _turn(x, cos, sin, rot, neighbours):
    y = x.float()
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if neighbours else (y[..., :rot // 2], y[..., rot // 2:rot])
    pair = (a * cos - b * sin, a * sin + b * cos)
    turned = torch.stack(pair, -1).flatten(-2) if neighbours else torch.cat(pair, -1)
    return torch.cat([turned, y[..., rot:]], -1).to(x.dtype)


def _rotary(s):
    c = s["case"]
    back = s["op"] == "rotary_bwd"
    if own:
        from gated_delta_rule_03_gb300 import rotary_bwd, rotary_fwd
        q, k = (rotary_bwd if back else rotary_fwd)(s["q"], s["k"], s["pos"], s["rates"], neighbours=c["neighbours"],
                                                    amplitude=s["amplitude"])
        return {"q": q, "k": k}
    angle = s["pos"].double()[:, None, None] * s["freq"]
    cos, sin = (s["amplitude"] * torch.cos(angle)).float(), (s["amplitude"] * torch.sin(angle)).float()
    return {n: _turn(s[n], cos, -sin if back else sin, c["rot"], c["neighbours"]) for n in "qk"}


def _plan(s):
    page, rows = s["case"]["page"], s["rows"]
    if own:
        from gated_delta_rule_03_gb300 import page_plan
        p = page_plan(s["table"], s["kv_lens"], s["free"], s["count"], page, q_lens=s["q_lens"], rows=rows)
        return {"table": s["table"], "kv_lens": p.kv_lens, "count": p.free_count, "cu": p.cu_q,
                "start": p.start, "positions": p.positions, "slots": p.slots}
    q, start, count = s["q_lens"].long(), s["kv_lens"].long(), s["count"].long()
    table, free = s["table"], s["free"]
    end = torch.cumsum(q, 0)
    held = -torch.div(-start, page, rounding_mode="floor")
    need = -torch.div(-(start + q), page, rounding_mode="floor") - held
    need = torch.where((end <= rows) & (held + need <= table.shape[1]), need, table.shape[1] * 2 + 1)
    fits = need <= table.shape[1]
    taken = torch.cumsum(need * fits, 0)
    granted = fits & ((need == 0) | (taken <= count))
    first = (taken - need)[:, None]
    j = torch.arange(table.shape[1], device="cuda")[None] - held[:, None]
    fresh = (j >= 0) & (j < need[:, None]) & granted[:, None]
    table.copy_(torch.where(fresh, free[(count - 1 - first - j).clamp(0, free.numel() - 1)], table))
    used = torch.where(granted & (need > 0), taken, 0).max()
    t = torch.arange(rows, device="cuda")
    n = torch.searchsorted(end, t, right=True)
    live = n < q.numel()
    n = n.clamp(max=q.numel() - 1)
    live &= granted[n]
    pos = torch.where(live, start[n] + t - (end - q)[n], 0)
    slot = table[n, pos // page].long() * page + pos % page
    cu = torch.cat([torch.zeros_like(end[:1]), end]).clamp(max=rows)
    return {"table": table, "kv_lens": torch.where(granted, start + q, start).int(), "count": (count - used).int(),
            "cu": cu.int(), "start": torch.where(granted, start, -1).int(), "positions": pos.int(),
            "slots": torch.where(live, slot, -1).int()}


def _scale_for(amax, top):
    """The least power of two whose `top`-fold reaches amax."""
    m, e = torch.frexp(amax)
    mt, et = math.frexp(top)
    k = (e - et + (m > mt).int()).clamp(LEAST, MOST)
    return torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, k, LEAST))


def _to_codes(x, codes):
    x = x.clamp(-TOP[codes], TOP[codes])
    return (x.round() if codes == "int8" else x).to(CODES[codes]).view(torch.uint8)


def _append(s):
    c = s["case"]
    if own:
        from gated_delta_rule_03_gb300 import cache_append
        cache_append(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        return {n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}
    page, top, N = c["page"], TOP[c["codes"]], c["N"]
    at, off = s["slots"].long() // page, s["slots"].long() % page
    start, col = s["start"].long(), torch.arange(page, device="cuda")
    # the page that every request had begun; else one of its own or none, which stays as it is
    begun = (start % page > 0) & (s["cu"][1:] > s["cu"][:-1])
    some = s["table"][torch.arange(N, device="cuda"), (start // page).clamp(max=s["table"].shape[1] - 1)].long()
    some = torch.where(begun, some, s["spare"])
    pages = s["k_cache"].shape[0]
    touched = torch.zeros(pages, dtype=torch.bool, device="cuda").index_fill_(0, at, True)[:, None]
    kept = torch.zeros(pages, dtype=torch.bool, device="cuda").index_fill_(0, some, True)[:, None]
    out = {}
    for x, n in ((s["k"], "k"), (s["v"], "v")):
        cache, scale = s[n + "_cache"], s[n + "_scale"]
        amax = torch.zeros_like(scale).index_reduce_(0, at, x.float().abs().amax(-1), "amax")
        new = torch.where(touched, torch.maximum(_scale_for(amax, top), torch.where(kept, scale, 0.0)), scale)
        held = cache.view(torch.uint8)[some]
        again = _to_codes(held.view(cache.dtype).float() * (scale / new)[some][..., None, None], c["codes"])
        begun_rows = (begun[:, None] & (col < (start % page)[:, None]))[:, None, :, None]
        cache.view(torch.uint8)[some] = torch.where(begun_rows, again, held)
        codes = _to_codes(x.float() / new[at][..., None], c["codes"])
        cache.view(torch.uint8)[at[:, None], torch.arange(c["Hkv"], device="cuda")[None], off[:, None]] = codes
        scale.copy_(new)
        out[n + "_cache"], out[n + "_scale"] = cache, scale
    return out


def _attn(s):
    c = s["case"]
    if own:
        from gated_delta_rule_03_gb300 import cache_attn
        o, lse = cache_attn(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["kv_lens"],
                            cu_q=None if c["T"] else s["cu"], max_q=s["max_q"], scale=s["scale"], softcap=c["cap"],
                            slopes=s["slopes"], causal=c["causal"], return_lse=True)
        return {"o": o, "lse": lse}
    N, H, Hkv, d, page, Q = c["N"], c["H"], c["Hkv"], c["d"], c["page"], s["max_q"]
    pages = s["table"].long().clamp_min(0)
    S = pages.shape[1] * page

    def whole(codes, scale):
        x = codes.view(torch.uint8)[pages].view(codes.dtype).float() * scale[pages][..., None, None]
        return x.transpose(1, 2).reshape(N, Hkv, 1, S, d)

    cu = s["cu"].long()
    lens, at = cu[1:] - cu[:-1], torch.arange(Q, device="cuda")
    live = at < lens[:, None]
    row = torch.where(live, cu[:-1, None] + at, 0)
    q = s["q"].float()[row.clamp(max=max(0, s["rows"] - 1))].reshape(N, Q, Hkv, H // Hkv, d).permute(0, 2, 3, 1, 4)
    score = (q @ whole(s["k_cache"], s["k_scale"]).transpose(-1, -2)).mul_(s["scale"])  # [N, Hkv, G, Q, S]
    if c["cap"]:
        score.div_(c["cap"]).tanh_().mul_(c["cap"])
    key = torch.arange(S, device="cuda")
    pos = (s["kv_lens"].long() - lens)[:, None] + at                                     # [N, Q]
    away = pos[..., None] - key
    if s["slopes"] is not None:
        score.sub_(s["slopes"].reshape(1, Hkv, -1, 1, 1) * away.abs().float()[:, None, None])
    seen = key < s["kv_lens"].long()[:, None, None]
    if c["causal"]:
        seen = seen & (away >= 0)
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp_min(-1e30)
    w = score.sub_(top).exp_()
    total = w.sum(-1, keepdim=True)
    o = w @ whole(s["v_cache"], s["v_scale"]) / total.clamp_min(1e-30)
    lse = (torch.log(total) + top)[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(N, Q, H, d)[live]
    return {"o": o.to(s["q"].dtype), "lse": lse.permute(0, 3, 1, 2).reshape(N, Q, H)[live]}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"].startswith("rotary"):
        e = 2 if case["dtype"] == "bf16" else 4
        T, heads = case["T"], case["Hq"] + case["Hk"]
        return {"bytes": 2 * T * heads * case["d"] * e + 4 * T + 4 * case["rot"], "flops": 3 * T * heads * case["rot"]}
    new, past, page = _new(case), _past(case), case["page"]
    N, T = case["N"], int(new.sum())
    fresh = int((-(-(past + new) // page) - -(-past // page)).sum())
    if case["op"] == "page_plan":
        # lengths in and out with offsets and starts, pages from the free list into the table, tokens
        return {"bytes": 4 * (5 * N + 1) + 8 * fresh + 8 * (T + case["rows"]), "flops": 0}
    Hkv, d = case["Hkv"], case["d"]
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "cache_append":
        begun = int(((past % page > 0) & (new > 0)).sum())
        return {"bytes": 2 * Hkv * (T * d * (e + 1) + 4 * (fresh + 2 * begun)) + 4 * T, "flops": 4 * T * Hkv * d}
    held = past + new
    # pairs of a query and a key that it sees
    pairs = float((new * past + new * (new + 1) // 2).sum() if case["causal"] else (new * held).sum())
    used = held * (new > 0)
    cache = 2 * Hkv * (int(used.sum()) * d + 4 * int((-(-used // page)).sum()))
    return {"bytes": cache + T * case["H"] * (2 * d * e + 4) + 4 * int((-(-used // page)).sum()) + 8 * N,
            "flops": 4 * pairs * case["H"] * d}


# ------------------------------------------------------------------ 64 bits, from the definitions

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("rotary"):
        return _exact_rotary(case, s)
    if case["op"] == "cache_attn":
        return _exact_attn(case, s)
    if case["op"] == "cache_append":
        return _exact_append(case, s)
    return None  # whole numbers


def _exact_rotary(case, s):
    """Pairs as complex numbers, turned by exp(i angle)."""
    rot, sign = case["rot"], -1 if case["op"] == "rotary_bwd" else 1
    angle = sign * s["pos"].double()[:, None] * s["freq"]
    turn = torch.polar(torch.full_like(angle, s["amplitude"]), angle)[:, None]
    out = {}
    for n in "qk":
        x = s[n].double().clone()
        even, odd = (slice(0, rot, 2), slice(1, rot, 2)) if case["neighbours"] else (slice(0, rot // 2), slice(rot // 2, rot))
        z = torch.complex(x[..., even], x[..., odd]) * turn
        x[..., even], x[..., odd] = z.real, z.imag
        out[n] = x
    return out


def _exact_append(case, s):
    """The scales alone: the codes are what the scales make of the inputs."""
    page, top = case["page"], TOP[case["codes"]]
    slots = s["slots"].cpu().numpy().astype(np.int64)
    out = {}
    for n in "kv":
        big = s[n].double().abs().amax(-1).cpu().numpy()
        scale = s[n + "_scale"].double().cpu().numpy().copy()
        first, most = {}, {}
        for t, slot in enumerate(slots.tolist()):
            p = slot // page
            first.setdefault(p, slot % page)
            most[p] = np.maximum(most[p], big[t]) if p in most else big[t]
        for p, m in most.items():
            with np.errstate(divide="ignore"):
                k = np.clip(np.ceil(np.log2(m / top)), LEAST, MOST)
            k = np.where(np.exp2(k - 1) * top >= m, np.maximum(k - 1, LEAST), k)
            k = np.where(np.exp2(k) * top < m, np.minimum(k + 1, MOST), k)
            scale[p] = np.maximum(np.exp2(k), scale[p] if first[p] else 0.0)
        out[n + "_cache"], out[n + "_scale"] = None, torch.tensor(scale, device="cuda")
    return out


def _exact_attn(case, s):
    """Request by request and head by head."""
    new, held = _new(case), _past(case) + _new(case)
    H, G, page = case["H"], case["H"] // case["Hkv"], case["page"]
    T = int(new.sum())
    o = torch.zeros(T, H, case["d"], dtype=torch.float64, device="cuda")
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device="cuda")
    row = 0
    for n in range(case["N"]):
        nq, nk = int(new[n]), int(held[n])
        if nq == 0 or nk == 0:
            row += nq
            continue
        pages = s["table"][n, :-(-nk // page)].long()
        k, v = ((s[a + "_cache"].view(torch.uint8)[pages].view(s[a + "_cache"].dtype).double()
                 * s[a + "_scale"][pages].double()[:, :, None, None]).transpose(0, 1).flatten(1, 2)[:, :nk] for a in "kv")
        away = torch.arange(nk - nq, nk, device="cuda")[:, None] - torch.arange(nk, device="cuda")
        for g in range(case["Hkv"]):
            for lo in range(0, G, max(1, (1 << 27) // (nq * nk))):
                heads = slice(g * G + lo, g * G + min(G, lo + max(1, (1 << 27) // (nq * nk))))
                z = torch.einsum("thd,jd->htj", s["q"][row:row + nq, heads].double(), k[g]) * s["scale"]
                if case["cap"]:
                    z = case["cap"] * torch.tanh(z / case["cap"])
                if s["slopes"] is not None:
                    z = z - s["slopes"][heads].double()[:, None, None] * away.abs()
                if case["causal"]:
                    z = torch.where(away >= 0, z, -math.inf)
                lse[row:row + nq, heads] = torch.logsumexp(z, -1).T
                o[row:row + nq, heads] = torch.einsum("htj,jd->thd", torch.softmax(z, -1), v[g])
        row += nq
    return {"o": o, "lse": lse}
