"""The operators around the paged cache together, as a serving program uses them: pages planned, queries and keys
turned to their positions, keys and values appended, attention over the cache; prompts of odd lengths first, then
single tokens from a captured graph, requests that end and others that take their pages. Every output against
attention in 64 bits over the exact keys and values of the tokens, the cache held to what its codes may be off by."""
import math

import pytest
import torch

from tests import cache_ref as ref

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
E4M3, INT8 = torch.float8_e4m3fn, torch.int8


class Program:
    """A layer of a serving program with room for `n` requests."""

    def __init__(self, n, width, pages, page, H, Hkv, d, dtype, codes, rot, neighbours):
        from gated_delta_rule_03_gb300 import rotary_amplitude, rotary_rates
        i32 = dict(dtype=torch.int32, device="cuda")
        self.n, self.page, self.H, self.Hkv, self.d, self.dtype, self.neighbours = n, page, H, Hkv, d, dtype, neighbours
        self.table = torch.full((n, width), -1, **i32)
        self.kv = torch.zeros(n, **i32)
        self.free = torch.randperm(pages, device="cuda").int()
        self.count = torch.tensor([pages], **i32)
        self.rates, self.amplitude = rotary_rates(rot, factor=4.0, trained_length=64), rotary_amplitude(4.0)
        junk = 0x7f if codes == E4M3 else 0x80  # pages that were never written hold no numbers
        self.k, self.v = (torch.full((pages, Hkv, page, d), junk, dtype=torch.uint8, device="cuda").view(codes) for _ in "kv")
        self.ks, self.vs = (torch.full((pages, Hkv), math.nan, device="cuda") for _ in "kv")
        self.keys, self.values = [[] for _ in range(n)], [[] for _ in range(n)]  # exact, request by request

    def layer(self, w, q_lens=None, rows=None, max_q=None):
        """One pass over the fused projections w [rows, (H + 2 Hkv) d]."""
        from gated_delta_rule_03_gb300 import cache_append, cache_attn, page_plan, rotary_fwd
        H, Hkv, d = self.H, self.Hkv, self.d
        q, k, v = w[:, :H * d].view(-1, H, d), w[:, H * d:(H + Hkv) * d].view(-1, Hkv, d), w[:, (H + Hkv) * d:].view(-1, Hkv, d)
        p = page_plan(self.table, self.kv, self.free, self.count, self.page, q_lens=q_lens, rows=rows, kv_lens_out=self.kv,
                      free_count_out=self.count)
        q, k = rotary_fwd(q, k, p.positions, self.rates, neighbours=self.neighbours, amplitude=self.amplitude)
        cache_append(k, v, p.slots, self.k, self.v, self.ks, self.vs)
        o = cache_attn(q, self.k, self.v, self.ks, self.vs, self.table, self.kv, cu_q=None if q_lens is None else p.cu_q, max_q=max_q)
        return o, p

    def expect(self, w, lens, o):
        """The same in 64 bits; a value's code is off by half a step of its page's scale at most."""
        H, Hkv, d = self.H, self.Hkv, self.d
        at = 0
        for i, n in enumerate(lens):
            if n == 0:
                continue
            x = w[at:at + n].double().cpu()
            past = len(self.keys[i])
            pos = torch.arange(past, past + n)
            turned = lambda t: ref.rotary(t, pos, self.rates.cpu(), self.neighbours, self.amplitude)  # noqa: E731
            q = turned(x[:, :H * d].view(n, H, d))
            self.keys[i] += list(turned(x[:, H * d:(H + Hkv) * d].view(n, Hkv, d)))
            self.values[i] += list(x[:, (H + Hkv) * d:].view(n, Hkv, d))
            k, v = torch.stack(self.keys[i]).repeat_interleave(H // Hkv, 1), torch.stack(self.values[i]).repeat_interleave(H // Hkv, 1)
            s = torch.einsum("thd,jhd->htj", q, k) * d ** -0.5
            s = torch.where(torch.arange(past + n) <= pos[:, None], s, -math.inf)
            want = torch.einsum("htj,jhd->thd", torch.softmax(s, -1), v)
            # Entries of a page are off by up to e = half a step of its largest: e4m3 2^-4 of themselves and 2^-10 of the scale
            # below its normal numbers, int8 half a scale, and once more for each time that a page was rescaled (int8; a
            # scale at least doubles, so half, a quarter .. a step: two halves in all). A scale is at most 2 / top of the
            # largest entry. bf16 rounds a key, a query and the output, 2^-8 each.
            codes = 2.0 ** -4 + 2.0 ** -10 * 2 / 448 if self.k.dtype == E4M3 else 0.0
            flat = 0.0 if self.k.dtype == E4M3 else 2 / 127
            half = ref.HALF_STEP[self.dtype]
            ks, vs = k.abs().amax(), v.abs().amax()
            key_off = (codes + half) * k.abs() + flat * ks
            score = (torch.einsum("thd,jhd->htj", q.abs(), key_off) + half * torch.einsum("thd,jhd->htj", q.abs(), k.abs())) * d ** -0.5
            score = torch.where(torch.isfinite(s), score, 0.0).amax(-1).T[..., None]
            size = torch.einsum("htj,jhd->thd", torch.softmax(s, -1), v.abs())
            # weights off by e^(2 score) - 1, values by their codes
            bound = (torch.exp(2 * score) - 1) * (size + want.abs()) + torch.exp(2 * score) * (codes * size + flat * vs) + half * want.abs() + 1e-3 * size
            off = (o[at:at + n].double().cpu() - want).abs()
            assert bool((off <= bound).all()), float((off / bound).max())
            # and on the whole far nearer than that: the errors of many entries are not all of one sign
            assert float(off.norm() / want.norm()) < 0.1
            at += n
        return at


@gpu
@pytest.mark.parametrize("dtype,codes,H,Hkv,d,page,rot,neighbours", [
    (BF16, E4M3, 8, 2, 64, 16, 64, False), (BF16, INT8, 4, 4, 128, 32, 32, True), (F32, E4M3, 3, 1, 64, 16, 16, False),
    (BF16, E4M3, 20, 1, 256, 64, 128, True)])
def test_prompts_and_then_single_tokens(dtype, codes, H, Hkv, d, page, rot, neighbours):
    from gated_delta_rule_03_gb300 import page_release
    g = torch.Generator(device="cuda").manual_seed(1)
    prog = Program(4, 400 // page + 2, 4 * (300 // page + 1), page, H, Hkv, d, dtype, codes, rot, neighbours)
    proj = lambda rows: torch.randn(rows, (H + 2 * Hkv) * d, generator=g, device="cuda").to(dtype)  # noqa: E731
    lens = [37, 0, 200, 1]
    w = proj(sum(lens) + 5)  # padded
    o, p = prog.layer(w, torch.tensor(lens, dtype=torch.int32, device="cuda"), rows=len(w), max_q=max(lens))
    assert p.start.tolist() == [0] * 4 and prog.kv.tolist() == lens
    prog.expect(w, lens, o)
    # pieces of prompts behind them
    lens = [9, 70, 3, 64]
    w = proj(sum(lens))
    o, p = prog.layer(w, torch.tensor(lens, dtype=torch.int32, device="cuda"), rows=len(w), max_q=70)
    prog.expect(w, lens, o)
    # single tokens, from a graph
    w = proj(4)
    state = [t.clone() for t in (prog.table, prog.kv, prog.count, prog.k.view(torch.uint8), prog.v.view(torch.uint8), prog.ks, prog.vs)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        prog.layer(w)  # (a first call outside the graph; then everything as it was)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, p = prog.layer(w)
    for t, old in zip((prog.table, prog.kv, prog.count, prog.k.view(torch.uint8), prog.v.view(torch.uint8), prog.ks, prog.vs), state):
        t.copy_(old)
    for _ in range(20):
        w.copy_(proj(4))
        graph.replay()
        prog.expect(w, [1] * 4, o)
    # two requests end, others take their places and pages
    held = int((prog.table >= 0).sum())
    page_release(prog.table, prog.kv, torch.tensor([True, False, True, False], device="cuda"), prog.free, prog.count, page)
    assert prog.kv.tolist()[::2] == [0, 0] and held - int((prog.table >= 0).sum()) == -(-66 // page) + -(-223 // page)
    for i in (0, 2):
        prog.keys[i], prog.values[i] = [], []
    lens = [150, 1, 60, 2]
    w = proj(sum(lens))
    o, p = prog.layer(w, torch.tensor(lens, dtype=torch.int32, device="cuda"), rows=len(w), max_q=150)
    prog.expect(w, lens, o)
    live = prog.table[prog.table >= 0].tolist()
    assert len(live) == len(set(live)) and not set(live) & set(prog.free[:int(prog.count)].tolist())
