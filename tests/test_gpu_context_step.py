"""The longer-context operators as a user runs them together: whole prompts are
attended to in bf16 and kept in 4 bits, decode steps read the 4-bit pool and sum the
weights, requests over a budget are cut, their blocks go back to the free list that
the step plan takes from.  Against fp64 over the values that the pool should hold."""

import math

import numpy as np
import pytest
import torch

from tests import context_reference as ctx
from tests import step_reference as ref
from tests.test_gpu_fp4_cache import i32, pa  # noqa: F401  (pa: the fixture)

pytestmark = pytest.mark.gpu
HQ, HKV, D, BS, BUDGET, RECENT, FIRST = 8, 2, 64, 16, 40, 6, 2


class Engine:
    def __init__(self, pa, n, blocks=40, width=8, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)
        self.pa, self.n, self.scale, self.ks, self.vs = pa, n, 1 / math.sqrt(D), 0.02, 0.03
        self.pool = pa.fp4_pool(blocks, BS, HKV, D)
        self.pool.fill_(0x7F)
        self.table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(blocks, generator=g, device="cuda").int()
        self.start = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ctx = torch.zeros(n, dtype=torch.int32, device="cuda")     # cached tokens
        self.seen = torch.zeros(n, dtype=torch.int32, device="cuda")    # tokens so far
        self.scores = torch.zeros((n, HKV, width * BS), device="cuda")
        self.w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
        self.rope = pa.rope_table(400, D)
        size = pa.pa_decode_fp4_workspace_bytes(n, HQ, HKV, D, width * BS, True)
        self.ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        # What the pool should hold, by request and head.
        self.held = [[[np.zeros((0, D)), np.zeros((0, D))] for _ in range(HKV)] for _ in range(n)]

    def project(self, packed, positions):
        """Normed and rotated queries, keys and values of a step, in a block of their own."""
        t = packed.shape[0]
        own = torch.empty((1, 2, -(-t // BS) * BS, HKV, D), dtype=torch.bfloat16, device="cuda")
        q, k, v = (x.view(t, -1, D) for x in packed.split([HQ * D, HKV * D, HKV * D], dim=1))
        q = self.pa.pa_qk_norm_rope_cache(
            q, k, v, own, torch.arange(t, device="cuda"), q_weight=self.w, k_weight=self.w,
            cos_sin=self.rope, positions=positions)
        return q, own[0, 0, :t], own[0, 1, :t]

    def plan(self, qlens, cap):
        qsl, seq, pos, slots, totals = self.pa.pa_plan_step(
            self.ctx, qlens, self.table, self.free, BS, self.pool.shape[0], max_tokens=cap,
            free_start=self.start)
        self.start.copy_(totals[1:])
        return qsl, seq, pos, slots

    def prompts(self, packed, qlens):
        qsl, seq, pos, slots = self.plan(i32(qlens), packed.shape[0])
        q, k, v = self.project(packed, pos)
        got = self.pa.pa_prompt_fwd(q, k, v, qsl, max(qlens), self.scale)
        self.pa.pa_reshape_and_cache_fp4(k, v, self.pool, slots, self.ks, self.vs)
        self.ctx.copy_(seq)
        self.seen.copy_(seq)
        return got, (q, k, v)

    def decode(self, packed):
        one = torch.ones(self.n, dtype=torch.int32, device="cuda")
        _, seq, _, slots = self.plan(one, self.n)
        q, k, v = self.project(packed, self.seen)
        self.pa.pa_reshape_and_cache_fp4(k, v, self.pool, slots, self.ks, self.vs)
        got = self.pa.pa_decode_scores_fp4(
            q, self.pool, self.table, seq, self.scale, self.ks, self.vs, self.scores, self.ws,
            max_seq_len=self.scores.shape[2])
        self.ctx.copy_(seq)
        self.seen += 1
        return got, (q, k, v)

    def evict(self):
        return self.pa.pa_evict_fp4(self.pool, self.table, self.ctx, self.scores, BUDGET, RECENT,
                                    FIRST, free_blocks=self.free, free_start=self.start)[2]

    # ------------------------------------------------------------ the model

    def keep(self, k, v, lens):
        t = 0
        for i, m in enumerate(lens):
            for h in range(HKV):
                for w, (x, step) in enumerate(((k, self.ks), (v, self.vs))):
                    tile = np.zeros((1, 1, -(-m // 16), 2, 9 * D), np.uint8)
                    ctx.fp4_store(tile, 0, range(m), x[t:t + m, h:h + 1].float().cpu().numpy(), step)
                    vals = ctx.fp4_values(torch.from_numpy(tile), step, step)[0, 0, :m, 0].numpy()
                    self.held[i][h][w] = np.concatenate([self.held[i][h][w], vals])
            t += m

    def held_pool(self):
        most = max(len(h[0]) for r in self.held for h in r)
        pool = torch.zeros((self.n, 2, most, HKV, D), dtype=torch.float64)
        for i in range(self.n):
            for h in range(HKV):
                for w in (0, 1):
                    x = self.held[i][h][w]
                    pool[i, w, :len(x), h] = torch.from_numpy(x)
        return pool.cuda(), np.arange(self.n)[:, None], [len(r[0][0]) for r in self.held]

    def check_decode(self, got, q, before, what):
        pool, table, lens = self.held_pool()
        refs = ctx.decode(q, pool, table, lens, self.scale)
        ref.check_attention(*got, refs, D, True, float(pool.abs().max()), what)
        want, tol = ctx.weight_sums(q, pool, table, lens, self.scale, refs, before)
        assert ((self.scores.double() - want).abs() <= tol).all(), what
        assert self.ctx.tolist() == lens, what

    def check_evict(self, before, lens, kept, what):
        want, new, _ = ctx.evict(before.cpu().numpy(), lens, np.zeros((self.n, 99), int), BS, BUDGET,
                                 RECENT, FIRST)
        for i in range(self.n):
            for h in range(HKV):
                assert kept[i, h, :new[i]].tolist() == want[i][h], what
                self.held[i][h] = [x[want[i][h]] for x in self.held[i][h]]
        assert self.ctx.tolist() == new, what

    def check_blocks(self):
        """Every block is either a request's or free, once."""
        used = [b for i, m in enumerate(self.ctx.tolist()) for b in
                self.table[i, :-(-m // BS)].tolist()]
        assert sorted(used + self.free[int(self.start[0]):].tolist()) == list(
            range(self.pool.shape[0]))


def packed(g, t):
    return torch.randn((t, (HQ + 2 * HKV) * D), generator=g, device="cuda").bfloat16()


@pytest.mark.parametrize("graphed", [False, True], ids=["eager", "graph"])
def test_prompts_decode_evict(pa, graphed):
    g = torch.Generator("cuda").manual_seed(1)
    lens = [70, 3, 39]
    e = Engine(pa, 3)
    got, (q, k, v) = e.prompts(packed(g, sum(lens)), lens)
    refs = ctx.prompts(q, k, v, np.concatenate([[0], np.cumsum(lens)]), e.scale)
    ref.check_attention(*got, refs, D, False, 0.0, "prompts")
    e.keep(k, v, lens)
    x = packed(g, 3)
    run, cut = e.decode, e.evict
    if graphed:
        before = e.scores.clone()
        got, (q, k, v) = e.decode(x)             # (the first calls load the modules)
        e.keep(k, v, [1] * 3)
        e.check_decode(got, q, before, "first step")
        state = [t.clone() for t in (e.pool, e.table, e.free, e.start, e.ctx, e.scores)]
        e.evict()
        for t, old in zip((e.pool, e.table, e.free, e.start, e.ctx, e.scores), state):
            t.copy_(old)
        torch.cuda.synchronize()
        step, drop = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(step):
            out = e.decode(x)
        with torch.cuda.graph(drop):
            kept = e.evict()

        def run(x):
            step.replay()
            return out

        def cut():
            drop.replay()
            return kept
    for n in range(30):
        x.copy_(packed(g, 3))
        before = e.scores.clone()
        got, (q, k, v) = run(x)
        torch.cuda.synchronize()
        e.keep(k, v, [1] * 3)
        if n % 4 == 0:
            e.check_decode(got, q, before, f"step {n}")
        if n % 5 == 4:
            before, was = e.scores.clone(), e.ctx.tolist()
            e.check_evict(before, was, cut(), f"eviction after step {n}")
            e.check_blocks()
    assert e.ctx.tolist() == [40, 33 + graphed, 40]
    assert e.seen.tolist() == [m + 30 + graphed for m in lens]
    assert pa.pa_get_device_error() == 0


def test_sums_of_a_prompts_last_rows(pa):
    """A prompt's own sums, from the weights of its last rows: each row is a request of
    its own length over the same blocks, the rows' sums are added up."""
    g = torch.Generator("cuda").manual_seed(2)
    e = Engine(pa, 1)
    _, (q, k, v) = e.prompts(packed(g, 70), [70])
    e.keep(k, v, [70])
    rows = torch.arange(62, 70, device="cuda")
    table = e.table.expand(8, -1).contiguous()
    s = torch.zeros((8, HKV, 70), device="cuda")
    ws = torch.empty(pa.pa_decode_fp4_workspace_bytes(8, HQ, HKV, D, 70, True), dtype=torch.uint8,
                     device="cuda")
    got = pa.pa_decode_scores_fp4(q[rows].contiguous(), e.pool, table, (rows + 1).int(), e.scale,
                                  e.ks, e.vs, s, ws, max_seq_len=70)
    pool, _, _ = e.held_pool()
    at, lens = np.zeros((8, 1), int), (rows + 1).tolist()
    refs = ctx.decode(q[rows], pool, at, lens, e.scale)
    ref.check_attention(*got, refs, D, True, float(pool.abs().max()), "rows")
    want, tol = ctx.weight_sums(q[rows], pool, at, lens, e.scale, refs, torch.zeros_like(s))
    assert ((s.double() - want).abs() <= tol).all()
    total = s.sum(0, keepdim=True).contiguous()
    lens, _, kept = pa.pa_evict_fp4(e.pool, e.table, e.ctx, total, 32, RECENT, FIRST)
    assert lens.tolist() == [32] and kept[0, :, -RECENT:].tolist() == [list(range(64, 70))] * HKV
    assert pa.pa_get_device_error() == 0
