"""Sums of attention weights against fp64, and eviction by them exactly."""

import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from tests import context_reference as ctx
from tests import step_reference as ref
from tests.test_gpu_fp4_cache import DEVERR, SHAPES, Cache, i32, pa  # noqa: F401

pytestmark = pytest.mark.gpu


class Plain(Cache):
    """The same cache in bf16, poisoned with NaN."""

    def __init__(self, *args):
        super().__init__(*args)
        v = self.values()
        nb, _, bs, hkv, d = v.shape
        self.pool = v.bfloat16().contiguous()

    def values(self):
        return self.pool.double() if self.pool.dtype == torch.bfloat16 else super().values()

    def check(self, got, what):
        pool = self.values()
        refs = ctx.decode(self.q, pool, self.table, self.seqs, self.scale)
        ref.check_attention(*got, refs, self.d, False, 0.0, what)
        return refs, pool


def sums(pa, c, scores, **kw):
    four = type(c) is Cache
    if "workspace" not in kw:
        n = (pa.pa_decode_fp4_workspace_bytes(len(c.seqs), c.hq, c.hkv, c.d, c.longest, True) if four
             else pa.pa_decode_scores_workspace_bytes(len(c.seqs), c.hq, c.hkv, c.d, c.longest))
        kw["workspace"] = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    kw = {"max_seq_len": c.longest, **kw}
    if four:
        return pa.pa_decode_scores_fp4(c.q, c.pool, c.dev_table, c.dev_seq, c.scale, c.ks, c.vs,
                                       scores, **kw)
    return pa.pa_decode_scores(c.q, c.pool, c.dev_table, c.dev_seq, c.scale, scores, **kw)


@pytest.mark.parametrize("kind", [Cache, Plain], ids=["fp4", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "h%d_%d_d%d_bs%d" % s)
def test_sums(pa, kind, shape):
    g = torch.Generator("cuda").manual_seed(1)
    for n, seqs in enumerate(([0, 1, 15, 16, 17, 33, 257, 600], [2300, 3], [1], [0], [5003])):
        c = kind(n, seqs, *shape)
        before = torch.rand((len(seqs), c.hkv, c.longest + 5), generator=g, device="cuda")
        got_s = before.clone()
        got = sums(pa, c, got_s)
        refs, pool = c.check(got, f"{shape} {seqs}")
        want, tol = ctx.weight_sums(c.q, pool, c.table, c.seqs, c.scale, refs, before)
        over = (got_s.double() - want).abs() - tol
        assert over.max() <= 0, (shape, seqs, float(over.max()))
        again = before.clone()
        sums(pa, c, again)
        assert torch.equal(again, got_s)          # in a fixed order
        assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("kind", [Cache, Plain], ids=["fp4", "bf16"])
def test_sums_of_one_long_stream(pa, kind):
    """One kv head cut into as many parts as there may be, merged row by row."""
    for n, (seqs, hq, d, bs) in enumerate((([20011], 16, 128, 16), ([9000, 40], 5, 64, 32))):
        c = kind(60 + n, seqs, hq, 1, d, bs)
        got_s = torch.zeros((len(seqs), 1, c.longest), device="cuda")
        refs, pool = c.check(sums(pa, c, got_s), f"{seqs}")
        want, tol = ctx.weight_sums(c.q, pool, c.table, c.seqs, c.scale, refs,
                                    torch.zeros_like(got_s))
        assert ((got_s.double() - want).abs() <= tol).all(), seqs
        assert pa.pa_get_device_error() == 0


def test_sums_of_shared_blocks_and_short_max(pa):
    """Two requests over the same blocks keep sums of their own; tokens past
    max_seq_len are attended to, get none and are flagged."""
    c = Cache(2, [400, 400], 8, 2, 64, 16)
    c.table[1] = c.table[0]
    c.dev_table[1] = c.dev_table[0]
    s = torch.zeros((2, 2, 400), device="cuda")
    refs, pool = c.check(sums(pa, c, s), "shared")
    want, tol = ctx.weight_sums(c.q, pool, c.table, c.seqs, c.scale, refs, torch.zeros_like(s))
    assert ((s.double() - want).abs() <= tol).all()
    total = s.double().sum(-1)
    assert (total - 4).abs().max() < 1e-4        # four heads' weights each
    short = torch.zeros((2, 2, 300), device="cuda")
    n = pa.pa_decode_fp4_workspace_bytes(2, 8, 2, 64, 290, True)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    c.check(sums(pa, c, short, max_seq_len=290, workspace=ws), "short")
    assert ((short[..., :290].double() - want[..., :290]).abs() <= tol[..., :290]).all()
    assert not short[..., 290:].any()
    assert pa.pa_get_device_error() == DEVERR["LENGTH"]


@pytest.mark.parametrize("kind", [Cache, Plain], ids=["fp4", "bf16"])
def test_sums_without_a_block(pa, kind):
    """Tokens of a block that is not there get nothing, also where all are gone."""
    c = kind(3, [70, 40, 33], 8, 2, 64, 16)
    c.dev_table[0, 1] = 10 ** 7
    c.dev_table[2, :3] = -1
    s = torch.zeros((3, 2, 70), device="cuda")
    out, lse = sums(pa, c, s)
    assert not s[0, :, 16:32].any() and not s[2].any()
    assert (s.double().sum(-1)[:2] - 4).abs().max() < 1e-4
    assert torch.isneginf(lse[2]).all() and not out[2].any()
    assert pa.pa_get_device_error() == DEVERR["BLOCK_ID"]


# ---------------------------------------------------------------- eviction

KINDS = ("bf16", "e4m3", "fp4")


class Store:
    """A pool of random bytes, its requests' tables, sums and a free list."""

    def __init__(self, seed, kind, seqs, hkv, d, bs, cap=None, values=None, spare=5):
        rng = np.random.default_rng(seed)
        self.kind, self.seqs, self.hkv, self.d, self.bs = kind, np.array(seqs), hkv, d, bs
        need = -(-self.seqs // bs)
        nb = int(need.sum()) + spare
        ids = rng.permutation(nb)
        self.table = np.full((len(seqs), int(need.max(initial=0)) + 2), -1, np.int32)
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = ids[at:at + n]
            at += n
        shape = (nb, hkv, bs // 16, 2, 9 * d) if kind == "fp4" else \
            (nb, 2, bs, hkv, d * (2 if kind == "bf16" else 1))
        self.bytes = rng.integers(0, 256, shape, dtype=np.uint8)
        self.cap = int(max(1, self.seqs.max(initial=0))) + 3 if cap is None else cap
        s = rng.exponential(size=(len(seqs), hkv, self.cap)).astype(np.float32)
        self.scores = s if values is None else rng.choice(np.float32(values), s.shape)
        self.free = np.full(nb + 4, -9, np.int32)
        self.start = nb + 2

    def pool(self):
        t = torch.from_numpy(self.bytes).cuda()
        return {"bf16": lambda: t.view(torch.bfloat16), "e4m3": lambda: t.view(torch.float8_e4m3fn),
                "fp4": lambda: t}[self.kind]()

    def rows(self, b, blk, off, h):
        """The bytes of a token of a head, in a list of views."""
        if self.kind != "fp4":
            return [b[blk, 0, off, h], b[blk, 1, off, h]]
        d, g, r = self.d, off // 16, off % 16
        t = b[blk, h, g]
        return [x for w in (0, 1) for x in (t[w, r * d // 2:(r + 1) * d // 2],
                                            t[w, 8 * d + r * d // 16:8 * d + (r + 1) * d // 16])]

    def run(self, pa, budget, recent, first, inplace, stream=None):
        n = len(self.seqs)
        pool, table, seq = self.pool(), i32(self.table), i32(self.seqs)
        sc = torch.from_numpy(self.scores).cuda()
        free, start = i32(self.free), i32([self.start])
        new = {} if inplace else dict(
            new_lens=torch.full_like(seq, 77), new_scores=torch.full_like(sc, 5.0),
            kept=torch.full((n, self.hkv, budget), 55, dtype=torch.int32, device="cuda"),
            new_free_start=i32([99]))
        f = pa.pa_evict_fp4 if self.kind == "fp4" else pa.pa_evict
        lens, fresh, kept = f(pool, table, seq, sc, budget, num_recent=recent, num_first=first,
                              free_blocks=free, free_start=start, stream=stream, **new)
        assert (lens is seq and fresh is sc) == inplace
        torch.cuda.synchronize()
        assert np.array_equal(table.cpu().numpy(), self.table)
        return (pool.view(torch.uint8).cpu().numpy(), lens.cpu().numpy(), fresh.cpu().numpy(),
                kept.cpu().numpy(), free.cpu().numpy(),
                int(new.get("new_free_start", start)[0]))

    def check(self, pa, budget, recent=0, first=0, inplace=False, what=""):
        got = self.run(pa, budget, recent, first, inplace)
        kept, lens, back = ctx.evict(self.scores, self.seqs, self.table, self.bs, budget, recent,
                                     first)
        want = self.bytes.copy()
        fresh = self.scores.copy() if inplace else np.zeros_like(self.scores)
        places = np.full((len(self.seqs), self.hkv, budget), -1, np.int32)
        for i, m in enumerate(self.seqs):
            for h in range(self.hkv):
                ks = kept[i][h]
                places[i, h, :len(ks)] = ks
                if inplace:
                    fresh[i, h, len(ks):m] = 0
                fresh[i, h, :len(ks)] = self.scores[i, h, ks]
                for j, p in enumerate(ks):
                    if j != p:
                        for a, b in zip(
                                self.rows(want, self.table[i, j // self.bs], j % self.bs, h),
                                self.rows(self.bytes, self.table[i, p // self.bs], p % self.bs, h)):
                            a[...] = b
        free, start = self.free.copy(), self.start - len(back)
        free[start:self.start] = back
        what = (what, budget, recent, first, inplace)
        assert got[1].tolist() == lens, what
        assert np.array_equal(got[3], places), what
        assert np.array_equal(got[0], want), what
        assert np.array_equal(got[2].view(np.uint32), fresh.view(np.uint32)), what
        assert np.array_equal(got[4], free) and got[5] == start, what
        assert pa.pa_get_device_error() == 0, what


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hkv,d,bs", [(2, 128, 16), (3, 64, 48), (1, 128, 64), (8, 64, 32)])
def test_evict(pa, kind, hkv, d, bs):
    for n, (seqs, budget, recent, first) in enumerate((
            ([0, 1, 16, 17, 100, 33, 64, 65], 16, 3, 2), ([300, 40], 290, 0, 0), ([77], 1, 0, 0),
            ([77], 1, 1, 0), ([77, 5], 4, 0, 4), ([700, 2], 300, 300, 0), ([513], 512, 100, 17),
            ([20, 20], 20, 5, 5), ([1500, 1400, 3], 700, 64, 4))):
        for inplace in (False, True):
            Store(n, kind, seqs, hkv, d, bs).check(pa, budget, recent, first, inplace, kind)


@pytest.mark.parametrize("kind", KINDS)
def test_evict_long(pa, kind):
    """One and several CTAs for a request, steps of many rows."""
    Store(20, kind, [9001], 1, 64, 16).check(pa, 4000, 500, 4)
    Store(21, kind, [6000, 5001, 100], 2, 128, 32).check(pa, 2500, 30, 0, True)
    Store(22, kind, list(range(150, 400)), 3, 64, 16).check(pa, 200, 16, 1, True)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("seqs,hkv,budget", [([9000], 8, 2100), ([6000, 5500], 8, 1700),
                                             ([3000] * 4, 8, 1100), ([2600], 2, 2100),
                                             ([700] * 19, 8, 300), ([300] * 70, 8, 140)])
def test_evict_cluster_sizes(pa, kind, seqs, hkv, budget):
    """As many CTAs for a head as fit beside the others', odd numbers of them among these."""
    Store(50, kind, seqs, hkv, 64, 16).check(pa, budget, budget // 9, 3, len(seqs) % 2 == 1)


@pytest.mark.parametrize("kind", KINDS)
def test_evict_far_beyond_the_budget(pa, kind):
    """More tokens than a CTA holds the ranks of, one CTA and several for a head."""
    Store(51, kind, [40000, 21000, 30], 1, 64, 16).check(pa, 100, 10, 4)
    Store(52, kind, [33000], 2, 128, 32).check(pa, 300, 0, 0, True)
    Store(53, kind, [33000], 1, 64, 16, values=[1.0, 2.0, -1.0]).check(pa, 90, 30, 0)


def test_evict_first_call_captured():
    """A process whose first eviction is captured: the launch's sizes are found then."""
    code = """
import torch, paged_kv_cache_50_gb300 as pa
t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
g = torch.Generator("cuda").manual_seed(0)
pool = torch.randn((24, 2, 16, 8, 64), generator=g, device="cuda").bfloat16()
table, seq = torch.arange(24, dtype=torch.int32, device="cuda")[None], t([380])
sums = torch.rand((1, 8, 384), generator=g, device="cuda")
sums[:, :, 380:] = 0
pools = [pool.clone(), pool.clone()]
new = [dict(new_lens=t([0]), new_scores=torch.zeros_like(sums),
            kept=torch.zeros((1, 8, 200), dtype=torch.int32, device="cuda")) for _ in pools]
run = lambda k: pa.pa_evict(pools[k], table, seq, sums, 200, num_recent=9, num_first=2, **new[k])
assert pa.pa_get_device_error() == 0
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    run(0)
graph.replay()
run(1)
torch.cuda.synchronize()
assert new[0]["new_lens"].tolist() == [200] and torch.equal(pools[0], pools[1])
assert all(torch.equal(new[0][k], new[1][k]) for k in new[0])
assert not torch.equal(pools[0], pool) and pa.pa_get_device_error() == 0
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("values", [[1.0], [0.0, -0.0], [1.0, 2.0], [-1.0, 0.0, 1e-45, -1e-45],
                                    [math.nan, 1.0, -1.0], [math.nan], [math.inf, -math.inf, 0.0],
                                    [-math.inf, math.nan], [3.4e38, -3.4e38, 1e-38]],
                         ids=lambda v: "_".join(map(str, v)))
def test_evict_ties_and_odd_sums(pa, values):
    for inplace in (False, True):
        s = Store(30, "bf16", [200, 90, 41], 2, 64, 16, values=values)
        s.check(pa, 40, 7, 3, inplace, values)


def test_evict_again(pa):
    """Twice in a row, in place: the second finds nothing over the budget."""
    s = Store(31, "fp4", [200, 90], 2, 64, 16)
    f = dict(num_recent=5, num_first=2)
    pool, table, seq = s.pool(), i32(s.table), i32(s.seqs)
    sc = torch.from_numpy(s.scores).cuda()
    pa.pa_evict_fp4(pool, table, seq, sc, 60, **f)
    once = pool.clone(), sc.clone()
    _, _, kept = pa.pa_evict_fp4(pool, table, seq, sc, 60, **f)
    assert torch.equal(pool, once[0]) and torch.equal(sc, once[1]) and seq.tolist() == [60, 60]
    assert (kept == torch.arange(60, device="cuda")).all() and pa.pa_get_device_error() == 0


def test_evict_free_list(pa):
    """Blocks are pushed by request over more than one round of requests; without room
    none is, and the rest is done all the same."""
    s = Store(32, "bf16", [40 + k % 30 for k in range(2500)], 1, 64, 16)
    s.check(pa, 17, 4, 0)
    s = Store(33, "bf16", [100, 100], 1, 64, 16)
    s.start = 9                               # ten blocks come back
    got = s.run(pa, 20, 0, 0, False)
    assert got[1].tolist() == [20, 20] and got[5] == 9 and np.array_equal(got[4], s.free)
    assert pa.pa_get_device_error() == DEVERR["LENGTH"]
    s.start = len(s.free) + 1
    got = s.run(pa, 20, 0, 0, False)
    assert got[5] == s.start and np.array_equal(got[4], s.free)
    assert pa.pa_get_device_error() == DEVERR["LENGTH"]


def test_evict_refused_requests(pa):
    """Longer than the sums or the table: left alone, the others are not."""
    s = Store(34, "bf16", [100, 60, 90], 2, 64, 16, cap=95)
    got = s.run(pa, 50, 5, 0, False)
    other = Store(34, "bf16", [100, 60, 90], 2, 64, 16, cap=95)
    blocks = other.table[0, :7]
    assert np.array_equal(got[0][blocks], s.bytes[blocks])
    assert got[1].tolist() == [100, 50, 50]
    assert (got[3][0] == np.arange(50)).all()
    assert pa.pa_get_device_error() == DEVERR["LENGTH"]
    s = Store(35, "bf16", [100, 60], 2, 64, 16, cap=500)
    s.seqs = np.array([16 * s.table.shape[1] + 1, 60])
    got = s.run(pa, 50, 5, 0, False)
    assert got[1].tolist() == [int(s.seqs[0]), 50]
    assert pa.pa_get_device_error() == DEVERR["LENGTH"]
    s.seqs = np.array([ctx.BIG, -5])
    assert s.run(pa, 50, 5, 0, False)[1].tolist() == [ctx.BIG, 0]
    assert pa.pa_get_device_error() == DEVERR["LENGTH"]


@pytest.mark.parametrize("kind", KINDS)
def test_evict_bad_blocks(pa, kind):
    """Rows of a block that is not there stay; nothing else is touched."""
    s = Store(36, kind, [100], 1, 64, 16)
    good = s.table.copy()
    s.table[0, 1], s.table[0, 4] = -3, 10 ** 8
    got = s.run(pa, 60, 0, 0, False)
    assert pa.pa_get_device_error() == DEVERR["BLOCK_ID"]
    kept, _, _ = ctx.evict(s.scores, s.seqs, good, 16, 60, 0, 0)
    want = s.bytes.copy()
    for j, p in enumerate(kept[0][0]):
        if p // 16 not in (1, 4) and j // 16 not in (1, 4):
            for a, b in zip(s.rows(want, good[0, j // 16], j % 16, 0),
                            s.rows(s.bytes, good[0, p // 16], p % 16, 0)):
                a[...] = b
    assert np.array_equal(got[0], want) and np.array_equal(got[3][0, 0], kept[0][0])


def test_evict_captured_beside_another_stream(pa):
    s, o = Store(37, "fp4", [300, 50, 200], 2, 128, 16), Store(38, "bf16", [3000], 2, 64, 16)
    want, other = s.run(pa, 100, 10, 2, False), o.run(pa, 1000, 10, 2, False)
    pool, table, seq = s.pool(), i32(s.table), i32(s.seqs)
    sc, free, start = torch.from_numpy(s.scores).cuda(), i32(s.free), i32([s.start])
    new = dict(new_lens=torch.zeros_like(seq), new_scores=torch.zeros_like(sc),
               kept=torch.zeros((3, 2, 100), dtype=torch.int32, device="cuda"),
               new_free_start=i32([0]))
    f = lambda: pa.pa_evict_fp4(pool, table, seq, sc, 100, 10, 2, free_blocks=free,   # noqa: E731
                                free_start=start, **new)
    f()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f()
    side = torch.cuda.Stream()
    for _ in range(3):
        pool.copy_(s.pool())
        for t in new.values():
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            got_other = o.run(pa, 1000, 10, 2, False, stream=side)
        got = [pool.cpu().numpy(), *(new[k].cpu().numpy() for k in ("new_lens", "new_scores", "kept")),
               free.cpu().numpy(), int(new["new_free_start"][0])]
        assert all(np.array_equal(a, b) for a, b in zip(got, want))
        assert all(np.array_equal(a, b) for a, b in zip(got_other, other))
    assert pa.pa_get_device_error() == 0


def test_evict_past_32_bits(pa):
    """Blocks whose bytes lie past 4 GiB, moved within them."""
    d, hkv, bs = 128, 8, 16
    nb = (1 << 32) // (2 * bs * hkv * d * 2) + 50
    pool = torch.empty((nb, 2, bs, hkv, d), dtype=torch.bfloat16, device="cuda")
    s = Store(39, "bf16", [500], hkv, d, bs, spare=0)
    pool[nb - 32:] = s.pool()
    table = i32(s.table + (s.table >= 0) * (nb - 32))
    lens, _, kept = pa.pa_evict(pool, table, i32(s.seqs), torch.from_numpy(s.scores).cuda(), 200, 8, 1)
    want = s.run(pa, 200, 8, 1, False)
    assert np.array_equal(pool[nb - 32:].contiguous().view(torch.uint8).cpu().numpy(), want[0])
    assert np.array_equal(kept.cpu().numpy(), want[3]) and pa.pa_get_device_error() == 0
