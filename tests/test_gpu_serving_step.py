"""The serving step as a user runs it: plan, norm + rotation + cache write,
windowed attention -- a prefill step and decode steps after it, eagerly and as
a captured graph, against fp64 from the unnormalised projections on."""

import math

import numpy as np
import pytest
import torch

from tests import step_reference as ref

pytestmark = pytest.mark.gpu
HQ, HKV, D, BS, W, SINKS, EPS = 8, 2, 64, 16, 24, 5, 1e-6


@pytest.fixture(scope="module")
def pa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_50_gb300 import build
    build.build()
    import paged_kv_cache_50_gb300 as pa
    pa.lib()
    assert pa.pa_get_device_error() == 0
    return pa


class Engine:
    """Device state of a little engine: pool, table, free list, weights."""

    def __init__(self, pa, n, fp8, seed=0, width=20, blocks=120):
        g = torch.Generator("cuda").manual_seed(seed)
        self.pa, self.n, self.fp8, self.scale = pa, n, fp8, 1 / math.sqrt(D)
        shape = (blocks, 2, BS, HKV, D)
        self.pool = (torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda") if fp8 else
                     torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda"))
        self.table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(blocks, generator=g, device="cuda").int()
        self.start = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ctx = torch.zeros(n, dtype=torch.int32, device="cuda")
        self.qw = (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).bfloat16()
        self.kw = (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).bfloat16()
        self.rope = pa.rope_table(400, D)
        self.ks, self.vs = 0.02, 0.02

    def step(self, packed, qlens, cap, max_q):
        """Attention of the step's tokens; advances the state on the device."""
        pa = self.pa
        qsl, seq, pos, slots, totals = pa.pa_plan_step(
            self.ctx, qlens, self.table, self.free, BS, self.pool.shape[0], max_tokens=cap,
            free_start=self.start)
        q, k, v = (t.view(cap, -1, D) for t in
                   packed.split([HQ * D, HKV * D, HKV * D], dim=1))
        more = dict(q_weight=self.qw, k_weight=self.kw, eps=EPS, cos_sin=self.rope, positions=pos)
        if self.fp8:
            q = pa.pa_qk_norm_rope_cache_fp8(q, k, v, self.pool, slots, self.ks, self.vs, **more)
        else:
            q = pa.pa_qk_norm_rope_cache(q, k, v, self.pool, slots, **more)
        if max_q > 1:
            out, lse = pa.pa_varlen_fwd_sinks(q, self.pool, self.table, qsl, seq, max_q, self.scale,
                                              W, SINKS)
        elif self.fp8:
            out, lse = pa.pa_decode_window_fp8(q[:self.n], self.pool, self.table, seq, self.scale,
                                               self.ks, self.vs, W, SINKS)
        else:
            out, lse = pa.pa_decode_window(q[:self.n], self.pool, self.table, seq, self.scale, W,
                                           SINKS)
        self.ctx.copy_(seq)
        self.start.copy_(totals[1:])
        return out, lse


class Plain:
    """The same in fp64 without a cache: every request's keys and values in order."""

    def __init__(self, e):
        self.e, self.k, self.v = e, [[] for _ in range(e.n)], [[] for _ in range(e.n)]

    def step(self, packed, qlens):
        """[(out, lse, slack)] of each request's rows."""
        e, t, res = self.e, 0, []
        x = packed.double().cpu().numpy()
        rope = e.rope.cpu().numpy()
        for i, m in enumerate(qlens):
            rows = x[t:t + m].reshape(m, HQ + 2 * HKV, D)
            pos = np.arange(len(self.k[i]), len(self.k[i]) + m)
            t += m
            q, _ = ref.norm_rope(rows[:, :HQ], e.qw.double().cpu().numpy(), EPS, rope, pos, False)
            k, _ = ref.norm_rope(rows[:, HQ:HQ + HKV], e.kw.double().cpu().numpy(), EPS, rope, pos,
                                 False)
            self.k[i] += list(k)
            self.v[i] += list(rows[:, HQ + HKV:])
            K, V = np.array(self.k[i]), np.array(self.v[i])
            out, lse = np.zeros((m, HQ, D)), np.zeros((m, HQ))
            slack, lslack = np.zeros((m, HQ, D)), np.zeros((m, HQ))
            for j in range(m):
                keys = [p for p in range(len(K)) if ref.sees(pos[j], p, W, SINKS)]
                for h in range(HQ):
                    kk, vv = K[keys, h // (HQ // HKV)], V[keys, h // (HQ // HKV)]
                    s = kk @ q[j, h] * e.scale
                    w = np.exp(s - s.max())
                    lse[j, h] = s.max() + math.log(w.sum())
                    w /= w.sum()
                    o = w @ vv
                    # Rounding q and k (to bf16, or k to e4m3) moves a logit by
                    # at most r = (uq + uk) scale sum |q k| (+ the floor of
                    # e4m3), so o by at most (exp(2 r) - 1) A, A = sum w |v -
                    # o|; v's own rounding by uv sum w |v|; and the kernel's
                    # bounds of step_reference, here 2^-7 (A + |o|) + 2^-10.
                    uk = 2.0 ** -4 if e.fp8 else 2.0 ** -8
                    mag = (np.abs(kk) @ np.abs(q[j, h])).max()
                    r = (2.0 ** -8 + uk + 2.0 ** -12) * e.scale * mag
                    if e.fp8:
                        r += 2.0 ** -10 * e.ks * e.scale * np.abs(q[j, h]).sum()
                    A, B = w @ np.abs(vv - o), w @ np.abs(vv)
                    uv = 2.0 ** -4 * B + 2.0 ** -10 * e.vs if e.fp8 else 0.0
                    out[j, h] = o
                    slack[j, h] = (math.exp(2 * r) - 1) * A + uv * (1 + math.exp(2 * r)) + \
                        2.0 ** -7 * (A + np.abs(o)) + 2.0 ** -10
                    lslack[j, h] = r + 2.0 ** -12
            res.append((out, lse, slack, lslack))
        return res


def check(got, want, qlens, what):
    out, lse = got[0].double().cpu().numpy(), got[1].double().cpu().numpy()
    t = 0
    for i, m in enumerate(qlens):
        o, l, slack, lslack = want[i]
        err = np.abs(out[t:t + m] - o) - slack
        assert err.max(initial=0) <= 0, (what, i, err.max())
        err = np.abs(lse[t:t + m] - l) - lslack
        assert err.max(initial=0) <= 0, (what, i, err.max())
        t += m


def packed(g, cap):
    return torch.randn((cap, (HQ + 2 * HKV) * D), generator=g, device="cuda").bfloat16()


def test_prefill_then_decode_steps(pa):
    g = torch.Generator("cuda").manual_seed(1)
    e = Engine(pa, 4, fp8=False)
    plain = Plain(e)
    for n, qlens in enumerate([[40, 1, 70, 16], [3, 33, 1, 17], [1] * 4, [1] * 4, [20, 1, 1, 2]]):
        cap = sum(qlens) + (7 if n % 2 else 0)     # padding tokens behind the step
        x = packed(g, cap)
        got = e.step(x, torch.tensor(qlens, dtype=torch.int32, device="cuda"), cap, max(qlens))
        check(got, plain.step(x, qlens), qlens, f"step {n}")
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_captured_decode_steps(pa, fp8):
    """One decode step captured once and replayed: the graph reads its
    lengths, tables and free list from the device and advances them."""
    n, steps = 3, 40
    g = torch.Generator("cuda").manual_seed(2)
    e = Engine(pa, n, fp8, seed=3)
    plain = Plain(e)
    ones = torch.ones(n, dtype=torch.int32, device="cuda")
    x = packed(g, n)
    check(e.step(x, ones, n, 1), plain.step(x, [1] * n), [1] * n, "eager step")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            got = e.step(x, ones, n, 1)
    for k in range(steps):
        x.copy_(packed(g, n))
        graph.replay()
        torch.cuda.synchronize()
        want = plain.step(x, [1] * n)
        if k in (0, 13, 14, 15, 30, steps - 1):
            check(got, want, [1] * n, f"replay {k}")
    assert e.ctx.tolist() == [steps + 1] * n
    assert pa.pa_get_device_error() == 0


def test_two_graphs_and_two_streams(pa):
    """Two engines' captured steps replayed in turn and at once: no state is
    shared between calls."""
    n = 3
    ones = torch.ones(n, dtype=torch.int32, device="cuda")
    gens = [torch.Generator("cuda").manual_seed(s) for s in (4, 5)]
    engines = [Engine(pa, n, False, seed=s) for s in (6, 7)]
    plains = [Plain(e) for e in engines]
    xs, graphs, outs, streams = [], [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for e, gen, st in zip(engines, gens, streams):
        x = packed(gen, n)
        graph = torch.cuda.CUDAGraph()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=st):
            outs.append(e.step(x, ones, n, 1))
        xs.append(x)
        graphs.append(graph)
    for k in range(20):
        for x, gen in zip(xs, gens):
            x.copy_(packed(gen, n))
        torch.cuda.synchronize()
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        for x, plain, out in zip(xs, plains, outs):
            want = plain.step(x, [1] * n)
            if k % 6 == 5:
                check(out, want, [1] * n, f"round {k}")
    assert pa.pa_get_device_error() == 0
