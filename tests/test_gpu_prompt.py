"""Causal attention over packed prompts against fp64.  What lies behind the prompts is
NaN.  Bounds: see step_reference."""

import math

import numpy as np
import pytest
import torch

from tests import context_reference as ctx
from tests import step_reference as ref
from tests.test_gpu_fp4_cache import i32, pa  # noqa: F401  (pa: the fixture)

pytestmark = pytest.mark.gpu


class Prompts:
    """Queries, keys and values as views of one packed projection with `pad` elements
    behind each row, and rows of no prompt behind the last."""

    def __init__(self, seed, lens, hq, hkv, d, pad=0, gain=1.0, behind=9):
        g = torch.Generator("cuda").manual_seed(seed)
        self.lens, self.d, self.scale = lens, d, gain / math.sqrt(d)
        self.qsl = np.concatenate([[0], np.cumsum(lens)])
        t = int(self.qsl[-1]) + behind
        w = (hq + 2 * hkv) * d
        x = torch.randn((t, w + pad), generator=g, device="cuda").bfloat16()
        x[int(self.qsl[-1]):] = float("nan")
        self.q, self.k, self.v = (y.view(t, -1, d) for y in
                                  x[:, :w].split([hq * d, hkv * d, hkv * d], dim=1))
        self.dev_qsl, self.longest = i32(self.qsl), max(lens, default=0)

    def run(self, pa, **kw):
        return pa.pa_prompt_fwd(self.q, self.k, self.v, self.dev_qsl,
                                kw.pop("max_query_len", self.longest), self.scale, **kw)

    def check(self, pa, got, what):
        n = int(self.qsl[-1])
        refs = ctx.prompts(self.q[:n], self.k, self.v, self.qsl, self.scale)
        ref.check_attention(got[0][:n], got[1][:n], refs, self.d, False, 0.0, what)
        assert pa.pa_get_device_error() == 0, what


RAGGED = [1, 127, 0, 128, 129, 16, 300, 2, 255, 257, 64]
SHAPES = [(8, 8, 128), (32, 8, 128), (8, 4, 64), (10, 2, 64), (16, 1, 128), (100, 1, 64),
          (128, 1, 128), (3, 3, 64), (24, 8, 64)]


@pytest.mark.parametrize("hq,hkv,d", SHAPES)
def test_prompts(pa, hq, hkv, d):
    for n, lens in enumerate((RAGGED, [1], [5, 40, 17], [640], [0, 0, 3, 0])):
        p = Prompts(n, lens, hq, hkv, d, pad=8 * n)
        p.check(pa, p.run(pa), f"{hq}/{hkv} d{d} {lens}")


def test_longer_prompts(pa):
    p = Prompts(10, [2100, 1000, 513], 8, 2, 128)
    p.check(pa, p.run(pa), "longer")
    p = Prompts(11, [1500, 900], 4, 4, 64)
    p.check(pa, p.run(pa), "longer, 64-wide")


def test_large_logits(pa):
    for gain in (8.0, 60.0):
        p = Prompts(12, [300, 129], 8, 2, 64, gain=gain)
        p.check(pa, p.run(pa), f"gain {gain}")


def test_many_prompts(pa):
    """More prompts than are ordered as a whole, long runs of empty ones among them."""
    rng = np.random.default_rng(13)
    for n, lens in enumerate((list(rng.integers(0, 40, 300)), [0] * 700 + [90] + [0] * 900 + [3],
                              [1] * 64 + [200], [7] * 64, [7] * 65)):
        p = Prompts(20 + n, [int(x) for x in lens], 4, 2, 64)
        p.check(pa, p.run(pa), f"{len(lens)} prompts")


def test_most_prompts(pa):
    p = Prompts(30, [1] * 65535, 2, 1, 64)
    out, lse = p.run(pa)
    n = 65535                                     # a row of one token is its value
    assert torch.equal(out[:n], p.v[:n].expand(n, 2, 64))
    want = (p.q[:n].double() * p.k[:n].double()).sum(-1) * p.scale
    assert (lse[:n].double() - want).abs().max() < 1e-4
    assert pa.pa_get_device_error() == 0


def test_rows_of_no_prompt_stay(pa):
    """Rows behind the last prompt and past max_query_len, at both store widths."""
    p = Prompts(31, [60, 200, 5], 8, 2, 64)
    t = p.q.shape[0]
    for shift in (0, 8):                          # 32- and 16-byte aligned rows
        base = torch.full((t * 8 * 64 + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
        out = base[shift:shift + t * 8 * 64].view(t, 8, 64)
        lse = torch.full((t, 8), 7.0, device="cuda")
        p.check(pa, p.run(pa, out=out, lse=lse), "all rows")
        assert (out[265:] == 7).all() and (lse[265:] == 7).all()
        assert (base[:shift] == 7).all() and (base[shift + t * 8 * 64:] == 7).all()
        full = out.clone()
        out.fill_(7.0)
        p.run(pa, out=out, lse=lse, max_query_len=70)
        assert (out[60 + 70:260] == 7).all()
        keep = list(range(130)) + list(range(260, 265))
        assert torch.equal(out[keep], full[keep])
    assert pa.pa_get_device_error() == 0


def test_neighbours_do_not_matter(pa):
    """A prompt's results do not depend on the prompts beside it, NaN among them."""
    p = Prompts(32, [100, 130, 70], 8, 2, 128)
    want = p.run(pa)
    p.q[:100] = p.k[:100] = p.v[:100] = float("nan")
    p.k[230:], p.v[230:] = float("inf"), float("nan")
    got = p.run(pa)
    for a, b in zip(got, want):
        assert torch.equal(a[100:230], b[100:230])
    assert torch.isnan(got[0][:100]).all()
    assert pa.pa_get_device_error() == 0


def test_without_lse_and_empty_batches(pa):
    p = Prompts(33, [40, 3], 4, 2, 64)
    want, _ = p.run(pa)
    out, lse = p.run(pa, return_lse=False)
    assert lse is None and torch.equal(out[:43], want[:43])
    none = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = pa.pa_prompt_fwd(none, none[:, :2], none[:, :2], i32([0]), 0, 0.1)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)


def test_odd_start_locations(pa):
    """Starts that are negative, fall or pass the rows are read as far as they make
    sense, and nothing else is written."""
    p = Prompts(34, [50, 60], 4, 2, 64)
    t = p.q.shape[0]
    want = p.run(pa)
    for qsl, rows in (([0, 50, 10 ** 6], range(50)), ([-5, 50, 110], range(50, 110)),
                      ([0, 50, 40], range(50))):
        out = torch.full((t, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        p.dev_qsl = i32(qsl)
        p.run(pa, out=out)
        assert torch.equal(out[rows.start:rows.stop], want[0][rows.start:rows.stop])
        assert (out[:rows.start] == 7).all()
    assert pa.pa_get_device_error() == 0


def test_captured_beside_another_stream(pa):
    """One graph for prompts of other lengths; another call beside it; the same each time."""
    p, o = Prompts(35, [200, 40, 90], 8, 2, 64), Prompts(36, [700], 4, 4, 128)
    other = o.run(pa)
    out, lse = p.run(pa, max_query_len=330)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run(pa, max_query_len=330, out=out, lse=lse)
    side = torch.cuda.Stream()
    for lens in ([200, 40, 90], [330, 0, 0], [1, 1, 328], [0, 330, 0]):
        p.lens, p.qsl = lens, np.concatenate([[0], np.cumsum(lens)])
        p.dev_qsl.copy_(i32(p.qsl))
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            got = o.run(pa, stream=side)
        torch.cuda.synchronize()
        p.check(pa, (out, lse), f"replay {lens}")
        assert all(torch.equal(a[:700], b[:700]) for a, b in zip(got, other))
        first = out.clone()
        graph.replay()
        assert torch.equal(out[:330], first[:330])


def test_against_the_pool(pa):
    """The same prompts through a block pool (pa_varlen_fwd)."""
    p = Prompts(37, [300, 77], 8, 2, 128)
    out, lse = p.run(pa)
    pool = torch.zeros((2, 2, 304, 2, 128), dtype=torch.bfloat16, device="cuda")
    for i, m in enumerate(p.lens):
        pool[i, 0, :m], pool[i, 1, :m] = (x[p.qsl[i]:p.qsl[i] + m] for x in (p.k, p.v))
    o2, l2 = pa.pa_varlen_fwd(p.q[:377].contiguous(), pool, i32([[0], [1]]), p.dev_qsl,
                              i32(p.lens), 300, p.scale)
    assert (lse[:377] - l2).abs().max() < 1e-5
    assert (out[:377].double() - o2.double()).abs().max() < 2.0 ** -6
