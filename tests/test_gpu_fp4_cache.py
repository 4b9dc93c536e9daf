"""The 4-bit pool: the quantising write bit for bit against the formula, and decode
attention over it against fp64.  Bounds: see context_reference."""

import math

import numpy as np
import pytest
import torch

from tests import context_reference as ctx
from tests import step_reference as ref

pytestmark = pytest.mark.gpu
DEVERR = dict(BLOCK_ID=1, SLOT=2, LENGTH=8)


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


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def garbage(shape, g):
    return torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)


# ---------------------------------------------------------------- write

def write_and_compare(pa, k, v, slots, nb, bs, ks, vs, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    hkv, d = k.shape[1:]
    pool = garbage((nb, hkv, bs // 16, 2, 9 * d), g)
    want = pool.cpu().numpy()
    ctx.fp4_store(want, 0, slots, k.float().cpu().numpy(), ks)
    ctx.fp4_store(want, 1, slots, v.float().cpu().numpy(), vs)
    pa.pa_reshape_and_cache_fp4(k, v, pool, torch.from_numpy(slots).cuda(), ks, vs)
    assert np.array_equal(pool.cpu().numpy(), want)


@pytest.mark.parametrize("T,hkv,d,bs", [(1, 1, 64, 16), (67, 8, 128, 16), (300, 3, 64, 48),
                                        (129, 2, 128, 128), (1000, 5, 128, 32)])
def test_write(pa, T, hkv, d, bs):
    """Views of one packed projection with a padded row; scattered, skipped slots."""
    g = torch.Generator("cuda").manual_seed(T)
    rng = np.random.default_rng(T)
    packed = torch.randn((T, 2 * hkv * d + 24), generator=g, device="cuda").bfloat16()
    packed *= torch.exp(2 * torch.randn((T, 1), generator=g, device="cuda")).bfloat16()
    k, v = packed[:, :hkv * d].view(T, hkv, d), packed[:, hkv * d:2 * hkv * d].view(T, hkv, d)
    nb = -(-T // bs) + 2
    slots = rng.permutation(nb * bs)[:T].astype(np.int64)
    slots[rng.random(T) < 0.1] = -1
    write_and_compare(pa, k, v, slots, nb, bs, 0.0153, 1.0)
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("step", [1.0, 0.0153, 1 / 3, 1e-3, 2.0 ** -70, 2.0 ** 70, 1e-36, 1e-44,
                                  1e36, 3.4e38])
def test_write_edge_values(pa, step):
    """Every bf16 value once as a block's first, its neighbours fractions of it at and
    beside the codes' midpoints; scales whose products leave the normal range."""
    bits = np.arange(65536, dtype=np.uint32) << 16
    top = bits.view(np.float32)
    part = np.array([1, -0.25 / 6, 0.75 / 6, -1.25 / 6, 1.75 / 6, 2.5 / 6, -3.5 / 6, 5 / 6, -0.0, 0,
                     1 / 24, -1 / 12, 0.5, -1 / 3, 0.3, 1e-8], np.float32)
    with np.errstate(all="ignore"):
        x = torch.from_numpy(top[:, None] * part[None, :]).bfloat16()
    x = x.view(-1, 1, 64).cuda()                      # four blocks a row
    slots = np.arange(len(x), dtype=np.int64)
    write_and_compare(pa, x, x.flip(-1), slots, len(x) // 64, 64, step, step)
    assert pa.pa_get_device_error() == 0


def test_write_quotients_at_the_midpoints(pa):
    """Random scales, elements that are a scale times a midpoint or the next bf16."""
    rng = np.random.default_rng(5)
    for n in range(40):
        step = float(np.float32(np.exp(rng.uniform(-20, 20))))
        top = (rng.choice([-1, 1], (256, 4)) * np.exp(rng.uniform(-3, 6, (256, 4))) * step)
        scale = np.clip(np.abs(top) / step / 6, 0, 448)
        scale = torch.from_numpy(scale).float().to(torch.float8_e4m3fn).double().numpy()
        mid = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], (256, 4, 15))
        x = np.concatenate([top[..., None], mid * (scale * step)[..., None]], -1)
        bits = (x.astype(np.float32).view(np.uint32) >> 16) + rng.integers(0, 2, x.shape)
        x = torch.from_numpy((bits.astype(np.uint32) << 16).view(np.float32)).bfloat16()
        x = x.reshape(256, 1, 64).cuda()
        write_and_compare(pa, x, -x, np.arange(256, dtype=np.int64), 16, 16, step, step)


def test_write_bad_slots(pa):
    g = torch.Generator("cuda").manual_seed(3)
    k = torch.randn((4, 2, 64), generator=g, device="cuda").bfloat16()
    slots = np.array([5, 64, 1 << 40, 2], np.int64)
    write_and_compare(pa, k, k, slots, 4, 16, 0.1, 0.1)
    assert pa.pa_get_device_error() == DEVERR["SLOT"]


# ---------------------------------------------------------------- decode

class Cache:
    """A 4-bit pool of random contents; what lies past the requests is poisoned: NaN
    scales, and table entries that are no block ids."""

    def __init__(self, seed, seqs, hq, hkv, d, bs, gain=1.0):
        rng = np.random.default_rng(seed)
        g = torch.Generator("cuda").manual_seed(seed)
        self.seqs, self.hq, self.hkv, self.d, self.bs = np.array(seqs), hq, hkv, d, bs
        self.ks, self.vs, self.scale = 0.021, 0.013, 1 / math.sqrt(d)
        need = -(-self.seqs // bs)
        nb = int(need.sum()) + 1
        self.table = np.full((len(seqs), int(need.max(initial=0)) + 1), -1, np.int32)
        ids, at = rng.permutation(nb), 0
        self.pool = garbage((nb, hkv, bs // 16, 2, 9 * d), g)
        _, scales = ctx.fp4_parts(self.pool)
        s = (torch.randn(scales.shape, generator=g, device="cuda").abs() * 40 * gain + 0.1)
        scales = s.clamp(max=448).to(torch.float8_e4m3fn).view(torch.uint8)
        dead = np.ones((nb, bs), bool)
        for i, n in enumerate(need):
            self.table[i, :n] = ids[at:at + n]
            at += n
            cells = np.arange(n * bs) >= seqs[i]
            dead[self.table[i, :n]] = cells.reshape(n, bs)
        where = torch.from_numpy(dead).cuda().view(nb, 1, bs // 16, 1, 16, 1).expand(scales.shape)
        scales = torch.where(where, torch.full_like(scales, 0x7F), scales)
        self.pool[..., 8 * d:] = scales.flatten(-2)
        bad = self.table.copy()
        bad[bad < 0] = rng.choice([-1, nb, nb + 99, ctx.BIG, -ctx.BIG], int((bad < 0).sum()))
        self.dev_table, self.dev_seq = i32(bad), i32(self.seqs)
        self.q = torch.randn((len(seqs), hq, d), generator=g, device="cuda").bfloat16()
        self.longest = int(self.seqs.max(initial=0))

    def workspace(self, pa, sums=False):
        n = pa.pa_decode_fp4_workspace_bytes(len(self.seqs), self.hq, self.hkv, self.d,
                                             self.longest, sums)
        return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN floats

    def decode(self, pa, **kw):
        kw = {"max_seq_len": self.longest, **kw}
        return pa.pa_decode_fp4(self.q, self.pool, self.dev_table, self.dev_seq, self.scale, self.ks,
                                self.vs, kw.pop("workspace", self.workspace(pa)), **kw)

    def values(self):
        return ctx.fp4_values(self.pool, self.ks, self.vs)

    def check(self, got, what):
        pool = self.values()
        refs = ctx.decode(self.q, pool, self.table, self.seqs, self.scale)
        vmax = float(torch.nan_to_num(pool[:, 1]).abs().max())
        ref.check_attention(*got, refs, self.d, True, vmax, what)
        return refs, pool


EDGES = [0, 1, 2, 15, 16, 17, 31, 32, 33, 47, 255, 256, 257, 300, 511, 512, 513, 1000]
SHAPES = [(8, 8, 128, 16), (32, 8, 128, 16), (64, 8, 64, 32), (16, 1, 128, 48), (16, 1, 64, 64),
          (10, 2, 64, 256), (12, 1, 128, 80), (7, 7, 64, 16), (6, 2, 128, 128)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "h%d_%d_d%d_bs%d" % s)
def test_decode(pa, shape):
    """All lengths in one batch (one or two splits), then few requests (many splits)."""
    for n, seqs in enumerate((EDGES, [1000, 3], [1], [0], [5003], [256, 0, 777])):
        c = Cache(n, seqs, *shape)
        c.check(c.decode(pa), f"{shape} {seqs}")
        assert pa.pa_get_device_error() == 0


def test_decode_large_logits(pa):
    for gain in (3.0, 11.0):
        c = Cache(7, [700, 90, 2000], 16, 4, 128, 16, gain)
        c.check(c.decode(pa), f"gain {gain}")


def test_decode_long(pa):
    c = Cache(8, [70001, 131072], 8, 1, 128, 16)
    c.check(c.decode(pa), "long")
    c = Cache(9, [100003], 4, 2, 64, 32)
    c.check(c.decode(pa), "long, 64-wide")


def test_decode_many_requests(pa):
    """The largest batch."""
    rng = np.random.default_rng(11)
    c = Cache(10, rng.integers(0, 40, 65535), 2, 1, 64, 16)
    out, lse = c.decode(pa)
    some = np.arange(0, 65535, 131)
    c.q, c.table, c.seqs = c.q[some], c.table[some], c.seqs[some]
    c.check((out[some], lse[some]), "65535 requests")
    assert pa.pa_get_device_error() == 0


def test_decode_sees_no_bad_block(pa):
    """A missing block and columns past the table are masked and flagged; a longer
    request than max_seq_len is read to its end."""
    c = Cache(12, [200, 100], 8, 2, 64, 16)
    t = c.dev_table.clone()
    t[0, 3], t[1, 0], t[1, 6] = 10 ** 6, -7, 10 ** 8
    gone = {0: range(48, 64), 1: list(range(16)) + list(range(96, 100))}
    c.dev_table = t
    got = c.decode(pa)
    pool = c.values()
    for i in (0, 1):
        keys = np.array([p for p in range(c.seqs[i]) if p not in gone[i]])
        pad = np.full((1, 40), -1, np.int32)
        cut = torch.zeros((1, 2, 200, 2, 64), dtype=torch.float64, device="cuda")
        blk = torch.from_numpy(c.table[i][keys // 16]).long().cuda()
        cut[0, :, :len(keys)] = pool[blk, :, torch.from_numpy(keys % 16).cuda()].transpose(0, 1)
        pad[0, 0] = 0
        refs = ctx.decode(c.q[i:i + 1], cut, pad, [len(keys)], c.scale)
        ref.check_attention(got[0][i:i + 1], got[1][i:i + 1], refs, 64, True, 100.0, f"request {i}")
    assert pa.pa_get_device_error() == DEVERR["BLOCK_ID"]
    c = Cache(13, [3000, 100], 8, 2, 64, 16)
    short = torch.empty(pa.pa_decode_fp4_workspace_bytes(2, 8, 2, 64, 1200), dtype=torch.uint8,
                        device="cuda")
    c.check(c.decode(pa, workspace=short, max_seq_len=1200), "max_seq_len too short")
    assert pa.pa_get_device_error() == 0
    c.dev_seq = i32([16 * c.dev_table.shape[1] + 1, ctx.BIG])
    c.decode(pa)
    assert pa.pa_get_device_error() == DEVERR["BLOCK_ID"]


def test_decode_nan_query_and_nan_block(pa):
    """NaN stays where it belongs: one query, or one head of one request."""
    c = Cache(14, [100, 300, 40], 8, 2, 128, 16)
    want = c.decode(pa)
    c.q[1, 5, 3] = float("nan")
    got = c.decode(pa)
    bad = torch.zeros((3, 8), dtype=torch.bool, device="cuda")
    bad[1, 5] = True
    assert torch.isnan(got[1])[bad].all() and torch.equal(got[1][~bad], want[1][~bad])
    assert torch.isnan(got[0])[bad].all() and torch.equal(got[0][~bad], want[0][~bad])


def test_decode_past_32_bits(pa):
    """Blocks whose bytes lie past 4 GiB."""
    d, hkv, bs = 128, 8, 16
    nb = (1 << 32) // (hkv * 2 * 9 * d) + 200
    pool = torch.empty((nb, hkv, 1, 2, 9 * d), dtype=torch.uint8, device="cuda")
    g = torch.Generator("cuda").manual_seed(15)
    ids = np.arange(nb - 70, nb).astype(np.int32)[::-1]
    T = 70 * bs - 5
    k = torch.randn((T, hkv, d), generator=g, device="cuda").bfloat16()
    slots = torch.from_numpy(ids[np.arange(T) // bs].astype(np.int64) * bs + np.arange(T) % bs).cuda()
    pa.pa_reshape_and_cache_fp4(k, k, pool, slots, 0.01, 0.01)
    q = torch.randn((1, 32, d), generator=g, device="cuda").bfloat16()
    ws = torch.empty(pa.pa_decode_fp4_workspace_bytes(1, 32, 8, d, T), dtype=torch.uint8,
                     device="cuda")
    got = pa.pa_decode_fp4(q, pool, i32(ids[None]), i32([T]), 0.09, 0.01, 0.01, ws, max_seq_len=T)
    vals = ctx.fp4_values(pool[nb - 70:], 0.01, 0.01)
    refs = ctx.decode(q, vals, (ids - (nb - 70))[None], [T], 0.09)
    ref.check_attention(*got, refs, d, True, float(vals[:, 1].abs().max()), "past 32 bits")
    assert pa.pa_get_device_error() == 0


def test_decode_captured_beside_another_stream(pa):
    """One graph for all steps: lengths and tables are read when it runs; a second
    call with a workspace of its own runs beside it, with the same results each time."""
    c = Cache(16, [900, 33, 300, 0], 8, 2, 64, 16)
    o = Cache(17, [2000, 77], 16, 2, 128, 32)
    want_other = o.decode(pa)
    ws, ows = c.workspace(pa), o.workspace(pa)
    out, lse = c.decode(pa, workspace=ws)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.decode(pa, workspace=ws, out=out, lse=lse)
    for seqs in ([900, 33, 300, 0], [1, 20, 0, 0], [513, 1, 299, 0]):
        c.seqs = np.array(seqs)
        c.dev_seq.copy_(i32(seqs))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            got_other = o.decode(pa, workspace=ows, stream=side)
        graph.replay()
        torch.cuda.synchronize()
        c.check((out, lse), f"replay {seqs}")
        first = (out.clone(), lse.clone())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
        assert all(torch.equal(a, b) for a, b in zip(got_other, want_other))
    assert pa.pa_get_device_error() == 0


def test_decode_workspace_is_checked(pa):
    c = Cache(18, [5003], 8, 2, 64, 16)
    small = c.workspace(pa)[:-16]
    with pytest.raises(pa.PaError):
        c.decode(pa, workspace=small)
    with pytest.raises(pa.PaError):
        c.decode(pa, workspace=None)
    with pytest.raises(TypeError):
        c.decode(pa, workspace=small.float())
