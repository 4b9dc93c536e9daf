"""Attention with a sliding window and first tokens that stay visible, prefill
and decode, against fp64.  What no row sees is poisoned: NaN contents, and
table entries that are no block ids where a whole block is unseen.  Bounds:
see step_reference."""

import math

import numpy as np
import pytest
import torch

from tests import step_reference as ref

pytestmark = pytest.mark.gpu
BIG = 2 ** 31 - 1


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


class Batch:
    def __init__(self, seed, seqs, qlens, hq, hkv, d, bs, window, sinks, fp8=False, gain=1.0,
                 poison=True):
        rng = np.random.default_rng(seed)
        g = torch.Generator("cuda").manual_seed(seed)
        self.seqs, self.d, self.fp8 = np.array(seqs), d, fp8
        self.qsl = np.concatenate([[0], np.cumsum(qlens)])
        self.window, self.sinks, self.scale = window, sinks, 1.0 / math.sqrt(d)
        self.ks, self.vs = 0.02, 0.03
        need = -(-self.seqs // bs)
        nb, width = int(need.sum()) + 1, int(need.max(initial=1)) + 1
        ids, k = rng.permutation(nb), 0
        table = np.full((len(seqs), width), -1, np.int32)
        shape = (nb, 2, bs, hkv, d)
        if fp8:
            x = (torch.randn(shape, generator=g, device="cuda") * 40 * gain).clamp(-448, 448)
            self.pool = x.to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            self.pool = (torch.randn(shape, generator=g, device="cuda") * gain).bfloat16()
        dead = np.ones((nb, bs), bool)      # cells that nothing may use
        for i, n in enumerate(need):
            table[i, :n] = ids[k:k + n]
            k += n
            seen = ref.seen_by_any(int(seqs[i]) - int(qlens[i]), int(seqs[i]), window, sinks)
            cells = np.zeros(n * bs, bool)
            cells[:len(seen)] = seen
            dead[table[i, :n]] = ~cells.reshape(n, bs)
        self.table = table.copy()
        if poison:
            for i, n in enumerate(need):
                for b in range(n):
                    if dead[table[i, b]].all():
                        table[i, b] = rng.choice([-1, nb, nb + 99, BIG, -BIG])
            where = torch.from_numpy(dead).cuda()[:, None, :].expand(nb, 2, bs)
            self.pool[where] = 0x7F if fp8 else float("nan")
        self.dev_table = torch.from_numpy(table).cuda()
        self.q = torch.randn((int(self.qsl[-1]), hq, d), generator=g, device="cuda").bfloat16()
        self.dev_seq = torch.from_numpy(self.seqs.astype(np.int32)).cuda()
        self.dev_qsl = torch.from_numpy(self.qsl.astype(np.int32)).cuda()
        self.max_q = int(max(qlens, default=0))

    def reference(self):
        if self.fp8:
            pool = self.pool.view(torch.float8_e4m3fn).double()
            pool = torch.stack([pool[:, 0] * self.ks, pool[:, 1] * self.vs], 1)
        else:
            pool = self.pool.double()
        self.vmax = float(torch.nan_to_num(pool[:, 1], nan=0.0).abs().max())
        return ref.window_attention(self.q.double(), pool, self.table, self.qsl, self.seqs,
                                    self.scale, self.window, self.sinks)

    def prefill(self, pa, **kw):
        return pa.pa_varlen_fwd_sinks(self.q, self.pool, self.dev_table, self.dev_qsl,
                                      self.dev_seq, self.max_q, self.scale, self.window,
                                      self.sinks, **kw)

    def decode(self, pa, **kw):
        if self.fp8:
            return pa.pa_decode_window_fp8(self.q, self.pool, self.dev_table, self.dev_seq,
                                           self.scale, self.ks, self.vs, self.window, self.sinks,
                                           **kw)
        return pa.pa_decode_window(self.q, self.pool, self.dev_table, self.dev_seq, self.scale,
                                   self.window, self.sinks, **kw)

    def check(self, pa, got, what):
        ref.check_attention(*got, self.reference(), self.d, self.fp8, self.vmax, what)
        assert pa.pa_get_device_error() == 0, what


PREFILL = {
    "ragged": ([1, 700, 130, 64, 333, 0, 20], [1, 260, 130, 0, 17, 0, 20], 32, 8, 128, 16),
    "d64": ([45, 300, 97, 1500], [45, 120, 3, 1], 8, 4, 64, 32),
    "g16": ([900, 81], [700, 81], 16, 1, 128, 64),
    "g5_bs48": ([400, 290], [150, 257], 10, 2, 64, 48),
    "g1_bs256": ([513, 1030], [513, 400], 3, 3, 128, 256),
    "late_chunk": ([2100], [70], 12, 4, 128, 16),
    "g128_d64": ([40, 300], [7, 33], 128, 1, 64, 16),
    "g100": ([70, 140], [12, 5], 100, 1, 128, 32),
    "one_long_many_short": ([5 + k for k in range(70)] + [700] + [40] * 30,
                            [1] * 70 + [500] + [1] * 30, 8, 4, 64, 16),
    "many_empty": ([1, 400, 2, 3, 1, 30], [1, 400, 1, 2, 1, 1], 8, 4, 64, 16),
}
MASKS = [(1, 0), (1, 1), (7, 2), (16, 16), (100, 4), (128, 0), (129, 17), (64, 15), (250, 130),
         (300, 256), (33, 400), (BIG, 0), (5, BIG)]


@pytest.mark.parametrize("name", sorted(PREFILL))
def test_prefill(pa, name):
    for n, (window, sinks) in enumerate(MASKS):
        b = Batch(n, *PREFILL[name], window, sinks)
        b.check(pa, b.prefill(pa), f"{name} window={window} sinks={sinks}")


def test_prefill_without_sinks_is_the_window_call(pa):
    b = Batch(50, *PREFILL["ragged"], 100, 0, poison=False)
    o1, l1 = b.prefill(pa)
    o2, l2 = pa.pa_varlen_fwd_window(b.q, b.pool, b.dev_table, b.dev_qsl, b.dev_seq, b.max_q,
                                     b.scale, 100)
    refs = b.reference()
    ref.check_attention(o1, l1, refs, b.d, False, b.vmax, "sinks=0")
    assert (l1[~torch.isinf(l1)] - l2[~torch.isinf(l2)]).abs().max() < 1e-5


def test_prefill_longer_rows(pa):
    b = Batch(51, [5000, 2600], [2200, 2600], 8, 2, 128, 16, 1024, 4)
    b.check(pa, b.prefill(pa), "longer rows")


def test_prefill_leaves_other_rows(pa):
    """Rows past the last request and past max_query_len stay as they were."""
    b = Batch(52, [60, 200], [40, 90], 8, 2, 64, 16, 32, 4)
    T = 150   # 20 rows behind the batch
    q = torch.cat([b.q, torch.full((T - 130, 8, 64), float("nan"), device="cuda").bfloat16()])
    out = torch.full_like(q, 3.0)
    lse = torch.full((T, 8), 5.0, device="cuda")
    pa.pa_varlen_fwd_sinks(q, b.pool, b.dev_table, b.dev_qsl, b.dev_seq, b.max_q, b.scale, 32, 4,
                           out=out, lse=lse)
    b.check(pa, (out[:130], lse[:130]), "padded batch")
    assert (out[130:] == 3.0).all() and (lse[130:] == 5.0).all()


def test_prefill_rows_past_the_batch(pa):
    """A last request that reaches past total_q or max_query_len: the rows that
    exist are computed, the others are left as they were."""
    b = Batch(58, [60, 200], [40, 90], 8, 2, 64, 16, 32, 4, poison=False)
    full = b.reference()
    for T, longest, rows in ((110, 90, [(0, 110)]), (130, 50, [(0, 40), (40, 90)])):
        out = torch.full((200, 8, 64), 3.0, device="cuda").bfloat16()
        lse = torch.full((200, 8), 5.0, device="cuda")
        pa.pa_varlen_fwd_sinks(b.q[:T], b.pool, b.dev_table, b.dev_qsl, b.dev_seq, longest,
                               b.scale, 32, 4, out=out[:T], lse=lse[:T])
        done = torch.zeros(200, dtype=torch.bool, device="cuda")
        for lo, hi in rows:
            done[lo:hi] = True
            ref.check_attention(out[lo:hi], lse[lo:hi], tuple(t[lo:hi] for t in full), b.d, False,
                                b.vmax, f"rows {lo}:{hi}")
        assert (out[~done] == 3.0).all() and (lse[~done] == 5.0).all()
    assert pa.pa_get_device_error() == 0


def test_prefill_most_requests(pa):
    """65535 requests and 64 kv heads, nearly all requests without queries."""
    n, heads, last = 65535, 64, 40
    seq = torch.full((n,), 16, dtype=torch.int32, device="cuda")
    qsl = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    qsl[1:], qsl[n] = 16, 16 + last      # the first and the last one
    seq[n - 1] = last
    table = torch.zeros((n, 3), dtype=torch.int32, device="cuda")
    table[n - 1] = torch.tensor([1, 2, 3])
    pool = torch.randn(4, 2, 16, heads, 64, device="cuda").bfloat16()
    q = torch.randn(16 + last, heads, 64, device="cuda").bfloat16()
    out, lse = pa.pa_varlen_fwd_sinks(q, pool, table, qsl, seq, last, 0.125, 16, 2)
    short = torch.tensor([0, 16, 16 + last], dtype=torch.int32, device="cuda")
    want, wl = pa.pa_varlen_fwd_sinks(q, pool, table[[0, n - 1]], short, seq[[0, n - 1]], last,
                                      0.125, 16, 2)
    assert torch.equal(out, want) and torch.equal(lse, wl)
    assert pa.pa_get_device_error() == 0


def test_nan_query_stays_in_its_row(pa):
    b = Batch(59, [300, 70], [90, 70], 8, 2, 128, 16, 64, 4, poison=False)
    want, wl = b.prefill(pa)
    b.q[33, 5, 7] = float("nan")
    got, gl = b.prefill(pa)
    assert torch.isnan(got[33, 5]).all() and torch.isnan(gl[33, 5])
    got[33, 5], gl[33, 5] = want[33, 5], wl[33, 5]
    assert torch.equal(got, want) and torch.equal(gl, wl)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("window", [64, 4096])
def test_nan_query_stays_in_its_row_of_decode(pa, window, fp8):
    b = Batch(69, [4200, 70], [1, 1], 8, 2, 128, 16, window, 4, fp8, poison=False)
    want, wl = b.decode(pa)
    b.q[0, 5, 7] = float("nan")
    got, gl = b.decode(pa)
    assert torch.isnan(got[0, 5]).all() and torch.isnan(gl[0, 5])
    got[0, 5], gl[0, 5] = want[0, 5], wl[0, 5]
    assert torch.equal(got, want) and torch.equal(gl, wl)


@pytest.mark.parametrize("length", [16 * 21, BIG])
def test_lengths_past_the_table(pa, length):
    """Positions past the table's columns are not seen, and not walked over."""
    b = Batch(68, [300, 40], [1, 1], 8, 2, 64, 16, BIG, 4, poison=False)
    assert b.dev_table.shape[1] == 20
    want = Batch(68, [300, 40], [1, 1], 8, 2, 64, 16, BIG, 4, poison=False).decode(pa)
    b.dev_seq[0] = length
    b.dev_table[0, 19] = 0        # the last column
    for call in (b.decode, b.prefill):
        got = call(pa)
        assert pa.pa_get_device_error() == pa.PA_DEVERR_BLOCK_ID
        assert torch.isfinite(got[0]).all() and torch.isfinite(got[1]).all()
        assert (got[1][1] - want[1][1]).abs().max() < 1e-5
        b.dev_seq[0] = 320
        o, l = b.decode(pa)       # what the table holds
        assert pa.pa_get_device_error() == 0
        assert (got[1][0] - l[0]).abs().max() < 1e-5
        assert (got[0].float() - o.float()).abs().max() < 0.02
        b.dev_seq[0] = length


def test_prefill_more_queries_than_tokens(pa):
    """Requests whose queries reach before position 0: those rows see nothing
    (0, -inf), whole units of them included; the others are aligned to the end."""
    b = Batch(54, [20, 5, 300, 1], [150, 200, 40, 65], 8, 2, 64, 16, 24, 3, poison=False)
    o, l = b.prefill(pa)
    b.check(pa, (o, l), "queries before position 0")
    assert torch.isneginf(l[:130]).all() and not torch.isneginf(l[130:150]).any()


def test_prefill_is_repeatable_and_without_lse(pa):
    b = Batch(55, *PREFILL["ragged"], 100, 4)
    o1, l1 = b.prefill(pa)
    for _ in range(4):
        o2, l2 = b.prefill(pa)
        assert torch.equal(o1, o2) and torch.equal(l1, l2)
    o3, l3 = b.prefill(pa, return_lse=False)
    assert l3 is None and torch.equal(o1, o3)


def test_prefill_captured_and_beside_another(pa):
    """A captured call replayed with other lengths and inputs, while another
    stream runs the same kernel on its own batch."""
    b = Batch(56, [500, 90, 700], [300, 90, 256], 8, 2, 128, 16, 200, 4, poison=False)
    other = Batch(57, [4000], [2500], 16, 4, 128, 16, 1024, 4)
    want = other.prefill(pa)
    out, lse = torch.empty_like(b.q), torch.empty(b.q.shape[:2], device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        b.prefill(pa, out=out, lse=lse)
    for seqs, qlens in (([500, 90, 700], [300, 90, 256]), ([496, 60, 640], [290, 0, 1]),
                        ([300, 90, 650], [300, 1, 200])):
        b.seqs = np.array(seqs)
        b.qsl = np.concatenate([[0], np.cumsum(qlens)])
        b.dev_seq.copy_(torch.from_numpy(b.seqs.astype(np.int32)))
        b.dev_qsl.copy_(torch.from_numpy(b.qsl.astype(np.int32)))
        b.q.normal_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(3):
                graph.replay()
        for _ in range(3):
            got = other.prefill(pa)
        torch.cuda.synchronize()
        n = int(b.qsl[-1])
        ref.check_attention(out[:n], lse[:n], tuple(t[:n] for t in b.reference()), b.d, False,
                            b.vmax, f"replay {qlens}")
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert pa.pa_get_device_error() == 0


def test_prefill_bad_visible_block_is_masked(pa):
    b = Batch(53, [300], [40], 8, 2, 64, 16, 64, 4, poison=False)
    b.dev_table[0, 17] = 10 ** 6      # positions 272..287: in the window
    out, lse = b.prefill(pa)
    assert pa.pa_get_device_error() == pa.PA_DEVERR_BLOCK_ID
    assert torch.isfinite(out).all()


DECODE = {
    "one_stream": ([5000], 64, 8, 128, 16),
    "ragged": ([1, 700, 130, 0, 64, 333, 17, 16, 15], 32, 8, 128, 16),
    "d64_g2": ([45, 300, 97, 1500], 8, 4, 64, 32),
    "g16": ([900, 81, 2050], 16, 1, 128, 64),
    "d64_g12": ([900, 31], 24, 2, 64, 256),
    "g5_bs48": ([400, 290, 49], 10, 2, 64, 48),
    "g1": ([513, 1030], 3, 3, 128, 16),
    "many": (list(range(1, 400, 4)), 8, 8, 64, 16),
}


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("name", sorted(DECODE))
def test_decode(pa, name, fp8):
    seqs, *rest = DECODE[name]
    for n, (window, sinks) in enumerate(MASKS + [(4096, 4), (512, 64), (2000, 1)]):
        b = Batch(n, seqs, [1] * len(seqs), *rest, window, sinks, fp8)
        # A request without tokens has no query position: it sees nothing.
        b.check(pa, b.decode(pa), f"{name} fp8={fp8} window={window} sinks={sinks}")


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_decode_large_logits(pa, fp8):
    """Logits in the hundreds: one token takes nearly all the weight."""
    b = Batch(60, [1200, 300], [1, 1], 8, 2, 128, 16, 512, 8, fp8, gain=1.0 if fp8 else 8.0)
    b.q *= 16
    b.check(pa, b.decode(pa), "large logits")
    if not fp8:
        b.check(pa, b.prefill(pa), "large logits, prefill")


def test_decode_equals_prefill_of_one_row(pa):
    b = Batch(61, [900, 33, 70], [1, 1, 1], 16, 4, 128, 16, 200, 20)
    o1, l1 = b.decode(pa)
    o2, l2 = b.prefill(pa)
    assert (l1 - l2).abs().max() < 1e-5 and (o1.float() - o2.float()).abs().max() < 0.02


def test_decode_is_repeatable_and_without_lse(pa):
    b = Batch(62, [5000, 4000], [1, 1], 32, 8, 128, 16, 4096, 4)
    o1, l1 = b.decode(pa)
    for _ in range(5):
        o2, l2 = b.decode(pa)
        assert torch.equal(o1, o2) and torch.equal(l1, l2)
    o3, l3 = b.decode(pa, return_lse=False)
    assert l3 is None and torch.equal(o1, o3)


def test_decode_float8_pool_is_its_codes(pa):
    b = Batch(67, [900, 33], [1, 1], 16, 4, 128, 16, 200, 20, fp8=True)
    want = b.decode(pa)
    b.pool = b.pool.view(torch.float8_e4m3fn)
    got = b.decode(pa)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_decode_unaligned_query_and_output(pa):
    """q 4-byte aligned and out 2-byte aligned only."""
    b = Batch(63, [900, 33], [1, 1], 16, 4, 64, 16, 200, 20)
    n = b.q.numel()
    q = torch.empty(n + 2, dtype=torch.bfloat16, device="cuda")[2:].view_as(b.q).copy_(b.q)
    out = torch.empty(n + 1, dtype=torch.bfloat16, device="cuda")[1:].view_as(b.q)
    want, _ = b.decode(pa)
    b.q = q
    got, _ = b.decode(pa, out=out)
    assert torch.equal(got, want)


def test_decode_bad_visible_block_is_masked(pa):
    for fp8 in (False, True):
        b = Batch(64, [300, 40], [1, 1], 8, 2, 64, 16, 64, 4, fp8, poison=False)
        b.dev_table[0, 17] = -1
        keep = b.seqs.copy()
        out, lse = b.decode(pa)
        assert pa.pa_get_device_error() == pa.PA_DEVERR_BLOCK_ID
        # Request 1 is as without the fault.
        b.seqs = keep
        o, l = out[1:], lse[1:]
        b.qsl, b.q, b.seqs, b.table = np.array([0, 1]), b.q[1:], keep[1:], b.table[1:]
        b.check(pa, (o, l), "the other request")


def test_decode_past_32_bit_offsets(pa):
    """Blocks whose byte and element offsets pass 2^32."""
    hkv, d, bs = 8, 128, 16
    nb = (1 << 32) // (2 * bs * hkv * d) + 40       # elements > 2^32, bytes > 2^33
    pool = torch.zeros((nb, 2, bs, hkv, d), dtype=torch.bfloat16, device="cuda")
    b = Batch(65, [300], [1], 16, 8, 128, 16, 64, 4, poison=False)
    small = b.pool.shape[0]
    pool[nb - small:] = b.pool
    b.dev_table = torch.where(b.dev_table >= 0, b.dev_table + (nb - small), b.dev_table)
    keep, b.pool = b.pool, pool
    dec, pre = b.decode(pa), b.prefill(pa)
    b.pool = keep
    b.check(pa, dec, "far blocks")
    b.check(pa, pre, "far blocks, prefill")


def test_argument_checks(pa):
    b = Batch(66, [300, 20], [1, 1], 8, 2, 64, 16, 64, 4)
    ok = dict(q=b.q, kv_cache=b.pool, block_table=b.dev_table, seq_lens=b.dev_seq, scale=0.1,
              sliding_window=8, num_sinks=2)
    for bad in (dict(q=b.q.half()), dict(q=b.q[:1]), dict(q=b.q.transpose(1, 2)),
                dict(block_table=b.dev_table[:1]), dict(seq_lens=b.dev_seq.long()),
                dict(out=torch.empty(1, 8, 64, dtype=torch.bfloat16, device="cuda")),
                dict(lse=torch.empty(2, 9, device="cuda")), dict(sliding_window=0),
                dict(num_sinks=-1), dict(kv_cache=b.pool.float()), dict(kv_cache=b.pool[0])):
        with pytest.raises((ValueError, TypeError, pa.PaError)):
            pa.pa_decode_window(**{**ok, **bad})
        with pytest.raises((ValueError, TypeError, pa.PaError)):
            if "q" in bad and bad["q"].shape[0] == 1:
                raise ValueError("a shorter batch is a valid prefill call")
            pa.pa_varlen_fwd_sinks(query_start_loc=b.dev_qsl, max_query_len=1, **{**ok, **bad})
    with pytest.raises(ValueError):
        pa.pa_varlen_fwd_sinks(query_start_loc=b.dev_qsl[:2], max_query_len=1, **ok)
    assert pa.pa_get_device_error() == 0
