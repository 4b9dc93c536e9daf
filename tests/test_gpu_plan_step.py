"""The step plan (block tables, slot maps and positions from request lengths)
on the GPU: whole numbers, equal to the reference in every entry."""

import numpy as np
import pytest
import torch

from tests import step_reference as ref

pytestmark = pytest.mark.gpu


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
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def make(seed, n, q_hi, c_hi, bs, spare_cols=2, spare_free=3, zero=0.2):
    """Random lengths (some requests without context or new tokens), the
    context's blocks in the table, the rest of a permuted pool as free list."""
    rng = np.random.default_rng(seed)
    ctx, q = rng.integers(0, c_hi + 1, n), rng.integers(1, q_hi + 1, n)
    ctx[rng.random(n) < zero] = 0
    q[rng.random(n) < zero] = 0
    have, need = -(-ctx // bs), -(-(ctx + q) // bs)
    width = max(1, int(need.max(initial=1))) + spare_cols
    nb = int(need.sum()) + spare_free + 1
    ids = rng.permutation(nb)
    table = np.full((n, width), -1, np.int32)
    k = 0
    for i in range(n):
        table[i, :have[i]] = ids[k:k + have[i]]
        k += have[i]
    start = int(rng.integers(0, 3))
    free = np.concatenate([rng.integers(0, nb, start), ids[k:]]).astype(np.int32)
    return ctx, q, table, free, start, nb


def run(pa, ctx, q, table, free, start, bs, nb, cap, **kw):
    """Every output in a buffer with a guard behind it."""
    n = len(ctx)
    buf = {k: torch.full((m + 8,), -77, dtype=t, device="cuda") for k, m, t in (
        ("query_start_loc", n + 1, torch.int32), ("seq_lens", n, torch.int32),
        ("positions", cap, torch.int32), ("slot_mapping", cap, torch.int64),
        ("totals", 2, torch.int32))}
    views = {k: b[:b.numel() - 8] for k, b in buf.items()}
    tab = i32(table)
    got = pa.pa_plan_step(i32(ctx), i32(q), tab, i32(free), bs, nb,
                          free_start=None if start is None else i32([start]), **views, **kw)
    err = pa.pa_get_device_error()
    for k, b in buf.items():
        assert (b[-8:] == -77).all(), k
    return [g.cpu().numpy() for g in got] + [tab.cpu().numpy(), err]


def compare(got, want):
    names = ("query_start_loc", "seq_lens", "positions", "slot_mapping", "totals", "table", "error")
    for name, g, w in zip(names, got, want):
        assert np.array_equal(g, w), (name, g, w)


@pytest.mark.parametrize("bs", [16, 48, 64])
@pytest.mark.parametrize("n,q_hi,c_hi", [(1, 1, 0), (1, 1, 40), (3, 5, 39), (64, 1, 4095),
                                         (256, 3, 50), (257, 9, 80), (512, 1, 99), (513, 4, 70),
                                         (16, 300, 4096), (7, 2500, 100), (1023, 3, 70),
                                         (1024, 2, 70), (1025, 4, 33), (2500, 9, 200)])
def test_plan_equals_reference(pa, n, q_hi, c_hi, bs):
    ctx, q, table, free, start, nb = make(n + bs, n, q_hi, c_hi, bs)
    total = int(q.sum())
    for cap in {max(total, 1), total + 1, total + 1500}:
        want = ref.plan(ctx, q, table, free, start, bs, nb, cap)
        assert want[-1] == 0
        compare(run(pa, ctx, q, table, free, start, bs, nb, cap), want)


def test_plan_without_tokens_or_requests(pa):
    compare(run(pa, [5, 0, 32], [0, 0, 0], [[1, -1], [-1, -1], [0, 2]], [3], 0, 16, 4, 0),
            ref.plan([5, 0, 32], [0, 0, 0], [[1, -1], [-1, -1], [0, 2]], [3], 0, 16, 4, 0))
    got = run(pa, np.zeros(0), np.zeros(0), np.zeros((0, 2)), [3], 0, 16, 4, 5)
    assert got[0].tolist() == [0] and got[2].tolist() == [0] * 5 and got[3].tolist() == [-1] * 5
    assert got[4].tolist() == [0, 0] and got[-1] == 0
    # No new block needed: an empty free list is enough; free_start defaults to 0.
    got = run(pa, [5], [11], [[2]], np.zeros(0), None, 16, 4, 11)
    assert got[-1] == 0 and got[3].tolist() == list(range(37, 48)) and got[4].tolist() == [11, 0]


def test_plan_most_requests(pa):
    ctx, q, table, free, start, nb = make(5, 65535, 2, 20, 16)
    cap = int(q.sum()) + 10
    compare(run(pa, ctx, q, table, free, start, 16, nb, cap),
            ref.plan(ctx, q, table, free, start, 16, nb, cap))


def test_plan_one_long_request_among_short(pa):
    q = np.ones(40, np.int64)
    q[17] = 131072
    ctx = np.arange(40) * 3
    need, have = -(-(ctx + q) // 16), -(-ctx // 16)
    nb = int(need.sum())
    ids = np.random.default_rng(8).permutation(nb)
    table = np.full((40, int(need.max())), -1, np.int32)
    k = 0
    for i in range(40):
        table[i, :have[i]] = ids[k:k + have[i]]
        k += have[i]
    cap = int(q.sum())
    compare(run(pa, ctx, q, table, ids[k:], 0, 16, nb, cap),
            ref.plan(ctx, q, table, ids[k:], 0, 16, nb, cap))


@pytest.mark.parametrize("what", ["out_of_blocks", "bad_free_id", "bad_table_id", "narrow_table",
                                  "negative", "negative_start", "capacity"])
def test_plan_refusals_on_the_device(pa, what):
    """Each refused case keeps to its buffers, marks its tokens and sets its bit."""
    ctx, q, table, free, start, nb = make(77, 50, 40, 100, 16, zero=0.0)
    ctx[:] = np.maximum(ctx, 1)
    cap = int(q.sum())
    bit = dict(out_of_blocks="NO_BLOCKS", bad_free_id="BLOCK_ID", bad_table_id="BLOCK_ID").get(
        what, "LENGTH")
    if what == "out_of_blocks":
        free = free[:start + 20]
    elif what == "bad_free_id":
        free = free.copy()
        free[start + 5], free[start + 9] = nb, -4
    elif what == "bad_table_id":
        for i in range(50):
            table[i, max(0, -(-ctx[i] // 16) - 1)] = nb + 3
    elif what == "narrow_table":
        table = table[:, :4].copy()
    elif what == "negative":
        ctx[3], q[5] = -9, -1
    elif what == "negative_start":
        start = -2
    else:
        cap -= 37
    want = ref.plan(ctx, q, table, free, start, 16, nb, cap)
    assert want[-1] & ref.DEVERR[bit]
    compare(run(pa, ctx, q, table, free, start, 16, nb, cap), want)


def test_plan_sums_saturate(pa):
    """Lengths whose sum leaves 32 bits: no wrap, tokens in range, LENGTH."""
    big = 2 ** 31 - 1
    got = run(pa, [0, 0, 0], [big, big, 4], [[1], [2], [3]], [5, 6], 0, 16, 8, 40)
    assert got[-1] & ref.DEVERR["LENGTH"] and got[0].tolist() == [0, 40, 40, 40]
    assert got[2].tolist() == list(range(40)) and got[3].tolist()[:16] == list(range(80, 96))
    assert got[3].tolist()[16:] == [-1] * 24
    got = run(pa, [big], [5], [[1]], [5], 0, 16, 8, 5)
    assert got[-1] & ref.DEVERR["LENGTH"] and got[1].tolist() == [big]


def test_plan_allocates_its_outputs_and_steps_chain(pa):
    """Two steps in a row, the second from the first one's outputs."""
    ctx, q, table, free, start, nb = make(9, 20, 30, 60, 16, spare_cols=4, spare_free=40)
    tab, fr = i32(table), i32(free)
    out = pa.pa_plan_step(i32(ctx), i32(q), tab, fr, 16, nb, max_tokens=700,
                          free_start=i32([start]))
    one = torch.ones(20, dtype=torch.int32, device="cuda")
    out2 = pa.pa_plan_step(out[1], one, tab, fr, 16, nb, max_tokens=20, free_start=out[4][1:])
    w = ref.plan(ctx, q, table, free, start, 16, nb, 700)
    w2 = ref.plan(w[1], np.ones(20), w[5], free, int(w[4][1]), 16, nb, 20)
    assert w[-1] == w2[-1] == 0
    compare([t.cpu().numpy() for t in out2] + [tab.cpu().numpy(), pa.pa_get_device_error()], w2)


def test_plan_lengths_at_any_address(pa):
    """More than 1024 requests whose lengths start 4, 8 or 12 bytes past 16."""
    ctx, q, table, free, start, nb = make(31, 1500, 5, 60, 16)
    want = ref.plan(ctx, q, table, free, start, 16, nb, int(q.sum()))
    for off in (1, 2, 3):
        buf = torch.zeros((2, 1504), dtype=torch.int32, device="cuda")
        c, n = buf[0, off:off + 1500], buf[1, off:off + 1500]
        c.copy_(i32(ctx))
        n.copy_(i32(q))
        tab = i32(table)
        got = pa.pa_plan_step(c, n, tab, i32(free), 16, nb, max_tokens=int(q.sum()),
                              free_start=i32([start]))
        compare([t.cpu().numpy() for t in got] + [tab.cpu().numpy(), pa.pa_get_device_error()],
                want)


def test_plan_beyond_capacity_keeps_attention_in_range(pa):
    """A step of more tokens than its buffers hold: attention over the plan's
    outputs neither leaves them nor touches another row."""
    ctx, q = np.array([20, 0, 7]), np.array([30, 40, 50])
    tab, cap = i32(np.full((3, 8), -1)), 64
    tab[0, :2], tab[2, 0] = i32([0, 1]), 2
    qsl, seq, pos, slot, tot = pa.pa_plan_step(i32(ctx), i32(q), tab, i32(np.arange(3, 24)), 16, 24,
                                               max_tokens=cap)
    assert qsl.tolist() == [0, 30, 64, 64] and tot.tolist()[0] == 120
    assert pa.pa_get_device_error() == pa.PA_DEVERR_LENGTH
    pool = torch.randn(24, 2, 16, 2, 64, device="cuda").bfloat16()
    x = torch.randn(cap + 80, 8, 64, device="cuda").bfloat16()
    out, lse = torch.full_like(x, 3.0), torch.full((cap + 80, 8), 5.0, device="cuda")
    pa.pa_varlen_fwd_sinks(x[:cap], pool, tab, qsl, seq, 50, 0.1, 16, 2, out=out[:cap],
                           lse=lse[:cap])
    torch.cuda.synchronize()
    pa.pa_get_device_error()      # the blocks that were never opened
    assert torch.isfinite(out[:30]).all()
    assert (out[cap:] == 3.0).all() and (lse[cap:] == 5.0).all()


def test_plan_argument_checks(pa):
    t, one = i32([[0, 1]]), i32([1])
    for kw in (dict(context_lens=i32([1, 2])), dict(query_lens=one.long()),
               dict(free_blocks=i32([[1]])), dict(free_start=i32([1, 2])), dict(totals=i32([1])),
               dict(positions=i32([1, 2])), dict(slot_mapping=torch.zeros(2, device="cuda")),
               dict(query_start_loc=one), dict(seq_lens=one.cpu()), dict(block_size=20),
               dict(max_tokens=None)):
        args = dict(context_lens=one, query_lens=one, block_table=t, free_blocks=one,
                    block_size=16, num_blocks=4, max_tokens=1)
        args.update(kw)
        with pytest.raises((ValueError, TypeError, pa.PaError)):
            pa.pa_plan_step(**args)
    assert pa.pa_get_device_error() == 0
