"""Host-side checks of the longer-context entry points (no GPU needed): every bad
argument is refused before a launch, and the references agree with direct
computations."""

import ctypes
import math

import numpy as np
import pytest
import torch

from tests import context_reference as ctx
from tests.test_boundary_steps import _shape, pa  # noqa: F401  (pa: the fixture)

NULL = None
P = 64   # a well-aligned pointer that nothing reads before a launch
BAD_SCALES = (0.0, -1.0, float("inf"), float("nan"))


def test_write_refusals(pa):
    def write(shape=None, k=P, v=P, ks=128, vs=128, cache=P, slots=P, n=4, k_scale=1.0, v_scale=1.0):
        s = shape if shape is not None else _shape(pa)
        return pa.lib().pa_reshape_and_cache_fp4(k, v, ks, vs, cache, slots, n, ctypes.byref(s),
                                                 k_scale, v_scale, NULL)

    for bad in (dict(k=NULL), dict(v=NULL), dict(cache=NULL), dict(slots=NULL), dict(k=72),
                dict(v=72), dict(cache=72), dict(slots=68), dict(n=-1), dict(ks=120), dict(vs=120),
                dict(ks=132), dict(vs=132)):
        assert write(**bad) == pa.PA_ERR_INVALID, bad
    for x in BAD_SCALES:
        assert write(k_scale=x) == write(v_scale=x) == pa.PA_ERR_INVALID
    for bad in (dict(num_kv_heads=0), dict(head_size=0), dict(block_size=0), dict(block_size=24),
                dict(num_blocks=0), dict(num_kv_heads=70000)):
        assert write(_shape(pa, **bad)) == pa.PA_ERR_INVALID, bad
    assert write(_shape(pa, head_size=96), ks=192, vs=192) == pa.PA_ERR_UNSUPPORTED
    assert write(n=0, k=NULL, cache=NULL) == pa.PA_OK


def test_workspace_sizes(pa):
    # A state for each of eight warps of at most two CTAs for each SM; longer contexts two
    # more for each CTA, whatever the batch; sums a log-sum-exp for each row, a pair of
    # numbers for each (request, kv head) and the logits.
    held = 304 * 8 * 9 * 512
    assert pa.pa_decode_fp4_workspace_bytes(64, 32, 8, 128, 200) == held
    assert pa.pa_decode_fp4_workspace_bytes(64, 32, 8, 128, 200, True) == \
        held + 64 * 8 * 8 + 64 * 32 * 4 + 64 * 32 * 200 * 4
    n = pa.pa_decode_fp4_workspace_bytes(1, 64, 8, 128, 131072)
    assert n == held + 304 * (16 + 2 * 8 * 130 * 4)
    assert pa.pa_decode_fp4_workspace_bytes(4096, 64, 8, 128, 131072) == n
    assert pa.pa_decode_fp4_workspace_bytes(1, 2, 1, 64, 16) == 8 * 5 * 512
    n = pa.pa_decode_scores_workspace_bytes(3, 6, 2, 64, 1000)
    assert n == (3 * 6 * 2 * 65 * 4 + 15) // 16 * 16 + 3 * 6 * 1000 * 4
    for bad in ((-1, 4, 2, 64, 10), (1, 0, 2, 64, 10), (1, 4, 0, 64, 10), (1, 4, 2, 0, 10),
                (1, 4, 2, 64, -1)):
        assert pa.pa_decode_fp4_workspace_bytes(*bad) == 0
        assert pa.pa_decode_scores_workspace_bytes(*bad) == 0


def test_decode_refusals(pa):
    L = pa.lib()
    room = 1 << 20

    def four(shape=None, ptrs=(P,) * 4, scale=0.1, ks=1.0, vs=1.0, longest=600, ws=P, size=room,
             out=P, lse=NULL, **_):
        s = shape if shape is not None else _shape(pa)
        return L.pa_decode_fp4(*ptrs, ctypes.byref(s), scale, ks, vs, longest, ws, size, out, lse,
                               NULL)

    def sums(shape=None, ptrs=(P,) * 4, scale=0.1, longest=600, ws=P, size=room, scores=P, cap=600,
             out=P, lse=NULL, **_):
        s = shape if shape is not None else _shape(pa)
        return L.pa_decode_scores(*ptrs, ctypes.byref(s), scale, longest, ws, size, scores, cap, out,
                                  lse, NULL)

    def sums4(shape=None, ptrs=(P,) * 4, scale=0.1, ks=1.0, vs=1.0, longest=600, ws=P, size=room,
              scores=P, cap=600, out=P, lse=NULL):
        s = shape if shape is not None else _shape(pa)
        return L.pa_decode_scores_fp4(*ptrs, ctypes.byref(s), scale, ks, vs, longest, ws, size,
                                      scores, cap, out, lse, NULL)

    for f in (four, sums, sums4):
        for bad in (dict(longest=-1), dict(ws=NULL), dict(ws=72), dict(size=100), dict(out=NULL),
                    dict(lse=66), dict(out=65)):
            assert f(**bad) == pa.PA_ERR_INVALID, (f.__name__, bad)
        for x in BAD_SCALES + (3e38,):
            assert f(scale=x) == pa.PA_ERR_INVALID
        for k in range(4):
            assert f(ptrs=tuple(NULL if j == k else P for j in range(4))) == pa.PA_ERR_INVALID
            assert f(ptrs=tuple(P + 2 if j == k else P for j in range(4))) == pa.PA_ERR_INVALID
        assert f(shape=_shape(pa, head_size=96)) == pa.PA_ERR_UNSUPPORTED
        assert f(shape=_shape(pa, num_q_heads=34)) == pa.PA_ERR_UNSUPPORTED
        assert f(shape=_shape(pa, block_size=24)) == pa.PA_ERR_INVALID
        assert f(shape=_shape(pa, num_q_heads=5)) == pa.PA_ERR_INVALID
        assert f(shape=_shape(pa, num_seqs=65536)) == pa.PA_ERR_INVALID
        assert f(shape=_shape(pa, num_seqs=0), ptrs=(NULL,) * 4) == pa.PA_OK
    for f in (four, sums4):
        for x in BAD_SCALES:
            assert f(ks=x) == f(vs=x) == pa.PA_ERR_INVALID
        assert f(scale=1e20, ks=1e19) == pa.PA_ERR_INVALID
    for f in (sums, sums4):
        for bad in (dict(scores=NULL), dict(scores=66), dict(cap=599)):
            assert f(**bad) == pa.PA_ERR_INVALID, (f.__name__, bad)


def test_evict_refusals(pa):
    L = pa.lib()
    apart = dict(table=2 << 12, seq=3 << 12, scores=4 << 12, lens=5 << 12, fresh=6 << 12,
                 kept=7 << 12, free=8 << 12, start=9 << 12, new=10 << 12)

    def call(four, shape=None, cache=P, el=2, cap=40, budget=20, recent=4, first=2, nfree=8, **kw):
        s = shape if shape is not None else _shape(pa)
        p = {**apart, **kw}
        f = L.pa_evict_fp4 if four else L.pa_evict
        return f(cache, ctypes.byref(s), *(() if four else (el,)), p["table"], p["seq"], p["scores"],
                 cap, budget, recent, first, p["lens"], p["fresh"], p["kept"], p["free"], nfree,
                 p["start"], p["new"], NULL)

    size = dict(table=32, seq=8, scores=640, lens=8, fresh=640, kept=320, free=32, start=4, new=4)
    same = {("lens", "seq"), ("fresh", "scores"), ("new", "start")}
    for four in (False, True):
        for bad in (dict(cap=0), dict(cap=-1), dict(budget=0), dict(budget=-5), dict(recent=-1),
                    dict(first=-1), dict(recent=19), dict(first=17), dict(nfree=-1), dict(cache=NULL),
                    dict(cache=72), dict(budget=(1 << 30) + 1)):
            assert call(four, **bad) == pa.PA_ERR_INVALID, bad
        for name in apart:
            assert call(four, **{name: NULL}) == pa.PA_ERR_INVALID, name
            assert call(four, **{name: apart[name] + 2}) == pa.PA_ERR_INVALID, name
        for out in ("lens", "fresh", "kept", "free", "new"):
            for other in apart:
                if out == other:
                    continue
                for at in (apart[other], apart[other] + size[other] - 4,
                           apart[other] - size[out] + 4):
                    if (out, other) in same and at == apart[other]:
                        continue
                    assert call(four, **{out: at}) == pa.PA_ERR_INVALID, (out, other, at)
        assert call(four, _shape(pa, head_size=96)) == pa.PA_ERR_UNSUPPORTED
        assert call(four, _shape(pa, block_size=24)) == pa.PA_ERR_INVALID
        assert call(four, _shape(pa, num_seqs=0), table=NULL, cache=NULL) == pa.PA_OK
        far = 1 << 20   # nothing may lie in the pool
        for name in apart:
            for at in (far, far + 64, far - size[name] + 4):
                assert call(four, cache=far, **{name: at}) == pa.PA_ERR_INVALID, (name, at)
        s = _shape(pa)
        pool = s.num_blocks * s.num_kv_heads * s.block_size * 2 * s.head_size * 9 // 16
        assert not four or call(four, cache=far, kept=far + pool - 4) == pa.PA_ERR_INVALID
    assert call(False, el=4) == call(False, el=0) == pa.PA_ERR_INVALID


def test_prompt_refusals(pa):
    L = pa.lib()

    def call(q=1 << 16, k=2 << 16, v=3 << 16, qs=256, ks=128, vs=128, qsl=P, n=2, total=4, longest=3,
             hq=4, hkv=2, d=64, scale=0.1, out=4 << 16, lse=NULL):
        return L.pa_prompt_fwd(q, k, v, qs, ks, vs, qsl, n, total, longest, hq, hkv, d, scale, out,
                               lse, NULL)

    for bad in (dict(q=NULL), dict(k=NULL), dict(v=NULL), dict(qsl=NULL), dict(out=NULL),
                dict(q=72), dict(k=72), dict(v=72), dict(out=72), dict(qsl=66), dict(lse=66),
                dict(n=-1), dict(n=65536), dict(total=-1), dict(longest=-1), dict(hq=0), dict(hkv=0),
                dict(hq=5), dict(d=0), dict(qs=248), dict(ks=120), dict(vs=120), dict(qs=260),
                dict(ks=132), dict(vs=132), dict(ks=1 << 40), dict(hkv=70000, hq=70000)):
        assert call(**bad) == pa.PA_ERR_INVALID, bad
    for x in BAD_SCALES + (3e38,):
        assert call(scale=x) == pa.PA_ERR_INVALID
    assert call(d=96, qs=384, ks=192, vs=192) == pa.PA_ERR_UNSUPPORTED
    assert call(hq=258, qs=258 * 64) == pa.PA_ERR_UNSUPPORTED
    # The output in a part of an input: 4 tokens of 512, 256 and 256 bytes.
    for name, at, size in (("q", 1 << 16, 2048), ("k", 2 << 16, 1024), ("v", 3 << 16, 1024)):
        for off in (0, 16, size - 16, 16 - 2048):
            assert call(out=at + off) == pa.PA_ERR_INVALID, (name, off)
    for none in (dict(n=0), dict(total=0), dict(longest=0)):
        assert call(q=NULL, out=NULL, **none) == pa.PA_OK


def test_binding_refuses_host_tensors_and_shapes(pa):
    bf, i32, i64 = torch.bfloat16, torch.int32, torch.int64
    q, kv = torch.zeros(2, 4, 64, dtype=bf), torch.zeros(8, 2, 16, 2, 64, dtype=bf)
    four = pa.fp4_pool(8, 32, 4, 64, device="cpu")
    assert four.shape == (8, 4, 2, 2, 576) and four.dtype == torch.uint8
    table, seq, sums = torch.zeros(2, 4, dtype=i32), torch.ones(2, dtype=i32), torch.zeros(2, 2, 64)
    out, lse, slots = torch.zeros_like(q), torch.zeros(2, 4), torch.zeros(2, dtype=i64)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    more = dict(out=out, lse=lse, max_seq_len=64)
    for bad, word in ((lambda: pa.fp4_pool(8, 24, 2, 64), "multiples of 16"),
                      (lambda: pa.pa_reshape_and_cache_fp4(q, q, four, slots, 1., 1.),
                       "CUDA tensor"),
                      (lambda: pa.pa_reshape_and_cache_fp4(q[:, :2], q[:, :2], kv, slots, 1., 1.),
                       "9 [*] head_size"),
                      (lambda: pa.pa_decode_fp4(q, four, table, seq, 0.1, 1., 1., ws, **more),
                       "CUDA tensor"),
                      (lambda: pa.pa_decode_fp4(q, kv, table, seq, 0.1, 1., 1., ws, **more),
                       "9 [*] head_size"),
                      (lambda: pa.pa_decode_fp4(q[..., :32], four, table, seq, 0.1, 1., 1., ws,
                                                **more), "head_size does not match"),
                      (lambda: pa.pa_decode_fp4(q[:1], four, table, seq, 0.1, 1., 1., ws, **more),
                       "one row per request"),
                      (lambda: pa.pa_decode_scores(q, kv, table[:1], seq, 0.1, sums, ws, **more),
                       "block_table"),
                      (lambda: pa.pa_decode_scores(q, four, table, seq, 0.1, sums, ws, **more),
                       "num_blocks, 2"),
                      (lambda: pa.pa_evict(four, table, seq, sums, 4, kept=table), "num_blocks, 2"),
                      (lambda: pa.pa_evict(kv, table, seq, sums[:1], 4, kept=table), "scores"),
                      (lambda: pa.pa_evict_fp4(kv, table, seq, sums, 4, kept=table),
                       "9 [*] head_size"),
                      (lambda: pa.pa_evict_fp4(four, table, seq, sums.repeat(1, 2, 1), 4, kept=table),
                       "CUDA tensor"),
                      (lambda: pa.pa_prompt_fwd(q, q[:, :2], q[:, :2], seq, 2, 0.1, out=out,
                                                lse=lse), "CUDA tensor"),
                      (lambda: pa.pa_prompt_fwd(q[0], q, q, seq, 2, 0.1, out=out, lse=lse),
                       "num_q_heads"),
                      (lambda: pa.pa_prompt_fwd(q, q, q, table, 2, 0.1, out=out, lse=lse),
                       "query_start_loc")):
        with pytest.raises(ValueError, match=word):
            bad()
    with pytest.raises(TypeError):
        pa.pa_decode_scores(q, kv, table, seq, 0.1, None, ws, **more)
    with pytest.raises(TypeError):
        pa.pa_decode_fp4(None, four, table, seq, 0.1, 1., 1., ws, **more)


def test_reference_quantisation_by_hand():
    x = np.zeros((1, 32), np.float32)
    x[0, :4] = [6, -0.25, 0.75, -5]          # scale 1: 6, -0 (a tie to even), 1, -4 (a tie)
    x[0, 16:19] = [1000, 3, np.nan]
    code, scale = ctx.quantise(x, 1.0)
    assert scale[0].tolist() == [0x38, 0x7F]
    assert code[0, :4].tolist() == [7, 8, 2, 14] and not code[0, 4:].any()
    pool = np.zeros((2, 1, 2, 2, 9 * 32), np.uint8)
    ctx.fp4_store(pool, 1, [32 + 17], x[None], 1.0)
    v = ctx.fp4_values(torch.from_numpy(pool), 5.0, 2.0)
    assert v.shape == (2, 2, 32, 1, 32) and not torch.nan_to_num(v[0]).any()
    assert v[1, 1, 17, 0, :4].tolist() == [12.0, 0.0, 2.0, -8.0]
    assert torch.isnan(v[1, 1, 17, 0, 16:]).all()


def test_reference_eviction_by_hand():
    s = np.array([[[5., 1., math.nan, 3., -0., 0., 9., 2.]]])
    kept, lens, back = ctx.evict(s, [8], np.array([[4, 7, -1]]), 4, 5, 1, 1)
    assert kept == [[[0, 1, 3, 6, 7]]] and lens == [5] and back == []
    kept, lens, back = ctx.evict(s, [8], np.array([[4, 7, -1]]), 4, 4, 0, 0)
    assert kept == [[[0, 3, 6, 7]]] and back == [7]
    assert ctx.evict(s, [6], np.array([[4, 7]]), 4, 5, 0, 0)[0] == [[[0, 1, 3, 4, 5]]]
