"""Host-side checks of the serving-step entry points (no GPU needed): every
bad argument is refused before a launch, and the fp64 references that the GPU
tests use agree with direct computations."""

import ctypes
import math

import numpy as np
import pytest
import torch

from tests import step_reference as ref

NULL = None
P = 64   # a well-aligned pointer that nothing reads before a launch


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_50_gb300 import build
    build.build()
    import paged_kv_cache_50_gb300 as pa
    pa.lib()
    return pa


def _shape(pa, **kw):
    f = dict(num_seqs=2, num_q_heads=4, num_kv_heads=2, head_size=64, block_size=16, num_blocks=8,
             max_blocks_per_seq=4)
    f.update(kw)
    return pa.PaShape(*f.values())


def _plan(pa, **kw):
    f = dict(ctx=P, q=P, free=P, start=P, num_free=4, n=2, width=4, bs=16, nb=8, cap=10, table=P,
             qsl=P, seq=P, pos=P, slot=P, totals=P, stream=NULL)
    f.update(kw)
    return pa.lib().pa_plan_step(*f.values())


def test_plan_step_refusals(pa):
    for bad in (dict(num_free=-1), dict(n=-1), dict(n=65536), dict(width=0), dict(bs=0),
                dict(bs=24), dict(nb=0), dict(cap=-1), dict(ctx=NULL), dict(q=NULL),
                dict(free=NULL), dict(table=NULL), dict(qsl=NULL), dict(seq=NULL), dict(pos=NULL),
                dict(slot=NULL), dict(totals=NULL), dict(slot=68), dict(ctx=66), dict(start=65),
                dict(totals=67)):
        assert _plan(pa, **bad) == pa.PA_ERR_INVALID, bad


def test_plan_step_refuses_overlaps(pa):
    """No output may lie in an input or in another output."""
    apart = dict(ctx=1 << 12, q=2 << 12, free=3 << 12, start=4 << 12, table=5 << 12, qsl=6 << 12,
                 seq=7 << 12, pos=8 << 12, slot=9 << 12, totals=10 << 12)
    size = dict(ctx=8, q=8, free=16, start=4, table=32, qsl=12, seq=8, pos=40, slot=80, totals=8)
    inputs = ("ctx", "q", "free", "start")
    for out in apart:
        for other in apart:
            if out == other or out in inputs:
                continue
            for at in (apart[other], apart[other] + size[other] - 4,
                       apart[other] - size[out] + 4):
                if out == "slot" and at % 8:
                    continue
                assert _plan(pa, **{**apart, out: at}) == pa.PA_ERR_INVALID, (out, other, at)


def _norm(pa, shape=None, fp8=False, **kw):
    f = dict(q=P, k=P, v=P, qs=256, ks=128, vs=128, qw=P, kw=P, eps=1e-6, cs=P, rows=16, rot=64,
             inter=0, pos=P, cache=P, slots=P, n=4)
    f.update({k: v for k, v in kw.items() if k in f})
    s = shape if shape is not None else _shape(pa)
    args = list(f.values()) + [ctypes.byref(s)]
    if fp8:
        return pa.lib().pa_qk_norm_rope_cache_fp8(*args, kw.get("kscale", 1.0),
                                                  kw.get("vscale", 1.0), kw.get("out", P), NULL)
    return pa.lib().pa_qk_norm_rope_cache(*args, kw.get("out", P), NULL)


@pytest.mark.parametrize("fp8", [False, True])
def test_norm_rope_refusals(pa, fp8):
    inf, nan = float("inf"), float("nan")
    for bad in (dict(q=NULL), dict(k=NULL), dict(v=NULL), dict(cache=NULL), dict(slots=NULL),
                dict(out=NULL), dict(qw=NULL), dict(kw=NULL), dict(cs=NULL), dict(pos=NULL),
                dict(q=72), dict(k=72), dict(v=72), dict(cache=72), dict(out=72), dict(slots=68),
                dict(cs=68), dict(pos=66), dict(qw=72), dict(kw=72), dict(qs=248), dict(ks=120),
                dict(vs=120), dict(qs=260), dict(ks=132), dict(vs=132), dict(n=-1), dict(rot=-16),
                dict(rot=80), dict(rows=0), dict(eps=-1.0), dict(eps=nan), dict(eps=inf),
                dict(qs=512, out=P)):   # in place needs dense queries
        assert _norm(pa, fp8=fp8, **bad) == pa.PA_ERR_INVALID, bad
    # The output in a part of an input: 4 tokens of 512, 256 and 256 bytes.
    at = dict(q=1 << 12, k=2 << 12, v=3 << 12, out=4 << 12)
    for name, size in (("q", 2048), ("k", 1024), ("v", 1024)):
        for off in (16 - 2048, 16, size - 16) + ((0,) if name != "q" else ()):
            assert _norm(pa, fp8=fp8, **{**at, "out": at[name] + off}) == pa.PA_ERR_INVALID
    for bad in (dict(num_q_heads=0), dict(num_kv_heads=0), dict(head_size=0), dict(block_size=0),
                dict(block_size=24), dict(num_blocks=0), dict(num_q_heads=70000)):
        assert _norm(pa, _shape(pa, **bad), fp8=fp8) == pa.PA_ERR_INVALID, bad
    assert _norm(pa, _shape(pa, head_size=96), fp8=fp8, qs=384, ks=192, vs=192) == \
        pa.PA_ERR_UNSUPPORTED
    assert _norm(pa, fp8=fp8, rot=24) == pa.PA_ERR_UNSUPPORTED
    assert _norm(pa, fp8=fp8, n=0, q=NULL, out=NULL) == pa.PA_OK
    if fp8:
        for bad in (0.0, -1.0, inf, nan):
            assert _norm(pa, fp8=True, kscale=bad) == pa.PA_ERR_INVALID
            assert _norm(pa, fp8=True, vscale=bad) == pa.PA_ERR_INVALID


def test_windowed_attention_refusals(pa):
    L = pa.lib()
    s = _shape(pa)

    def varlen(shape=s, window=8, sinks=2, ptrs=(P,) * 5, out=P, lse=NULL, total=4, scale=0.1):
        return L.pa_varlen_fwd_sinks(*ptrs, total, 2, ctypes.byref(shape), scale, window, sinks, out,
                                     lse, NULL)

    def decode(shape=s, window=8, sinks=2, ptrs=(P,) * 4, out=P, lse=NULL, scale=0.1):
        return L.pa_decode_window(*ptrs, ctypes.byref(shape), scale, window, sinks, out, lse, NULL)

    def decode8(shape=s, window=8, sinks=2, ptrs=(P,) * 4, out=P, lse=NULL, ks=1.0, vs=1.0,
                scale=0.1):
        return L.pa_decode_window_fp8(*ptrs, ctypes.byref(shape), scale, ks, vs, window, sinks, out,
                                      lse, NULL)

    for f, n in ((varlen, 5), (decode, 4), (decode8, 4)):
        assert f(window=0) == f(window=-3) == f(sinks=-1) == f(out=NULL) == pa.PA_ERR_INVALID
        assert f(lse=66) == pa.PA_ERR_INVALID
        for bad in (0.0, -0.1, float("inf"), float("nan")):
            assert f(scale=bad) == pa.PA_ERR_INVALID
        for k in range(n):
            assert f(ptrs=tuple(NULL if j == k else P for j in range(n))) == pa.PA_ERR_INVALID
            assert f(ptrs=tuple(P + 2 if j == k else P for j in range(n))) == pa.PA_ERR_INVALID
        assert f(shape=_shape(pa, head_size=96)) == pa.PA_ERR_UNSUPPORTED
        assert f(shape=_shape(pa, block_size=24)) == pa.PA_ERR_INVALID
        assert f(shape=_shape(pa, num_q_heads=5)) == pa.PA_ERR_INVALID
        assert f(shape=_shape(pa, num_seqs=0), ptrs=(NULL,) * n) == pa.PA_OK
    assert varlen(total=-1) == pa.PA_ERR_INVALID
    assert varlen(total=0, ptrs=(NULL,) * 5) == pa.PA_OK
    assert varlen(shape=_shape(pa, num_q_heads=258)) == pa.PA_ERR_UNSUPPORTED
    wide = _shape(pa, num_q_heads=34)
    assert decode(shape=wide) == decode8(shape=wide) == pa.PA_ERR_UNSUPPORTED
    for bad in (0.0, -1.0, float("inf"), float("nan")):
        assert decode8(ks=bad) == decode8(vs=bad) == pa.PA_ERR_INVALID


def test_binding_refuses_host_tensors(pa):
    i32 = torch.int32
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    kv = torch.zeros(8, 2, 16, 2, 64, dtype=torch.bfloat16)
    table, seq = torch.zeros(2, 4, dtype=i32), torch.ones(2, dtype=i32)
    with pytest.raises(ValueError):
        pa.pa_plan_step(seq, seq, table, seq, 16, 8, max_tokens=4)
    with pytest.raises(ValueError):
        pa.pa_qk_norm_rope_cache(q, q[:, :2], q[:, :2], kv, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        pa.pa_varlen_fwd_sinks(q, kv, table, seq, seq, 1, 0.1, 8, 2)
    with pytest.raises(ValueError):
        pa.pa_decode_window(q, kv, table, seq, 0.1, 8)
    with pytest.raises(TypeError):
        pa.pa_decode_window(None, kv, table, seq, 0.1, 8)


def test_binding_refuses_another_device(pa):
    pa._binding().check_device(0, 0, "q")
    with pytest.raises(ValueError, match="q is on cuda:1, the current device is cuda:0"):
        pa._binding().check_device(1, 0, "q")


def test_binding_checks_shapes_and_types(pa):
    """The compiled checks with host tensors: shapes and types are refused
    first, then the device, all before the library is called."""
    bf, i32, i64 = torch.bfloat16, torch.int32, torch.int64
    q, kv = torch.zeros(2, 4, 64, dtype=bf), torch.zeros(8, 2, 16, 2, 64, dtype=bf)
    table, seq = torch.zeros(2, 4, dtype=i32), torch.ones(2, dtype=i32)
    out, lse = torch.zeros_like(q), torch.zeros(2, 4)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        pa.pa_decode_window(q, kv, table, seq, 0.1, 8, out=out, lse=lse)
    with pytest.raises(ValueError, match="block_table"):
        pa.pa_decode_window(q, kv, table[:1], seq, 0.1, 8, out=out, lse=lse)
    with pytest.raises(ValueError, match="head_size"):
        pa.pa_varlen_fwd_sinks(q[..., :32], kv, table, seq, seq, 1, 0.1, 8, 2, out=out, lse=lse)
    with pytest.raises(TypeError, match="torch.Tensor"):
        pa.pa_decode_window_fp8(q, None, table, seq, 0.1, 1.0, 1.0, 8, out=out, lse=lse)
    with pytest.raises(ValueError, match="num_blocks, 2, block_size"):
        pa.pa_decode_window(q, kv[:, :1], table, seq, 0.1, 8, out=out, lse=lse)
    slots, pos = torch.zeros(2, dtype=i64), torch.zeros(2, dtype=i32)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        pa.pa_qk_norm_rope_cache(q, q[:, :2], q[:, :2], kv, slots, q_out=out)
    with pytest.raises(ValueError, match="num_seqs, max_blocks"):
        pa.pa_plan_step(seq, seq, seq, seq, 16, 8, query_start_loc=pos, seq_lens=seq,
                        positions=pos, slot_mapping=slots, totals=pos)
    with pytest.raises(ValueError, match="out of range"):
        pa.pa_plan_step(seq, seq, table, seq, 16, 8, max_tokens=1 << 40, query_start_loc=pos,
                        seq_lens=seq, positions=pos, slot_mapping=slots, totals=pos)
    with pytest.raises(TypeError):
        pa._binding().plan_step(1, 2)


def test_reference_plan_by_hand():
    # Two requests, blocks of 16: 15 cached + 3 new tokens (one block opens at
    # position 16), 0 cached + 17 new (two blocks).
    qsl, seq, pos, slot, totals, table, err = ref.plan(
        [15, 0], [3, 17], [[7, -1, -1], [-1, -1, -1]], [9, 4, 2, 5], 1, 16, 10, 22)
    assert err == 0 and qsl.tolist() == [0, 3, 20] and seq.tolist() == [18, 17]
    assert table.tolist() == [[7, 4, -1], [2, 5, -1]]
    assert slot.tolist() == [7 * 16 + 15, 64, 65] + list(range(32, 48)) + [80, -1, -1]
    assert pos.tolist() == [15, 16, 17] + list(range(17)) + [0, 0]
    assert totals.tolist() == [20, 4]


def test_reference_rotation_by_hand():
    x = np.arange(1.0, 17.0).reshape(1, 1, 16)
    table = np.zeros((3, 16))
    ang = 0.1 * np.arange(1, 9)
    table[2, :8], table[2, 8:] = np.cos(ang), np.sin(ang)
    z = (x[0, 0, :8] + 1j * x[0, 0, 8:]) * np.exp(1j * ang)
    y, _ = ref.norm_rope(x, None, 0.0, table, np.array([2]), False)
    assert np.allclose(y[0, 0], np.concatenate([z.real, z.imag]), atol=1e-14)
    z = (x[0, 0, 0::2] + 1j * x[0, 0, 1::2]) * np.exp(1j * ang)
    y, _ = ref.norm_rope(x, None, 0.0, table, np.array([2]), True)
    assert np.allclose(y[0, 0, 0::2], z.real) and np.allclose(y[0, 0, 1::2], z.imag)
    y, _ = ref.norm_rope(x, np.full(16, 2.0), 0.0, None, None, False)
    assert math.isclose((y ** 2).mean(), 4.0)


def test_reference_window_by_hand():
    g = torch.Generator().manual_seed(3)
    q = torch.randn((5, 2, 8), generator=g, dtype=torch.float64)
    pool = torch.randn((3, 2, 16, 1, 8), generator=g, dtype=torch.float64)
    table, seq, window, sinks = np.array([[2, 0]], np.int32), 21, 3, 2
    out, lse, *_ = ref.window_attention(q, pool, table, [0, 5], [seq], 0.3, window, sinks)
    flat = torch.cat([pool[2], pool[0]], 1)[:, :seq, 0]              # [2, seq, 8]
    for t in range(5):
        p = 16 + t
        keys = [k for k in range(seq) if ref.sees(p, k, window, sinks)]
        assert keys == [0, 1, p - 2, p - 1, p]
        for h in range(2):
            x = 0.3 * flat[0, keys] @ q[t, h]
            assert torch.allclose(lse[t, h], torch.logsumexp(x, 0))
            assert torch.allclose(out[t, h], torch.softmax(x, 0) @ flat[1, keys])
