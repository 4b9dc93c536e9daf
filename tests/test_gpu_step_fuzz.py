"""Random shapes through the serving-step operators: the axes that their own
tests walk one at a time (block and head sizes, group sizes, windows, first
tokens, lengths, layouts, pool types), crossed.  Bounds: see step_reference."""

import numpy as np
import pytest
import torch

from tests import step_reference as ref
from tests import test_gpu_plan_step as plans
from tests import test_gpu_qk_norm_rope as norms
from tests import test_gpu_window_sinks as windows

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


@pytest.mark.parametrize("seed", range(90))
def test_windowed_attention(pa, seed):
    r = np.random.default_rng(90000 + seed)

    def pick(*options):
        return int(r.choice(options))

    d, bs, hkv = pick(64, 128), pick(16, 32, 48, 64, 80, 128), pick(1, 2, 3, 4, 8)
    window = pick(1, 5, 16, 33, 64, 100, 128, 257, 400, 512, 1024, 4096, BIG)
    sinks = pick(0, 0, 1, 4, 15, 16, 17, 64, 130, 500)
    n = pick(1, 1, 2, 3, 5, 9, 20, 64)
    longest = pick(3, 40, 300, 1500, 6000) if n < 10 else pick(40, 300, 1500)
    seqs = r.integers(0, longest + 1, n)
    mode = ("decode", "decode over e4m3", "prefill")[seed % 3]
    if mode == "prefill":
        grp = pick(1, 2, 3, 4, 8, 12, 32, 100)
        new = np.minimum(seqs, r.integers(0, pick(2, 8, 70, 300) + 1, n))
        if new.sum() == 0:
            seqs[0] = max(seqs[0], 1)
            new[0] = 1
    else:
        grp, new = pick(1, 2, 3, 4, 5, 7, 8, 9, 12, 16), np.ones(n, int)
    fp8 = mode == "decode over e4m3"
    b = windows.Batch(seed, [int(x) for x in seqs], [int(x) for x in new], hkv * grp, hkv, d, bs,
                      window, sinks, fp8, gain=1.0 if fp8 else float(r.choice([0.5, 1, 3])))
    got = b.prefill(pa) if mode == "prefill" else b.decode(pa)
    b.check(pa, got, f"{mode} d={d} bs={bs} heads={hkv}x{grp} window={window} sinks={sinks} n={n}")


@pytest.mark.parametrize("seed", range(40))
def test_plan(pa, seed):
    r = np.random.default_rng(70000 + seed)
    n = int(r.choice([1, 2, 31, 33, 64, 255, 256, 257, 400, 511, 513, 900, 1030, 4096, 4097, 5000]))
    bs = int(r.choice([16, 32, 48, 80, 128]))
    ctx, q, table, free, start, nb = plans.make(
        seed, n, int(r.choice([1, 3, 40, 300] if n < 1000 else [1, 3, 20])),
        int(r.choice([0, 5, 100, 3000])), bs, zero=float(r.choice([0, 0.2, 0.9])))
    cap = max(0, int(q.sum()) + int(r.choice([0, 0, 1, 700, -3])))
    plans.compare(plans.run(pa, ctx, q, table, free, start, bs, nb, cap),
                  ref.plan(ctx, q, table, free, start, bs, nb, cap))


@pytest.mark.parametrize("seed", range(40))
def test_norm_rope(pa, seed):
    r = np.random.default_rng(50000 + seed)
    d, hkv = int(r.choice([64, 128])), int(r.choice([1, 2, 3, 4, 8, 16]))
    hq, bs = hkv * int(r.choice([1, 2, 3, 4, 8])), int(r.choice([16, 32, 48, 64, 256]))
    T, rot = int(r.choice([1, 2, 7, 40, 130, 513, 1500])), int(r.choice([0, 16, 32, 48, d // 2, d]))
    inter, norm, fp8 = bool(r.integers(2)), bool(r.integers(4)), bool(r.integers(2))
    c = norms.Case(seed, T, hq, hkv, d, bs, fp8, pad=int(r.choice([0, 8, 24])))
    c.ks, c.vs = float(r.choice([0.001, 0.031, 0.5, 1.0])), float(r.choice([0.027, 0.0077]))
    before = c.pool.cpu().clone()
    got = c.call(pa, norm, rot, inter)
    assert pa.pa_get_device_error() == 0
    c.check(got, before, norm, inter, 1e-5, f"d={d} heads={hq}/{hkv} T={T} rot={rot} {inter} {norm}")
