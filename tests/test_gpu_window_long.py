"""Windowed prefill at windows up to the largest int, which users pass for "no
window".  Bounds: see step_reference."""

import numpy as np
import pytest
import torch

from tests.test_gpu_window_sinks import BIG, Batch, pa  # noqa: F401  (pa: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window", [BIG, BIG - 1, BIG - 100, BIG - 300, BIG // 2 + 1])
def test_more_queries_than_tokens(pa, d, window):
    """Rows before position 0 see nothing, the others everything up to their
    own position: a unit's first row may lie anywhere before 0."""
    for sinks in (0, 3, BIG):
        b = Batch(54, [20, 5, 300, 1, 64], [150, 200, 40, 65, 64], 8, 2, d, 16, window, sinks,
                  poison=False)
        o, l = b.prefill(pa)
        what = f"d={d} window={window} sinks={sinks}"
        b.check(pa, (o, l), what)
        for i, (seq, n) in enumerate(zip(b.seqs, np.diff(b.qsl))):
            rows = l[int(b.qsl[i]):int(b.qsl[i + 1])]
            dead = max(0, int(n - seq))
            assert torch.isneginf(rows[:dead]).all() and torch.isfinite(rows[dead:]).all(), what


@pytest.mark.parametrize("d", [64, 128])
def test_largest_window_is_no_window(pa, d):
    b = Batch(3, [700, 90], [300, 90], 8, 2, d, 16, BIG, 0, poison=False)
    o, l = b.prefill(pa)
    o2, l2 = pa.pa_varlen_fwd(b.q, b.pool, b.dev_table, b.dev_qsl, b.dev_seq, b.max_q, b.scale)
    b.check(pa, (o, l), f"d={d}")
    assert (l - l2).abs().max() < 1e-5 and (o.float() - o2.float()).abs().max() < 0.02
