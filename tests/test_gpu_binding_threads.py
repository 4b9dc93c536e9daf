"""The compiled calls beside other threads of the interpreter."""

import ctypes
import threading

import pytest
import torch

from tests.test_gpu_window_sinks import Batch, pa  # noqa: F401  (pa: the fixture)

pytestmark = pytest.mark.gpu


def entry_points(L):
    return (L.pa_plan_step, L.pa_qk_norm_rope_cache, L.pa_qk_norm_rope_cache_fp8,
            L.pa_varlen_fwd_sinks, L.pa_decode_window, L.pa_decode_window_fp8)


def address(f):
    return ctypes.cast(f, ctypes.c_void_p).value


def test_library_calls_leave_the_interpreter_free(pa):
    """Every entry point in turn replaced by the interpreter's own question
    whether this thread holds its lock; the answer is the call's status."""
    b = pa._binding()
    held = address(ctypes.pythonapi.PyGILState_Check)
    assert ctypes.pythonapi.PyGILState_Check() == 1    # the question itself works

    def i32(*s):
        return torch.zeros(s, dtype=torch.int32, device="cuda")

    x = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros((2, 2, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    kv8, lse, slots = kv.to(torch.uint8), torch.zeros((1, 2), device="cuda"), i32(1).long()
    b.bind(*[held] * 6)
    try:
        got = [
            b.plan_step(i32(1), i32(1), i32(1), None, i32(1, 1), 16, 2, 1, i32(2), i32(1), i32(1),
                        slots, i32(2), None),
            b.norm_rope(x, x, x, kv, slots, None, None, None, 1e-6, None, None, False, x, None),
            b.norm_rope(x, x, x, kv8, slots, (1.0, 1.0), None, None, 1e-6, None, None, False, x,
                        None),
            b.varlen_sinks(x, kv, i32(1, 1), i32(1), x, lse, i32(2), 1, 0.1, 8, 2, None),
            b.decode_window(x, kv, i32(1, 1), i32(1), x, lse, None, 0.1, 8, 2, None),
            b.decode_window(x, kv8, i32(1, 1), i32(1), x, lse, (1.0, 1.0), 0.1, 8, 2, None)]
    finally:
        b.bind(*(address(f) for f in entry_points(pa.lib())))
    assert got == [0] * 6
    with pytest.raises(ValueError):      # refusals are raised with the lock held
        pa.pa_decode_window(x, kv, i32(1, 1), i32(2), 0.1, 8)


def test_calls_from_several_threads(pa):
    """Four threads, each on a stream of its own, give what one gives."""
    b = Batch(70, [900, 33, 300], [70, 33, 1], 8, 2, 64, 16, 64, 4, poison=False)
    want = b.prefill(pa)
    torch.cuda.synchronize()
    wrong = []

    def work():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(50):
                got = b.prefill(pa)
                s.synchronize()
                if not (torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])):
                    wrong.append(threading.current_thread().name)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and pa.pa_get_device_error() == 0
