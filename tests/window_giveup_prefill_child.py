"""Child process of test_gpu_window_giveup.py: windowed prefill in a test build
of the library, through its C ABI; prints one JSON line with what it saw.

  python -m tests.window_giveup_prefill_child <path of the test build>

A CTA's first unit loses the weights of its second Q tile in the last tile but
one, so that the CTA gives up between the next unit's two query copies: the
first is on its way (it comes late) and has to be waited for.
"""

import ctypes
import json
import math
import sys

import torch

from tests.timeout_child import Shape

HQ, HKV, BS, WINDOW, SINKS = 32, 8, 16, 512, 8
CTX, NEW = 1000, 8000      # 126 slots x 8 heads: every CTA takes several units


def main(path):
    L = ctypes.CDLL(path)
    P, i32, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    L.pa_varlen_fwd_sinks.argtypes = [P, P, P, P, P, i32, i32, ctypes.POINTER(Shape), f32, i32,
                                      i32, P, P, P]
    L.pa_get_device_error.argtypes = [ctypes.POINTER(i32), P]
    g = torch.Generator("cuda").manual_seed(75)
    records = []
    for d in (128, 64):
        nb = -(-(CTX + NEW) // BS)
        table = torch.randperm(nb, generator=g, device="cuda").int().view(1, nb)
        pool = torch.randn((nb, 2, BS, HKV, d), generator=g, device="cuda").bfloat16()
        q = torch.randn((NEW, HQ, d), generator=g, device="cuda").bfloat16()
        seq = torch.tensor([CTX + NEW], dtype=torch.int32, device="cuda")
        qsl = torch.tensor([0, NEW], dtype=torch.int32, device="cuda")
        shape = Shape(1, HQ, HKV, d, BS, nb, nb)

        def run():
            out = torch.full_like(q, 7.0)
            lse = torch.full((NEW, HQ), 7.0, device="cuda")
            rc = L.pa_varlen_fwd_sinks(q.data_ptr(), pool.data_ptr(), table.data_ptr(),
                                       qsl.data_ptr(), seq.data_ptr(), NEW, NEW,
                                       ctypes.byref(shape), 1 / math.sqrt(d), WINDOW, SINKS,
                                       out.data_ptr(), lse.data_ptr(), None)
            torch.cuda.synchronize()
            code, left = i32(-1), i32(-1)
            rc2 = L.pa_get_device_error(ctypes.byref(code), None)
            rc3 = L.pa_test_window_left(ctypes.byref(left))
            return [rc, rc2, rc3, code.value], left.value, out, lse

        status, left, out1, lse1 = run()
        rec = dict(d=d, plain=status, plain_left=left)
        # CTA 0: rows 0-63 of kv head 0 see positions 489 to 1063 and the first
        # eight: 37 pieces from 480 on and one, five tiles; the last but one is 3.
        assert L.pa_test_mute_window_tile(0, 3) == 0
        status, left, out2, lse2 = run()
        assert L.pa_test_mute_window_tile(-1, -1) == 0
        differ = ((lse1 != lse2) | (out1 != out2).any(-1)).view(-1, 4 * 16, HKV, HQ // HKV)
        rec.update(muted=status, left=left,
                   units=differ.any(3).any(1).nonzero().tolist())
        status, left, out3, lse3 = run()
        rec.update(after=status, left_after=left,
                   same=bool(torch.equal(out1, out3) and torch.equal(lse1, lse3)))
        records.append(rec)
    print(json.dumps(records), flush=True)


if __name__ == "__main__":
    main(sys.argv[1])
