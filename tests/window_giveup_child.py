"""Child process of test_gpu_window_giveup.py: drives a test build of the
library (short bounded waits, the skip hooks) through its C ABI and prints one
JSON line with what it saw.

  python -m tests.window_giveup_child <path of the test build>

Windowed decode in its ring forms (K and V in a box each: bf16, d 128; both in
one: bf16, d 64, and e4m3), on clusters of eight CTAs and on lone CTAs, with
warps that walk their ring several times.  One box of one warp is left out, or
issued only after the wait for it has run out: a warp that gives up must issue
nothing more and wait for every box that is on its way.
"""

import ctypes
import json
import math
import sys

import torch

from tests.timeout_child import Shape

HQ, HKV, BS, SINKS = 16, 4, 16, 8


def main(path):
    L = ctypes.CDLL(path)
    P, i32, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    SP = ctypes.POINTER(Shape)
    L.pa_decode_window.argtypes = [P, P, P, P, SP, f32, i32, i32, P, P, P]
    L.pa_decode_window_fp8.argtypes = [P, P, P, P, SP, f32, f32, f32, i32, i32, P, P, P]
    L.pa_get_device_error.argtypes = [ctypes.POINTER(i32), P]
    g = torch.Generator("cuda").manual_seed(74)
    records = []
    for d, fp8 in ((128, False), (64, False), (128, True)):
        for clusters in (True, False):
            # Eight shares of ~2000 tokens over 16 warps, or one CTA of four warps
            # per request and kv head.
            seqs = [20000, 300] if clusters else [2100] + [40 + k for k in range(90)]
            window = 16384 if clusters else 2048
            blocks = [-(-n // BS) for n in seqs]
            nb, width = sum(blocks), max(blocks)
            ids = torch.randperm(nb, generator=g, device="cuda").int()
            table = torch.full((len(seqs), width), -1, dtype=torch.int32, device="cuda")
            k = 0
            for i, n in enumerate(blocks):
                table[i, :n] = ids[k:k + n]
                k += n
            pool = torch.randn((nb, 2, BS, HKV, d), generator=g, device="cuda")
            pool = (pool * 40).clamp(-448, 448).to(torch.float8_e4m3fn) if fp8 else pool.bfloat16()
            q = torch.randn((len(seqs), HQ, d), generator=g, device="cuda").bfloat16()
            seq = torch.tensor(seqs, dtype=torch.int32, device="cuda")
            shape = Shape(len(seqs), HQ, HKV, d, BS, nb, width)
            scales = (0.02, 0.03) if fp8 else ()
            call = L.pa_decode_window_fp8 if fp8 else L.pa_decode_window

            def run():
                out = torch.full_like(q, 7.0)
                lse = torch.full((len(seqs), HQ), 7.0, device="cuda")
                rc = call(q.data_ptr(), pool.data_ptr(), table.data_ptr(), seq.data_ptr(),
                          ctypes.byref(shape), 1 / math.sqrt(d), *scales, window, SINKS,
                          out.data_ptr(), lse.data_ptr(), None)
                torch.cuda.synchronize()
                code, left = i32(-1), (i32 * 2)(-1, -1)
                rc2 = L.pa_get_device_error(ctypes.byref(code), None)
                rc3 = L.pa_test_decode_left(left)
                return [rc, rc2, rc3, code.value], list(left), out, lse

            status, left, out1, lse1 = run()
            name = f"d{d}{' e4m3' if fp8 else ''}{' clusters' if clusters else ''}"
            records.append(dict(name=name, box=None, status=status, left=left))
            # Sub-blocks of the share's first warp: share 3 has 129 of 1025 (the first
            # tokens' one and 1024 of the window) for 16 warps, the lone CTA 130 (one
            # and 129, from position 48 on) for 4.
            per_warp = 9 if clusters else 33
            boxes = per_warp if d * (1 if fp8 else 2) <= 128 else 2 * per_warp
            share = 3 if clusters else 0
            for hook in (L.pa_test_skip_decode_box, L.pa_test_late_decode_box):
                for box in (0, 1, 2, 3, 4, 5, boxes - 2, boxes - 1):
                    assert hook(share, box) == 0
                    status, left, out2, lse2 = run()
                    assert L.pa_test_skip_decode_box(-1, -1) == 0
                    differ = (lse1 != lse2) | (out1 != out2).any(-1)
                    rows = differ.nonzero().tolist()
                    status3, left3, out3, lse3 = run()
                    records.append(dict(
                        name=name, box=box, late=hook is L.pa_test_late_decode_box, status=status,
                        left=left, rows=rows, after=status3, left_after=left3,
                        same=bool(torch.equal(out1, out3) and torch.equal(lse1, lse3))))
    print(json.dumps(records), flush=True)


if __name__ == "__main__":
    main(sys.argv[1])
