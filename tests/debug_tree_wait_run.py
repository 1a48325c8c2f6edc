"""Run in a process of its own (see test_tree_wait_gpu.py).

Loads the debug build of the library, whose waits in ffd_decode_tree can be given a
limit of their own, and lets them run out in every form of the kernels.  Exits
non-zero on the first failure; prints one summary line on success."""
import ctypes
import os
import sys
import time

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, HERE)
sys.path.insert(0, os.path.dirname(HERE))

from sparse_long_context_ffd_b200 import ffd  # noqa: E402
from test_tree_gpu import FORMATS, Case  # noqa: E402


def flags(ws):
    f = ctypes.c_uint32(0)
    status = ffd.load_library().ffd_check_device_status(ws.data_ptr(), ctypes.byref(f),
                                                        torch.cuda.current_stream().cuda_stream)
    return status, f.value


def main():
    ffd.use_debug_library()
    lib = ffd.load_library()
    lib.ffd_debug_tree_wait_limit.argtypes = [ctypes.c_uint64]
    lib.ffd_debug_tree_wait_limit.restype = None
    runs = 0
    for fmt in FORMATS:
        for n, G in [(4, 2), (4, 8), (8, 8), (16, 8), (32, 8), (63, 8)]:
            # one unit a CTA with many tiles (the ring goes round), and CTAs with many units
            for B, Hkv, cap, lengths in [(1, 4, 64 * 1024, [64 * 1024 - 5]),
                                         (40, 3, 768, [(131 * i) % 700 + n for i in range(40)])]:
                c = Case(fmt, B, n, G, Hkv, cap, lengths, seed=n).device()
                # what lies around the output and the workspace stays as it is
                ws = torch.full((c.ws.numel() + 512,), 0x5A, dtype=torch.uint8, device="cuda")
                ws[256:256 + 256] = 0
                c.ws, guarded = ws[256:-256], ws
                out = torch.full((c.out.numel() + 256,), 7.0, dtype=torch.bfloat16, device="cuda")
                c.out = out[128:-128].view(c.out.shape)
                want = c.run().clone()
                assert flags(c.ws) == (ffd.FFD_OK, 0)
                for limit in (0, 1000, 10000):
                    lib.ffd_debug_tree_wait_limit(limit)
                    t0 = time.monotonic()
                    c.run()
                    took = time.monotonic() - t0
                    status, bits = flags(c.ws)
                    assert took < 1.0, f"{took} s: the CTA's waits did not end together"
                    if limit == 0:
                        assert (status, bits) == (ffd.FFD_ERR_TIMEOUT, ffd.FFD_DEVICE_FLAG_TIMEOUT), (status, bits)
                    else:
                        assert bits in (0, ffd.FFD_DEVICE_FLAG_TIMEOUT)
                    assert (guarded[:256] == 0x5A).all() and (guarded[-256:] == 0x5A).all()
                    assert (out[:128] == 7.0).all() and (out[-128:] == 7.0).all()
                    runs += 1
                lib.ffd_debug_tree_wait_limit(2 * 10 ** 9)
                c.out.fill_(9.0)
                assert torch.equal(c.run().view(torch.int16), want.view(torch.int16))
                assert flags(c.ws) == (ffd.FFD_OK, 0)
    torch.cuda.synchronize()
    print(f"tree waits: {runs} calls with short limits ended and were reported", flush=True)


if __name__ == "__main__":
    main()
