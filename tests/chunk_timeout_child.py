"""Child process of test_gpu_chunk_timeout.py (run with TREEVERIFY_LIB naming
the development build): a call whose CTA 0 never receives the loads of one
K or V tile, then the same call without the hook on the same stream.  Prints
one JSON line per withheld tile."""

import ctypes
import json
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, HERE)
sys.path.insert(0, os.path.dirname(HERE))

import torch  # noqa: E402

import test_gpu_chunk as TC  # noqa: E402
from speculative_decoding_tree_attn_gb300 import capi  # noqa: E402

SHORT_NS = 200_000  # 0.2 ms wait limit while the hook is set


def main():
    set_hooks = capi.lib().tv_test_set_chunk_hooks
    set_hooks.restype, set_hooks.argtypes = ctypes.c_int, [ctypes.c_ulonglong, ctypes.c_int]
    for D, entry in ((128, 4), (128, 7), (64, 0), (64, 21)):  # K of tile 2, V of tile 3, K of tile 0, V of tile 10
        c = TC._case([700, 900], [100, 70], 8, 2, D, "bf16", 16, seed=3)
        assert set_hooks(SHORT_NS, entry) == 0
        _, _, timed_out = TC._run(c, capi.TV_ATTN_TCGEN05, num_ctas=2)
        assert set_hooks(2_000_000_000, -1) == 0
        out, lse, status = TC._run(c, capi.TV_ATTN_TCGEN05, num_ctas=2)
        TC._check(c, out, lse, True)
        print(json.dumps({"tile": [D, entry], "status": timed_out, "after": status}), flush=True)
    torch.cuda.synchronize()


if __name__ == "__main__":
    main()
