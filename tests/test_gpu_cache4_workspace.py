"""One workspace of pa_decode_fp4 under calls of both types, with and without
weights, in turn: what one leaves behind must not be where another counts."""

import numpy as np
import pytest

from test_gpu_fp4 import assert_out, decode_case, dev, expected, status
from test_gpu_weights import assert_weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,G", [(64, 1), (64, 8), (128, 2), (128, 8)])
def test_types_and_weights_in_turn(cuda_device, D, G):
    import torch

    import paged_kv_cache_357_b200 as pa

    lens, H, width = [3000, 5, 2500, 1300], 2, 200
    ws, sets = None, {}
    for dtype in ("bf16", "fp16"):
        c = decode_case([41, D, G], lens, G * H, H, D, 16, dtype, width=width)
        sets[dtype] = c, expected(c), dev(c["kp"], cuda_device), dev(c["vp"], cuda_device)
    ws = pa.alloc_decode_fp4_workspace(4, G * H, sets["bf16"][2], width)
    for i in range(16):
        dtype, weighted = ("bf16", "fp16")[i // 2 % 2], (i + i // 4) % 2 == 0
        c, (out, _, added, tol, wtol), kp, vp = sets[dtype]
        q = c["q"].to(cuda_device)
        got, st = torch.full_like(q, float("nan")), status(cuda_device)
        w = torch.zeros((4, H, width * 16), device=cuda_device) if weighted else None
        pa.pa_decode_fp4(q, kp, vp, dev(c["tables"], cuda_device), dev(c["lens"], cuda_device), c["scale"], got, ws,
                         weights=w, dev_status=st)
        assert int(st) == 0
        assert_out(got, out, tol, dtype, f"call {i}")
        if weighted:
            assert_weights(w, np.zeros(tuple(w.shape), np.float32), added, wtol, c["lens"], 1)


@pytest.mark.parametrize("D", [64, 128])
def test_sizes_do_not_depend_on_the_type(cuda_device, D):
    import ctypes

    import torch

    import paged_kv_cache_357_b200 as pa
    from paged_kv_cache_357_b200 import _lib

    sms = torch.cuda.get_device_properties(cuda_device).multi_processor_count
    for Hq in (2, 4, 8, 16):
        base = set()
        for dtype in (_lib.PA_FP16, _lib.PA_BF16):
            d = _lib.PoolDesc(9, 16, 2, D, dtype)
            for ctas in (0, 3 * sms):
                o = _lib.DecodeOpts(ctas, 0)
                sizes = [_lib.load().pa_decode_fp4_workspace_bytes(5, Hq, width, ctypes.byref(d), ctypes.byref(o))
                         for width in (0, 7)]
                assert sizes[1] > sizes[0] > 0
                base.add(tuple(sizes))
        assert len(base) == 1
