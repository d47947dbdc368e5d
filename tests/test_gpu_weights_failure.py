"""What a decode that fails does to accumulated weights: they outlast the call,
so the rows that it cannot finish stay as they were."""

import numpy as np
import pytest

import cache4_testlib as ref
from test_gpu_fp4 import decode_case, dev, status
from test_gpu_weights import assert_weights, case16, expected16, prior

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,D", [("16", 128), ("16", 64), ("fp4", 128), ("fp4", 64)])
@pytest.mark.parametrize("bad", [-1, 10**6])
def test_a_bad_block_leaves_its_sequence(cuda_device, kind, D, bad):
    import torch

    import paged_kv_cache_357_b200 as pa

    lens = [40, 700, 5, 33]
    if kind == "16":
        c = case16([D, 5], lens, 8, 2, D, 16, "bf16")
        _, _, added, _, wtol = expected16(c)
        q, kp, vp = (c[k].to(cuda_device) for k in ("q", "kp", "vp"))
        rng = c["rng"]
    else:
        c = decode_case([D, 5], lens, 8, 2, D, 16, "bf16")
        _, _, added, _, wtol = ref.attend(ref.f64(c["q"]), ref.pool_values(c["kp"], D), ref.pool_values(c["vp"], D),
                                          c["tables"], c["lens"], c["scale"], 16)
        q, kp, vp = c["q"].to(cuda_device), dev(c["kp"], cuda_device), dev(c["vp"], cuda_device)
        rng = np.random.default_rng(5)
    width = c["tables"].shape[1]
    before = prior(rng, 4, 2, width * 16)
    tables = c["tables"].copy()
    tables[1, 30] = bad
    tables[3, 2] = bad  # the last block, of one token
    tables[0, 5] = 10**6  # behind the last block: not read
    w, st, out = dev(before, cuda_device), status(cuda_device), torch.empty_like(q)
    args = (q, kp, vp, dev(tables, cuda_device), dev(c["lens"], cuda_device), c["scale"])
    if kind == "16":
        pa.pa_decode_weights(*args, w, out, pa.alloc_decode_weights_workspace(4, 8, kp, width), dev_status=st)
    else:
        pa.pa_decode_fp4(*args, out, pa.alloc_decode_fp4_workspace(4, 8, kp, width), weights=w, dev_status=st)
    assert int(st) == 101
    assert np.array_equal(w.cpu().numpy()[[1, 3]], before[[1, 3]])
    some = [0, 2]
    assert_weights(w[some], before[some], added[some], wtol[some], c["lens"][some], 1)


def test_a_timeout_leaves_every_row(cuda_device):
    """The hook that withholds the copies: the decode's waits run out, and
    nothing is added, by this call or by one on the same workspace before it
    is zeroed again (one CTA: no unit is split, so no other count is left)."""
    import time

    import torch

    import paged_kv_cache_357_b200 as pa

    c = case16(7, [300, 40, 129], 8, 2, 128, 16, "bf16")
    q, kp, vp = (c[k].to(cuda_device) for k in ("q", "kp", "vp"))
    width = c["tables"].shape[1]
    before = prior(c["rng"], 3, 2, width * 16)
    w, st, out = dev(before, cuda_device), status(cuda_device), torch.empty_like(q)
    ws = pa.alloc_decode_weights_workspace(3, 8, kp, width, 1)
    args = (q, kp, vp, dev(c["tables"], cuda_device), dev(c["lens"], cuda_device), c["scale"], w, out, ws)
    t0 = time.time()
    pa.pa_decode_weights(*args, dev_status=st, num_ctas=1, flags=pa.PA_DECODE_TEST_WITHHOLD_COPIES)
    torch.cuda.synchronize()
    assert time.time() - t0 < 10.0
    assert int(st) == 105 and np.array_equal(w.cpu().numpy(), before)
    st.zero_()
    pa.pa_decode_weights(*args, dev_status=st, num_ctas=1)
    assert int(st) == 105 and np.array_equal(w.cpu().numpy(), before)
    st.zero_()
    ws.zero_()
    pa.pa_decode_weights(*args, dev_status=st, num_ctas=1)
    _, _, added, _, wtol = expected16(c)
    assert int(st) == 0
    assert_weights(w, before, added, wtol, c["lens"], 1)


def test_the_hook_is_refused_where_nothing_waits(cuda_device):
    import paged_kv_cache_357_b200 as pa

    c = case16(8, [30], 4, 2, 64, 16, "bf16")
    with pytest.raises(pa.PaError):
        pa.alloc_decode_weights_workspace(1, 4, c["kp"].to(cuda_device), 2, 1, pa.PA_DECODE_TEST_WITHHOLD_COPIES)
