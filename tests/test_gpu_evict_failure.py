"""The eviction's bounded wait, made to run out on the host's word: one chunk
loads its rows and tells nobody (PA_EVICT_TEST_WITHHOLD), the chunks that
store where it reads give up after about 20 ms."""

import time

import numpy as np
import pytest

from test_gpu_evict import case, check, from_pool, to_pool
from test_gpu_fp4 import dev, status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,D", [("bf16", 128), ("bf16", 64), ("fp4", 128), ("fp4", 64)])
def test_a_chunk_that_never_says_it_is_loaded(cuda_device, kind, D):
    import torch

    import paged_kv_cache_357_b200 as pa

    c = case([51, D], [3000, 900, 40], 2, D, 16, kind)
    w = c["rng"].random((3, 2, c["tokens"])).astype(np.float32)
    # the first chunk's rows of sequence 0 come from far behind, where later chunks store
    w[0, :, :2000] *= 0.01
    budgets = np.array([1500, 600, 30], np.int32)
    want = check(c, cuda_device, w, budgets, 0, 5, room=1500)
    kp, vp = (to_pool(c, p, cuda_device) for p in c["pools"])
    wd, st = dev(w.copy(), cuda_device), status(cuda_device)
    kept = torch.full((3, 2, 1500), -9, dtype=torch.int32, device=cuda_device)
    new_lens = torch.zeros(3, dtype=torch.int32, device=cuda_device)
    args = (dev(c["tables"], cuda_device), dev(c["lens"], cuda_device), dev(budgets, cuda_device), wd, kept, new_lens)
    t0 = time.time()
    pa.pa_evict(*args, kp, vp, 0, 5, dev_status=st, flags=pa.PA_EVICT_TEST_WITHHOLD)
    torch.cuda.synchronize()
    assert time.time() - t0 < 10.0
    assert int(st) == 105
    # every other (sequence, kv head) is as it should be
    others = [(0, 1), (1, 0), (1, 1), (2, 0), (2, 1)]
    for s, h in others:
        n, m = int(c["lens"][s]), int(budgets[s])
        assert torch.equal(kept[s, h, :m], want[3][s, h, :m]) and torch.equal(wd[s, h, :n], want[2][s, h, :n])
        for got, good in zip((kp, vp), want):
            blocks = c["tables"][s, : -(-n // 16)]
            assert np.array_equal(from_pool(c, got)[blocks, h], from_pool(c, good)[blocks, h])
    assert torch.equal(new_lens, want[4])
    # and the next call, on the same context
    check(c, cuda_device, w, budgets, 0, 5, room=1500)


def test_the_hook_without_a_wait(cuda_device):
    """Nobody stores where the withheld chunk reads: nothing runs out."""
    import torch

    import paged_kv_cache_357_b200 as pa

    c = case(52, [40], 1, 64, 16, "bf16")
    kp, vp = (to_pool(c, p, cuda_device) for p in c["pools"])
    w, st = torch.rand((1, 1, c["tokens"]), device=cuda_device), status(cuda_device)
    kept = torch.zeros((1, 1, 20), dtype=torch.int32, device=cuda_device)
    new_lens = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    pa.pa_evict(dev(c["tables"], cuda_device), dev(c["lens"], cuda_device), dev(np.array([20], np.int32), cuda_device), w,
                kept, new_lens, kp, vp, dev_status=st, flags=pa.PA_EVICT_TEST_WITHHOLD)
    assert int(st) == 0
    assert np.array_equal(from_pool(c, kp), c["pools"][0])  # its own rows are not stored either
    with pytest.raises(pa.PaError):
        pa.pa_evict(dev(c["tables"], cuda_device), dev(c["lens"], cuda_device), dev(np.array([20], np.int32), cuda_device),
                    w, kept, new_lens, kp, vp, flags=512)
