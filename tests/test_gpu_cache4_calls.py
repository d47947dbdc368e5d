"""Whole numbers of the wrappers that a C int does not hold: refused, not cut
to their low 32 bits; and flags of the eviction that are none."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wrong", [1 << 31, 1 << 32, (1 << 32) + 1, -(1 << 31) - 1])
def test_numbers_past_32_bits(cuda_device, wrong):
    import torch

    import paged_kv_cache_357_b200 as pa

    i32 = dict(dtype=torch.int32, device=cuda_device)
    for fp4 in (False, True):
        shape = pa.fp4_pool_shape(4, 1, 16, 128) if fp4 else (4, 1, 16, 128)
        kp = torch.zeros(shape, dtype=torch.uint8 if fp4 else torch.bfloat16, device=cuda_device)
        q = torch.ones((1, 1, 128), dtype=torch.bfloat16, device=cuda_device)
        tables, lens = torch.tensor([[1, 2]], **i32), torch.tensor([20], **i32)
        w, kept, new_lens = torch.zeros((1, 1, 32), device=cuda_device), torch.zeros((1, 1, 9), **i32), torch.zeros(1, **i32)
        for name in ("sinks", "recent"):
            with pytest.raises(ValueError, match=name):
                pa.pa_evict(tables, lens, torch.tensor([9], **i32), w, kept, new_lens, kp, kp.clone(), **{name: wrong})
        with pytest.raises(ValueError, match="num_new"):
            if fp4:
                pa.pa_decode_fp4(q, kp, kp.clone(), tables, lens, 1.0, torch.empty_like(q),
                                 pa.alloc_decode_fp4_workspace(1, 1, kp, 2), weights=w, num_new=wrong)
            else:
                pa.pa_decode_weights(q, kp, kp.clone(), tables, lens, 1.0, w, torch.empty_like(q),
                                     pa.alloc_decode_weights_workspace(1, 1, kp, 2), num_new=wrong)


@pytest.mark.parametrize("flags", [1, 2, 4, 257, 512, 1 << 32, -1])
def test_flags_of_the_eviction(cuda_device, flags):
    """Only the test hook is one: 1 would say that 16-bit pools are 4-bit pools."""
    import torch

    import paged_kv_cache_357_b200 as pa

    i32 = dict(dtype=torch.int32, device=cuda_device)
    kp = torch.ones((4, 1, 16, 128), dtype=torch.bfloat16, device=cuda_device)
    kept, new_lens = torch.zeros((1, 1, 9), **i32), torch.zeros(1, **i32)
    with pytest.raises(pa.PaError):
        pa.pa_evict(torch.tensor([[1, 2]], **i32), torch.tensor([20], **i32), torch.tensor([9], **i32),
                    torch.zeros((1, 1, 32), device=cuda_device), kept, new_lens, kp, kp.clone(), flags=flags)
    assert (kept == 0).all() and (new_lens == 0).all()
