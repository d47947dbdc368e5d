"""How many bits a softmax weight keeps on its way to V, where outputs nearly
cancel: pairs of rows v, -v under weights that differ in their last bits.

Tolerance.  q has one element that is not zero, so a score is one product,
exact in fp32, and the reference (a running max, the same for a row's tokens)
leaves a sum of at most 8 + 2^-6, rounded by 2^-21.  A weight is then off by at
most 2^-21 (that sum), 2^-22 (the exponential), 2^-22 (its split into 16-bit
values) and its share of the roundings of the products' sum (n of at most 6,
2^-23 each, and as many of merges): under 2^-19 of itself.  Of A = sum p |v|
that is 2^-19 * A, and the output's own rounding comes on top.
"""

import numpy as np
import pytest

import cache4_testlib as ref
from test_gpu_fp4 import dev

pytestmark = pytest.mark.gpu

LENS = [2, 4, 6] * 30


def pairs(seed, G, D, dtype):
    """(q, keys, values, tables, out, A) of sequences of nearly cancelling
    pairs over blocks of 8; keys and values are held exactly by 4-bit pools."""
    rng = np.random.default_rng(seed)
    S, H, block = len(LENS), 2, 8
    k, v = np.zeros((S, H, block, D)), np.zeros((S, H, block, D))
    k[..., 0] = ref.E2M1[rng.integers(0, 8, (S, H, block))] * rng.choice([-1, 1], (S, H, block))
    k[..., 1] = 6.0  # the group's scale is 1
    half = ref.E2M1[rng.integers(0, 8, (S, H, block // 2, D))] * rng.choice([-1, 1], (S, H, block // 2, D))
    half[..., ::16] = 6.0
    v[:, :, 0::2], v[:, :, 1::2] = half, -half
    q = ref.normal16(rng, (S, H * G, D), dtype, 2.0**-8)
    q[..., 1:] = 0.0
    out, A = np.zeros((S, H * G, D)), np.zeros((S, H * G, D))
    for s, n in enumerate(LENS):
        for i in range(H * G):
            x = k[s, i // G, :n] @ ref.f64(q)[s, i]
            p = np.exp(x - x.max())
            p /= p.sum()
            out[s, i], A[s, i] = p @ v[s, i // G, :n], p @ np.abs(v[s, i // G, :n])
    tables = np.arange(S, dtype=np.int32)[:, None]
    return q, k, v, tables, out, A


def assert_close(got, out, A, dtype):
    small = 2.0**-25 if dtype == "fp16" else 0.0
    worst = np.abs(ref.f64(got) - out) - (2.0**-19 * A + ref.HALF_STEP[dtype] * np.abs(out) * 1.01 + small)
    assert (worst <= 0).all(), f"{worst.max():.3e} beyond its bound"


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("G", [1, 4, 8])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("weighted", [False, True])
def test_weights_over_4_bit_pools_keep_their_bits(cuda_device, dtype, G, D, weighted):
    import torch

    import paged_kv_cache_357_b200 as pa

    q, k, v, tables, out, A = pairs([G, D], G, D, dtype)
    kp, vp = (dev(ref.join_tiles(*ref.quantise(x)), cuda_device) for x in (k, v))
    assert np.array_equal(ref.pool_values(kp.cpu().numpy(), D), k)
    assert np.array_equal(ref.pool_values(vp.cpu().numpy(), D), v)
    S, width = len(LENS), 1
    w = torch.zeros((S, 2, 8), device=cuda_device) if weighted else None
    got = torch.full_like(q, float("nan")).to(cuda_device)
    pa.pa_decode_fp4(q.to(cuda_device), kp, vp, dev(tables, cuda_device), dev(np.array(LENS, np.int32), cuda_device), 1.0,
                     got, pa.alloc_decode_fp4_workspace(S, 2 * G, kp, width if weighted else 0), weights=w)
    assert_close(got, out, A, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_weights_over_16_bit_pools_at_head_dim_64_keep_their_bits(cuda_device, dtype, G):
    import torch

    import paged_kv_cache_357_b200 as pa

    q, k, v, tables, out, A = pairs([G, 64], G, 64, dtype)
    kp, vp = (torch.from_numpy(x).to(ref.torch_type(dtype)).to(cuda_device) for x in (k, v))
    S = len(LENS)
    got, w = torch.full_like(q, float("nan")).to(cuda_device), torch.zeros((S, 2, 8), device=cuda_device)
    pa.pa_decode_weights(q.to(cuda_device), kp, vp, dev(tables, cuda_device), dev(np.array(LENS, np.int32), cuda_device),
                         1.0, w, got, pa.alloc_decode_weights_workspace(S, 2 * G, kp, 1))
    assert_close(got, out, A, dtype)
