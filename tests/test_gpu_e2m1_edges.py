"""4-bit caches where the other tests do not reach: infinite queries."""
import pytest
import torch

from speculative_decoding_verify_paged_gb300 import ScoreMod

import test_gpu_e2m1_attention as A
import test_gpu_scored as T

pytestmark = pytest.mark.gpu

# heads of 64, 128 and 256 values with a warp's rows, one block and two of the wide kernel, CUDA cores
KERNELS = [(64, 4, 5), (64, 4, 20), (128, 4, 1), (128, 8, 6), (128, 8, 7), (128, 16, 5), (128, 8, 20), (128, 8, 40), (256, 4, 3), (256, 4, 12), (96, 4, 5)]


@pytest.mark.parametrize("d,hq,n", KERNELS)
def test_infinite_queries_under_a_cap(d, hq, n):
    """An infinite query value makes its row's scores the cap's ends, whatever finite values stand beside it: none of them is an
    infinity of its own in fp16."""
    kv, step, buf, msl = A.make(93, [300, 37], [n, n], hq, 2, d, 16, ScoreMod(softcap=3.0))
    clean = A.attend(kv, step, buf, msl)
    codes = kv.k_pool[..., 0]  # the first two values of every key: of opposite signs, and not zero
    kv.k_pool[..., 0] = torch.where((codes & 8) > 0, torch.full_like(codes, 0x2A), torch.full_like(codes, 0xA2))
    kv.k_block_scales[..., 0] = torch.where((kv.k_block_scales[..., 0] & 127) == 0, torch.full_like(codes, 0x38), kv.k_block_scales[..., 0])
    for row, big in ((0, 1e6), (n, 1e30)):
        step.q[row, :, 0], step.q[row, :, 1] = float("inf"), big
        step.q[row, 1::2, 0] = -float("inf")
    out = A.attend(kv, step, buf, msl)
    assert clean.shape == out.shape
    T.assert_near(out, A.reference(kv, step, step.mod), False)
