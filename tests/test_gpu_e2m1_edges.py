"""4-bit caches where the other tests do not reach: pool scales of any size in attention, infinite queries, gathered values to
the bit, and appends of more rows than one wave of CTAs takes."""
import numpy as np
import pytest
import torch

from speculative_decoding_verify_paged_gb300 import ScoreMod
from speculative_decoding_verify_paged_gb300 import _lib as L

import _e2m1 as E
import test_gpu_e2m1 as C
import test_gpu_e2m1_attention as A
import test_gpu_scored as T

pytestmark = pytest.mark.gpu

# heads of 64, 128 and 256 values with a warp's rows, one block and two of the wide kernel, CUDA cores
KERNELS = [(64, 4, 5), (64, 4, 20), (128, 4, 1), (128, 8, 6), (128, 8, 7), (128, 16, 5), (128, 8, 20), (128, 8, 40), (256, 4, 3), (256, 4, 12), (96, 4, 5)]


@pytest.mark.parametrize("cap", [0.0, 20.0, 1000.0])
@pytest.mark.parametrize("scales", [(2.0 ** -64, 2.0 ** 64), (1e-6, 3e4), (3e4, 1e-6), (2.0 ** 64, 2.0 ** -64)], ids=str)
@pytest.mark.parametrize("d,hq,n", KERNELS)
def test_pool_scales_of_any_size(d, hq, n, scales, cap):
    """Keys that are larger or smaller by their pool's scale, with the softmax scale the other way, and values by theirs: the
    tolerance of these caches (test_gpu_e2m1_attention.py), relative to the values."""
    kv, step, buf, msl = A.make(92, [300, 37], [n, max(1, n - 1)], hq, 2, d, 16, ScoreMod(softcap=cap))
    step.scale *= kv.k_scale / scales[0]
    kv.k_scale, kv.v_scale = scales
    T.assert_near(A.attend(kv, step, buf, msl), A.reference(kv, step, step.mod, step.scale), False)


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


@pytest.mark.parametrize("d", [32, 96, 128, 256])
@pytest.mark.parametrize("scales", [(0.75, 1.25), (1e-6, 3.3e4), (2.0 ** -64, 2.0 ** 64)], ids=str)
def test_gathered_values_to_the_bit(d, scales):
    """A code times fp32(s * scale) in fp32, rounded once to bf16."""
    ctx, hkv, bs = [300, 0, 17, 64, 1], 3, 16
    kv, _ = C.filled("e2m1", 24, ctx, hkv, d, bs)
    kv.k_scale, kv.v_scale = scales
    kv.v_block_scales[int(kv.block_table[0, 1]), :, 3, 0] = 0xB4  # a negative scale
    kv.v_block_scales[int(kv.block_table[0, 1]), :, 4, 1] = 0x7F  # NaN
    cu = torch.tensor(np.concatenate([[0], np.cumsum(ctx)]), dtype=torch.int32, device="cuda")
    outs = [torch.empty((sum(ctx), hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    L.kv_gather(kv, *outs, cu, first=torch.zeros(len(ctx), dtype=torch.int32, device="cuda"))
    table = kv.block_table.cpu().numpy()
    for got, name, scale in zip(outs, "kv", scales):
        codes, block_scales = (np.concatenate([getattr(kv, name + x).cpu().numpy()[table[b, np.arange(c) // bs], :, np.arange(c) % bs]
                                               for b, c in enumerate(ctx)]) for x in ("_pool", "_block_scales"))
        code = E.values(codes, np.full_like(block_scales, 0x38), 1.0).astype(np.float32)
        s = np.where(block_scales & 128, -1, 1) * np.append(E.e4m3_table(), np.nan)[block_scales & 127]
        step = (s.astype(np.float32) * np.float32(scale)).astype(np.float32).repeat(16, -1)
        want = torch.from_numpy(code * step).to(torch.bfloat16)
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(got.cpu()), nan) and torch.equal(got.cpu()[~nan].view(torch.int16), want[~nan].view(torch.int16))


@pytest.mark.parametrize("n", [48, 49, 64])
def test_append_of_very_many_rows(n):
    """400 sequences of 48 to 64 rows: just within one wave of CTAs with 32 rows each, just past it, and well past."""
    _, kv, step, buf = C.make(25, [3 + b % 60 for b in range(400)], [n] * 400, hq=1, hkv=1, d=32, bs=64)
    before = C.host(kv)
    L.kv_append(kv, step.new_k, step.new_v, step.cu_q, buf.status)
    torch.cuda.synchronize()
    assert int(buf.status) == 0
    C.assert_stored(kv, before, step.cu_q, step.new_k, step.new_v)
