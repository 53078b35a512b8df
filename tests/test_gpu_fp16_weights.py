"""Attention whose softmax weights are fp16 for the product with V: weights next to scores of any size."""
import numpy as np
import pytest
import torch

from speculative_decoding_verify_paged_gb300 import PagedKV, ScoreMod
from speculative_decoding_verify_paged_gb300 import _lib as L

import test_gpu_scored_edges as X

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("far,slope", [(2000000000, 0.05), (120000000, 0.8)])
@pytest.mark.parametrize("d,hq,n", [(64, 8, 6), (128, 8, 1), (128, 8, 6), (128, 16, 5), (256, 8, 6)])
def test_biased_scores_whose_step_is_sixteen(d, hq, n, far, slope):
    """E4M3 pools: the committed keys' biased scores (base 2) lie between 2^27 and 2^28, where fp32's step is 16: one step above
    the running maximum is past what a weight may be. The new keys, at a distance of nothing, take it all (the usual
    tolerance of these caches)."""
    ctx = [1500, 37]
    slopes = torch.linspace(slope, 1.8 * slope, hq, device="cuda")
    pos = np.concatenate([c + far + np.arange(n) for c in ctx])
    assert 2 ** 27 < slope * far / np.log(2) and 1.8 * slope * far / np.log(2) < 2 ** 28
    X.make(91, ctx, [n, n], hq, 2, d, "e4m3", ScoreMod(slopes=slopes), positions=torch.from_numpy(pos.astype(np.int32)).cuda())


def flat_cache(dt, d, ctx, n, batch, hkv=2, bs=16):
    """Sequences that share their blocks: every key zero, every value 1."""
    blocks = -(-(ctx + n) // bs)
    table = torch.arange(blocks, dtype=torch.int32, device="cuda").expand(batch, -1).contiguous()
    lens = torch.full((batch,), ctx, dtype=torch.int32, device="cuda")
    free = torch.full((blocks,), -1, dtype=torch.int32, device="cuda")
    top = torch.zeros(1, dtype=torch.int32, device="cuda")
    wide = d if dt == "e4m3" else d // 2
    pools = [torch.full((blocks, hkv, bs, wide), code, dtype=torch.uint8, device="cuda") for code in (0, 0x38 if dt == "e4m3" else 0x22)]
    scales = [None, None] if dt == "e4m3" else [torch.full((blocks, hkv, bs, d // 16), 0x38, dtype=torch.uint8, device="cuda") for _ in range(2)]
    return PagedKV(*pools, table, lens, free, top, k_block_scales=scales[0], v_block_scales=scales[1])


def attend(kv, q, out, cu, n, ctx, scale, status, plain):
    """The scored call with nothing modified, or the plain one."""
    args = dict(max_q=n, max_seq_len=ctx + n, scale=scale, status=status)
    if plain:
        need = L.spec_verify_attn_workspace_bytes(kv, q.shape[1], q.shape[0], n, ctx + n)
        L.spec_verify_attn(kv, q, out, cu, workspace=torch.empty(max(256, need), dtype=torch.uint8, device="cuda"), **args)
    else:
        L.spec_verify_attn_scored(kv, q, out, cu, mod=ScoreMod(), **args)
    torch.cuda.synchronize()


@pytest.mark.parametrize("plain", [False, True], ids=["scored", "plain"])
@pytest.mark.parametrize("d,hq,n", [(64, 8, 6), (128, 8, 1), (128, 8, 6), (128, 16, 5), (256, 8, 6), (96, 8, 6)])
def test_scores_whose_step_is_sixteen(d, hq, n, plain):
    """The same without a bias, for the scored call or the plain one: each key's score is one step above that of the key 64
    before it, or equal to it. Outputs are averages of values between 1 and 2."""
    ctx = 1500
    kv = flat_cache("e4m3", d, ctx, n, 2)
    blocks, _, bs, _ = kv.k_pool.shape
    block, slot = (torch.from_numpy(x).cuda() for x in np.divmod(np.arange(blocks * bs), bs))
    kv.k_pool[:, :, :, 0] = 0x38  # 1
    rise = torch.from_numpy((np.arange(blocks * bs) // 64).astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    kv.k_pool[block, :, slot, 1] = rise[:, None]  # (whole numbers: rounded to four bits past 15, still ascending)
    kv.v_pool[block, :, slot] = torch.from_numpy((0x38 + np.arange(blocks * bs) % 9).astype(np.uint8)).cuda()[:, None, None]
    q = torch.zeros((2 * n, hq, d), dtype=torch.bfloat16, device="cuda")
    q[:, :, 0], q[:, :, 1] = 12288.0, 2.0 ** -10
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
    out = torch.full_like(q, float("nan"))
    attend(kv, q, out, cu, n, ctx, 16.0 * 2 ** 10 * float(np.log(2)), status, plain)
    assert int(status) == 0 and bool(((out >= 1) & (out <= 2)).all())


TAILS = [(dt, d, hq, n) for dt in ("e2m1", "e4m3") for d, hq, n in (
    (64, 4, 5), (64, 4, 12), (128, 4, 1), (128, 8, 6), (128, 8, 7), (128, 16, 5), (128, 8, 20), (128, 8, 40), (256, 4, 3), (96, 4, 5))]


@pytest.mark.parametrize("plain", [False, True], ids=["scored", "plain"])
@pytest.mark.parametrize("x", [20.5, 24.5, 27.5])
@pytest.mark.parametrize("dt,d,hq,n", TAILS)
def test_a_flat_tail_next_to_one_large_weight(dt, d, hq, n, x, plain):
    """The first key has weight 1 and a value of 0, all others a weight of 2^-x and values of 1: the output is the tail's share
    alone. A weight counts to 2^-32 of the row's largest (half of the smallest fp16 number, with the largest weight at 2^7 or more), and
    to 2^-11 of itself; the output is rounded to bf16 (2^-8), and the sums' own errors are far below. As many units as there
    are CTAs and more, so that one warp meets the first key and much of the tail."""
    ctx, batch = 640, 400
    kv = flat_cache(dt, d, ctx, n, batch)
    kv.k_pool[0, :, 0], kv.v_pool[0, :, 0] = 0x38 if dt == "e4m3" else 0x22, 0
    q = torch.ones((batch * n, hq, d), dtype=torch.bfloat16, device="cuda")
    out, status = torch.full_like(q, float("nan")), torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = torch.arange(0, batch * n + 1, n, dtype=torch.int32, device="cuda")
    attend(kv, q, out, cu, n, ctx, x * float(np.log(2)) / d, status, plain)
    assert int(status) == 0
    others = (ctx + torch.arange(n, dtype=torch.float64, device="cuda")).repeat(batch)[:, None, None]
    total = 1 + others * 2.0 ** -x
    want = others * 2.0 ** -x / total
    assert bool(((out.double() - want).abs() <= want * (2.0 ** -8 + 2.0 ** -11 + 1e-5) + others * 2.0 ** -32 / total).all())
