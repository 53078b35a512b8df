"""The transforming append at its edges: tables with bad ids, and what an 8-bit pool holds of awkward values."""
import numpy as np
import pytest
import torch

from speculative_decoding_verify_paged_gb300 import _lib as L
from speculative_decoding_verify_paged_gb300 import step as S
from speculative_decoding_verify_paged_gb300 import workloads as W

import test_gpu_heads as T
from _helpers import status_of, upload

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("batch,which", [(3, 1), (40, 0), (40, 39), (1500, 1400)])
def test_a_bad_id_of_a_partly_filled_block(batch, which, shared):
    """The id that a sequence's first new row goes to is out of range: SV_ERR_BAD_BLOCK_ID. With reference counts nothing
    is written at all; without them no row goes through that id, committed rows stay, and what is written of
    the other rows is as it should be."""
    n = 12
    case = W.custom(71, batch=batch, ctx_lens=[5 + b % 11 for b in range(batch)], n_q=[n] * batch, num_q_heads=4, num_kv_heads=2, head_dim=64,
                    block_size=16, vocab=16, use_bank=False)
    q, k, v, t, _ = T.make(batch * n, 4, 2, 64, torch.bfloat16, 64)

    def call(bad):
        kv, d, buf = upload(case)
        if shared:
            kv.ref_count = torch.zeros(case.state.k_pool.shape[0], dtype=torch.int32, device="cuda")
            kv.ref_count[kv.block_table[kv.block_table >= 0].long()] = 1
        if bad is not None:
            kv.block_table[which, 0] = bad
        qo = torch.full(q.shape, 5.0, dtype=q.dtype, device="cuda")
        held = [x for x in (kv.k_pool, kv.v_pool, qo, kv.block_table, kv.free_list, kv.free_top, kv.ref_count) if x is not None]
        before = [x.clone() for x in held]
        L.kv_append_rope(kv, t, k, v, d.cu_q, buf.status, q=q, q_out=qo)
        torch.cuda.synchronize()
        assert status_of(buf) == (0 if bad is None else 6)
        return before, held

    _, good = call(None)
    for bad in (-1, case.state.k_pool.shape[0], 1 << 30):
        before, held = call(bad)
        if shared:
            for x, y in zip(before, held):
                assert torch.equal(x, y)
            continue
        for x, y, z in zip(before[:3], held, good):  # the pools and the queries
            assert ((y == x) | (y == z)).all()
        block = int(case.state.block_table[which, 0])  # what the bad id stands in for: untouched
        assert torch.equal(held[0][block], before[0][block]) and torch.equal(held[1][block], before[1][block])


def nearest_code(y):
    """The E4M3 code nearest to each y (ties to the even mantissa, saturating), and how far y is from the border to the
    code on its other side, from the format: sign, exponent with bias 7, three mantissa bits, 448 the largest."""
    c = np.arange(0x7F)
    size = np.where(c < 8, c * 2.0 ** -9, (1 + c % 8 / 8) * 2.0 ** (c // 8 - 7.0))
    a = np.minimum(np.abs(y), size[-1])
    hi = np.searchsorted(size, a).clip(1, len(c) - 1)
    lo = hi - 1
    middle = (size[lo] + size[hi]) / 2
    code = np.where((a > middle) | ((a == middle) & (hi % 2 == 0)), hi, lo)
    other = np.minimum(np.abs(a - middle), np.where(code == hi, np.where(hi + 1 < len(c), (size[hi] + size[np.minimum(hi + 1, len(c) - 1)]) / 2 - a, np.inf),
                                                    np.where(lo > 0, a - (size[np.maximum(lo - 1, 0)] + size[lo]) / 2, np.inf)))
    return np.where(np.signbit(y), code | 0x80, code), other


def test_keys_are_the_nearest_codes():
    """Normalised and rotated keys in an E4M3 pool: the code nearest to the 64-bit y / scale wherever y is further from
    a border between two codes than the fp32 arithmetic is off (2^-20 of the pair's size, as for the rows). Many of the values
    would get another code if they went through bf16."""
    for d, rot, kw in ((128, 128, {}), (64, 32, {"interleaved": True, "offset": 1.0}), (128, 64, {"norm": False})):
        n, hkv = 64, 4
        case = W.custom(72, batch=1, ctx_lens=[7], n_q=[n], num_q_heads=hkv, num_kv_heads=hkv, head_dim=d, block_size=16, vocab=16, dtype="e4m3",
                        use_bank=False)
        kv, step, buf = upload(case)
        _, k, v, t, _ = T.make(n, hkv, hkv, d, torch.bfloat16, rot, **kw)
        L.kv_append_rope(kv, t, k, v, step.cu_q, buf.status)
        torch.cuda.synchronize()
        assert status_of(buf) == 0
        at = torch.arange(7, 7 + n, device="cuda")
        got = kv.k_pool[kv.block_table[0][at // 16].long(), :, at % 16].cpu().numpy()
        y, size = T.want_of(k, t.k_weight, np.arange(7, 7 + n), t)
        want, room = nearest_code(y / kv.k_scale)
        clear = room > 2.0 ** -20 * size / kv.k_scale
        if t.k_weight is None:  # values that are neither normalised nor rotated are exact, ties (one in 32 of them) among them
            clear[:, :, rot:] = True
        assert clear.mean() > 0.99
        # signs of zeros are the arithmetic's own
        same = (got == want) | (((got | want) & 0x7F) == 0)
        assert same[clear].all()
        through_bf16, _ = nearest_code(torch.from_numpy(y).to(torch.bfloat16).double().numpy() / kv.k_scale)
        assert (through_bf16 != want)[clear].sum() > 100


def test_codes_of_nonfinite_values():
    """A NaN is stored as the code 0x7F, an infinity as the largest finite value, by both appends alike."""
    case = W.custom(73, batch=1, ctx_lens=[3], n_q=[4], num_q_heads=2, num_kv_heads=2, head_dim=64, block_size=16, vocab=16, dtype="e4m3", use_bank=False)
    x = torch.randn(4, 2, 64, device="cuda").to(torch.bfloat16)
    x[0, :, 3], x[1, :, 4] = float("nan"), -float("nan")
    x[2, :, 5], x[3, :, 6] = float("inf"), -float("inf")
    x.view(torch.int16)[0, 0, 9] = -1  # a NaN with every bit set
    for rope in (False, True):
        kv, d, buf = upload(case)
        if rope:
            L.kv_append_rope(kv, L.HeadTransform(), x, x, d.cu_q, buf.status)
        else:
            L.kv_append(kv, x, x, d.cu_q, buf.status)
        torch.cuda.synchronize()
        assert status_of(buf) == 0
        at = torch.arange(3, 7, device="cuda")
        for pool in (kv.k_pool, kv.v_pool):
            got = pool[kv.block_table[0][at // 16].long(), :, at % 16]
            assert (got[0, :, 3] == 0x7F).all() and (got[1, :, 4] == 0x7F).all() and got[0, 0, 9] == 0x7F
            assert (got[2, :, 5] == 0x7E).all() and (got[3, :, 6] == 0xFE).all()
            assert ((got & 0x7F) == 0x7F).sum() == 5


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d,rot,kw", [(128, 128, {}), (64, 64, {"interleaved": True}), (40, 24, {})])
def test_a_frequency_that_is_no_number(d, rot, kw, dtype):
    """The angle of an infinite or NaN frequency is a NaN, in its pair of every head and nowhere else."""
    q, k, _, t, pos = T.make(5, 4, 2, d, dtype, rot, **kw)
    qo, ko, q1, k1 = (torch.empty(x.shape, dtype=dtype, device="cuda") for x in (q, k, q, k))
    L.qk_norm_rope(t, q, k, pos, qo, ko)
    t.inv_freq[1], t.inv_freq[3], t.inv_freq[4] = float("nan"), float("inf"), -float("inf")
    L.qk_norm_rope(t, q, k, pos, q1, k1)
    bad = [x for i in (1, 3, 4) for x in ((2 * i, 2 * i + 1) if kw.get("interleaved") else (i, i + rot // 2))]
    good = [x for x in range(d) if x not in bad]
    for x, y in ((qo, q1), (ko, k1)):
        assert torch.isnan(y[:, :, bad]).all() and torch.equal(y[:, :, good], x[:, :, good])
