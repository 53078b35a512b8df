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
