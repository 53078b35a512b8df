"""kv_append refuses rows that do not fit the cache before anything is launched (pools of every type; no GPU is needed)."""
from types import SimpleNamespace

import pytest
import torch

from speculative_decoding_verify_paged_gb300 import _lib as L


def cache(dtype, hkv=2, d=64):
    """A cache's numbers; no pointer of it is looked at."""
    s = L.sv_paged_kv(num_blocks=16, block_size=16, max_blocks_per_seq=4, num_kv_heads=hkv, head_dim=d, batch=1, dtype=dtype, k_scale=1.0, v_scale=1.0)
    return SimpleNamespace(is_e2m1=False, struct=lambda: s)


@pytest.mark.parametrize("dtype,rows", [(L.SV_DTYPE_BF16, torch.bfloat16), (L.SV_DTYPE_F32, torch.float32), (L.SV_DTYPE_E4M3, torch.bfloat16)])
def test_rows_that_do_not_fit(dtype, rows):
    kv = cache(dtype)
    x = torch.zeros((5, 2, 64), dtype=rows)
    other = torch.float32 if rows == torch.bfloat16 else torch.bfloat16
    for k, v in ((x, x[:4]), (x[:4], x), (x[:, :1], x[:, :1]), (x, x[:, :, :32]), (x.to(other), x), (x, x.to(other)), (x.to(other), x.to(other)),
                 (x, torch.zeros((5, 2, 72), dtype=rows))):
        with pytest.raises(ValueError):
            L.kv_append(kv, k, v, None, None)
    with pytest.raises(TypeError):
        L.kv_append(kv, x, x, None, None)  # rows that fit, and are not on a GPU
