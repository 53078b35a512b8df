"""The 32-bit positions of scored attention's work order, asked on the host: a call whose positions would not
fit goes to the CUDA-core kernels, which have none. Nothing here touches a GPU."""
import ctypes

import pytest

from speculative_decoding_verify_paged_gb300 import _lib as L
from speculative_decoding_verify_paged_gb300 import build as B


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


def workspace(lib, *, d, dtype, batch, rows, length, hq=64, hkv=8):
    """More than 608 sequences and heads: the CUDA-core kernels do not split them and need no workspace."""
    kv = L.sv_paged_kv(num_blocks=1 << 16, block_size=64, max_blocks_per_seq=1 << 17, num_kv_heads=hkv, head_dim=d, batch=batch, dtype=dtype)
    return lib.sv_spec_verify_attn_scored_workspace_bytes(ctypes.byref(kv), hq, 1, rows, length)


# A unit (a KV head of a sequence, up to `block` rows of it) has a position for each tile of keys and `lead` more.
# `lead` is 4 for warps of up to 16 rows (blocks of 16 to 32 here), 5 for wider ones.
INSTANCES = [
    # head_dim, dtype (0 bf16, 2 E4M3), batch, rows a sequence (8 query heads a KV head), block, tile, lead
    (256, 0, 1024, 64, 32, 16, 4),  # sequences that share a long prefix
    (256, 0, 4096, 64, 32, 16, 4),
    (256, 0, 4096, 1, 16, 16, 4),
    (256, 2, 2048, 64, 32, 32, 4),
    (256, 2, 4096, 2, 16, 32, 4),
    (128, 0, 4096, 3, 24, 32, 5),
    (128, 0, 4096, 64, 96, 32, 5),
    (128, 2, 4096, 64, 96, 64, 5),
    (64, 0, 4096, 8, 64, 64, 5),
    (64, 2, 4096, 64, 128, 128, 5),
]


@pytest.mark.parametrize("d,dtype,batch,n,block,tile,lead", INSTANCES)
def test_positions_stay_within_32_bits(lib, d, dtype, batch, n, block, tile, lead):
    units = batch * 8 * -(-8 * n // block)
    most = (2 ** 31 - 1) // units - lead  # tiles of the longest sequences that fit
    assert most * tile < 1 << 30
    assert workspace(lib, d=d, dtype=dtype, batch=batch, rows=n, length=most * tile) > 0
    assert workspace(lib, d=d, dtype=dtype, batch=batch, rows=n, length=most * tile + 1) == 0
    assert workspace(lib, d=d, dtype=dtype, batch=batch, rows=n, length=1 << 30) == 0


def test_named_shapes(lib):
    """Two shapes whose positions pass 2^31, and rows of a KV head that do not fit 32 bits."""
    assert workspace(lib, d=256, dtype=0, batch=1024, rows=64, length=262144) == 0
    assert workspace(lib, d=256, dtype=0, batch=4096, rows=64, length=131072) == 0
    assert workspace(lib, d=256, dtype=0, batch=1024, rows=64, length=32768) > 0
    assert workspace(lib, d=128, dtype=0, batch=1, rows=64, length=64, hq=1 << 30, hkv=1) == 0
