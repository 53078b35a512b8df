"""Attention over E4M3 pools with as many query rows a KV head as a unit of the tcgen05 kernel holds (128), and more: every tile
of every unit is the pool's, call after call."""
import pytest
import torch

from speculative_decoding_verify_paged_gb300 import PagedKV
from speculative_decoding_verify_paged_gb300 import _lib as L

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [6, 20, 31, 32, 40, 64])
def test_many_rows_of_many_sequences(n):
    """400 sequences that share one context of random codes and differ in their last rows. Each of 20 calls gives the bits of
    the first, and the first is the CUDA-core kernel's (fp32) but for fp16 weights (2^-11 each, and queries that fp16 holds) and
    the outputs' rounding to bf16 (2^-8), both relative to the values' size: 2^-7 of a row's norm over its values'."""
    batch, ctx, hq, hkv, d, bs = 400, 640, 8, 2, 128, 16
    g = torch.Generator(device="cuda").manual_seed(n)
    shared, own = ctx // bs, -(-n // bs)
    blocks = shared + batch * own
    pools = [torch.randn((blocks, hkv, bs, d), generator=g, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8) for _ in range(2)]
    first = torch.arange(shared, dtype=torch.int32, device="cuda").expand(batch, -1)
    rest = (shared + torch.arange(batch * own, dtype=torch.int32, device="cuda")).view(batch, own)
    kv = PagedKV(*pools, torch.cat((first, rest), 1).contiguous(), torch.full((batch,), ctx, dtype=torch.int32, device="cuda"),
                 torch.full((blocks,), -1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"))
    q = torch.randn((batch * n, hq, d), generator=g, device="cuda").to(torch.bfloat16)
    cu = torch.arange(0, batch * n + 1, n, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(256, L.spec_verify_attn_workspace_bytes(kv, hq, batch * n, n, ctx + n)), dtype=torch.uint8, device="cuda")

    def attend():
        out = torch.full_like(q, float("nan"))
        L.spec_verify_attn(kv, q, out, cu, max_q=n, max_seq_len=ctx + n, scale=d ** -0.5, status=status, workspace=ws)
        torch.cuda.synchronize()
        assert int(status) == 0
        return out
    outs = attend()
    for _ in range(20):
        assert torch.equal(attend(), outs)
    L.set_attn_path("cuda_cores")
    try:
        want = attend().double()
    finally:
        L.set_attn_path("auto")
    err = (outs.double() - want).norm(dim=-1)
    assert bool((err <= 2.0 ** -7 * want.norm(dim=-1).clamp(min=0.05 * float(want.norm(dim=-1).max()))).all())
