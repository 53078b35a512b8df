"""Scored attention where rows see different keys: infinities and NaN next to finite values, tile after tile.

A row that does not see such a key has the bits that it has with a finite value in the key's place: weights of unseen
keys are zero either way. Nothing here is compared within a tolerance unless a test says so."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from speculative_decoding_verify_paged_gb300 import ScoreMod
from speculative_decoding_verify_paged_gb300 import _lib as L
from speculative_decoding_verify_paged_gb300 import step as S
from speculative_decoding_verify_paged_gb300 import workloads as W

import test_gpu_scored as T
from _helpers import max_seq_len, status_of

pytestmark = pytest.mark.gpu


def make(seed, ctx, nq, hq, hkv, d, dt, mod, **kw):
    case = W.custom(seed, batch=len(ctx), ctx_lens=ctx, n_q=nq, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=16, vocab=16, dtype=dt,
                    use_bank=False)
    kv, step, buf = T.run(case, mod, **kw)
    return kv, step, buf, max_seq_len(case.state, case.step)


def put(kv, b, t, value, pool="v_pool"):
    """The value (an E4M3 pool: the code) in every head's first place of key t of sequence b, and in one more."""
    rows = getattr(kv, pool)[int(kv.block_table[b, t // 16]), :, t % 16]
    rows[:, 0] = value
    rows[:, rows.shape[1] // 2 + 1] = value


def again(kv, step, buf, msl):
    buf.attn_out.zero_()
    S.attention(kv, step, buf, msl)
    torch.cuda.synchronize()
    assert status_of(buf) == 0
    return buf.attn_out.clone()


@pytest.mark.parametrize("n", [16, 32, 40, 64])  # 64 and 128 rows a unit: one block; 160 and 256: two
def test_nonfinite_values_in_some_of_many_edge_tiles(n):
    """Wide units whose tiles are all at an edge (a window as long as the draft), some with an infinity or NaN and some
    without, in many short sequences: rows that do not see them keep their bits, over and over."""
    window, count = 64, 24
    ctx = [130 + 7 * i for i in range(count)]
    kv, step, buf, msl = make(60, ctx, [n] * count, 8, 2, 128, "bf16", ScoreMod(softcap=20.0, window=window))
    clean = buf.attn_out.clone()
    hit = np.zeros(len(clean), bool)
    for b, c in enumerate(ctx):
        if b % 3 != 2:  # the window's first key: row 0 alone sees it
            put(kv, b, c - window + 1, float("inf"))
            hit[b * n] = True
        if b % 3 != 1:  # the last new row: itself alone
            put(kv, b, c + n - 1, float("nan"))
            hit[b * n + n - 1] = True
    first = None
    for _ in range(30):
        out = again(kv, step, buf, msl)
        assert torch.equal(out[~hit], clean[~hit])
        assert not torch.isfinite(out[hit].float()).all(-1).any()
        assert first is None or torch.equal(first.view(torch.int16), out.view(torch.int16))
        first = out


@pytest.mark.parametrize("dt,d,hq", [("e4m3", 64, 8), ("e4m3", 64, 64), ("e4m3", 128, 8), ("e4m3", 128, 24), ("e4m3", 128, 64), ("e4m3", 256, 8),
                                     ("e4m3", 256, 32), ("e4m3", 96, 8), ("bf16", 64, 8), ("bf16", 128, 8), ("bf16", 128, 48), ("bf16", 256, 8),
                                     ("bf16", 96, 8), ("f32", 64, 8)])
def test_a_seen_nan_reaches_its_rows_and_no_others(dt, d, hq):
    """A NaN among the values of a draft row and of the window's first key: it stands in the same places of the rows that
    see the key, and nowhere else."""
    window = 50
    masks = torch.tensor([1, 3, 5, 9, 17, 1, 3, 5, 9, 17, 33], dtype=torch.int64, device="cuda")
    kv, step, buf, msl = make(61, [200, 37], [5, 6], hq, 2, d, dt, ScoreMod(softcap=20.0, window=window), tree_mask=masks)
    want = buf.attn_out.clone()
    nan = 0x7F if dt == "e4m3" else float("nan")
    minus = 0xFF if dt == "e4m3" else float("nan")
    for b, t, row, code in ((0, 200 + 4, 4, nan), (0, 200 - window + 1, 0, minus), (1, 37 + 2, 7, minus)):
        put(kv, b, t, code)
        want[row, :, 0] = want[row, :, d // 2 + 1] = float("nan")
    out = again(kv, step, buf, msl)
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    keep = ~torch.isnan(want)
    assert torch.equal(out[keep], want[keep])


@pytest.mark.parametrize("dt,d,hq", [("bf16", 64, 8), ("bf16", 128, 8), ("bf16", 128, 32), ("bf16", 128, 48), ("bf16", 256, 8), ("bf16", 96, 8),
                                     ("e4m3", 128, 8), ("e4m3", 256, 8), ("f32", 64, 8)])
def test_a_seen_nonfinite_value_counts_whatever_its_weight(dt, d, hq):
    """A bias so steep that all weights but the nearest key's are zero in fp32: an infinity (E4M3: a NaN) among the
    values of a key that is further back still reaches the rows that see it."""
    kv, step, buf, msl = make(62, [200, 37], [5, 6], hq, 2, d, dt, ScoreMod(slopes=torch.full((hq,), 1000.0, device="cuda")))
    clean = buf.attn_out.clone()
    put(kv, 0, 202, 0x7F if dt == "e4m3" else float("inf"))  # the third of the new keys: rows 2 to 4 see it
    out = again(kv, step, buf, msl)
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[2:5, :, 0] = hit[2:5, :, d // 2 + 1] = True
    assert not torch.isfinite(out[hit].float()).any()
    assert torch.equal(out[~hit], clean[~hit])


@pytest.mark.parametrize("dt,d,hq", [("bf16", 128, 8), ("bf16", 128, 64), ("bf16", 96, 8), ("e4m3", 128, 8), ("f32", 64, 8)])
@pytest.mark.parametrize("cap", [2.5e38, 3.4028234e38])
def test_the_largest_caps_change_nothing(dt, d, hq, cap):
    """Caps whose product with log2(e) is past fp32's range."""
    make(63, [200, 33], [4, 2], hq, 2, d, dt, ScoreMod(softcap=cap))


@pytest.mark.parametrize("dt,d,hq,n", [("bf16", 128, 8, 6), ("bf16", 128, 32, 6), ("bf16", 128, 8, 40), ("bf16", 64, 8, 6), ("e4m3", 128, 8, 6),
                                       ("e4m3", 256, 8, 6), ("f32", 64, 8, 6)])
@pytest.mark.parametrize("far", [1000, 1000000, 2000000000])
def test_a_bias_between_positions_far_past_the_cache(dt, d, hq, n, far):
    """Rows whose positions begin far past the committed keys: the bias goes by the distance between them, however
    large the positions are (the usual tolerance of these caches)."""
    ctx = [200, 37]
    pos = np.concatenate([c + far + np.arange(n) // 2 for c in ctx])
    make(64, ctx, [n, n], hq, 2, d, dt, ScoreMod(slopes=T.slopes(hq)), positions=torch.from_numpy(pos.astype(np.int32)).cuda())


@pytest.mark.parametrize("dt,d,n", [("bf16", 128, 2), ("e4m3", 64, 1), ("bf16", 128, 17), ("f32", 32, 1)])
def test_more_sequences_than_threads(dt, d, n):
    """Batches past the 256 and 384 sequences that a CTA's threads take at once."""
    count = 900
    ctx = [(13 * b) % 50 for b in range(count)]
    nq = [1 + b % n for b in range(count)]
    make(65, ctx, nq, 4, 1, d, dt, ScoreMod(softcap=20.0, window=33))


FIRST_CALL_IN_A_CAPTURE = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
from speculative_decoding_verify_paged_gb300 import HeadTransform, ScoreMod, _lib as L, step as S, workloads as W
case = W.custom(66, batch=2, ctx_lens=[40, 90], n_q=[{n}, {n}], num_q_heads=8, num_kv_heads=2, head_dim={d}, block_size=16, vocab=16, dtype={dt!r}, use_bank=False)
kv, d = S.device_kv(case.state, "cuda"), S.DeviceStep.from_host(case.step, "cuda")
inv = torch.full(({d} // 2,), 0.1, device="cuda")
d.transform, d.mod = HeadTransform(inv_freq=inv), ScoreMod(softcap=20.0, window=30)
buf = S.StepBuffers.make(kv, d, 90 + {n})
table, free, top = kv.block_table.clone(), kv.free_list.clone(), kv.free_top.clone()
buf.attn_out.zero_()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    S.append(kv, d, buf)
    S.attention(kv, d, buf, 90 + {n})
g.replay()
torch.cuda.synchronize()
assert int(buf.status.item()) == 0
first = buf.attn_out.clone()
kv.block_table.copy_(table), kv.free_list.copy_(free), kv.free_top.copy_(top)
S.append(kv, d, buf)
S.attention(kv, d, buf, 90 + {n})
torch.cuda.synchronize()
assert int(buf.status.item()) == 0 and torch.equal(first, buf.attn_out) and bool((first != 0).any())
"""


@pytest.mark.parametrize("dt,d,n", [("bf16", 128, 3), ("bf16", 128, 40), ("e4m3", 64, 3), ("f32", 64, 3)])
def test_the_first_call_of_a_process_may_be_captured(dt, d, n):
    """Nothing has run yet when the transforming append and the attention are captured; the graph gives the bits of the
    calls."""
    here = os.path.dirname(os.path.abspath(__file__))
    code = FIRST_CALL_IN_A_CAPTURE.format(root=os.path.dirname(here), tests=here, dt=dt, d=d, n=n)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("hq,n", [(2, 1), (8, 1), (8, 3)])  # the CUDA-core kernels' three layouts of rows
def test_small_products_next_to_large_ones(hq, n):
    """fp32 caches: a score is a sum of sums of 32 products, so products that are each less than half a step of the whole
    are not lost one by one. Key 0 has 224 products of 2^-5 next to one of 2^20 (a step there is 2^-3), the others none:
    their scores differ by 7 scale. What is left is the rounding of the scores themselves, in base 2 of 378000, to half of 2^-5:
    two of them move a weight p by 2 * 2^-6 ln 2 p (1 - p) <= 0.0055."""
    kv, step, buf, msl = make(67, [1], [n], hq, 1, 256, "f32", ScoreMod())
    blk, scale = int(kv.block_table[0, 0]), 0.25
    kv.k_pool.zero_(), kv.v_pool.zero_(), step.q.fill_(1.0)
    kv.k_pool[blk, 0, :1 + n, 0] = 2.0 ** 20
    kv.k_pool[blk, 0, 0, 32:] = 2.0 ** -5
    kv.v_pool[blk, 0, 0] = 1.0
    step.scale = scale
    out = T.f64(again(kv, step, buf, msl))
    e = np.exp(7 * scale)
    for i in range(n):
        assert np.all(np.abs(out[i] - e / (e + i + 1)) <= 0.0055)


@pytest.mark.parametrize("dt,d,hq", [("e4m3", 128, 8), ("e4m3", 64, 48), ("bf16", 128, 8), ("bf16", 128, 64), ("f32", 64, 8)])
def test_nan_among_committed_and_new_keys_of_long_sequences(dt, d, hq):
    """A NaN in the middle of the committed keys reaches every row, one in a new key the rows from it on; over many splits."""
    n = 5
    kv, step, buf, msl = make(68, [9000, 40], [n, n], hq, 2, d, dt, ScoreMod(softcap=20.0))
    want = buf.attn_out.clone()
    nan = 0x7F if dt == "e4m3" else float("nan")
    for t, first in ((9002, 2), (4321, 0)):
        put(kv, 0, t, nan)
        want[first:n, :, 0] = want[first:n, :, d // 2 + 1] = float("nan")
        out = again(kv, step, buf, msl)
        assert torch.equal(torch.isnan(out), torch.isnan(want))
        assert torch.equal(out[~torch.isnan(want)], want[~torch.isnan(want)])


def test_no_memory_for_the_workspace():
    """The workspace that a call takes for itself fails as any tensor does, and the call is none the worse for it."""
    kv, step, buf, _ = make(69, [300], [40], 8, 2, 128, "bf16", ScoreMod())
    clean = buf.attn_out.clone()
    out = torch.zeros_like(clean)
    call = lambda: L.spec_verify_attn_scored(kv, step.q, out, step.cu_q, max_q=40, max_seq_len=1 << 20, scale=step.scale, mod=ScoreMod(), status=buf.status)  # noqa: E731
    need = L.spec_verify_attn_scored_workspace_bytes(kv, 8, 40, 40, 1 << 20)
    assert need > 20 << 20  # not from the allocator's small blocks
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda.set_per_process_memory_fraction(1e-6)
    try:
        with pytest.raises(torch.OutOfMemoryError):
            call()
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert not out.any()
    call()
    torch.cuda.synchronize()
    assert status_of(buf) == 0 and torch.isfinite(out.float()).all() and out.any()
