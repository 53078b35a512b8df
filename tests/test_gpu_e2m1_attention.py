"""Attention over a 4-bit cache against the plain 64-bit form.

Tolerance: 2^-7 of a query head's row, as over E4M3 pools (test_gpu_scored.py): codes and block scales are operands of
the products exactly, queries are fp16 with a power of two of their own (2^-39 of the row's largest value at most), each
weight is rounded to fp16 (2^-11 of itself, 2^-25 where that is more) and the output to bf16 (2^-8)."""
import os
import subprocess
import sys
import time
from types import SimpleNamespace

import numpy as np
import pytest
import torch

from speculative_decoding_verify_paged_gb300 import ScoreMod
from speculative_decoding_verify_paged_gb300 import _lib as L
from speculative_decoding_verify_paged_gb300 import step as S
from speculative_decoding_verify_paged_gb300 import workloads as W

import _e2m1 as E
import test_gpu_scored as T
from _helpers import max_seq_len, status_of

pytestmark = pytest.mark.gpu


def reference(kv, d, mod, scale=None):
    k, v = E.pools(kv)
    wide = SimpleNamespace(k_pool=torch.from_numpy(k), v_pool=torch.from_numpy(v), block_table=kv.block_table, seq_lens=kv.seq_lens)
    return T.reference(wide, d.q, d.cu_q, mod, d.positions, d.tree_mask if d.mask_kind == L.SV_MASK_TREE else None, scale)


def make(seed, ctx, nq, hq, hkv, d, bs, mod, *, positions=None, tree_mask=None, slack=0, q_scale=1.0, **kw):
    case = W.custom(seed, batch=len(ctx), ctx_lens=ctx, n_q=[max(1, n) for n in nq], num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=bs,
                    vocab=16, dtype="bf16", use_bank=False, **kw)
    kv, step = E.device_kv(case.state), S.DeviceStep.from_host(case.step)
    if 0 in nq:  # sequences without rows
        some = torch.from_numpy(np.repeat(np.array(nq) > 0, case.step.n_q)).cuda()
        step.q, step.new_k, step.new_v = step.q[some], step.new_k[some], step.new_v[some]
        step.cu_q = torch.tensor(np.concatenate([[0], np.cumsum(nq)]), dtype=torch.int32, device="cuda")
    step.mod, step.positions = mod, positions
    if tree_mask is not None:
        step.tree_mask, step.mask_kind = tree_mask, L.SV_MASK_TREE
    step.q = (step.q * q_scale).to(step.q.dtype)
    msl = max_seq_len(case.state, case.step, slack)
    buf = S.StepBuffers.make(kv, step, msl)
    S.append(kv, step, buf)
    buf.attn_out.fill_(float("nan"))
    return kv, step, buf, msl


def attend(kv, step, buf, msl):
    S.attention(kv, step, buf, msl)
    torch.cuda.synchronize()
    assert status_of(buf) == 0
    return buf.attn_out.clone()


def check(kv, step, buf, msl):
    out = attend(kv, step, buf, msl)
    T.assert_near(out, reference(kv, step, step.mod or ScoreMod()), False)
    return out


SMALL = {
    # name: (seed, ctx, n_q, hq, hkv, d, bs)
    "g4-bs16": (11, [700, 65, 1, 300], [6, 6, 6, 6], 32, 8, 128, 16),
    "one-token": (12, [513, 64, 63, 0], [1, 1, 1, 1], 16, 2, 128, 16),
    "two-tokens-g8": (32, [513, 64, 63, 0], [2, 1, 2, 2], 16, 2, 128, 32),
    "g8-ragged": (13, [16, 900, 255, 129, 1], [3, 9, 2, 5, 1], 64, 8, 128, 128),
    "d64": (14, [333, 47], [5, 3], 8, 2, 64, 16),
    "d64-one-token": (33, [333, 47, 2000], [1, 1, 1], 8, 2, 64, 64),
    "d64-g4x6": (34, [333, 47, 2000], [6, 6, 6], 8, 2, 64, 16),
    "d64-many-rows": (35, [333, 47], [33, 64], 4, 2, 64, 16),
    "d64-bs1": (15, [33, 70], [5, 2], 4, 1, 64, 1),
    "d64-bs4": (36, [33, 70], [5, 2], 4, 1, 64, 4),
    "bs8": (27, [75, 8, 140], [6, 1, 3], 8, 2, 128, 8),
    "d64-bs8": (28, [300, 9], [2, 1], 8, 2, 64, 8),
    "d256": (16, [290, 31], [2, 4], 8, 2, 256, 32),
    "d256-bs8": (37, [290, 31], [1, 3], 2, 2, 256, 8),
    "d96": (17, [130, 31], [2, 4], 6, 2, 96, 8),
    "d32": (38, [130, 31, 5], [2, 4, 1], 6, 2, 32, 4),
    "d160": (44, [100, 31], [9, 3], 8, 2, 160, 16),
    "rows-27": (39, [200, 90, 1000], [9, 7, 9], 6, 2, 128, 16),
    "rows-28": (82, [200, 90, 1000], [7, 1, 6], 8, 2, 128, 16),
    "rows-32-bs8": (83, [200, 0, 333], [4, 4, 2], 16, 2, 128, 8),
    "rows-40": (40, [600, 90, 17], [5, 5, 5], 16, 2, 128, 16),
    "wide": (18, [200, 90], [64, 33], 8, 1, 128, 64),
    "wide-bs256": (50, [700, 255], [40, 64], 8, 2, 128, 256),
    "one-block": (29, [300, 129], [26, 25], 8, 2, 128, 16),
    "two-blocks-ragged": (30, [1000, 5, 127, 128], [33, 64, 1, 40], 16, 4, 128, 32),
    "d256-many-rows": (19, [150], [30], 8, 1, 256, 16),
    "mha": (20, [400, 20], [7, 1], 3, 3, 128, 256),
    "no-rows": (45, [400, 20, 70], [0, 3, 0], 4, 2, 128, 16),
    "one-block-no-rows": (77, [400, 20, 70, 300], [0, 20, 0, 1], 8, 2, 128, 16),
    "two-blocks-no-rows": (78, [400, 20, 70, 300], [0, 33, 0, 50], 8, 2, 128, 16),
    "one-block-bs8": (79, [75, 8, 140], [20, 1, 13], 8, 2, 128, 8),
    "two-blocks-bs8": (80, [75, 0, 140], [40, 1, 33], 8, 2, 128, 8),
}


@pytest.mark.parametrize("mod", list(T.MODS))
@pytest.mark.parametrize("name", list(SMALL))
def test_small(name, mod):
    seed, ctx, nq, hq, hkv, d, bs = SMALL[name]
    check(*make(seed, ctx, nq, hq, hkv, d, bs, T.MODS[mod](hq)))


def tree(rng, n, count):
    depth, bits = [], []
    for _ in range(count):
        dd, mm = [0], [1]
        for j in range(1, n):
            p = int(rng.randint(max(0, j - 6) // 2, j))
            dd.append(dd[p] + 1)
            mm.append(mm[p] | (1 << j))
        depth += dd
        bits += mm
    return np.array(depth), torch.from_numpy(np.array(bits, np.uint64).view(np.int64)).cuda()


@pytest.mark.parametrize("d,hq,n", [(64, 4, 12), (128, 8, 12), (128, 4, 31), (128, 8, 61), (128, 2, 64), (256, 4, 20), (96, 4, 12)])
@pytest.mark.parametrize("mod", ["none", "cap", "all"])
def test_trees(d, hq, n, mod):
    ctx = [300, 0, 63]
    depth, bits = tree(np.random.RandomState(n), n, 3)
    where = torch.from_numpy(np.repeat(ctx, n) + depth).int().cuda()
    check(*make(41, ctx, [n] * 3, hq, 2, d, 16, T.MODS[mod](hq), positions=where, tree_mask=bits))


@pytest.mark.parametrize("d,hq,n", [(64, 4, 5), (128, 4, 1), (128, 8, 6), (128, 16, 5), (128, 8, 8), (128, 8, 20), (128, 8, 40), (256, 4, 3), (96, 4, 5)])
def test_long_contexts(d, hq, n):
    """Many CTAs share a unit; the bound of the lengths is far above them."""
    check(*make(42, [5000, 37, 2900], [n, max(1, n - 2), n], hq, 2, d, 16, None, slack=3000))
    check(*make(43, [5000], [n], hq, 2, d, 64, ScoreMod(window=1500)))


@pytest.mark.parametrize("d,hq,n", [(128, 4, 1), (128, 8, 6), (128, 8, 40), (64, 4, 5)])
def test_many_sequences(d, hq, n):
    rng = np.random.RandomState(0)
    ctx = rng.randint(0, 90, 700).tolist()
    check(*make(44, ctx, rng.randint(1, n + 1, 700).tolist(), hq, 2, d, 16, None))


@pytest.mark.parametrize("d,hq,n", [(64, 4, 5), (128, 4, 1), (128, 8, 6), (128, 8, 8), (128, 8, 20), (128, 8, 40), (256, 4, 3), (96, 4, 5)])
def test_plain_call_is_the_scored_one(d, hq, n):
    """spec_verify_attn and its form without a workspace of the caller's: the bits of the scored call with nothing modified."""
    kv, step, buf, msl = make(46, [500, 37, 290], [n, 1, n], hq, 2, d, 16, ScoreMod())
    want = attend(kv, step, buf, msl)
    step.mod = None
    got = attend(kv, step, S.StepBuffers.make(kv, step, msl), msl)
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    L.spec_verify_attn_no_alloc(kv, step.q, out, step.cu_q, max_q=step.max_q, max_seq_len=msl, scale=step.scale, status=buf.status)
    assert torch.equal(out, want)


@pytest.mark.parametrize("d,hq,n", [(64, 4, 5), (128, 4, 1), (128, 8, 6), (128, 8, 8), (128, 8, 20), (128, 8, 40), (256, 4, 3)])
def test_queries_of_any_size(d, hq, n):
    """Queries far outside fp16's range, rows of very different sizes, zero rows: nothing is lost or refused."""
    for q_scale in (1e-30, 1e30):
        kv, step, buf, msl = make(47, [200, 37], [n, 1], hq, 2, d, 16, ScoreMod(), q_scale=q_scale)
        step.scale /= q_scale
        T.assert_near(attend(kv, step, buf, msl), reference(kv, step, ScoreMod(), step.scale), False)
    kv, step, buf, msl = make(48, [200, 37], [n, 1], hq, 2, d, 16, None)
    step.q[:, 0] = 0.0
    step.q[:, 1, : d // 2] *= 2.0 ** -30
    step.q[-1, 2] *= 1e-3
    check(kv, step, buf, msl)


def gaps(kv, step):
    """The least distance between a row's two largest scores, over the sum of the sizes of the largest's products."""
    keys, _ = E.pools(kv)
    table, lens, cu, q = kv.block_table.cpu().numpy(), kv.seq_lens.tolist(), step.cu_q.tolist(), T.f64(step.q)
    least = np.inf
    for b, c in enumerate(lens):
        for i in range(cu[b + 1] - cu[b]):
            t = np.arange(c + i + 1)
            k = keys[table[b, t // 16], :, t % 16]
            for h in range(q.shape[1]):
                kh = k[:, h // (q.shape[1] // k.shape[1])]
                s = kh @ q[cu[b] + i, h]
                first, second = np.argsort(s)[-1:-3:-1]
                size = max(np.abs(kh[x] * q[cu[b] + i, h]).sum() for x in (first, second))
                least = min(least, (s[first] - s[second]) / (2 * size))
    return least


@pytest.mark.parametrize("d,hq,n", [(64, 4, 5), (128, 4, 1), (128, 8, 6), (128, 8, 8), (128, 8, 20), (128, 8, 40), (256, 4, 3)])
def test_scores_of_any_size(d, hq, n):
    """Scores of up to 2^34 in base 2, where fp32's steps are past 16: the weights stay within fp16, and a row's largest score
    takes it all. (A sum of 256 products in fp32 is off by 256 2^-24 = 2^-16 of the sum of their sizes at most; the rows here
    have their two largest scores further apart, which is looked at.)"""
    for up in (2.0 ** 22, 2.0 ** 26, 2.0 ** 30):
        kv, step, buf, msl = make(76, [200, 37], [n, 1], hq, 2, d, 16, ScoreMod())
        assert gaps(kv, step) > 2.0 ** -16
        step.scale *= up
        want = reference(kv, step, ScoreMod(), step.scale)
        T.assert_near(attend(kv, step, buf, msl), want, False)


def put(kv, b, t, group=0, code=0x7F, pool="v"):
    """A NaN scale for 16 values of key t of sequence b, every head."""
    getattr(kv, pool + "_block_scales")[int(kv.block_table[b, t // 16]), :, t % 16, group] = code


KINDS = [(64, 4), (64, 64), (128, 2), (128, 8), (128, 12), (128, 16), (128, 20), (128, 24), (128, 64), (256, 8), (256, 32), (96, 8)]


@pytest.mark.parametrize("d,hq", KINDS)
def test_a_seen_nan_reaches_its_rows_and_no_others(d, hq):
    window = 50
    masks = torch.tensor([1, 3, 5, 9, 17, 1, 3, 5, 9, 17, 33], dtype=torch.int64, device="cuda")
    kv, step, buf, msl = make(61, [200, 37], [5, 6], hq, 2, d, 16, ScoreMod(softcap=20.0, window=window), tree_mask=masks)
    want = check(kv, step, buf, msl)
    last = d // 16 - 1
    for b, t, row, code in ((0, 200 + 4, 4, 0x7F), (0, 200 - window + 1, 0, 0xFF), (1, 37 + 2, 7, 0x7F)):
        put(kv, b, t, 0, code)
        put(kv, b, t, last, code)
        want[row, :, :16] = want[row, :, -16:] = float("nan")
    out = attend(kv, step, buf, msl)
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    keep = ~torch.isnan(want)
    assert torch.equal(out[keep], want[keep])


@pytest.mark.parametrize("d,hq", KINDS)
def test_a_nan_key_reaches_its_rows_and_no_others(d, hq):
    kv, step, buf, msl = make(62, [200, 37], [5, 6], hq, 2, d, 16, ScoreMod())
    want = check(kv, step, buf, msl)
    put(kv, 0, 202, d // 16 - 1, pool="k")  # the third of the new keys: rows 2 to 4 see it
    want[2:5] = float("nan")
    out = attend(kv, step, buf, msl)
    assert torch.equal(torch.isnan(out), torch.isnan(want)) and torch.equal(out[~torch.isnan(want)], want[~torch.isnan(want)])


@pytest.mark.parametrize("d,hq", KINDS)
def test_a_seen_nan_counts_whatever_its_weight(d, hq):
    kv, step, buf, msl = make(63, [200, 37], [5, 6], hq, 2, d, 16, ScoreMod(slopes=torch.full((hq,), 1000.0, device="cuda")))
    clean = check(kv, step, buf, msl)
    put(kv, 0, 202)
    out = attend(kv, step, buf, msl)
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[2:5, :, :16] = True
    assert torch.isnan(out[hit]).all() and torch.equal(out[~hit], clean[~hit])


@pytest.mark.parametrize("d,hq", KINDS)
def test_slots_of_nobody_reach_nobody(d, hq):
    """NaN scales in every block that no sequence holds, in the slots behind the rows, and before a window."""
    kv, step, buf, msl = make(64, [200, 37, 0], [5, 6, 1], hq, 2, d, 16, ScoreMod(window=40))
    want = check(kv, step, buf, msl)
    table, lens, cu = kv.block_table.cpu().numpy(), kv.seq_lens.tolist(), step.cu_q.tolist()
    keep = torch.zeros(kv.k_pool.shape[0], 16, dtype=torch.bool)
    for b, c in enumerate(lens):
        t = np.arange(max(0, c - 39), c + cu[b + 1] - cu[b])
        keep[table[b, t // 16], t % 16] = True
    for f in (kv.k_block_scales, kv.v_block_scales):
        f.masked_fill_(~keep.cuda()[:, None, :, None], 0xFF)
    assert torch.equal(attend(kv, step, buf, msl), want)


@pytest.mark.parametrize("d,hq,n", [(64, 4, 5), (128, 4, 1), (128, 8, 6), (128, 8, 8), (128, 8, 20), (128, 8, 40), (256, 4, 3), (96, 4, 5)])
def test_rows_that_see_nothing(d, hq, n):
    """Tree masks without a bit and no committed key: zeros."""
    masks = torch.zeros(2 * n, dtype=torch.int64, device="cuda")
    kv, step, buf, msl = make(65, [0, 50], [n, n], hq, 2, d, 16, ScoreMod(), tree_mask=masks)
    out = check(kv, step, buf, msl)
    assert (out[:n] == 0).all() and (out[n:] != 0).any()


@pytest.mark.parametrize("d,hq,n", [(64, 4, 5), (128, 4, 1), (128, 8, 6), (128, 8, 8), (128, 8, 20), (128, 8, 40), (256, 4, 3), (96, 4, 5)])
def test_errors(d, hq, n):
    """Bad lengths and ids are recorded; the sequences beside them are right."""
    for spoil, code in (("length", 7), ("rows", 7), ("id", 6), ("hole", 6)):
        kv, step, buf, msl = make(66, [300, 290, 310], [n] * 3, hq, 2, d, 16, ScoreMod())
        want = attend(kv, step, buf, msl)
        ref = reference(kv, step, ScoreMod())
        buf.attn_out.fill_(3.0)
        if spoil == "length":
            kv.seq_lens[1] = msl + 100
        elif spoil == "rows":
            kv.seq_lens[1] = -1
        else:
            kv.block_table[1, 3] = kv.k_pool.shape[0] + 5 if spoil == "id" else -1
        S.attention(kv, step, buf, msl)
        torch.cuda.synchronize()
        assert status_of(buf) == code, spoil
        for rows in (slice(0, n), slice(2 * n, 3 * n)):  # (the work is cut elsewhere without a sequence's keys)
            T.assert_near(buf.attn_out[rows], ref[rows], False)
            assert code == 7 or torch.equal(buf.attn_out[rows], want[rows])
        if code == 7:
            assert (buf.attn_out[n:2 * n] == 3.0).all()


@pytest.mark.parametrize("d,hq,n", [(64, 4, 5), (128, 8, 6), (128, 8, 8), (128, 8, 20), (128, 8, 40), (96, 4, 5)])
def test_blocks_past_32_bits(d, hq, n):
    """Blocks that lie more than 2^31 (heads of 64 and 96 values) or 2^32 bytes (of 128) behind their pool's start."""
    mod = ScoreMod(softcap=20.0)
    kv, step, buf, msl = make(81, [300, 37], [n, n], hq, 2, d, 16, mod)
    want = attend(kv, step, buf, msl)
    k, v = torch.empty_like(step.new_k), torch.empty_like(step.new_v)
    L.kv_gather(kv, k, v, step.cu_q, buf.status)
    few, blocks = kv.k_pool.shape[0], 2200000
    base = E.device_kv(W.custom(81, batch=2, ctx_lens=[300, 37], n_q=[n, n], num_q_heads=hq, num_kv_heads=2, head_dim=d, block_size=16, vocab=16,
                                dtype="bf16", use_bank=False).state)
    far = {}
    for f in ("k_pool", "v_pool", "k_block_scales", "v_block_scales"):
        small = getattr(base, f)
        far[f] = torch.full((blocks, *small.shape[1:]), 0xFF, dtype=torch.uint8, device="cuda")
        far[f][blocks - few:] = small
    assert far["k_pool"].numel() > 2 ** (32 if d == 128 else 31)
    for f, x in far.items():
        setattr(base, f, x)
    base.block_table = torch.where(base.block_table >= 0, base.block_table + (blocks - few), base.block_table)
    free = torch.full((blocks,), -1, dtype=torch.int32, device="cuda")
    free[:few] = torch.where(base.free_list >= 0, base.free_list + (blocks - few), base.free_list)
    base.free_list = free
    far_buf = S.StepBuffers.make(base, step, msl)
    S.append(base, step, far_buf)
    assert torch.equal(attend(base, step, far_buf, msl), want)
    far_k, far_v = torch.empty_like(k), torch.empty_like(v)
    L.kv_gather(base, far_k, far_v, step.cu_q, far_buf.status)
    assert status_of(far_buf) == 0 and torch.equal(far_k, k) and torch.equal(far_v, v)


def test_rows_behind_the_last_sequence_stay():
    kv, step, buf, msl = make(67, [300, 29], [6, 6], 8, 2, 128, 16, ScoreMod())
    want = attend(kv, step, buf, msl)
    cu = torch.tensor([0, 6, 10], dtype=torch.int32, device="cuda")
    out = torch.full_like(want, 3.0)
    L.spec_verify_attn_scored(kv, step.q, out, cu, max_q=6, max_seq_len=msl, scale=step.scale, mod=ScoreMod(), status=buf.status)
    T.assert_near(out[:10], reference(kv, step, ScoreMod())[:10], False)
    assert (out[10:] == 3.0).all()


@pytest.mark.parametrize("d,hq,n", [(64, 4, 5), (128, 4, 1), (128, 8, 6), (128, 8, 8), (128, 8, 20), (128, 8, 40), (256, 4, 3)])
def test_calls_repeat_and_replay(d, hq, n):
    """The same bits from call to call, from a captured graph (append, attention and gather together) replayed, and from
    two streams at once with workspaces of their own."""
    ctx = (900, 37, 290, 3000)
    kv, step, buf, msl = make(68, list(ctx), [n] * 4, hq, 2, d, 16, ScoreMod(softcap=30.0))
    want = attend(kv, step, buf, msl)
    for _ in range(5):
        assert torch.equal(attend(kv, step, buf, msl), want)
    k, v = torch.empty_like(step.new_k), torch.empty_like(step.new_v)
    L.kv_gather(kv, k, v, step.cu_q, buf.status)
    first = (k.clone(), v.clone())
    # the step's blocks, back on the stack in the order in which they went: each replay takes them again
    top, table, free = int(kv.free_top), kv.block_table.clone(), kv.free_list.clone()
    ids = [int(table[b, j]) for b, c in enumerate(ctx) for j in range(-(-c // 16), -(-(c + n) // 16))]
    free[top:top + len(ids)] = torch.tensor(ids[::-1], dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.kv_append(kv, step.new_k, step.new_v, step.cu_q, buf.status)
        S.attention(kv, step, buf, msl)
        L.kv_gather(kv, k, v, step.cu_q, buf.status)
    for _ in range(3):
        for x in (k, v, buf.attn_out):
            x.zero_()
        kv.free_top.fill_(top + len(ids))
        kv.free_list.copy_(free)
        graph.replay()
        torch.cuda.synchronize()
        assert status_of(buf) == 0 and torch.equal(kv.block_table, table)
        assert torch.equal(buf.attn_out, want) and torch.equal(k, first[0]) and torch.equal(v, first[1])
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(want) for _ in streams]
    for _ in range(10):
        for s, o in zip(streams, outs):
            s.wait_stream(torch.cuda.current_stream())
            L.spec_verify_attn_scored(kv, step.q, o, step.cu_q, max_q=step.max_q, max_seq_len=msl, scale=step.scale, mod=step.mod, status=buf.status,
                                      stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("d,hq,n", [(64, 4, 5), (128, 8, 6), (128, 8, 8), (128, 8, 20), (128, 8, 40), (256, 4, 3), (96, 4, 5)])
@pytest.mark.parametrize("cap", [150.0, 1000.0, 3.4028234e38])
def test_large_caps(d, hq, n, cap):
    """Either side of what the two-instruction tanh takes, and a cap whose product with log2(e) is past fp32's range."""
    check(*make(73, [200, 33], [n, 2], hq, 2, d, 16, ScoreMod(softcap=cap)))


@pytest.mark.parametrize("d,hq,n", [(64, 4, 5), (128, 8, 6), (128, 8, 8), (128, 8, 20), (128, 8, 40), (256, 4, 3), (96, 4, 5)])
@pytest.mark.parametrize("far", [1000, 2000000000])
def test_a_bias_between_positions_far_past_the_cache(d, hq, n, far):
    ctx = [200, 37]
    pos = np.concatenate([c + far + np.arange(n) // 2 for c in ctx])
    check(*make(74, ctx, [n, n], hq, 2, d, 16, ScoreMod(slopes=T.slopes(hq)), positions=torch.from_numpy(pos.astype(np.int32)).cuda()))


FIRST_CALLS_IN_A_CAPTURE = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
from speculative_decoding_verify_paged_gb300 import ScoreMod, _lib as L, step as S, workloads as W
import _e2m1 as E
case = W.custom(75, batch=2, ctx_lens=[40, 90], n_q=[{n}, {n}], num_q_heads=8, num_kv_heads=2, head_dim={d}, block_size=16, vocab=16, dtype="bf16", use_bank=False)
kv, d = E.device_kv(case.state), S.DeviceStep.from_host(case.step, "cuda")
d.mod = ScoreMod(softcap=20.0, window=30)
buf = S.StepBuffers.make(kv, d, 90 + {n})
k, v = torch.empty_like(d.new_k), torch.empty_like(d.new_v)
table, free, top = kv.block_table.clone(), kv.free_list.clone(), kv.free_top.clone()
torch.cuda.synchronize()
def run():
    S.append(kv, d, buf)
    S.attention(kv, d, buf, 90 + {n})
    L.kv_gather(kv, k, v, d.cu_q, buf.status)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    run()
g.replay()
torch.cuda.synchronize()
assert int(buf.status.item()) == 0
first = [x.clone() for x in (buf.attn_out, k, v)]
kv.block_table.copy_(table), kv.free_list.copy_(free), kv.free_top.copy_(top)
run()
torch.cuda.synchronize()
assert int(buf.status.item()) == 0 and all(torch.equal(x, y) and bool((x != 0).any()) for x, y in zip(first, (buf.attn_out, k, v)))
"""


@pytest.mark.parametrize("d,n", [(64, 3), (128, 3), (128, 20), (128, 40), (96, 3)])
def test_the_first_calls_of_a_process_may_be_captured(d, n):
    here = os.path.dirname(os.path.abspath(__file__))
    code = FIRST_CALLS_IN_A_CAPTURE.format(root=os.path.dirname(here), tests=here, d=d, n=n)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("hq,n", [(8, 20), (8, 40)])
def test_a_wait_runs_out_then_the_call_is_right(hq, n):
    """The kernels for many rows wait for their converters. The test hook lets these wait for what nothing ends: the call
    records a timeout within its budget, and the next one on the stream is right (up to 128 rows a KV head, and more)."""
    kv, step, buf, msl = make(72, [900, 37, 290], [n, 1, n], hq, 2, 128, 16, ScoreMod())
    want = attend(kv, step, buf, msl)
    L.set_wait_budget_us(2000)
    L.set_stall_for_test("attention")
    try:
        t0 = time.perf_counter()
        S.attention(kv, step, buf, msl)
        torch.cuda.synchronize()
        seconds = time.perf_counter() - t0
    finally:
        L.set_stall_for_test("none")
        L.set_wait_budget_us(L.DEFAULT_WAIT_BUDGET_US)
    assert status_of(buf) == L.SV_ERR_TIMEOUT and seconds < 1.0
    buf.status.zero_()
    buf.attn_out.fill_(float("nan"))
    assert torch.equal(attend(kv, step, buf, msl), want)


def test_whole_steps():
    """Ten verify steps of a ragged batch: append, attention, sampling, rollback, with the cache's rows held against the
    plain format all the way."""
    rng = np.random.RandomState(5)
    ctx = [37, 0, 130, 700, 64]
    first = W.custom(70, batch=5, ctx_lens=ctx, n_q=[1] * 5, num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16, vocab=64, dtype="bf16",
                     use_bank=False, growth_tokens=200, pool_factor=2.0)
    kv = E.device_kv(first.state)
    rows = [[], []]  # what each sequence's places hold, by the plain format
    k0, v0 = E.pools(kv)
    table = kv.block_table.cpu().numpy()
    for pool, out in ((k0, rows[0]), (v0, rows[1])):
        for b, c in enumerate(ctx):
            t = np.arange(c)
            out.append(pool[table[b, t // 16], :, t % 16])
    for it in range(10):
        nq = rng.randint(1, 9, 5).tolist()
        case = W.custom(71 + it, batch=5, ctx_lens=ctx, n_q=nq, num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16, vocab=64, dtype="bf16",
                        use_bank=False)
        step = S.DeviceStep.from_host(case.step)
        step.mod = ScoreMod(softcap=20.0) if it % 2 else None
        lens = kv.seq_lens.tolist()
        msl = max(c + n for c, n in zip(lens, nq))
        buf = S.StepBuffers.make(kv, step, msl)
        S.append(kv, step, buf)
        S.attention(kv, step, buf, msl)
        T.assert_near(buf.attn_out, reference(kv, step, step.mod or ScoreMod()), False)
        S.sample(step, buf)
        S.rollback(kv, step, buf)
        torch.cuda.synchronize()
        assert status_of(buf) == 0
        cu, acc = step.cu_q.tolist(), buf.accept.tolist()
        for which, (new, scale) in enumerate(((step.new_k, kv.k_scale), (step.new_v, kv.v_scale))):
            stored = E.values(*E.quantise(new.float().cpu().numpy(), scale), scale)
            for b in range(5):
                rows[which][b] = np.concatenate([rows[which][b], stored[cu[b]:cu[b] + acc[b] + 1]])
    lens = kv.seq_lens.tolist()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    out = [torch.empty((int(cu[-1]), 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    L.kv_gather(kv, *out, cu, first=torch.zeros(5, dtype=torch.int32, device="cuda"))
    for got, want in zip(out, rows):
        want = np.concatenate(want)
        assert np.all(np.abs(got.double().cpu().numpy() - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -22))
