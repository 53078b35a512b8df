"""Attention with capped scores, a distance bias and a window (spec_verify_attn_scored) against
the plain 64-bit form.

Tolerances, as a norm over a query head's output row (|got - want|_2 <= tol |.|_2 with the norm
over sqrt(sum p^2 |v|^2), the size of an average of independent values, and |want| itself):
 * fp32 caches: scores are fp32 dot products of D terms, off by at most about D 2^-24 of the sum of
   |q k| scale; with N(0, 1) values and D <= 256 that is under 2^-16 absolute, and a softmax weight
   moves by as much relatively: 1e-4 (the framework's own bar for fp32 caches) covers it with the sums;
 * bf16 and E4M3 caches: each weight p is rounded to bf16 (2^-8, fp16 2^-11 for E4M3) and the
   output to bf16 (2^-8); fp16 queries add 2^-11 to each product: at most 2^-7 in all, compared
   against the row's norm plus that of the weighted values' root sum of squares."""
import time

import numpy as np
import pytest
import torch

from speculative_decoding_verify_paged_gb300 import HeadTransform, ScoreMod, SVError
from speculative_decoding_verify_paged_gb300 import _lib as L
from speculative_decoding_verify_paged_gb300 import step as S
from speculative_decoding_verify_paged_gb300 import workloads as W

import _plain64 as P
from _helpers import max_seq_len, status_of, upload

pytestmark = pytest.mark.gpu


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def pools(kv):
    """Both pools as float64 [blocks, hkv, bs, d]."""
    if kv.k_pool.dtype == torch.uint8:
        return f64(kv.k_pool.view(torch.float8_e4m3fn)) * kv.k_scale, f64(kv.v_pool.view(torch.float8_e4m3fn)) * kv.v_scale
    return f64(kv.k_pool), f64(kv.v_pool)


def reference(kv, q, cu, mod, positions=None, tree_mask=None, scale=None):
    """The plain form over the cache as it is (after the append), and the norms to compare against."""
    kp, vp = pools(kv)
    table, lens, cu = kv.block_table.cpu().numpy(), kv.seq_lens.cpu().numpy(), cu.cpu().numpy()
    bs, d = kp.shape[2], kp.shape[3]
    q = f64(q)
    slopes = None if mod.slopes is None else mod.slopes.cpu().numpy()
    tm = None if tree_mask is None else tree_mask.cpu().numpy().view(np.uint64)
    pos = None if positions is None else positions.cpu().numpy()
    out = np.zeros(q.shape)
    for b in range(len(lens)):
        lo, hi, c = int(cu[b]), int(cu[b + 1]), int(lens[b])
        t = np.arange(c + hi - lo)
        k, v = (x[table[b, t // bs], :, t % bs] for x in (kp, vp))
        out[lo:hi] = P.attention(k, v, q[lo:hi], c, scale=1.0 / np.sqrt(d) if scale is None else scale, softcap=mod.softcap, slopes=slopes,
                                 window=mod.window, positions=None if pos is None else pos[lo:hi], tree_mask=None if tm is None else tm[lo:hi])
    return out


def assert_near(got, want, f32):
    """Row by row; a floor of 5% of the largest row keeps rows of cancelling values comparable (a sum
    of n independent values of size 1 is at least that, for the lengths here)."""
    got, tol = f64(got), 1e-4 if f32 else 2.0 ** -7
    assert np.isfinite(got).all()
    err = np.linalg.norm(got - want, axis=-1)
    size = np.linalg.norm(want, axis=-1)
    assert np.all(err <= tol * np.maximum(size, 0.05 * size.max())), float((err / np.maximum(size, 0.05 * size.max())).max())


def run(case, mod, *, slack=0, positions=None, tree_mask=None, q_scale=1.0, window_first=None):
    kv, d, buf = upload(case)
    d.mod, d.positions = mod, positions
    if tree_mask is not None:
        d.tree_mask, d.mask_kind = tree_mask, L.SV_MASK_TREE
    d.q = d.q * q_scale
    S.append(kv, d, buf)
    msl = max_seq_len(case.state, case.step, slack)
    buf = S.StepBuffers.make(kv, d, msl)
    buf.attn_out.fill_(float("nan"))
    S.attention(kv, d, buf, msl)
    torch.cuda.synchronize()
    assert status_of(buf) == 0
    want = reference(kv, d.q, d.cu_q, mod, positions, d.tree_mask if d.mask_kind == L.SV_MASK_TREE else None)
    assert_near(buf.attn_out, want, case.state.dtype == "f32")
    return kv, d, buf


def slopes(hq):
    return 2.0 ** (-8.0 * torch.arange(1, hq + 1, dtype=torch.float32, device="cuda") / hq)


MODS = {
    "none": lambda hq: ScoreMod(),
    "cap": lambda hq: ScoreMod(softcap=5.0),
    "bias": lambda hq: ScoreMod(slopes=slopes(hq)),
    "window": lambda hq: ScoreMod(window=100),
    "window1": lambda hq: ScoreMod(window=1),
    "all": lambda hq: ScoreMod(softcap=2.0, slopes=slopes(hq), window=37),
}

SMALL = {
    # name: (seed, ctx, n_q, hq, hkv, d, bs, dtype)
    "bf16-g4-bs16": (11, [700, 65, 1, 300], [6, 6, 6, 6], 32, 8, 128, 16, "bf16"),
    "bf16-one-token": (12, [513, 64, 63, 0], [1, 1, 1, 1], 16, 2, 128, 16, "bf16"),
    "bf16-g8-ragged": (13, [16, 900, 255, 129, 1], [3, 9, 2, 5, 1], 64, 8, 128, 128, "bf16"),
    "bf16-d64": (14, [333, 47], [5, 3], 8, 2, 64, 16, "bf16"),
    "bf16-d64-bs1": (15, [33, 70], [5, 2], 4, 1, 64, 1, "bf16"),
    "bf16-bs8": (27, [75, 8, 140], [6, 1, 3], 8, 2, 128, 8, "bf16"),
    "e4m3-d64-bs8": (28, [300, 9], [2, 1], 8, 2, 64, 8, "e4m3"),
    "bf16-d256": (16, [290, 31], [2, 4], 8, 2, 256, 32, "bf16"),
    "bf16-d96": (17, [130, 31], [2, 4], 6, 2, 96, 8, "bf16"),
    "bf16-wide": (18, [200, 90], [64, 33], 8, 1, 128, 64, "bf16"),
    "bf16-wide-bs256": (50, [700, 255], [40, 64], 8, 2, 128, 256, "bf16"),
    "bf16-one-block": (29, [300, 129], [26, 25], 8, 2, 128, 16, "bf16"),
    "bf16-two-blocks-ragged": (30, [1000, 5, 127, 128], [33, 64, 1, 40], 16, 4, 128, 32, "bf16"),
    "bf16-d256-wide": (19, [150], [30], 8, 1, 256, 16, "bf16"),
    "bf16-mha": (20, [400, 20], [7, 1], 3, 3, 128, 256, "bf16"),
    "e4m3-g4": (21, [700, 3, 129], [6, 6, 6], 32, 8, 128, 16, "e4m3"),
    "e4m3-d64": (22, [333, 47], [5, 3], 4, 4, 64, 16, "e4m3"),
    "e4m3-d256": (23, [150, 47], [5, 1], 8, 2, 256, 64, "e4m3"),
    "e4m3-wide": (24, [170, 0], [40, 64], 8, 2, 128, 16, "e4m3"),
    "f32-d128": (25, [400, 3], [6, 4], 8, 2, 128, 32, "f32"),
    "f32-d32": (26, [100, 3], [1, 4], 2, 1, 32, 4, "f32"),
    "f32-few-rows": (41, [200, 33, 0], [2, 1, 2], 4, 2, 160, 16, "f32"),
    "f32-d256-many-rows": (42, [150, 70], [9, 20], 8, 2, 256, 32, "f32"),
    "e4m3-d96-few-rows": (43, [100, 31], [1, 1], 4, 2, 96, 16, "e4m3"),
    "bf16-d160": (44, [100, 31], [9, 3], 8, 2, 160, 16, "bf16"),
}


@pytest.mark.parametrize("mod", list(MODS))
@pytest.mark.parametrize("name", list(SMALL))
def test_small(name, mod):
    seed, ctx, nq, hq, hkv, d, bs, dt = SMALL[name]
    case = W.custom(seed, batch=len(ctx), ctx_lens=ctx, n_q=nq, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=bs, vocab=16,
                    dtype=dt, use_bank=False)
    run(case, MODS[mod](hq))


@pytest.mark.parametrize("dt", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("mod", ["cap", "all"])
def test_trees(dt, mod):
    """Draft trees: positions are depths, and a row's window goes by position, not by place in the cache."""
    if dt == "f32":
        n, hq = 12, 4
        case = W.custom(31, batch=2, ctx_lens=[90, 0], n_q=[n, n], num_q_heads=hq, num_kv_heads=2, head_dim=64, block_size=16, vocab=16, dtype=dt,
                        use_bank=False)
        rng = np.random.RandomState(1)
        depth, bits = [], []
        for _ in range(2):
            dd, mm = [0], [1]
            for j in range(1, n):
                p = int(rng.randint(0, j))
                dd.append(dd[p] + 1)
                mm.append(mm[p] | (1 << j))
            depth += dd
            bits += mm
        masks = np.array(bits, np.uint64)
    else:
        case = W.tree(batch=2, ctx=333, vocab=256, kv_dtype=dt) if dt == "e4m3" else W.tree(batch=2, ctx=333, vocab=256)
        hq = 32
        masks = case.step.tree_mask
        depth = [bin(int(m)).count("1") - 1 for m in masks]
    pos = np.repeat(case.state.seq_lens, case.step.n_q) + np.array(depth)
    run(case, MODS[mod](hq), positions=torch.from_numpy(pos.astype(np.int32)).cuda(),
        tree_mask=torch.from_numpy(np.ascontiguousarray(masks).view(np.int64)).cuda())


@pytest.mark.parametrize("dt", ["bf16", "e4m3", "f32"])
def test_rows_that_see_nothing(dt):
    """Tree rows without a bit set in a sequence without committed keys, and a window that leaves a
    row only keys that its mask hides: zeros, not NaN."""
    case = W.custom(32, batch=2, ctx_lens=[0, 50], n_q=[3, 4], num_q_heads=8, num_kv_heads=2, head_dim=64, block_size=16, vocab=16, dtype=dt,
                    use_bank=False)
    masks = torch.tensor([1, 0, 5, 1, 0, 7, 0], dtype=torch.int64, device="cuda")
    _, _, buf = run(case, ScoreMod(softcap=3.0, window=1), tree_mask=masks)
    out = f64(buf.attn_out)
    assert (out[[1, 4, 6]] == 0).all() and (np.abs(out[[0, 2, 3, 5]]).max(-1) > 0).all()


def test_large_scores():
    """Scores far past the cap, far apart without one, and negative ones throughout."""
    case = W.custom(33, batch=2, ctx_lens=[300, 80], n_q=[4, 2], num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16, vocab=16, use_bank=False)
    run(case, ScoreMod(softcap=30.0), q_scale=64.0)
    run(case, ScoreMod(softcap=1000.0), q_scale=16.0)
    run(case, ScoreMod(slopes=1000.0 * slopes(8)), q_scale=1.0)
    run(case, ScoreMod(slopes=-0.01 * slopes(8)), q_scale=1.0)  # a bias that grows with distance


@pytest.mark.parametrize("dt,d,hq", [("bf16", 128, 8), ("bf16", 128, 64), ("bf16", 128, 128), ("e4m3", 128, 8), ("f32", 64, 8)])
@pytest.mark.parametrize("cap", [1e-38, 1e-3, 250.0, 1e5])
def test_caps_of_any_size(dt, d, hq, cap):
    """Caps so small that a score is all or nothing, and so large that they change nothing (there the scores
    keep their precision); queries of zeros score zero under any."""
    case = W.custom(45, batch=2, ctx_lens=[200, 33], n_q=[4, 2], num_q_heads=hq, num_kv_heads=2, head_dim=d, block_size=16, vocab=16, dtype=dt,
                    use_bank=False)
    if cap >= 1.0:
        run(case, ScoreMod(softcap=cap))
    run(case, ScoreMod(softcap=cap), q_scale=0.0)


WIDE = {
    # name: (seed, ctx, n_q): eight query heads on two KV heads of 128 values
    "one-block-many": (46, [(37 * i) % 250 for i in range(40)], [17 + i % 16 for i in range(40)]),
    "one-block-long": (47, [9000, 2500, 70], [30, 20, 32]),
    "two-blocks-many": (48, [(37 * i) % 250 for i in range(40)], [1 + (7 * i) % 64 for i in range(40)]),
    "two-blocks-long": (49, [9000, 2500, 70], [64, 50, 33]),
}


@pytest.mark.parametrize("name", list(WIDE))
def test_wide_units(name):
    """Units of more than 64 rows: many short sequences (several a CTA, some of a single tile of keys) and long
    ones (tiles over many CTAs); the same bits every time."""
    seed, ctx, nq = WIDE[name]
    case = W.custom(seed, batch=len(ctx), ctx_lens=ctx, n_q=nq, num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16, vocab=16, use_bank=False)
    run(case, ScoreMod(window=150))
    kv, d, buf = run(case, ScoreMod(softcap=20.0, slopes=slopes(8)))
    first = buf.attn_out.clone()
    for _ in range(20):
        buf.attn_out.zero_()
        S.attention(kv, d, buf, max_seq_len(case.state, case.step))
        torch.cuda.synchronize()
        assert status_of(buf) == 0 and torch.equal(buf.attn_out, first)


def test_long_context_and_loose_bound():
    case = W.custom(34, batch=3, ctx_lens=[9000, 10, 2500], n_q=[6, 6, 1], num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16, vocab=16)
    run(case, ScoreMod(softcap=10.0, slopes=slopes(8)))
    run(case, ScoreMod(window=3000), slack=30000)
    run(case, ScoreMod(softcap=10.0, window=64))


@pytest.mark.parametrize("dt,d,hq", [("bf16", 128, 8), ("bf16", 96, 8), ("f32", 64, 8), ("f32", 160, 2), ("bf16", 128, 32), ("bf16", 128, 48), ("bf16", 64, 32), ("bf16", 256, 8)])
def test_nonfinite_where_nothing_is_seen(dt, d, hq):
    """NaN and infinities in slots past the end of a sequence, before its window, and in draft rows
    that a row does not see: the rows that do not see them are as if they were not there."""
    case = W.custom(35, batch=2, ctx_lens=[200, 37], n_q=[5, 6], num_q_heads=hq, num_kv_heads=2, head_dim=d, block_size=16, vocab=16, dtype=dt,
                    use_bank=False)
    mod = ScoreMod(softcap=20.0, window=50)
    masks = torch.tensor([1, 3, 5, 9, 17] * 1 + [1, 3, 5, 9, 17, 33], dtype=torch.int64, device="cuda")
    kv, dd, buf = run(case, mod, tree_mask=masks)
    clean = buf.attn_out.clone()
    for pool, bad in ((kv.k_pool, float("nan")), (kv.v_pool, float("inf"))):
        for b, (c, n) in enumerate(((200, 5), (37, 6))):
            t = np.arange(c + n, (c + n + 15) // 16 * 16)
            gone = np.concatenate([t, np.arange(0, max(0, c - 49))])
            for x in gone:
                pool[int(kv.block_table[b, x // 16]), :, x % 16] = bad
        # draft row 4 of sequence 0 (bit 4: only row 4 sees it)
        pool[int(kv.block_table[0, 204 // 16]), :, 204 % 16] = bad
    S.attention(kv, dd, buf, max_seq_len(case.state, case.step))
    torch.cuda.synchronize()
    keep = [0, 1, 2, 3, 5, 6, 7, 8, 9, 10]
    assert torch.equal(buf.attn_out[keep], clean[keep])
    assert not torch.isfinite(buf.attn_out[4].float()).any()


def test_rows_behind_the_last_sequence_stay():
    case = W.custom(36, batch=2, ctx_lens=[100, 40], n_q=[3, 2], num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16, vocab=16, use_bank=False)
    kv, d, buf = upload(case)
    S.append(kv, d, buf)
    q = torch.cat([d.q, d.q])
    out = torch.full_like(q, 9.0)
    L.spec_verify_attn_scored(kv, q, out, d.cu_q, max_q=3, max_seq_len=103, scale=0.1, mod=ScoreMod(softcap=9.0), status=buf.status)
    torch.cuda.synchronize()
    assert status_of(buf) == 0 and (out[5:] == 9.0).all() and (out[:5] != 9.0).any()


def test_errors_on_the_device():
    case = W.custom(37, batch=2, ctx_lens=[100, 40], n_q=[3, 3], num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16, vocab=16, use_bank=False)
    kv, d, buf = upload(case)
    S.append(kv, d, buf)

    def status_with(**kw):
        buf.status.zero_()
        args = dict(max_q=3, max_seq_len=103, scale=0.1, mod=ScoreMod(), status=buf.status)
        args.update(kw)
        L.spec_verify_attn_scored(kv, d.q, buf.attn_out, d.cu_q, **args)
        torch.cuda.synchronize()
        return status_of(buf)

    assert status_with() == 0
    assert status_with(max_seq_len=50) == 7  # sequence 0 has 103 tokens
    assert status_with(max_q=2) == 7
    early = torch.tensor([99, 101, 102, 40, 41, 42], dtype=torch.int32, device="cuda")
    assert status_with(positions=early) == 7  # before the committed keys' end
    good = kv.block_table[1, 0].clone()
    for bad in (case.state.num_blocks + 5, -1):
        kv.block_table[1, 0] = bad
        assert status_with() == 6
        assert status_with(mod=ScoreMod(window=8)) == 0  # the window leaves that block out
    kv.block_table[1, 0] = good
    assert status_with() == 0
    with pytest.raises(SVError):
        status_with(workspace=torch.empty(1, dtype=torch.uint8, device="cuda"), max_seq_len=103000)


def test_no_sequences_rows_or_context():
    case = W.custom(38, batch=3, ctx_lens=[20, 40, 0], n_q=[3, 3, 1], num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16, vocab=16, use_bank=False)
    kv, d, buf = upload(case)
    S.append(kv, d, buf)
    out = torch.full_like(d.q, 9.0)
    cu = torch.tensor([0, 3, 3, 3], dtype=torch.int32, device="cuda")  # sequences without rows
    L.spec_verify_attn_scored(kv, d.q, out, cu, max_q=3, max_seq_len=43, scale=0.1, mod=ScoreMod(), status=buf.status)
    L.spec_verify_attn_scored(kv, d.q[:0], out[:0], cu * 0, max_q=3, max_seq_len=43, scale=0.1, mod=ScoreMod(), status=buf.status)
    torch.cuda.synchronize()
    assert status_of(buf) == 0 and (out[3:] == 9.0).all()
    L.spec_verify_attn_scored(kv, d.q, buf.attn_out, d.cu_q, max_q=3, max_seq_len=43, scale=0.1, mod=ScoreMod(), status=buf.status)
    torch.cuda.synchronize()
    assert torch.equal(out[:3], buf.attn_out[:3])


@pytest.mark.parametrize("nq", [[6, 1, 4, 2], [32, 1, 20, 2], [64, 3, 40, 1]])
def test_repeatable_on_two_streams_and_in_graphs(nq):
    """The same call twice, two at once on their own streams, and captured: the same bits."""
    case = W.custom(39, batch=4, ctx_lens=[900, 40, 2000, 3], n_q=nq, num_q_heads=32, num_kv_heads=8, head_dim=128, block_size=16, vocab=16,
                    use_bank=False)
    mod = ScoreMod(softcap=20.0, slopes=slopes(32))
    kv, d, buf = run(case, mod)
    first = buf.attn_out.clone()
    outs = [torch.empty_like(first) for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    call = lambda o, st: L.spec_verify_attn_scored(kv, d.q, o, d.cu_q, max_q=nq[0], max_seq_len=2000 + nq[2], scale=d.scale, mod=mod, stream=st)  # noqa: E731
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for o, s in zip(outs, streams):
            call(o, s)
    for s in streams:
        s.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(outs[2], None)
        graphs.append(g)
    for g in graphs:
        outs[2].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[2], first)
    assert torch.equal(outs[0], first) and torch.equal(outs[1], first)


@pytest.mark.parametrize("n", [6, 20, 40])  # rows of a warp-matrix unit, of a wide one, of two blocks
def test_wait_that_runs_out_then_recovers(n):
    """The failure-path hook: nothing is issued, every wait runs out, the call records SV_ERR_TIMEOUT and
    the next one on the stream is right."""
    case = W.custom(51, batch=4, ctx_lens=[700, 65, 1, 300], n_q=[n, n, n, n], num_q_heads=32, num_kv_heads=8, head_dim=128, block_size=16, vocab=16,
                    use_bank=False)
    mod = ScoreMod(softcap=20.0)
    kv, d, buf = run(case, mod)
    first = buf.attn_out.clone()
    L.set_wait_budget_us(2000)
    L.set_stall_for_test("attention")
    try:
        t0 = time.perf_counter()
        S.attention(kv, d, buf, 700 + n)
        torch.cuda.synchronize()
        assert time.perf_counter() - t0 < 1.0
    finally:
        L.set_stall_for_test("none")
        L.set_wait_budget_us(L.DEFAULT_WAIT_BUDGET_US)
    assert status_of(buf) == L.SV_ERR_TIMEOUT
    buf.status.zero_()
    S.attention(kv, d, buf, 700 + n)
    torch.cuda.synchronize()
    assert status_of(buf) == 0 and torch.equal(buf.attn_out, first)


@pytest.mark.parametrize("dt", ["bf16", "e4m3"])
def test_whole_steps(dt):
    """Three verify steps of a model with head norms, rotary positions, capped scores and a window:
    the cache holds the transformed keys and attention over it is the plain form's, with what earlier
    steps accepted among the committed keys."""
    case = W.custom(40, batch=3, ctx_lens=[60, 5, 130], n_q=[4, 6, 1], num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16, vocab=64, dtype=dt,
                    use_bank=False)
    kv, d, _ = upload(case)
    g = torch.Generator().manual_seed(1)
    inv = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).float().cuda()
    weight = (1 + 0.2 * torch.randn(128, generator=g)).to(torch.bfloat16).cuda()
    d.transform = HeadTransform(inv_freq=inv, q_weight=weight, k_weight=weight)
    d.mod = ScoreMod(softcap=15.0, window=70)
    kept = []
    for it in range(3):
        buf = S.StepBuffers.make(kv, d, 160)
        lens = kv.seq_lens.cpu().numpy().copy()
        d.new_k, d.new_v, d.q = ((torch.randn(x.shape, generator=g) * 2).to(x.dtype).cuda() for x in (d.new_k, d.new_v, d.q))
        S.append(kv, d, buf)
        S.attention(kv, d, buf, 160)
        torch.cuda.synchronize()
        assert status_of(buf) == 0
        pos = np.concatenate([c + np.arange(m) for c, m in zip(lens, case.step.n_q)])
        want_q = P.transform(f64(d.q), f64(weight), pos, inv.cpu().numpy(), eps=1e-6, offset=0.0, interleaved=False)
        assert np.all(np.abs(f64(buf.q_rot) - want_q) <= 2.0 ** -8 * np.abs(want_q) + 2.0 ** -17)
        want_k = P.transform(f64(d.new_k), f64(weight), pos, inv.cpu().numpy(), eps=1e-6, offset=0.0, interleaved=False)
        kept.append((pos, want_k, lens))
        kp, _ = pools(kv)
        table = kv.block_table.cpu().numpy()
        owner = np.repeat(np.arange(3), case.step.n_q)
        step = 2.0 ** -4 if dt == "e4m3" else 2.0 ** -8
        got = kp[table[owner, pos // 16], :, pos % 16]
        assert np.all(np.abs(got - want_k) <= step * np.abs(want_k) + (kv.k_scale * 2.0 ** -10 if dt == "e4m3" else 0) + 2.0 ** -17)
        assert_near(buf.attn_out, reference(kv, buf.q_rot, d.cu_q, d.mod), False)
        S.sample(d, buf)
        S.rollback(kv, d, buf)
        torch.cuda.synchronize()
        assert status_of(buf) == 0
        assert (kv.seq_lens.cpu().numpy() == lens + buf.accept.cpu().numpy() + 1).all()
