"""The 4-bit cache: rows into it, rows out of it and the bookkeeping that moves them, against the plain format.

Appended rows are determined to the bit (each operation of the format is one rounding in fp32). Gathered values are a code
times fp32(s * scale): against 64 bits two roundings of fp32 (2^-24 each) and the one to bf16 (2^-8 of the value).
Rows that are normalised and rotated on their way in are off by 2^-20 of the pair's size before (test_gpu_heads.py says
why), so a code may be the next one where the value lies that close to a border."""
import numpy as np
import pytest
import torch

import oracle
from speculative_decoding_verify_paged_gb300 import HeadTransform, SVError
from speculative_decoding_verify_paged_gb300 import _lib as L
from speculative_decoding_verify_paged_gb300 import step as S
from speculative_decoding_verify_paged_gb300 import workloads as W

import _e2m1 as E
import _plain64 as P
from _helpers import assert_kv_equal, max_seq_len, status_of

pytestmark = pytest.mark.gpu

FIELDS = ("k_pool", "v_pool", "k_block_scales", "v_block_scales")


def host(kv):
    return {f: getattr(kv, f).cpu().numpy().copy() for f in FIELDS}


def make(seed, ctx, nq, *, hq=4, hkv=2, d=128, bs=16, ref_count=None, **kw):
    case = W.custom(seed, batch=len(ctx), ctx_lens=ctx, n_q=nq, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=bs, vocab=16, dtype="bf16",
                    use_bank=False, **kw)
    kv = E.device_kv(case.state, ref_count=ref_count)
    step = S.DeviceStep.from_host(case.step)
    buf = S.StepBuffers.make(kv, step, max_seq_len(case.state, case.step))
    return case, kv, step, buf


def places(kv, cu):
    """(sequence, block, slot) of every new row."""
    table, lens, cu, bs = kv.block_table.cpu().numpy(), kv.seq_lens.cpu().numpy(), cu.cpu().numpy(), kv.k_pool.shape[2]
    return [(b, table[b, (lens[b] + i) // bs], (lens[b] + i) % bs) for b in range(len(lens)) for i in range(cu[b + 1] - cu[b])]


def assert_stored(kv, before, cu, new_k, new_v):
    """Every new row is stored as the plain format says, and nothing else has changed."""
    want = {f: x.copy() for f, x in before.items()}
    for name, rows in (("k", new_k), ("v", new_v)):
        codes, scales = E.quantise(rows.float().cpu().numpy(), getattr(kv, name + "_scale"))
        for r, (_, blk, slot) in enumerate(places(kv, cu)):
            want[name + "_pool"][blk, :, slot] = codes[r]
            want[name + "_block_scales"][blk, :, slot] = scales[r]
    got = host(kv)
    for f in FIELDS[2:]:
        np.testing.assert_array_equal(got[f], want[f])
    for name in "kv":  # (the codes of 16 NaN are open)
        nan = np.repeat((want[name + "_block_scales"] & 127) == 127, 8, -1)
        np.testing.assert_array_equal(np.where(nan, 0, got[name + "_pool"]), np.where(nan, 0, want[name + "_pool"]))


SHAPES = {
    # name: ctx, n_q, hkv, d, bs
    "one-row": ([37], [1], 1, 128, 16),
    "ragged": ([0, 15, 16, 700], [3, 9, 1, 6], 8, 128, 16),
    "d32-bs1": ([5, 9], [4, 2], 3, 32, 1),
    "d64-bs8": ([300, 7], [5, 1], 2, 64, 8),
    "d96": ([33, 64], [2, 7], 5, 96, 32),
    "d160": ([100], [13], 2, 160, 64),
    "d256-bs256": ([255, 513], [64, 33], 4, 256, 256),
    "many": ([20] * 300, [64] * 300, 1, 64, 128),  # several rows a CTA, rows of several sequences
}


@pytest.mark.parametrize("name", list(SHAPES))
def test_append(name):
    ctx, nq, hkv, d, bs = SHAPES[name]
    case, kv, step, buf = make(3, ctx, nq, hq=hkv, hkv=hkv, d=d, bs=bs)
    before = host(kv)
    S.append(kv, step, buf)
    torch.cuda.synchronize()
    assert status_of(buf) == 0
    okv = oracle.OracleKV(case.state)
    assert okv.append(case.step) is None
    assert_kv_equal(kv, okv, pools=False)
    assert_stored(kv, before, step.cu_q, step.new_k, step.new_v)


@pytest.mark.parametrize("aligned", [True, False])
def test_append_special_values(aligned):
    """Zeros of either sign, subnormals, the largest values, infinities and NaN, borders between codes; rows that start
    on a 16-byte border alone."""
    _, kv, step, buf = make(4, [30, 3], [5, 4], hkv=2, hq=2, d=64)
    n = step.total_q * 2 * 64
    store = torch.empty(2 * n + 64, dtype=torch.bfloat16, device="cuda")
    k, v = (store[o + (0 if aligned else 8):][:n].view(step.total_q, 2, 64) for o in (0, n + 32))
    k.copy_(step.new_k)
    v.copy_(step.new_v)
    k[0, 0, :16] = 0.0
    k[0, 0, 16:32] = -0.0
    k[0, 1, 3] = float("nan")
    k[1, 0, 20] = float("inf")
    k[1, 1, 40] = -float("inf")
    k[2, 0] = 1e-39
    k[2, 1] = torch.finfo(torch.bfloat16).max
    k[3, 0, :16] = torch.tensor([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5, 0]) * 0.75
    v[4, 0, 5] = float("nan")
    v[4, 0, 6] = float("inf")
    v[5] *= 1e30
    v[6] *= 1e-30
    v[7, 0, ::16] = 3000.0
    before = host(kv)
    L.kv_append(kv, k, v, step.cu_q, buf.status)
    torch.cuda.synchronize()
    assert status_of(buf) == 0
    assert_stored(kv, before, step.cu_q, k, v)


@pytest.mark.parametrize("scale", [2.0 ** -64, 1e-6, 1.0, 3.3e4, 2.0 ** 64])
def test_append_pool_scales(scale):
    _, kv, step, buf = make(5, [30], [7], hkv=2, hq=2, d=64)
    kv.k_scale, kv.v_scale = scale, 1.0 / scale
    k, v = (step.new_k * scale).to(torch.bfloat16), (step.new_v / scale).to(torch.bfloat16)
    before = host(kv)
    L.kv_append(kv, k, v, step.cu_q, buf.status)
    torch.cuda.synchronize()
    assert_stored(kv, before, step.cu_q, k, v)


def test_append_refusals_write_nothing():
    """All or nothing: too few blocks, a bad popped id, a length that does not fit, an error in the status word; and rows
    past cu_q[batch]."""
    for spoil in ("blocks", "id", "length", "status"):
        _, kv, step, buf = make(6, [16, 32], [3, 2])
        if spoil == "blocks":
            kv.free_top.fill_(1)
        elif spoil == "id":
            kv.free_list[int(kv.free_top) - 1] = kv.k_pool.shape[0]
        elif spoil == "length":
            kv.seq_lens[1] = kv.block_table.shape[1] * 16 - 1
        else:
            buf.status.fill_(4)
        before = host(kv)
        S.append(kv, step, buf)
        torch.cuda.synchronize()
        assert status_of(buf) != 0
        after = host(kv)
        assert all(np.array_equal(before[f], after[f]) for f in FIELDS)
    _, kv, step, buf = make(6, [16, 32], [3, 2])
    before = host(kv)
    cu = torch.tensor([0, 3, 4], dtype=torch.int32, device="cuda")  # the last of five rows is nobody's
    L.kv_append(kv, step.new_k, step.new_v, cu, buf.status)
    torch.cuda.synchronize()
    assert status_of(buf) == 0
    assert_stored(kv, before, cu, step.new_k[:4], step.new_v[:4])


def transform(d, rot, seed=0, axes=None, interleaved=False, norm=True):
    g = torch.Generator().manual_seed(seed)
    w = lambda: (1 + 0.2 * torch.randn(d, generator=g)).bfloat16().cuda() if norm else None  # noqa: E731
    inv = (10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / max(1, rot // 2))).float().cuda() if rot else None
    return HeadTransform(inv_freq=inv, q_weight=w(), k_weight=w(), axes=axes, interleaved=interleaved)


@pytest.mark.parametrize("d,rot,interleaved,norm", [(128, 128, False, True), (64, 32, True, True), (256, 256, False, True), (96, 40, False, True),
                                                    (32, 32, True, False), (128, 0, False, False)])
def test_rotating_append(d, rot, interleaved, norm):
    ctx, nq, hkv = [30, 3, 0], [5, 40, 1], 3
    _, kv, step, buf = make(7, ctx, nq, hq=6, hkv=hkv, d=d)
    t = transform(d, rot, interleaved=interleaved, norm=norm)
    before = host(kv)
    plain = S.device_kv(W.custom(7, batch=3, ctx_lens=ctx, n_q=nq, num_q_heads=6, num_kv_heads=hkv, head_dim=d, block_size=16, vocab=16, dtype="bf16",
                                 use_bank=False).state)
    q_out, q_plain = torch.empty_like(step.q), torch.empty_like(step.q)
    status = torch.zeros_like(buf.status)
    L.kv_append_rope(kv, t, step.new_k, step.new_v, step.cu_q, buf.status, q=step.q, q_out=q_out)
    L.kv_append_rope(plain, t, step.new_k, step.new_v, step.cu_q, status, q=step.q, q_out=q_plain)
    torch.cuda.synchronize()
    assert status_of(buf) == 0 and torch.equal(q_out, q_plain)
    if rot == 0 and not norm:
        assert_stored(kv, before, step.cu_q, step.new_k, step.new_v)
        return
    where = np.concatenate([np.arange(c, c + n) for c, n in zip(ctx, nq)])
    want = P.transform(step.new_k.double().cpu().numpy(), None if t.k_weight is None else t.k_weight.double().cpu().numpy(), where,
                       np.zeros(0, np.float32) if t.inv_freq is None else t.inv_freq.cpu().numpy(), eps=t.eps, offset=0.0, interleaved=interleaved)
    codes, scales = E.quantise(want.astype(np.float32), kv.k_scale)
    vc, vs = E.quantise(step.new_v.float().cpu().numpy(), kv.v_scale)
    got = host(kv)
    blk, slot = np.array([p[1:] for p in places(kv, step.cu_q)]).T
    np.testing.assert_array_equal(got["v_pool"][blk, :, slot], vc)
    np.testing.assert_array_equal(got["v_block_scales"][blk, :, slot], vs)
    # values next to a border (2^-20 of the pair, some 2^-18 of a step) may take the next code: one in thousands
    stored = E.values(got["k_pool"][blk, :, slot], got["k_block_scales"][blk, :, slot], kv.k_scale)
    plain_values = E.values(codes, scales, kv.k_scale)
    assert np.mean(stored != plain_values) < 1e-3
    top = np.abs(want).reshape(*want.shape[:2], -1, 16).max(-1).repeat(16, -1)
    assert np.all(np.abs(stored - want) <= top / 6 * (17 / 16) + 1e-6 * top)


def test_copy_on_write():
    """Children that share their parents' partly filled blocks write into copies, codes and scales; the parents' rows stay."""
    for rope in (False, True):
        ctx, nq = [37, 5, 64], [2, 3, 1]
        _, kv, step, buf = make(8, ctx + [0, 0, 0], nq + nq, d=96, growth_tokens=256, pool_factor=4.0)
        kv.ref_count = torch.zeros(kv.k_pool.shape[0], dtype=torch.int32, device="cuda")
        kv.ref_count[kv.block_table[kv.block_table >= 0].long()] = 1
        L.kv_fork(kv, torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"), torch.tensor([3, 4, 5], dtype=torch.int32, device="cuda"), buf.status)

        def rows(b, n):
            t = np.arange(n)
            blk = kv.block_table[b].cpu().numpy()[t // 16]
            h = host(kv)
            return [h[f][blk, :, t % 16] for f in FIELDS]
        before = [rows(b, c) for b, c in enumerate(ctx)]
        if rope:
            L.kv_append_rope(kv, HeadTransform(), step.new_k, step.new_v, step.cu_q, buf.status)
        else:
            L.kv_append(kv, step.new_k, step.new_v, step.cu_q, buf.status)
        torch.cuda.synchronize()
        assert status_of(buf) == 0
        table = kv.block_table.cpu().numpy()
        assert table[0, 2] != table[3, 2] and table[1, 0] != table[4, 0] and table[2, 3] == table[5, 3]
        cu = step.cu_q.cpu().numpy()
        for b in range(6):
            c, n = ctx[b % 3], nq[b % 3]
            got = rows(b, c + n)
            for x, (f, old) in enumerate(zip(got, before[b % 3])):
                np.testing.assert_array_equal(f[:c], old)
            for name, at in (("k", 0), ("v", 1)):
                codes, scales = E.quantise(getattr(step, "new_" + name)[cu[b]:cu[b + 1]].float().cpu().numpy(), getattr(kv, name + "_scale"))
                np.testing.assert_array_equal(got[at][c:], codes)
                np.testing.assert_array_equal(got[at + 2][c:], scales)
        assert (kv.ref_count >= 0).all()


@pytest.mark.parametrize("d", [32, 128])
def test_tree_rollback_moves_codes_and_scales(d):
    _, kv, step, buf = make(9, [37, 14], [7, 9], hkv=3, hq=3, d=d)
    S.append(kv, step, buf)
    torch.cuda.synchronize()
    at = places(kv, step.cu_q)
    before = host(kv)
    path = torch.full((2, 9), -1, dtype=torch.int32, device="cuda")
    path[0, :3] = torch.tensor([2, 3, 6])
    path[1, :4] = torch.tensor([1, 4, 5, 8])
    accept = torch.tensor([3, 4], dtype=torch.int32, device="cuda")
    L.kv_rollback(kv, step.cu_q, accept, buf.status, max_q=9, path_nodes=path)
    torch.cuda.synchronize()
    assert status_of(buf) == 0 and kv.seq_lens.tolist() == [41, 19]
    want = {f: x.copy() for f, x in before.items()}
    for b, first in ((0, 0), (1, 7)):
        for j in range(int(accept[b])):
            _, sb, ss = at[first + int(path[b, j])]
            _, db, ds = at[first + 1 + j]
            for f in FIELDS:
                want[f][db, :, ds] = want[f][sb, :, ss]
    after = host(kv)
    for f in FIELDS:
        np.testing.assert_array_equal(after[f], want[f])


# ----------------------------------------------------------------------------
# gather
# ----------------------------------------------------------------------------
def filled(dt, seed, ctx, hkv, d, bs):
    state = W.custom(seed, batch=len(ctx), ctx_lens=ctx, n_q=[1] * len(ctx), num_q_heads=hkv, num_kv_heads=hkv, head_dim=d, block_size=bs, vocab=16,
                     dtype="bf16" if dt == "e2m1" else dt, use_bank=False, growth_tokens=64).state
    kv = E.device_kv(state) if dt == "e2m1" else S.device_kv(state)
    if dt == "e2m1":
        return kv, E.pools(kv)
    if dt == "e4m3":
        return kv, tuple(p.view(torch.float8_e4m3fn).double().cpu().numpy() * 0.125 for p in (kv.k_pool, kv.v_pool))
    return kv, tuple(p.double().cpu().numpy() for p in (kv.k_pool, kv.v_pool))


@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("dt,d", [("bf16", 8), ("bf16", 24), ("bf16", 128), ("f32", 8), ("f32", 96), ("e4m3", 16), ("e4m3", 128), ("e2m1", 32),
                                  ("e2m1", 96), ("e2m1", 256)])
def test_gather(dt, d, aligned):
    ctx, hkv, bs = [300, 0, 17, 64, 1], 3, 16
    kv, pools = filled(dt, 20, ctx, hkv, d, bs)
    first, count = [3, 0, 0, 15, 0], [290, 0, 17, 49, 1]
    rows = sum(count)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(count)]), dtype=torch.int32, device="cuda")
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    skip = 0 if aligned else 16 // torch.empty(0, dtype=dtype).element_size()
    store = torch.full((2, (rows + 2) * hkv * d + 32), 7.0, dtype=dtype, device="cuda")
    k, v = (x[skip:skip + (rows + 2) * hkv * d].view(rows + 2, hkv, d) for x in store)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.kv_gather(kv, k, v, cu, status, first=torch.tensor(first, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert int(status) == 0
    table = kv.block_table.cpu().numpy()
    at = np.concatenate([np.stack([np.full(n, b), f + np.arange(n)]) for b, (f, n) in enumerate(zip(first, count))], 1)
    for got, pool in ((k, pools[0]), (v, pools[1])):
        assert (got[rows:] == 7.0).all()  # rows past cu[batch]
        want = pool[table[at[0], at[1] // bs], :, at[1] % bs]
        got = got[:rows].double().cpu().numpy()
        if dt in ("bf16", "f32", "e4m3"):
            np.testing.assert_array_equal(got, want)
        else:
            assert np.all(np.abs(got - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -22))
    one = torch.full_like(k[:rows], 5.0)  # values alone
    L.kv_gather(kv, None, one, cu, first=torch.tensor(first, dtype=torch.int32, device="cuda"))
    assert torch.equal(one, v[:rows])


@pytest.mark.parametrize("dt", ["bf16", "e2m1"])
def test_gather_errors(dt):
    """A range past the block table, a negative start, a block that is not there: recorded, the other rows written."""
    kv, pools = filled(dt, 21, [40, 40, 40], 2, 64, 16)
    for spoil, code in (("first", 7), ("past", 7), ("id", 6), ("hole", 6)):
        first = torch.tensor([0, 0, 5], dtype=torch.int32, device="cuda")
        table = kv.block_table.clone()
        if spoil == "first":
            first[1] = -1
        elif spoil == "past":
            first[1] = table.shape[1] * 16 - 9
        else:
            kv.block_table[1, 0] = kv.k_pool.shape[0] if spoil == "id" else -1
        cu = torch.tensor([0, 10, 20, 30], dtype=torch.int32, device="cuda")
        out = torch.full((30, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        L.kv_gather(kv, out, None, cu, status, first=first)
        torch.cuda.synchronize()
        assert int(status) == code, spoil
        assert (out[10:20] == 7.0).all() and (out[:10] != 7.0).any() and (out[20:] != 7.0).any()
        kv.block_table.copy_(table)


def test_gather_nan_and_new_rows():
    """Without `first` the rows that an append has just written; a NaN comes back as 16."""
    _, kv, step, buf = make(22, [30, 3], [5, 4], d=64)
    step.new_k[2, 1, 17] = float("nan")
    S.append(kv, step, buf)
    k, v = torch.empty_like(step.new_k), torch.empty_like(step.new_v)
    L.kv_gather(kv, k, v, step.cu_q, buf.status)
    torch.cuda.synchronize()
    assert status_of(buf) == 0
    for got, new, scale in ((k, step.new_k, kv.k_scale), (v, step.new_v, kv.v_scale)):
        want = E.values(*E.quantise(new.float().cpu().numpy(), scale), scale)
        got = got.double().cpu().numpy()
        np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
        assert np.all((np.abs(got - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -22)) | np.isnan(want))
    assert torch.isnan(k[2, 1, 16:32]).all() and int(torch.isnan(k).sum()) == 16


def test_binding_refusals():
    _, kv, step, buf = make(23, [30], [5], d=64)
    out = torch.empty_like(step.new_k)
    for bad in (out[:, :1], out.float(), out[:, :, :32], out.view(5, -1)):
        with pytest.raises((ValueError, TypeError)):
            L.kv_gather(kv, bad, None, step.cu_q)
        with pytest.raises((ValueError, TypeError)):
            L.kv_append(kv, bad, bad, step.cu_q, buf.status)
    with pytest.raises(ValueError):
        L.kv_gather(kv, None, None, step.cu_q)
    with pytest.raises(ValueError):
        L.kv_gather(kv, out, out[:4], step.cu_q)
    with pytest.raises(ValueError):
        L.kv_gather(kv, out, None, step.cu_q[:1])
    with pytest.raises(ValueError):
        L.kv_gather(kv, out, None, step.cu_q, first=step.cu_q)  # one start a sequence
    with pytest.raises(TypeError):
        L.kv_gather(kv, out.cpu(), None, step.cu_q)
    scales = kv.k_block_scales
    for bad in (None, scales[:, :, :, :2].contiguous(), scales.to(torch.int8), scales.transpose(0, 1)):
        kv.k_block_scales = bad
        with pytest.raises((ValueError, TypeError)):
            L.kv_gather(kv, out, None, step.cu_q)
    kv.k_block_scales = scales
    kv.k_scale = 0.0
    with pytest.raises(SVError):
        L.kv_gather(kv, out, None, step.cu_q)


# ----------------------------------------------------------------------------
# rotary positions with several axes
# ----------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d,rot,interleaved,sections,in_turn", [(128, 128, False, (16, 24, 24), False), (128, 128, False, (24, 20, 20), True),
                                                                (64, 32, True, (8, 4, 4), False), (96, 44, False, (22, 0), False),
                                                                (256, 256, True, (16,) * 8, True), (40, 24, False, (12,), False)])
def test_axes(dtype, d, rot, interleaved, sections, in_turn):
    import test_gpu_heads as H
    q, k, _, t, _ = H.make(9, 6, 2, d, dtype, rot, interleaved=interleaved)
    t.axes = L.rotary_axes(sections, in_turn=in_turn)
    g = torch.Generator().manual_seed(1)
    pos = torch.randint(-3, 70000, (len(sections), 9), generator=g, dtype=torch.int32).cuda()
    outs = [torch.empty(x.shape, dtype=dtype, device="cuda") for x in (q, k)]
    L.qk_norm_rope(t, q, k, pos, *outs)
    torch.cuda.synchronize()
    inv, axis = t.inv_freq.cpu().numpy(), np.frombuffer(t.axes, np.uint8)
    for x, w, got in ((q, t.q_weight, outs[0]), (k, t.k_weight, outs[1])):
        x, w = x.double().cpu().numpy(), w.double().cpu().numpy()
        want = flat = P.transform(x, w, np.zeros(9), inv[:0], eps=t.eps, offset=0.0, interleaved=interleaved)
        for a in range(len(sections)):  # an axis's pairs, with the others' frequencies at zero
            only = np.where(axis == a, inv, np.float32(0))
            want = P.transform(want, None, pos[a].cpu().numpy(), only, eps=0.0, offset=0.0, interleaved=interleaved)
        H.assert_rounded(got, want, H.pair_size(flat, rot, interleaved), dtype)


def test_axes_with_equal_positions_change_nothing():
    """One axis, the same positions on all and (append) none at all: the bits of the call without axes."""
    import test_gpu_heads as H
    q, k, v, t, pos = H.make(40, 8, 2, 128, torch.bfloat16, 128)
    want = [torch.empty(x.shape, dtype=x.dtype, device="cuda") for x in (q, k)]
    L.qk_norm_rope(t, q, k, pos, *want)
    for axes, n in ((bytes(64), 1), (L.rotary_axes((16, 24, 24)), 3), (L.rotary_axes((32, 32)), 5)):
        got = [torch.empty_like(x) for x in want]
        t.axes = axes
        L.qk_norm_rope(t, q, k, pos.expand(n, -1).contiguous(), *got)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        with pytest.raises(ValueError):
            L.qk_norm_rope(t, q, k, pos, *got)  # one axis's positions
    for bad in (bytes(63), list(range(64)), "x" * 64):
        t.axes = bad
        with pytest.raises((ValueError, TypeError)):
            L.qk_norm_rope(t, q, k, pos.expand(3, -1).contiguous(), *want)
    t.axes = bytes([0] * 63 + [3])
    with pytest.raises(ValueError):
        L.qk_norm_rope(t, q, k, pos.expand(3, -1).contiguous(), *want)
    stored = []
    for axes in (None, L.rotary_axes((16, 24, 24))):
        case = W.custom(30, batch=2, ctx_lens=[30, 3], n_q=[5, 4], num_q_heads=4, num_kv_heads=2, head_dim=128, block_size=16, vocab=16, dtype="bf16",
                        use_bank=False)
        kv, step = S.device_kv(case.state), S.DeviceStep.from_host(case.step)
        step.transform = HeadTransform(inv_freq=t.inv_freq, k_weight=t.k_weight, axes=axes)
        buf = S.StepBuffers.make(kv, step, 64)
        S.append(kv, step, buf)
        torch.cuda.synchronize()
        assert status_of(buf) == 0
        stored.append((kv.k_pool, kv.v_pool, buf.q_rot))
    assert all(torch.equal(a, b) for a, b in zip(*stored))


@pytest.mark.parametrize("dt", ["bf16", "e4m3", "e2m1"])
def test_appending_with_axes(dt):
    """The stored keys are those of the rows' own transform (bf16), or as near as the pool's codes."""
    case = W.custom(31, batch=2, ctx_lens=[30, 3], n_q=[5, 40], num_q_heads=4, num_kv_heads=2, head_dim=128, block_size=16, vocab=16,
                    dtype="bf16" if dt == "e2m1" else dt, use_bank=False)
    kv = E.device_kv(case.state) if dt == "e2m1" else S.device_kv(case.state)
    step = S.DeviceStep.from_host(case.step)
    step.transform = transform(128, 128, axes=L.rotary_axes((16, 24, 24)))
    step.axis_positions = torch.randint(0, 5000, (3, 45), generator=torch.Generator().manual_seed(2), dtype=torch.int32).cuda()
    buf = S.StepBuffers.make(kv, step, 64)
    S.append(kv, step, buf)
    q, k = torch.empty_like(step.q), torch.empty_like(step.new_k)
    L.qk_norm_rope(step.transform, step.q, step.new_k, step.axis_positions, q, k)
    got = torch.empty_like(k)
    L.kv_gather(kv, got, None, step.cu_q, buf.status)
    torch.cuda.synchronize()
    assert status_of(buf) == 0 and torch.equal(q, buf.q_rot)
    if dt == "bf16":
        assert torch.equal(got, k)
    elif dt == "e4m3":  # half a code's step (2^-4, or 2^-10 of the scale 0.125 below the normal codes) and bf16's rounding of k
        err = (got.float() - k.float()).abs()
        assert (err <= k.float().abs() * (2.0 ** -4 + 2.0 ** -7) + 2.0 ** -13).all()
    else:
        top = k.float().abs().unflatten(-1, (-1, 16)).amax(-1).repeat_interleave(16, -1)
        assert ((got.float() - k.float()).abs() <= top * (17 / 96 + 2.0 ** -7)).all()
    step.positions, step.axis_positions = torch.zeros(45, dtype=torch.int32, device="cuda"), None
    with pytest.raises(ValueError):
        S.append(kv, step, buf)
