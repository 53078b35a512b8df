"""Head norms and rotation (qk_norm_rope), and the append that applies them (kv_append_rope),
against the plain 64-bit form.

Tolerances. The arithmetic is fp32. A normalised value y = x r (w + offset) is off by a few
roundings of 2^-24 each and by the error of the mean of squares (8 + 5 roundings at most, halved by
the root): under 16 * 2^-24 |y| with the rsqrt's own error. A rotated value a cos t - b sin t adds
three roundings and the error of cos and sin: the fraction of a turn is rounded to fp32 (2^-24 of
an angle of at most pi: 2^-22.3) and the function itself is within 2^-23. Altogether under
2^-20 * (|a| + |b|). The output's own rounding adds half a step: 2^-8 (bf16) or 2^-24 (fp32)
relative."""
import numpy as np
import pytest
import torch

import oracle
from speculative_decoding_verify_paged_gb300 import HeadTransform, SVError
from speculative_decoding_verify_paged_gb300 import _lib as L
from speculative_decoding_verify_paged_gb300 import step as S
from speculative_decoding_verify_paged_gb300 import workloads as W

import _plain64 as P
from _helpers import assert_kv_equal, status_of, upload

pytestmark = pytest.mark.gpu

STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def assert_rounded(got, want, size, dtype):
    """|got - want| within the fp32 arithmetic's error (of values of magnitude `size`) and one rounding to dtype."""
    err = np.abs(f64(got) - want)
    assert np.all(err <= 2.0 ** -20 * size + STEP[dtype] * (np.abs(want) + 2.0 ** -20 * size) + 1e-38), float(err.max())


def pair_size(y, rot, interleaved):
    """|a| + |b| of every value's pair."""
    s = np.abs(y).copy()
    half = rot // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        both = np.abs(y[:, :, a]) + np.abs(y[:, :, b])
        s[:, :, a] = s[:, :, b] = both
    return s


def make(n, hq, hkv, d, dtype, rot, *, norm=True, offset=0.0, interleaved=False, seed=0, far=5000):
    g = torch.Generator().manual_seed(seed)
    wide = (torch.randn(n, hq + 2 * hkv, d, generator=g) * 2).to(dtype).cuda()
    inv = (10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / max(rot // 2, 1))).float().cuda()
    weight = lambda: (1.0 - offset + 0.3 * torch.randn(d, generator=g)).to(dtype).cuda() if norm else None  # noqa: E731
    t = HeadTransform(inv_freq=inv if rot else None, q_weight=weight(), k_weight=weight(), eps=1e-6, weight_offset=offset,
                      interleaved=interleaved)
    pos = torch.randint(0, far, (n,), generator=g, dtype=torch.int32).cuda()
    return wide[:, :hq], wide[:, hq:hq + hkv], wide[:, hq + hkv:], t, pos


def want_of(x, weight, pos, t):
    inv = np.zeros(0, np.float32) if t.inv_freq is None else t.inv_freq.cpu().numpy()
    kw = dict(eps=t.eps, offset=t.weight_offset, interleaved=t.interleaved)
    w = None if weight is None else f64(weight)
    flat = P.transform(f64(x), w, np.zeros(x.shape[0]), inv[:0], **kw)
    size = pair_size(flat, 2 * len(inv), t.interleaved)
    return P.transform(f64(x), w, pos, inv, **kw), size


CASES = {
    # name: n, hq, hkv, d, rot, keyword arguments
    "one-token": (1, 32, 8, 128, 128, {}),
    "one-head": (3, 1, 1, 128, 128, {}),
    "wide": (37, 64, 8, 128, 128, {"offset": 1.0}),
    "partial": (5, 8, 2, 128, 32, {}),
    "interleaved": (5, 8, 2, 64, 64, {"interleaved": True}),
    "interleaved-partial": (5, 8, 2, 64, 20, {"interleaved": True}),
    "d8": (9, 4, 2, 8, 8, {}),  # partners through shared memory: half the rotation is not a multiple of 8
    "d40-rot24": (9, 3, 1, 40, 24, {}),
    "d40-rot22": (9, 3, 1, 40, 22, {}),
    "d80": (9, 5, 5, 80, 80, {}),
    "d256": (7, 4, 2, 256, 256, {}),
    "d256-many": (3, 40, 8, 256, 128, {}),
    "no-norm": (6, 8, 2, 128, 128, {"norm": False}),
    "no-rotation": (6, 8, 2, 128, 0, {}),
    "far": (64, 2, 1, 128, 128, {"far": 1 << 30}),
}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name", list(CASES))
def test_rows(name, dtype):
    n, hq, hkv, d, rot, kw = CASES[name]
    q, k, _, t, pos = make(n, hq, hkv, d, dtype, rot, **kw)
    qo, ko = torch.full(q.shape, 7.0, dtype=dtype, device="cuda"), torch.full(k.shape, 7.0, dtype=dtype, device="cuda")
    L.qk_norm_rope(t, q, k, pos, qo, ko)
    for x, w, o in ((q, t.q_weight, qo), (k, t.k_weight, ko)):
        want, size = want_of(x, w, pos.cpu().numpy(), t)
        assert_rounded(o, want, size, dtype)


def test_in_place_and_strided_outputs():
    """q_out = q, and outputs that are parts of wider rows: the rest of those rows stays as it was."""
    q, k, _, t, pos = make(11, 6, 2, 64, torch.bfloat16, 64)
    qo, ko = torch.empty(q.shape, dtype=q.dtype, device="cuda"), torch.empty(k.shape, dtype=k.dtype, device="cuda")
    L.qk_norm_rope(t, q, k, pos, qo, ko)
    wide = torch.full((11, 12, 64), 3.0, dtype=q.dtype, device="cuda")
    L.qk_norm_rope(t, q, k, pos, wide[:, 1:7], wide[:, 8:10])
    assert torch.equal(wide[:, 1:7], qo) and torch.equal(wide[:, 8:10], ko)
    assert (wide[:, [0, 7, 10, 11]] == 3.0).all()
    qi, ki = q.clone(), k.clone()
    L.qk_norm_rope(t, qi, ki, pos, qi, ki)
    assert torch.equal(qi, qo) and torch.equal(ki, ko)


def test_queries_or_keys_alone_and_no_rows():
    q, k, _, t, pos = make(4, 6, 2, 64, torch.float32, 64)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    q1, k1 = torch.empty_like(q), torch.empty_like(k)
    L.qk_norm_rope(t, q, k, pos, qo, ko)
    L.qk_norm_rope(t, q, None, pos, q1, None)
    L.qk_norm_rope(t, None, k, pos, None, k1)
    assert torch.equal(q1, qo) and torch.equal(k1, ko)
    L.qk_norm_rope(t, q[:0], k[:0], pos[:0], q1[:0], k1[:0])


def test_nonfinite_values_stay_in_their_head():
    q, k, _, t, pos = make(3, 4, 2, 128, torch.bfloat16, 64)
    qo, ko, q1, k1 = (torch.empty(x.shape, dtype=x.dtype, device="cuda") for x in (q, k, q, k))
    L.qk_norm_rope(t, q, k, pos, qo, ko)
    q[1, 2, 5] = float("nan")
    k[0, 1, 100] = float("inf")
    L.qk_norm_rope(t, q, k, pos, q1, k1)
    assert torch.isnan(q1[1, 2]).any()
    q1[1, 2] = qo[1, 2]
    k1[0, 1] = ko[0, 1]
    assert torch.equal(q1, qo) and torch.equal(k1, ko)


def test_other_stream_and_graph():
    q, k, _, t, pos = make(16, 8, 2, 128, torch.bfloat16, 128)
    qo, ko, q1, k1 = (torch.empty(x.shape, dtype=x.dtype, device="cuda") for x in (q, k, q, k))
    L.qk_norm_rope(t, q, k, pos, qo, ko)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        L.qk_norm_rope(t, q, k, pos, q1, k1)
    q1.zero_(), k1.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(q1, qo) and torch.equal(k1, ko)
    q1.zero_(), k1.zero_()
    torch.cuda.synchronize()
    L.qk_norm_rope(t, q, k, pos, q1, k1, stream=side)
    side.synchronize()
    assert torch.equal(q1, qo) and torch.equal(k1, ko)


# ---------------------------------------------------------------------------
# the append
# ---------------------------------------------------------------------------
APPENDS = {
    # name: custom arguments, rot, transform arguments
    "bf16": (dict(ctx_lens=[37, 64, 0, 200], n_q=[5, 1, 7, 16], num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16), 128, {}),
    "f32": (dict(ctx_lens=[15, 16], n_q=[5, 3], num_q_heads=4, num_kv_heads=4, head_dim=64, block_size=16), 32, {"interleaved": True}),
    "e4m3": (dict(ctx_lens=[100, 17, 260], n_q=[4, 6, 2], num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16), 128, {"offset": 1.0}),
    "e4m3-d64-no-norm": (dict(ctx_lens=[7], n_q=[64], num_q_heads=2, num_kv_heads=1, head_dim=64, block_size=8), 64, {"norm": False}),
    "bs1-d40": (dict(ctx_lens=[3, 0], n_q=[2, 1], num_q_heads=3, num_kv_heads=1, head_dim=40, block_size=1), 40, {}),
}


@pytest.mark.parametrize("name", list(APPENDS))
def test_append(name):
    """Blocks, lengths and free list as kv_append leaves them; the stored keys are the transformed
    ones, the values the given ones, every other row of the pools untouched; q_out as qk_norm_rope's."""
    kw, rot, tkw = APPENDS[name]
    dt = name.split("-")[0] if name.split("-")[0] in ("f32", "e4m3") else "bf16"
    case = W.custom(41, batch=len(kw["ctx_lens"]), vocab=16, dtype=dt, use_bank=False, **kw)
    kv, d, buf = upload(case)
    rows = torch.float32 if dt == "f32" else torch.bfloat16
    n = d.total_q
    q, k, v, t, _ = make(n, kw["num_q_heads"], kw["num_kv_heads"], kw["head_dim"], rows, rot, **tkw)
    d.q, d.new_k, d.new_v, d.transform = q, k, v, t
    buf.q_rot = torch.empty(q.shape, dtype=rows, device="cuda")
    kp0, vp0 = kv.k_pool.clone(), kv.v_pool.clone()
    S.append(kv, d, buf)
    torch.cuda.synchronize()
    assert status_of(buf) == 0
    okv = oracle.OracleKV(case.state)
    assert okv.append(case.step) is None
    assert_kv_equal(kv, okv, pools=False)
    pos = np.concatenate([c + np.arange(m) for c, m in zip(case.state.seq_lens, case.step.n_q)])
    want_q, size_q = want_of(q, t.q_weight, pos, t)
    assert_rounded(buf.q_rot, want_q, size_q, rows)
    want_k, size_k = want_of(k, t.k_weight, pos, t)
    r = 0
    bs = kw["block_size"]
    for b, (c, m) in enumerate(zip(case.state.seq_lens, case.step.n_q)):
        for j in range(int(m)):
            blk, slot = okv.bt[b][(c + j) // bs], (c + j) % bs
            got = kv.k_pool[blk, :, slot]
            if dt == "e4m3":
                # the nearest code to y / scale, up to the fp32 error of y: half a step of a code (2^-4
                # of normal values, 2^-10 of subnormal ones) and that error
                x = f64(got.view(torch.float8_e4m3fn))
                y = want_k[r] / kv.k_scale
                assert np.all(np.abs(x - np.clip(y, -448, 448)) <= 2.0 ** -20 * size_k[r] / kv.k_scale + np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10))
                plain = (v[r].float() / kv.v_scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                assert torch.equal(kv.v_pool[blk, :, slot], plain)
            else:
                assert_rounded(got[None], want_k[r:r + 1], size_k[r:r + 1], rows)
                assert torch.equal(kv.v_pool[blk, :, slot], v[r])
            kp0[blk, :, slot], vp0[blk, :, slot] = got, kv.v_pool[blk, :, slot]
            r += 1
    assert torch.equal(kp0.view(torch.uint8), kv.k_pool.view(torch.uint8))
    assert torch.equal(vp0.view(torch.uint8), kv.v_pool.view(torch.uint8))


def test_identity_transform_is_kv_append():
    """Without a norm and a rotation the pools hold kv_append's bits (bf16 and E4M3, copy-on-write pools among them)."""
    for dt in ("bf16", "e4m3"):
        case = W.custom(42, batch=3, ctx_lens=[20, 33, 5], n_q=[3, 14, 1], num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16,
                        vocab=16, dtype=dt, use_bank=False)
        a, d, buf = upload(case)
        b, _, buf2 = upload(case)
        for kv in (a, b):
            # sequence 2 shares its partly filled block with sequence 0's slot in the counts: it takes a private copy
            kv.ref_count = torch.zeros(case.state.num_blocks, dtype=torch.int32, device="cuda")
            held = kv.block_table[kv.block_table >= 0].long()
            kv.ref_count[held] = 1
            kv.ref_count[int(kv.block_table[2, 0])] = 2
        S.append(a, d, buf)
        d.transform = HeadTransform()
        buf2.q_rot = torch.empty_like(d.q)
        S.append(b, d, buf2)
        torch.cuda.synchronize()
        assert status_of(buf) == 0 and status_of(buf2) == 0
        for x, y in ((a.k_pool, b.k_pool), (a.v_pool, b.v_pool), (a.block_table, b.block_table), (a.free_list, b.free_list),
                     (a.free_top, b.free_top), (a.ref_count, b.ref_count), (d.q, buf2.q_rot)):
            assert torch.equal(x, y)


def test_append_in_place_without_queries_and_with_positions():
    case = W.custom(43, batch=2, ctx_lens=[9, 40], n_q=[4, 3], num_q_heads=4, num_kv_heads=2, head_dim=64, block_size=16, vocab=16, use_bank=False)
    q, k, v, t, _ = make(7, 4, 2, 64, torch.bfloat16, 64)
    pos = torch.tensor([9, 10, 10, 11, 40, 41, 41], dtype=torch.int32, device="cuda")
    qo, ko = torch.empty(q.shape, dtype=q.dtype, device="cuda"), torch.empty(k.shape, dtype=k.dtype, device="cuda")
    L.qk_norm_rope(t, q, k, pos, qo, ko)
    ref, d, buf = upload(case)
    d.new_k, d.new_v = ko, v.contiguous()
    S.append(ref, d, buf)
    for with_q in (False, True):
        kv, _, buf = upload(case)
        qi = q.clone()
        L.kv_append_rope(kv, t, k, v, d.cu_q, buf.status, q=qi if with_q else None, q_out=qi if with_q else None, positions=pos)
        assert torch.equal(kv.k_pool, ref.k_pool) and torch.equal(kv.v_pool, ref.v_pool)
        assert torch.equal(qi, qo if with_q else q)


def test_failed_append_changes_nothing():
    """Out of blocks, an error already held, and rows past cu_q[batch]."""
    case = W.custom(44, batch=2, ctx_lens=[16, 32], n_q=[3, 2], num_q_heads=4, num_kv_heads=2, head_dim=64, block_size=16, vocab=16, use_bank=False)
    q, k, v, t, _ = make(5, 4, 2, 64, torch.bfloat16, 64)
    for held, code in ((0, 4), (7, 7)):
        kv, d, buf = upload(case)
        qo = torch.full(q.shape, 5.0, dtype=q.dtype, device="cuda")
        if code == 4:
            kv.free_top.zero_()
        buf.status.fill_(held)
        before = [x.clone() for x in (kv.k_pool, kv.v_pool, kv.block_table, kv.free_list, kv.free_top)]
        L.kv_append_rope(kv, t, k, v, d.cu_q, buf.status, q=q, q_out=qo)
        torch.cuda.synchronize()
        assert status_of(buf) == code and (qo == 5.0).all()
        for x, y in zip(before, (kv.k_pool, kv.v_pool, kv.block_table, kv.free_list, kv.free_top)):
            assert torch.equal(x, y)
    kv, d, buf = upload(case)
    more = torch.cat([k, k[:2]]), torch.cat([v, v[:2]]), torch.cat([q, q[:2]])
    qo = torch.full(more[2].shape, 5.0, dtype=q.dtype, device="cuda")
    L.kv_append_rope(kv, t, more[0], more[1], d.cu_q, buf.status, q=more[2], q_out=qo)
    torch.cuda.synchronize()
    assert status_of(buf) == 0 and (qo[5:] == 5.0).all() and not (qo[:5] == 5.0).all()


def test_bindings_refuse_what_does_not_fit():
    q, k, v, t, pos = make(4, 6, 2, 64, torch.bfloat16, 64)
    qo, ko = torch.empty(q.shape, dtype=q.dtype, device="cuda"), torch.empty(k.shape, dtype=k.dtype, device="cuda")
    with pytest.raises(ValueError):
        L.qk_norm_rope(t, q, k, pos[:3], qo, ko)
    with pytest.raises(ValueError):
        L.qk_norm_rope(t, q, k, pos, qo.float(), ko)
    with pytest.raises(ValueError):
        L.qk_norm_rope(t, q.transpose(0, 1), None, pos, qo.transpose(0, 1), None)
    with pytest.raises(ValueError):
        L.qk_norm_rope(HeadTransform(q_weight=torch.ones(32, dtype=q.dtype, device="cuda")), q, k, pos, qo, ko)
    with pytest.raises(TypeError):
        L.qk_norm_rope(t, q.cpu(), k, pos, qo, ko)
    with pytest.raises(TypeError):
        L.qk_norm_rope(t, q, k, pos.cpu(), qo, ko)
    with pytest.raises(TypeError):
        L.qk_norm_rope(HeadTransform(), q.half(), None, pos, qo.half(), None)
    with pytest.raises(ValueError):
        L.qk_norm_rope(t, q, k, pos, None, ko)
    with pytest.raises(ValueError):
        L.qk_norm_rope(t, None, None, pos, None, None)
    with pytest.raises(SVError):
        L.qk_norm_rope(t, q, k, None, qo, ko)  # a rotation without positions
    odd = torch.empty(4 * 6 * 64 + 8, dtype=q.dtype, device="cuda")[1:1 + 4 * 6 * 64].view(4, 6, 64)
    with pytest.raises(SVError):
        L.qk_norm_rope(t, odd, None, pos, qo, None)
