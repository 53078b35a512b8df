"""4-bit pools, the gather and rotary axes on the host: argument checks without a GPU, and the plain format's
own pins (torch's E4M3 conversion, hand-worked codes)."""
import ctypes

import numpy as np
import pytest
import torch

import _e2m1 as E
from speculative_decoding_verify_paged_gb300 import HeadTransform, PagedKV, rotary_axes
from speculative_decoding_verify_paged_gb300 import _lib as L
from speculative_decoding_verify_paged_gb300 import build as B

P = ctypes.c_void_p
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 10


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


def cache(**kw):
    s = L.sv_paged_kv()
    s.k_pool = s.v_pool = s.block_table = s.seq_lens = s.free_list = s.free_top = s.k_block_scales = s.v_block_scales = 256  # never read
    s.num_blocks, s.block_size, s.max_blocks_per_seq, s.num_kv_heads, s.head_dim, s.batch = 16, 16, 4, 2, 128, 2
    s.dtype, s.k_scale, s.v_scale = L.SV_DTYPE_E2M1, 1.0, 1.0
    for k, v in kw.items():
        setattr(s, k, v)
    return s


BAD = [dict(k_block_scales=None), dict(v_block_scales=None), dict(k_block_scales=264), dict(v_block_scales=260), dict(head_dim=48),
       dict(head_dim=16), dict(k_scale=0.0), dict(v_scale=-1.0), dict(k_scale=float("nan")), dict(v_scale=float("inf")),
       dict(k_scale=2.0 ** -65), dict(v_scale=2.0 ** 64.5), dict(k_pool=264), dict(block_size=12)]


@pytest.mark.parametrize("bad", BAD, ids=str)
def test_every_call_refuses_a_bad_cache(lib, bad):
    kv = ctypes.byref(cache(**bad))
    t, m = L.sv_head_transform(), L.sv_score_mod()
    assert lib.sv_kv_append(kv, P(256), P(256), P(256), 4, P(256), None) == INVALID
    assert lib.sv_kv_append_rope(kv, ctypes.byref(t), P(256), 256, P(256), 256, None, 0, None, 0, 0, P(256), 4, None, P(256), None) == INVALID
    assert lib.sv_kv_gather(kv, P(256), P(256), P(256), 4, None, None, None) == INVALID
    assert lib.sv_spec_verify_attn(kv, P(256), P(256), P(256), 4, 4, 4, 64, 0.1, 0, None, None, 0, None, None) == INVALID
    assert lib.sv_spec_verify_attn_scored(kv, P(256), P(256), P(256), 4, 4, 4, 64, 0.1, ctypes.byref(m), None, 0, None, None, 0, None, None) == INVALID
    assert lib.sv_kv_rollback(kv, P(256), P(256), None, 4, P(256), None) == INVALID
    assert lib.sv_kv_release(kv, P(256), 1, P(256), None) == INVALID


def test_attention_refusals(lib):
    kv = cache()
    m = L.sv_score_mod()

    def plain(kv=kv, hq=4, rows=4, max_q=4, max_len=64, scale=0.1, mask=0, q=256, cu=256):
        return lib.sv_spec_verify_attn(ctypes.byref(kv), P(q), P(256), P(cu), hq, rows, max_q, max_len, scale, mask, None, None, 0, None, None)
    assert plain(rows=0) == 0
    assert plain(kv=cache(batch=0)) == 0
    for bad in (dict(hq=3), dict(hq=0), dict(rows=-1), dict(max_q=65), dict(max_len=0), dict(scale=float("nan")), dict(mask=2), dict(mask=1),
                dict(q=None), dict(q=264), dict(cu=None)):
        assert plain(**bad) == INVALID, bad
    assert plain(max_len=(1 << 30) + 1) == UNSUPPORTED
    assert plain(kv=cache(batch=65536)) == UNSUPPORTED
    big = cache(max_blocks_per_seq=1000)
    need = lib.sv_spec_verify_attn_workspace_bytes(ctypes.byref(big), 4, 8, 4, 10000)
    assert need == lib.sv_spec_verify_attn_scored_workspace_bytes(ctypes.byref(big), 4, 8, 4, 10000) > 0
    args = (ctypes.byref(big), P(256), P(256), P(256), 4, 8, 4, 10000, 0.1)
    for ws, n in ((None, 0), (256, need - 1), (264, need)):
        assert lib.sv_spec_verify_attn(*args, 0, None, P(ws), n, None, None) == WORKSPACE
        assert lib.sv_spec_verify_attn_scored(*args, ctypes.byref(m), None, 0, None, P(ws), n, None, None) == WORKSPACE
    for bad in ((3, 8, 4, 64), (4, -1, 4, 64), (4, 8, 0, 64), (4, 8, 65, 64), (4, 8, 4, 0), (4, 8, 4, (1 << 30) + 1)):
        assert lib.sv_spec_verify_attn_workspace_bytes(ctypes.byref(big), *bad) == 0


@pytest.mark.parametrize("dtype", [0, 1, 2, 3])
def test_gather_refusals(lib, dtype):
    def call(kv=None, k=256, v=256, cu=256, rows=4):
        return lib.sv_kv_gather(ctypes.byref(cache(dtype=dtype) if kv is None else kv), P(k), P(v), P(cu), rows, None, None, None)
    assert call(rows=0, cu=None) == 0
    assert call(kv=cache(dtype=dtype, batch=0)) == 0
    for bad in (dict(rows=-1), dict(cu=None), dict(k=264), dict(v=260), dict(k=None, v=None)):
        assert call(**bad) == INVALID, bad
    assert lib.sv_kv_gather(None, P(256), P(256), P(256), 4, None, None, None) == INVALID


def test_axes_refusals(lib):
    t = L.sv_head_transform(inv_freq=256, rotary_dim=64)

    def axes(n, values=(0,) * 32):
        a = L.sv_rotary_axes(num_axes=n)
        a.axis[:len(values)] = list(values)
        return a

    def heads(a, rows=4, pos=256):
        return lib.sv_qk_norm_rope_axes(ctypes.byref(t), None if a is None else ctypes.byref(a), P(256), 512, P(256), 512, 4, P(256), 256, P(256), 256, 2,
                                        128, 0, rows, P(pos), None)

    def append(a, batch=0):
        return lib.sv_kv_append_rope_axes(ctypes.byref(cache(batch=batch)), ctypes.byref(t), None if a is None else ctypes.byref(a), P(256), 256, P(256),
                                          256, P(256), 512, P(256), 512, 4, P(256), 4, None, P(256), None)
    assert heads(axes(3, (0, 1, 2) * 10 + (0, 0)), rows=0) == 0
    assert append(axes(8, (7,) * 32)) == 0
    for a in (None, axes(0), axes(-1), axes(9), axes(2, (0, 1, 2)), axes(1, (0,) * 31 + (1,)), axes(8, (8,))):
        assert heads(a, rows=0) == INVALID
        assert append(a) == INVALID
    assert heads(axes(2, (1,) * 40), rows=0) == 0  # entries past the pairs are not looked at
    assert heads(axes(1, (0,) * 32 + (9,)), rows=0) == 0
    assert heads(axes(2), pos=None) == INVALID


def test_rotary_axes():
    assert rotary_axes((2, 1, 1)) == bytes((0, 0, 1, 2))
    assert rotary_axes((3, 2, 2), in_turn=True) == bytes((0, 1, 2, 0, 1, 2, 0))
    assert rotary_axes((6, 2, 1), in_turn=True) == bytes((0, 1, 2, 0, 1, 0, 0, 0, 0))
    assert rotary_axes((4,)) == bytes(4)
    for bad in ((), (1,) * 9, (2, -1)):
        with pytest.raises(ValueError):
            rotary_axes(bad)
    with pytest.raises(ValueError):
        rotary_axes((1, 5), in_turn=True)  # the second's share would run past the end
    assert HeadTransform().axes is None


def test_python_refusals():
    """A cache whose tensors do not fit together, before anything is loaded or launched."""
    z = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    i = torch.zeros(1, dtype=torch.int32)

    def kv(**kw):
        d = dict(k_pool=z(2, 1, 16, 64), v_pool=z(2, 1, 16, 64), block_table=i[None], seq_lens=i, free_list=i, free_top=i, k_block_scales=z(2, 1, 16, 8),
                 v_block_scales=z(2, 1, 16, 8))
        return PagedKV(**{**d, **kw})
    for bad in (dict(v_block_scales=None), dict(k_block_scales=None), dict(k_block_scales=z(2, 1, 16, 4)), dict(v_block_scales=z(1, 1, 16, 8)),
                dict(k_pool=z(2, 1, 16, 72)), dict(v_pool=z(2, 1, 16, 32)), dict(k_block_scales=torch.zeros((2, 1, 16, 8)))):
        with pytest.raises((ValueError, TypeError)):
            kv(**bad).struct()
    with pytest.raises(TypeError):
        kv().struct()  # not on a GPU
    assert kv().is_e2m1


# ---- the plain format ----
def test_plain_scales_are_torchs_e4m3():
    x = np.concatenate([np.random.RandomState(0).uniform(0, 460, 20000), np.exp(np.random.RandomState(1).uniform(-9, 6.1, 20000)), E.e4m3_table(),
                        (E.e4m3_table()[1:] + E.e4m3_table()[:-1]) / 2]).astype(np.float32)
    want = torch.from_numpy(np.minimum(x, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(E.nearest(x.astype(np.float64), E.e4m3_table()), want)


def test_plain_codes_by_hand():
    row = np.array([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.3, -0.2, 5.1, 2.6, -6, 0.0, 1, -4], np.float32)  # scale 1: s = 1
    codes, s = E.quantise(row[None], 1.0)
    assert s.tolist() == [[0x38]]  # 1.0
    assert (codes[0] & 15).tolist() == [7, 2, 4, 6, 9, 7, 15, 2]
    assert (codes[0] >> 4).tolist() == [0, 2, 4, 6, 8, 5, 0, 14]
    np.testing.assert_array_equal(E.values(codes, s, 1.0)[0], [6, 0, 1, 1, 2, 2, 4, 4, -0.5, 0, 6, 3, -6, 0, 1, -4])
    # a group of zeros, one whose scale rounds to zero, one with an infinity, one with a NaN
    rows = np.zeros((4, 16), np.float32)
    rows[1, 3], rows[2, 5], rows[2, 6], rows[3, 0] = 2.0 ** -12, -np.inf, 3.0, np.nan
    codes, s = E.quantise(rows, 1.0)
    assert s[:, 0].tolist() == [0, 0, 0x7E, 0x7F]
    v = E.values(codes, s, 1.0)
    assert not v[0].any() and not v[1].any() and v[2, 5] == -6 * 448 and v[2, 6] == 0 and np.isnan(v[3]).all()


def test_plain_error_is_bounded():
    """Half a step of the codes (a quarter of the smallest magnitudes' distance up to one of six), and what a block scale
    rounded down leaves past six: 1/16 of it."""
    x = np.random.RandomState(3).randn(200, 256).astype(np.float32)
    v = E.values(*E.quantise(x, 0.75), 0.75)
    top = np.abs(x).reshape(200, -1, 16).max(-1).repeat(16, -1)
    assert np.all(np.abs(v - x) <= top * (1 / 6) * (17 / 16))


@pytest.mark.parametrize("d,n,hq,block,tile,lead", [
    (256, 1, 64, 8, 64, 4), (256, 64, 64, 16, 64, 4), (128, 1, 64, 8, 128, 2), (128, 2, 64, 16, 128, 2), (128, 4, 64, 32, 64, 4), (128, 5, 64, 24, 128, 2),
    (128, 64, 64, 24, 128, 2), (64, 1, 64, 8, 128, 2), (64, 64, 64, 32, 128, 2)])
def test_positions_stay_within_32_bits(lib, d, n, hq, block, tile, lead):
    """A unit (`block` rows of a KV head) has a position for each tile of keys and `lead` more; a call whose positions pass 32
    bits goes to the CUDA-core kernels, which need no workspace for this many sequences. (Many rows: the kernel for caps past
    the fast form has the most.)"""
    def workspace(length):
        kv = L.sv_paged_kv(num_blocks=1 << 16, block_size=64, max_blocks_per_seq=1 << 17, num_kv_heads=8, head_dim=d, batch=4096, dtype=L.SV_DTYPE_E2M1)
        return lib.sv_spec_verify_attn_scored_workspace_bytes(ctypes.byref(kv), hq, 1, n, length)
    units = 4096 * 8 * -(-8 * n // block)
    most = (2 ** 31 - 1) // units - lead
    assert most * tile < 1 << 30
    assert workspace(most * tile) > 0 and workspace(most * tile + 1) == 0 and workspace(1 << 30) == 0
