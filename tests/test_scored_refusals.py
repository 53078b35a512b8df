"""Host-side argument checks of the head transform, the transforming append and attention with
modified scores: each answers without touching a GPU."""
import ctypes

import pytest

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
    s.k_pool = s.v_pool = s.block_table = s.seq_lens = s.free_list = s.free_top = 256  # never read
    s.num_blocks, s.block_size, s.max_blocks_per_seq, s.num_kv_heads, s.head_dim, s.batch = 16, 16, 4, 2, 128, 2
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def heads(lib, t, rows=4, q=256, hq=4, k=256, hkv=2, d=128, dtype=0, qs=512, ks=256, pos=256):
    return lib.sv_qk_norm_rope(None if t is None else ctypes.byref(t), P(q), qs, P(q), qs, hq, P(k), ks, P(k), ks, hkv, d, dtype, rows, P(pos), None)


def test_heads(lib):
    good = lambda **kw: L.sv_head_transform(**{**dict(inv_freq=256, eps=1e-6, rotary_dim=128), **kw})  # noqa: E731
    assert heads(lib, good(), rows=0) == 0
    assert heads(lib, good(), hq=0, hkv=0) == 0
    assert heads(lib, None) == INVALID
    for bad in (dict(rotary_dim=130), dict(rotary_dim=-2), dict(rotary_dim=3), dict(inv_freq=None), dict(interleaved=2), dict(q_weight=264),
                dict(q_weight=256, eps=-1.0), dict(k_weight=256, eps=float("nan")), dict(q_weight=256, weight_offset=float("inf"))):
        assert heads(lib, good(**bad)) == INVALID, bad
    for bad in (dict(rows=-1), dict(hq=-1), dict(d=12), dict(d=264), dict(d=0), dict(dtype=2), dict(dtype=7), dict(qs=504), dict(qs=516),
                dict(ks=128), dict(q=None), dict(k=264), dict(pos=None), dict(qs=1 << 40)):
        assert heads(lib, good(), **bad) == INVALID, bad


def append(lib, kv, t, rows=4, k=256, ks=256, v=256, q=256, qs=512, hq=4, cu=256, status=256):
    return lib.sv_kv_append_rope(None if kv is None else ctypes.byref(kv), None if t is None else ctypes.byref(t), P(k), ks, P(v), ks, P(q), qs,
                                 P(q), qs, hq, P(cu), rows, None, P(status), None)


def test_append(lib):
    t = L.sv_head_transform(inv_freq=256, rotary_dim=64)
    assert append(lib, cache(batch=0), t) == 0
    assert append(lib, None, t) == INVALID
    assert append(lib, cache(), None) == INVALID
    for bad in (dict(block_size=3), dict(head_dim=12), dict(dtype=9), dict(free_list=None), dict(k_pool=264), dict(dtype=2, k_scale=0.0)):
        assert append(lib, cache(**bad), t) == INVALID, bad
    for bad in (dict(rows=-1), dict(k=None), dict(v=264), dict(q=None), dict(hq=-1), dict(ks=250), dict(cu=None), dict(status=None)):
        assert append(lib, cache(), t, **bad) == INVALID, bad
    assert append(lib, cache(), L.sv_head_transform(inv_freq=256, rotary_dim=130)) == INVALID
    assert append(lib, cache(ref_count=256, batch=5000), t) == UNSUPPORTED


def attend(lib, kv, mod, hq=4, rows=4, max_q=4, max_len=64, scale=0.1, mask=0, tree=None, q=256, cu=256, ws=None, wb=0):
    return lib.sv_spec_verify_attn_scored(None if kv is None else ctypes.byref(kv), P(q), P(256), P(cu), hq, rows, max_q, max_len, scale,
                                          None if mod is None else ctypes.byref(mod), None, mask, P(tree), P(ws), wb, None, None)


def test_attention(lib):
    mod = lambda **kw: L.sv_score_mod(**kw)  # noqa: E731
    assert attend(lib, cache(batch=0), mod()) == 0
    assert attend(lib, cache(), mod(), rows=0) == 0
    assert attend(lib, None, mod()) == INVALID
    assert attend(lib, cache(), None) == INVALID
    for bad in (dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=float("inf")), dict(window=-1)):
        assert attend(lib, cache(), mod(**bad)) == INVALID, bad
    for bad in (dict(hq=3), dict(hq=0), dict(rows=-1), dict(max_q=0), dict(max_q=65), dict(max_len=0), dict(scale=float("nan")), dict(mask=2),
                dict(mask=1), dict(q=None), dict(q=264), dict(cu=None)):
        assert attend(lib, cache(), mod(), **bad) == INVALID, bad
    assert attend(lib, cache(head_dim=40), mod()) == UNSUPPORTED
    assert attend(lib, cache(), mod(), max_len=(1 << 30) + 1) == UNSUPPORTED
    assert attend(lib, cache(batch=65536), mod()) == UNSUPPORTED


def test_workspace(lib):
    kv = cache(max_blocks_per_seq=1000)
    need = lib.sv_spec_verify_attn_scored_workspace_bytes(ctypes.byref(kv), 4, 8, 4, 10000)
    assert need > 0
    assert attend(lib, kv, L.sv_score_mod(), rows=8, max_len=10000) == WORKSPACE
    assert attend(lib, kv, L.sv_score_mod(), rows=8, max_len=10000, ws=256, wb=need - 1) == WORKSPACE
    assert attend(lib, kv, L.sv_score_mod(), rows=8, max_len=10000, ws=264, wb=need) == WORKSPACE
    for bad in ((3, 8, 4, 64), (4, -1, 4, 64), (4, 8, 0, 64), (4, 8, 65, 64), (4, 8, 4, 0), (4, 8, 4, (1 << 30) + 1)):
        assert lib.sv_spec_verify_attn_scored_workspace_bytes(ctypes.byref(kv), *bad) == 0
