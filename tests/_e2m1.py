"""The 4-bit pool's format, plainly (not collected as tests): numpy, nearest neighbours by search."""
import numpy as np
import torch

from speculative_decoding_verify_paged_gb300 import step as S

MAGNITUDES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def e4m3_table():
    """Values of the codes 0 .. 126; 127 is NaN."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))


def nearest(x, table):
    """Index of the nearest of an ascending table, ties to the even index, saturating. x: finite, >= 0."""
    at = np.clip(np.searchsorted(table, x), 1, len(table) - 1)
    lo, hi = table[at - 1], table[at]
    up = (x - lo > hi - x) | ((x - lo == hi - x) & (at % 2 == 0))
    return np.where(x >= table[-1], len(table) - 1, np.where(up, at, at - 1))


def quantise(x, scale):
    """Rows [..., d] (values of bf16 or fp32) -> codes uint8 [..., d / 2], block scales uint8 [..., d / 16]."""
    x = np.asarray(x, np.float32).reshape(*x.shape[:-1], -1, 16)
    one, scale = np.float32(1), np.float32(scale)
    with np.errstate(all="ignore"):
        top = np.abs(x).max(-1)
        nan = np.isnan(top)
        s = nearest(np.where(nan, 0, np.minimum(np.nan_to_num(top * (one / (np.float32(6) * scale)), nan=0.0), np.float32(1e30))).astype(np.float64),
                    e4m3_table())
        step = e4m3_table()[s].astype(np.float32) * scale
        r = np.where(step > 0, one / np.where(step > 0, step, one), np.float32(0))[..., None]
        y = x * r
        code = nearest(np.minimum(np.nan_to_num(np.abs(y), nan=0.0, posinf=1e30), 1e30).astype(np.float64), MAGNITUDES) | (np.signbit(y) << 3)
    s = np.where(nan, 127, s).astype(np.uint8)
    code = code.astype(np.uint8).reshape(*x.shape[:-2], -1)
    return code[..., 0::2] | (code[..., 1::2] << 4), s


def values(codes, scales, scale):
    """What they stand for, in 64 bits."""
    n = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1)
    v = MAGNITUDES[n & 7] * np.where(n & 8, -1.0, 1.0)
    table = np.append(e4m3_table(), np.nan)
    s = np.where(scales & 128, -1.0, 1.0) * table[scales & 127] * float(np.float32(scale))
    return v * np.repeat(s, 16, -1)


def device_kv(state, k_scale=0.75, v_scale=1.25, ref_count=None):
    """The cache of a bf16 state with its rows as E2M1 codes."""
    kv = S.device_kv(state, "cuda", ref_count=ref_count)
    for name, scale in (("k", k_scale), ("v", v_scale)):
        codes, scales = quantise(getattr(kv, name + "_pool").float().cpu().numpy(), scale)
        setattr(kv, name + "_pool", torch.from_numpy(codes).cuda())
        setattr(kv, name + "_block_scales", torch.from_numpy(scales).cuda())
        setattr(kv, name + "_scale", scale)
    return kv


def pools(kv):
    """Both pools in 64 bits, [blocks, heads, block_size, head_dim]."""
    return tuple(values(getattr(kv, n + "_pool").cpu().numpy(), getattr(kv, n + "_block_scales").cpu().numpy(), getattr(kv, n + "_scale"))
                 for n in "kv")
