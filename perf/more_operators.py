"""Cases and plain forms of the operators around a paged cache held in 4 bits.

Four operators, as a decoder layer over such a cache uses them:

* ``append``  a step's key and value rows into the cache, as E2M1 codes with a scale per 16 values, and
              back out as the values that the codes stand for (what a prompt's attention has to see, so that
              it agrees with the later steps),
* ``gather``  rows of the sequences' contexts out of the cache as dense rows,
* ``attend``  attention of the step's rows over the cache, for chains and draft trees, with capped scores, a
              bias that falls with distance and a window of visible distances where the model has them,
* ``axes``    head norms and rotation of queries and keys whose positions have several axes (time, height,
              width of an image's or a video's tokens).

``own`` selects the plain torch forms (False) or the framework's entry points (True).
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
K_SCALE, V_SCALE = 0.75, 1.25  # of the pools
GROUP = 16                     # values that share a scale
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def listed():
    shape = dict(hq=32, hkv=8, d=128, bs=16)
    append = dict(op="append", hkv=8, d=128, bs=16)
    gather = dict(op="gather", hkv=8, d=128, bs=16, lens="uniform", share=1.0)
    attend = dict(shape, op="attend", n_lo=6, n_hi=6, lens="uniform", tree=False, softcap=0.0, slopes=False, window=0)
    axes = dict(op="axes", dtype="bf16", hq=32, hkv=8, d=128, sections="16,24,24", turns=False, interleaved=False, norm=True)
    return [
        # the verify step of the 32-sequence benchmark: six rows a sequence
        dict(append, name="append-32x6", batch=32, n_lo=6, n_hi=6, ctx_lo=512, ctx_hi=4096),
        # prompt chunks of 64 rows into young sequences
        dict(append, name="append-256x64-chunks", batch=256, n_lo=64, n_hi=64, ctx_lo=0, ctx_hi=64, bs=128),
        # a few short contexts leave the cache: launch and latency alone
        dict(gather, name="gather-4-short", batch=4, ctx_lo=37, ctx_hi=200, hkv=2, d=64),
        # the 32-sequence benchmark's whole contexts, for a dense kernel or another pool
        dict(gather, name="gather-32-contexts", batch=32, ctx_lo=512, ctx_hi=4096),
        # the smallest heads and the shortest contexts
        dict(attend, name="attend-4-short", batch=4, n_lo=5, n_hi=5, ctx_lo=37, ctx_hi=200, hq=4, hkv=2, d=64, softcap=20.0),
        # the 32-sequence benchmark's step
        dict(attend, name="attend-32x6", batch=32, ctx_lo=512, ctx_hi=4096),
        # plain decoding: one new token a sequence, few long sequences, wide query groups
        dict(attend, name="attend-4-long", batch=4, n_lo=1, n_hi=1, ctx_lo=32000, ctx_hi=32700, hq=64),
        # continuous batching: ragged draft lengths, contexts from a few tokens to thousands, large blocks, capped scores
        dict(attend, name="attend-128-ragged", batch=128, n_lo=3, n_hi=9, ctx_lo=16, ctx_hi=8192, bs=128, lens="log", softcap=30.0),
        # short contexts of many sequences, wide query groups
        dict(attend, name="attend-128x5-wide-groups", batch=128, n_lo=5, n_hi=5, ctx_lo=512, ctx_hi=640, hq=64),
        # draft trees of 61 rows over long contexts: limited by the products, not by memory
        dict(attend, name="attend-16-trees", batch=16, n_lo=61, n_hi=61, ctx_lo=8192, ctx_hi=8192, bs=64, tree=True),
        # one new token of each of four sequences: launch and latency alone
        dict(axes, name="axes-4-tokens", rows=4, far=4096),
        # the prompt chunks of a large batch of images: limited by memory, not by latency
        dict(axes, name="axes-16384-rows", rows=16384, far=32768),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(("append", "gather", "attend", "attend", "attend", "axes"))
    d = rng.choice((64, 128, 128, 256))
    hkv = rng.choice((1, 2, 4, 8))
    hq = hkv * rng.choice((1, 2, 4, 8))
    if op == "axes":
        dtype = rng.choice(("bf16", "bf16", "f32"))
        rows = min(_log_int(rng, 1, 16384), 16384 * 40 * 128 // ((hq + hkv) * d) // (2 if dtype == "f32" else 1))
        half = rng.choice((d, d, d // 2)) // 2
        side = rng.randint(1, half // 3)
        parts = rng.choice(((half - 2 * side, side, side), (half - side, side)))
        return dict(op=op, dtype=dtype, rows=rows if rng.random() < 0.5 else rows // 2 + 1, hq=hq, hkv=hkv, d=d,
                    sections=",".join(map(str, parts)), turns=rng.random() < 0.4, interleaved=rng.random() < 0.3,
                    norm=rng.random() < 0.7, far=_log_int(rng, 64, 1 << 20))
    if op == "append":
        n_hi = _log_int(rng, 1, 64)
        ctx_hi = _log_int(rng, 64, 2048)
        room = min(2 ** 18 * 8 * 128 // (ctx_hi * hkv * d), 256 * 64 * 8 * 128 // (n_hi * hkv * d))
        return dict(op=op, batch=max(1, min(_log_int(rng, 1, 256), room)), n_lo=rng.randint(1, n_hi), n_hi=n_hi, ctx_lo=0, ctx_hi=ctx_hi,
                    hkv=hkv, d=d, bs=rng.choice((64, 128, 256)))
    if op == "gather":
        ctx_hi = _log_int(rng, 16, 32768)
        room = 32 * 4096 * 8 * 128 // (ctx_hi * hkv * d)
        return dict(op=op, batch=max(1, min(_log_int(rng, 1, 128), room)), ctx_lo=rng.choice((0, 1, ctx_hi // 2)), ctx_hi=ctx_hi, hkv=hkv, d=d,
                    bs=rng.choice((16, 16, 32, 64, 128)), lens=rng.choice(("uniform", "log")), share=rng.choice((1.0, 0.5)))
    tree = rng.random() < 0.2
    n_hi = rng.randint(8, 61) if tree else rng.choice((1, 1, rng.randint(2, 9), rng.randint(2, 9), rng.randint(10, 64)))
    ctx_hi = _log_int(rng, 16, 32768)
    # no more keys and no more products than the listed trees have
    room = min(2 ** 17 * 8 * 128 // ((ctx_hi + n_hi) * hkv * d), 16 * 61 * 8192 * 32 * 128 // (n_hi * (ctx_hi + n_hi) * hq * d))
    return dict(op=op, batch=max(1, min(_log_int(rng, 1, 128), room)), n_lo=n_hi if tree else rng.randint(1, n_hi), n_hi=n_hi,
                ctx_lo=rng.choice((0, 1, ctx_hi // 2)), ctx_hi=ctx_hi, hq=hq, hkv=hkv, d=d, bs=rng.choice((16, 16, 32, 64, 128)),
                lens=rng.choice(("uniform", "log")), tree=tree, softcap=rng.choice((0.0, 0.0, 15.0, 30.0, 50.0)),
                slopes=rng.random() < 0.3, window=rng.choice((0, 0, 0, _log_int(rng, 16, 4096))))


def _lengths(c):
    """Context lengths and row counts of a case's sequences: part of the case, whatever the seed."""
    r = np.random.RandomState(c["batch"] * 7919 + c["ctx_hi"] * 31 + c.get("n_hi", 0))
    if c.get("lens") == "log":
        ctx = np.exp(r.uniform(math.log(max(1, c["ctx_lo"])), math.log(c["ctx_hi"] + 1), c["batch"])).astype(np.int64)
        ctx = np.clip(ctx, c["ctx_lo"], c["ctx_hi"])
    else:
        ctx = r.randint(c["ctx_lo"], c["ctx_hi"] + 1, c["batch"]).astype(np.int64)
    if c["op"] == "gather":  # the first part of each context, or all of it
        return ctx, np.maximum((ctx * c["share"]).astype(np.int64), np.minimum(ctx, 1))
    n = r.randint(c["n_lo"], c["n_hi"] + 1, c["batch"]).astype(np.int64)
    if c["op"] == "append":
        # the rows fit the block that is being filled (slots 1 .. bs - n), so that a pass can be repeated on the same cache
        n = np.minimum(n, c["bs"] - 1)
        ctx = ctx - ctx % c["bs"] + 1 + ctx % c["bs"] % (c["bs"] - n)
    return ctx, n


def _axes(c):
    """The axis of each rotated pair: in sections, or (turns) dealt out in turn until an axis has its share, the rest to the first."""
    parts = [int(x) for x in c["sections"].split(",")]
    if not c["turns"]:
        return np.repeat(np.arange(len(parts)), parts)
    i = np.arange(sum(parts))
    a = i % len(parts)
    return np.where(i < len(parts) * np.array(parts)[a], a, 0)


def work(c):
    held = 0.5 + 1 / GROUP  # bytes of a value in the cache
    if c["op"] == "axes":
        values = c["rows"] * (c["hq"] + c["hkv"]) * c["d"]
        return {"bytes": 2 * values * (2 if c["dtype"] == "bf16" else 4) + 4 * c["rows"] * len(c["sections"].split(",")), "flops": 8 * values}
    ctx, n = _lengths(c)
    rows = int(n.sum())
    if c["op"] != "attend":
        values = 2 * rows * c["hkv"] * c["d"]
        return {"bytes": int(values * (2 + held) * (2 if c["op"] == "append" else 1)) + 4 * rows, "flops": 4 * values}
    seen = ctx + n if c["window"] == 0 else np.minimum(ctx + n, c["window"] + n - 1)  # keys that some row sees
    pairs = n * (np.minimum(ctx, c["window"]) if c["window"] else ctx) + n * (n + 1) // 2
    return {"bytes": int(int(seen.sum()) * 2 * c["hkv"] * c["d"] * held) + 4 * rows * c["hq"] * c["d"] + 4 * c["batch"],
            "flops": 4 * c["hq"] * c["d"] * int(pairs.sum())}


# ----------------------------------------------------------------------------
# the 4-bit format
# ----------------------------------------------------------------------------
def _quantised(x, pool_scale):
    """Codes (two a byte, the even value's below) and E4M3 scales of rows [..., d], in 32 bits: s the E4M3 number nearest to
    max|x| / (6 pool_scale) over 16 values, the codes nearest to x / (s pool_scale); ties to even, saturating."""
    x = x.float().unflatten(-1, (-1, GROUP))
    pool = torch.tensor(pool_scale, dtype=torch.float32, device=x.device)
    s = (x.abs().amax(-1, keepdim=True) * (1.0 / (6.0 * pool))).clamp(max=448.0).to(torch.float8_e4m3fn)
    step = s.float() * pool
    y = (x * torch.where(step == 0, torch.zeros_like(step), 1.0 / step))
    m = y.abs()
    # a border belongs to the even code of the two beside it
    code = (m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)
    code = (code | (torch.signbit(y).to(torch.uint8) << 3)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.squeeze(-1).view(torch.uint8)


def _values(codes, scales, pool_scale):
    """What codes and scales stand for, in 32 bits."""
    table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), dtype=torch.float32, device=codes.device)
    v = table[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()]
    s = scales.view(torch.float8_e4m3fn).float() * torch.tensor(pool_scale, dtype=torch.float32, device=codes.device)
    return (v.unflatten(-1, (-1, GROUP)) * s[..., None]).flatten(-2)


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _normal(g, shape, dtype="bf16", sigma=1.0):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    return (x * sigma).to(torch.float32 if dtype == "f32" else torch.bfloat16)


def _trees(n, r):
    """Random draft trees in breadth-first order: each row's depth and its ancestors' bits (its own among them)."""
    depth, bits = [], []
    for k in n.tolist():
        d, m = [0], [1]
        for j in range(1, k):
            p = int(r.randint(max(0, j - 6) // 2, j))
            d.append(d[p] + 1)
            m.append(m[p] | (1 << j))
        depth += d
        bits += m
    return np.array(depth, np.int64), np.array(bits, np.uint64).view(np.int64)


def _pool(g, shape, pool_scale):
    """A pool that holds N(0, 1) rows."""
    codes = torch.empty(shape[:-1] + (shape[-1] // 2,), dtype=torch.uint8, device="cuda")
    scales = torch.empty(shape[:-1] + (shape[-1] // GROUP,), dtype=torch.uint8, device="cuda")
    part = max(1, 2 ** 25 // (shape[1] * shape[2] * shape[3]))
    for k in range(0, shape[0], part):
        codes[k:k + part], scales[k:k + part] = _quantised(_normal(g, (min(part, shape[0] - k),) + shape[1:]), pool_scale)
    return codes, scales


def _cache(c, g, held_tokens):
    """A shuffled pool with the sequences' blocks and as many free ones."""
    bs, batch = c["bs"], c["batch"]
    held = (held_tokens + bs - 1) // bs
    width = int(held.max()) + 1
    total = int(held.sum())
    blocks = total + batch
    order = torch.randperm(blocks, generator=g, device="cuda", dtype=torch.int32)
    first = np.concatenate([[0], np.cumsum(held)])[:-1]
    col = torch.arange(width, device="cuda")[None, :]
    start, count = (torch.from_numpy(x).cuda()[:, None] for x in (first, held))
    table = torch.where(col < count, order[(start + col).clamp(max=blocks - 1)], torch.full((), -1, dtype=torch.int32, device="cuda"))
    shape = (blocks, c["hkv"], bs, c["d"])
    k, ks = _pool(g, shape, K_SCALE)
    v, vs = _pool(g, shape, V_SCALE)
    free = torch.full((blocks,), -1, dtype=torch.int32, device="cuda")
    free[:batch] = order[total:]
    return {"k_pool": k, "k_scales": ks, "v_pool": v, "v_scales": vs, "table": table.contiguous(), "free": free,
            "top": torch.full((1,), batch, dtype=torch.int32, device="cuda"), "status": torch.zeros(1, dtype=torch.int32, device="cuda")}


def _i32(x):
    return torch.from_numpy(np.asarray(x, np.int32)).cuda()


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = np.random.RandomState(seed & 0x7FFFFFFF)
    s = {"case": c}
    if c["op"] == "axes":
        # one projection's output holds queries, keys and values of a row side by side
        qkv = _normal(g, (c["rows"], c["hq"] + 2 * c["hkv"], c["d"]), c["dtype"], 2.0)
        axis = _axes(c)
        half = len(axis)
        s.update(q=qkv[:, :c["hq"]], k=qkv[:, c["hq"]:c["hq"] + c["hkv"]], axis=torch.from_numpy(axis).cuda(), axes=bytes(axis.tolist()),
                 inv_freq=(10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)).float(), q_weight=None, k_weight=None)
        # the first axis runs far, the others stay within a picture
        far = torch.tensor([c["far"]] + [min(c["far"], 256)] * (int(axis.max())), device="cuda")[:, None]
        s["positions"] = (torch.rand((far.shape[0], c["rows"]), generator=g, device="cuda", dtype=torch.float64) * far).int()
        if c["norm"]:
            for name in ("q_weight", "k_weight"):
                s[name] = (1.0 + 0.2 * torch.randn(c["d"], generator=g, device="cuda")).to(qkv.dtype)
        s["q_out"], s["k_out"] = (torch.empty(x.shape, dtype=x.dtype, device="cuda") for x in (s["q"], s["k"]))
        return s
    ctx, n = _lengths(c)
    rows, n_max = int(n.sum()), int(n.max())
    s.update(_cache(c, g, ctx if c["op"] == "gather" else ctx + n), lens=_i32(ctx), cu=_i32(np.concatenate([[0], np.cumsum(n)])), rows=rows)
    if c["op"] == "gather":
        s["first"] = _i32(np.zeros(c["batch"]))
    if c["op"] == "append":
        # keys with a few large values a head, as rotated keys have them
        kv = _normal(g, (rows, 2 * c["hkv"], c["d"]))
        kv[:, :c["hkv"], :4] *= 6.0
        s["new_k"], s["new_v"] = kv[:, :c["hkv"]].contiguous(), kv[:, c["hkv"]:].contiguous()
    if c["op"] != "attend":
        s["k_out"], s["v_out"] = (torch.empty((rows, c["hkv"], c["d"]), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        return s
    s.update(n_max=n_max, l_max=int((ctx + n).max()), tree_mask=None, positions=None, slopes=None)
    if c["tree"]:
        depth, bits = _trees(n, r)
        s["tree_mask"] = torch.from_numpy(bits).cuda()
        s["positions"] = _i32(np.repeat(ctx, n) + depth)
    if c["slopes"]:
        s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, c["hq"] + 1, device="cuda", dtype=torch.float32) / c["hq"])
    s["q"] = _normal(g, (rows, c["hq"], c["d"]), sigma=3.0)
    s["out"] = torch.empty_like(s["q"])
    return s


# ----------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------
def _owner(cu, total):
    """The sequence and the place in it of every row."""
    rows = torch.arange(total, device=cu.device, dtype=cu.dtype)
    seq = torch.searchsorted(cu, rows, right=True) - 1
    return seq, rows - cu[seq]


def _gather_plain(s, c, first):
    seq, i = _owner(s["cu"], s["rows"])
    at = first[seq] + i
    block, slot = s["table"][seq, at // c["bs"]].long(), (at % c["bs"]).long()
    s["k_out"].copy_(_values(s["k_pool"][block, :, slot], s["k_scales"][block, :, slot], K_SCALE))
    s["v_out"].copy_(_values(s["v_pool"][block, :, slot], s["v_scales"][block, :, slot], V_SCALE))
    return s["k_out"], s["v_out"]


def _append_plain(s, c):
    seq, i = _owner(s["cu"], s["rows"])
    at = s["lens"][seq] + i
    block, slot = s["table"][seq, at // c["bs"]].long(), (at % c["bs"]).long()
    s["k_pool"][block, :, slot], s["k_scales"][block, :, slot] = _quantised(s["new_k"], K_SCALE)
    s["v_pool"][block, :, slot], s["v_scales"][block, :, slot] = _quantised(s["new_v"], V_SCALE)
    return (*_gather_plain(s, c, s["lens"]), s["table"], s["free"], s["top"])


def _attend_plain(s, c):
    hkv, d, bs, batch, n_max = c["hkv"], c["d"], c["bs"], c["batch"], s["n_max"]
    group, width = c["hq"] // hkv, -(-s["l_max"] // bs)
    table = s["table"][:, :width].clamp(min=0).long()

    def gathered(codes, scales, pool_scale):
        codes, scales = (x[table].permute(0, 2, 1, 3, 4).reshape(batch, hkv, width * bs, -1) for x in (codes, scales))
        return _values(codes, scales, pool_scale)

    k, v = gathered(s["k_pool"], s["k_scales"], K_SCALE), gathered(s["v_pool"], s["v_scales"], V_SCALE)
    cu, lens = s["cu"].long(), s["lens"].long()
    n = cu[1:] - cu[:-1]
    i = torch.arange(n_max, device="cuda")
    row = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)  # [batch, n_max]
    live = i < n[:, None]
    q = s["q"][row].float().reshape(batch, n_max, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(batch, hkv, group * n_max, d)
    t = torch.arange(width * bs, device="cuda")
    j = t - lens[:, None]  # the new row that a key is, if it is one
    where_q = lens[:, None] + i if s["positions"] is None else s["positions"].long()[row]
    new = (cu[:-1, None] + j).clamp(min=0, max=s["q"].shape[0] - 1)
    where_k = t.expand(batch, -1) if s["positions"] is None else torch.where(j >= 0, s["positions"].long()[new], t)
    if s["tree_mask"] is None:
        sees = j[:, None, :] <= i[:, None]
    else:
        sees = (j[:, None, :] < 0) | (((s["tree_mask"][row][:, :, None] >> j.clamp(0, 63)[:, None, :]) & 1) == 1)
    sees = sees & (t < (lens + n)[:, None])[:, None, :] & live[:, :, None]
    far = where_q[:, :, None] - where_k[:, None, :]  # [batch, n_max, keys]
    if c["window"]:
        sees = sees & (far < c["window"])
    x = (q @ k.transpose(-1, -2)).reshape(batch, hkv, group, n_max, -1) * (1.0 / math.sqrt(d))
    if c["softcap"]:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    if s["slopes"] is not None:
        x = x - s["slopes"].reshape(hkv, group, 1, 1) * far[:, None, None].float()
    x = x.masked_fill(~sees[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    o = (p.reshape(batch, hkv, group * n_max, -1) @ v).reshape(batch, hkv, group, n_max, d).permute(0, 3, 1, 2, 4)
    s["out"].copy_(o.reshape(batch, n_max, c["hq"], d)[live])
    return s["out"]


def _rotated(x, weight, s, c):
    """Heads normalised (where a weight is given) and rotated, in 32 bits; the angles in 64."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    rot = 2 * s["inv_freq"].numel()
    angle = (s["positions"].double()[s["axis"]].T * s["inv_freq"].double())[:, None, :]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if c["interleaved"] else (x[..., :rot // 2], x[..., rot // 2:rot])
    u, w = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((u, w), -1).flatten(-2) if c["interleaved"] else torch.cat((u, w), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _axes_plain(s, c):
    s["q_out"].copy_(_rotated(s["q"], s["q_weight"], s, c))
    s["k_out"].copy_(_rotated(s["k"], s["k_weight"], s, c))
    return s["q_out"], s["k_out"]


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def _own(s, c):
    from speculative_decoding_verify_paged_gb300 import HeadTransform, PagedKV, ScoreMod, _lib as L
    if c["op"] == "axes":
        t = HeadTransform(inv_freq=s["inv_freq"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, interleaved=c["interleaved"],
                          axes=s["axes"])
        L.qk_norm_rope(t, s["q"], s["k"], s["positions"], s["q_out"], s["k_out"])
        return s["q_out"], s["k_out"]
    kv = PagedKV(s["k_pool"], s["v_pool"], s["table"], s["lens"], s["free"], s["top"], k_scale=K_SCALE, v_scale=V_SCALE,
                 k_block_scales=s["k_scales"], v_block_scales=s["v_scales"])
    if c["op"] == "append":
        L.kv_append(kv, s["new_k"], s["new_v"], s["cu"], s["status"])
        L.kv_gather(kv, s["k_out"], s["v_out"], s["cu"], s["status"])
        return s["k_out"], s["v_out"], s["table"], s["free"], s["top"]
    if c["op"] == "gather":
        L.kv_gather(kv, s["k_out"], s["v_out"], s["cu"], s["status"], first=s["first"])
        return s["k_out"], s["v_out"]
    L.spec_verify_attn_scored(
        kv, s["q"], s["out"], s["cu"], max_q=s["n_max"], max_seq_len=s["l_max"], scale=1.0 / math.sqrt(c["d"]),
        mod=ScoreMod(softcap=c["softcap"], slopes=s["slopes"], window=c["window"]), positions=s["positions"],
        mask_kind=L.SV_MASK_TREE if c["tree"] else L.SV_MASK_CAUSAL, tree_mask=s["tree_mask"], status=s["status"])
    return s["out"]


def run(s):
    c = s["case"]
    if own:
        return _own(s, c)
    if c["op"] == "gather":
        return _gather_plain(s, c, s["first"])
    return {"append": _append_plain, "attend": _attend_plain, "axes": _axes_plain}[c["op"]](s, c)


# ----------------------------------------------------------------------------
# the definitions in 64 bits, one head vector and one sequence at a time
# ----------------------------------------------------------------------------
def _value64(codes, scales, pool_scale):
    """A code is a sign, two exponent bits and one of the mantissa; a scale stands for 16 codes."""
    nibble = torch.empty(codes.shape + (2,), dtype=torch.int64, device="cuda")
    nibble[..., 0], nibble[..., 1] = codes % 16, torch.div(codes, 16, rounding_mode="floor")
    e, m = (nibble >> 1) % 4, nibble % 2
    v = torch.where(e == 0, m * 0.5, (1.0 + 0.5 * m) * 2.0 ** (e.double() - 1.0))
    v = torch.where(nibble >= 8, -v, v).reshape(*codes.shape[:-1], -1)
    return v * torch.repeat_interleave(scales.view(torch.float8_e4m3fn).double() * pool_scale, GROUP, -1)


def _turn64(x, weight, where, inv_freq, interleaved):
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * weight.double()
    half = inv_freq.numel()
    z = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), where.double() * inv_freq.double())[:, None]
    out = x.clone()
    even, odd = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    y = torch.complex(x[..., even].contiguous(), x[..., odd].contiguous()) * z
    out[..., even], out[..., odd] = y.real, y.imag
    return out


def exact(c, seed):
    if c["op"] == "append":
        return None  # what the codes stand for is already rounded, and the rest are whole numbers
    s = prepare(c, seed)
    if c["op"] == "axes":
        where = torch.stack([s["positions"][a] for a in _axes(c).tolist()], -1)  # a pair's position
        return tuple(_turn64(s[x], s[x + "_weight"], where, s["inv_freq"], c["interleaved"]) for x in ("q", "k"))
    ctx, n = _lengths(c)
    first = np.concatenate([[0], np.cumsum(n)])
    bs = c["bs"]

    def rows_of(b, total):
        ids = s["table"][b, :(total + bs - 1) // bs].long()
        return [_value64(*(s[x + y][ids].transpose(1, 2).flatten(0, 1)[:total] for y in ("_pool", "_scales")), scale)
                for x, scale in (("k", K_SCALE), ("v", V_SCALE))]

    if c["op"] == "gather":
        got = [rows_of(b, int(n[b])) for b in range(c["batch"])]
        return torch.cat([x[0] for x in got]), torch.cat([x[1] for x in got])
    if work(c)["flops"] > 3e11:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group = c["hq"] // c["hkv"]
    for b in range(c["batch"]):
        lo, hi, have, rows = int(first[b]), int(first[b + 1]), int(ctx[b]), int(n[b])
        total = have + rows
        k, v = rows_of(b, total)
        place = torch.arange(total, device="cuda")
        if s["positions"] is not None:
            place[have:] = s["positions"][lo:hi].long()
        mask = torch.ones((rows, total), dtype=torch.bool, device="cuda")
        new = torch.arange(rows, device="cuda")
        mask[:, have:] = new[None] <= new[:, None] if s["tree_mask"] is None else ((s["tree_mask"][lo:hi, None] >> new) & 1).bool()
        gap = place[have:, None] - place[None]
        if c["window"]:
            mask &= gap < c["window"]
        q = s["q"][lo:hi].double().reshape(rows, c["hkv"], group, c["d"])
        x = torch.einsum("ihgd,thd->hgit", q, k) / math.sqrt(c["d"])
        if c["softcap"]:
            x = torch.tanh(x / c["softcap"]) * c["softcap"]
        if s["slopes"] is not None:
            x = x - s["slopes"].double().reshape(c["hkv"], group, 1, 1) * gap
        p = torch.softmax(x.masked_fill(~mask, -math.inf), -1).nan_to_num(0.0)
        out[lo:hi] = torch.einsum("hgit,thd->ihgd", p, v).reshape(rows, c["hq"], c["d"])
    return out
