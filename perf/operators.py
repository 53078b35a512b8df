"""Cases and plain forms of the operators that a verify step runs around its paged cache.

Three operators, as a decoder layer with normalised and rotated heads uses them:

* ``heads``   norms of queries and keys per head with the position rotation in the same pass,
* ``append``  the same on the way into the paged cache: keys are normalised, rotated and stored
              (as E4M3 codes in an 8-bit pool), values stored, queries written beside it,
* ``attend``  attention of the step's rows over the paged cache with scores capped by a tanh, a
              bias that falls with distance, and a window of visible distances, for chains and
              draft trees.

``own`` selects the plain torch forms (False) or the framework's entry points (True).
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
SCALE_8BIT = 0.125  # scale of the 8-bit pools


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def listed():
    heads = dict(op="heads", dtype="bf16", hq=32, hkv=8, d=128, rot=128, interleaved=False, norm=True, offset=0.0, far=4096)
    append = dict(op="append", dtype="bf16", hq=32, hkv=8, d=128, rot=128, interleaved=False, norm=True, offset=0.0, bs=16,
                  tree=False)
    attend = dict(op="attend", dtype="bf16", hq=32, hkv=8, d=128, bs=16, n_lo=6, n_hi=6, lens="uniform", tree=False, softcap=0.0,
                  slopes=False, window=0)
    return [
        # one new token of each of four sequences: launch and latency alone
        dict(heads, name="heads-4-tokens", rows=4),
        # a verify step of 128 sequences with 5 rows each, wide query groups, part of each head rotated, weights stored as w - 1
        dict(heads, name="heads-640-rows-partial", rows=640, hq=64, rot=64, interleaved=True, offset=1.0, far=131072),
        # the prompt chunks of a large batch: limited by memory, not by latency
        dict(heads, name="heads-16384-rows", rows=16384, far=32768),
        # the verify step of the 32-sequence benchmark: six rows a sequence
        dict(append, name="append-32x6", batch=32, n_lo=6, n_hi=6, ctx_lo=512, ctx_hi=4096),
        # continuous batching: ragged draft lengths, large blocks, an 8-bit pool
        dict(append, name="append-256-ragged-e4m3", dtype="e4m3", batch=256, n_lo=3, n_hi=9, ctx_lo=16, ctx_hi=2048, bs=128),
        # prompt chunks of 64 rows into young sequences
        dict(append, name="append-256x64-chunks", batch=256, n_lo=64, n_hi=64, ctx_lo=0, ctx_hi=64, bs=128),
        # fp32, the smallest heads and the shortest contexts
        dict(attend, name="attend-4-f32", dtype="f32", batch=4, n_lo=5, n_hi=5, ctx_lo=37, ctx_hi=200, hq=4, hkv=2, d=64, softcap=20.0),
        # the 32-sequence benchmark's step with capped scores
        dict(attend, name="attend-32x6-capped", batch=32, ctx_lo=512, ctx_hi=4096, softcap=30.0),
        # plain decoding: one new token a sequence, few long sequences, an 8-bit pool
        dict(attend, name="attend-4-long-e4m3", dtype="e4m3", batch=4, n_lo=1, n_hi=1, ctx_lo=32000, ctx_hi=32700, hq=64, softcap=50.0),
        # continuous batching with a distance bias and a sliding window: most keys of the long sequences are out of sight
        dict(attend, name="attend-128-window-biased", batch=128, n_lo=3, n_hi=9, ctx_lo=16, ctx_hi=8192, bs=128, lens="log",
             slopes=True, window=1024),
        # short contexts of many sequences, wide query groups
        dict(attend, name="attend-128x5-wide-groups", batch=128, n_lo=5, n_hi=5, ctx_lo=512, ctx_hi=640, hq=64, softcap=30.0),
        # draft trees of 61 rows over long contexts: limited by the products, not by memory
        dict(attend, name="attend-16-trees", batch=16, n_lo=61, n_hi=61, ctx_lo=8192, ctx_hi=8192, bs=64, tree=True, softcap=30.0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(("heads", "append", "attend", "attend"))
    d = rng.choice((64, 128, 128, 256))
    hkv = rng.choice((1, 2, 4, 8))
    hq = hkv * rng.choice((1, 2, 4, 8))
    if op == "heads":
        dtype = rng.choice(("bf16", "bf16", "f32"))
        rows = min(_log_int(rng, 1, 16384), 16384 * 40 * 128 // ((hq + hkv) * d) // (2 if dtype == "f32" else 1))
        return dict(op=op, dtype=dtype, rows=rows if rng.random() < 0.5 else rows // 2 + 1, hq=hq, hkv=hkv, d=d,
                    rot=rng.choice((d, d, d // 2, d // 4)), interleaved=rng.random() < 0.3, norm=rng.random() < 0.7,
                    offset=rng.choice((0.0, 1.0)), far=_log_int(rng, 64, 1 << 20))
    if op == "append":
        n_hi = _log_int(rng, 1, 64)
        ctx_hi = _log_int(rng, 64, 2048)
        dtype = rng.choice(("bf16", "bf16", "e4m3", "f32"))
        room = min(2 ** 18 * 8 * 128 // (ctx_hi * hkv * d), 256 * 64 * 40 * 128 // (n_hi * (hq + hkv) * d) // (2 if dtype == "f32" else 1))
        batch = max(1, min(_log_int(rng, 1, 256), room))
        return dict(op=op, dtype=dtype, batch=batch, n_lo=rng.randint(1, n_hi), n_hi=n_hi, ctx_lo=0,
                    ctx_hi=ctx_hi, hq=hq, hkv=hkv, d=d, rot=rng.choice((d, d, d // 2)), interleaved=rng.random() < 0.3,
                    norm=rng.random() < 0.7, offset=rng.choice((0.0, 1.0)), bs=rng.choice((64, 128, 256)),
                    tree=rng.random() < 0.25)
    dtype = rng.choice(("bf16", "bf16", "bf16", "e4m3", "e4m3", "f32"))
    tree = rng.random() < 0.2
    n_hi = rng.randint(8, 61) if tree else rng.choice((1, 1, rng.randint(2, 9), rng.randint(2, 9), rng.randint(10, 64)))
    ctx_hi = _log_int(rng, 16, 2048 if dtype == "f32" else 32768)
    # no more keys and no more products than the listed trees have
    room = min(2 ** 17 * 8 * 128 // ((ctx_hi + n_hi) * hkv * d), 16 * 61 * 8192 * 32 * 128 // (n_hi * (ctx_hi + n_hi) * hq * d))
    if dtype == "f32":
        room //= 16
    batch = max(1, min(_log_int(rng, 1, 128), room))
    return dict(op=op, dtype=dtype, batch=batch, n_lo=n_hi if tree else rng.randint(1, n_hi), n_hi=n_hi, ctx_lo=rng.choice((0, 1, ctx_hi // 2)),
                ctx_hi=ctx_hi, hq=hq, hkv=hkv, d=d, bs=rng.choice((16, 16, 32, 64, 128)), lens=rng.choice(("uniform", "log")), tree=tree,
                softcap=rng.choice((0.0, 15.0, 30.0, 50.0)), slopes=rng.random() < 0.4,
                window=rng.choice((0, 0, _log_int(rng, 16, 4096))))


def _lengths(c):
    """Context lengths and row counts of a case's sequences: part of the case, whatever the seed."""
    r = np.random.RandomState(c["batch"] * 7919 + c["ctx_hi"] * 31 + c["n_hi"])
    if c.get("lens") == "log":
        ctx = np.exp(r.uniform(math.log(max(1, c["ctx_lo"])), math.log(c["ctx_hi"] + 1), c["batch"])).astype(np.int64)
        ctx = np.clip(ctx, c["ctx_lo"], c["ctx_hi"])
    else:
        ctx = r.randint(c["ctx_lo"], c["ctx_hi"] + 1, c["batch"]).astype(np.int64)
    n = r.randint(c["n_lo"], c["n_hi"] + 1, c["batch"]).astype(np.int64)
    if c["op"] == "append":
        # the rows fit the block that is being filled (slots 1 .. bs - n), so that a pass can be repeated on the same cache
        n = np.minimum(n, c["bs"] - 1)
        ctx = ctx - ctx % c["bs"] + 1 + ctx % c["bs"] % (c["bs"] - n)
    return ctx, n


def _size(dtype):
    return {"bf16": 2, "f32": 4, "e4m3": 1}[dtype]


def work(c):
    row = 2 if c["dtype"] != "f32" else 4  # queries, new rows and outputs
    if c["op"] == "heads":
        heads = c["rows"] * (c["hq"] + c["hkv"])
        return {"bytes": 2 * heads * c["d"] * row + 4 * c["rows"], "flops": heads * c["d"] * 8}
    ctx, n = _lengths(c)
    rows = int(n.sum())
    if c["op"] == "append":
        values = rows * c["d"]
        return {"bytes": values * (2 * c["hq"] * row + 2 * c["hkv"] * (row + _size(c["dtype"]))) + 4 * rows,
                "flops": values * (c["hq"] + c["hkv"]) * 8}
    seen = ctx + n if c["window"] == 0 else np.minimum(ctx + n, c["window"] + n - 1)  # keys that some row sees
    pairs = n * (np.minimum(ctx, c["window"]) if c["window"] else ctx) + n * (n + 1) // 2
    return {"bytes": int(seen.sum()) * 2 * c["hkv"] * c["d"] * _size(c["dtype"]) + 2 * rows * c["hq"] * c["d"] * row + 4 * c["batch"],
            "flops": 4 * c["hq"] * c["d"] * int(pairs.sum())}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _normal(g, shape, dtype, sigma=1.0):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    return (x * sigma).to(torch.float32 if dtype == "f32" else torch.bfloat16)


def _transform(c, g):
    """Rotation frequencies and the heads' norm weights."""
    half = c["rot"] // 2
    inv = (10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / max(half, 1))).float()
    t = {"inv_freq": inv, "q_weight": None, "k_weight": None}
    if c["norm"]:
        for name in ("q_weight", "k_weight"):
            w = 1.0 - c["offset"] + 0.2 * torch.randn(c["d"], generator=g, device="cuda")
            t[name] = w.to(torch.float32 if c["dtype"] == "f32" else torch.bfloat16)
    return t


def _trees(c, n, r):
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


def _cache(c, g, ctx, n):
    """A shuffled pool with the sequences' blocks, as many free ones, and the ragged rows' offsets."""
    bs, batch = c["bs"], c["batch"]
    held = (ctx + n + bs - 1) // bs
    width = int(held.max()) + 1
    total = int(held.sum())
    blocks = total + batch
    order = torch.randperm(blocks, generator=g, device="cuda", dtype=torch.int32)
    first = np.concatenate([[0], np.cumsum(held)])[:-1]
    col = torch.arange(width, device="cuda")[None, :]
    start, count = (torch.from_numpy(x).cuda()[:, None] for x in (first, held))
    table = torch.where(col < count, order[(start + col).clamp(max=blocks - 1)], torch.full((), -1, dtype=torch.int32, device="cuda"))
    shape = (blocks, c["hkv"], bs, c["d"])
    if c["dtype"] == "e4m3":
        # codes with exponent fields 3 .. 9: magnitudes 1/16 .. 7.5 before the scale
        def codes():
            e = torch.randint(3 * 8, 10 * 8, shape, generator=g, device="cuda", dtype=torch.uint8)
            return e | (torch.randint(0, 2, shape, generator=g, device="cuda", dtype=torch.uint8) << 7)
        k, v = codes(), codes()
    else:
        k, v = _normal(g, shape, c["dtype"]), _normal(g, shape, c["dtype"])
    free = torch.full((blocks,), -1, dtype=torch.int32, device="cuda")
    free[:batch] = order[total:]
    cu = np.concatenate([[0], np.cumsum(n)])
    i32 = lambda x: torch.from_numpy(np.asarray(x, np.int32)).cuda()  # noqa: E731
    return {"k_pool": k, "v_pool": v, "table": table.contiguous(), "lens": i32(ctx), "free": free, "top": i32([batch]), "cu": i32(cu),
            "status": torch.zeros(1, dtype=torch.int32, device="cuda")}


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = np.random.RandomState(seed & 0x7FFFFFFF)
    s = {"case": c}
    if c["op"] == "heads":
        # one projection's output holds queries, keys and values of a row side by side
        qkv = _normal(g, (c["rows"], c["hq"] + 2 * c["hkv"], c["d"]), c["dtype"], 2.0)
        s.update(_transform(c, g), q=qkv[:, :c["hq"]], k=qkv[:, c["hq"]:c["hq"] + c["hkv"]])
        s["positions"] = torch.randint(0, c["far"], (c["rows"],), generator=g, device="cuda", dtype=torch.int32)
        s["q_out"], s["k_out"] = (torch.empty(x.shape, dtype=x.dtype, device="cuda") for x in (s["q"], s["k"]))
        return s
    ctx, n = _lengths(c)
    rows, n_max = int(n.sum()), int(n.max())
    s.update(_cache(c, g, ctx, n), n_max=n_max, l_max=int((ctx + n).max()))
    s["tree_mask"] = s["positions"] = None
    if c["tree"]:
        depth, bits = _trees(c, n, r)
        s["tree_mask"] = torch.from_numpy(bits).cuda()
        s["positions"] = torch.from_numpy((np.repeat(ctx, n) + depth).astype(np.int32)).cuda()
    if c["op"] == "append":
        qkv = _normal(g, (rows, c["hq"] + 2 * c["hkv"], c["d"]), c["dtype"], 2.0)
        s.update(_transform(c, g), q=qkv[:, :c["hq"]], k=qkv[:, c["hq"]:c["hq"] + c["hkv"]], v=qkv[:, c["hq"] + c["hkv"]:])
        s["q_out"] = torch.empty((rows, c["hq"], c["d"]), dtype=qkv.dtype, device="cuda")
        return s
    s["q"] = _normal(g, (rows, c["hq"], c["d"]), c["dtype"], 3.0)
    s["out"] = torch.empty_like(s["q"])
    s["slopes"] = None
    if c["slopes"]:
        s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, c["hq"] + 1, device="cuda", dtype=torch.float32) / c["hq"])
    return s


# ----------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------
def _owner(cu, total):
    """The sequence and the place in it of every row."""
    rows = torch.arange(total, device=cu.device, dtype=cu.dtype)
    seq = torch.searchsorted(cu, rows, right=True) - 1
    return seq, rows - cu[seq]


def _rotated(x, weight, positions, s, c):
    """Heads normalised (where a weight is given) and rotated, in 32 bits; the angles in 64."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * (weight.float() + c["offset"])
    rot = c["rot"]
    angle = (positions.double()[:, None] * s["inv_freq"].double())[:, None, :]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if c["interleaved"] else (x[..., :rot // 2], x[..., rot // 2:rot])
    u, w = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((u, w), -1).flatten(-2) if c["interleaved"] else torch.cat((u, w), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _heads_plain(s, c):
    s["q_out"].copy_(_rotated(s["q"], s["q_weight"], s["positions"], s, c))
    s["k_out"].copy_(_rotated(s["k"], s["k_weight"], s["positions"], s, c))
    return s["q_out"], s["k_out"]


def _append_plain(s, c):
    seq, i = _owner(s["cu"], s["q"].shape[0])
    at = s["lens"][seq] + i
    positions = at if s["positions"] is None else s["positions"]
    block, slot = s["table"][seq, at // c["bs"]].long(), (at % c["bs"]).long()
    k, v = _rotated(s["k"], s["k_weight"], positions, s, c), s["v"].float()
    if c["dtype"] == "e4m3":
        k, v = ((x / SCALE_8BIT).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8) for x in (k, v))
    s["k_pool"][block, :, slot] = k.to(s["k_pool"].dtype)
    s["v_pool"][block, :, slot] = v.to(s["v_pool"].dtype)
    s["q_out"].copy_(_rotated(s["q"], s["q_weight"], positions, s, c))
    return _append_outputs(s, c)


def _append_outputs(s, c):
    k, v = ((s[p].view(torch.float8_e4m3fn) if c["dtype"] == "e4m3" else s[p]) for p in ("k_pool", "v_pool"))
    return s["q_out"], k, v, s["table"], s["free"], s["top"]


def _attend_plain(s, c):
    hkv, d, bs, batch, n_max = c["hkv"], c["d"], c["bs"], c["batch"], s["n_max"]
    group, width = c["hq"] // hkv, -(-s["l_max"] // bs)
    table = s["table"][:, :width].clamp(min=0).long()

    def gathered(pool):
        x = pool.view(torch.float8_e4m3fn).float() * SCALE_8BIT if c["dtype"] == "e4m3" else pool
        return x[table].permute(0, 2, 1, 3, 4).reshape(batch, hkv, width * bs, d).float()

    k, v = gathered(s["k_pool"]), gathered(s["v_pool"])
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


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def _own(s, c):
    from speculative_decoding_verify_paged_gb300 import HeadTransform, PagedKV, ScoreMod, _lib as L
    if c["op"] == "attend":
        kv = PagedKV(s["k_pool"], s["v_pool"], s["table"], s["lens"], s["free"], s["top"], k_scale=SCALE_8BIT, v_scale=SCALE_8BIT)
        L.spec_verify_attn_scored(
            kv, s["q"], s["out"], s["cu"], max_q=s["n_max"], max_seq_len=s["l_max"], scale=1.0 / math.sqrt(c["d"]),
            mod=ScoreMod(softcap=c["softcap"], slopes=s["slopes"], window=c["window"]), positions=s["positions"],
            mask_kind=L.SV_MASK_TREE if c["tree"] else L.SV_MASK_CAUSAL, tree_mask=s["tree_mask"], status=s["status"])
        return s["out"]
    t = HeadTransform(inv_freq=s["inv_freq"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, weight_offset=c["offset"],
                      interleaved=c["interleaved"])
    if c["op"] == "heads":
        L.qk_norm_rope(t, s["q"], s["k"], s["positions"], s["q_out"], s["k_out"])
        return s["q_out"], s["k_out"]
    kv = PagedKV(s["k_pool"], s["v_pool"], s["table"], s["lens"], s["free"], s["top"], k_scale=SCALE_8BIT, v_scale=SCALE_8BIT)
    L.kv_append_rope(kv, t, s["k"], s["v"], s["cu"], s["status"], q=s["q"], q_out=s["q_out"], positions=s["positions"])
    return _append_outputs(s, c)


def run(s):
    c = s["case"]
    if own:
        return _own(s, c)
    return {"heads": _heads_plain, "append": _append_plain, "attend": _attend_plain}[c["op"]](s, c)


# ----------------------------------------------------------------------------
# the definitions in 64 bits, one head vector and one sequence at a time
# ----------------------------------------------------------------------------
def _turn64(x, weight, offset, where, inv_freq, interleaved):
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * (weight.double() + offset)
    half = inv_freq.numel()
    z = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), where.double()[:, None] * inv_freq.double())[:, None]
    out = x.clone()
    even, odd = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    y = torch.complex(x[..., even].contiguous(), x[..., odd].contiguous()) * z
    out[..., even], out[..., odd] = y.real, y.imag
    return out


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "heads":
        return tuple(_turn64(s[x], s[x + "_weight"], c["offset"], s["positions"], s["inv_freq"], c["interleaved"]) for x in ("q", "k"))
    ctx, n = _lengths(c)
    first = np.concatenate([[0], np.cumsum(n)])
    bs = c["bs"]
    if c["op"] == "append":
        at = torch.from_numpy(np.concatenate([np.arange(a, a + b) for a, b in zip(ctx, n)])).cuda()
        where = at if s["positions"] is None else s["positions"]
        q, k = (_turn64(s[x], s[x + "_weight"], c["offset"], where, s["inv_freq"], c["interleaved"]) for x in ("q", "k"))
        if c["dtype"] == "e4m3":
            return q, None, None, None, None, None  # the pools hold codes: what they stand for is already rounded
        pools = [s["k_pool"].double(), s["v_pool"].double()]
        seq = torch.from_numpy(np.repeat(np.arange(c["batch"]), n)).cuda()
        block = s["table"].long()[seq, at // bs]
        pools[0][block, :, at % bs], pools[1][block, :, at % bs] = k, s["v"].double()
        return q, pools[0], pools[1], None, None, None
    if work(c)["flops"] > 3e11:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group = c["hq"] // c["hkv"]
    for b in range(c["batch"]):
        lo, hi, have, rows = int(first[b]), int(first[b + 1]), int(ctx[b]), int(n[b])
        total = have + rows
        ids = s["table"][b, :(total + bs - 1) // bs].long()
        pool = []
        for p in (s["k_pool"], s["v_pool"]):
            x = p[ids].transpose(1, 2).reshape(-1, c["hkv"], c["d"])[:total]
            pool.append(x.view(torch.float8_e4m3fn).double() * SCALE_8BIT if c["dtype"] == "e4m3" else x.double())
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
        x = torch.einsum("ihgd,thd->hgit", q, pool[0]) / math.sqrt(c["d"])
        if c["softcap"]:
            x = torch.tanh(x / c["softcap"]) * c["softcap"]
        if s["slopes"] is not None:
            x = x - s["slopes"].double().reshape(c["hkv"], group, 1, 1) * gap
        p = torch.softmax(x.masked_fill(~mask, -math.inf), -1).nan_to_num(0.0)
        out[lo:hi] = torch.einsum("hgit,thd->ihgd", p, pool[1]).reshape(rows, c["hq"], c["d"])
    return out
