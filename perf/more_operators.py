"""The operators of a serving step around and inside the attention block, as they are measured.

Each case names one operator ("op") and its sizes. `run` with `own` false
computes it in elementary torch operations; with `own` true it makes the calls
a user of the library makes. The operators:

  norm    a layer's input: residual sum, root-mean-square norm and gain, as
          16 / 32-bit numbers or as e4m3 numbers with one scale a row
  back    its backward pass: the gradient of the sum's terms, and of the gain
  linear  a projection whose weights are held in 4 bits, of 16 / 32-bit rows or
          of e4m3 rows with their scales, with the residual added
  tree    attention of each request's tree of drafted tokens over the 4-bit
          paged cache (which holds the drafted tokens too, behind the others),
          with the tree's positions and visibility made from its parents
  move    accepted tokens moved to their places in the cache, and read back

Weights are uint8 [N / 16, K / 64, 544] (both rounded up): 512 bytes of 4-bit
numbers of 16 rows and 64 columns, and the rows' 16 scales, bf16. A number n
stands for s (n - 8). With lane = 4 r + j (r = 0..7, j = 0..3), word w = 0..3 of
a lane's 16 bytes holds, low nibble first, for e = 0, 1, q = 0, 1, hi = 0, 1 the
number of row r + 8 hi, column 16 j + 4 w + 2 q + e. Scale 2 r + hi is that of
row r + 8 hi.

The cache is that of kv4_append: uint8 [pages, kv heads, page / 16, 18 d], per
16 tokens 8 d bytes of keys, 8 d of values and one bf16 pair (s, z) per token
and 64 channels for each; a number n stands for s (n - 8) + z.
"""

import math
import random

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6
BASE = 10000.0
TOP8 = 448.0    # largest e4m3 number


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token for each of a batch's requests, in front of 8-bit projections: latency
        {"name": "norm_step", "op": "norm", "rows": 64, "C": 768, "type": "bf16", "add": True, "gain": True, "fp8": True},
        # a layer of the benchmark's block, whole batch
        {"name": "norm_layer", "op": "norm", "rows": 32768, "C": 768, "type": "bf16", "add": True, "gain": True, "fp8": False},
        # its backward pass
        {"name": "back_layer", "op": "back", "rows": 32768, "C": 768, "type": "bf16", "gain": True, "dh": True},
        # a wide model in 32 bits, an odd number of rows
        {"name": "back_wide", "op": "back", "rows": 5001, "C": 8192, "type": "fp32", "gain": True, "dh": False},
        # q, k and v of one token in the benchmark's block: latency
        {"name": "linear_token", "op": "linear", "M": 1, "N": 1536, "K": 768, "type": "bf16", "fp8": False, "add": False},
        # a few drafted tokens of a few requests through a wide model's projection, 8-bit rows
        {"name": "linear_drafts", "op": "linear", "M": 24, "N": 8192, "K": 8192, "type": "bf16", "fp8": True, "add": False},
        # a prompt of the training length through the output projection of sixteen heads of 128
        {"name": "linear_prompt", "op": "linear", "M": 2048, "N": 2048, "K": 2048, "type": "bf16", "fp8": False, "add": True},
        # one request of the small model, four drafted tokens: latency
        {"name": "tree_tiny", "op": "tree", "B": 1, "max_new": 4, "Hq": 2, "Hkv": 1, "d": 64, "page": 16, "max_len": 256,
         "window": 128, "even": True, "rot": 64, "interleaved": False, "type": "bf16"},
        # a batch of long contexts on a full layer, four query heads to a kv head, sixteen drafted tokens
        {"name": "tree_long", "op": "tree", "B": 16, "max_new": 16, "Hq": 16, "Hkv": 4, "d": 128, "page": 64, "max_len": 32768,
         "window": -1, "even": True, "rot": 128, "interleaved": False, "type": "bf16"},
        # plain multi-head attention in 32 bits, ragged, small pages
        {"name": "tree_fp32", "op": "tree", "B": 16, "max_new": 11, "Hq": 6, "Hkv": 6, "d": 128, "page": 16, "max_len": 5000,
         "window": -1, "even": False, "rot": 32, "interleaved": True, "type": "fp32"},
        # the accepted tokens of one layer of the benchmark's stack
        {"name": "move_step", "op": "move", "B": 32, "T": 8, "Hkv": 3, "d": 128, "page": 64},
        # of a large batch with large trees
        {"name": "move_batch", "op": "move", "B": 2048, "T": 32, "Hkv": 4, "d": 128, "page": 32},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "back", "back", "linear", "linear", "linear", "tree", "tree", "tree", "move"])
    t = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("norm", "back"):
        C = 8 * _log(rng, 1, 2048)
        rows = _log(rng, 1, max(1, min(32768, 32768 * 768 // C)))
        case = {"op": op, "rows": rows, "C": C, "type": t, "gain": rng.random() < 0.8}
        return {**case, "add": rng.random() < 0.7, "fp8": rng.random() < 0.4} if op == "norm" else {**case, "dh": rng.random() < 0.6}
    if op == "linear":
        N, K = _log(rng, 1, 8192), 8 * _log(rng, 1, 1024)
        M = _log(rng, 1, max(1, min(2048, 2048 ** 3 // (N * K))))
        if t == "fp32":
            M = min(M, 128)
        return {"op": op, "M": M, "N": N, "K": K, "type": t, "fp8": rng.random() < 0.3, "add": rng.random() < 0.4}
    d = rng.choice([64, 128, 128])
    page = 16 * rng.choice([1, 2, 3, 4, 8])
    if op == "move":
        T = _log(rng, 2, 64)
        return {"op": op, "B": _log(rng, 1, max(1, min(2048, 65536 // T))), "T": T, "Hkv": rng.randint(1, 4), "d": d, "page": page}
    G, Hkv, T = rng.choice([1, 2, 3, 4, 4, 6, 8]), rng.randint(1, 4), _log(rng, 1, 64)
    if t == "fp32":
        T = min(T, 24)
    max_len = max(T + 1, _log(rng, 1, 32768))
    most = max(1, min(64, 32768 * 64 * 16 * 3 // (max_len * Hkv * max(16, G * T))))
    return {"op": op, "B": _log(rng, 1, most), "max_new": T, "Hq": G * Hkv, "Hkv": Hkv, "d": d, "page": page, "max_len": max_len,
            "window": rng.choice([-1, -1, _log(rng, 1, 8192)]), "even": rng.random() < 0.3,
            "rot": rng.choice([16 * rng.randint(1, d // 16), d]), "interleaved": rng.random() < 0.5, "type": t}


def _fixed(case):
    """Lengths are part of the case, not of the seed: a pass always has the same work."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _tree_sizes(case):
    """Cached tokens of each request (the drafted ones among them), and its drafted tokens."""
    r, top, T = _fixed(case), case["max_len"], case["max_new"]
    lens = [r.randint(max(1, top - top // 8), top) if case["even"] else _log(r, 1, top) for _ in range(case["B"])]
    lens[r.randrange(case["B"])] = top
    new = [min(n, T if case["even"] else r.randint(1, T)) for n in lens]
    return lens, new


def _move_sizes(case):
    """Accepted tokens of each request that have to move: tokens 1 .. a - 1 of its path (the first is in place)."""
    r = _fixed(case)
    return [r.randint(1, max(1, case["T"] // 2)) for _ in range(case["B"])]


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _tables(rows, rot):
    ang = torch.arange(rows, device=DEV, dtype=torch.float64)[:, None] * (
        BASE ** (-torch.arange(rot // 2, device=DEV, dtype=torch.float64) * 2.0 / rot))
    return ang.cos().float(), ang.sin().float()


def _cache(n_pages, case, g):
    """A cache full of tokens: steps near 0.2, centres near 0."""
    d = case["d"]
    c = torch.randint(0, 256, (n_pages, case["Hkv"], case["page"] // 16, 18 * d), generator=g, device=DEV, dtype=torch.uint8)
    pairs = c[..., 16 * d:].view(torch.bfloat16)
    shape = pairs[..., 0::2].shape
    pairs[..., 0::2] = (0.2 + 0.05 * torch.rand(shape, generator=g, device=DEV)).bfloat16()
    pairs[..., 1::2] = (0.1 + 0.1 * torch.randn(shape, generator=g, device=DEV)).bfloat16()
    return c


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    if op in ("norm", "back"):
        t, rows, C = TYPES[case["type"]], case["rows"], case["C"]
        s["x"] = (2.0 * randn(rows, C)).to(t)
        s["g"] = 1.0 + 0.1 * randn(C) if case["gain"] else None
        if op == "norm":
            s["r"] = randn(rows, C).to(t) if case["add"] else None
        else:  # what the forward pass left, and the gradients that come back
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(-1) + EPS)
            s["dy"] = randn(rows, C).to(t)
            s["gh"] = randn(rows, C).to(t) if case["dh"] else None
        return s
    if op == "linear":
        t, M, N, K = TYPES[case["type"]], case["M"], case["N"], case["K"]
        x = randn(M, K)
        s["scale"] = None
        if case["fp8"]:
            s["scale"] = x.abs().amax(-1) / TOP8
            s["x"] = (x / s["scale"][:, None]).to(torch.float8_e4m3fn)
        else:
            s["x"] = x.to(t)
        P, Q = -(-N // 16), -(-K // 64)
        w = torch.randint(0, 256, (P, Q, 544), generator=g, device=DEV, dtype=torch.uint8)
        w[..., 512:].view(torch.bfloat16).copy_((0.2 + 0.1 * torch.rand(P, Q, 16, generator=g, device=DEV)) / math.sqrt(K))
        s["w"] = w
        s["r"] = randn(M, N).to(t) if case["add"] else None
        return s
    d, Hkv, page, B = case["d"], case["Hkv"], case["page"], case["B"]
    if op == "move":
        T = case["T"]
        per = -(-(T + page) // page)
        pages = torch.randperm(B * per + 2, generator=g, device=DEV)[:B * per].view(B, per)
        first = torch.randint(0, page, (B, 1), generator=g, device=DEV)
        at = first + torch.arange(T, device=DEV)[None, :]
        slot = torch.gather(pages, 1, at // page) * page + at % page
        took = torch.tensor(_move_sizes(case), device=DEV)[:, None]
        # the path's tokens lie behind the places that they go to, in the order of their depth
        i = torch.arange(T, device=DEV)[None, :]
        picked = torch.rand(B, T, generator=g, device=DEV).masked_fill(i < took, 2.0)
        path = picked.argsort(-1)[:, :max(_move_sizes(case))]
        path = path.masked_fill(torch.arange(path.shape[1], device=DEV)[None, :] >= took, T).sort(-1).values
        on = (torch.arange(path.shape[1], device=DEV)[None, :] < took) & (path < T)
        s["src"] = torch.where(on, torch.gather(slot, 1, path.clamp(max=T - 1)), -1)
        s["dst"] = torch.where(on, slot[:, :path.shape[1]], -1)
        s["cache"] = _cache(B * per + 2, case, g)
        return s
    (lens, new), t = _tree_sizes(case), TYPES[case["type"]]
    cap = -(-case["max_len"] // page) + 2
    held = [-(-n // page) for n in lens]
    n_pages, total = sum(held) + 1, sum(new)
    n_rows = -(-total // 8) * 8  # a step's token buffer is padded
    s["q"] = randn(n_rows, case["Hq"], d).to(t)
    s["gq"] = 1.0 + 0.1 * randn(d)
    s["tables"] = _tables(case["max_len"], case["rot"])
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["cu"] = torch.tensor([0] + new, device=DEV).cumsum(0).int()
    # a token's parent is one of the six in front of it, mostly the nearest; -1: the context's last token
    row = torch.repeat_interleave(torch.arange(B, device=DEV), torch.tensor(new, device=DEV))
    at = torch.arange(total, device=DEV) - s["cu"][row]
    back = (torch.rand(total, generator=g, device=DEV).square() * at.clamp(max=6)).long()
    s["parent"] = torch.zeros(n_rows, dtype=torch.int32, device=DEV)
    s["parent"][:total] = (at - 1 - back).int()
    held_t, i = torch.tensor(held, device=DEV), torch.arange(cap, device=DEV)[None, :]
    ids = torch.randperm(n_pages, generator=g, device=DEV)
    begin = torch.cumsum(held_t, 0) - held_t
    s["table"] = torch.where(i < held_t[:, None], ids[(begin[:, None] + i).clamp(max=n_pages - 1)], -1).int()
    s["cache"] = _cache(n_pages, case, g)
    return s


# ---------------------------------------------------------------------------
# The plain form
# ---------------------------------------------------------------------------

def _round8(t):
    """t (64 bits, at most 448 in size) rounded to the nearest e4m3 number, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6))) - 3.0)
    return torch.round(t / step) * step


def _norm_plain(s):
    x = s["x"].float()
    h = (x if s["r"] is None else x + s["r"].float()).to(s["x"].dtype)
    f = h.float()
    rstd = torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS)
    out = {"h": h, "rstd": rstd[:, 0]}
    if not s["fp8"]:
        y = f * rstd
        out["y"] = (y if s["g"] is None else y * s["g"]).to(h.dtype)
        return out
    # numbers next to a border of e4m3: in 64 bits, where the norm's factor drops out of y / max |y|
    u = h.double() if s["g"] is None else h.double() * s["g"].double()
    top = u.abs().amax(-1, keepdim=True)
    n = _round8(torch.where(top > 0, u * TOP8 / top, 0.0))
    out["scale"] = (top.float() * rstd / TOP8)[:, 0]
    out["y"] = n.float() * out["scale"][:, None]
    return out


def _back_plain(s):
    h, dy, r = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    n = h * r
    d = dy if s["g"] is None else dy * s["g"]
    dx = r * (d - n * (d * n).mean(-1, keepdim=True))
    if s["gh"] is not None:
        dx = dx + s["gh"].float()
    return {"dx": dx.to(s["x"].dtype), "dgain": (dy * n).sum(0)}


def _weights(w, N, K):
    """The weights [N, K] in 32 bits."""
    P, Q = w.shape[:2]
    b = w[..., :512].reshape(P, Q, 8, 4, 4, 4)                                   # r, j, word, byte
    n = torch.stack([b & 15, b >> 4], -1).reshape(P, Q, 8, 4, 4, 2, 2, 2)        # r, j, word, e, q, hi
    n = n.permute(0, 7, 2, 1, 3, 4, 6, 5).reshape(P * 16, Q, 64).float() - 8.0
    sc = w[..., 512:].contiguous().view(torch.bfloat16).view(P, Q, 8, 2).permute(0, 3, 2, 1).reshape(P * 16, Q, 1).float()
    return (n * sc).reshape(P * 16, Q * 64)[:N, :K]


def _linear_plain(s):
    x = s["x"].float()
    if s["scale"] is not None:
        x = x * s["scale"][:, None]
    y = x @ _weights(s["w"], s["N"], s["K"]).T
    if s["r"] is not None:
        y = y + s["r"].float()
    return {"y": y.to(TYPES[s["type"]])}


def _turn(x, cos, sin, interleaved):
    half = cos.shape[-1]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * cos + b * sin, b * cos - a * sin
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half], y[..., half:2 * half] = a * cos + b * sin, b * cos - a * sin
    return y


def _values(tiles):
    """Tiles [..., 18 d] as the keys and values they stand for, [..., 16, d] in 32 bits."""
    d = tiles.shape[-1] // 18
    G, lead = d // 64, tiles.shape[:-1]
    pairs = tiles[..., 16 * d:].contiguous().view(torch.bfloat16).view(*lead, 2, 16, G, 1, 2).float()
    b = tiles[..., :8 * d].reshape(*lead, 16, 4, G, 8)
    n = torch.stack([b & 15, b >> 4], -1).transpose(-4, -3).reshape(*lead, 16, G, 64)
    k = (n.float() - 8.0) * pairs[..., 0, :, :, :, 0] + pairs[..., 0, :, :, :, 1]
    b = tiles[..., 8 * d:16 * d].reshape(*lead, 8, 8, G, 2, 2, 2)  # pair, r, g, u, token, byte
    n = torch.stack([b & 15, b >> 4], -1)
    m = n.dim()
    n = n.permute(*range(m - 7), m - 7, m - 3, m - 5, m - 6, m - 4, m - 2, m - 1).reshape(*lead, 16, G, 64)
    v = (n.float() - 8.0) * pairs[..., 1, :, :, :, 0] + pairs[..., 1, :, :, :, 1]
    return k.flatten(-2), v.flatten(-2)


def _tree_plain(s):
    B, T, Hq, Hkv, d, page = s["B"], s["max_new"], s["Hq"], s["Hkv"], s["d"], s["page"]
    dev, n_rows = s["q"].device, s["q"].shape[0]
    lens, cu = s["lens"].long(), s["cu"].long()
    new = cu[1:] - cu[:-1]
    ctx = lens - new
    i = torch.arange(T, device=dev)
    real = i[None, :] < new[:, None]                                             # [B, T]
    flat = (cu[:-1, None] + i).clamp(max=n_rows - 1)
    # who is above whom: the parent relation squared until it holds the whole way up
    parent = torch.where(real, s["parent"].long()[flat], -1)
    up = (parent[:, :, None] == i[None, None, :]) | torch.eye(T, dtype=torch.bool, device=dev)[None]
    for _ in range(max(1, math.ceil(math.log2(T)))):
        up = (up.float() @ up.float()) > 0
    up = up & real[:, :, None] & real[:, None, :]
    pos2 = ctx[:, None] + up.sum(-1) - 1
    seen2 = (up.long() << i).sum(-1)
    pos = torch.zeros(n_rows, dtype=torch.int64, device=dev)
    seen = torch.zeros(n_rows, dtype=torch.int64, device=dev)
    pos[flat[real]], seen[flat[real]] = pos2[real], seen2[real]
    # the queries
    at = torch.where(real, pos2, 0)
    cos, sin = (t[at][:, :, None] for t in s["tables"])
    q = _turn(s["q"].float()[flat], cos, sin, s["interleaved"])
    q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + EPS) * s["gq"]
    q = q.view(B, T, Hkv, Hq // Hkv, d).transpose(1, 2).reshape(B, Hkv, -1, d)    # rows (token, head of the group)
    # the tiles of 16 tokens that hold a visible key: all of them, or from the first token's window on
    n_tiles, first = -(-s["max_len"] // 16), torch.zeros_like(lens)
    if s["window"] >= 0:
        first = (ctx - s["window"]).clamp(min=0) // 16
        n_tiles = min(n_tiles, (s["window"] + T + 15) // 16 + 1)
    tile = first[:, None] + torch.arange(n_tiles, device=dev)[None, :]
    held = torch.gather(s["table"].long(), 1, (tile * 16 // page).clamp(max=s["table"].shape[1] - 1)).clamp(min=0)
    k, v = (x.reshape(B, Hkv, -1, d) for x in _values(s["cache"][held, :, tile % (page // 16)].transpose(1, 2)))
    j = (tile[:, :, None] * 16 + torch.arange(16, device=dev)).flatten(1)         # [B, keys]
    drafted = (j - ctx[:, None]).clamp(0, T - 1)
    mine = torch.gather(up, 2, drafted[:, None, :].expand(-1, T, -1)) & (j < lens[:, None])[:, None]
    shown = torch.where((j < ctx[:, None])[:, None], real[:, :, None], mine)      # [B, T, keys]
    if s["window"] >= 0:
        where = torch.where(j < ctx[:, None], j, torch.gather(pos2, 1, drafted))
        shown = shown & (pos2[:, :, None] - where[:, None, :] <= s["window"])
    shown = shown.repeat_interleave(Hq // Hkv, 1)[:, None]                       # [B, 1, rows, keys]
    z = (q @ k.transpose(-1, -2) / math.sqrt(d)).masked_fill(~shown, -math.inf)
    top = z.amax(-1, keepdim=True)
    e = (z - top.clamp(min=-1e30)).exp()
    total = e.sum(-1, keepdim=True)
    o2 = ((e @ v) / torch.where(total > 0, total, 1.0)).view(B, Hkv, T, -1, d).transpose(1, 2).reshape(B, T, Hq, d)
    lse2 = (top + total.log())[..., 0].view(B, Hkv, T, -1).transpose(1, 2).reshape(B, T, Hq)
    o = torch.zeros_like(s["q"])
    lse = torch.full((n_rows, Hq), -math.inf, device=dev)
    o[flat[real]], lse[flat[real]] = o2[real].to(o.dtype), lse2[real]
    return {"pos": pos.int(), "seen": seen, "o": o, "lse": lse}


def _move_plain(s):
    cache, page, d = s["cache"], s["page"], s["d"]
    on = s["src"] >= 0
    a, b = s["src"][on], s["dst"][on]

    def parts(c):  # views of a cache whose index 3 (values: 3 and 7) is the token's
        n, H, R = c.shape[:3]
        return (c[..., :8 * d].view(n, H, R, 16, d // 2), c[..., 8 * d:16 * d].view(n, H, R, 8, d // 4, 2, 2),
                c[..., 16 * d:].view(n, H, R, 2, 16, d // 16))
    k, v, sc = parts(cache)
    ap, at, ao, bp, bt, bo = a // page, a % page // 16, a % 16, b // page, b % page // 16, b % 16
    kk, vv, ss = k[ap, :, at, ao], v[ap, :, at, ao // 2, :, ao % 2], sc[ap, :, at, :, ao]
    k[bp, :, bt, bo] = kk
    v[bp, :, bt, bo // 2, :, bo % 2] = vv
    sc[bp, :, bt, :, bo] = ss
    p = s["dst"].clamp(min=0)
    keys, values = _values(cache[p // page, :, p % page // 16])                  # [B, T, Hkv, 16, d]
    take = (p % 16)[:, :, None, None, None].expand(-1, -1, cache.shape[1], 1, d)
    hide = (s["dst"] < 0)[:, :, None, None]
    return {x: torch.gather(y, 3, take)[..., 0, :].masked_fill(hide, 0.0).bfloat16() for x, y in (("k", keys), ("v", values))}


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    s, op = state, state["op"]
    if not own:
        return {"norm": _norm_plain, "back": _back_plain, "linear": _linear_plain, "tree": _tree_plain, "move": _move_plain}[op](s)
    import sliding_window_gqa_qk_gb300 as swa
    if op == "norm":
        r = swa.rms_norm(s["x"], s["g"], add=s["r"], eps=EPS, fp8=s["fp8"])
        out = {"h": r["h"], "rstd": r["rstd"]}
        if s["fp8"]:
            out["scale"] = r["scale"]
            out["y"] = r["y"].float() * r["scale"][:, None]
        else:
            out["y"] = r["y"]
        return out
    if op == "back":
        r = swa.rms_norm_backward(s["x"], s["rstd"], s["dy"], s["g"], dh=s["gh"])
        return {"dx": r["dx"], "dgain": r["dgain"]}
    if op == "linear":
        return {"y": swa.w4_linear(s["x"], s["w"], out_features=s["N"], scale=s["scale"], add=s["r"], dtype=TYPES[s["type"]])}
    if op == "tree":
        if "workspace" not in s:  # kept for the life of the program
            s["workspace"] = swa.new_kv4_workspace(s["cache"], s["B"], s["Hq"], max_pages=s["table"].shape[1], window=s["window"])
        pos, seen = swa.kv4_tree(s["parent"], s["cu"], s["lens"], max_new=s["max_new"])
        o, lse = swa.kv4_tree_attention(s["cache"], s["q"], s["table"], s["lens"], s["cu"], pos, seen, max_new=s["max_new"],
                                        rope=s["tables"], interleaved=s["interleaved"], gq=s["gq"], window=s["window"], eps=EPS,
                                        workspace=s["workspace"])
        return {"pos": pos, "seen": seen, "o": o, "lse": lse}
    swa.kv4_move(s["cache"], s["src"], s["dst"])
    k, v = swa.kv4_read(s["cache"], s["dst"])
    return {"k": k, "v": v}


def work(case):
    op = case["op"]
    if op in ("norm", "back"):
        es = 2 if case["type"] == "bf16" else 4
        n, gain = case["rows"] * case["C"], 4 * case["C"]
        if op == "norm":
            y = n + 4 * case["rows"] if case["fp8"] else n * es
            return {"bytes": n * es * (3 if case["add"] else 1) + y + 4 * case["rows"] + (gain if case["gain"] else 0), "flops": 5 * n}
        return {"bytes": n * es * (4 if case["dh"] else 3) + 4 * case["rows"] + gain * (2 if case["gain"] else 1), "flops": 10 * n}
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        es = 2 if case["type"] == "bf16" else 4
        w = N * (K / 2 + 2 * -(-K // 64))
        x = M * K + 4 * M if case["fp8"] else M * K * es
        return {"bytes": w + x + M * N * es * (2 if case["add"] else 1), "flops": 2 * M * N * K}
    d, Hkv = case["d"], case["Hkv"]
    if op == "move":
        n, rows = sum(min(a, case["T"] - a) for a in _move_sizes(case)), case["B"] * max(_move_sizes(case))
        # each moved token is read, written and read back; the rows go out
        return {"bytes": 3 * n * Hkv * 18 * d / 16 + 4 * rows * Hkv * d + 24 * rows, "flops": 0}
    lens, new = _tree_sizes(case)
    es = 2 if case["type"] == "bf16" else 4
    w = case["window"]
    seen = [n if w < 0 else min(n, w + t) for n, t in zip(lens, new)]
    rows = -(-sum(new) // 8) * 8 * case["Hq"]
    pages = sum(-(-n // case["page"]) for n in seen)
    return {"bytes": sum(seen) * Hkv * 18 * d / 16 + 2 * rows * d * es + 4 * rows + 4 * pages + 28 * sum(new) + 12 * case["B"],
            "flops": 4 * d * case["Hq"] * sum(t * (n - t if w < 0 else min(n - t, w)) for n, t in zip(lens, new))}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def _w64(w, row0, row1, K):
    """Rows row0 .. row1 - 1 of the weights, number by number."""
    rows = torch.arange(row0, row1, device=DEV)[:, None]
    col = torch.arange(K, device=DEV)[None, :]
    lane = 4 * (rows % 8) + col % 64 // 16
    nib = col % 2 * 4 + col % 4 // 2 * 2 + rows % 16 // 8
    byte = lane * 16 + col % 16 // 4 * 4 + nib // 2
    n = (w[rows // 16, col // 64, byte].long() >> (nib % 2 * 4)) & 15
    sc = w[..., 512:].contiguous().view(torch.bfloat16).double()
    return (n - 8).double() * sc[rows // 16, col // 64, 2 * (rows % 8) + rows % 16 // 8]


def _places(d):
    """Byte and shift of a channel in a token's row of keys, and in a pair's row of values (of its even token)."""
    kb, ks, vb, vs = [], [], [], []
    for c in range(d):
        g, x = divmod(c, 64)
        n = (x // 16) * (d // 4) + g * 16 + x % 16
        kb.append(n // 2), ks.append(4 * (n % 2))
        n = ((x // 8) * (d // 64) + g) * 16 + (x % 8 // 4) * 8 + x % 4
        vb.append(n // 2), vs.append(4 * (n % 2))
    return tuple(torch.tensor(t, device=DEV) for t in (kb, ks, vb, vs))


def _held64(cache, page, slot):
    """Keys and values of the cache's slots, [slots, heads, d] in 64 bits."""
    d = cache.shape[-1] // 18
    kb, ks, vb, vs = _places(d)
    t = slot % 16
    rows = cache[slot // page, :, slot % page // 16]
    group = torch.arange(d, device=DEV) // 64
    pairs = rows[..., 16 * d:].contiguous().view(torch.bfloat16).double()

    def take(at, shift, which):
        n = (torch.gather(rows, 2, at[:, None].expand(-1, rows.shape[1], -1)) >> shift.to(torch.uint8)) & 15
        p = ((which * 16 + t)[:, None] * (d // 64) + group) * 2
        p = p[:, None].expand(-1, rows.shape[1], -1)
        return torch.gather(pairs, 2, p) * (n.double() - 8.0) + torch.gather(pairs, 2, p + 1)

    return (take(t[:, None] * (d // 2) + kb, ks, 0), take(8 * d + (t // 2)[:, None] * d + (t % 2)[:, None] * 2 + vb, vs, 1))


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "norm":
        h = s["x"] if s["r"] is None else (s["x"].float() + s["r"].float()).to(s["x"].dtype)   # rounded: what the norm is of
        f = h.double()
        rstd = 1.0 / (f.pow(2).sum(-1) / case["C"] + EPS).sqrt()
        u = f * (1.0 if s["g"] is None else s["g"].double())
        out = {"h": f if s["r"] is None else s["x"].double() + s["r"].double(), "rstd": rstd}
        if not case["fp8"]:
            return {**out, "y": u * rstd[:, None]}
        top = u.abs().max(-1).values
        t = u * 448.0 / torch.where(top > 0, top, 1.0)[:, None]
        # e4m3: eight numbers to a power of two, from 2^-6 on; below that multiples of 2^-9
        _, e = torch.frexp(t.abs().clamp(min=0.015625))
        unit = torch.ldexp(torch.ones_like(t), e - 4)
        out["scale"] = top * rstd / 448.0
        return {**out, "y": torch.round(t / unit) * unit * out["scale"][:, None]}
    if op == "back":
        f, dy = s["x"].double(), s["dy"].double()
        r = s["rstd"].double()[:, None]
        w = dy * (1.0 if s["g"] is None else s["g"].double())
        dx = r * w - f * r.pow(3) * (w * f).sum(-1, keepdim=True) / case["C"]
        return {"dx": dx + (0.0 if s["gh"] is None else s["gh"].double()), "dgain": (dy * f * r).sum(0)}
    if op == "linear":
        x = s["x"].float().double() * (1.0 if s["scale"] is None else s["scale"].double()[:, None])
        y = torch.cat([x @ _w64(s["w"], a, min(a + 1024, case["N"]), case["K"]).T for a in range(0, case["N"], 1024)], 1)
        return {"y": y if s["r"] is None else y + s["r"].double()}
    if op == "move":
        page = case["page"]
        on = s["src"] >= 0
        k, v = (torch.zeros(*s["src"].shape, case["Hkv"], case["d"], device=DEV, dtype=torch.float64) for _ in range(2))
        k[on], v[on] = _held64(s["cache"], page, s["src"][on])
        return {"k": k, "v": v}
    Hq, Hkv, d, page = (case[x] for x in ("Hq", "Hkv", "d", "page"))
    n_rows, half = s["q"].shape[0], case["rot"] // 2
    o = torch.zeros(n_rows, Hq, d, device=DEV, dtype=torch.float64)
    lse = torch.full((n_rows, Hq), -math.inf, device=DEV, dtype=torch.float64)
    lens, new = _tree_sizes(case)
    parent, first = s["parent"].tolist(), 0
    for b, (n, t) in enumerate(zip(lens, new)):
        ctx = n - t
        above, depth = [], []
        for i in range(t):
            p = parent[first + i]
            above.append({i} if p < 0 else above[p] | {i})
            depth.append(0 if p < 0 else depth[p] + 1)
        lo = 0 if case["window"] < 0 else max(0, ctx - case["window"])
        j = torch.arange(lo, n, device=DEV)
        k, v = _held64(s["cache"], page, s["table"][b].long()[j // page] * page + j % page)
        at = torch.tensor(depth, device=DEV) + ctx
        cos, sin = (x.double()[at][:, None] for x in s["tables"])
        x = s["q"][first:first + t].double()
        y = x.clone()
        a, c = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if case["interleaved"] else (slice(0, half), slice(half, 2 * half))
        y[..., a] = x[..., a] * cos + x[..., c] * sin
        y[..., c] = x[..., c] * cos - x[..., a] * sin
        y = y / (y.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt() * s["gq"].double()
        hide = torch.zeros(t, n - lo, dtype=torch.bool, device=DEV)
        for i in range(t):
            hide[i, ctx - lo:] = torch.tensor([x not in above[i] or 0 <= case["window"] < depth[i] - depth[x] for x in range(t)], device=DEV)
        if case["window"] >= 0:
            hide[:, :ctx - lo] |= at[:, None] - j[None, :ctx - lo] > case["window"]
        for h in range(Hkv):
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            z = torch.einsum("tgd,kd->tgk", y[:, heads], k[:, h]) / math.sqrt(d)
            z = z.masked_fill(hide[:, None], -math.inf)
            lse[first:first + t, heads] = torch.logsumexp(z, -1)
            o[first:first + t, heads] = torch.softmax(z, -1) @ v[:, h]
        first += t
    return {"pos": None, "seen": None, "o": o, "lse": lse}
