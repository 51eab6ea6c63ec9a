"""The operators of the decode path, and of rotary positions, as they are measured.

Each case names one operator ("op") and its sizes. `run` with `own` false
computes it in elementary torch operations; with `own` true it makes the calls
a user of the library makes. The operators:

  tables  cosine / sine tables of rotary positions, scaled for long contexts
  rope    the rotation of a layer's q and k by such tables (and its transpose,
          the backward), in the split-half or the interleaved layout, of the
          whole head or its first channels
  plan    pages, slots and positions of a serving step from request lengths
  append  new keys (rotated and normed) and values (with their value
          embedding) quantised into the 4-bit paged cache, and read back
  attend  attention of one new token per request over that cache

The cache is uint8 [pages, kv heads, page / 16, 18 d]: per 16 tokens of one kv
head 8 d bytes of keys, 8 d bytes of values, and one bf16 pair (s, z) per
token and group of 64 channels for each. A value is s (n - 8) + z.
  keys    nibble x = 64-channel group g, j = 0..3, i = 0..15 of a token's row
          is at row position (j, g, i), low nibble first; token by token
  values  token pair by token pair: (r = 0..7, g, u = 0..1, token of the pair,
          i = 0..3) holds channel 64 g + 8 r + 4 u + i
"""

import math
import random

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6
VE_SCALE = 0.5
VOCAB = 8192
BASE = 10000.0


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # a training script's tables: ten times its sequence of 2048
        {"name": "tables_script", "op": "tables", "first": 0, "rows": 20480, "rot": 128, "scaling": "none", "factor": 1.0},
        # a context of 16384 stretched sixteenfold, low frequencies only
        {"name": "tables_far", "op": "tables", "first": 0, "rows": 262144, "rot": 128, "scaling": "by_parts", "factor": 16.0},
        # q and k of one layer of the benchmark's stack, forward
        {"name": "rope_layer", "op": "rope", "B": 16, "T": 2048, "Hq": 6, "Hkv": 3, "d": 128, "rot": 128,
         "interleaved": False, "inverse": False, "given": False, "type": "bf16"},
        # gradients of q and k of a long-context layer: half the head turned, pairs side by side, packed positions
        {"name": "rope_back_long", "op": "rope", "B": 2, "T": 16384, "Hq": 16, "Hkv": 4, "d": 128, "rot": 64,
         "interleaved": True, "inverse": True, "given": True, "type": "fp32"},
        # one token for each of a batch's requests
        {"name": "plan_step", "op": "plan", "B": 64, "page": 64, "max_pages": 256, "new": 1, "short": False},
        # a large batch of prompts and continuations, with too few pages for the last of them
        {"name": "plan_mixed", "op": "plan", "B": 1000, "page": 32, "max_pages": 512, "new": 700, "short": True},
        # one token for each of a batch's requests, on a layer with value embeddings
        {"name": "append_step", "op": "append", "B": 64, "T": 1, "Hkv": 3, "d": 128, "page": 64, "rot": 128,
         "interleaved": False, "ve": True},
        # eight prompts of the training length
        {"name": "append_prompt", "op": "append", "B": 8, "T": 2048, "Hkv": 3, "d": 128, "page": 64, "rot": 128,
         "interleaved": False, "ve": False},
        # one request of the small model: latency
        {"name": "attend_tiny", "op": "attend", "B": 1, "Hq": 2, "Hkv": 1, "d": 64, "page": 16, "max_len": 256,
         "window": 128, "even": True, "rot": 64, "interleaved": False, "type": "bf16"},
        # a batch on a sliding-window layer, requests of all lengths
        {"name": "attend_window", "op": "attend", "B": 64, "Hq": 6, "Hkv": 3, "d": 128, "page": 64, "max_len": 16384,
         "window": 1024, "even": False, "rot": 128, "interleaved": False, "type": "bf16"},
        # a batch of long contexts on a full layer, four query heads to a kv head
        {"name": "attend_long", "op": "attend", "B": 32, "Hq": 16, "Hkv": 4, "d": 128, "page": 64, "max_len": 65536,
         "window": -1, "even": True, "rot": 128, "interleaved": False, "type": "bf16"},
        # plain multi-head attention in 32 bits, ragged, small pages
        {"name": "attend_fp32", "op": "attend", "B": 16, "Hq": 6, "Hkv": 6, "d": 128, "page": 16, "max_len": 5000,
         "window": -1, "even": False, "rot": 32, "interleaved": True, "type": "fp32"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["tables", "rope", "plan", "append", "append", "attend", "attend", "attend"])
    d = rng.choice([64, 128, 128])
    rot = rng.choice([16 * rng.randint(1, d // 16), d])
    inter = rng.random() < 0.5
    if op == "tables":
        scaling = rng.choice(["none", "linear", "ntk", "by_parts"])
        return {"op": op, "first": rng.choice([0, rng.randint(1, 1 << 21)]), "rows": _log(rng, 1, 262144),
                "rot": 16 * rng.randint(1, 8), "scaling": scaling,
                "factor": 1.0 if scaling == "none" else round(rng.uniform(1.5, 32.0), 2)}
    if op == "plan":
        B = _log(rng, 1, 1000)
        page = 16 * rng.choice([1, 2, 3, 4, 8])
        return {"op": op, "B": B, "page": page, "max_pages": rng.randint(8192 // page, 16384 // page),
                "new": rng.choice([1, _log(rng, 2, 700)]), "short": rng.random() < 0.3}
    if op == "rope":
        Hkv = rng.randint(1, 4)
        Hq = Hkv * rng.randint(1, 4)
        T = _log(rng, 1, 16384)
        return {"op": op, "B": rng.randint(1, max(1, min(16, 600000 // (T * (Hq + Hkv))))), "T": T, "Hq": Hq, "Hkv": Hkv,
                "d": d, "rot": rot, "interleaved": inter, "inverse": rng.random() < 0.5, "given": rng.random() < 0.5,
                "type": rng.choice(["bf16", "fp32"])}
    page = 16 * rng.choice([1, 2, 3, 4, 8])
    if op == "append":
        T = rng.choice([1, _log(rng, 2, 2048)])
        return {"op": op, "B": _log(rng, 1, 256) if T == 1 else rng.randint(1, max(1, 16384 // T)) if T > 128 else rng.randint(1, 64),
                "T": T, "Hkv": rng.randint(1, 4 if T * 64 > 16384 else 6), "d": d, "page": page, "rot": rot, "interleaved": inter,
                "ve": rng.random() < 0.5}
    G = rng.choice([1, 2, 3, 4, 4, 6, 8])
    Hkv = rng.randint(1, 4)
    max_len = _log(rng, 1, 65536)
    most = max(1, min(256, 4000000 // (max_len * Hkv)))
    return {"op": op, "B": _log(rng, 1, most), "Hq": G * Hkv, "Hkv": Hkv, "d": d, "page": page, "max_len": max_len,
            "window": rng.choice([-1, -1, _log(rng, 1, 8192)]), "even": rng.random() < 0.3, "rot": rot, "interleaved": inter,
            "type": rng.choice(["bf16", "bf16", "bf16", "fp32"])}


def _fixed(case):
    """Lengths are part of the case, not of the seed: a pass always has the same work."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _plan_sizes(case):
    r, cap = _fixed(case), case["page"] * case["max_pages"]
    new = [1 if case["new"] == 1 else min(_log(r, 1, case["new"]), cap // 2) for _ in range(case["B"])]
    lens = [0 if r.random() < 0.2 and case["new"] > 1 else r.randint(1, cap - n) for n in new]
    return lens, new


def _attend_sizes(case):
    r, top = _fixed(case), case["max_len"]
    lens = [r.randint(max(1, top - top // 8), top) if case["even"] else _log(r, 1, top) for _ in range(case["B"])]
    lens[r.randrange(case["B"])] = top
    return lens


def _visible(case):
    w = case["window"]
    return [n if w < 0 else min(n, w + 1) for n in _attend_sizes(case)]


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


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case)
    if op == "tables":
        # the base is the input of the call: another seed, another base
        s["base"] = BASE * (1.0 + (seed % 997) / 997.0)
        return s

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    if op == "rope":
        t = TYPES[case["type"]]
        B, T, d = case["B"], case["T"], case["d"]
        s["q"], s["k"] = randn(B, T, case["Hq"], d).to(t), randn(B, T, case["Hkv"], d).to(t)
        s["tables"] = _tables(max(T, 2048), case["rot"])
        s["pos"] = None
        if case["given"]:  # documents packed into the rows: positions begin again
            start = torch.randint(1, T + 1, (B, 1), generator=g, device=DEV)
            at = torch.arange(T, device=DEV)[None, :]
            s["pos"] = torch.where(at < start, at, at - start).int()
        return s
    if op == "plan":
        lens, new = _plan_sizes(case)
        B, page, cap = case["B"], case["page"], case["max_pages"]
        held = [-(-n // page) for n in lens]
        want = sum(-(-(n + m) // page) - h for n, m, h in zip(lens, new, held))
        n_pages = sum(held) + want + 16
        ids = torch.randperm(n_pages, generator=g, device=DEV).int()
        held_t, at = torch.tensor(held, device=DEV), torch.arange(cap, device=DEV)[None, :]
        used = at < held_t[:, None]
        begin = torch.cumsum(held_t, 0) - held_t
        s["table"] = torch.where(used, ids[(begin[:, None] + at).clamp(max=n_pages - 1)], -1).int()
        head = 5
        s["free"] = torch.cat([ids[:head], ids[sum(held):sum(held) + (want * 3 // 4 if case["short"] else want + 11)]]).contiguous()
        s["head"] = torch.tensor([head], dtype=torch.int32, device=DEV)
        s["n_pages"] = n_pages
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["fresh"] = torch.tensor(new, dtype=torch.int32, device=DEV)
        s["n_tokens"] = -(-sum(new) // 64) * 64  # a step's token buffer is padded
        return s
    d, Hkv, page = case["d"], case["Hkv"], case["page"]
    if op == "append":
        B, T = case["B"], case["T"]
        s["k"], s["v"] = randn(B, T, Hkv, d).to(torch.bfloat16), randn(B, T, Hkv, d).to(torch.bfloat16)
        s["gk"] = 1.0 + 0.1 * randn(d)
        rows = T + 64
        s["tables"] = _tables(rows, case["rot"])
        first = torch.randint(0, 64, (B, 1), generator=g, device=DEV)
        s["pos"] = (first + torch.arange(T, device=DEV)[None, :]).int()
        per = -(-(T + 63) // page)
        pages = torch.randperm(B * per + 3, generator=g, device=DEV)[:B * per].view(B, per)
        at = s["pos"].long()
        s["slot"] = torch.gather(pages, 1, at // page) * page + at % page
        s["cache"] = torch.randint(0, 256, (B * per + 3, Hkv, page // 16, 18 * d), generator=g, device=DEV, dtype=torch.uint8)
        if case["ve"]:
            s["table"] = (0.02 * randn(VOCAB, Hkv * d)).to(torch.bfloat16)
            s["tok"] = torch.randint(0, VOCAB, (B, T), generator=g, device=DEV).int()
            s["gate"] = 2.0 * torch.sigmoid(randn(B, T, Hkv))
        return s
    lens, t = _attend_sizes(case), TYPES[case["type"]]
    B, cap = case["B"], -(-case["max_len"] // page) + 2
    held = [-(-n // page) for n in lens]
    n_pages = sum(held) + 1
    s["q"] = randn(B, case["Hq"], d).to(t)
    s["gq"] = 1.0 + 0.1 * randn(d)
    s["tables"] = _tables(case["max_len"], case["rot"])
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    held_t, at = torch.tensor(held, device=DEV), torch.arange(cap, device=DEV)[None, :]
    ids = torch.randperm(n_pages, generator=g, device=DEV)
    begin = torch.cumsum(held_t, 0) - held_t
    s["table"] = torch.where(at < held_t[:, None], ids[(begin[:, None] + at).clamp(max=n_pages - 1)], -1).int()
    s["cache"] = torch.randint(0, 256, (n_pages, Hkv, page // 16, 18 * d), generator=g, device=DEV, dtype=torch.uint8)
    pairs = s["cache"][..., 16 * d:].view(torch.bfloat16)  # (s, z): steps near 0.2, centres near 0
    shape = pairs[..., 0::2].shape
    pairs[..., 0::2] = (0.2 + 0.05 * torch.rand(shape, generator=g, device=DEV)).bfloat16()
    pairs[..., 1::2] = (0.1 + 0.1 * torch.randn(shape, generator=g, device=DEV)).bfloat16()
    return s


# ---------------------------------------------------------------------------
# The plain form
# ---------------------------------------------------------------------------

def _freqs(s, dev):
    """Angle per position of each pair of channels, in 64 bits."""
    rot, base, f = s["rot"], s["base"], s["factor"]
    c = torch.arange(rot // 2, device=dev, dtype=torch.float64)
    if s["scaling"] == "ntk" and rot > 2:
        base = base * f ** (rot / (rot - 2.0))
    theta = base ** (-2.0 * c / rot)
    if s["scaling"] == "linear":
        theta = theta / f
    if s["scaling"] == "by_parts":  # turns made over the original context decide: all kept, all stretched, or between
        turns = 16384 * theta / (2.0 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        theta = theta * keep + theta / f * (1.0 - keep)
    return theta


def _turn(x, cos, sin, interleaved, sign=1.0):
    """x [..., d] turned; cos, sin broadcast over x's pairs."""
    half = cos.shape[-1]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * cos + sign * b * sin, b * cos - sign * a * sin
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half], y[..., half:2 * half] = a * cos + sign * b * sin, b * cos - sign * a * sin
    return y


def _norm(x, gain):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gain


def _plan_plain(s):
    page, cap, n = s["page"], s["max_pages"], s["n_tokens"]
    lens, new, free, head = s["lens"].long(), s["fresh"].long(), s["free"].long(), s["head"].long()
    held = (lens + page - 1) // page
    want = (lens + new + page - 1) // page - held
    off = torch.cumsum(want, 0) - want
    fits = (want == 0) | (head + off + want <= free.numel())
    at = torch.arange(cap, device=lens.device)[None, :]
    mine = (at >= held[:, None]) & (at < (held + want)[:, None]) & fits[:, None]
    pick = (head + off)[:, None] + at - held[:, None]
    table = torch.where(mine, free[pick.clamp(0, free.numel() - 1)].int(), s["table"])
    cu = torch.zeros(lens.numel() + 1, dtype=torch.int64, device=lens.device)
    cu[1:] = torch.cumsum(new, 0)
    i = torch.arange(n, device=lens.device)
    row = torch.searchsorted(cu[1:].contiguous(), i, right=True)
    real = i < cu[-1]
    r = row.clamp(max=lens.numel() - 1)
    pos = lens[r] + i - cu[r]
    slot = table.long()[r, (pos // page).clamp(0, cap - 1)] * page + pos % page
    slot = torch.where(real & fits[r], slot, -1)
    s["table"].copy_(table)
    return {"table": s["table"], "slot": slot, "pos": torch.where(real, pos, 0).int(), "row": torch.where(real, r, -1).int(),
            "cu": cu.int(), "lens": torch.where(fits, lens + new, lens).int(),
            "head": (head + torch.where(fits, want, 0).sum()).int()}


def _codes(x):
    """4-bit codes of [..., d] in 64 bits, and the pairs (s, z) [..., d / 64, 2]."""
    g = x.unflatten(-1, (-1, 64))
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    step = ((hi - lo) / 15.0).bfloat16()
    mid = (lo + 8.0 * step.double()).bfloat16()
    n = torch.floor((g - mid.double()) / step.double() + 8.5).clamp(0, 15)
    n = torch.where(step == 0, 8.0, n)
    return n.to(torch.uint8), torch.cat([step, mid], -1)


def _append_plain(s):
    d, Hkv, page = s["d"], s["Hkv"], s["page"]
    cos, sin = (t[s["pos"].long()][:, :, None].double() for t in s["tables"])
    k = _norm(_turn(s["k"].double(), cos, sin, s["interleaved"]), s["gk"].double()).flatten(0, 1)
    v = s["v"].double()
    if s["ve"]:
        e = s["table"][s["tok"].long()].double().view(v.shape)
        v = v + VE_SCALE * s["gate"].double()[..., None] * e
    v = v.flatten(0, 1)
    N, cache, G = k.shape[0], s["cache"], d // 64
    slot = s["slot"].flatten()
    p, tile, t = slot // page, slot % page // 16, slot % 16
    nk, pk = _codes(k)
    nv, pv = _codes(v)
    # keys: [N, Hkv, G, 4, 16] -> (4, G, 16) and two to a byte
    b = nk.view(N, Hkv, G, 4, 8, 2).transpose(2, 3)
    cache[..., :8 * d].view(*cache.shape[:3], 16, d // 2)[p, :, tile, t] = (b[..., 0] | b[..., 1] << 4).reshape(N, Hkv, d // 2)
    # values: [N, Hkv, G, 8, 2, 4] -> (8, G, 2, 4) and two to a byte, at the token's place in its pair
    b = nv.view(N, Hkv, G, 8, 2, 2, 2).transpose(2, 3)
    cache[..., 8 * d:16 * d].view(*cache.shape[:3], 8, 8, G, 2, 2, 2)[p, :, tile, t // 2, :, :, :, t % 2] = b[..., 0] | b[..., 1] << 4
    pairs = cache[..., 16 * d:].view(torch.bfloat16).view(*cache.shape[:3], 2, 16, G, 2)
    pairs[p, :, tile, 0, t] = pk
    pairs[p, :, tile, 1, t] = pv
    # and back
    kv, vv = _values(cache)
    keys = kv.view(*cache.shape[:3], 16, d)[p, :, tile, t]
    values = vv.view(*cache.shape[:3], 16, d)[p, :, tile, t]
    return {"k": keys.view(s["k"].shape).bfloat16(), "v": values.view(s["k"].shape).bfloat16()}


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


def _attend_plain(s):
    B, Hq, Hkv, d, page = s["B"], s["Hq"], s["Hkv"], s["d"], s["page"]
    lens = s["lens"].long()
    at = (lens - 1).clamp(min=0)
    cos, sin = (t[at][:, None] for t in s["tables"])
    q = _norm(_turn(s["q"].float(), cos, sin, s["interleaved"]), s["gq"]).view(B, Hkv, Hq // Hkv, d)
    # the tiles of 16 tokens that hold a visible key: all of them, or those of the window
    n_tiles = -(-s["max_len"] // 16)
    first = torch.zeros_like(lens)
    if s["window"] >= 0:
        first = (lens - 1 - s["window"]).clamp(min=0) // 16
        n_tiles = min(n_tiles, (s["window"] + 15) // 16 + 1)
    tile = first[:, None] + torch.arange(n_tiles, device=lens.device)[None, :]
    held = torch.gather(s["table"].long(), 1, (tile * 16 // page).clamp(max=s["table"].shape[1] - 1)).clamp(min=0)
    tiles = s["cache"][held, :, tile % (page // 16)].transpose(1, 2)  # [B, Hkv, tiles, 18 d]
    k, v = (x.reshape(B, Hkv, -1, d) for x in _values(tiles))
    z = q @ k.transpose(-1, -2) / math.sqrt(d)
    j = (tile[:, :, None] * 16 + torch.arange(16, device=lens.device)).flatten(1)
    seen = j < lens[:, None]
    if s["window"] >= 0:
        seen = seen & (j >= lens[:, None] - 1 - s["window"])
    z = z.masked_fill(~seen[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    e = (z - top).exp()
    total = e.sum(-1, keepdim=True)
    o = (e / total) @ v
    return {"o": o.reshape(B, Hq, d).to(s["q"].dtype), "lse": (top + total.log()).reshape(B, Hq)}


def _plain(s):
    op = s["op"]
    if op == "tables":
        at = s["first"] + torch.arange(s["rows"], device=DEV, dtype=torch.float64)
        ang = at[:, None] * _freqs(s, DEV)
        return {"cos": ang.cos().float(), "sin": ang.sin().float()}
    if op == "rope":
        cos, sin = s["tables"]
        if s["pos"] is None:
            cos, sin = cos[None, :s["T"], None], sin[None, :s["T"], None]
        else:
            cos, sin = cos[s["pos"].long()][:, :, None], sin[s["pos"].long()][:, :, None]
        sign = -1.0 if s["inverse"] else 1.0
        return {x: _turn(s[x].float(), cos, sin, s["interleaved"], sign).to(s[x].dtype) for x in ("q", "k")}
    return {"plan": _plan_plain, "append": _append_plain, "attend": _attend_plain}[op](s)


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    if not own:
        return _plain(state)
    import sliding_window_gqa_qk_gb300 as swa
    s, op = state, state["op"]
    if op == "tables":
        cos, sin = swa.rope_tables(s["rows"], s["rot"], base=s["base"], scaling=s["scaling"], factor=s["factor"],
                                   orig_len=16384, first=s["first"])
        return {"cos": cos, "sin": sin}
    if op == "rope":
        q, k = swa.rope_apply(s["q"], s["k"], s["tables"], pos=s["pos"], interleaved=s["interleaved"], inverse=s["inverse"])
        return {"q": q, "k": k}
    if op == "plan":
        p = swa.kv4_plan(s["lens"], s["fresh"], s["table"], s["free"], s["head"], page=s["page"], n_pages=s["n_pages"],
                         n_tokens=s["n_tokens"])
        return {"table": s["table"], "slot": p["slot"], "pos": p["pos"], "row": p["row"], "cu": p["cu"], "lens": p["lens"],
                "head": p["free_head"]}
    if op == "append":
        more = dict(ve=s["table"], tok=s["tok"], ve_gate=s["gate"], ve_scale=VE_SCALE) if s["ve"] else {}
        swa.kv4_append(s["cache"], s["k"], s["v"], s["slot"], pos=s["pos"], rope=s["tables"], interleaved=s["interleaved"],
                       gk=s["gk"], eps=EPS, **more)
        k, v = swa.kv4_read(s["cache"], s["slot"])
        return {"k": k, "v": v}
    if "workspace" not in s:  # kept for the life of the program
        s["workspace"] = swa.new_kv4_workspace(s["cache"], s["B"], s["Hq"], max_pages=s["table"].shape[1], window=s["window"])
    o, lse = swa.kv4_attention(s["cache"], s["q"], s["table"], s["lens"], rope=s["tables"], interleaved=s["interleaved"],
                               gq=s["gq"], window=s["window"], eps=EPS, workspace=s["workspace"])
    return {"o": o, "lse": lse}


def work(case):
    op = case["op"]
    if op == "tables":
        n = case["rows"] * case["rot"] / 2
        return {"bytes": 8 * n, "flops": 4 * n}
    if op == "rope":
        es = 2 if case["type"] == "bf16" else 4
        rows = case["B"] * case["T"]
        n = rows * (case["Hq"] + case["Hkv"])
        angles = 4 * case["rot"] * (min(rows, max(case["T"], 2048)) if case["given"] else case["T"])
        return {"bytes": 2 * n * case["d"] * es + angles + (4 * rows if case["given"] else 0), "flops": 3 * n * case["rot"]}
    if op == "plan":
        lens, new = _plan_sizes(case)
        page, B, n = case["page"], case["B"], sum(new)
        fresh = sum(-(-(a + b) // page) - -(-a // page) for a, b in zip(lens, new))
        return {"bytes": 8 * B + 8 * fresh + 16 * (-(-n // 64) * 64) + 8 * B + 4 * sum(1 for a in lens if a % page), "flops": 8 * n}
    if op == "append":
        rows, d = case["B"] * case["T"], case["d"]
        n = rows * case["Hkv"]
        held = n * 18 * d / 16
        ve = n * (2 * d + 4) + 4 * rows if case["ve"] else 0
        return {"bytes": 4 * n * d + ve + held + held + 4 * n * d + 12 * rows + 4 * d, "flops": 30 * n * d}
    seen, d = sum(_visible(case)), case["d"]
    es = 2 if case["type"] == "bf16" else 4
    pages = sum(-(-n // case["page"]) for n in _visible(case))
    rows = case["B"] * case["Hq"]
    return {"bytes": seen * case["Hkv"] * 18 * d / 16 + 2 * rows * d * es + 4 * rows + 4 * pages + 4 * case["B"],
            "flops": 4 * seen * case["Hq"] * d}


# ---------------------------------------------------------------------------
# The definition in 64 bits, channel by channel
# ---------------------------------------------------------------------------

def _partner(d, rot, interleaved):
    """For each channel: its partner, its column of the tables, and the sign of the partner's sine."""
    c = list(range(d))
    if interleaved:
        to, col, sg = [x ^ 1 for x in c], [x // 2 for x in c], [1.0 if x % 2 == 0 else -1.0 for x in c]
    else:
        h = rot // 2
        to, col, sg = [(x + h) % rot for x in c], [x % h for x in c], [1.0 if x < h else -1.0 for x in c]
    to = [t if x < rot else x for x, t in zip(c, to)]
    col = [t if x < rot else 0 for x, t in zip(c, col)]
    return (torch.tensor(to, device=DEV), torch.tensor(col, device=DEV), torch.tensor(sg, device=DEV, dtype=torch.float64),
            torch.tensor([x < rot for x in c], device=DEV))


def _turn64(x, cos, sin, interleaved, inverse=False):
    """x [rows, heads, d] by tables [rows, rot / 2]."""
    rot = 2 * cos.shape[1]
    to, col, sg, on = _partner(x.shape[-1], rot, interleaved)
    c = torch.where(on, cos.double()[:, col], 1.0)[:, None]
    n = torch.where(on, sin.double()[:, col] * sg, 0.0)[:, None]
    x = x.double()
    return x * c + (-1.0 if inverse else 1.0) * x[..., to] * n


def _rms64(x, gain):
    return x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * gain.double()


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


def _nearest64(x):
    """The value each channel is held as: steps and centres are bf16."""
    y = torch.empty_like(x)
    for g in range(x.shape[-1] // 64):
        c = x[..., 64 * g:64 * g + 64]
        lo = c.min(-1, keepdim=True).values
        s = ((c.max(-1, keepdim=True).values - lo) / 15).to(torch.bfloat16).double()
        z = (lo + 8 * s).to(torch.bfloat16).double()
        n = ((c - z) / s + 0.5).floor().clamp(-8, 7)
        y[..., 64 * g:64 * g + 64] = torch.where(s > 0, z + s * n, z)
    return y


def exact(case, seed):
    op = case["op"]
    if op == "plan":
        return None
    s = prepare(case, seed)
    if op == "tables":
        half = case["rot"] // 2
        at = torch.arange(case["first"], case["first"] + case["rows"], device=DEV, dtype=torch.float64)
        cos, sin = (torch.empty(case["rows"], half, device=DEV, dtype=torch.float64) for _ in range(2))
        for c in range(half):
            base = s["base"]
            if case["scaling"] == "ntk":
                base *= case["factor"] ** (case["rot"] / (case["rot"] - 2.0))
            w = math.exp(-2.0 * c / case["rot"] * math.log(base))
            if case["scaling"] == "linear":
                w /= case["factor"]
            if case["scaling"] == "by_parts":
                keep = min(1.0, max(0.0, (16384 * w / (2.0 * math.pi) - 1.0) / 31.0))
                w = keep * w + (1.0 - keep) * w / case["factor"]
            cos[:, c], sin[:, c] = torch.cos(at * w), torch.sin(at * w)
        return {"cos": cos, "sin": sin}
    if op == "rope":
        at = (torch.arange(case["T"], device=DEV).repeat(case["B"]) if s["pos"] is None else s["pos"].flatten()).long()
        return {x: _turn64(s[x].flatten(0, 1), s["tables"][0][at], s["tables"][1][at], case["interleaved"],
                           case["inverse"]).view(s[x].shape) for x in ("q", "k")}
    if op == "append":
        at = s["pos"].flatten().long()
        k = _turn64(s["k"].flatten(0, 1), s["tables"][0][at], s["tables"][1][at], case["interleaved"])
        v = s["v"].flatten(0, 1).double()
        if case["ve"]:
            v = v + VE_SCALE * s["gate"].double().flatten(0, 1)[..., None] * s["table"].double()[s["tok"].flatten().long()].view(v.shape)
        return {"k": _nearest64(_rms64(k, s["gk"])).view(s["k"].shape), "v": _nearest64(v).view(s["v"].shape)}
    B, Hq, Hkv, d, page = (case[x] for x in ("B", "Hq", "Hkv", "d", "page"))
    o = torch.empty(B, Hq, d, device=DEV, dtype=torch.float64)
    lse = torch.empty(B, Hq, device=DEV, dtype=torch.float64)
    for b, n in enumerate(_attend_sizes(case)):
        j = torch.arange(0 if case["window"] < 0 else max(0, n - 1 - case["window"]), n, device=DEV)
        k, v = _held64(s["cache"], page, s["table"][b].long()[j // page] * page + j % page)
        at = torch.tensor([n - 1], device=DEV)
        q = _rms64(_turn64(s["q"][b:b + 1], s["tables"][0][at], s["tables"][1][at], case["interleaved"]), s["gq"])[0]
        for h in range(Hkv):
            rows = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            z = q[rows] @ k[:, h].T / math.sqrt(d)
            lse[b, rows] = torch.logsumexp(z, -1)
            o[b, rows] = torch.softmax(z, -1) @ v[:, h]
    return {"o": o, "lse": lse}
