"""The serving calls as they are used together: the block call against its parts
and the float64 oracle, drafted steps with acceptance and moves against plain
decoding, captured and replayed steps, streams, the binding's short way, and
where the tree attention's ranges end.

Bounds: as in test_serve_gpu.py. The block call makes the same launches as its
parts, so it gives their bits. Against the oracle (keys and values read back
from the cache, so that the quantiser's borders play no part) a bf16 block rounds
xn, q, o (half a step each, 2^-8) and P (2^-8) on the way, and weights in calls of
more than 32 tokens: the attention's part of out is held to 2 % in the 2-norm,
which a missing or misplaced row exceeds by far; an fp32 one to 1e-4."""

import numpy as np
import pytest
import torch

import sliding_window_gqa_qk_gb300 as swa
from oracle import decode as dec
from oracle import serve
from test_decode_gpu import build_cache, f64, randn
from test_serve_gpu import DT, KINDS, dev, i32, random_parents, random_w4, tree_case

pytestmark = pytest.mark.gpu


def step_case(kind, B, new, old, Hq, Hkv, d, C, page=32, seed=1, ve=False):
    """A cache with `old` tokens per request, a plan for `new` more, and a block's inputs and weights."""
    max_pages = max(-(-(o + n) // page) for o, n in zip(old, new)) + 1
    n_pages = B * max_pages + 2
    cache = swa.new_kv4_cache(n_pages, page, Hkv, d, dev())
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device=dev())
    free = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).int().to(dev())
    rope = swa.rope_tables(max_pages * page, d)
    gk = (1 + 0.1 * randn(seed + 1, d)).to(dev())
    plan = swa.kv4_plan(i32(*([0] * B)), i32(*old), table, free, i32(0), page=page, n_pages=n_pages, n_tokens=sum(old))
    n = sum(old)
    if n:
        k, v = (randn(seed + 2 + i, n, 1, Hkv, d, dtype=DT[kind]).to(dev()) for i in range(2))
        swa.kv4_append(cache, k, v, plan["slot"].view(n, 1), pos=plan["pos"].view(n, 1), rope=rope, gk=gk)
    pad = -(-sum(new) // 8) * 8
    plan = swa.kv4_plan(plan["lens"], i32(*new), table, free, plan["free_head"], page=page, n_pages=n_pages, n_tokens=pad)
    s = dict(cache=cache, table=table, plan=plan, rope=rope, gk=gk, gq=(1 + 0.1 * randn(seed + 4, d)).to(dev()), pad=pad, Hq=Hq, C=C,
             gain=(1 + 0.1 * randn(seed + 5, C)).to(dev()), x=randn(seed + 6, pad, C, dtype=DT[kind]).to(dev()),
             add=randn(seed + 7, pad, C, dtype=DT[kind]).to(dev()))
    s["w"] = [random_w4(seed + 8 + i, N, K) for i, (N, K) in enumerate(((Hq * d, C), (Hkv * d, C), (Hkv * d, C), (C, Hq * d)))]
    for w, K in zip(s["w"], (C, C, C, Hq * d)):      # a size that keeps activations near 1
        w[..., 512:].view(torch.bfloat16).mul_(2.0 / K ** 0.5)
    s["wd"] = [w.to(dev()) for w in s["w"]]
    if ve:
        s["ve"] = (0.05 * randn(seed + 20, 64, Hkv * d)).to(DT[kind]).to(dev())
        s["tok"] = torch.randint(0, 64, (pad,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32).to(dev())
        s["gate_w"] = (0.3 * randn(seed + 21, Hkv, 16)).to(dev())
    return s


def parts(s, cache, kind, tree, window, pos, cu=None, seen=None, max_new=1, ws=None, add=True):
    """The block by its parts."""
    n, d, Hkv = s["x"].shape[0], cache.shape[-1] // 18, cache.shape[1]
    r = swa.rms_norm(s["x"], s["gain"], add=s["add"] if add else None)
    q, k, v = (swa.w4_linear(r["y"], w, out_features=N).view(n, 1, N // d, d) for w, N in zip(s["wd"], (s["Hq"] * d, Hkv * d, Hkv * d)))
    more = {}
    if "ve" in s:
        more = dict(ve=s["ve"], tok=s["tok"].view(n, 1), gate_x=r["y"].view(n, 1, -1), gate_w=s["gate_w"])
    swa.kv4_append(cache, k, v, s["plan"]["slot"].view(n, 1), pos=pos.view(n, 1), rope=s["rope"], gk=s["gk"], workspace=ws, **more)
    kw = dict(rope=s["rope"], gq=s["gq"], window=window, workspace=ws)
    if tree:
        o, _ = swa.kv4_tree_attention(cache, q.view(n, s["Hq"], d), s["table"], s["plan"]["lens"], cu, pos, seen, max_new=max_new, **kw)
    else:
        o, _ = swa.kv4_attention(cache, q.view(n, s["Hq"], d), s["table"], s["plan"]["lens"], **kw)
    return swa.w4_linear(o.view(n, -1), s["wd"][3], out_features=s["C"], add=r["h"])


def oracle_out(s, cache, kind, window, pos, cu, seen, add=True):
    """out [tokens, C] in 64 bits, with the keys and values that the cache holds."""
    d, Hq, C = cache.shape[-1] // 18, s["Hq"], s["C"]
    Hkv, page = cache.shape[1], 16 * cache.shape[2]
    h = s["x"] if not add else (s["x"].float() + s["add"].float()).to(s["x"].dtype)
    xn, _ = serve.norm(f64(h), f64(s["gain"]))
    wq, wo = serve.w4_values(s["w"][0].numpy(), Hq * d, C), serve.w4_values(s["w"][3].numpy(), C, Hq * d)
    q = (xn @ wq.T).reshape(-1, Hq, d)
    o = np.zeros_like(q)
    lens, table = s["plan"]["lens"].tolist(), s["table"].cpu().long()
    cos, sin = (f64(t) for t in s["rope"])
    for b, n in enumerate(lens):
        j = torch.arange(n)
        slot = (table[b, j // page] * page + j % page).view(1, n).to(dev())
        k, v = (f64(t)[0] for t in swa.kv4_read(cache, slot, dtype=torch.float32))
        a, e = cu[b], cu[b + 1]
        o[a:e] = serve.tree_attend(q[a:e], k, v, pos[a:e], seen[a:e], window=window, gq=f64(s["gq"]), cos=cos, sin=sin)[0]
    return f64(h), o.reshape(len(q), -1) @ wo.T


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("ve,window,d,C,Hq,Hkv", [(False, -1, 128, 192, 4, 2), (True, 9, 64, 136, 6, 3), (True, -1, 128, 768, 6, 3)])
@pytest.mark.parametrize("tree", [False, True])
def test_block_is_its_parts_and_the_oracles(kind, ve, window, d, C, Hq, Hkv, tree):
    new = [3, 1, 7, 12, 0, 5] if tree else [1] * 8
    old = [20, 0, 33, 64, 5, 100] if tree else [20, 0, 33, 64, 5, 100, 7, 31]
    B = len(new)
    s = step_case(kind, B, new, old, Hq, Hkv, d, C, ve=ve)
    plan = s["plan"]
    ws = swa.new_kv4_block_workspace(s["cache"], s["pad"], C, Hq, kind=kind)
    cu = plan["cu"]
    kw = dict(rope=s["rope"], gq=s["gq"], gk=s["gk"], gain=s["gain"], window=window, workspace=ws, Hq=Hq)
    if ve:
        kw.update(ve=s["ve"], tok=s["tok"], gate_w=s["gate_w"])
    if tree:
        parent = torch.zeros(s["pad"], dtype=torch.int32)
        at = np.concatenate([[0], np.cumsum(new)])
        for b, n in enumerate(new):
            parent[at[b]:at[b + 1]] = torch.tensor(random_parents(n, b), dtype=torch.int32)
        pos, seen = swa.kv4_tree(parent.to(dev()), cu, plan["lens"], max_new=max(new))
        kw.update(cu=cu, seen=seen, max_new=max(new))
    else:
        pos, seen = plan["pos"], torch.ones(s["pad"], dtype=torch.int64, device=dev())
    for add in (True, False):
        c1, c2 = s["cache"].clone(), s["cache"].clone()
        out = swa.kv4_block(c1, s["x"], s["wd"], s["table"], plan["lens"], plan["slot"], pos, add=s["add"] if add else None, **kw)
        assert swa.swa_attn_check_status(ws, kind=kind) == swa.SWA_OK
        want = parts(s, c2, kind, tree, window, pos, cu, kw.get("seen"), max(new), ws, add)
        assert torch.equal(c1, c2)
        real = sum(new)
        assert torch.equal(out[:real], want[:real])
        h, part = oracle_out(s, c1, kind, window, pos.tolist(), cu.tolist(), seen.tolist(), add)
        got = f64(out)[:real] - h[:real]
        # out itself is rounded: half a step of it
        err = np.linalg.norm(got - part[:real])
        room = (2.0 ** -8 if kind == "bf16" else 2.0 ** -24) * np.linalg.norm(f64(out)[:real])
        assert err <= (2e-2 if kind == "bf16" else 1e-4) * np.linalg.norm(part[:real]) + room


def test_block_refuses():
    s = step_case("bf16", 2, [1, 1], [5, 9], 4, 2, 128, 64)
    p = s["plan"]
    n = 2
    x, slot, pos = s["x"][:n].contiguous(), p["slot"][:n].contiguous(), p["pos"][:n].contiguous()
    ok = swa.kv4_block(s["cache"], x, s["wd"], s["table"], p["lens"], slot, pos, Hq=4)
    assert ok.shape == x.shape
    with pytest.raises(ValueError):       # tokens without a tree, and not one a request
        swa.kv4_block(s["cache"], s["x"], s["wd"], s["table"], p["lens"], p["slot"], p["pos"], Hq=4)
    with pytest.raises(ValueError):
        swa.kv4_block(s["cache"], x, s["wd"][:3], s["table"], p["lens"], slot, pos, Hq=4)
    with pytest.raises(ValueError):
        swa.kv4_block(s["cache"], x, s["wd"], s["table"], p["lens"], slot, pos, Hq=2)
    with pytest.raises(swa.SwaError):     # onto its own input
        swa.kv4_block(s["cache"], x, s["wd"], s["table"], p["lens"], slot, pos, Hq=4, out=x)
    small = swa.new_kv4_workspace(s["cache"], 2, 4, max_pages=4)
    before = s["cache"].clone()
    with pytest.raises(swa.SwaError):
        swa.kv4_block(s["cache"], x, s["wd"], s["table"], p["lens"], slot, pos, Hq=4, workspace=small)
    assert torch.equal(before, s["cache"])
    empty = swa.kv4_block(s["cache"], x[:0], s["wd"], s["table"][:0], p["lens"][:0], slot[:0], pos[:0], Hq=4)
    assert empty.shape == (0, 64)


@pytest.mark.parametrize("kind", KINDS)
def test_accepted_tokens_moved_are_plain_decoding(kind):
    # a tree is appended and a path of it accepted: after the move the cache holds, token by token, what plain decoding
    # of the path would have put there, and the next token's attention is the same
    Hkv, Hq, d, page, old = 2, 4, 128, 16, 21
    T, path = 9, [0, 2, 5, 8]
    parent = [-1, 0, 0, 1, 1, 2, 2, 5, 5]
    max_pages = 3
    table = torch.tensor([[4, 2, 0]], dtype=torch.int32, device=dev())
    rope = swa.rope_tables(64, d)
    k, v = (randn(30 + i, old + T, Hkv, d, dtype=DT[kind]).to(dev()) for i in range(2))
    slots = lambda at: (table[0, at // page].long() * page + at % page).view(1, -1)   # noqa: E731
    every = torch.arange(old + T, device=dev())
    a = swa.new_kv4_cache(6, page, Hkv, d, dev())
    swa.kv4_append(a, k[None, :old], v[None, :old], slots(every[:old]), rope=rope)
    b = a.clone()
    pos, seen = swa.kv4_tree(i32(*parent), i32(0, T), i32(old + T), max_new=T)
    swa.kv4_append(a, k[None, old:].contiguous(), v[None, old:].contiguous(), slots(every[old:]), pos=pos.view(1, T), rope=rope)
    src = slots(every[old:][torch.tensor(path, device=dev())])
    dst = slots(every[old:old + len(path)])
    swa.kv4_move(a, src, dst)
    at = torch.tensor(path, device=dev()) + old
    swa.kv4_append(b, k[None, at], v[None, at], dst, pos=(old + torch.arange(len(path), device=dev(), dtype=torch.int32)).view(1, -1), rope=rope)
    n = old + len(path)
    for x, y in zip(swa.kv4_read(a, slots(every[:n]), dtype=DT[kind]), swa.kv4_read(b, slots(every[:n]), dtype=DT[kind])):
        assert torch.equal(x, y)
    q = randn(33, 1, Hq, d, dtype=DT[kind]).to(dev())
    for x, y in zip(swa.kv4_attention(a, q, table, i32(n), rope=rope), swa.kv4_attention(b, q, table, i32(n), rope=rope)):
        assert torch.equal(x, y)


def test_a_drafted_step_captured_and_replayed():
    # plan's tokens, tree, block and move in one graph, with another tree and other tokens in the replay
    s = step_case("bf16", 3, [8, 8, 8], [40, 17, 90], 6, 3, 128, 192)
    C, N = 192, 24
    ws = swa.new_kv4_block_workspace(s["cache"], N, C, 6)
    plan, cu = s["plan"], s["plan"]["cu"]
    parent = torch.tensor(random_parents(8, 1) + random_parents(8, 2) + random_parents(8, 3), dtype=torch.int32, device=dev())
    src = plan["slot"].view(3, 8)[:, 4:6].contiguous()
    dst = plan["slot"].view(3, 8)[:, 1:3].contiguous()
    cache = s["cache"]

    def run():
        pos, seen = swa.kv4_tree(parent, cu, plan["lens"], max_new=8, workspace=ws)
        out = swa.kv4_block(cache, s["x"], s["wd"], s["table"], plan["lens"], plan["slot"], pos, Hq=6, cu=cu, seen=seen, max_new=8,
                            gain=s["gain"], add=s["add"], rope=s["rope"], gq=s["gq"], gk=s["gk"], workspace=ws)
        r = swa.rms_norm(out, s["gain"], fp8=True)
        y = swa.w4_linear(r["y"], s["wd"][0], out_features=6 * 128, scale=r["scale"])
        swa.kv4_move(cache, src, dst)
        return pos, seen, out, y
    start = cache.clone()
    run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run()
    for seed in (1, 7):
        parent.copy_(torch.tensor(random_parents(8, seed) + random_parents(8, seed + 1) + random_parents(8, seed + 2), dtype=torch.int32))
        s["x"].copy_(randn(50 + seed, N, C, dtype=torch.bfloat16))
        cache.copy_(start)
        g.replay()
        torch.cuda.synchronize()
        replayed, held = [t.clone() for t in got], cache.clone()
        cache.copy_(start)
        want = run()
        assert all(torch.equal(a, b) for a, b in zip(replayed, want)) and torch.equal(held, cache)
    assert swa.swa_attn_check_status(ws) == swa.SWA_OK


def test_norm_and_its_backward_captured_beside_an_eager_graph_of_the_same_leaves():
    x = randn(60, 40, 256, dtype=torch.bfloat16).to(dev())
    dy, g = randn(61, 40, 256, dtype=torch.bfloat16).to(dev()), (1 + 0.1 * randn(62, 256)).to(dev())
    leaf = x.float().requires_grad_()
    kept = (leaf * 2).sum()               # an autograd graph that lives on

    def run():
        f = swa.rms_norm(x, g)
        return swa.rms_norm_backward(f["h"], f["rstd"], dy, g)
    want = run()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        got = run()
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(got["dx"], want["dx"]) and torch.equal(got["dgain"], want["dgain"])
    kept.backward()


def test_calls_on_two_streams_at_once():
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    cases = []
    for seed in (70, 80):
        w4 = random_w4(seed, 2048, 4096).to(dev())
        x = randn(seed + 1, 40, 4096, dtype=torch.bfloat16).to(dev())
        g = (1 + 0.1 * randn(seed + 2, 4096)).to(dev())
        cases.append((w4, x, g))

    def run(c, stream):
        r = swa.rms_norm(c[1], c[2], stream=stream)
        y = swa.w4_linear(r["y"], c[0], stream=stream)
        z = swa.w4_linear(r["y"][:5].contiguous() if stream is None else r["y"][:5], c[0], stream=stream)
        back = swa.rms_norm_backward(c[1], r["rstd"], r["y"], c[2], stream=stream)
        return [r["y"], y, z, back["dx"], back["dgain"]]
    want = [run(c, None) for c in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for c, st in zip(cases, (a, b)):
            st.wait_stream(torch.cuda.current_stream())
            got.append(run(c, st))
        for st in (a, b):
            st.synchronize()
        for w, x in zip(want, got):
            assert all(torch.equal(u, v) for u, v in zip(w, x))
    tree_case("bf16", [300, 77], [20, 9], 4, 2, 128, 32, -1, 64, False, stream=a)


def test_short_way_gives_the_long_ways_bits(monkeypatch):
    x, add = (randn(90 + i, 3, 7, 264, dtype=torch.bfloat16).to(dev()) for i in range(2))
    g = (1 + 0.1 * randn(92, 264)).to(dev())
    w4 = random_w4(93, 100, 264).to(dev())
    cache, table, _ = build_cache([50, 33], 2, 128, 16, 94)
    cd, td, lens, cu = cache.to(dev()), table.to(dev()), i32(50, 33), i32(0, 3, 5)
    parent, q = i32(-1, 0, 0, -1, 0, 0), randn(95, 6, 4, 128, dtype=torch.bfloat16).to(dev())
    ws = swa.new_kv4_workspace(cd, 2, 4, max_pages=td.shape[1])
    src, dst = torch.tensor([[3, 4]], device=dev()), torch.tensor([[5, -1]], device=dev())

    def run():
        f = swa.rms_norm(x, g, add=add)
        e = swa.rms_norm(x, g, add=add, fp8=True)
        b = swa.rms_norm_backward(f["h"], f["rstd"], add, g, dh=x)
        y = swa.w4_linear(f["y"], w4, out_features=100)
        z = swa.w4_linear(e["y"], w4, out_features=100, scale=e["scale"], dtype=torch.float32)
        pos, seen = swa.kv4_tree(parent, cu, lens, max_new=3, workspace=ws)
        o, lse = swa.kv4_tree_attention(cd, q, td, lens, cu, pos, seen, max_new=3, window=40, workspace=ws)
        c = cd.clone()
        swa.kv4_move(c, src, dst)
        return [f["y"], f["h"], f["rstd"], e["y"].view(torch.uint8), e["scale"], b["dx"], b["dgain"], y, z, pos, seen, o, lse, c]
    assert swa._fast is not None
    assert swa.load("fp32") is not None
    fast = run()
    calls = [n for n in ("rms_norm", "rms_norm_backward", "w4_linear", "kv4_tree", "kv4_tree_attention", "kv4_move")]
    assert all(callable(getattr(swa._fast, n)) for n in calls)
    assert swa._fast.rms_norm(x, g, add, 1e-6, False, False) is not None       # the short way takes it
    assert swa._fast.rms_norm(x.half(), g, None, 1e-6, False, False) is None   # and leaves the unusual
    assert swa._fast.w4_linear(x[:, :, ::2], w4, 100, None, None, 0, None, None) is None
    monkeypatch.setattr(swa, "_fast", None)
    for a, b in zip(fast, run()):
        assert a.dtype is b.dtype and a.shape == b.shape and torch.equal(a, b)
    assert swa.swa_attn_check_status(ws) == swa.SWA_OK


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,T", [(4, 3), (4, 16)])
@pytest.mark.parametrize("grow", [3.0, 30.0])
def test_tree_of_keys_whose_logits_grow(kind, Hq, T, grow):
    # keys of later blocks are much larger, so that the running maximum rises again and again, by up to hundreds; the
    # first block's are tiny. Compared relative to what a logit of that size may be off by.
    d, page, n = 128, 64, 900
    cache, table, rows = build_cache([n], 1, d, page, 40)
    sc = cache[..., 16 * d:].view(torch.bfloat16).view(*cache.shape[:3], 2, 16, 2, 2)
    for j in range(n):
        f = 0.01 if j < 128 else grow * (j // 128) / 7
        sc[int(table[0, j // page]), :, j % page // 16, 0, j % 16] *= f
    keys = []
    for j in range(n):
        keys.append(np.array([dec.read_row(cache.numpy(), page, int(table[0, j // page]) * page + j % page, 0)[0]]))
    keys, vals = np.array(keys), rows[0][1]
    parent = random_parents(T, 41)
    pos, seen = serve.tree(parent, n - T)
    q = randn(42, T, Hq, d, dtype=DT[kind])
    o, lse = swa.kv4_tree_attention(cache.to(dev()), q.to(dev()), table.to(dev()), i32(n), i32(0, T), i32(*pos),
                                    torch.tensor(seen, device=dev()), max_new=T)
    ro, rl = serve.tree_attend(f64(q), keys, vals, pos, seen)
    # a logit's products sum to |q|_1-like sizes: |q| |k| <= sqrt(d) * |k|; the error is 2.6e-6 of that (see test_serve_gpu.py)
    size = np.abs(keys).max() * d / np.sqrt(d) * np.sqrt(d)
    slip = 2.6e-6 * size
    assert np.all(np.abs(f64(lse) - rl) <= slip + 2e-6 * np.abs(rl))
    top = np.abs(vals).max()
    assert np.all(np.abs(f64(o) - ro) <= (2 * slip + 2.0 ** -8 + 2e-4) * top + 2.0 ** -8 * np.abs(ro))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [3, 20])
def test_tree_of_gains_and_scales_of_every_size(kind, T):
    d, page, n = 128, 16, 200
    for gain, scale in ((1e-3, 0.0), (50.0, 0.0), (1.0, 1e-4), (0.0, 0.0)):
        cache, table, rows = build_cache([n], 1, d, page, 43)
        pos, seen = serve.tree(random_parents(T, 44), n - T)
        q, gq = randn(45, T, 4, d, dtype=DT[kind]), torch.full((d,), gain)
        o, lse = swa.kv4_tree_attention(cache.to(dev()), q.to(dev()), table.to(dev()), i32(n), i32(0, T), i32(*pos),
                                        torch.tensor(seen, device=dev()), max_new=T, gq=gq.to(dev()), softmax_scale=scale)
        ro, rl = serve.tree_attend(f64(q), *rows[0], pos, seen, gq=f64(gq), scale=scale)
        slip = 8e-5 * max(gain, 1.0)
        assert np.all(np.abs(f64(lse) - rl) <= slip + 1e-5)
        top = np.abs(rows[0][1]).max()
        assert np.all(np.abs(f64(o) - ro) <= (2 * slip + 2.0 ** -8 + 1e-4) * top + 2.0 ** -8 * np.abs(ro))


@pytest.mark.parametrize("T", [2, 12])
def test_tree_over_a_cache_past_32_bits(T):
    # pages whose byte offsets, and slots, need more than 32 bits
    d, page, Hkv = 128, 1024, 4
    tile = 18 * d * Hkv * (page // 16)
    n_pages = (1 << 33) // tile + 40
    cache = torch.zeros(n_pages, Hkv, page // 16, 18 * d, dtype=torch.uint8, device=dev())
    ids = [n_pages - 1, 3, n_pages - 7]
    table = i32(*ids)[None].contiguous()
    n = 2 * page + 77
    at = torch.arange(n, device=dev())
    slot = (table[0, at // page].long() * page + at % page).view(1, n)
    k, v = (randn(46 + i, 1, n, Hkv, d, dtype=torch.bfloat16).to(dev()) for i in range(2))
    swa.kv4_append(cache, k, v, slot)
    kh, vh = (f64(t)[0] for t in swa.kv4_read(cache, slot, dtype=torch.float32))
    pos, seen = serve.tree(random_parents(T, 48), n - T)
    q = randn(49, T, 8, d, dtype=torch.bfloat16).to(dev())
    o, lse = swa.kv4_tree_attention(cache, q, table, i32(n), i32(0, T), i32(*pos), torch.tensor(seen, device=dev()), max_new=T)
    ro, rl = serve.tree_attend(f64(q), kh, vh, pos, seen)
    assert np.abs(f64(lse) - rl).max() <= 1e-4
    assert np.linalg.norm(f64(o) - ro) <= 9e-3 * np.linalg.norm(ro)
    far = slot[:, -3:]
    swa.kv4_move(cache, far, slot[:, 1030:1033].contiguous())
    moved = swa.kv4_read(cache, slot[:, 1030:1033].contiguous(), dtype=torch.float32)
    assert np.array_equal(f64(moved[0])[0], kh[-3:]) and np.array_equal(f64(moved[1])[0], vh[-3:])


# Tables of 4096 tokens and more: CTAs that find their shares from all the lengths.
RAGGED = [  # lens, new, Hq, Hkv, d, page, window, rot, interleaved
    ([4200, 0, 1, 17, 4100, 900, 2500], [4, 0, 1, 3, 2, 4, 4], 8, 2, 128, 64, -1, 128, False),
    ([4200, 0, 1, 17, 4100, 900, 2500], [4, 0, 1, 3, 2, 4, 4], 4, 4, 64, 16, -1, 64, False),
    ([17, 4200, 33, 64, 0], [16, 20, 33, 1, 0], 8, 2, 128, 64, -1, 0, False),           # two groups of 64 rows
    ([17, 4200, 33, 64, 0], [16, 20, 30, 1, 0], 6, 2, 64, 64, -1, 0, True),
    ([5000, 4999, 4097, 30], [8, 8, 7, 8], 2, 1, 128, 256, 4500, 64, False),
    ([9000], [3], 1, 1, 64, 64, -1, 64, False),
    ([9000], [64], 4, 1, 128, 64, -1, 128, False),
    ([1] * 60 + [4200] + [40 + i for i in range(67)], [1] * 128, 2, 1, 64, 16, -1, 0, False),        # 128 requests
    ([1] * 60 + [4200] + [40 + i for i in range(68)], [1] * 129, 2, 1, 64, 16, -1, 0, False),        # one more: the host's grid
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("case", range(len(RAGGED)))
def test_ragged_long_batches(kind, case):
    tree_case(kind, *RAGGED[case])


@pytest.mark.parametrize("T", [3, 12])
@pytest.mark.parametrize("kind", KINDS)
def test_shares_of_refused_requests_and_of_a_wide_table(kind, T):
    # a table far wider than its requests; two of them refused; lengths of a
    # captured call that grow between its replays
    B, Hq, Hkv, d, page = 5, 4, 2, 128, 16
    lens = [300, 260, 310, 5, 1200]
    new = [T, T, T, 0, T]
    cache, table, rows = build_cache(lens, Hkv, d, page, 61)
    wide = torch.full((B, 700), -1, dtype=torch.int32)
    wide[:, : table.shape[1]] = table
    cd, wide = cache.to(dev()), wide.to(dev())
    cu = np.concatenate([[0], np.cumsum(new)])
    trees = [serve.tree(random_parents(n, 62), m - n) for n, m in zip(new, lens)]
    seen = torch.tensor(np.array([s for t in trees for s in t[1]] + [0] * 3, dtype=np.uint64).view(np.int64), device=dev())
    q = randn(63, sum(new) + 3, Hq, d, dtype=DT[kind]).to(dev())
    ws = swa.new_kv4_workspace(cd, B, Hq, max_pages=700, kind=kind)
    held, where = i32(*lens), i32(*np.concatenate([t[0] for t in trees] + [[0] * 3]))

    def call():
        return swa.kv4_tree_attention(cd, q, wide, held, i32cu, where, seen, max_new=T, workspace=ws)

    i32cu = i32(*cu)

    def check(o, lse, dead=(), less=0):
        od, ld = f64(o), f64(lse)
        for b in range(B):
            at = slice(cu[b], cu[b + 1])
            if b in dead or b == 3:
                assert not od[at].any() and np.all(ld[at] == -np.inf)
                continue
            pos, vis = trees[b]
            n = lens[b] - less if b == 4 else lens[b]
            ro, rl = serve.tree_attend(f64(q)[at], rows[b][0][:n], rows[b][1][:n], np.asarray(pos) - (lens[b] - n), vis)
            top = np.abs(rows[b][1]).max()
            assert np.abs(ld[at] - rl).max() <= 1e-4
            assert np.all(np.abs(od[at] - ro) <= (1.7e-4 + 2.0 ** -8) * top + 2.0 ** -8 * np.abs(ro))
        assert not od[cu[-1]:].any() and np.all(ld[cu[-1]:] == -np.inf)

    o, lse = call()
    check(o, lse)
    assert swa.swa_attn_check_status(ws, kind=kind) == swa.SWA_OK
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go, gl = call()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(go, o) and torch.equal(gl, lse)
    full, at_full = held.clone(), where.clone()
    held[4] -= 900                                   # an earlier state of the long request
    where[cu[4]:cu[5]] -= 900
    g.replay()
    torch.cuda.synchronize()
    check(go, gl, less=900)
    held.copy_(full)
    where.copy_(at_full)
    held[0], held[2] = -1, 700 * page + 1            # refused
    g.replay()
    torch.cuda.synchronize()
    assert swa.swa_attn_check_status(ws, kind=kind) == swa.SWA_ERR_DEVICE_CHECK
    check(go, gl, dead=(0, 2))
    held.copy_(full)
    g.replay()
    torch.cuda.synchronize()
    assert swa.swa_attn_check_status(ws, kind=kind) == swa.SWA_OK
    assert torch.equal(go, o) and torch.equal(gl, lse)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("C", [96, 40000])
def test_norm_copies_its_input_where_h_is_wanted_without_an_addition(kind, C):
    x = randn(70, 5, C, dtype=DT[kind]).to(dev())
    want = swa.rms_norm(x)
    h, y = torch.zeros_like(x), torch.zeros_like(x)
    assert swa.swa_rms_norm(5, C, 1e-6, x, None, None, h, y, None, None, None, kind=kind) == swa.SWA_OK
    assert torch.equal(h, x) and torch.equal(y, want["y"])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("C", [248, 1000, 2048, 3000, 4096, 6008, 8192, 12000, 16384, 20000])
def test_norm_backward_of_more_rows_than_blocks(kind, C):
    # every width of row, blocks with several rows whose loads overlap, in place.
    # dx: half a step of its type (2^-8 or 2^-24) and fp32's own few roundings of
    # terms of size rstd (|d| + |xh mean|) + |dh|: 1e-6 of them; its mean over C of
    # products of size |d xh| is a sum of C / threads and then log terms: 1e-5.
    # dgain: at most ~700 additions in a row, 700 * 2^-24 of the sum of sizes.
    rows = 6000 if C <= 1000 else (1300 if C < 4096 else 700)
    h, dy, dh = (randn(71 + i, rows, C, dtype=DT[kind]).to(dev()) for i in range(3))
    g = (1 + 0.1 * randn(74, C)).to(dev())
    rstd = swa.rms_norm(h)["rstd"]
    r = swa.rms_norm_backward(h, rstd, dy, g, dh=dh)
    xh, d = h.double() * rstd.double()[:, None], dy.double() * g.double()
    mean = (d * xh).mean(-1, keepdim=True)
    want = rstd.double()[:, None] * (d - xh * mean) + dh.double()
    size = rstd.double()[:, None] * (d.abs() + xh.abs() * ((d * xh).abs().mean(-1, keepdim=True))) + dh.double().abs()
    half = 2.0 ** -8 if kind == "bf16" else 2.0 ** -24
    assert bool(((r["dx"].double() - want).abs() <= half * want.abs() + 1.1e-5 * size).all())
    dg, top = (dy.double() * xh).sum(0), (dy.double() * xh).abs().sum(0)
    assert bool(((r["dgain"].double() - dg).abs() <= 700 * 2.0 ** -24 * top).all())
    ws = torch.empty(swa.swa_rms_norm_workspace_size(rows, C, kind), dtype=torch.uint8, device=dev())
    for at in range(3):
        t = [h.clone(), dy.clone(), dh.clone()]
        dgain = torch.empty_like(g)
        assert swa.swa_rms_norm_bwd(rows, C, t[0], rstd, g, t[1], t[2], t[at], dgain, ws, kind=kind) == swa.SWA_OK
        assert torch.equal(t[at], r["dx"]) and torch.equal(dgain, r["dgain"])
