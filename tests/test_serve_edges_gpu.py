"""Edges of the serving calls that the other files' cases do not reach."""

import ctypes
import time

import numpy as np
import pytest
import torch

import sliding_window_gqa_qk_gb300 as swa
from oracle import serve
from test_decode_gpu import build_cache, f64, numbers_of, randn, scales_of
from oracle import decode as dec
from test_serve_gpu import DT, KINDS, check_linear, dev, i32, linear_case, random_parents, random_w4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,T,ahead", [(4, 20, 10), (2, 6, 3), (1, 64, 40), (6, 12, 5)])
@pytest.mark.parametrize("chunks,wide", [(1, 0), (4, 0), (9, 0), (20, 0), (32, 300), (33, 300)])
def test_rows_that_see_nothing_of_the_last_chunk(kind, Hq, T, ahead, chunks, wide):
    # The context ends `ahead` tokens in front of a multiple of 128, where a long request's last chunk begins: that holds
    # only drafted tokens, of a branch that the first `ahead` do not see. Every logit is near -200 in base 2 (each key is
    # a centre opposed to the queries), so that a chunk without a key must not count as one whose logits are 0.
    d, page = 128, 64
    ctx = 128 * chunks - ahead
    n = ctx + T
    cache, table, _ = build_cache([n], 1, d, page, 7)
    sc = cache[..., 16 * d:].view(torch.bfloat16).view(*cache.shape[:3], 2, 16, 2, 2)
    real = torch.isfinite(sc[..., 0, :, :, 0])
    sc[..., 0, :, :, 0] = torch.where(real, sc[..., 0, :, :, 0] * 0.1, sc[..., 0, :, :, 0])
    sc[..., 0, :, :, 1] = torch.where(real, torch.full_like(sc[..., 0, :, :, 1], -12.25), sc[..., 0, :, :, 1])
    keys, vals = [], []
    for j in range(n):
        slot = int(table[0, j // page]) * page + j % page
        nk, nv = numbers_of(cache, page, slot)
        s = scales_of(cache, page, slot)
        keys.append(dec.dequantise(nk, s[0, :, :, 0], s[0, :, :, 1]))
        vals.append(dec.dequantise(nv, s[1, :, :, 0], s[1, :, :, 1]))
    keys, vals = np.array(keys).reshape(n, 1, d), np.array(vals).reshape(n, 1, d)
    parent = list(range(-1, ahead - 1)) + [-1] + list(range(ahead, T - 1))      # two branches, each a chain
    pos, seen = serve.tree(parent, ctx)
    q = (1 + 0.1 * randn(8, T, Hq, d)).to(DT[kind])
    if wide:       # a table whose CTAs find their shares themselves
        table = torch.cat([table, torch.full((1, wide), -1, dtype=torch.int32)], 1).contiguous()
    ws = swa.new_kv4_workspace(cache.to(dev()), 1, Hq, max_pages=table.shape[1], kind=kind)
    o, lse = swa.kv4_tree_attention(cache.to(dev()), q.to(dev()), table.to(dev()), i32(n), i32(0, T), i32(*pos),
                                    torch.tensor(np.array(seen, dtype=np.uint64).view(np.int64), device=dev()), max_new=T, workspace=ws)
    assert swa.swa_attn_check_status(ws, kind=kind) == swa.SWA_OK
    ro, rl = serve.tree_attend(f64(q), keys, vals, pos, seen)
    assert rl.max() < -87 and rl.min() > -160
    # an error of 2.6e-6 of a logit's sum of products (test_decode_gpu.py): |q|_2 <= sqrt(d) |k|_2 / sqrt(d) at most
    size = np.sqrt((keys ** 2).sum(-1)).max()
    slip = 2.6e-6 * size
    assert np.all(np.abs(f64(lse) - rl) <= slip + 2e-6 * np.abs(rl)), (float(np.abs(f64(lse) - rl).max()), slip)
    top = np.abs(vals).max()
    assert np.all(np.abs(f64(o) - ro) <= (2 * slip + 2.0 ** -8 + 2e-4) * top + 2.0 ** -8 * np.abs(ro))


def long_batch(kind, B, T, Hq, Hkv, d, n, page=64):
    """Arguments of the tree attention of B requests of n cached tokens, T of them drafted in a chain, and their workspace."""
    per = -(-n // page)
    cache = torch.randint(0, 256, (B * per, Hkv, page // 16, 18 * d), dtype=torch.uint8, device=dev())
    sc = cache[..., 16 * d:].view(torch.bfloat16)
    sc[..., 0::2], sc[..., 1::2] = 0.2, 0.1
    table = torch.arange(B * per, dtype=torch.int32, device=dev()).view(B, per)
    lens = torch.full((B,), n, dtype=torch.int32, device=dev())
    cu = torch.arange(B + 1, dtype=torch.int32, device=dev()) * T
    pos, seen = swa.kv4_tree(torch.arange(-1, T - 1, dtype=torch.int32, device=dev()).repeat(B), cu, lens, max_new=T)
    q = randn(31, B * T, Hq, d, dtype=DT[kind]).to(dev())
    return cache, q, table, lens, cu, pos, seen, swa.new_kv4_workspace(cache, B, Hq, max_pages=per, kind=kind)


def out_of_time(call, check, ws, kind, tries=20):
    """Runs call under a limit of 1 ns, while another stream keeps the memory busy, until a wait has run out; check()
    after each. Whether one did, and the longest that a call took, in seconds."""
    side, big = torch.cuda.Stream(), [torch.zeros(1 << 28, device=dev()) for _ in range(2)]
    longest = 0.0
    for _ in range(tries):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(3):
                big[0].copy_(big[1])
        start = time.perf_counter()
        assert call(swa.make_extras(wait_limit_ns=1)) == swa.SWA_OK
        st = swa.swa_attn_check_status(ws, kind=kind)
        longest = max(longest, time.perf_counter() - start)
        assert st in (swa.SWA_OK, swa.SWA_ERR_TIMEOUT)
        assert swa.swa_attn_check_status(ws, kind=kind) == swa.SWA_OK      # read and cleared
        check()
        if st == swa.SWA_ERR_TIMEOUT:
            return True, longest
    return False, longest


@pytest.mark.parametrize("n", [100, 700, 768, 900])
@pytest.mark.parametrize("Hq,T", [(4, 16), (4, 5)])
def test_tree_waits_that_run_out_in_short_requests(n, Hq, T):
    # One to eight blocks a CTA, so that the loader has issued its last copies when the others give up. They land before
    # the CTA ends: calls behind it on the same SMs, and on the same workspace, give their bits.
    B = 600
    cache, q, table, lens, cu, pos, seen, ws = long_batch("bf16", B, T, Hq, 1, 128, n)
    want = swa.kv4_tree_attention(cache, q, table, lens, cu, pos, seen, max_new=T, workspace=ws)
    p, c = swa.make_params(B, 1, Hq, 1, 128), swa.swa_kv4_cache(cache.data_ptr(), cache.shape[0], 64)
    o, lse = torch.empty_like(q), torch.empty(B * T, Hq, device=dev())

    def call(ex):
        return swa.swa_kv4_tree_attn(p, ex, c, None, B * T, T, q, None, table, table.shape[1], lens, cu, pos, seen, o, lse, ws)

    def check():
        got = swa.kv4_tree_attention(cache, q, table, lens, cu, pos, seen, max_new=T, workspace=ws)
        assert swa.swa_attn_check_status(ws) == swa.SWA_OK
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    ran_out, longest = out_of_time(call, check, ws, "bf16")
    assert ran_out
    assert longest < 1.0          # the copies land in microseconds; nothing waits for what never comes


@pytest.mark.parametrize("kind,d,Hq,T", [("fp32", 128, 4, 8), ("fp32", 128, 4, 16), ("bf16", 64, 4, 8), ("bf16", 64, 4, 16)])
def test_tree_waits_that_run_out_among_warps_that_share_stages(kind, d, Hq, T):
    # 32 and 64 rows of the m16n8k16 form: two and four warps wait for each other's stages. None waits for one that was
    # never asked for (2 s each, and there are more CTAs than run at once).
    B, n = 32, 8192
    cache, q, table, lens, cu, pos, seen, ws = long_batch(kind, B, T, Hq, 1, d, n)
    want = swa.kv4_tree_attention(cache, q, table, lens, cu, pos, seen, max_new=T, workspace=ws)
    p, c = swa.make_params(B, 1, Hq, 1, d), swa.swa_kv4_cache(cache.data_ptr(), cache.shape[0], 64)
    o, lse = torch.empty_like(q), torch.empty(B * T, Hq, device=dev())

    def call(ex):
        return swa.swa_kv4_tree_attn(p, ex, c, None, B * T, T, q, None, table, table.shape[1], lens, cu, pos, seen, o, lse, ws)

    def check():
        got = swa.kv4_tree_attention(cache, q, table, lens, cu, pos, seen, max_new=T, workspace=ws)
        assert swa.swa_attn_check_status(ws, kind=kind) == swa.SWA_OK
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    _, longest = out_of_time(call, check, ws, kind)      # (the arithmetic may hide every copy)
    assert longest < 1.0


@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("M,N,K", [(33, 48, 4104), (64, 128, 8192), (65, 20000, 640), (100, 160, 6464), (128, 2048, 2048), (129, 130, 5000)])
def test_linear_rings_that_go_round(x8, M, N, K):
    # the pipelines of the form for many rows: more stages than their rings hold, parts of K of different lengths, more
    # tiles than CTAs run at once; every call gives the same bits
    w4, x, scale, r, want, size = linear_case("bf16", M, N, K, x8, True, 40)
    a = [t if t is None else t.to(dev()) for t in (x, w4, scale, r)]
    ws = torch.zeros(256, dtype=torch.uint8, device=dev())
    ys = [swa.w4_linear(a[0], a[1], out_features=N, scale=a[2], add=a[3], dtype=torch.bfloat16, workspace=ws) for _ in range(4)]
    check_linear(ys[0], "bf16", want, size, M, K, x8)
    assert all(torch.equal(y, ys[0]) for y in ys) and swa.swa_attn_check_status(ws) == swa.SWA_OK


@pytest.mark.parametrize("N", [40, 100, 300])
def test_projections_of_the_block_call_keep_its_wait_limit(N):
    # requests without a cached token, so that the attention has nothing to wait for: what runs out is the projections'
    # (N rows: each tile of x that they have). Calls behind it give their bits.
    C, Hq, Hkv, d = 4096, 8, 8, 64
    cache = swa.new_kv4_cache(2, 16, Hkv, d, dev())
    w = [random_w4(50 + i, n, k).to(dev()) for i, (n, k) in enumerate(((Hq * d, C), (Hkv * d, C), (Hkv * d, C), (C, Hq * d)))]
    x = randn(55, N, C, dtype=torch.bfloat16).to(dev())
    table, lens = torch.zeros(N, 1, dtype=torch.int32, device=dev()), torch.zeros(N, dtype=torch.int32, device=dev())
    slot, pos = torch.full((N,), -1, dtype=torch.int64, device=dev()), torch.zeros(N, dtype=torch.int32, device=dev())
    ws = swa.new_kv4_block_workspace(cache, N, C, Hq)
    p, c = swa.make_params(N, 1, Hq, Hkv, d), swa.swa_kv4_cache(cache.data_ptr(), 2, 16)
    weights, out = swa.swa_kv4_weights(C, *(t.data_ptr() for t in w)), torch.empty_like(x)
    want = [swa.w4_linear(x, w[0]), swa.w4_linear(x[:, :Hq * d].contiguous(), w[3])]

    def call(ex):
        return swa.swa_kv4_block(p, ex, c, None, weights, N, 1, x, None, None, None, None, None, None, slot, pos, None, None, table, 1,
                                 lens, out, ws)

    def check():
        got = [swa.w4_linear(x, w[0], workspace=ws), swa.w4_linear(x[:, :Hq * d].contiguous(), w[3], workspace=ws)]
        assert call(None) == swa.SWA_OK and swa.swa_attn_check_status(ws) == swa.SWA_OK
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(out, x)
    check()
    ran_out, longest = out_of_time(call, check, ws, "bf16")
    assert ran_out
    assert longest < 1.0


def test_the_short_way_leaves_numbers_that_are_no_size():
    x, w4 = randn(24, 3, 64, dtype=torch.bfloat16).to(dev()), torch.zeros(2, 1, 544, dtype=torch.uint8, device=dev())
    for n in (-1, -5, -(2 ** 31)):
        with pytest.raises(ValueError):
            swa.w4_linear(x, w4, out_features=n)
    assert swa.w4_linear(x, w4).shape == (3, 32)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,d,T", [(2, 128, 3), (4, 128, 12), (2, 64, 9)])
def test_rows_in_front_of_the_first_request_are_padding(kind, Hq, d, T):
    # some requests of a larger step: the rows of the others, in front and behind, hold nothing
    lens, page, front, behind = [40, 33], 16, 5, 3
    cache, table, rows = build_cache(lens, 1, d, page, 21)
    cd, td = cache.to(dev()), table.to(dev())
    N = front + 2 * T + behind
    cu = i32(front, front + T, front + 2 * T)
    parent = torch.arange(-1, T - 1).repeat(2)
    parent = torch.cat([torch.full((front,), 7), parent, torch.full((behind,), -1)]).int().to(dev())
    ws = swa.new_kv4_workspace(cd, 2, Hq, max_pages=td.shape[1], kind=kind)
    # (outputs of the C calls, so that what they leave alone is seen)
    pos, seen = torch.full((N,), 77, dtype=torch.int32, device=dev()), torch.full((N,), 77, dtype=torch.int64, device=dev())
    assert swa.swa_kv4_tree(2, N, T, parent, cu, i32(*lens), pos, seen, ws) == swa.SWA_OK
    assert pos[:front].tolist() == [0] * front and seen[:front].tolist() == [0] * front
    assert pos[-behind:].tolist() == [0] * behind and seen[-behind:].tolist() == [0] * behind
    q = randn(22, N, Hq, d, dtype=DT[kind]).to(dev())
    o, lse = torch.full_like(q, 5.0), torch.full((N, Hq), 5.0, device=dev())
    p, c = swa.make_params(2, 1, Hq, 1, d), swa.swa_kv4_cache(cd.data_ptr(), cd.shape[0], page)
    assert swa.swa_kv4_tree_attn(p, None, c, None, N, T, q, None, td, td.shape[1], i32(*lens), cu, pos, seen, o, lse, ws) == swa.SWA_OK
    assert swa.swa_attn_check_status(ws, kind=kind) == swa.SWA_OK
    for at in (slice(0, front), slice(N - behind, N)):
        assert not o[at].any() and torch.isneginf(lse[at]).all()
    for b, n in enumerate(lens):
        at = slice(front + b * T, front + (b + 1) * T)
        ro, rl = serve.tree_attend(f64(q)[at], *rows[b], *serve.tree(list(range(-1, T - 1)), n - T))
        assert np.abs(f64(lse)[at] - rl).max() <= 1e-4
        assert np.linalg.norm(f64(o)[at] - ro) <= (9e-3 if kind == "bf16" else 1e-5) * np.linalg.norm(ro)


def test_a_failed_launch_is_not_told_again():
    # A launch into a capture that is no longer valid fails on the host. The next call, which has nothing to do with it,
    # succeeds. (The capture is begun and ended by the driver's functions, so that torch knows nothing of it.)
    cu = ctypes.CDLL("libcuda.so.1")
    w4 = torch.randint(0, 128, (256, 64, 544), dtype=torch.uint8, device=dev())
    g = torch.ones(4096, device=dev())
    for M in (4, 40, 0):         # in a cluster, each form
        x = randn(23, max(M, 1), 4096, dtype=torch.bfloat16).to(dev())
        y = torch.empty_like(x)
        assert swa.swa_w4_linear(M, 4096, 4096, x, None, w4, None, y) == swa.SWA_OK
        torch.cuda.synchronize()
        stream = torch.cuda.Stream()
        h = ctypes.c_void_p(stream.cuda_stream)
        assert cu.cuStreamBeginCapture_v2(h, 2) == 0
        assert cu.cuStreamSynchronize(h) != 0                  # not allowed in a capture, which ends it
        if M:
            failed = swa.swa_w4_linear(M, 4096, 4096, x, None, w4, None, y, stream=stream)
        else:                    # the gradient of no rows: a memset
            failed = swa.swa_rms_norm_bwd(0, 4096, None, None, None, None, None, None, g, None, 0, stream=stream, kind="bf16")
        graph = ctypes.c_void_p()
        assert cu.cuStreamEndCapture(h, ctypes.byref(graph)) != 0 and not graph.value
        assert failed == swa.SWA_ERR_CUDA
        out = torch.empty_like(x)
        assert swa.swa_rms_norm(1, 4096, 1e-6, x, None, g, None, out, None, None, None) == swa.SWA_OK
        torch.cuda.synchronize()


def test_the_short_way_takes_the_ordinary_calls():
    # each of its functions itself, with what the Python functions pass: a result, and the long way's bits
    swa.load("fp32")
    f = swa._fast
    assert f is not None
    for dt in (torch.bfloat16, torch.float32):
        x, add = (randn(90 + i, 5, 264, dtype=dt).to(dev()) for i in range(2))
        g, w4 = (1 + 0.1 * randn(92, 264)).to(dev()), random_w4(93, 104, 264).to(dev())
        s = torch.cuda.current_stream()            # asked for by name: the long way

        def same(a, b):
            assert a is not None
            a, b = ([t[k] for k in sorted(t)] if isinstance(t, dict) else list(t) if isinstance(t, tuple) else [t] for t in (a, b))
            assert len(a) == len(b)
            for u, v in zip(a, b):
                assert (u is None) == (v is None) and (u is None or u.dtype is v.dtype and torch.equal(u.float(), v.float()))
        n = f.rms_norm(x, g, add, 1e-6, False, False)
        e = f.rms_norm(x, None, add, 1e-6, True, False)
        same(n, swa.rms_norm(x, g, add=add, stream=s))
        same(e, swa.rms_norm(x, add=add, fp8=True, stream=s))
        y = x.clone()
        assert f.rms_norm(y, g, add, 1e-6, False, True)["h"] is y and torch.equal(y, n["h"])
        ws = torch.empty(swa.swa_rms_norm_workspace_size(5, 264), dtype=torch.uint8, device=dev())
        for w in (None, ws):
            same(f.rms_norm_backward(n["h"], n["rstd"], add, g, x, w), swa.rms_norm_backward(n["h"], n["rstd"], add, g, dh=x, stream=s))
        which = 1 if dt is torch.bfloat16 else 2
        for args, kw in (((None, None, None, 0, None, None), dict()), ((97, None, add[:, :97].contiguous(), which, None, None),
                                                                      dict(out_features=97, add=add[:, :97].contiguous(), dtype=dt))):
            same(f.w4_linear(x, w4, *args) if args[0] else f.w4_linear(x, w4, None, None, None, 0, None, None)[:, :97],
                 swa.w4_linear(x, w4, stream=s, **kw)[:, :97])
        out, r = torch.empty(5, 104, dtype=dt, device=dev()), add[:, :104].contiguous()
        assert f.w4_linear(e["y"], w4, 104, e["scale"], r, which, out, None) is out
        same(out, swa.w4_linear(e["y"], w4, out_features=104, scale=e["scale"], add=r, dtype=dt, stream=s))
        cache, table, _ = build_cache([50, 33], 2, 128, 16, 94)
        cd, td, lens, cu = cache.to(dev()), table.to(dev()), i32(50, 33), i32(0, 3, 5)
        parent, q = i32(-1, 0, 0, -1, 0, 0), randn(95, 6, 4, 128, dtype=dt).to(dev())
        ws, rope, gq = swa.new_kv4_workspace(cd, 2, 4, max_pages=td.shape[1]), swa.rope_tables(64, 64), (1 + 0.1 * randn(96, 128)).to(dev())
        for w in (None, ws):
            tree = f.kv4_tree(parent, cu, lens, 3, w)
            same(tree, swa.kv4_tree(parent, cu, lens, max_new=3, workspace=w, stream=s))
        for pair in ((None, None), rope):
            same(f.kv4_tree_attention(cd, q, td, lens, cu, *tree, 3, *pair, False, gq, 40, 0.0, 1e-6, ws),
                 swa.kv4_tree_attention(cd, q, td, lens, cu, *tree, max_new=3, rope=None if pair[0] is None else pair, gq=gq, window=40,
                                        workspace=ws, stream=s))
        src, dst = torch.tensor([[3, 4]], device=dev()), torch.tensor([[5, -1]], device=dev())
        a, b = cd.clone(), cd.clone()
        assert f.kv4_move(a, src, dst, ws) is True
        swa.kv4_move(b, src, dst, workspace=ws, stream=s)
        assert torch.equal(a, b) and not torch.equal(a, cd)


MANY = [  # lens, new, Hq, Hkv, page: more than 16 (token, head) rows of a kv head, d = 128
    ([700, 40, 129], [16, 16, 5], 4, 1, 64),
    ([2500, 2499], [20, 24], 8, 2, 32),
    ([5000, 300], [30, 9], 2, 2, 64),
    ([9000], [64], 4, 4, 128),
]


@pytest.mark.parametrize("case", range(len(MANY)))
def test_tree_of_many_rows_keeps_its_bits(case):
    # P and the values have 11 bits each: beside o's own rounding they count little. A rounding to 8 bits has an rms of
    # 2^-8 / sqrt(3) times that of 1 / mantissa, 0.74 where mantissas are spread by their logarithm: 1.66e-3. One to 11
    # bits is an eighth of it, twice, of a sum's terms: 3e-4. Together 1.69e-3, and a tenth for how mantissas are spread.
    lens, new, Hq, Hkv, page = MANY[case]
    cache, table, rows = build_cache(lens, Hkv, 128, page, 60 + case)
    cu = np.concatenate([[0], np.cumsum(new)])
    trees = [serve.tree(random_parents(n, 61 + b), m - n) for b, (n, m) in enumerate(zip(new, lens))]
    q = randn(62, int(cu[-1]), Hq, 128, dtype=torch.bfloat16)
    o, _ = swa.kv4_tree_attention(cache.to(dev()), q.to(dev()), table.to(dev()), i32(*lens), i32(*cu), i32(*sum((t[0] for t in trees), [])),
                                  torch.tensor(np.array(sum((t[1] for t in trees), []), dtype=np.uint64).view(np.int64), device=dev()),
                                  max_new=max(new))
    want = np.concatenate([serve.tree_attend(f64(q)[cu[b]:cu[b + 1]], *rows[b], *trees[b])[0] for b in range(len(lens))])
    assert np.linalg.norm(f64(o) - want) <= 1.9e-3 * np.linalg.norm(want), np.linalg.norm(f64(o) - want) / np.linalg.norm(want)


@pytest.mark.parametrize("Hq,T", [(4, 16), (2, 40), (4, 3)])
@pytest.mark.parametrize("powers", [[0], [-14], [12], [13, 14], [-90, -60], [60], [100, 0], [-30, -13, -12, 0, 11, 12, 13, 14, 40], [110, 108]])
def test_tree_of_values_of_every_size(Hq, T, powers):
    # values of each key, or of some, times a power of two: far from fp16's range, in which more than 16 rows hold them
    d, page, n = 128, 64, 900
    cache, table, _ = build_cache([n], 1, d, page, 70)
    sc = cache[..., 16 * d:].view(torch.bfloat16).view(*cache.shape[:3], 2, 16, 2, 2)
    keys, vals, size = [], [], []
    for j in range(n):
        slot = int(table[0, j // page]) * page + j % page
        v = sc[slot // page, :, slot % page // 16, 1, j % 16]
        v *= 2.0 ** powers[(j * 7 + j // 128) % len(powers)]
        s = scales_of(cache, page, slot)
        nk, nv = numbers_of(cache, page, slot)
        keys.append(dec.dequantise(nk, s[0, :, :, 0], s[0, :, :, 1]))
        vals.append(dec.dequantise(nv, s[1, :, :, 0], s[1, :, :, 1]))
        size.append(np.repeat(8 * np.abs(s[1, :, :, 0]) + np.abs(s[1, :, :, 1]), 64, -1))
    keys, vals, size = (np.array(t).reshape(n, 1, d) for t in (keys, vals, size))
    pos, seen = serve.tree(random_parents(T, 71), n - T)
    q = randn(72, T, Hq, d, dtype=torch.bfloat16)
    o, lse = swa.kv4_tree_attention(cache.to(dev()), q.to(dev()), table.to(dev()), i32(n), i32(0, T), i32(*pos),
                                    torch.tensor(np.array(seen, dtype=np.uint64).view(np.int64), device=dev()), max_new=T)
    ro, rl = serve.tree_attend(f64(q), keys, vals, pos, seen)
    so = serve.tree_attend(f64(q), keys, size, pos, seen)[0]          # what a row's terms sum to
    assert np.all(np.abs(f64(lse) - rl) <= 1e-4)
    # P: 2^-8 up to 16 rows, 2^-11 above; a value: exact up to 16 rows, half a step of 2^-11 of four times a key's size
    # above (times size, which is at least a quarter of that); logits 2 * 8e-5
    each = 2.0 ** -8 if Hq * T <= 16 else 2.0 ** -11 + 2.0 ** -10
    assert np.all(np.abs(f64(o) - ro) <= (1.7e-4 + each) * so + 2.0 ** -8 * np.abs(ro))


@pytest.mark.parametrize("Hq,T", [(4, 16), (4, 3)])
def test_tree_of_one_key_far_above_many(Hq, T):
    # one key 25 powers of two above 20000 others, which together still count 6e-4: no P may be lost
    d, page, n = 128, 64, 20000
    per = -(-n // page)
    cache = torch.zeros(per, 1, page // 16, 18 * d, dtype=torch.uint8)
    cache[..., :16 * d] = 0x88                                           # n - 8 = 0 everywhere: keys and values are their centres
    sc = cache[..., 16 * d:].view(torch.bfloat16).view(per, 1, page // 16, 2, 16, 2, 2)
    sc[..., 0, :, :, 1], sc[..., 1, :, :, 1] = 0.0, 1.0
    sc[0, 0, 0, 0, 5, :, 1], sc[0, 0, 0, 1, 5, :, 1] = 1.53125, 0.0      # logits 128 * 1.53 / sqrt(128) = 17.3 and 0
    q = torch.ones(T, Hq, d, dtype=torch.bfloat16)
    pos, seen = serve.tree(list(range(-1, T - 1)), n - T)
    o, lse = swa.kv4_tree_attention(cache.to(dev()), q.to(dev()), torch.arange(per, dtype=torch.int32, device=dev())[None].contiguous(),
                                    i32(n), i32(0, T), i32(*pos), torch.tensor(seen, device=dev()), max_new=T)
    top = 1.53125 * 128 / np.sqrt(128) / np.sqrt(1 + 1e-6)
    count = n - T + np.arange(1, T + 1) - 1.0                             # keys at 0 that a token sees
    want = count * np.exp(-top) / (1 + count * np.exp(-top))
    assert np.abs(f64(lse)[:, 0] - (top + np.log1p(count * np.exp(-top)))).max() <= 1e-4
    # (the logit's 2.6e-6 of 17.3, o's rounding)
    assert np.all(np.abs(f64(o) - want[:, None, None]) <= (2.0 ** -8 + 1e-3) * want[:, None, None])


@pytest.mark.parametrize("Hq,T", [(4, 16), (2, 40)])
@pytest.mark.parametrize("seed", range(8))
def test_tree_of_likely_small_and_unlikely_large_values(Hq, T, seed):
    # logits tens apart and values of 2^-30 to 2^30: what counts in o are keys whose P is as small as their values are large
    d, page, n = 128, 64, 200
    cache, table, _ = build_cache([n], 1, d, page, 80 + seed)
    sc = cache[..., 16 * d:].view(torch.bfloat16).view(*cache.shape[:3], 2, 16, 2, 2)
    g = np.random.default_rng(seed)
    keys, vals, size = [], [], []
    for j in range(n):
        slot = int(table[0, j // page]) * page + j % page
        both = sc[slot // page, :, slot % page // 16, :, j % 16]
        both[:, 0, :, 0] *= 15.0
        both[:, 1] *= 2.0 ** int(g.integers(-30, 31))
        s = scales_of(cache, page, slot)
        nk, nv = numbers_of(cache, page, slot)
        keys.append(dec.dequantise(nk, s[0, :, :, 0], s[0, :, :, 1]))
        vals.append(dec.dequantise(nv, s[1, :, :, 0], s[1, :, :, 1]))
        size.append(np.repeat(8 * np.abs(s[1, :, :, 0]) + np.abs(s[1, :, :, 1]), 64, -1))
    keys, vals, size = (np.array(t).reshape(n, 1, d) for t in (keys, vals, size))
    pos, seen = serve.tree(random_parents(T, 81 + seed), n - T)
    q = randn(82 + seed, T, Hq, d, dtype=torch.bfloat16)
    o, lse = swa.kv4_tree_attention(cache.to(dev()), q.to(dev()), table.to(dev()), i32(n), i32(0, T), i32(*pos),
                                    torch.tensor(np.array(seen, dtype=np.uint64).view(np.int64), device=dev()), max_new=T)
    ro, rl = serve.tree_attend(f64(q), keys, vals, pos, seen)
    so = serve.tree_attend(f64(q), keys, size, pos, seen)[0]
    # as above; a logit is wrong by 2.6e-6 of the sum of its products' sizes
    qn = np.abs(f64(q) / np.sqrt((f64(q) ** 2).mean(-1, keepdims=True) + 1e-6))
    slip = 2.6e-6 * (qn @ np.abs(keys[:, 0]).T).max(-1) / np.sqrt(d) + 2e-5
    assert np.all(np.abs(f64(lse) - rl) <= slip + 2e-6 * np.abs(rl))
    assert np.all(np.abs(f64(o) - ro) <= (2.5 * slip[..., None] + 2.0 ** -11 + 2.0 ** -10) * so + 2.0 ** -8 * np.abs(ro))
