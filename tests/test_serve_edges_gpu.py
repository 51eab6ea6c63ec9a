"""Edges of the serving calls that the other files' cases do not reach."""

import numpy as np
import pytest
import torch

import sliding_window_gqa_qk_gb300 as swa
from oracle import serve
from test_decode_gpu import build_cache, f64, numbers_of, randn, scales_of
from oracle import decode as dec
from test_serve_gpu import DT, KINDS, dev, i32

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
