"""The positions, the cache, the kept blocks and block attention around the
indexer's own calls, launched back to back: what one call leaves on the
device (lengths, rows, lists) is what the next one reads."""
import math

import numpy as np
import pytest
import torch

import hierarchical_top_indexer_b200 as hisa
from tests import attn_ref as ref
from tests.test_gpu_block_attn import _f64, _i32

pytestmark = pytest.mark.gpu


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").bfloat16()


@pytest.mark.parametrize("dtype", ["bf16", "fp4"])
@pytest.mark.parametrize("graph", [False, True])
def test_decode_step_then_store_then_attend(dtype, graph):
    """hisa_decode_step advances the shared length in its last kernels; the store at the last position and the attention
    up to it follow without a wait on the host, as a captured step too."""
    g = torch.Generator("cuda").manual_seed(3)
    batch, cap, H, Hq, Hkv, d, B, m, k, steps = 5, 640, 16, 8, 2, 128, 64, 4, 64, 6
    start = np.array([600, 0, 63, 64, 320])
    kv = hisa.KVCache(batch, cap, 128, B)
    c = hisa.AttnCache(batch, cap, Hkv, d, dtype, lens=kv.len, status=kv.status)
    irope, arope = hisa.hisa_rope_init(128, rot=64), hisa.hisa_rope_init(d, layout="interleaved")
    kv.keys.copy_(_randn(g, batch, cap, 128) / 8)
    kv.len.copy_(_i32(start))
    hisa.hisa_pool_blocks(kv)
    n = int(start.sum())
    seq, pos = _i32(np.repeat(np.arange(batch), start)), _i32(np.concatenate([np.arange(s) for s in start]))
    hisa.hisa_cache_store(c, _randn(g, n, Hkv, d), _randn(g, n, Hkv, d), seq, pos)
    rows, w = _i32(np.arange(batch)), torch.rand((batch, H), generator=g, device="cuda")
    new = [[_randn(g, batch, *s) for s in ((128,), (H, 128), (Hq, d), (Hkv, d), (Hkv, d))] for _ in range(steps)]
    tok, Qi, Qa, K1, V1 = (torch.empty_like(x) for x in new[0])
    at, lists = torch.empty_like(kv.len), torch.empty((batch, m), dtype=torch.int32, device="cuda")
    size = max(hisa.hisa_select_blocks_workspace_bytes(kv, batch, H, m), hisa.hisa_decode_step_workspace_bytes(kv, H, m, k),
               hisa.hisa_block_attn_workspace_bytes(c, batch, Hq, B, m))
    ws, idx = hisa.workspace(size), torch.empty((batch, k), dtype=torch.int32, device="cuda")
    out = torch.empty((batch, Hq, d), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((batch, Hq), device="cuda")
    Qr, Kr = torch.empty_like(Qa), torch.empty_like(K1)

    def step():
        at.copy_(kv.len)
        hisa.hisa_rope(irope, tok, at, out=tok)
        hisa.hisa_rope(irope, Qi, at, out=Qi)
        hisa.hisa_rope(arope, K1, at, out=Kr)
        hisa.hisa_decode_step(kv, tok, Qi, w, m, k, ws=ws, idx=idx)
        hisa.hisa_cache_store(c, Kr, V1, rows)
        hisa.hisa_rope(arope, Qa, at, out=Qr)
        hisa.hisa_select_blocks(kv, Qi, w, rows, None, m, ws=ws, blocks=lists)
        hisa.hisa_block_attn(c, Qr, rows, None, lists, B=B, ws=ws, out=out, lse=lse)

    play = step
    if graph:
        for x, y in zip((tok, Qi, Qa, K1, V1), new[0]):
            x.copy_(y)
        keep = [t.clone() for t in (kv.len, kv.keys, kv.pooled, kv.pooled_hl, c.k, c.v)]
        step()
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            step()
        for t, x in zip((kv.len, kv.keys, kv.pooled, kv.pooled_hl, c.k, c.v), keep):
            t.copy_(x)
        play = captured.replay
    seen = []
    for i in range(steps):
        for x, y in zip((tok, Qi, Qa, K1, V1), new[i]):
            x.copy_(y)
        play()
        seen.append([t.clone() for t in (at, idx, lists, Qr, Kr, V1, out, lse)])
    assert kv.status_bits() == 0 and (kv.len.cpu().numpy() == start + steps).all()
    every = [(_i32(np.full(s + steps, b)), _i32(np.arange(s + steps))) for b, s in enumerate(start)]
    K, V = np.zeros((2, batch, Hkv, cap, d))
    for b, (sq, ps) in enumerate(every):
        kr, vr = hisa.hisa_cache_load(c, sq, ps)
        K[b, :, :len(ps)], V[b, :, :len(ps)] = _f64(kr).swapaxes(0, 1), _f64(vr).swapaxes(0, 1)
    for i, (at_, idx_, lists_, Qr_, Kr_, V1_, out_, lse_) in enumerate(seen):
        t = start + i
        assert (at_.cpu().numpy() == t).all()
        for b in range(batch):
            for rows_, x in ((K, Kr_), (V, V1_)):
                want = _f64(x[b]) if dtype == "bf16" else ref.fp4_rows(_f64(x[b]))[2]
                assert np.array_equal(rows_[b, :, t[b]], want)
            kept = {int(j) for j in lists_[b] if j >= 0}
            assert t[b] // B in kept and {int(s) // B for s in idx_[b] if s >= 0} <= kept    # one stage 1 for both
        r = ref.block_attn(_f64(Qr_), K, V, np.arange(batch), t, lists_.cpu().numpy(), B, 1 / math.sqrt(d))
        ref.check_block_attn(_f64(out_), _f64(lse_), r, d, dtype == "fp4")


@pytest.mark.parametrize("d,B,cap,H,n_q,m", [(64, 8, 8192, 1, 4, 1000), (128, 8, 8192, 128, 300, 70), (64, 16, 1 << 20, 8, 3, 600),
                                             (128, 1024, 3000, 5, 7, 2), (64, 8, 5000, 17, 1, 1)])
def test_select_blocks_of_many_blocks(d, B, cap, H, n_q, m):
    """Rows of more blocks than the scoring kernel keeps the best of itself, and sequences that end inside a block."""
    g = torch.Generator("cuda").manual_seed(cap + B)
    kv = hisa.KVCache(2, cap, d, B)
    kv.keys.copy_(_randn(g, 2, cap, d))
    kv.len.copy_(_i32([cap, cap // 2 - 3]))
    hisa.hisa_pool_blocks(kv)
    Q, w = _randn(g, n_q, H, d), torch.rand((n_q, H), generator=g, device="cuda")
    seq = _i32(np.arange(n_q) % 2)
    want = hisa.hisa_select_inspect(kv, Q, w, seq, None, m, 16)
    ws = hisa.workspace(hisa.hisa_select_blocks_workspace_bytes(kv, n_q, H, m))
    ws.fill_(0xFF)
    blocks, counts = hisa.hisa_select_blocks(kv, Q, w, seq, None, m, want_counts=True, ws=ws)
    assert torch.equal(blocks, want["blocks"]) and torch.equal(counts, want["nblocks"])
    assert (counts == torch.minimum((kv.len[seq.long()] - 1) // B + 1, torch.tensor(m, device="cuda"))).all()
    assert kv.status_bits() == 0
