"""Block attention where a tile holds values that a row must not feel: logits
past fp32's range of tokens that only its neighbours keep."""
import math

import numpy as np
import pytest
import torch

import hierarchical_top_indexer_b200 as hisa
from tests import attn_ref as ref
from tests.test_gpu_block_attn import _bf, _f64, _i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,G,B", [(128, 8, 128), (64, 3, 128), (128, 2, 64), (128, 8, 256)])
@pytest.mark.parametrize("every", [2, 5])
def test_unseen_logits_past_fp32(d, G, B, every):
    """A chunk whose groups read the union of their rows' blocks.  One block's
    keys are of 2^70: the rows that keep it have queries of 2^-70, the others
    queries of 2^62 and keys of 2^-62, so that every logit a row sees is of
    order 1 and the ones it does not see are infinite."""
    rng = np.random.default_rng(d + G + B + every)
    n, Hkv, cap = max(4 * (128 // G) + 3, 163), 2, 8192
    nblk, m = cap // B, 2048 // B
    big = nblk // 2                                     # in the middle of a CTA's run of tiles
    K, V = rng.standard_normal((2, 1, Hkv, cap, d))
    K *= 2.0 ** -62
    K[:, :, big * B:(big + 1) * B] *= 2.0 ** 132
    keeps = np.arange(n) % every == 0
    Q = rng.standard_normal((n, Hkv * G, d)) * np.where(keeps, 2.0 ** -70, 2.0 ** 62)[:, None, None]
    blocks = np.stack([rng.permutation(np.delete(np.arange(nblk), big))[:m] for _ in range(n)])
    blocks[keeps, 0] = big
    pos = np.full(n, cap - 1)
    k, v, q = _bf(K), _bf(V), _bf(Q)
    c = hisa.AttnCache.wrap(k, v, _i32([cap]))
    out, lse = hisa.hisa_block_attn(c, q, _i32(np.zeros(n)), _i32(pos), _i32(blocks), B=B)
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
    r = ref.block_attn(_f64(q), _f64(k), _f64(v), np.zeros(n, int), pos, blocks, B, 1 / math.sqrt(d))
    assert r["zabs"].max() < 64
    ref.check_block_attn(_f64(out), _f64(lse), r, d, False)


@pytest.mark.parametrize("dtype", ["bf16", "fp4"])
def test_select_then_attend_with_no_rows(dtype):
    kv = hisa.KVCache(2, 256, 128, 64)
    kv.len.fill_(256)
    hisa.hisa_pool_blocks(kv)
    c = hisa.AttnCache(2, 256, 1, 128, dtype, lens=kv.len, status=kv.status)
    none = _i32([])
    blocks = hisa.hisa_select_blocks(kv, torch.zeros((0, 16, 128), dtype=torch.bfloat16, device="cuda"),
                                     torch.zeros((0, 16), device="cuda"), none, none, 3)
    assert blocks.shape == (0, 3)
    Qa = torch.zeros((5, 4, 128), dtype=torch.bfloat16, device="cuda")
    for pos in (none, None):
        out, lse = hisa.hisa_block_attn(c, Qa[:0], none, pos, blocks, B=64)
        assert out.shape == (0, 4, 128) and lse.shape == (0, 4)
    assert kv.status_bits() == 0


@pytest.mark.parametrize("d,G,rows", [(128, 8, 1), (128, 8, 40), (64, 5, 1), (64, 20, 1), (64, 1, 140)])
def test_values_as_large_as_the_header_allows(d, G, rows):
    """Values around 2^87, weights of rows whose maximum keeps growing a little: the sums before the division are up to
    2^8 times the values and the number of tokens."""
    rng = np.random.default_rng(d + G)
    batch, cap, Hkv = 2, 2048, 2
    K, V = rng.standard_normal((2, batch, Hkv, cap, d))
    K += np.linspace(0, 6, cap)[:, None] / math.sqrt(d)
    V = np.clip(V, -4, 4) * 2.0 ** 86
    Q = 1 + 0.2 * rng.standard_normal((batch * rows, Hkv * G, d))
    seq, pos = np.repeat([0, 1], rows), np.tile(np.arange(cap - rows, cap), 2)
    k, v, q = _bf(K), _bf(V), _bf(Q)
    c = hisa.AttnCache.wrap(k, v, _i32([cap, cap]))
    out, lse = hisa.hisa_block_attn(c, q, _i32(seq), _i32(pos))
    assert torch.isfinite(out.float()).all() and float(v.float().abs().max()) <= 2.0 ** 88
    r = ref.block_attn(_f64(q), _f64(k), _f64(v), seq, pos, None, 1, 1 / math.sqrt(d))
    ref.check_block_attn(_f64(out), _f64(lse), r, d, False)
