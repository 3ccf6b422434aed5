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
