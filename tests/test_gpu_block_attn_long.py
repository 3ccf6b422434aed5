"""Block attention with many tiles to a CTA, so that every ring, buffer and
barrier of the kernels is used over and over within a segment, and with
logits that keep growing along the prefix, so that the softmax's reference
moves (and the output is rescaled) again and again.  Sampled rows against
the 64-bit form."""
import math

import numpy as np
import pytest
import torch

import hierarchical_top_indexer_b200 as hisa
from tests import attn_ref as ref
from tests.test_gpu_block_attn import Case, _f64, _i32

pytestmark = pytest.mark.gpu

SMS = 148
DEEPEST = 8          # stages of the deepest ring (4-bit rows of d = 64 in the lone-row kernel)


class Long:
    """Keys a(s) / sqrt(d) u + noise with a growing along the prefix, queries c u + noise with c from -1 to 1 over the
    heads: logits c a(s) + noise.  Rows at or past len hold NaN."""

    def __init__(self, dtype, d, Hkv, G, lens, q_seq, q_pos, slope, seed):
        g = torch.Generator("cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        lens = np.asarray(lens)
        batch, cap, n = len(lens), -(-int(lens.max()) // 16) * 16, int(lens.sum())
        self.dtype, self.d, self.G = dtype, d, G
        self.c = hisa.AttnCache(batch, cap, Hkv, d, dtype, lens=_i32(lens))
        if dtype == "bf16":
            self.c.k.fill_(math.nan), self.c.v.fill_(math.nan)
        else:
            for t, byte in ((self.c.k, 0xFF), (self.c.v, 0xFF), (self.c.k_scale, 0x7F), (self.c.v_scale, 0x7F)):
                t.fill_(byte)
        seq, pos = np.repeat(np.arange(batch), lens), np.concatenate([np.arange(x) for x in lens])
        u = torch.where(torch.randn(d, generator=g, device="cuda") > 0, 1.0, -1.0)
        a = torch.from_numpy(slope * pos / math.sqrt(d)).cuda().float()
        K = torch.randn((n, Hkv, d), generator=g, device="cuda") + a[:, None, None] * u
        V = torch.randn((n, Hkv, d), generator=g, device="cuda")
        hisa.hisa_cache_store(self.c, K.bfloat16(), V.bfloat16(), _i32(seq), _i32(pos))
        self.q_seq, self.q_pos = np.asarray(q_seq), np.asarray(q_pos)
        steep = torch.linspace(-1, 1, G, device="cuda").repeat(Hkv) if G > 1 else torch.ones(Hkv, device="cuda")
        Q = 0.3 * torch.randn((len(q_seq), Hkv * G, d), generator=g, device="cuda") + steep[None, :, None] * u
        self.Q, self.blocks, self.B = Q.bfloat16(), None, 128
        self.rng = rng

    def keep(self, B, m, alike=False):
        """Random kept blocks of every row, in no order (alike: most rows of a chunk keep much the same)."""
        self.B = B
        lists = [self.rng.permutation(t // B + 1)[:m] for t in self.q_pos]
        if alike:
            for i in range(1, len(lists)):
                if self.rng.random() < 0.8:
                    lists[i] = np.where(self.rng.random(len(lists[0])) < 0.9, lists[0], self.rng.integers(0, 20, len(lists[0])))
        self.blocks = np.full((len(lists), m), -1)
        for row, x in zip(self.blocks, lists):
            row[:len(x)] = x

    def tiles(self):
        """Tiles that the rows read one by one (a group's union is never fewer than its longest row's)."""
        per = [len(ref.visible(self.q_pos, self.blocks, self.B, i)) / 128 for i in range(len(self.q_pos))]
        return sum(math.ceil(x) for x in per) * self.c.heads

    def values(self, b, h, n):
        out = []
        for t, s in ((self.c.k, self.c.k_scale), (self.c.v, self.c.v_scale)):
            x = t[b, h, :n]
            out.append(_f64(x) if self.dtype == "bf16" else ref.fp4_values(x.cpu().numpy(), s[b, h, :n].cpu().numpy()))
        return out

    def run_and_check(self, pairs):
        seq, pos = _i32(self.q_seq), _i32(self.q_pos)
        blocks = None if self.blocks is None else _i32(self.blocks)
        out, lse = hisa.hisa_block_attn(self.c, self.Q, seq, pos, blocks, B=self.B)
        o2, l2 = hisa.hisa_block_attn(self.c, self.Q, seq, pos, blocks, B=self.B)
        assert torch.equal(out, o2) and torch.equal(lse, l2) and self.c.status_bits() == 0
        assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
        for i, h in pairs:
            k, v = self.values(self.q_seq[i], h, self.q_pos[i] + 1)
            heads = slice(h * self.G, (h + 1) * self.G)
            r = ref.block_attn(_f64(self.Q[i:i + 1, heads]), k[None, None], v[None, None], [0], self.q_pos[i:i + 1],
                               None if self.blocks is None else self.blocks[i:i + 1], self.B, 1 / math.sqrt(self.d))
            ref.check_block_attn(_f64(out[i:i + 1, heads]), _f64(lse[i:i + 1, heads]), r, self.d, self.dtype == "fp4")


@pytest.mark.parametrize("dtype", ["bf16", "fp4"])
@pytest.mark.parametrize("d,Hkv,G", [(128, 8, 8), (64, 8, 16), (128, 8, 1), (64, 8, 5), (128, 4, 32), (64, 4, 17)])
@pytest.mark.parametrize("B,m", [(128, 0), (128, 26), (16, 190)])
@pytest.mark.parametrize("slope", [0.1, 0.001])
def test_lone_rows(dtype, d, Hkv, G, B, m, slope):
    """A row per sequence, at its end or some way before it; up to 16 heads the lone-row kernel, else the other.  At
    slope 0.1 a head's logits grow by up to 2^18 a tile: without a moving reference they pass bf16's range."""
    rng = np.random.default_rng(G + B)
    lens = rng.integers(3500, 4097, 16)
    at = lens - 1 - np.where(np.arange(16) % 3 == 0, rng.integers(0, 300, 16), 0)
    x = Long(dtype, d, Hkv, G, lens, np.arange(16), at, slope, seed=G + B)
    if m:
        x.keep(B, m)
    assert x.tiles() >= (DEEPEST + 1) * SMS * (2 if dtype == "bf16" and G <= 16 else 1)
    x.run_and_check([(0, 0), (3, Hkv - 1), (7, 1), (11, 2), (15, Hkv - 1)])


@pytest.mark.parametrize("dtype", ["bf16", "fp4"])
@pytest.mark.parametrize("d,Hkv,G,rows", [(128, 2, 8, 160), (64, 2, 3, 420), (128, 1, 128, 12), (64, 3, 16, 80)])
@pytest.mark.parametrize("B,m", [(128, 0), (128, 40), (32, 150)])
@pytest.mark.parametrize("slope", [0.1, 0.001])
def test_chunks(dtype, d, Hkv, G, rows, B, m, slope):
    """The last rows of two sequences, causal: groups of rows over long prefixes or over the union of their lists."""
    lens = np.array([8190, 6001])
    seq = np.repeat([0, 1], rows)
    pos = np.concatenate([np.arange(n - rows, n) for n in lens])
    x = Long(dtype, d, Hkv, G, lens, seq, pos, slope, seed=G + B + rows)
    if m:
        x.keep(B, m, alike=True)
    # groups of 128 // G rows, each reading at least what one of its rows reads
    assert x.tiles() // (128 // G) >= 4 * SMS
    x.run_and_check([(0, 0), (rows - 1, Hkv - 1), (rows, 0), (rows + rows // 2, Hkv - 1), (2 * rows - 1, 0)])


@pytest.mark.parametrize("dtype", ["bf16", "fp4"])
@pytest.mark.parametrize("d,Hkv,G", [(64, 1, 4), (128, 1, 1)])
@pytest.mark.parametrize("n", [1024, 1025])
def test_both_sides_of_the_rows_without_a_plan(dtype, d, Hkv, G, n):
    """Lone rows over whole prefixes: up to 1024 every CTA works the tiles out itself, above it a plan does.  Empty
    sequences and bad rows among them, and the last positions read on the device."""
    rng = np.random.default_rng(n)
    lens = rng.integers(0, 145, 1025)
    lens[:4] = [0, 1, 144, 129]
    lens[rng.integers(0, 1025, 60)] = 0
    seq = rng.permutation(1025)[:n]
    pos = lens[seq] - 1 - rng.integers(0, 3, n)         # some rows before the start, all those of empty sequences bad
    pos[17], pos[n - 1] = lens[seq[17]], 1 << 30        # and some past their prefix
    seq[5] = 1025
    case = Case(dtype, d, Hkv, G, 144, lens, seq, pos, 128, 0, seed=n)
    out, lse = case.call()
    r = case.check(out, lse)
    bad = torch.from_numpy(case.valid < 0).cuda()
    assert 60 < int(bad.sum()) < n // 2 and (out[bad] == 0).all() and torch.isneginf(lse[bad]).all()
    # fewer rows of the same: the other side of 1024, within both sides' tolerances
    some = n // 2
    o2, l2 = hisa.hisa_block_attn(case.c, case.Q[:some].contiguous(), _i32(seq[:some]), _i32(pos[:some]), scale=case.scale)
    ref.check_block_attn(_f64(o2), _f64(l2), {k: v[:some] for k, v in r.items()}, d, dtype == "fp4")
    case.c.clear_status()
    case.valid = np.where((seq >= 0) & (seq < 1025), lens[np.minimum(seq, 1024)] - 1, -1)
    case.check(*case.call(q_pos=None))
