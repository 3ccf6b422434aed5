"""Rotary positions, the attention cache and block attention on the GPU,
against the 64-bit forms of attn_ref (tolerances derived there)."""
import math

import numpy as np
import pytest
import torch

import hierarchical_top_indexer_b200 as hisa
from tests import attn_ref as ref

pytestmark = pytest.mark.gpu


def _bf(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).cuda()


def _f64(t):
    return t.to(torch.float64).cpu().numpy()


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


# ------------------------------------------------------------------- rope

@pytest.mark.parametrize("d,rot,off,layout,rows,heads,scaling", [
    (128, 64, 64, "half", 64, 64, "none"), (128, 64, 0, "interleaved", 33, 17, "yarn"), (64, 64, 0, "half", 1, 1, "none"),
    (64, 32, 16, "half", 499, 5, "ntk"), (64, 20, 6, "half", 31, 3, "linear"), (64, 20, 6, "interleaved", 31, 3, "linear"),
    (64, 20, 7, "interleaved", 31, 3, "none"), (70, 16, 8, "half", 9, 2, "none"), (6, 2, 1, "half", 11, 1, "none"),
    (512, 256, 128, "half", 5, 2, "none"), (128, 128, 0, "half", 700, 1, "none"), (64, 16, 48, "interleaved", 3, 130, "none")])
@pytest.mark.parametrize("transpose", [False, True])
def test_rope(d, rot, off, layout, rows, heads, scaling, transpose):
    rng = np.random.default_rng(d + rot + rows)
    x = _bf(rng.standard_normal((rows, heads, d)))
    pos = rng.integers(-5, 1 << 20, rows)
    pos[0] = (1 << 31) - 1
    if rows > 2:
        pos[1], pos[2] = 0, -(1 << 31)
    kw = dict(scaling=scaling, factor=1.0 if scaling == "none" else 8.0, orig_len=4096)
    plan = hisa.hisa_rope_init(d, rot=rot, off=off, layout=layout, **kw)
    y = hisa.hisa_rope(plan, x, _i32(pos), transpose=transpose)
    gain = 0.1 * math.log(8.0) + 1 if scaling == "yarn" else 1.0
    want = ref.rope(_f64(x), pos, ref.rope_rates(rot, **kw), off, layout, gain, transpose)
    # one rounding to bf16 (2^-8 of the value); the angle is off by 2^-25 of half a turn in
    # fp32, by 2^-53 times the position's angle in the float64 form, the rotation by a few 2^-24
    xa = np.abs(_f64(x)).max(-1, keepdims=True)
    tol = 2.0 ** -8 * np.abs(want) + xa * (2.0 ** -20 + 2.0 ** -50 * np.abs(pos.astype(np.float64))[:, None, None])
    assert (np.abs(_f64(y) - want) <= tol).all()
    keep = np.r_[0:off, off + rot:d]
    assert torch.equal(y[..., keep], x[..., keep])
    z = x.clone()
    assert hisa.hisa_rope(plan, z, _i32(pos), out=z, transpose=transpose) is z and torch.equal(z, y)


def test_rope_gradient_is_the_transpose():
    """<g, J dx> by differences of the 64-bit form equals <J^T g, dx> of the kernel's transpose."""
    rng = np.random.default_rng(7)
    x, dx, pos = rng.standard_normal((6, 2, 64)), rng.standard_normal((6, 2, 64)), rng.integers(0, 9999, 6)
    g = _bf(rng.standard_normal((6, 2, 64)))
    for layout in ("half", "interleaved"):
        plan = hisa.hisa_rope_init(64, rot=32, off=16, layout=layout, gain=1.25)
        f = lambda a: ref.rope(a, pos, ref.rope_rates(32), 16, layout, 1.25)  # noqa: E731,B023
        diff = (f(x + 1e-4 * dx) - f(x - 1e-4 * dx)) / 2e-4
        back = _f64(hisa.hisa_rope(plan, g, _i32(pos), transpose=True))
        tol = (2.0 ** -8 * 1.25 * 1.5 * np.abs(_f64(g)).max() * np.abs(dx)).sum()
        assert abs((_f64(g) * diff).sum() - (back * dx).sum()) <= tol
        t = hisa.hisa_rope(plan, g[:, 0].contiguous(), _i32(pos), transpose=True)      # [rows, d]
        assert torch.equal(t, hisa.hisa_rope(plan, g, _i32(pos), transpose=True)[:, 0])


def test_rope_refuses_an_overlapping_output():
    plan = hisa.hisa_rope_init(64)
    buf = torch.zeros((9, 1, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        hisa.hisa_rope(plan, buf[:8], _i32(np.zeros(8)), out=buf[1:])


# ------------------------------------------------------------------ cache

def _names(rng, n, batch, cap):
    slot = rng.permutation(batch * cap)[:n]
    return slot // cap, slot % cap


@pytest.mark.parametrize("n,heads,d,batch,cap,mul", [(1, 1, 64, 1, 16, 1.0), (65, 3, 128, 4, 48, 1.0), (700, 2, 64, 5, 1008, 0.25),
                                                     (64, 8, 128, 64, 16, 2.0 ** -40)])
def test_cache_rows_in_4_bits(n, heads, d, batch, cap, mul):
    rng = np.random.default_rng(n)
    x = [_bf(rng.standard_normal((n, heads, d)) * np.exp(2 * rng.standard_normal((n, heads, 1))) * mul) for _ in "kv"]
    x[0][0, 0, :16] = 0                                                   # a group of zeros
    seq, pos = _names(rng, n, batch, cap)
    c = hisa.AttnCache(batch, cap, heads, d, "fp4", k_mul=mul, v_mul=mul)
    for t in (c.k, c.v, c.k_scale, c.v_scale):
        t.fill_(0xAB)
    hisa.hisa_cache_store(c, x[0], x[1], _i32(seq), _i32(pos))
    got = hisa.hisa_cache_load(c, _i32(seq), _i32(pos))
    for x_, codes, scales, back in zip(x, (c.k, c.v), (c.k_scale, c.v_scale), got):
        wc, ws, values = ref.fp4_rows(_f64(x_), mul)
        sc, cc = scales.cpu().numpy()[seq, :, pos], codes.cpu().numpy()[seq, :, pos]
        assert np.array_equal(sc, ws)
        assert np.array_equal(ref.fp4_values(cc, sc, mul), values) and np.array_equal(_f64(back), values)
        others = np.ones((batch, cap), bool)
        others[seq, pos] = False
        assert (codes.cpu().numpy().transpose(0, 2, 1, 3)[others] == 0xAB).all()     # nothing else is written
        assert (scales.cpu().numpy().transpose(0, 2, 1, 3)[others] == 0xAB).all()
    assert c.status_bits() == 0


def test_every_tie_and_boundary_of_the_4_bit_rounding():
    """All bf16 significands against all e4m3 significands: 16 x 256 groups whose scale is set by their first element."""
    rows = []
    for s in range(8, 16):                                # scale s / 8 * 2^e
        top = 6 * s / 8.0
        x = np.arange(128, 256) / 128.0
        for e in (-4, -3, -2, -1, 0, 1, 2):
            v = x * 2.0 ** e
            v = v[v <= top]
            for i in range(0, len(v), 15):
                g = np.zeros(16)
                g[0] = top
                g[1:1 + len(v[i:i + 15])] = v[i:i + 15] * np.where(np.arange(len(v[i:i + 15])) % 2, -1, 1)
                rows.append(g)
    rows += [np.zeros(16)] * (-len(rows) % 4)
    x = np.stack(rows).reshape(-1, 1, 64)
    n = len(x)
    c = hisa.AttnCache(1, -(-n // 16) * 16, 1, 64, "fp4")
    seq, pos = _i32(np.zeros(n)), _i32(np.arange(n))
    hisa.hisa_cache_store(c, _bf(x), _bf(-x), seq, pos)
    k, v = hisa.hisa_cache_load(c, seq, pos)
    assert np.array_equal(_f64(_bf(x)), x)
    want = ref.fp4_rows(x)[2]
    assert np.array_equal(_f64(k), want) and np.array_equal(_f64(v), -want)


def test_cache_rows_in_bf16_and_bad_names():
    rng = np.random.default_rng(3)
    K, V = (_bf(rng.standard_normal((6, 2, 64))) for _ in "kv")
    for dtype in ("bf16", "fp4"):
        c = hisa.AttnCache(3, 32, 2, 64, dtype, lens=_i32([5, 0, 32]))
        before = [t.clone() for t in (c.k, c.v)]
        hisa.hisa_cache_store(c, K[:2].contiguous(), V[:2].contiguous(), _i32([-1, 3]), _i32([0, 0]))
        assert c.status_bits() == hisa.HISA_DEV_BAD_QUERY
        c.clear_status()
        hisa.hisa_cache_store(c, K[:3].contiguous(), V[:3].contiguous(), _i32([0, 1, 1]), _i32([32, -1, 1 << 30]))
        assert c.status_bits() == hisa.HISA_DEV_CAPACITY
        assert torch.equal(c.k, before[0]) and torch.equal(c.v, before[1])
        c.clear_status()
        # the last positions: 4, none, 31
        hisa.hisa_cache_store(c, K[:3].contiguous(), V[:3].contiguous(), _i32([0, 1, 2]))
        assert c.status_bits() == hisa.HISA_DEV_CAPACITY
        k, v = hisa.hisa_cache_load(c, _i32([0, 2, 1, 9]), _i32([4, 31, 0, 0]))
        assert c.status_bits() == hisa.HISA_DEV_CAPACITY | hisa.HISA_DEV_BAD_QUERY
        if dtype == "bf16":
            assert torch.equal(k[:2], K[[0, 2]]) and torch.equal(v[:2], V[[0, 2]])
        else:
            assert np.array_equal(_f64(k[:2]), ref.fp4_rows(_f64(K[[0, 2]]))[2])
        assert (k[2:] == 0).all() and (v[2:] == 0).all()


# -------------------------------------------------------------- attention

class Case:
    """A cache with rows past len that hold NaN, queries, kept blocks in no order, with repeats, padding and bad ids."""

    def __init__(self, dtype, d, Hkv, G, cap, lens, q_seq, q_pos, B, m, seed=0, mul=1.0, sharp=1.0):
        rng = np.random.default_rng(seed)
        batch, n = len(lens), len(q_seq)
        K, V = rng.standard_normal((2, batch, Hkv, cap, d)) * mul
        K *= np.exp(0.5 * rng.standard_normal((1, Hkv, 1, d)))
        self.Q = _bf(rng.standard_normal((n, Hkv * G, d)) * sharp / mul)
        past = np.arange(cap)[None, :] >= np.asarray(lens)[:, None]                 # [batch, cap]
        past = np.broadcast_to(past[:, None, :], (batch, Hkv, cap))
        if dtype == "bf16":
            k, v = _bf(K), _bf(V)
            self.K, self.V = _f64(k), _f64(v)
            for t in (k, v):
                t[torch.from_numpy(past.copy()).cuda()] = math.nan
            self.c = hisa.AttnCache.wrap(k, v, _i32(lens))
        else:
            out = []
            for x in (K, V):
                codes, scales, val = ref.fp4_rows(_f64(_bf(x)), mul)
                codes[past], scales[past] = 0xFF, 0x7F                              # an e4m3 NaN
                out += [torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), val]
            self.K, self.V = out[2], out[5]
            self.c = hisa.AttnCache.wrap(out[0], out[3], _i32(lens), k_scale=out[1], v_scale=out[4], k_mul=mul, v_mul=mul)
        self.dtype, self.d, self.B, self.scale = dtype, d, B, 1 / math.sqrt(d)
        self.q_seq, self.q_pos = np.asarray(q_seq), np.asarray(q_pos)
        ok = (self.q_seq >= 0) & (self.q_seq < batch)
        ln = np.where(ok, np.asarray(lens)[np.where(ok, self.q_seq, 0)], 0)
        self.valid = np.where(ok & (self.q_pos >= 0) & (self.q_pos < ln), self.q_pos, -1)
        self.blocks = None
        if m:
            nblk = -(-cap // B)
            self.blocks = rng.integers(0, nblk, (n, m))
            own = rng.random(n) < 0.8
            self.blocks[own, rng.integers(0, m)] = np.maximum(self.valid, 0)[own] // B
            bad = rng.random((n, m))
            self.blocks[bad < 0.1] = -1
            self.blocks[(bad > 0.1) & (bad < 0.15)] = nblk + 7
            self.blocks[(bad > 0.15) & (bad < 0.17)] = (1 << 31) - 1

    def call(self, **kw):
        return hisa.hisa_block_attn(self.c, self.Q, _i32(self.q_seq), kw.pop("q_pos", _i32(self.q_pos)),
                                    None if self.blocks is None else _i32(self.blocks), B=self.B, scale=self.scale, **kw)

    def check(self, out, lse):
        assert self.c.status_bits() == (hisa.HISA_DEV_BAD_QUERY if (self.valid < 0).any() else 0)
        r = ref.block_attn(_f64(self.Q), self.K, self.V, np.where(self.valid < 0, 0, self.q_seq), self.valid, self.blocks,
                           self.B, self.scale)
        assert torch.isfinite(out.float()).all()
        ref.check_block_attn(_f64(out), _f64(lse), r, self.d, self.dtype == "fp4")
        return r


DTYPES = pytest.mark.parametrize("dtype", ["bf16", "fp4"])


@DTYPES
@pytest.mark.parametrize("d,Hkv,G", [(64, 1, 1), (128, 2, 4), (128, 1, 128), (64, 3, 5), (128, 1, 17), (64, 1, 96)])
@pytest.mark.parametrize("B,m", [(128, 0), (128, 5), (64, 9), (8, 40), (16, 3), (32, 31), (256, 2), (384, 3), (1024, 1)])
def test_single_tokens(dtype, d, Hkv, G, B, m):
    """One row per sequence at its last position, lengths from one token on."""
    lens = [1, 700, 129, 128, 1504, 2]
    c = Case(dtype, d, Hkv, G, 1504, lens, [4, 0, 2, 1, 3, 5], [1503, 0, 128, 699, 127, 1], B, m, seed=B + G)
    c.check(*c.call())
    out, lse = c.call(q_pos=None)                       # the last positions, read on the device
    c.check(out, lse)


@DTYPES
@pytest.mark.parametrize("d,Hkv,G", [(128, 2, 8), (64, 1, 3), (64, 2, 1), (128, 1, 128)])
@pytest.mark.parametrize("B,m", [(128, 0), (128, 3), (64, 6), (8, 20), (512, 2)])
def test_chunks(dtype, d, Hkv, G, B, m):
    """More rows than sequences: groups of rows, causal, some of two sequences, some rows bad."""
    n = 23 if G == 128 else 61
    rng = np.random.default_rng(n)
    q_seq = np.sort(rng.integers(0, 2, n))
    q_pos = np.where(q_seq == 0, 640, 300) - rng.permutation(n) % 90
    q_pos[0], q_pos[1], q_pos[2] = 0, -1, 5000
    q_seq[3], q_seq[4] = 2, -3
    c = Case(dtype, d, Hkv, G, 656, [641, 301], q_seq, q_pos, B, m, seed=B + G)
    c.check(*c.call())


@DTYPES
@pytest.mark.parametrize("d,Hkv,G", [(128, 2, 8), (64, 1, 3), (64, 1, 1), (128, 1, 32)])
@pytest.mark.parametrize("B,m", [(128, 3), (64, 6), (16, 9), (384, 1)])
def test_chunks_of_many_rows(dtype, d, Hkv, G, B, m):
    """Enough rows for groups over kept blocks: the union of a group's lists, each row masking what it did not keep."""
    n = max(100, 4 * (128 // G) + 3)
    rng = np.random.default_rng(n + B)
    q_seq = np.sort(rng.integers(0, 2, n))
    q_pos = np.where(q_seq == 0, 640, 300) - rng.integers(0, 300, n)
    q_pos[5], q_pos[6], q_seq[7] = -1, 641, 9
    c = Case(dtype, d, Hkv, G, 656, [641, 301], q_seq, q_pos, B, m, seed=B + G)
    near = rng.random(n) < 0.7                          # neighbours keep much the same blocks, some a list of their own
    c.blocks[near] = c.blocks[0]
    c.blocks[20:30] = -1
    c.check(*c.call())


@DTYPES
def test_rows_of_many_sequences_in_one_group(dtype):
    """Rows in no order of sequences: a group's tiles mix pieces of several."""
    rng = np.random.default_rng(5)
    lens = [40, 1, 130, 0, 64, 17, 99]
    q_seq = rng.integers(0, 7, 460)
    q_pos = np.maximum(np.asarray(lens)[q_seq] - 1 - rng.integers(0, 3, 460), 0)
    for B, m in ((128, 0), (16, 4), (8, 9)):
        c = Case(dtype, 64, 1, 4, 144, lens, q_seq, q_pos, B, m, seed=B)
        c.check(*c.call())


@DTYPES
def test_long_prefixes_split_over_the_ctas(dtype):
    """A few rows over a long prefix (parts of a row joined), and more tiles than CTAs with ragged ends."""
    for lens, seed in (([20011], 1), ([20011, 3, 9000], 2)):
        n = len(lens)
        c = Case(dtype, 128, 2, 4, 20016, lens, np.arange(n), np.asarray(lens) - 1, 128, 0, seed=seed)
        c.check(*c.call())


@DTYPES
def test_empty_lists_and_sequences(dtype):
    c = Case(dtype, 64, 2, 2, 256, [256, 0, 100], [0, 1, 2, 0], [255, 0, 99, 10], 64, 4, seed=3)
    c.blocks[:] = -1
    c.blocks[2] = [1, 1, 1, 1]
    c.blocks[3] = [2, 1, 3, -1]                         # all past the row's position
    out, lse = c.call()
    c.check(out, lse)
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all() and (out[3] == 0).all()
    c.blocks[2] = -1                                    # nothing at all to read
    c.c.clear_status()
    out, lse = c.call()
    assert (out == 0).all() and torch.isneginf(lse).all()
    assert hisa.hisa_block_attn(c.c, c.Q[:0], _i32([]), None)[0].shape == (0, 4, 64)


@DTYPES
@pytest.mark.parametrize("sharp", [1e-3, 30.0])
def test_flat_and_sharp_weights(dtype, sharp):
    """Nearly equal weights, and one weight near 1 whose maximum keeps growing along the prefix."""
    c = Case(dtype, 128, 1, 8, 3008, [3000], [0], [2999], 128, 0, seed=9, sharp=sharp)
    k = torch.linspace(0.1, 3.0, 3008, device="cuda")[None, None, :, None]
    if dtype == "bf16":
        c.c.k[:, :, :3000] = (c.c.k * k)[:, :, :3000].to(torch.bfloat16)
        c.K = np.nan_to_num(_f64(c.c.k))
    c.check(*c.call())


def test_powers_of_two_scale_a_4_bit_cache():
    for mul in (2.0 ** -20, 2.0 ** 20):
        c = Case("fp4", 128, 1, 4, 512, [500], [0, 0, 0], [499, 17, 0], 128, 0, seed=4, mul=mul)
        c.check(*c.call())


@DTYPES
def test_given_buffers_streams_and_graphs(dtype):
    c = Case(dtype, 128, 2, 8, 2048, [2048, 1000, 1500], [0, 1, 2], [2047, 999, 1499], 64, 6, seed=6)
    n, Hq = c.Q.shape[:2]
    ws = hisa.workspace(hisa.hisa_block_attn_workspace_bytes(c.c, n, Hq, 64, 6))
    ws.fill_(0xFF)                                      # nothing in it needs to start at zero
    out = torch.full((n, Hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n, Hq), 7.0, device="cuda")
    a, b = c.call(ws=ws, out=out, lse=lse)
    assert a is out and b is lse
    c.check(out, lse)
    first = out.clone(), lse.clone()
    for _ in range(3):                                  # the same bits every time, back to back
        c.call(ws=ws, out=out, lse=lse)
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    o2, l2 = c.call(stream=other)
    other.synchronize()
    assert torch.equal(o2, first[0]) and torch.equal(l2, first[1])
    seq, pos, blk = _i32(c.q_seq), _i32(c.q_pos), _i32(c.blocks)
    call = lambda: hisa.hisa_block_attn(c.c, c.Q, seq, pos, blk, B=64, scale=c.scale, ws=ws, out=out, lse=lse)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first[0])
    pos.sub_(1)                                         # the replay reads its inputs anew
    graph.replay()
    torch.cuda.synchronize()
    c.valid = c.valid - 1
    c.check(out, lse)
    guard = torch.full((n + 1, Hq, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    hisa.hisa_block_attn(c.c, c.Q, seq, pos, blk, B=64, scale=c.scale, out=guard[:n])
    assert (guard[n] == 5).all()                        # rows behind the last stay


@DTYPES
def test_rows_of_one_sequence_alone(dtype):
    """No more rows than sequences, yet several of one sequence: each row alone."""
    c = Case(dtype, 128, 2, 4, 640, [640, 500, 1], [0, 0, 0], [639, 100, 0], 64, 5, seed=8)
    c.check(*c.call())


@DTYPES
def test_two_calls_at_once(dtype):
    """Two streams, a workspace each, on one cache; then both replayed as graphs that share a workspace in turn."""
    one = Case(dtype, 128, 2, 8, 4096, [4096, 3000], [0, 1], [4095, 2999], 64, 20, seed=12)
    two = Case(dtype, 128, 2, 8, 4096, [4096, 3000], np.repeat([0, 1], 100), np.r_[3900:4000, 2900:3000], 64, 20, seed=12)
    two.c, two.K, two.V = one.c, one.K, one.V
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(10):
        outs = [x.call(stream=s) for x, s in zip((one, two), streams)]
    torch.cuda.synchronize()
    for x, (out, lse) in zip((one, two), outs):
        x.check(out, lse)
    size = lambda x: hisa.hisa_block_attn_workspace_bytes(x.c, x.Q.shape[0], 16, 64, 20)  # noqa: E731
    ws = hisa.workspace(max(size(one), size(two)))
    args = [(x, _i32(x.q_seq), _i32(x.q_pos), _i32(x.blocks)) for x in (one, two)]
    graphs, got = [], []
    for x, seq, pos, blk in args:
        run = lambda: hisa.hisa_block_attn(x.c, x.Q, seq, pos, blk, B=64, scale=x.scale, ws=ws)  # noqa: E731,B023
        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(run())
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for (out, lse), (o2, l2) in zip(outs, got):
        assert torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("dtype,d,cap,B", [("bf16", 128, 9_000_000, 128), ("fp4", 128, 34_000_000, 256), ("bf16", 64, 1 << 23, 8)])
def test_offsets_past_32_bits(dtype, d, cap, B):
    """Rows whose bytes lie past 2^31 from the cache's start (and 2^20 blocks in a sequence): stored, read back, attended to."""
    c = hisa.AttnCache(1, cap, 1, d, dtype, lens=_i32([cap]))
    rng = np.random.default_rng(1)
    last = (cap - 1) // B
    blocks = np.array([[last, last - 2, 0, last // 2]])
    tok = np.concatenate([np.arange(j * B, min((j + 1) * B, cap)) for j in blocks[0]])
    K, V = (_bf(rng.standard_normal((len(tok), 1, d))) for _ in "kv")
    seq = _i32(np.zeros(len(tok)))
    hisa.hisa_cache_store(c, K, V, seq, _i32(tok))
    k, v = hisa.hisa_cache_load(c, seq, _i32(tok))
    Q = _bf(rng.standard_normal((1, 4, d)))
    order = np.argsort(tok)
    near = [np.array_equal(_f64(a), _f64(b) if dtype == "bf16" else ref.fp4_rows(_f64(b))[2]) for a, b in ((k, K), (v, V))]
    assert all(near)
    r = ref.block_attn(_f64(Q), _f64(k)[order].swapaxes(0, 1)[None], _f64(v)[order].swapaxes(0, 1)[None], [0], [len(tok) - 1], None, 1,
                       1 / math.sqrt(d))
    out, lse = hisa.hisa_block_attn(c, Q, _i32([0]), None, _i32(blocks), B=B)
    ref.check_block_attn(_f64(out), _f64(lse), r, d, dtype == "fp4")
    # 120 rows of one sequence: the other kernel
    out, lse = hisa.hisa_block_attn(c, Q.repeat(120, 1, 1), _i32(np.zeros(120)), None, _i32(blocks.repeat(120, 0)), B=B)
    r = {x: np.repeat(y, 120, 0) for x, y in r.items()}
    ref.check_block_attn(_f64(out), _f64(lse), r, d, dtype == "fp4")
    assert c.status_bits() == 0


def test_scales_at_the_ends_of_their_range():
    c = Case("fp4", 64, 1, 2, 64, [64], [0], [63], 128, 0, seed=2)
    c.c._struct.k_mul = 2.0 ** 60
    with pytest.raises(hisa.HisaError) as e:
        hisa.hisa_block_attn(c.c, c.Q, _i32([0]), scale=1e30)
    assert e.value.code == hisa.HISA_E_INVAL
    c.c._struct.k_mul = 1.0
    for scale in (1e-30, 1e-3, 40.0):
        c.scale = scale
        c.check(*c.call())
    c = Case("fp4", 128, 1, 3, 256, [256], [0], [255], 128, 0, seed=2)
    for size in (2.0 ** -120, 2.0 ** 100):               # queries far from 1, brought back by the scale
        q = c.Q
        c.Q, c.scale = (q.double() * size).to(torch.bfloat16), 1 / (math.sqrt(128) * size)
        if size > 1 or c.scale < 3e38:
            c.check(*c.call())
        c.Q = q


# --------------------------------------------------------------- together

@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("m", [4, 100])
@pytest.mark.parametrize("n_q", [4, 600])
def test_select_blocks_is_stage_one(m, n_q, dtype):
    from hisa_inputs import make_case
    rng = np.random.default_rng(n_q)
    case = make_case(batch=2, L=[4096, 3000], H=16, d=128, B=64, m=m, k=64, seed=3, dtype=dtype,
                     positions=[np.sort(rng.integers(0, 4096, n_q // 2)), np.sort(rng.integers(0, 3000, n_q // 2))])
    kv = hisa.KVCache.from_case(case)
    hisa.hisa_pool_blocks(kv)
    dev = lambda x, dt: torch.from_numpy(x.view(np.int16) if x.dtype == np.uint16 else x).cuda().view(dt)  # noqa: E731
    Q, w = dev(case.Q, torch.bfloat16), dev(case.w, torch.float32)
    seq, pos = dev(case.q_seq, torch.int32), dev(case.q_pos, torch.int32)
    want = hisa.hisa_select_inspect(kv, Q, w, seq, pos, m, 64)
    blocks, counts = hisa.hisa_select_blocks(kv, Q, w, seq, pos, m, want_counts=True)
    assert torch.equal(blocks, want["blocks"]) and torch.equal(counts, want["nblocks"])
    pos[0] = 1 << 20
    bad, counts = hisa.hisa_select_blocks(kv, Q, w, seq, pos, m, want_counts=True)
    assert (bad[0] == -1).all() and int(counts[0]) == 0 and torch.equal(bad[1:], want["blocks"][1:])
    assert kv.status_bits() == hisa.HISA_DEV_BAD_QUERY


@DTYPES
def test_decode_steps_with_a_shared_length(dtype):
    """A few decode steps as a model runs them: positions on the indexer's and the attention's queries and keys, the
    indexer key appended, its blocks selected, key and value rows stored, attention over the blocks.  Each step is
    checked against the 64-bit attention over everything stored so far."""
    rng = np.random.default_rng(11)
    batch, cap, H, Hq, Hkv, B, m = 3, 512, 16, 8, 2, 64, 3
    kv = hisa.KVCache(batch, cap, 128, B)
    c = hisa.AttnCache(batch, cap, Hkv, 128, dtype, lens=kv.len, status=kv.status)
    start = np.array([300, 0, 63])
    irope, arope = hisa.hisa_rope_init(128, rot=64, off=64, layout="interleaved"), hisa.hisa_rope_init(128)
    total = int(start.sum())
    seq = np.repeat(np.arange(batch), start)
    pos = np.concatenate([np.arange(s) for s in start])
    ik = hisa.hisa_rope(irope, _bf(rng.standard_normal((total, 128)) / 8), _i32(pos))
    kv.keys[torch.from_numpy(seq).cuda(), torch.from_numpy(pos).cuda()] = ik
    kv.len.copy_(_i32(start))
    hisa.hisa_pool_blocks(kv)
    K, V = (_bf(rng.standard_normal((total, Hkv, 128))) for _ in "kv")
    hisa.hisa_cache_store(c, hisa.hisa_rope(arope, K, _i32(pos)), V, _i32(seq), _i32(pos))
    rows = _i32(np.arange(batch))
    for step in range(3):
        at = kv.len.clone()                            # the new token's positions
        tok = hisa.hisa_rope(irope, _bf(rng.standard_normal((batch, 128)) / 8), at)
        Qi = hisa.hisa_rope(irope, _bf(rng.standard_normal((batch, H, 128))), at)
        Qa, K1 = (hisa.hisa_rope(arope, _bf(rng.standard_normal((batch, h, 128))), at) for h in (Hq, Hkv))
        V1 = _bf(rng.standard_normal((batch, Hkv, 128)))
        w = torch.from_numpy(rng.random((batch, H), np.float32)).cuda()
        hisa.hisa_append(kv, tok)
        blocks = hisa.hisa_select_blocks(kv, Qi, w, rows, None, m)
        hisa.hisa_cache_store(c, K1, V1, rows)
        out, lse = hisa.hisa_block_attn(c, Qa, rows, None, blocks, B=B)
        n = kv.len.cpu().numpy()
        assert (n == start + step + 1).all() and kv.status_bits() == 0
        Kf, Vf = np.zeros((2, batch, Hkv, cap, 128))
        for b in range(batch):
            k, v = hisa.hisa_cache_load(c, _i32(np.full(n[b], b)), _i32(np.arange(n[b])))
            Kf[b, :, :n[b]], Vf[b, :, :n[b]] = _f64(k).swapaxes(0, 1), _f64(v).swapaxes(0, 1)
            last = _f64(K1[b]) if dtype == "bf16" else ref.fp4_rows(_f64(K1[b]))[2]
            assert np.array_equal(Kf[b, :, n[b] - 1], last)
        r = ref.block_attn(_f64(Qa), Kf, Vf, np.arange(batch), n - 1, blocks.cpu().numpy(), B, 1 / math.sqrt(128))
        ref.check_block_attn(_f64(out), _f64(lse), r, 128, dtype == "fp4")
