"""Refusals of rotary positions, the attention cache and block attention: the
library's host checks (no CUDA call is possible on a machine without a GPU, so
reaching one would give HISA_E_CUDA) and the binding's."""
import ctypes
import math

import pytest
import torch

import hierarchical_top_indexer_b200 as hisa
from tests import attn_ref as ref

P = ctypes.c_void_p


def _kv(**over):
    f = dict(k=256, v=512, k_scale=None, v_scale=None, len=64, status=128, batch=2, cap=4096, heads=2, d=128, dtype=0,
             k_mul=1.0, v_mul=1.0)
    f.update(over)
    return hisa.hisa_attn_kv(**f)


def _fp4(**over):
    return _kv(**{**dict(dtype=1, k_scale=1024, v_scale=2048), **over})


def _attn(c, Qa=P(16), Hq=16, q_seq=P(16), q_pos=None, n_q=4, blocks=P(16), mb=8, B=128, scale=0.1, out=P(16), lse=None,
          ws=P(256), ws_bytes=1 << 40):
    return hisa.lib().hisa_block_attn(ctypes.byref(c) if c else None, Qa, Hq, q_seq, q_pos, n_q, blocks, mb, B, scale, out,
                                      lse, ws, ws_bytes, None)


@pytest.mark.parametrize("bad", [dict(k=None), dict(v=None), dict(len=None), dict(batch=0), dict(cap=0), dict(heads=0),
                                 dict(dtype=2), dict(k=264), dict(len=66), dict(status=130)])
def test_cache_descriptor_is_checked(bad):
    for make in (_kv, _fp4):
        c = make(**bad)
        assert _attn(c) == hisa.HISA_E_INVAL
        assert hisa.lib().hisa_cache_store(ctypes.byref(c), P(16), P(16), P(16), None, 1, None) == hisa.HISA_E_INVAL
        assert hisa.lib().hisa_block_attn_workspace_bytes(ctypes.byref(c), 4, 16, 128, 8) == 0


def test_fp4_descriptor_is_checked():
    for bad in (dict(k_scale=None), dict(v_scale=None), dict(k_scale=1032), dict(k_mul=3.0), dict(v_mul=0.0),
                dict(v_mul=-1.0), dict(k_mul=math.inf), dict(k_mul=2.0 ** 61), dict(v_mul=2.0 ** -61)):
        assert _attn(_fp4(**bad)) == hisa.HISA_E_INVAL, bad
    assert _attn(_fp4(cap=4100)) == hisa.HISA_E_UNSUPPORTED
    assert _attn(_kv(d=96)) == hisa.HISA_E_UNSUPPORTED
    assert _attn(_kv(batch=1 << 23)) == hisa.HISA_E_UNSUPPORTED
    for ok in (dict(k_mul=2.0 ** 60), dict(v_mul=2.0 ** -60), dict(k_mul=0.5)):
        assert _attn(_fp4(**ok), n_q=0) == hisa.HISA_OK


def test_block_attn_arguments():
    c = _kv()
    assert _attn(None) == hisa.HISA_E_INVAL
    for bad in (dict(Qa=None), dict(Qa=P(8)), dict(q_seq=None), dict(q_seq=P(18)), dict(q_pos=P(18)), dict(out=None),
                dict(out=P(8)), dict(lse=P(18)), dict(blocks=P(18)), dict(n_q=-1), dict(mb=-1), dict(Hq=0), dict(Hq=15),
                dict(blocks=None), dict(mb=0), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf),
                dict(scale=math.nan)):
        assert _attn(c, **bad) == hisa.HISA_E_INVAL, bad
    assert _attn(c, Hq=2 * 129) == hisa.HISA_E_UNSUPPORTED
    for B in (0, 1, 4, 12, 96, 100, 1152):
        assert _attn(c, B=B) == hisa.HISA_E_UNSUPPORTED, B
    assert _attn(_kv(cap=(1 << 23) + 8, batch=1), B=8) == hisa.HISA_E_UNSUPPORTED   # over 2^20 blocks
    assert _attn(c, ws=None) == hisa.HISA_E_WORKSPACE
    assert _attn(c, ws=P(128)) == hisa.HISA_E_WORKSPACE
    need = hisa.lib().hisa_block_attn_workspace_bytes(ctypes.byref(c), 4, 16, 128, 8)
    assert need > 0 and _attn(c, ws_bytes=need - 1) == hisa.HISA_E_WORKSPACE
    assert _attn(c, n_q=0, Qa=None, ws=None, ws_bytes=0) == hisa.HISA_OK
    # the whole prefix does not read B
    assert _attn(c, n_q=0, blocks=None, mb=0, B=0) == hisa.HISA_OK


def test_cache_rows_arguments():
    lib, c = hisa.lib(), _fp4()
    for fn in (lib.hisa_cache_store, lib.hisa_cache_load):
        call = lambda K=P(16), V=P(16), seq=P(16), pos=P(16), n=3: fn(ctypes.byref(c), K, V, seq, pos, n, None)  # noqa: E731,B023
        assert call(K=None) == call(V=None) == call(seq=None) == call(n=-1) == hisa.HISA_E_INVAL
        assert call(K=P(8)) == call(V=P(24)) == call(seq=P(2)) == call(pos=P(2)) == hisa.HISA_E_INVAL
        assert call(n=0, K=None) == hisa.HISA_OK
        assert fn(None, P(16), P(16), P(16), None, 1, None) == hisa.HISA_E_INVAL


def test_select_blocks_arguments():
    lib = hisa.lib()
    kv = hisa.hisa_kv(keys=16, key_scale=None, pooled=32, pooled_hl=48, len=64, status=128, batch=1, cap=4096, d=128, B=128,
                      dtype=0)
    call = lambda Q=P(16), w=P(16), s=P(16), pos=None, n=4, H=64, m=8, out=P(16), nb=None, ws=P(256), size=1 << 30: \
        lib.hisa_select_blocks(ctypes.byref(kv), Q, w, s, pos, n, H, m, out, nb, ws, size, None)  # noqa: E731
    assert call(Q=None) == call(w=None) == call(s=None) == call(out=None) == call(m=0) == hisa.HISA_E_INVAL
    assert call(pos=P(2)) == call(nb=P(2)) == call(Q=P(8)) == hisa.HISA_E_INVAL
    assert call(H=0) == call(H=129) == hisa.HISA_E_UNSUPPORTED
    assert call(ws=None) == call(ws=P(128)) == call(size=16) == hisa.HISA_E_WORKSPACE
    assert call(n=0, Q=None) == hisa.HISA_OK
    ws = lib.hisa_select_blocks_workspace_bytes(ctypes.byref(kv), 4, 64, 8)
    assert 0 < ws < lib.hisa_select_workspace_bytes(ctypes.byref(kv), 4, 64, 8, 64)
    assert lib.hisa_select_blocks_workspace_bytes(ctypes.byref(kv), 4, 64, 0) == 0


@pytest.mark.parametrize("bad", [dict(d=1), dict(d=514), dict(rot=0), dict(rot=7), dict(rot=66), dict(off=-1), dict(off=1),
                                 dict(base=1.0), dict(base=math.inf), dict(factor=0.5), dict(factor=math.nan),
                                 dict(gain=math.inf), dict(scaling="yarn"), dict(scaling="yarn", orig_len=4096, beta_slow=0),
                                 dict(scaling="yarn", orig_len=4096, beta_fast=0.5), dict(d=512, rot=258),
                                 dict(scaling="ntk", rot=2, factor=2.0)])
def test_rope_plans_are_checked(bad):
    with pytest.raises(hisa.HisaError) as e:
        hisa.hisa_rope_init(**{**dict(d=64, rot=64), **bad})
    assert e.value.code == hisa.HISA_E_INVAL


def test_rope_names_are_checked():
    for bad in (dict(layout="both"), dict(scaling="linear ")):
        with pytest.raises(ValueError):
            hisa.hisa_rope_init(64, **bad)


@pytest.mark.parametrize("rot,scaling,factor", [(64, "none", 1.0), (128, "linear", 8.0), (32, "ntk", 4.0), (64, "yarn", 16.0),
                                                (2, "none", 1.0), (256, "yarn", 40.0), (64, "yarn", 1.0)])
def test_rope_rates(rot, scaling, factor):
    """The plan's turns are the rates / 2 pi in 64-bit fixed point, and the gain the scaling's own.  The fixed point
    itself is off by up to half its step of 2^-64, the float64 rates by a few of their own 2^-53."""
    p = hisa.hisa_rope_init(max(rot, 64), rot=rot, base=10000.0, scaling=scaling, factor=factor, orig_len=8192)
    w = ref.rope_rates(rot, 10000.0, scaling, factor, 8192)
    for i, x in enumerate(w):
        assert abs(p.turns[i] / 2.0 ** 64 - x / (2 * math.pi)) <= 4 * 2.0 ** -53 * x + 2.0 ** -65
    assert all(p.turns[i] == 0 for i in range(rot // 2, hisa.HISA_ROPE_MAX_PAIRS))
    assert abs(p.gain - (0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0)) < 1e-6
    assert hisa.hisa_rope_init(max(rot, 64), rot=rot, scaling=scaling, factor=factor, orig_len=8192, gain=0.75).gain == 0.75


def test_rope_arguments():
    lib, p = hisa.lib(), hisa.hisa_rope_init(64)
    call = lambda plan=p, x=P(16), y=P(16), pos=P(16), rows=4, heads=2: \
        lib.hisa_rope(ctypes.byref(plan) if plan else None, x, y, pos, rows, heads, 0, None)  # noqa: E731
    assert call(plan=None) == call(plan=hisa.hisa_rope_plan()) == hisa.HISA_E_INVAL
    assert call(x=None) == call(y=None) == call(pos=None) == call(x=P(8)) == call(y=P(8)) == call(pos=P(2)) == hisa.HISA_E_INVAL
    assert call(rows=-1) == call(heads=0) == hisa.HISA_E_INVAL
    assert call(rows=0, x=None) == hisa.HISA_OK


def test_the_binding_refuses_tensors_the_call_cannot_read():
    k = torch.zeros((2, 2, 64, 64), dtype=torch.bfloat16)
    lens = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        hisa.AttnCache.wrap(k, k[:, :1].clone(), lens)
    with pytest.raises(ValueError):
        hisa.AttnCache.wrap(k, k, lens.long())
    with pytest.raises(ValueError):
        hisa.AttnCache.wrap(k, k, lens, k_scale=lens)
    with pytest.raises(ValueError):
        hisa.AttnCache.wrap(k.transpose(1, 2), k.transpose(1, 2), lens)
    with pytest.raises(ValueError):
        hisa.AttnCache.wrap(k.view(torch.uint8), k.view(torch.uint8), lens, k_scale=lens, v_scale=lens)
    with pytest.raises(ValueError):
        hisa.AttnCache(2, 64, 2, 64, "int4", device="cpu")
    c = hisa.AttnCache.wrap(k, k, lens)
    q, seq = torch.zeros((3, 4, 64), dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    for bad in (dict(Qa=q.float()), dict(Qa=q[..., :32]), dict(q_seq=seq[:2]), dict(q_seq=seq.long()), dict(q_pos=seq[:1]),
                dict(blocks=seq), dict(blocks=torch.zeros((3, 0), dtype=torch.int32)),
                dict(blocks=torch.zeros((2, 4), dtype=torch.int32))):
        with pytest.raises(ValueError):
            hisa.hisa_block_attn(c, **{**dict(Qa=q, q_seq=seq), **bad})
    rows = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    for bad in (dict(K=rows[:2]), dict(V=rows.float()), dict(seq=seq.long()), dict(pos=seq[:2])):
        with pytest.raises(ValueError):
            hisa.hisa_cache_store(c, **{**dict(K=rows, V=rows, seq=seq), **bad})
    with pytest.raises(ValueError):
        hisa.hisa_rope(hisa.hisa_rope_init(64), rows, seq)      # not a CUDA tensor


def test_outputs_that_overlap_their_inputs_are_refused():
    c = _kv()
    size = 4 * 16 * 128 * 2   # n_q rows of Hq heads
    for out in (1 << 20, (1 << 20) + size - 16, (1 << 20) - size + 16):
        assert _attn(c, Qa=P(1 << 20), out=P(out)) == hisa.HISA_E_INVAL, out
    lib, p = hisa.lib(), hisa.hisa_rope_init(64)
    size = 4 * 2 * 64 * 2
    for y in ((1 << 20) + 16, (1 << 20) + size - 16, (1 << 20) - size + 16):
        assert lib.hisa_rope(ctypes.byref(p), P(1 << 20), P(y), P(16), 4, 2, 0, None) == hisa.HISA_E_INVAL, y


def test_a_gain_past_fp32_is_refused():
    with pytest.raises(hisa.HisaError) as e:
        hisa.hisa_rope_init(64, gain=1e39)
    assert e.value.code == hisa.HISA_E_INVAL


def test_an_empty_batch_with_kept_blocks_is_no_error():
    """A tensor without elements has no address: hisa_select_blocks of no rows gives such a list."""
    assert torch.zeros((0, 8), dtype=torch.int32).data_ptr() == 0
    for c in (_kv(), _fp4()):
        assert _attn(c, n_q=0, blocks=None, mb=8, Qa=None, q_seq=None, out=None, ws=None, ws_bytes=0) == hisa.HISA_OK
        assert _attn(c, n_q=0, blocks=None, mb=8, B=12) == hisa.HISA_E_UNSUPPORTED     # sizes are checked all the same
        assert _attn(c, n_q=1, blocks=None, mb=8) == hisa.HISA_E_INVAL


def test_lists_longer_than_the_plan_counts_are_refused():
    """The plan counts the entries of up to 128 rows in an int and steps 256 at a time: 128 * mb + 256 < 2^31."""
    most = (1 << 24) - 4
    assert 128 * most + 256 < 1 << 31 <= 128 * (most + 4) + 256
    for make in (_kv, _fp4):
        for Hq in (2, 16, 256):
            size = lambda mb: hisa.lib().hisa_block_attn_workspace_bytes(ctypes.byref(make()), 1, Hq, 128, mb)  # noqa: E731,B023
            assert size(most) > 0
            for mb in (most + 1, (1 << 31) - 200, (1 << 31) - 1):
                assert size(mb) == 0 and _attn(make(), Hq=Hq, n_q=1, mb=mb) == hisa.HISA_E_UNSUPPORTED, mb


def _apart(make):
    """A cache whose rows and scales lie apart: k from 16 MB on, v 32 MB further, the scales behind."""
    mb = 1 << 20
    over = dict(k=16 * mb, v=48 * mb, len=64, status=128)
    if make is _fp4:
        over.update(k_scale=80 * mb, v_scale=96 * mb)
    return make(**over)


def test_rows_inside_the_cache_are_refused():
    mb, lib, free = 1 << 20, hisa.lib(), P(128 << 20)
    size = 3 * 2 * 128 * 2                                       # n tokens of heads rows
    for make in (_kv, _fp4):
        c = _apart(make)
        rows = 2 * 2 * 4096 * (256 if make is _kv else 64)
        inside = [16 * mb, 16 * mb + rows - 16, 16 * mb - size + 16, 48 * mb, 48 * mb + rows - 16]
        if make is _fp4:
            scales = 2 * 2 * 4096 * 128 // 16
            inside += [80 * mb, 80 * mb + scales - 16, 96 * mb - size + 16, 96 * mb + scales - 16]
        for fn in (lib.hisa_cache_store, lib.hisa_cache_load):
            for at in inside:
                assert fn(ctypes.byref(c), P(at), free, P(64), None, 3, None) == hisa.HISA_E_INVAL, at
                assert fn(ctypes.byref(c), free, P(at), P(64), None, 3, None) == hisa.HISA_E_INVAL, at


def test_loaded_keys_and_values_that_overlap_are_refused():
    """Where nothing overlaps the call goes on to the launch, which fails on a machine without a GPU."""
    at, size, lib = 128 << 20, 3 * 2 * 128 * 2, hisa.lib()
    for make in (_kv, _fp4):
        c = _apart(make)
        for v in (at, at + size - 16, at - size + 16):
            assert lib.hisa_cache_load(ctypes.byref(c), P(at), P(v), P(64), None, 3, None) == hisa.HISA_E_INVAL, v
        if not torch.cuda.is_available():                        # next to one another, and the same rows stored twice
            for fn, v in ((lib.hisa_cache_load, at + size), (lib.hisa_cache_load, at - size), (lib.hisa_cache_store, at)):
                assert fn(ctypes.byref(c), P(at), P(v), P(64), None, 3, None) == hisa.HISA_E_CUDA, v


def test_outputs_that_overlap_each_other_or_the_cache_are_refused():
    mb, size, lse = 1 << 20, 4 * 16 * 128 * 2, 4 * 16 * 4           # n_q rows of Hq heads
    at, far = 128 * mb, 256 * mb
    for make in (_kv, _fp4):
        c = _apart(make)
        call = lambda **kw: _attn(c, **{**dict(Qa=P(at), out=P(far), lse=P(64 * mb + far)), **kw})  # noqa: E731,B023
        for x in (at, at + size - 4, at - lse + 4):
            assert call(lse=P(x)) == hisa.HISA_E_INVAL, x
        for x in (far, far + size - 4, far - lse + 4):
            assert call(lse=P(x)) == hisa.HISA_E_INVAL, x
        for x in (16 * mb, 48 * mb) + (() if make is _kv else (80 * mb, 96 * mb)):
            assert call(out=P(x)) == call(out=P(x - size + 16)) == call(lse=P(x)) == call(lse=P(x - 4)) == hisa.HISA_E_INVAL
        if not torch.cuda.is_available():                        # next to one another: the call goes on to the device
            assert call(lse=P(far + size)) == call(lse=P(at - lse)) == call(lse=None) == hisa.HISA_E_CUDA


def test_a_gain_below_fp32_is_refused():
    """It would come out as 0 (or lose bits), which as an argument stands for the scaling's own gain."""
    for gain in (1e-46, -1e-60, 1e-39):
        with pytest.raises(hisa.HisaError) as e:
            hisa.hisa_rope_init(64, gain=gain)
        assert e.value.code == hisa.HISA_E_INVAL
    for gain in (2.0 ** -126, -3.0, 3e38):
        assert hisa.hisa_rope_init(64, gain=gain).gain == torch.tensor(gain, dtype=torch.float32).item()


@pytest.mark.parametrize("field,value", [("d", 62), ("d", 513), ("rot", 0), ("rot", 63), ("rot", 258), ("off", -1), ("off", 1),
                                         ("layout", 2), ("layout", -1), ("ready", 0), ("ready", 2)])
def test_a_plan_that_was_written_over_is_refused(field, value):
    """A plan is plain memory; one whose sizes or layout hisa_rope_init would have refused is refused by the call too
    (an odd rot left an element of y unwritten, an unknown layout ran as HALF)."""
    p = hisa.hisa_rope_init(64)
    setattr(p, field, value)
    assert hisa.lib().hisa_rope(ctypes.byref(p), P(16), P(16), P(16), 4, 2, 0, None) == hisa.HISA_E_INVAL
