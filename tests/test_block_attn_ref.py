"""The 64-bit forms the GPU tests compare with, against closed forms and torch."""
import math

import numpy as np
import torch

from tests import attn_ref as ref


def test_fp4_rows_are_the_nearest_codes():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((40, 64)) * np.exp(rng.standard_normal((40, 64)))
    x = torch.from_numpy(x).to(torch.bfloat16).to(torch.float64).numpy()
    codes, scales, values = ref.fp4_rows(x)
    assert np.array_equal(ref.fp4_values(codes, scales), values)
    s = np.repeat(torch.from_numpy(scales).view(torch.float8_e4m3fn).to(torch.float64).numpy(), 16, -1)
    grid = np.concatenate([ref.E2M1, -ref.E2M1])
    best = np.abs(x[..., None] - s[..., None] * grid).min(-1)
    assert np.allclose(np.abs(x - values), best, rtol=0, atol=1e-15)


def test_fp4_ties_go_to_the_even_code():
    x = np.zeros((1, 16))
    x[0, :9] = [6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.0]     # scale 1
    _, _, v = ref.fp4_rows(x)
    assert v[0, :9].tolist() == [6.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, -4.0]


def test_fp4_zero_group_and_saturation():
    x = np.zeros((1, 32))
    x[0, 16:] = 1e5
    codes, scales, v = ref.fp4_rows(x)
    assert scales[0, 0] == 0 and (v[0, :16] == 0).all() and (v[0, 16:] == 6 * 448).all()


def test_rope_is_a_rotation_and_its_transpose_undoes_it():
    rng = np.random.default_rng(1)
    x, pos = rng.standard_normal((7, 3, 32)), np.arange(-3, 4) * 1000
    w = ref.rope_rates(16)
    for layout in ("half", "interleaved"):
        y = ref.rope(x, pos, w, 8, layout)
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
        assert np.allclose(ref.rope(y, pos, w, 8, layout, transpose=True), x)
        assert np.array_equal(y[..., :8], x[..., :8]) and np.array_equal(y[..., 24:], x[..., 24:])
    assert w[0] == 1.0 and math.isclose(w[1], 10000 ** (-1 / 8))


def test_block_attn_equals_torch_on_a_causal_prefix():
    rng = np.random.default_rng(2)
    Q, K, V = rng.standard_normal((5, 4, 16)), rng.standard_normal((1, 2, 20, 16)), rng.standard_normal((1, 2, 20, 16))
    pos = np.arange(15, 20)
    r = ref.block_attn(Q, K, V, np.zeros(5, int), pos, None, 0, 0.25)
    mask = torch.arange(20)[None] <= torch.from_numpy(pos)[:, None]
    t = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(Q).transpose(0, 1), torch.from_numpy(K[0]).repeat_interleave(2, 0),
        torch.from_numpy(V[0]).repeat_interleave(2, 0), mask, scale=0.25)
    assert np.allclose(r["out"], t.transpose(0, 1).numpy())
    every = np.tile(np.arange(5), (5, 1))
    some = ref.block_attn(Q, K, V, np.zeros(5, int), pos, every, 4, 0.25)
    assert np.allclose(some["out"], r["out"]) and np.allclose(some["lse"], r["lse"])
    none = ref.block_attn(Q, K, V, np.zeros(5, int), pos, np.full((5, 2), -1), 4, 0.25)
    assert (none["out"] == 0).all() and np.isneginf(none["lse"]).all()
