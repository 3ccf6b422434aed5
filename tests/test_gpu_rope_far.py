"""Rotary positions at the ends of the sizes the header allows."""
import numpy as np
import pytest
import torch

import hierarchical_top_indexer_b200 as hisa
from tests import attn_ref as ref
from tests.test_gpu_block_attn import _bf, _f64, _i32

pytestmark = pytest.mark.gpu


def test_as_many_rows_as_an_int_counts():
    """2^31 - 1 rows of 16 bytes (34 GB, in place): the number of blocks is computed without passing an int."""
    rows = (1 << 31) - 1
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    rng = np.random.default_rng(0)
    x = torch.zeros((rows, 8), dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(rows, dtype=torch.int32, device="cuda")
    at = np.array([0, 1, 511, 512, 1 << 28, rows // 2, rows - 513, rows - 512, rows - 2, rows - 1])
    some, where = _bf(rng.standard_normal((len(at), 8))), torch.from_numpy(at).cuda()
    p = rng.integers(-(1 << 20), 1 << 20, len(at))
    x[where], pos[where] = some, _i32(p)
    plan = hisa.hisa_rope_init(8, rot=2, off=4, layout="interleaved")
    y = hisa.hisa_rope(plan, x, pos, out=x)
    assert y is x
    want = ref.rope(_f64(some)[:, None], p, ref.rope_rates(2), 4, "interleaved")[:, 0]
    mag = np.abs(_f64(some)[:, 4:6]).sum(1)[:, None]
    # bf16's rounding, the angle (2^-26 of a turn) and fp32's sine, cosine and products (some 2^-22)
    assert (np.abs(_f64(x[where]) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * mag).all()
    assert np.array_equal(_f64(x[where])[:, [0, 1, 2, 3, 6, 7]], _f64(some)[:, [0, 1, 2, 3, 6, 7]])
    assert int(torch.count_nonzero(x[1 << 30:(1 << 30) + (1 << 20)])) == 0
    del x, y, pos
    torch.cuda.empty_cache()


@pytest.mark.parametrize("d,rot,heads", [(8, 2, 1 << 16), (512, 256, 1 << 16), (2, 2, 1 << 16), (16, 16, 40000)])
def test_as_many_heads_as_a_row_has(d, rot, heads):
    rng = np.random.default_rng(d)
    x, pos = _bf(rng.standard_normal((2, heads, d))), np.array([77, -(1 << 31)])
    plan = hisa.hisa_rope_init(d, rot=rot, layout="interleaved" if d == 8 else "half")
    y = _f64(hisa.hisa_rope(plan, x, _i32(pos)))
    want = ref.rope(_f64(x), pos, ref.rope_rates(rot), 0, "interleaved" if d == 8 else "half")
    # bf16's rounding; then, times |a| + |b|: the 64-bit form's own angle at -2^31 (2^-21 and 2^-22 rad from the rate and
    # the product), 2^-26 of a turn (2^-23.3 rad), and fp32's sine, cosine and products (2^-22): together below 2^-19
    mag = 2 * np.abs(_f64(x)).max()
    assert (np.abs(y - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * mag).all()
