"""Plain 64-bit forms of rotary positions, the 4-bit cache rows and block
attention, for the tests (numpy, written from the definitions)."""
import math

import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def rope_rates(rot, base=10000.0, scaling="none", factor=1.0, orig_len=0.0, beta_fast=32.0, beta_slow=1.0):
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    w = base ** (-2.0 * i / rot)
    if scaling == "linear":
        w = w / factor
    if scaling == "yarn":
        c = lambda t: rot * math.log(orig_len / (2 * math.pi * t)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(c(beta_fast)), 0), min(math.ceil(c(beta_slow)), rot - 1)
        r = np.clip((i - lo) / max(hi - lo, 0.001), 0, 1)
        w = w * (1 - r) + w / factor * r
    return w


def rope(x, pos, w, off, layout, gain=1.0, transpose=False):
    """x [rows, heads, d] float64 rotated."""
    y, rot = x.copy(), 2 * len(w)
    t = pos.astype(np.float64)[:, None] * w[None, :]
    c, s = gain * np.cos(t)[:, None], gain * np.sin(t)[:, None] * (-1 if transpose else 1)
    ia = off + (np.arange(rot // 2) if layout == "half" else 2 * np.arange(rot // 2))
    ib = ia + (rot // 2 if layout == "half" else 1)
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ib] * c + x[..., ia] * s
    return y


def e4m3_round(x):
    """Nearest e4m3 value (ties to even) of x >= 0 in float64, as (byte, value)."""
    b = torch.from_numpy(np.minimum(x, 448.0)).to(torch.float32).to(torch.float8_e4m3fn)
    return b.view(torch.uint8).numpy(), b.to(torch.float64).numpy()


def fp4_rows(x, mul=1.0):
    """(codes [.., d / 2], scales [.., d / 16], values [.., d]) of rows x [.., d] float64."""
    g = x.reshape(*x.shape[:-1], -1, 16)
    sb, s = e4m3_round(np.abs(g).max(-1) / (6.0 * mul))
    step = (s * mul)[..., None]
    y = np.minimum(np.abs(g) / np.where(step > 0, step, 1.0), 6.0) * (step > 0)
    dist = np.abs(y[..., None] - E2M1)
    best = dist.min(-1, keepdims=True)
    near = dist == best                               # one code, or the two of a tie
    code = np.where(near[..., 0::2].any(-1), near[..., 0::2].argmax(-1) * 2, near.argmax(-1))   # ties: the even code
    code = code + 8 * ((g < 0) & (code > 0))
    values = np.where(code >= 8, -1.0, 1.0) * E2M1[code & 7] * step
    code = code.reshape(x.shape).astype(np.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), sb, values.reshape(x.shape)


def fp4_values(codes, scales, mul=1.0):
    n = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = np.where(n >= 8, -1.0, 1.0) * E2M1[n & 7]
    s = torch.from_numpy(scales.copy()).view(torch.float8_e4m3fn).to(torch.float64).numpy()
    return v * np.repeat(s, 16, -1) * mul


def visible(q_pos, blocks, B, i):
    """Token positions that row i attends to (blocks None: its whole prefix)."""
    t = int(q_pos[i])
    if t < 0:
        return np.zeros(0, np.int64)
    if blocks is None:
        return np.arange(t + 1)
    keep = sorted({int(j) for j in blocks[i] if 0 <= j <= t // B})
    s = np.concatenate([np.arange(j * B, (j + 1) * B) for j in keep]) if keep else np.zeros(0, np.int64)
    return s[s <= t]


def block_attn(Q, K, V, q_seq, q_pos, blocks, B, scale):
    """Per row and head: out, lse, and what a tolerance needs (sum of weight
    * |v|, largest |scale q.k| by absolute products, tokens, largest |v|).
    Q [n, Hq, d], K, V [batch, Hkv, cap, d] float64; q_pos -1: an invalid row."""
    n, Hq, d = Q.shape
    G = Hq // K.shape[1]
    out, lse = np.zeros((n, Hq, d)), np.full((n, Hq), -np.inf)
    wv, zabs = np.zeros((n, Hq, d)), np.zeros((n, Hq))
    ntok, vmax = np.zeros(n), np.zeros((n, Hq))
    for i in range(n):
        s = visible(q_pos, blocks, B, i)
        ntok[i] = len(s)
        if not len(s):
            continue
        for h in range(Hq):
            k, v = K[q_seq[i], h // G][s], V[q_seq[i], h // G][s]
            z = scale * (k @ Q[i, h])
            zabs[i, h] = scale * (np.abs(k) @ np.abs(Q[i, h])).max()
            m = z.max()
            p = np.exp(z - m)
            lse[i, h] = m + math.log(p.sum())
            p /= p.sum()
            out[i, h], wv[i, h], vmax[i, h] = p @ v, p @ np.abs(v), np.abs(v).max()
    return dict(out=out, lse=lse, wv=wv, zabs=zabs, ntok=ntok, vmax=vmax)


def check_block_attn(out, lse, ref, d, fp4):
    """Tolerances from the arithmetic: a logit is a sum of d exact products in
    fp32, off by at most d * 2^-23 of the sum of their magnitudes (2^-23: the
    tensor core may cut instead of round); a weight is off by that, by the 2^x
    unit's 2^-22 and by its rounding, 2^-8 (bf16) or 2^-11 (f16, with 2^-25 of
    the largest as its smallest step: kept 2^7 larger, 2^-32); the output is
    rounded to bf16, 2^-8 of itself.  The fp32 sums over tokens add 2^-16."""
    dz = d * 2.0 ** -23 * ref["zabs"]
    rel = (2.0 ** -11 if fp4 else 2.0 ** -8) + 2.0 ** -16
    tiny = ref["ntok"][:, None] * ref["vmax"] * 2.0 ** -32
    tol = (rel + 2 * dz)[..., None] * ref["wv"] + tiny[..., None]
    tol = tol + 2.0 ** -8 * (np.abs(ref["out"]) + tol) + 1e-30
    bad = np.abs(out - ref["out"]) > tol
    assert not bad.any(), (f"{bad.sum()} of {bad.size} outputs off, worst "
                           f"{(np.abs(out - ref['out']) / tol).max():.2f} of the tolerance at {np.argwhere(bad)[0]}")
    empty = np.isneginf(ref["lse"])
    assert np.array_equal(np.isneginf(lse), empty)
    lt = dz + 2.0 ** -18 * (1 + np.abs(np.where(empty, 0, ref["lse"])))
    err = np.abs(np.where(empty, 0, lse) - np.where(empty, 0, ref["lse"]))
    assert (err <= lt).all(), f"lse off by {err.max()}, {(err / lt).max():.2f} of the tolerance"
