"""Work of the attention side of the indexer, case by case: rotary positions, the attention cache held in 4 bits,
and attention over the blocks a cheap score selected (or over the whole prefix).

Three kinds of case, by case["op"]:

  rope    x [rows, heads, d] bf16 and a position per row -> the rotated rows, bf16
  cache   new key and value rows [n, heads, d] bf16 stored in a 4-bit cache at (sequence, position), then read back
  attn    grouped-query attention of query rows over a cache of bf16 rows or of 4-bit rows: over each row's kept
          blocks (m > 0), or over its whole prefix (m = 0) -> out [n_q, Hq, d] bf16, lse [n_q, Hq] fp32

A 4-bit row holds e2m1 codes, two to a byte, the first of a pair in the low half, and one e4m3 scale for each 16
elements; the value is code * scale.  Sequences' rows lie head after head: [batch, heads, cap, ...].
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases

def _rope(rows, heads, d, rot, off, layout, scaling, factor, far, back):
    return dict(op="rope", rows=rows, heads=heads, d=d, rot=rot, off=off, layout=layout, scaling=scaling, factor=factor,
                far=far, back=back)


def _cache(n, heads, d, batch, cap):
    return dict(op="cache", n=n, heads=heads, d=d, batch=batch, cap=cap)


def _attn(dtype, batch, length, rows, Hq, Hkv, d, B, m, ragged):
    return dict(op="attn", dtype=dtype, batch=batch, length=length, rows=rows, Hq=Hq, Hkv=Hkv, d=d, B=B, m=m, ragged=ragged)


def listed():
    return [
        # one decode step's indexer queries of 64 sequences: the last 64 of 128 dimensions carry the position
        dict(_rope(64, 64, 128, 64, 64, "half", "none", 1.0, 32768, False), name="rope decode 64x64"),
        # a prefill chunk's queries far out in a context stretched sixteen times
        dict(_rope(4096, 64, 128, 64, 0, "interleaved", "yarn", 16.0, 131072, False), name="rope chunk 4096x64"),
        # the way back (the gradient of the rotated keys), few heads, odd row count, short head
        dict(_rope(4999, 5, 64, 32, 16, "half", "ntk", 4.0, 32768, True), name="rope back 4999x5"),
        # one new token of 64 sequences into the 4-bit cache
        dict(_cache(64, 8, 128, 64, 4096), name="cache decode 64x8"),
        # a prefill chunk into the 4-bit cache
        dict(_cache(16384, 8, 128, 1, 32768), name="cache chunk 16384x8"),
        # the smallest decode step: latency
        dict(_attn("bf16", 4, 2048, 1, 8, 2, 64, 64, 8, True), name="attn decode 2K b4"),
        # the 32K decode batch, 64 blocks of 128 tokens each
        dict(_attn("bf16", 64, 32768, 1, 64, 8, 128, 128, 64, False), name="attn decode 32K b64"),
        # a chunk of 4096 rows, each with blocks of its own
        dict(_attn("bf16", 1, 32768, 4096, 16, 2, 128, 128, 64, False), name="attn chunk 4096 of 32K"),
        # one user's decode step over the whole 4-bit prefix: few rows, split over the length
        dict(_attn("fp4", 1, 8000, 1, 16, 2, 128, 128, 0, False), name="attn4 decode 8K b1"),
        # long 4-bit prefixes, no selection
        dict(_attn("fp4", 16, 131072, 1, 32, 4, 128, 128, 0, True), name="attn4 decode 128K b16"),
        # 128 heads over one key and value head, the kept blocks of a 4-bit cache
        dict(_attn("fp4", 64, 32768, 1, 128, 1, 128, 128, 64, False), name="attn4 blocks 32K b64 mqa"),
        # a chunk against its 4-bit prefix, causal
        dict(_attn("fp4", 2, 8191, 512, 32, 4, 128, 128, 0, False), name="attn4 chunk 512 of 8K b2"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "cache", "attn", "attn", "attn", "attn"])
    d = rng.choice([64, 128])
    if op == "rope":
        rot = rng.choice([d // 4, d // 2, d])
        off = rng.choice([0, d - rot])
        rows = _log(rng, 1, 8192)
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        return _rope(rows, _log(rng, 1, max(2, min(128, 262144 // rows))), d, rot, off, rng.choice(["half", "interleaved"]), scaling,
                     1.0 if scaling == "none" else rng.choice([2.0, 8.0, 16.0]), _log(rng, 1024, 1 << 20), rng.random() < 0.3)
    if op == "cache":
        n = _log(rng, 1, 16384)
        return _cache(n, rng.randint(1, 8), d, rng.randint(1, 16), 16 * _log(rng, max(1, -(-n // 16)), 4096))
    dtype = rng.choice(["bf16", "fp4"])
    Hkv = rng.choice([1, 1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16, 32, 128 if Hkv == 1 else 6])
    B = rng.choice([16, 32, 64, 128, 256])
    if rng.random() < 0.6:   # single tokens
        batch = _log(rng, 1, 64)
        length = _log(rng, 17, min(131072, 4194304 // (batch * Hkv)))
        m = rng.choice([0, max(1, _log(rng, 1, 8192) // B)])
        return _attn(dtype, batch, length, 1, Hkv * G, Hkv, d, B, m, rng.random() < 0.5)
    batch = rng.randint(1, 3)
    rows = _log(rng, 2, 512)
    length = _log(rng, rows, min(32768, 134217728 // (batch * rows * Hkv * G)) + rows)
    m = rng.choice([0, max(1, _log(rng, 1, 4096) // B)])
    return _attn(dtype, batch, length, rows, Hkv * G, Hkv, d, B, m, False)


# ----------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _quantise(x):
    """Rows of bf16 values as (e2m1 codes, e4m3 scales): the scale of 16 elements is their largest magnitude / 6 rounded to
    e4m3, a code is the element / scale rounded to the nearest e2m1 value (ties to the even code), saturated at 6."""
    x = x.float().unflatten(-1, (-1, 16))
    s = (x.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    y = x / s.float().clamp(min=2.0 ** -10).unsqueeze(-1) * (s.float() > 0).unsqueeze(-1)
    a = y.abs()
    code = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte() + (a >= 3.5).byte()
            + (a > 5.0).byte())
    code = (code | ((y < 0) & (code > 0)).byte() * 8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.view(torch.uint8)


def _values(codes, scales, dtype=torch.float32):
    """The values that codes and scales stand for."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=dtype, device=codes.device)
    v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1).flatten(-2)
    return v.unflatten(-1, (-1, 16)).mul_(scales.view(torch.float8_e4m3fn).to(dtype).unsqueeze(-1)).flatten(-2)


def _kept_blocks(g, c, q_seq, q_pos):
    """Each row's own block and the m - 1 others of the highest score, ascending, -1 padded.  The score drifts along a
    sequence, as neighbouring queries look at much the same blocks, and every row has some of its own."""
    nblk = -(-c["length"] // c["B"])
    n = q_seq.numel()
    anchors = torch.randn((c["batch"], c["rows"] // 64 + 2, nblk), generator=g, device="cuda")
    at = (torch.arange(n, device="cuda") % c["rows"]).float() / 64.0
    lo = at.long()
    w = (at - lo).unsqueeze(1)
    score = (1 - w) * anchors[q_seq.long(), lo] + w * anchors[q_seq.long(), lo + 1]
    score += 0.5 * torch.randn((n, nblk), generator=g, device="cuda")
    j = torch.arange(nblk, device="cuda")
    mine = (q_pos // c["B"]).unsqueeze(1)
    score = score.masked_fill(j > mine, -math.inf).masked_fill(j == mine, math.inf)
    top, idx = score.topk(min(c["m"], nblk), dim=1)
    idx = idx.masked_fill(top == -math.inf, nblk).sort(dim=1).values
    return idx.masked_fill(idx == nblk, -1).int().contiguous()


def prepare(case, seed):
    g, c = _gen(seed), case
    s = dict(case=c)
    if c["op"] == "rope":
        s["x"] = _normal(g, c["rows"], c["heads"], c["d"])
        s["pos"] = torch.randint(0, c["far"], (c["rows"],), generator=g, device="cuda", dtype=torch.int32)
        if own:
            import hierarchical_top_indexer_b200 as hisa
            s["rope"] = hisa.hisa_rope_init(c["d"], rot=c["rot"], off=c["off"], layout=c["layout"], base=10000.0, scaling=c["scaling"],
                                            factor=c["factor"], orig_len=8192)
        return s
    if c["op"] == "cache":
        s["k"], s["v"] = _normal(g, c["n"], c["heads"], c["d"]), _normal(g, c["n"], c["heads"], c["d"])
        s["k"] *= torch.exp(torch.randn((c["heads"], c["d"]), generator=g, device="cuda")).bfloat16()  # some channels of a key run larger
        slots = torch.randperm(c["batch"] * c["cap"], generator=g, device="cuda")[:c["n"]].sort().values
        s["seq"], s["pos"] = (slots // c["cap"]).int(), (slots % c["cap"]).int()
        shape = (c["batch"], c["heads"], c["cap"])
        lens = torch.full((c["batch"],), c["cap"], dtype=torch.int32, device="cuda")
        s["cache"] = [torch.zeros((*shape, c["d"] // 2), dtype=torch.uint8, device="cuda") for _ in range(2)]
        s["cache"] += [torch.zeros((*shape, c["d"] // 16), dtype=torch.uint8, device="cuda") for _ in range(2)]
        if own:
            import hierarchical_top_indexer_b200 as hisa
            s["handle"] = hisa.AttnCache.wrap(s["cache"][0], s["cache"][1], lens, k_scale=s["cache"][2], v_scale=s["cache"][3])
        return s
    batch, rows, cap = c["batch"], c["rows"], -(-c["length"] // 16) * 16
    lens = torch.full((batch,), c["length"], dtype=torch.int32, device="cuda")
    if c["ragged"]:
        lens -= torch.randint(0, max(1, c["length"] // 4), (batch,), generator=g, device="cuda", dtype=torch.int32)
    s["len"] = lens
    s["q"] = _normal(g, batch * rows, c["Hq"], c["d"])
    s["q_seq"] = torch.arange(batch, device="cuda", dtype=torch.int32).repeat_interleave(rows)
    s["q_pos"] = (lens[s["q_seq"].long()] - rows + torch.arange(rows, device="cuda", dtype=torch.int32).repeat(batch)).int()
    s["k"], s["v"] = _normal(g, batch, c["Hkv"], cap, c["d"]), _normal(g, batch, c["Hkv"], cap, c["d"])
    # keys of one block lie around a centre of their own
    nblk = -(-cap // 128)
    s["k"].mul_(0.5).add_(_normal(g, batch, c["Hkv"], nblk, 1, c["d"]).expand(-1, -1, -1, 128, -1).flatten(2, 3)[:, :, :cap])
    if c["dtype"] == "fp4":
        s["k"], s["k_scale"] = _quantise(s["k"])
        s["v"], s["v_scale"] = _quantise(s["v"])
    s["blocks"] = _kept_blocks(g, c, s["q_seq"], s["q_pos"]) if c["m"] else None
    s["scale"] = 1.0 / math.sqrt(c["d"])
    if own:
        import hierarchical_top_indexer_b200 as hisa
        s["handle"] = hisa.AttnCache.wrap(s["k"], s["v"], lens, k_scale=s.get("k_scale"), v_scale=s.get("v_scale"))
        s["ws"] = hisa.workspace(hisa.hisa_block_attn_workspace_bytes(s["handle"], batch * rows, c["Hq"], c["B"], c["m"]))
    return s


# ------------------------------------------------------------ plain forms

def _inv_freq(c):
    """Rotation per position of each pair, in radians, with the context stretched as asked."""
    i = torch.arange(c["rot"] // 2, dtype=torch.float64, device="cuda")
    base, f = 10000.0, c["factor"]
    if c["scaling"] == "ntk":
        base = base * f ** (c["rot"] / (c["rot"] - 2))
    inv = base ** (-2.0 * i / c["rot"])
    if c["scaling"] == "linear":
        inv = inv / f
    if c["scaling"] == "yarn":   # pairs that turn often keep their rate, those that hardly turn are stretched
        at = lambda turns: c["rot"] * math.log(8192 / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), c["rot"] - 1)
        keep = 1 - ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        inv = inv * keep + inv / f * (1 - keep)
    return inv


def _plain_rope(s):
    c, x = s["case"], s["x"].float()
    ang = s["pos"].double().unsqueeze(1) * _inv_freq(c)
    m = 0.1 * math.log(c["factor"]) + 1.0 if c["scaling"] == "yarn" else 1.0
    cos, sin = (m * ang.cos()).float().unsqueeze(1), (m * ang.sin()).float().unsqueeze(1)
    sin = -sin if c["back"] else sin
    part = x[..., c["off"]:c["off"] + c["rot"]]
    y = x.clone()
    out = y[..., c["off"]:c["off"] + c["rot"]]
    if c["layout"] == "half":
        a, b = part[..., :c["rot"] // 2], part[..., c["rot"] // 2:]
        out[..., :c["rot"] // 2], out[..., c["rot"] // 2:] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        out[..., 0::2], out[..., 1::2] = a * cos - b * sin, b * cos + a * sin
    return y.bfloat16()


def _plain_cache(s):
    seq, pos = s["seq"].long(), s["pos"].long()
    kq, vq = _quantise(s["k"]), _quantise(s["v"])
    k, v, ks, vs = s["cache"]
    k[seq, :, pos], ks[seq, :, pos] = kq
    v[seq, :, pos], vs[seq, :, pos] = vq
    return [_values(x[seq, :, pos], sc[seq, :, pos]).bfloat16() for x, sc in ((k, ks), (v, vs))]


def _plain_attn(s):
    c = s["case"]
    n, Hkv, G = s["q"].shape[0], c["Hkv"], c["Hq"] // c["Hkv"]
    f = lambda x, sc: _values(x, sc) if c["dtype"] == "fp4" else x.float()  # noqa: E731
    q = s["q"].float().unflatten(1, (Hkv, G))
    if c["rows"] == 1 and c["m"]:   # single tokens: their kept tokens gathered
        tok = (s["blocks"].unsqueeze(2) * c["B"] + torch.arange(c["B"], device="cuda")).flatten(1)
        on = (s["blocks"] >= 0).repeat_interleave(c["B"], 1) & (tok <= s["q_pos"].unsqueeze(1))
        tok = tok.masked_fill(~on, 0).long()
        at = (s["q_seq"].long().view(-1, 1, 1), torch.arange(Hkv, device="cuda").view(1, -1, 1), tok.unsqueeze(1))
        k = f(s["k"][at], s["k_scale"][at] if "k_scale" in s else None)
        v = f(s["v"][at], s["v_scale"][at] if "v_scale" in s else None)
        on = on.view(n, 1, 1, -1)
        z = torch.einsum("nhgd,nhtd->nhgt", q, k)
        combine = "nhgt,nhtd->nhgd"
    else:                           # a chunk: every token of its prefix, the others masked
        k, v = f(s["k"], s.get("k_scale")), f(s["v"], s.get("v_scale"))
        t = torch.arange(k.shape[2], device="cuda")
        on = t <= s["q_pos"].unsqueeze(1)
        if c["m"]:
            kept = torch.zeros((n, -(-k.shape[2] // c["B"]) + 1), dtype=torch.bool, device="cuda")
            kept.scatter_(1, s["blocks"].long() % kept.shape[1], True)   # -1 falls on the last, unused one
            on &= kept[:, t // c["B"]]
        q = q.unflatten(0, (c["batch"], c["rows"]))
        on = on.view(c["batch"], c["rows"], 1, 1, -1)
        z = torch.einsum("brhgd,bhtd->brhgt", q, k)
        combine = "brhgt,bhtd->brhgd"
    z.mul_(s["scale"]).masked_fill_(~on, -math.inf)
    top = z.amax(-1, keepdim=True)
    z.sub_(top).exp_()
    total = z.sum(-1, keepdim=True)
    out = torch.einsum(combine, z, v) / total
    return out.reshape(n, c["Hq"], c["d"]).bfloat16(), (top + total.log()).reshape(n, c["Hq"])


def run(state):
    op = state["case"]["op"]
    if own:
        import hierarchical_top_indexer_b200 as hisa
        if op == "rope":
            return hisa.hisa_rope(state["rope"], state["x"], state["pos"], transpose=state["case"]["back"])
        if op == "cache":
            hisa.hisa_cache_store(state["handle"], state["k"], state["v"], state["seq"], state["pos"])
            return list(hisa.hisa_cache_load(state["handle"], state["seq"], state["pos"]))
        return hisa.hisa_block_attn(state["handle"], state["q"], state["q_seq"], state["q_pos"], state["blocks"], B=state["case"]["B"],
                                    scale=state["scale"], ws=state["ws"])
    return _plain_rope(state) if op == "rope" else _plain_cache(state) if op == "cache" else _plain_attn(state)


# ------------------------------------------------------- work and 64 bits

def _token_bytes(c):
    return c["Hkv"] * (2 * c["d"] * 2 if c["dtype"] == "bf16" else 2 * (c["d"] // 2 + c["d"] // 16))


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["rows"] * c["heads"]
        return {"bytes": 4.0 * n * c["d"] + 4 * c["rows"], "flops": 3.0 * n * c["rot"]}
    if c["op"] == "cache":   # bf16 rows in, codes and scales out; then codes and scales in, values out
        n = 2 * c["n"] * c["heads"] * c["d"]
        return {"bytes": 2 * (2.0 * n + 0.5625 * n) + 16.0 * c["n"], "flops": 4.0 * n}
    n_q = c["batch"] * c["rows"]
    length = c["length"] * (0.875 if c["ragged"] else 1.0)
    seen = min(c["m"] * c["B"], length) if c["m"] else length - (c["rows"] - 1) / 2
    read = c["batch"] * min(length, c["rows"] * seen if c["m"] else length)   # a chunk's tokens are read once
    return {"bytes": read * _token_bytes(c) + n_q * (c["Hq"] * (4.0 * c["d"] + 4) + 4 * c["m"] + 8), "flops": 4.0 * c["d"] * c["Hq"] * n_q * seen}


def _exact_rope(s):
    c = s["case"]
    x, pos = s["x"].double(), s["pos"].double()
    y, base, f, r = x.clone(), 10000.0, c["factor"], c["rot"]
    if c["scaling"] == "ntk":
        base *= math.pow(f, r / (r - 2))
    turn = lambda t: r * math.log(8192 / (2 * math.pi * t)) / (2 * math.log(base))  # noqa: E731
    first, last = max(math.floor(turn(32)), 0), min(math.ceil(turn(1)), r - 1)
    gain = 1 + 0.1 * math.log(f) if c["scaling"] == "yarn" else 1.0
    for i in range(r // 2):
        rate = math.pow(base, -2 * i / r)
        if c["scaling"] == "linear":
            rate /= f
        if c["scaling"] == "yarn":
            slow = min(max((i - first) / max(last - first, 0.001), 0.0), 1.0)
            rate = rate * (1 - slow) + rate / f * slow
        p, q = (c["off"] + i, c["off"] + i + r // 2) if c["layout"] == "half" else (c["off"] + 2 * i, c["off"] + 2 * i + 1)
        z = torch.complex(x[:, :, p], x[:, :, q]) * torch.polar(torch.full_like(pos, gain), (-pos if c["back"] else pos) * rate).unsqueeze(1)
        y[:, :, p], y[:, :, q] = z.real, z.imag
    return y


def _exact_cached(x):
    """The values that stored rows come back as: nearest code of the sixteen, per group of 16."""
    x = x.double().reshape(*x.shape[:-1], -1, 16)
    s = torch.clamp(x.abs().max(-1).values / 6, max=448.0).float().to(torch.float8_e4m3fn).double().unsqueeze(-1)
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    y = torch.where(s > 0, x.abs() / torch.where(s > 0, s, 1.0), 0.0).clamp(max=6.0)
    hi = torch.searchsorted(grid, y).clamp(max=7)
    lo = (hi - 1).clamp(min=0)
    up = (grid[hi] - y < y - grid[lo]) | ((grid[hi] - y == y - grid[lo]) & (hi % 2 == 0))
    return (torch.where(up, grid[hi], grid[lo]) * s * x.sign()).flatten(-2)


def _exact_values(x, scale):
    if scale is None:
        return x.double()
    n = torch.stack((x % 16, x // 16), -1).flatten(-2).long()
    e, m = n // 2 % 4, n % 2
    v = torch.where(e > 0, (1 + 0.5 * m) * torch.pow(2.0, (e - 1).double()), 0.5 * m) * (1.0 - 2.0 * (n // 8))
    return v * scale.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "rope":
        return _exact_rope(s)
    if c["op"] == "cache":
        return [_exact_cached(s["k"]), _exact_cached(s["v"])]
    G, d = c["Hq"] // c["Hkv"], c["d"]
    out = torch.empty((s["q"].shape[0], c["Hq"], d), dtype=torch.float64, device="cuda")
    lse = torch.empty(out.shape[:2], dtype=torch.float64, device="cuda")
    for b in range(c["batch"]):
        n = int(s["len"][b])
        t = torch.arange(n, device="cuda")
        for h in range(c["Hkv"]):
            k, v = (_exact_values(s[x][b, h, :n], s[x + "_scale"][b, h, :n] if x + "_scale" in s else None) for x in "kv")
            for r in range(b * c["rows"], (b + 1) * c["rows"], 256):
                e = min(r + 256, (b + 1) * c["rows"])
                z = torch.matmul(s["q"][r:e, h * G:(h + 1) * G].double(), k.T) * s["scale"]
                seen = t[None] <= s["q_pos"][r:e, None]
                if c["m"]:
                    seen &= torch.stack([torch.isin(t // c["B"], row) for row in s["blocks"][r:e]])
                z = z.masked_fill(~seen[:, None], -math.inf)
                lse[r:e, h * G:(h + 1) * G] = torch.logsumexp(z, -1)
                out[r:e, h * G:(h + 1) * G] = torch.matmul(torch.softmax(z, -1), v)
    return out, lse
