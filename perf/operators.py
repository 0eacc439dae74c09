"""The 4-bit latent cache's operators as a program uses them: writing latent rows to the cache (whole prompts, chunks
and single tokens), reading them back, and decoding over them; each in a plain form of elementary torch operations
and as the package's own calls.

Cache row (r values): r / 2 bytes of e2m1 codes (element 2j in the low half of byte j: sign, then the index of
0, 0.5, 1, 1.5, 2, 3, 4, 6), then r / 32 scale bytes, one per 32 consecutive elements, then padding to a multiple of
16 bytes.  A scale byte X stands for 2^(X - 127) with X taken into [87, 167]; 255 is NaN.  The writer picks the
smallest exponent e in [-40, 40] with max|group| <= 7 * 2^e (up to there, 6 is no further off than half a step), and
rounds x * 2^-e to the nearest code, ties to the even code, saturating at 6; a group that holds a NaN or an infinity
gets scale 255 and zero codes.
"""
import math

import torch

own = False

GROUP = 32
D_V = 128
STD = 0.02   # weights; queries as q_abs = q . W_UK with q ~ N(0, 1) and d_q = 128


def _row_bytes(r):
    return -(-(r // 2 + r // GROUP) // 16) * 16


# ------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the cached-latent decode of the benchmark: 64 ragged sequences up to 32768 rows, all 96 heads
        dict(name="decode_64x32768_h96", kind="decode", B=64, H=96, lo=1024, hi=32768, max_len=32768, ld=272,
             gate=False, edges=False),
        # the mid-size layer's 16 heads (or a 96-head layer on six devices), gated, mid-length conversations
        dict(name="decode_32x4096_h16", kind="decode", B=32, H=16, lo=512, hi=4096, max_len=4096, ld=272, gate=True,
             edges=False),
        # one user with a very long document: the work is split along the rows
        dict(name="decode_1x130999_h96", kind="decode", B=1, H=96, lo=130999, hi=130999, max_len=131072, ld=272,
             gate=True, edges=False),
        # a handful of fresh conversations at the toy layer's 8 heads: latency
        dict(name="decode_4x300_h8", kind="decode", B=4, H=8, lo=1, hi=300, max_len=300, ld=272, gate=True,
             edges=False),
        # odd head count, rows inside a wider record, an empty and a one-row sequence among the others
        dict(name="decode_7x5000_h37", kind="decode", B=7, H=37, lo=2, hi=5000, max_len=5001, ld=320, gate=True,
             edges=True),
        # a serving step: the new token's latent goes into the cache, then all heads attend to it and the past
        dict(name="step_64x8192_h96", kind="step", B=64, H=96, lo=1024, hi=8191, max_len=8192, ld=272, gate=True,
             edges=False),
        # the same for a single user
        dict(name="step_1x1000_h16", kind="step", B=1, H=16, lo=1000, hi=1000, max_len=1024, ld=272, gate=True,
             edges=False),
        # chunked prefill: ragged sequences take a chunk of 512 tokens each, and the context is read back for it
        dict(name="append_8x512", kind="append", B=8, T=512, lo=0, hi=3584, max_len=4096, ld=272, r=512,
             dtype="bfloat16"),
        # one token for each of 64 short conversations, then the context is read back
        dict(name="append_64x1", kind="append", B=64, T=1, lo=0, hi=255, max_len=256, ld=272, r=512,
             dtype="bfloat16"),
        # sixteen prompts of 8192 tokens written and read back
        dict(name="write_131072x512", kind="write", rows=131072, r=512, dtype="bfloat16"),
        # the toy layer's latent in fp32: two sequences of 128 tokens, 32 values each
        dict(name="write_256x32_f32", kind="write", rows=256, r=32, dtype="float32"),
        # ragged contexts read back as bf16 rows, padding left as it was
        dict(name="read_16x4096", kind="read", B=16, lo=100, hi=4096, max_len=4096, ld=288, r=512, dtype="bfloat16"),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "decode", "step", "append", "write", "read"])
    if kind in ("decode", "step"):
        B = _between(rng, 1, 64)
        hi = _between(rng, 1, min(131072, 64 * 32768 // B // 2))
        lo = _between(rng, 1, hi)
        max_len = hi + 1 + rng.randrange(0, 64)
        return dict(kind=kind, B=B, H=_between(rng, 1, 96), lo=lo, hi=hi, max_len=max_len,
                    ld=272 + 16 * rng.choice([0, 0, 1, 3, 15]), gate=rng.random() < 0.5,
                    edges=B > 2 and rng.random() < 0.5)
    r = 32 * _between(rng, 1, 16)
    dtype = rng.choice(["bfloat16", "float32"])
    ld = _row_bytes(r) + 16 * rng.choice([0, 0, 1, 3])
    if kind == "write":
        return dict(kind=kind, rows=_between(rng, 1, 131072), r=r, dtype=dtype)
    B = _between(rng, 1, 64)
    max_len = _between(rng, 2, 131072 // B)
    if kind == "read":
        return dict(kind=kind, B=B, lo=0, hi=max_len, max_len=max_len, ld=ld, r=r, dtype=dtype)
    T = _between(rng, 1, max_len)
    return dict(kind=kind, B=B, T=T, lo=0, hi=max_len - T, max_len=max_len, ld=ld, r=r, dtype=dtype)


def _lens(case):
    """Ragged lengths, evenly spread over [lo, hi] (their order comes from the seed)."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    lens = [lo + int((hi - lo) * (i + 0.5) / B) for i in range(B)]
    if case.get("edges"):
        lens[:2] = [0, 1]
    return lens


# ------------------------------------------------------------------------------------------------- inputs
def _normal(gen, shape, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std


def _latent(gen, shape):
    """Latent rows as RMSNorm with unit gain leaves them."""
    x = _normal(gen, shape)
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)
    kind = case["kind"]
    state = dict(case=case)
    r = case.get("r", 512)
    dtype = getattr(torch, case.get("dtype", "bfloat16"))
    if kind == "write":
        state["c"] = _latent(gen, (case["rows"], r)).to(dtype)
        return state
    B, max_len, ld = case["B"], case["max_len"], case["ld"]
    lens = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
    state["lens"] = lens[torch.randperm(B, generator=gen, device="cuda")].contiguous()
    records = torch.zeros((B, max_len, ld), dtype=torch.uint8, device="cuda")
    state["cache"] = records[:, :, :_row_bytes(r)]
    for b in range(B):
        state["cache"][b] = _pack(_latent(gen, (max_len, r)))
    if kind == "read":
        state["out"] = torch.zeros((B, max_len, r), dtype=dtype, device="cuda")
        return state
    if kind == "append":
        state["new"] = _latent(gen, (B, case["T"], r)).to(dtype)
        return state
    H = case["H"]
    state["scale"] = 1.0 if H > 48 else 1.0 / math.sqrt(128.0)
    state["q_abs"] = _normal(gen, (B, H, r), math.sqrt(128.0) * STD).to(torch.bfloat16)
    state["w_uv"] = _normal(gen, (H, D_V, r), STD).to(torch.bfloat16)
    state["gate"] = _normal(gen, (B, H * D_V)).to(torch.bfloat16) if case["gate"] else None
    if kind == "step":
        state["new"] = _latent(gen, (B, 1, r)).to(torch.bfloat16)
        state["lens_after"] = state["lens"] + 1
    return state


# ------------------------------------------------------------------------------------------------- plain forms
def _pack(x):
    """Cache rows [..., row_bytes(r)] of latent rows x [..., r]."""
    r = x.shape[-1]
    g = x.float().unflatten(-1, (r // GROUP, GROUP))
    a = g.abs().amax(-1)
    bad = ~torch.isfinite(g).all(-1)
    mant, expo = torch.frexp(a)                      # a = mant * 2^expo, mant in [0.5, 1)
    e = torch.where(mant <= 0.875, expo - 3, expo - 2).clamp(-40, 40)
    e = torch.where(a == 0, -40, e)
    s = torch.ldexp(g, -e.unsqueeze(-1))
    m = s.abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    code = code + 8 * torch.signbit(s)
    code = torch.where(bad.unsqueeze(-1), 0, code).flatten(-2)
    scale = torch.where(bad, 255, e + 127).to(torch.uint8)
    rows = torch.cat([code[..., 0::2] + 16 * code[..., 1::2], scale], -1)
    return torch.nn.functional.pad(rows.to(torch.uint8), (0, _row_bytes(r) - rows.shape[-1]))


def _unpack(rows, r):
    """fp32 values of cache rows."""
    codes = rows[..., :r // 2]
    codes = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=rows.device)
    v = torch.where(codes >= 8, -1.0, 1.0) * grid[codes & 7]
    X = rows[..., r // 2:r // 2 + r // GROUP].int()
    scale = torch.where(X == 255, math.nan, torch.exp2((X.clamp(87, 167) - 127).float()))
    return (v.unflatten(-1, (r // GROUP, GROUP)) * scale.unsqueeze(-1)).flatten(-2)


def _put(cache, new, lens):
    """new [B, T, r] into rows lens[b] .. lens[b] + T - 1 of each sequence."""
    B, T = new.shape[:2]
    at = lens.long()[:, None] + torch.arange(T, device=lens.device)
    cache[torch.arange(B, device=lens.device)[:, None], at] = _pack(new)


def _attend(q_abs, cache, lens, w_uv, gate, scale):
    B, H, r = q_abs.shape
    c = _unpack(cache, r)
    seen = torch.arange(c.shape[1], device=c.device) < lens[:, None]
    c = torch.where(seen[:, :, None], c, 0.0)
    s = torch.matmul(q_abs.float(), c.transpose(1, 2)) * scale
    s = torch.where(seen[:, None, :], s, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(top), 0.0, top))
    norm = p.sum(-1, keepdim=True)
    o_lat = torch.matmul(p, c) / torch.where(lens[:, None, None] == 0, 1.0, norm)
    o = torch.matmul(o_lat.transpose(0, 1), w_uv.float().transpose(1, 2)).transpose(0, 1).reshape(B, -1)
    if gate is not None:
        o = o / (1.0 + torch.exp(-gate.float()))
    return o.to(torch.bfloat16)


def run(state):
    case = state["case"]
    kind = case["kind"]
    if own:
        import latent_compressed_attention_gb300 as lca

        if kind == "write":
            c4 = lca.mla_quantize_latent_fp4(state["c"])
            return lca.mla_dequantize_latent_fp4(c4, case["r"], dtype=state["c"].dtype)
        if kind == "read":
            return lca.mla_dequantize_latent_fp4(state["cache"], case["r"], lens=state["lens"], out=state["out"])
        if kind == "append":
            lca.mla_append_latent_fp4(state["new"], state["cache"], state["lens"])
            return lca.mla_dequantize_latent_fp4(state["cache"], case["r"], dtype=state["new"].dtype)
        lens = state["lens"]
        if kind == "step":
            lca.mla_append_latent_fp4(state["new"], state["cache"], lens)
            lens = state["lens_after"]
        return lca.mla_latent_decode_fp4(state["q_abs"], state["cache"], lens, state["w_uv"], state["gate"],
                                         state["scale"])
    if kind == "write":
        return _unpack(_pack(state["c"]), case["r"]).to(state["c"].dtype)
    if kind == "read":
        rows = torch.arange(case["max_len"], device="cuda")
        seen = rows < state["lens"][:, None]
        c = _unpack(state["cache"], case["r"]).to(state["out"].dtype)
        state["out"].copy_(torch.where(seen[:, :, None], c, state["out"]))
        return state["out"]
    if kind == "append":
        _put(state["cache"], state["new"], state["lens"])
        return _unpack(state["cache"], case["r"]).to(state["new"].dtype)
    lens = state["lens"]
    if kind == "step":
        _put(state["cache"], state["new"], lens)
        lens = state["lens_after"]
    return _attend(state["q_abs"], state["cache"], lens, state["w_uv"], state["gate"], state["scale"])


# ------------------------------------------------------------------------------------------------- floors
def work(case):
    kind = case["kind"]
    r = case.get("r", 512)
    row = r // 2 + r // GROUP
    es = 4 if case.get("dtype") == "float32" else 2
    if kind == "write":   # the rows in, the cache out, the values read back out
        return dict(bytes=case["rows"] * (r * es + row + r * es), flops=0)
    B = case["B"]
    rows = sum(_lens(case))
    if kind == "read":
        return dict(bytes=rows * (row + r * es) + 4 * B, flops=0)
    if kind == "append":   # the new rows in and into the cache, the whole cache out as values
        new, all_rows = B * case["T"], B * case["max_len"]
        return dict(bytes=new * (r * es + row) + (all_rows - new) * row + all_rows * r * es + 4 * B, flops=0)
    H = case["H"]
    bytes_ = rows * row + B * H * r * 2 + H * D_V * r * 2 + B * H * D_V * 2 * (2 if case["gate"] else 1) + 4 * B
    if kind == "step":
        bytes_ += B * (r * 2 + row)
        rows += B
    return dict(bytes=bytes_, flops=4 * rows * H * r + 2 * B * H * r * D_V)


# ------------------------------------------------------------------------------------------------- in 64 bits
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _values64(rows, r):
    """The values that cache rows [n, row_bytes] stand for."""
    table = torch.tensor(_E2M1, dtype=torch.float64, device=rows.device)
    both = torch.empty((rows.shape[0], r), dtype=torch.float64, device=rows.device)
    both[:, 0::2] = table[(rows[:, :r // 2] % 16).long()]
    both[:, 1::2] = table[(rows[:, :r // 2] // 16).long()]
    X = rows[:, r // 2:r // 2 + r // GROUP].double()
    scale = torch.where(X == 255, math.nan, torch.exp2(X.clamp(87, 167) - 127))
    return both * scale.repeat_interleave(GROUP, 1)


def _nearest64(x):
    """What latent rows x [n, r] become in the cache, from the format's definition."""
    g = x.double().unflatten(1, (-1, GROUP))
    top = g.abs().amax(-1, keepdim=True)
    units = torch.exp2(torch.arange(-40, 41, dtype=torch.float64, device=x.device))
    unit = units[(top > 7.0 * units[:-1]).sum(-1, keepdim=True)]
    order = [0, 2, 4, 6, 1, 3, 5, 7]   # even codes first: of two equally near ones the first is taken
    grid = torch.tensor([_E2M1[k] for k in order], dtype=torch.float64, device=x.device)
    near = grid[((g.abs() / unit).unsqueeze(-1) - grid).abs().argmin(-1)]
    return torch.where(torch.isfinite(g).all(-1, keepdim=True), torch.copysign(near, g) * unit, math.nan).flatten(1)


def exact(case, seed):
    state = prepare(case, seed)
    kind = case["kind"]
    r = case.get("r", 512)
    if kind == "write":
        return _nearest64(state["c"])
    lens = state["lens"].tolist()
    B, cache = case["B"], state["cache"]
    if kind == "read":
        out = state["out"].double()
        for b in range(B):
            out[b, :lens[b]] = _values64(cache[b, :lens[b]], r)
        return out
    if kind == "append":
        out = torch.empty((B, case["max_len"], r), dtype=torch.float64, device="cuda")
        for b in range(B):
            out[b] = _values64(cache[b], r)
            out[b, lens[b]:lens[b] + case["T"]] = _nearest64(state["new"][b])
        return out
    outs = []
    for b in range(B):
        c = _values64(cache[b, :lens[b]], r)
        if kind == "step":
            c = torch.cat([c, _nearest64(state["new"][b])])
        if not len(c):
            outs.append(torch.zeros(case["H"] * D_V, dtype=torch.float64, device="cuda"))
            continue
        weights = torch.softmax(state["q_abs"][b].double() @ c.T * state["scale"], -1)
        o = ((weights @ c)[:, None, :] * state["w_uv"].double()).sum(-1).flatten()
        outs.append(o * torch.sigmoid(state["gate"][b].double()) if case["gate"] else o)
    return torch.stack(outs)
