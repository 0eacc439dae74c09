"""Serving over a paged latent cache, a run of tokens per sequence at a time: block tables and slot maps kept on the GPU,
latent rows appended through them, and the attention of each sequence's new tokens (a chunk of text or a tree of drafts)
to its cached rows, all of them or a sliding window and the first few; each in a plain form of elementary torch
operations and as the package's own calls.

The pool is [blocks, block_size, r] bf16; cache row u of sequence b is row u % block_size of block
block_table[b, u // block_size].  A sequence has lens[b] rows cached; its T new tokens' latents are rows lens[b] + t.

reserve  each sequence holds ceil((lens + counts) / block_size) blocks afterwards.  Blocks given up (in order of sequence
         and index) serve the sequences that need more, in the same order, then the top of the free stack does; those
         left over go back on the stack so that the first one given up is on top.  slots[b, t] is the pool row of token t,
         -1 from counts[b] on.
append   pool row slots[b, t] becomes c[b, t].
attend   token t of a chunk sees rows u <= lens + t; a drafted token sees the cached rows, its ancestors and itself.
         With a window of w, only rows whose position is among the last w up to its own, and those at positions below
         `sinks`, count; a draft's position is lens + its depth.
"""
import math

import torch

own = False

R = 512
D_V = 128
STD = 0.02   # weights; queries as q_abs = q . W_UK with q ~ N(0, 1) and d_q = 128


# ------------------------------------------------------------------------------------------------- cases
def _attend_case(B, T, H, lo, hi, bs=64, ld=R, tree=False, window=0, sinks=0, gate=True, ragged=False, edges=False):
    return dict(kind="attend", B=B, T=T, H=H, lo=lo, hi=hi, bs=bs, ld=ld, tree=tree, window=window, sinks=sinks, gate=gate,
                ragged=ragged, edges=edges)


def listed():
    return [
        # one step of speculative serving: room for 8 drafts in each of 64 conversations, then the drafts are dropped
        dict(name="reserve_64x8", kind="reserve", B=64, T=8, lo=1024, hi=32768, bs=64, fresh=False),
        # 512 prompts admitted to an empty cache and, later, all of them finished
        dict(name="reserve_512x2048", kind="reserve", B=512, T=2048, lo=1, hi=2048, bs=64, fresh=True),
        # 8 drafted tokens of 64 conversations
        dict(name="append_64x8", kind="append", B=64, T=8, lo=0, hi=1000, bs=64, ld=R, dtype="bfloat16"),
        # sixteen ragged prompts of up to 8192 tokens, straight from an fp32 norm
        dict(name="append_16x8192_f32", kind="append", B=16, T=8192, lo=0, hi=0, bs=256, ld=R, dtype="float32"),
        # one user's short conversation, 8 drafts, 16 heads: latency
        dict(name="tree_1x8_h16", **_attend_case(1, 8, 16, 1000, 1000, tree=True)),
        # drafts of 16 tokens in 32 conversations, all 96 heads
        dict(name="tree_32x16_h96", **_attend_case(32, 16, 96, 1024, 8192, tree=True)),
        # odd sizes: 61 drafts, 37 heads, rows inside wider records, token counts of their own, an empty and a one-row context
        dict(name="tree_7x61_h37", **_attend_case(7, 61, 37, 2, 5000, bs=128, ld=520, tree=True, ragged=True, edges=True)),
        # plain decode over the paged cache: 64 ragged conversations, one token each
        dict(name="decode_64x32768_h96", **_attend_case(64, 1, 96, 1024, 32768, gate=False)),
        # the same under a window of 4096 with 4 sinks
        dict(name="window_64x1_h96", **_attend_case(64, 1, 96, 1024, 32768, window=4096, sinks=4)),
        # a handful of conversations at the toy layer's 8 heads under a short window: latency
        dict(name="window_4x1_h8", **_attend_case(4, 1, 8, 1, 2000, window=256, sinks=4)),
        # chunked prefill of long documents under the window
        dict(name="window_8x512_h96", **_attend_case(8, 512, 96, 0, 30000, bs=256, window=4096, sinks=64)),
        # chunked prefill without one: mid-size layer's 16 heads, ragged chunks
        dict(name="chunk_16x256_h16", **_attend_case(16, 256, 16, 100, 4096, bs=128, ragged=True)),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    kind = rng.choice(["reserve", "append", "attend", "attend", "attend", "attend"])
    if kind == "reserve":
        B = _between(rng, 1, 1024)
        bs = 64 * rng.choice([1, 2, 4])
        if rng.random() < 0.5:
            T = _between(rng, 1, 64)
            hi = _between(rng, 1, 32768)
            return dict(kind=kind, B=B, T=T, lo=_between(rng, 1, hi), hi=hi, bs=bs, fresh=False)
        T = _between(rng, 1, min(8192, (1 << 20) // B))
        return dict(kind=kind, B=B, T=T, lo=1, hi=T, bs=bs, fresh=True)
    ld = R + 8 * rng.choice([0, 0, 1, 3, 8])
    bs = 64 * rng.choice([1, 1, 2, 3, 4])
    if kind == "append":
        B = _between(rng, 1, 64)
        T = _between(rng, 1, 131072 // B)
        return dict(kind=kind, B=B, T=T, lo=0, hi=rng.choice([0, 100, 1000]), bs=bs, ld=ld,
                    dtype=rng.choice(["bfloat16", "float32"]))
    tree = rng.random() < 0.5
    T = rng.choice([1, _between(rng, 1, 64), _between(rng, 1, 64 if tree else 512)])
    H = _between(rng, 1, 128)
    B = _between(rng, 1, 64)
    while B * T * H > 400000:
        B = (B + 1) // 2
        if B == 1:
            T = min(T, 400000 // H)
    # a score per (token, head, row): 1.5e9 of them are what the largest listed case has
    hi = _between(rng, 1, max(1, min(131072, 1300000 // B, 1500000000 // (B * T * H))))
    window = rng.choice([0, 0, _between(rng, 1, 8192)])
    lo = _between(rng, 1, hi) if rng.random() < 0.8 else 0
    return _attend_case(B, T, H, lo, hi, bs=bs, ld=ld, tree=tree, window=window,
                        sinks=_between(rng, 1, 128) - 1 if window else 0, gate=rng.random() < 0.5,
                        ragged=rng.random() < 0.5, edges=B > 2 and rng.random() < 0.5)


def _lens(case):
    """Ragged numbers of cached rows, evenly spread over [lo, hi] (their order comes from the seed)."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    lens = [lo + int((hi - lo) * (i + 0.5) / B) for i in range(B)]
    if case.get("edges"):
        lens[:2] = [0, 1]
    return lens


def _counts(case):
    """New tokens of the sequences, in the order of _lens: T each, or spread over [1, T] with one that has none."""
    B, T = case["B"], case["T"]
    if not case.get("ragged"):
        return [T] * B
    counts = [max(1, T - (5 * i) % T) for i in range(B)]
    if case.get("edges"):
        counts[2] = 0
    return counts


def _order(case, seed):
    """The sequences' order: positions in _lens and _counts."""
    gen = torch.Generator().manual_seed(int(seed) * 31 + 7)
    return torch.randperm(case["B"], generator=gen).tolist()


# ------------------------------------------------------------------------------------------------- inputs
def _normal(gen, shape, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std


def _latent(gen, shape):
    """Latent rows as RMSNorm with unit gain leaves them."""
    x = _normal(gen, shape)
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True))


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _pages(gen, rows, bs):
    """A block table for sequences of these many rows, blocks in any order, and how many blocks there are."""
    held = [-(-n // bs) for n in rows]
    total, wide = sum(held), max(max(held), 1)
    ids = torch.randperm(total + 1, generator=gen, device="cuda").int()
    at = torch.tensor([0] + held, device="cuda").cumsum(0)[:-1]
    j = torch.arange(wide, device="cuda")
    table = ids[(at[:, None] + j).clamp(max=total)]
    return torch.where(j < _ints(held)[:, None], table, -1).contiguous(), total + 1


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 29)
    kind, B, T, bs = case["kind"], case["B"], case["T"], case["bs"]
    order = _order(case, seed)
    lens = [_lens(case)[i] for i in order]
    if kind == "reserve":
        counts = lens if case["fresh"] else [T] * B
        lens = [0] * B if case["fresh"] else lens
        held = [-(-n // bs) for n in lens]
        wide = -(-(max(lens) + T) // bs)
        used, more = sum(held), sum(-(-(n + c) // bs) for n, c in zip(lens, counts)) - sum(held)
        ids = torch.randperm(used + more + 100, generator=gen, device="cuda").int()
        table = torch.full((B, wide), -1, dtype=torch.int32, device="cuda")
        j = torch.arange(wide, device="cuda")
        at = torch.tensor([0] + held, device="cuda").cumsum(0)[:-1]
        table = torch.where(j < _ints(held)[:, None], ids[(at[:, None] + j).clamp(max=len(ids) - 1)], table).contiguous()
        free = torch.cat([ids[used:], torch.full((used,), -1, dtype=torch.int32, device="cuda")])
        return dict(case=case, lens=_ints(lens), counts=_ints(counts), none=_ints([0] * B), table=table, held=_ints(held),
                    free=free, free_count=_ints([more + 100]))
    counts = [T] * B if kind == "append" else [_counts(case)[i] for i in order]
    rows = [n + c for n, c in zip(lens, counts)]
    table, blocks = _pages(gen, rows, bs)
    records = torch.zeros((blocks, bs, case["ld"]), dtype=torch.bfloat16, device="cuda")
    pool = records[:, :, :R]
    for i in range(0, blocks, 512):
        part = pool[i:i + 512]
        part.copy_(_latent(gen, part.shape))
    state = dict(case=case, lens=_ints(lens), host_lens=lens, host_counts=counts, table=table, pool=pool)
    t = torch.arange(T, device="cuda")
    if kind == "append":
        u = state["lens"].long()[:, None] + t
        state["slots"] = (table.long().gather(1, u // bs) * bs + u % bs).int()
        state["new"] = _latent(gen, (B, T, R)).to(getattr(torch, case["dtype"]))
        return state
    H = case["H"]
    state["scale"] = 1.0 if H > 48 else 1.0 / math.sqrt(128.0)
    state["q_abs"] = _normal(gen, (B, T, H, R), math.sqrt(128.0) * STD).to(torch.bfloat16)
    state["w_uv"] = _normal(gen, (H, D_V, R), STD).to(torch.bfloat16)
    state["gate"] = _normal(gen, (B, T, H * D_V)).to(torch.bfloat16) if case["gate"] else None
    state["counts"] = _ints(counts) if case["ragged"] else None
    state["out"] = torch.zeros((B, T, H * D_V), dtype=torch.bfloat16, device="cuda")
    state["parents"] = None
    if case["tree"]:   # a few roots; every other draft hangs on one of those before it, more often on a recent one
        r = torch.rand((B, T), generator=gen, device="cuda")
        up = torch.where(r < 0.5, t - 1, (r.square() * t).long() - 1)
        state["parents"] = torch.minimum(up, t - 1).int().contiguous()
    return state


# ------------------------------------------------------------------------------------------------- plain forms
def _reserve(state, lens, counts):
    case, table, held, free, free_count = state["case"], state["table"], state["held"], state["free"], state["free_count"]
    bs, T = case["bs"], case["T"]
    B, wide = table.shape
    need = (lens + counts + bs - 1) // bs
    up, down = (need - held).clamp(min=0).long(), (held - need).clamp(min=0).long()
    a0, r0 = up.cumsum(0) - up, down.cumsum(0) - down
    A, Rel, F = up.sum(), down.sum(), free_count.long()[0]
    j = torch.arange(wide, device="cuda")
    # the blocks given up, by their number; the others' go to a place behind the last
    gone = (j >= need[:, None]) & (j < held[:, None])
    k = torch.where(gone, r0[:, None] + j - need[:, None], B * wide)
    released = torch.zeros(B * wide + 1, dtype=torch.int32, device="cuda").scatter_(0, k.flatten(), table.flatten())
    new = (j >= held[:, None]) & (j < need[:, None])
    k = a0[:, None] + j - held[:, None]
    took = torch.where(k < Rel, released[k.clamp(0, B * wide)], free[(F - 1 - (k - Rel)).clamp(0, len(free) - 1)])
    table.copy_(torch.where(new, took, table))
    k = F + Rel - 1 - torch.arange(len(free), device="cuda")      # of each place of the stack
    back = (k >= A) & (k < Rel)
    free.copy_(torch.where(back, released[k.clamp(0, B * wide)], free))
    free_count.copy_((F + Rel - A).int().reshape(1))
    held.copy_(need)
    t = torch.arange(T, device="cuda")
    u = (lens[:, None] + t).long()
    slots = table.gather(1, (u // bs).clamp(max=wide - 1)).long() * bs + u % bs
    return torch.where(t < counts[:, None], slots, -1).int()


def _ancestors(parents):
    """[T, T] truth values: whether token a is token t or above it (rows t)."""
    T = parents.shape[0]
    t = torch.arange(T, device=parents.device)
    hang = (t[None, :] == parents.long()[:, None]).float()
    seen = torch.eye(T, device=parents.device)
    for _ in range(max(T - 1, 1).bit_length()):      # paths of up to 1, 2, 4, ... steps
        seen = ((seen + seen @ hang) > 0).float()
        hang = hang @ hang
    return seen > 0


def _attend(state):
    case, lens, counts = state["case"], state["host_lens"], state["host_counts"]
    bs, H, w, sinks, out = case["bs"], case["H"], case["window"], case["sinks"], state["out"]
    w_uv = state["w_uv"].float()
    for b, (n, c) in enumerate(zip(lens, counts)):
        if c == 0:
            continue
        lo = max(n - w + 1, 0) if w else 0           # rows that no token's window reaches are left out
        head = min(sinks, lo)
        u = torch.cat([torch.arange(head, device="cuda"), torch.arange(lo, n + c, device="cuda")])
        k = state["pool"][state["table"][b].long()[u // bs], u % bs].float()
        t = torch.arange(c, device="cuda")
        if case["tree"]:
            above = _ancestors(state["parents"][b, :c])
            depth = above.sum(1) - 1
            at = torch.where(u < n, u, n + depth[(u - n).clamp(min=0)])
            p = n + depth
            seen = (u < n) | above[:, (u - n).clamp(min=0)]
        else:
            at, p = u, n + t
            seen = u <= p[:, None]
        if w:
            seen = seen & ((at > p[:, None] - w) | (at < sinks))
        s = torch.matmul(state["q_abs"][b, :c].float().reshape(c * H, R), k.T).reshape(c, H, -1) * state["scale"]
        s = torch.where(seen[:, None, :], s, -math.inf)
        s = torch.exp(s - s.amax(-1, keepdim=True))
        o = torch.matmul(s.reshape(c * H, -1), k).reshape(c, H, R) / s.sum(-1, keepdim=True)
        o = torch.matmul(o.transpose(0, 1), w_uv.transpose(1, 2)).transpose(0, 1).reshape(c, H * D_V)
        if state["gate"] is not None:
            o = o / (1.0 + torch.exp(-state["gate"][b, :c].float()))
        out[b, :c] = o.to(torch.bfloat16)
    return out


def run(state):
    case = state["case"]
    kind, bs = case["kind"], case["bs"]
    if kind == "reserve":
        if own:
            import latent_compressed_attention_gb300 as lca

            def step(lens, counts, T):
                return lca.mla_reserve_latent_blocks(lens, counts, T, state["table"], state["held"], state["free"],
                                                     state["free_count"], bs)
        else:
            def step(lens, counts, T):
                return _reserve(state, lens, counts)
        slots = step(state["lens"], state["counts"], case["T"])
        step(state["none"] if case["fresh"] else state["lens"], state["none"], 0)
        return [slots, state["table"], state["held"], state["free"], state["free_count"]]
    if kind == "append":
        if own:
            import latent_compressed_attention_gb300 as lca

            return lca.mla_append_latent_paged(state["new"], state["pool"], state["slots"])
        at = state["slots"].long().flatten()
        state["pool"][at // bs, at % bs] = state["new"].flatten(0, 1).to(torch.bfloat16)
        return state["pool"]
    if own:
        import latent_compressed_attention_gb300 as lca

        return lca.mla_latent_attend_paged(state["q_abs"], state["pool"], state["table"], state["lens"], state["w_uv"],
                                           counts=state["counts"], parents=state["parents"], gate=state["gate"],
                                           scale=state["scale"], window=case["window"], sinks=case["sinks"],
                                           out=state["out"])
    return _attend(state)


# ------------------------------------------------------------------------------------------------- floors
def _seen(case, n, c):
    """Rows that a sequence's tokens see between them, and how many each sees, added up (a tree as its chain)."""
    w, sinks = case["window"], case["sinks"]
    if not w:
        return n + c, sum(n + t + 1 for t in range(c))
    lo = max(n - w + 1, 0)
    each = sum(min(w, n + t + 1) + min(sinks, max(n + t + 1 - w, 0)) for t in range(c))
    return min(sinks, lo) + n + c - lo, each


def work(case):
    kind, B, T, bs = case["kind"], case["B"], case["T"], case["bs"]
    if kind == "reserve":   # lengths, counts and held blocks in, held out, a block moved from the stack to the table; twice
        lens = [0] * B if case["fresh"] else _lens(case)
        counts = _lens(case) if case["fresh"] else [T] * B
        moved = sum(-(-(n + c) // bs) + -n // bs for n, c in zip(lens, counts))
        return dict(bytes=2 * (16 * B + 8 * moved) + 4 * B * T, flops=0)
    if kind == "append":
        es = 4 if case["dtype"] == "float32" else 2
        return dict(bytes=B * T * (R * es + R * 2 + 4), flops=0)
    H = case["H"]
    bytes_, flops, tokens = H * D_V * R * 2, 0, 0
    for n, c in zip(_lens(case), _counts(case)):
        if c:
            rows, each = _seen(case, n, c)
            bytes_ += rows * R * 2 + -(-rows // bs) * 4
            flops += 4 * R * H * each
            tokens += c
    bytes_ += tokens * H * (R * 2 + D_V * 2 * (2 if case["gate"] else 1)) + 4 * B + (4 * tokens if case["tree"] else 0)
    return dict(bytes=bytes_, flops=flops + 2 * tokens * H * R * D_V)


# ------------------------------------------------------------------------------------------------- in 64 bits
def _reserve_one_by_one(state):
    case = state["case"]
    bs, T = case["bs"], case["T"]
    lens, counts = state["lens"].tolist(), state["counts"].tolist()
    table, held = state["table"].tolist(), state["held"].tolist()
    free, left = state["free"].tolist(), state["free_count"].item()
    stack = free[:left]

    def step(lens, counts):
        need = [-(-(n + c) // bs) for n, c in zip(lens, counts)]
        given = [table[b][j] for b in range(len(lens)) for j in range(need[b], held[b])]
        for block in reversed(given):
            stack.append(block)
        for b in range(len(lens)):
            for j in range(held[b], need[b]):
                table[b][j] = stack.pop()
            held[b] = need[b]

    step(lens, counts)
    slots = [[table[b][(n + t) // bs] * bs + (n + t) % bs if t < c else -1 for t in range(T)]
             for b, (n, c) in enumerate(zip(lens, counts))]
    step([0] * len(lens) if case["fresh"] else lens, [0] * len(lens))
    free[:len(stack)] = stack
    return [torch.tensor(x, device="cuda") for x in (slots, table, held, free, [len(stack)])]


def exact(case, seed):
    state = prepare(case, seed)
    if case["kind"] == "reserve":
        return _reserve_one_by_one(state)
    bs = case["bs"]
    if case["kind"] == "append":
        rows = state["pool"].double().reshape(-1, R)
        rows[state["slots"].long().reshape(-1)] = state["new"].double().reshape(-1, R)
        return rows.reshape(state["pool"].shape)
    H, w, sinks = case["H"], case["window"], case["sinks"]
    out = torch.zeros((case["B"], case["T"], H * D_V), dtype=torch.float64, device="cuda")
    flat = state["pool"].reshape(-1, R) if state["pool"].is_contiguous() else state["pool"].flatten(0, 1)
    for b, (n, c) in enumerate(zip(state["host_lens"], state["host_counts"])):
        if c == 0:
            continue
        at = [(state["table"][b, u0] * bs + torch.arange(bs, device="cuda"))
              for u0 in range(-(-(n + c) // bs))]
        cache = flat[torch.cat(at).long()[:n + c]].double()
        parents = state["parents"][b, :c].tolist() if case["tree"] else list(range(-1, c - 1))
        hidden = torch.ones((c, n + c), dtype=torch.bool, device="cuda")
        depth = []
        for t in range(c):
            up = parents[t]
            depth.append(0 if up < 0 else depth[up] + 1)
            first = max(n + depth[t] - w + 1, 0) if w else 0      # the first position inside the window
            hidden[t, first:n] = False
            hidden[t, :min(sinks, n)] = False
        if case["tree"]:
            lines = []
            for t in range(c):
                a = t
                while a >= 0:
                    if not w or depth[t] - depth[a] < w or n + depth[a] < sinks:
                        lines.append((t, n + a))
                    a = parents[a]
            lines = torch.tensor(lines, device="cuda")
            hidden[lines[:, 0], lines[:, 1]] = False
        else:
            t, u = torch.arange(c, device="cuda")[:, None], torch.arange(c, device="cuda")
            hidden[:, n:] = (u > t) | ((t - u >= w) & (n + u >= sinks) if w else u > t)
        for h in range(0, H, 16):
            q = state["q_abs"][b, :c, h:h + 16].double()
            s = torch.einsum("thr,ur->htu", q, cache) * state["scale"]
            p = torch.softmax(s.masked_fill(hidden, -math.inf), -1)
            o = torch.einsum("htr,hvr->thv", p @ cache, state["w_uv"][h:h + 16].double())
            out[b, :c, h * D_V:(h + 16) * D_V] = o.reshape(c, -1)
        if case["gate"]:
            out[b, :c] *= torch.sigmoid(state["gate"][b, :c].double())
    return out
