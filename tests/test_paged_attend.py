"""GPU parity of mla_latent_attend_paged (chunks, drafted trees, windows with sinks over a paged cache) against the
definition in 64 bits, within an elementwise bound that counts the roundings of the call's documentation.

With weights a_u, latent o = sum a_u c_u and y = W o, a value is off by at most
    2^-8 |out|                                   the output's rounding to bf16 (half a step: 2^-8 relative)
  + s 2^-10 sum_j |W_j| A_j                      o kept as f16 (s the gate's sigmoid, A_j as below): with parts i of weights
                                                 g_i, sum g_i = 1, the parts' roundings sum to 2^-11 sum_i g_i |o_ij| <=
                                                 2^-11 A_j, and the joined row is rounded again, by 2^-11 |o_j| <= 2^-11 A_j
  + s 2^-16 sum_j |W_j| |o_j|                    o in two bf16 parts before W_UV
  + s 2^-8 sum_j |W_j| A_j,  A_j = sum a_u |c_uj|   the weights' rounding to bf16
  + s E sum_j |W_j| A_j                          everything in fp32
where E covers, relative to a weight, the scores' sums of 512 products, exact one by one, in fp32 (each of 512 additions
rounds a partial sum of at most S = max_u |scale| sum_j |q_j c_uj| by 2^-24 of it: 512 * 2^-24 * S, twice because the
normaliser moves too), the exponent's FMA on scores and maxima of up to S log2(e) (2^-23 S each way), ex2's own error (2^-21),
and the sums over n rows, the rescalings and the join (each rounds a sum by 2^-24, at most n + 2^10 of them, in the
numerator and the normaliser: (n + 2^10) 2^-23) and the two products with 512 terms (2^-14).  Second-order terms take
another 2 %.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

R, D_V, BOUNDS = 512, 128, -9


@pytest.fixture(scope="module")
def env():
    import torch

    import latent_compressed_attention_gb300 as lca
    lca.build()
    lca.mla_get_device_error()
    return torch, lca


def problem(env, T, H, lens, counts=None, bs=64, ld=R, tree=None, window=0, sinks=0, gate=True, scale=None, q_std=0.25,
            seed=0, spare=3):
    """A call's arguments.  The pool holds NaN wherever no sequence has a row, and the table a block that does not exist
    wherever a sequence has none."""
    torch, _ = env
    gen = torch.Generator(device="cuda").manual_seed(seed * 1009 + T * 31 + H)
    rng = np.random.default_rng([seed, T, H])
    B = len(lens)
    rows = [n + c for n, c in zip(lens, counts or [T] * B)]
    held = [-(-n // bs) for n in rows]
    ids = rng.permutation(sum(held) + spare)
    table = np.full((B, max(held) + 1), -7)
    records = torch.full((sum(held) + spare, bs, ld), float("nan"), dtype=torch.bfloat16, device="cuda")
    pool, at = records[:, :, :R], 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
        x = torch.randn((rows[b], R), generator=gen, device="cuda")
        x = (x * torch.rsqrt(x.square().mean(-1, keepdim=True))).to(torch.bfloat16)
        for j in range(held[b]):
            part = x[j * bs:(j + 1) * bs]
            pool[int(table[b, j]), :len(part)] = part
    i32 = dict(dtype=torch.int32, device="cuda")
    parents = None
    if tree is not None:
        t = np.arange(T)
        near = np.maximum(rng.integers(-1, np.maximum(t, 1)), t - 1 - rng.integers(0, 4, T))
        up = {"star": t * 0 - 1, "chain": t - 1, "mixed": near}[tree]
        parents = torch.tensor(np.tile(np.minimum(up, t - 1), (B, 1)), **i32)
        if tree == "mixed" and B > 1:
            parents[1:] = torch.tensor(np.stack([rng.integers(-1, np.maximum(t, 1)) * (t > 0) - (t == 0) for _ in range(B - 1)]), **i32)
    return dict(q_abs=(torch.randn((B, T, H, R), generator=gen, device="cuda") * q_std).to(torch.bfloat16), pool=pool,
                block_table=torch.tensor(table, **i32), lens=torch.tensor(lens, **i32),
                w_uv=(torch.randn((H, D_V, R), generator=gen, device="cuda") * 0.05).to(torch.bfloat16),
                counts=None if counts is None else torch.tensor(counts, **i32), parents=parents,
                gate=(torch.randn((B, T, H * D_V), generator=gen, device="cuda") * 2).to(torch.bfloat16) if gate else None,
                scale=1 / math.sqrt(128) if scale is None else scale, window=window, sinks=sinks)


def visible(n, c, parents, window, sinks):
    """[c, n + c] truth values, one token after the other."""
    seen, depth = np.zeros((c, n + c), bool), []
    for t in range(c):
        up = t - 1 if parents is None else parents[t]
        depth.append(depth[up] + 1 if up >= 0 else 0)
        position = np.concatenate([np.arange(n), n + np.array(depth)])
        near = position > n + depth[t] - window if window else np.ones(n + t + 1, bool)
        seen[t, :n] = (near | (position < sinks))[:n]
        a = t
        while a >= 0:
            seen[t, n + a] = near[n + a] or position[n + a] < sinks
            a = a - 1 if parents is None else parents[a]
    return seen


def reference(env, d):
    """Per sequence (b, count): the exact outputs and what they may be off by, [count, H * 128] in 64 bits."""
    torch, _ = env
    T, H = d["q_abs"].shape[1:3]
    bs = d["pool"].shape[1]
    w = d["w_uv"].double()
    for b, n in enumerate(d["lens"].tolist()):
        c = T if d["counts"] is None else int(d["counts"][b])
        if c == 0:
            continue
        u = torch.arange(n + c, device="cuda")
        k = d["pool"][d["block_table"][b].long()[u // bs], u % bs].double()
        seen = visible(n, c, None if d["parents"] is None else d["parents"][b].tolist(), d["window"], d["sinks"])
        seen = torch.tensor(seen, device="cuda")
        used = seen.any(0)
        k, seen = k[used], seen[:, used]
        q = d["q_abs"][b, :c].double()
        out, off = torch.empty((2, c, H, D_V), dtype=torch.float64, device="cuda")
        for h in range(H):
            s = q[:, h] @ k.T * d["scale"]
            a = torch.softmax(s.masked_fill(~seen, -math.inf), -1)
            o, A = a @ k, a @ k.abs()
            out[:, h] = o @ w[h].T
            S = (q[:, h].abs() @ k.abs().T * abs(d["scale"])).max(-1, keepdim=True).values
            E = 2 * 512 * 2.0**-24 * S + 4 * 2.0**-23 * 1.45 * S + 2.0**-20 + (len(k) + 2**10) * 2.0**-23 + 2.0**-14
            off[:, h] = 2.0**-16 * (o.abs() @ w[h].abs().T) + (2.0**-8 + 2.0**-10 + E) * (A @ w[h].abs().T)
        if d["gate"] is not None:
            g = torch.sigmoid(d["gate"][b, :c].double()).view(c, H, D_V)
            out, off = out * g, off * g
        off = 1.02 * (off + 2.0**-8 * out.abs()) + 1e-30
        yield b, c, out.reshape(c, -1), off.reshape(c, -1)


def attend(env, d, **more):
    return env[1].mla_latent_attend_paged(**(d | more))


def check(env, d, got=None, error=0):
    torch, lca = env
    if got is None:
        out = torch.full((*d["q_abs"].shape[:2], d["q_abs"].shape[2] * D_V), 7.0, dtype=torch.bfloat16, device="cuda")
        got = attend(env, d, out=out)
    assert lca.mla_get_device_error() == error
    left = torch.ones(got.shape[:2], dtype=torch.bool, device="cuda")
    for b, c, out, off in reference(env, d):
        err = (got[b, :c].double() - out).abs()
        assert bool((err <= off).all()), f"sequence {b}: {float((err / off).max()):.3f} of what it may be off by"
        left[b, :c] = False
    assert bool((got[left] == 7.0).all())
    return got


@pytest.mark.parametrize("T,H,lens,kw", [
    (1, 1, [0], dict()),
    (1, 1, [62, 63, 64, 65], dict()),
    (1, 96, [0, 63, 1000], dict(gate=False, scale=1.0)),
    (1, 128, [64, 129, 5], dict(bs=128)),
    (1, 16, [5000], dict(bs=192)),
    (2, 64, [126, 127, 128], dict()),
    (2, 20, [70000], dict()),
    (5, 96, [127, 124, 0], dict(ld=520)),
    (3, 16, [100, 200, 300, 400], dict(counts=[0, 1, 2, 3])),
    (1, 8, [10, 20, 30], dict(counts=[0, 0, 0])),
    (200, 8, [0, 100], dict(bs=256)),
    (130, 3, [0, 1, 640], dict(counts=[130, 129, 7])),
    (257, 37, [3], dict()),
    (16, 96, [333, 1], dict(tree="mixed")),
    (64, 5, [300, 0], dict(tree="mixed")),
    (64, 128, [191], dict(tree="chain")),
    (61, 37, [5, 777], dict(tree="star", counts=[61, 13], bs=128, ld=576)),
    (8, 16, [1000], dict(tree="mixed")),
    (1, 33, [64], dict(tree="star"))])
def test_shapes(env, T, H, lens, kw):
    check(env, problem(env, T, H, lens, **kw))


@pytest.mark.parametrize("T,H,lens,kw", [
    (1, 96, [5000, 4095, 4096, 10], dict(window=4096, sinks=4)),
    (1, 8, [0, 1, 255, 256, 257, 1000], dict(window=256, sinks=4)),
    (1, 16, [1000, 3], dict(window=1)),
    (1, 16, [1000, 0, 130], dict(window=1, sinks=1)),
    (9, 24, [500, 0, 60], dict(window=50, sinks=200)),
    (130, 3, [0, 500], dict(window=50, sinks=4)),
    (130, 20, [3000], dict(window=1000, sinks=130)),
    (300, 4, [70], dict(window=64)),
    (5, 16, [5, 700], dict(window=2**31 - 1, sinks=2**31 - 1)),
    (5, 16, [5, 700], dict(sinks=9)),
    (40, 12, [1, 100], dict(window=3, sinks=2, tree="mixed")),
    (40, 12, [0, 700], dict(window=7, sinks=300, tree="chain")),
    (64, 3, [2, 900], dict(window=100, sinks=70, tree="mixed")),
    (64, 2, [2, 900], dict(window=1, tree="mixed"))])
def test_windows(env, T, H, lens, kw):
    check(env, problem(env, T, H, lens, **kw))


@pytest.mark.parametrize("scale", [0.0, -0.1, 1e-20, 3.0])
@pytest.mark.parametrize("T,tree", [(1, None), (6, "mixed"), (150, None)])
def test_scales(env, T, tree, scale):
    check(env, problem(env, T, 24, [700, 130], tree=tree, scale=scale, window=200 if tree else 0, sinks=2))


def test_many_sequences(env):
    rng = np.random.default_rng(3)
    check(env, problem(env, 2, 3, rng.integers(0, 400, 333).tolist(), counts=rng.integers(0, 3, 333).tolist()))


@pytest.mark.parametrize("lens", [[0, 0, 0, 700], [0, 300], [0], [130, 0, 0, 0, 0, 1500]])
def test_short_sequences_before_long_ones(env, lens):
    """Clusters that take several tiles of one unit of the cache each and then longer ones, in many orders."""
    check(env, problem(env, 1, 2, (lens * 400)[:400 if len(lens) > 1 else 1000]))


@pytest.mark.parametrize("T,lens", [(24, [20000, 9000, 24000, 6000, 21000, 13000, 700, 12500, 25000]), (40, [9000] * 14)])
def test_rounds_of_shares(env, T, lens):
    """Sequences of many tiles whose rows are more than a round's: every cluster has several shares."""
    d = problem(env, T, 64, lens, gate=False)
    got = attend(env, d)
    assert env[1].mla_get_device_error() == 0
    rng = np.random.default_rng(5)
    pick = sorted(rng.choice(64, 6, replace=False).tolist())    # heads to compare: the reference takes long
    some = dict(d, q_abs=d["q_abs"][:, :, pick].contiguous(), w_uv=d["w_uv"][pick].contiguous())
    for b, c, out, off in reference(env, some):
        err = (got[b, :c].view(c, 64, D_V)[:, pick].reshape(c, -1).double() - out).abs()
        assert bool((err <= off).all()), f"sequence {b}: {float((err / off).max()):.3f} of what it may be off by"


def test_rising_scores(env):
    """Each token's scores rise along the cache by far more than a softmax keeps, in a different direction per head."""
    torch, _ = env
    d = problem(env, 3, 48, [3000], seed=8, gate=False)
    u = torch.arange(3003, device="cuda")
    ramp = torch.linspace(0, 1, 3003, device="cuda")
    k = torch.randn(3003, R, device="cuda") * 0.1
    k[:, 0], k[:, 1], k[:, 2] = ramp * 4, (1 - ramp) * 4, torch.sin(ramp * 60) * 4
    d["pool"][d["block_table"][0].long()[u // 64], u % 64] = k.to(torch.bfloat16)
    d["q_abs"][..., :3] = 0
    for h in range(48):
        d["q_abs"][:, :, h, h % 3] = 40.0 * (1 + h // 3)
    d["scale"] = 1.0
    check(env, d)


def test_hidden_rows_have_no_effect(env):
    """NaN and infinities in rows that some tokens see and others do not: a sibling's, a later token's, one outside the
    window.  Those that see one get NaN; the others what they get without it."""
    torch, _ = env
    for bad in (float("nan"), float("inf"), -float("inf")):
        d = problem(env, 12, 96, [200], tree="star", seed=9)
        clean = attend(env, d)
        d["pool"][int(d["block_table"][0, 203 // 64]), 203 % 64, 17] = bad
        got = attend(env, d)
        assert bool(got[0, 3].isnan().all())
        rest = [t for t in range(12) if t != 3]
        assert torch.equal(got[0, rest], clean[0, rest])
        d = problem(env, 70, 6, [200], window=30, sinks=3, seed=10)
        clean = attend(env, d)
        for row in (1, 171 + 40, 268):     # a sink, one that tokens 11 .. 40 see, one that 68 and 69 see
            c = d["pool"][int(d["block_table"][0, row // 64]), row % 64]
            kept = c.clone()
            c[400] = bad
            got = attend(env, d)
            hit = [t for t in range(70) if row < 3 or row <= 200 + t < row + 30]
            rest = [t for t in range(70) if t not in hit]
            assert bool(got[0, hit].isnan().all()) and torch.equal(got[0, rest], clean[0, rest])
            c.copy_(kept)
    assert env[1].mla_get_device_error() == 0


@pytest.mark.parametrize("tree", [None, "mixed"])
@pytest.mark.parametrize("bs", [64, 192])
def test_blocks_behind_the_window_may_be_given_back(env, bs, tree):
    """Table entries of blocks of which no token sees a row are not read, wherever they end in a unit of 128 rows."""
    for T, lens, window, sinks in ((1, [500, 640, 1000], 70, 3), (5, [700, 449, 66], 129, 65), (7, [2000], 1, 0), (3, [900], 192, 0)):
        d = problem(env, T, 40, lens, bs=bs, tree=tree, window=window, sinks=sinks, seed=bs)
        gone = 0
        for b, n in enumerate(lens):
            for j in range(-(-n // bs)):
                if j * bs >= sinks and (j + 1) * bs <= n - window + 1:
                    d["block_table"][b, j] = -1
                    gone += 1
        assert gone
        d["block_table"] = d["block_table"][:, :-1]   # as wide as the longest sequence and no wider
        check(env, d)


def test_nan_in_a_row_that_all_see(env):
    torch, _ = env
    d = problem(env, 2, 96, [700, 700])
    d["pool"][int(d["block_table"][0, 3]), 5, 9] = float("nan")
    got = attend(env, d)
    assert bool(got[0].isnan().all()) and bool(got[1].isfinite().all())
    d = problem(env, 2, 16, [100])
    d["q_abs"][0, 1, 3, 77] = float("nan")
    got = attend(env, d).view(2, 16, D_V)
    assert bool(got[1, 3].isnan().all()) and int(got.isnan().sum()) == D_V


def test_reports(env):
    """Lengths, counts, blocks and parents out of range are reported; the other sequences' results stand."""
    torch, lca = env
    for key, value in (("lens", -1), ("lens", 2**31 - 1), ("lens", 4 * 64 - 1), ("counts", -1), ("counts", 4)):
        d = problem(env, 3, 16, [100, 130, 150], counts=[3, 2, 3])
        assert d["block_table"].shape[1] == 4
        want = attend(env, d, out=torch.full((3, 3, 16 * D_V), 7.0, dtype=torch.bfloat16, device="cuda"))
        d[key][1] = value
        got = attend(env, d, out=torch.full((3, 3, 16 * D_V), 7.0, dtype=torch.bfloat16, device="cuda"))
        assert lca.mla_get_device_error() == BOUNDS
        assert torch.equal(got[[0, 2]], want[[0, 2]]) and bool((got[1] == 7.0).all())
    for block in (-1, 10**6, 2**31 - 1, -2**31):
        d = problem(env, 2, 16, [100, 200])
        want = d["pool"][int(d["block_table"][0, 1])].clone()
        d["block_table"][0, 1] = block
        got = attend(env, d)
        assert lca.mla_get_device_error() == BOUNDS
        spare = problem(env, 2, 16, [100, 200])
        spare["pool"][int(spare["block_table"][0, 1])] = 0
        assert torch.equal(got, attend(env, spare))
        assert want.isfinite().any()
    for t, up in ((0, 0), (3, 3), (3, 7), (5, -2), (2, -2**31), (2, 2**31 - 1)):
        d = problem(env, 8, 16, [100, 200], tree="star")
        want = attend(env, d)
        d["parents"][1, t] = up
        got = attend(env, d)
        assert lca.mla_get_device_error() == BOUNDS and torch.equal(got, want)


def test_repeatable_and_shared_workspace(env):
    """The same bits whatever the workspace holds, on any stream, and from two captured graphs that share one."""
    torch, lca = env
    one = problem(env, 16, 96, [3000, 100, 900], tree="mixed", seed=1)
    two = problem(env, 1, 40, [9000, 20], window=2000, sinks=5, seed=2)
    need = max(lca.mla_latent_attend_paged_workspace_size(*d["q_abs"].shape) for d in (one, two))
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    want = [check(env, d) for d in (one, two)]
    for d, w in zip((one, two), want):
        for _ in range(4):
            assert torch.equal(attend(env, d, workspace=ws), w)
    outs, graphs = [torch.zeros_like(w) for w in want], []
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert torch.equal(attend(env, one), want[0])
    torch.cuda.synchronize()
    got = attend(env, two, stream=side)
    side.synchronize()
    assert torch.equal(got, want[1])
    for d, o in zip((one, two), outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            attend(env, d, workspace=ws, out=o)
        graphs.append(graph)
    for _ in range(3):
        for g in graphs:
            g.replay()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
            o.zero_()
    # a replay takes the lengths that it finds
    one["lens"].copy_(torch.tensor([2900, 90, 800], dtype=torch.int32, device="cuda"))
    graphs[0].replay()
    check(env, one, outs[0])
    assert lca.mla_get_device_error() == 0


@pytest.mark.parametrize("B,T", [(2, 3), (2, 40)])
def test_least_alignment(env, B, T):
    """Every tensor at the alignment that the call asks for and no more: 16 bytes, whole numbers 4."""
    torch, lca = env

    def moved(t, by):
        if t is None:
            return None
        flat = torch.empty(t.numel() + 64, dtype=t.dtype, device="cuda")
        at = next(i for i in range(64) if (flat.data_ptr() + i * t.element_size()) % 64 == by)
        return flat[at:at + t.numel()].view(t.shape).copy_(t)

    d = problem(env, T, 16, [100, 300][:B], counts=[T, T - 1], tree="mixed", window=50, sinks=3)
    want = attend(env, d)
    for key in d:
        if isinstance(d[key], torch.Tensor):
            d[key] = moved(d[key], 16 if d[key].dtype == torch.bfloat16 else 4)
    ws = torch.empty(lca.mla_latent_attend_paged_workspace_size(B, T, 16, R) + 64, dtype=torch.uint8, device="cuda")
    out = moved(torch.zeros_like(want), 16)
    got = attend(env, d, out=out, workspace=ws[next(i for i in range(64) if (ws.data_ptr() + i) % 64 == 16):])
    assert got.data_ptr() % 32 == 16 and torch.equal(got, want)


def test_queries_that_are_no_tokens(env):
    """Whatever the queries behind a sequence's last token hold, which share its last tile, has no effect."""
    torch, _ = env
    d = problem(env, 9, 20, [300, 70, 10], counts=[4, 9, 0], window=90, sinks=2)
    want = attend(env, d)
    for bad in (float("nan"), float("inf"), 3e38):
        for b, c in enumerate((4, 9, 0)):
            d["q_abs"][b, c:] = bad
        assert torch.equal(attend(env, d), want)
    assert env[1].mla_get_device_error() == 0


def test_views(env):
    """Tables and pools that are views, a pool of one block, a call without tokens or sequences."""
    torch, lca = env
    d = problem(env, 2, 16, [100, 200])
    want = attend(env, d)
    wide = torch.full((2, 40), -9, dtype=torch.int32, device="cuda")
    wide[:, 5:5 + d["block_table"].shape[1]] = d["block_table"]
    assert torch.equal(attend(env, d, block_table=wide[:, 5:5 + d["block_table"].shape[1]]), want)
    bigger = torch.zeros(d["pool"].shape[0] + 4, 64, R, dtype=torch.bfloat16, device="cuda")
    bigger[4:] = d["pool"]
    assert torch.equal(attend(env, d, pool=bigger[4:]), want)
    check(env, problem(env, 2, 16, [20], spare=0))
    for B, T in ((0, 2), (2, 0)):
        empty = dict(q_abs=d["q_abs"][:B, :T].contiguous(), lens=d["lens"][:B], block_table=d["block_table"][:B],
                     gate=d["gate"][:B, :T].contiguous())
        assert attend(env, d, **empty).shape == (B, T, 16 * D_V)
    assert lca.mla_get_device_error() == 0


def test_far_blocks(env):
    """Cache rows whose element offsets pass 2^32."""
    torch, _ = env
    d = problem(env, 3, 16, [500])
    pool = torch.empty(137000, 64, R, dtype=torch.bfloat16, device="cuda")
    n = d["pool"].shape[0]
    pool[-n:] = d["pool"]
    table = d["block_table"]
    table[table >= 0] += 137000 - n
    d["pool"] = pool
    check(env, d)


def test_refusals(env):
    torch, lca = env
    d = problem(env, 2, 16, [100, 200], counts=[1, 2], tree="star")
    q = d["q_abs"]
    for bad in (dict(q_abs=q.float()), dict(q_abs=q[0]), dict(q_abs=q[:, :, ::2]), dict(q_abs=q.cpu()), dict(lens=d["lens"][:1]),
                dict(lens=d["lens"].long()), dict(pool=d["pool"][:, :, :256]), dict(pool=d["pool"].float()),
                dict(pool=d["pool"][:, :32]), dict(w_uv=d["w_uv"][:15]), dict(gate=d["gate"][:, :1]), dict(counts=d["counts"][:1]),
                dict(parents=d["parents"][:, :1]), dict(parents=d["parents"].long()), dict(block_table=d["block_table"][:1]),
                dict(out=torch.empty(2, 2, 1, device="cuda")), dict(window=2**31), dict(sinks=-2**31 - 1),
                dict(workspace=torch.empty(64, 64, device="cuda")[:, ::2])):
        with pytest.raises((TypeError, ValueError)):
            attend(env, d, **bad)
    for bad in (dict(window=-1), dict(sinks=-1), dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(lca.MLAError):
            attend(env, d, **bad)
    with pytest.raises(lca.MLAError):
        attend(env, problem(env, 65, 2, [10], tree="star"))
    with pytest.raises(lca.MLAError):
        attend(env, problem(env, 1, 2, [10], bs=32))


def test_serving_steps(env):
    """Speculative serving as a program runs it: prompts in chunks, then rounds of a drafted tree of which a path is kept,
    sequences that end and start meanwhile, all through the block tables; every attention against 64 bits."""
    torch, lca = env
    rng = np.random.default_rng(12)
    B, H, bs, wide, blocks = 3, 12, 64, 12, 30
    i32 = dict(dtype=torch.int32, device="cuda")
    pool = torch.full((blocks, bs, R), float("nan"), dtype=torch.bfloat16, device="cuda")
    table, held = torch.full((B, wide), -1, **i32), torch.zeros(B, **i32)
    free, left = torch.randperm(blocks, device="cuda").int(), torch.tensor([blocks], **i32)
    w_uv = (torch.randn((H, D_V, R), device="cuda") * 0.05).to(torch.bfloat16)
    rows = [torch.empty(0, R, dtype=torch.bfloat16, device="cuda") for _ in range(B)]   # what each sequence has cached

    def step(T, counts, parents, window):
        lens_t, counts_t = torch.tensor([len(r) for r in rows], **i32), torch.tensor(counts, **i32)
        c = torch.randn((B, T, R), device="cuda").to(torch.bfloat16)
        slots = lca.mla_reserve_latent_blocks(lens_t, counts_t, T, table, held, free, left, bs)
        lca.mla_append_latent_paged(c, pool, slots)
        q = (torch.randn((B, T, H, R), device="cuda") * 0.25).to(torch.bfloat16)
        args = dict(q_abs=q, pool=pool, block_table=table, lens=lens_t, w_uv=w_uv, counts=counts_t, gate=None, scale=0.1,
                    parents=None if parents is None else torch.tensor(parents, **i32), window=window, sinks=3)
        out = attend(env, args)
        flat = torch.cat([torch.cat([rows[b], c[b, :counts[b]]]) for b in range(B)])
        alone = torch.zeros((B, wide * bs, R), dtype=torch.bfloat16, device="cuda")
        at = 0
        for b in range(B):
            n = len(rows[b]) + counts[b]
            alone[b, :n] = flat[at:at + n]
            at += n
        # the same rows in blocks one after the other
        same = dict(args, pool=alone.view(B * wide, bs, R), block_table=torch.arange(B * wide, **i32).view(B, wide))
        for b, n, want, off in reference(env, same):
            assert bool(((out[b, :n].double() - want).abs() <= off).all())
        assert bool((out[[b for b in range(B) if counts[b] == 0]] == 0).all())
        return c, slots

    for i in range(12):
        window = 0 if i % 2 else 100
        if i % 4 == 0:      # a chunk of prompt for some
            counts = [int(x) for x in rng.integers(0, 90, B)]
            c, _ = step(90, counts, None, window)
            rows = [torch.cat([rows[b], c[b, :counts[b]]]) for b in range(B)]
        else:
            T = 10
            parents = [[int(rng.integers(-1, t)) if t else -1 for t in range(T)] for _ in range(B)]
            counts = [T if len(rows[b]) else 0 for b in range(B)]
            c, slots = step(T, counts, parents, window)
            for b in range(B):
                if counts[b]:
                    path, a = [], int(rng.integers(0, T))
                    while a >= 0:
                        path.insert(0, a)
                        a = parents[b][a]
                    kept = c[b, path]    # the path's rows, one after the other, over the drafts'
                    lca.mla_append_latent_paged(kept, pool, slots[b, :len(path)])
                    rows[b] = torch.cat([rows[b], kept])
        if i == 6:
            rows[1] = rows[1][:0]   # this one ends; its blocks go back at the next step
    zero = torch.zeros(B, **i32)
    lca.mla_reserve_latent_blocks(zero, zero, 0, table, held, free, left, bs)
    assert int(left) == blocks and sorted(free.tolist()) == list(range(blocks))
    assert lca.mla_get_device_error() == 0
