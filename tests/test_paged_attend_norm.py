"""mla_latent_attend_paged over long caches, in norm.  An elementwise bound that adds up what every weight's rounding can do
at worst does not shrink with the number of rows, but the outputs do: over 20,000 rows it holds for zeros.  The bound here is
one on the error of a tile's outputs together, 128 (token, head) rows or those of them that are compared, and shrinks as they
do.  Its own tests, on the CPU, plant mistakes in the reference (a unit of rows left out or counted twice, a part's weight
off, a part's maximum forgotten) and see that it does not hold for them.

With y = G W o, o = sum_u a_u c_u (G the gate's sigmoid, a the softmax weights) the error is a sum of
  - the output's rounding to bf16: 2^-8 |y|;
  - sum_u a_u d_u G W c_u with |d_u| <= e = 2^-8 + E: a weight's rounding to bf16 (half a step) and the errors E of its score,
    E = 2 * 512 * 2^-24 S + 4 * 2^-23 * 1.45 S + 2^-20 with S = max_u |scale| sum_j |q_j c_uj| (512 exact products added in fp32
    for it and the maximum, the exponent's FMA, ex2);
  - twice sum_ij d_ij v_ij G W_j with |d_ij| <= 2^-11: a part i of o in f16, v_i = sum of a_u c_u over its rows, and the joined
    row in f16 again;
  - what is added in fp32, off by 2^-22 of a partial sum each time (a step of fp32, twice for a tensor core that truncates),
    once per 8 rows at most and 2^10 times more for the join, the rescalings, the normaliser and the product with W;
  - o in two bf16 parts, off by 2^-16 |o_j|, and the product's 512 terms: 2^-10 |D o| together, D_j = |G W_j| (Cauchy-Schwarz
    over 512 j: 2^-16 sqrt(512) and 64 * 2^-22 sqrt(512), together less than 2^-10).
The roundings d are of unrelated numbers: taken as independent, of mean 0 and uniform within their half steps (variance at
most 1/3 of the bound's square).  The norm of a sum M d with independent d in [-1, 1] is a convex function of d with Lipschitz
constant |M| (the operator norm), so that it passes its mean, at most sqrt(|M|_F^2 / 3), by t with a probability of at most
exp(-t^2 / (8 |M|^2)) (Boucheron, Lugosi and Massart, Concentration Inequalities, theorem 6.10, scaled to [-1, 1]): 14 |M| is
1e-10.  |M|^2 is the largest eigenvalue of G = M M^T, at most (tr G^8)^(1/8).  The rows' parts i are not known here.  For rows c_u = mean + independent rest, sum_i v_ij^2 is at most 2 mean_j^2 +
2 sum_u a_u^2 c_uj^2 and mean_j^2 at most 2 o_j^2 + 2 sum_u a_u^2 c_uj^2 (as means over the rest; the f16 roundings are an
eighth of the weights'): w_j^2 = 4 o_j^2 + 6 sum_u a_u^2 c_uj^2 takes sum_i v_ij^2's place.  Second-order terms take 2 %."""
import math

import numpy as np
import pytest
import torch

R, D_V, TILE = 512, 128, 128


def visible(positions, n, window, sinks, tree=None):
    """[tokens, n + new] truth values for tokens at these places of a chunk, or of a tree (each token's parent)."""
    new = max(positions) + 1 if tree is None else len(tree)
    u = torch.arange(n + new)
    seen = []
    for t in positions:
        if tree is None:
            p, row = n + t, u <= n + t
        else:
            above, a = [], t
            while a >= 0:
                above.append(a)
                a = tree[a]
            p, row = n + len(above) - 1, u < n
            row[[n + a for a in above]] = True
            assert not window
        if window:
            row = row & ((u > p - window) | (u < sinks))
        seen.append(row)
    return torch.stack(seen)


def exact(k, q, w, gate, seen, scale):
    """Of the rows k [n, R] with q [t, h, R], w [h, D_V, R], gate [t, h, D_V] or None and seen [t, n], all in 64 bits: y
    [t, h, D_V] and what the bound needs, per (t, h)."""
    t, h = q.shape[:2]
    y = torch.empty((t, h, D_V), dtype=torch.float64, device=k.device)
    s_max = torch.zeros((t, h), dtype=torch.float64, device=k.device)
    numbers = {name: torch.empty((t, h), dtype=torch.float64, device=k.device)
               for name in ("weights", "weights_top", "parts", "parts_top", "o")}
    for i in range(h):
        Y = k @ w[i].T
        s = (q[:, i] @ k.T) * scale
        a = torch.softmax(s.masked_fill(~seen, -math.inf), -1)
        s_max[:, i] = ((q[:, i].abs() @ k.abs().T) * abs(scale)).max(-1).values
        o = a @ k
        g = torch.ones((t, D_V), dtype=torch.float64, device=k.device) if gate is None else torch.sigmoid(gate[:, i])
        y[:, i] = g * (o @ w[i].T)
        W = g[:, :, None] * w[i]
        w2 = 4 * o ** 2 + 6 * a ** 2 @ k ** 2
        for name, grams in (("weights", torch.stack([(a[j, :, None] * Y * g[j]).T @ (a[j, :, None] * Y * g[j]) for j in range(t)])),
                            ("parts", (W * w2[:, None]) @ W.transpose(1, 2))):
            numbers[name][:, i] = grams.diagonal(dim1=1, dim2=2).sum(-1)
            two = (grams / numbers[name][:, i, None, None]) @ (grams / numbers[name][:, i, None, None])
            numbers[name + "_top"][:, i] = numbers[name][:, i] * (two @ two).square().sum((1, 2)) ** (1 / 8)
        numbers["o"][:, i] = (W.square().sum(1) * o ** 2).sum(-1)
    return y, dict(numbers, S=s_max, n=seen.sum(-1, keepdim=True).expand(t, h))


def allowed(y, x, rows):
    """What the error of these (token, head) rows may be in norm."""
    at = {name: v[rows] for name, v in x.items()}
    S = float(at["S"].max())
    e = 2.0**-8 + 2 * 512 * 2.0**-24 * S + 4 * 2.0**-23 * 1.45 * S + 2.0**-20
    near = lambda name: float((at[name].sum() / 3).sqrt() + 14 * at[name + "_top"].max().sqrt())   # noqa: E731
    added = (int(at["n"].max()) / 8 + 2**10) * 2.0**-22 * float(at["parts"].sum().sqrt())
    return 1.02 * (2.0**-8 * float(y[rows].norm()) + e * near("weights") + 2 * 2.0**-11 * near("parts") + added
                   + 2.0**-10 * float(at["o"].sum().sqrt()))


def share_of_allowed(got, y, x, tile):
    """The largest error of a tile's rows, as a part of what it may be; tile [t, h]: the tile of each row."""
    return max(float((got[tile == i] - y[tile == i]).norm()) / allowed(y, x, tile == i) for i in tile.unique().tolist())


# ------------------------------------------------------------------------------------------------- the bound itself (CPU)
def rows_of(gen, n, device):
    x = torch.randn((n, R), generator=gen, device=device)
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True))).to(torch.bfloat16)


def bits(x, n):
    """x rounded to n bits of mantissa."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(m * 2.0**n), e - n)


def in_parts(k, q, w, cuts, scale, weight=None, forget=None):
    """The outputs as the kernels compute them, with their roundings: rows [cuts[i], cuts[i + 1]) are a part each, with
    weights against the part's own maximum; the parts' weights times weight, one maximum forgotten."""
    t, h = q.shape[:2]
    y = torch.empty((t, h, D_V), dtype=torch.float64)
    for i in range(h):
        o, m, l = [], [], []
        for lo, hi in zip(cuts, cuts[1:]):
            s = (q[:, i] @ k[lo:hi].T) * scale
            m.append(s.max(-1, keepdim=True).values)
            p = torch.exp(s - m[-1])
            l.append(p.sum(-1, keepdim=True))
            o.append(bits(bits(p, 8) @ k[lo:hi] / l[-1], 11))
        top = torch.stack(m).max(0).values
        f = [torch.exp(m_i - top) * l_i for m_i, l_i in zip(m, l)]
        if weight is not None:
            f = [x * v for x, v in zip(f, weight)]
        if forget is not None:
            f[forget] = l[forget]
        row = bits(sum(x * v for x, v in zip(f, o)) / sum(f), 11)
        y[:, i] = row @ w[i].T
    return bits(y, 8)


@pytest.mark.parametrize("n,scale,parts", [(1000, 0.09, 3), (9000, 0.02, 5), (9000, 0.12, 9), (20000, 0.02, 4), (40000, 0.01, 8)])
def test_the_bound_sees_mistakes(n, scale, parts):
    gen = torch.Generator().manual_seed(n + parts)
    k = rows_of(gen, n, "cpu").double()
    q = (torch.randn((2, 3, R), generator=gen) * 0.25).to(torch.bfloat16).double()
    w = (torch.randn((3, D_V, R), generator=gen) * 0.05).to(torch.bfloat16).double()
    seen, tile = torch.ones((2, n), dtype=torch.bool), torch.zeros((2, 3), dtype=torch.int64)
    y, x = exact(k, q, w, None, seen, scale)
    cuts = [0] + sorted(int(c) * 128 for c in np.random.default_rng(n).choice(np.arange(1, n // 128), parts - 1, replace=False)) + [n]
    assert share_of_allowed(in_parts(k, q, w, cuts, scale), y, x, tile) < 0.8
    # a unit in the middle or at a part's border is left out, or counted twice
    for u0 in (n // 256 * 128, cuts[1], cuts[-2] - 128):
        left = torch.cat([torch.arange(u0), torch.arange(u0 + 128, n)])
        assert share_of_allowed(exact(k[left], q, w, None, seen[:, left], scale)[0], y, x, tile) > 1
        twice = torch.cat([torch.arange(n), torch.arange(u0, u0 + 128)])
        assert share_of_allowed(exact(k[twice], q, w, None, seen[:, twice % n], scale)[0], y, x, tile) > 1
    # a part is lost, or weighs a third more (one that has some of the rows: 128 of 9000 hardly count)
    for i in range(parts):
        for f in [0] + [4 / 3] * (cuts[i + 1] - cuts[i] > n / 16):
            weight = [f if j == i else 1.0 for j in range(parts)]
            assert share_of_allowed(in_parts(k, q, w, cuts, scale, weight=weight), y, x, tile) > 1
    if scale > 0.05:
        assert max(share_of_allowed(in_parts(k, q, w, cuts, scale, forget=i), y, x, tile) for i in range(parts)) > 1
    assert share_of_allowed(torch.zeros_like(y), y, x, tile) > 10


# ------------------------------------------------------------------------------------------------- the kernels (GPU)
@pytest.fixture(scope="module")
def lca():
    import latent_compressed_attention_gb300 as lca
    lca.build()
    lca.mla_get_device_error()
    return lca


def trees(rng, B, T):
    return [[int(rng.integers(max(t - 4, 0), t + 1)) - 1 for t in range(T)] for _ in range(B)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,lens,kernels,kw", [
    (1, 16, [5000], 2, dict(bs=192)),
    (2, 20, [70000], 2, dict(scale=0.01)),
    (2, 20, [9000, 33], 2, dict(scale=0.12, gate=True)),
    (1, 96, [1000 + 700 * i for i in range(40)], 2, dict()),
    (1, 96, [300 + 400 * i for i in range(80)], 2, dict(gate=True, window=2000, sinks=4)),
    (16, 96, [8000, 3000, 12000], 2, dict(tree=True)),
    (32, 96, [8000, 3000, 5, 12000], 3, dict(tree=True, gate=True, ld=520)),
    # several shares per cluster
    (24, 64, [20000, 9000, 24000, 6000, 21000, 13000, 700, 12500, 25000], 3, dict()),
    (40, 64, [9000] * 14, 3, dict(gate=True, heads=2)),
    (120, 32, [9000, 30000, 12000, 100, 25000, 18000], 3, dict(counts=[120, 7, 61, 120, 1, 90], window=20000, sinks=100)),
    # long chunks
    (300, 96, [20000, 100, 9000], 3, dict(window=4096, sinks=64, bs=256)),
    (1100, 16, [3000, 40], 3, dict(counts=[1100, 1051])),
    (8192, 3, [0, 500], 3, dict(counts=[8192, 7001], gate=True)),
    (8192, 2, [9000], 3, dict(window=1000, sinks=10))])
def test_long_caches(lca, T, H, lens, kernels, kw):
    counts, bs, ld, window, sinks = kw.get("counts"), kw.get("bs", 64), kw.get("ld", R), kw.get("window", 0), kw.get("sinks", 0)
    scale, B = kw.get("scale", 0.02), len(lens)
    gen = torch.Generator(device="cuda").manual_seed(T * 100 + H + B)
    rng = np.random.default_rng([T, H, B])
    rows = [n + c for n, c in zip(lens, counts or [T] * B)]
    held = [-(-n // bs) for n in rows]
    ids = rng.permutation(sum(held) + 3)
    records = torch.full((sum(held) + 3, bs, ld), float("nan"), dtype=torch.bfloat16, device="cuda")
    pool = records[:, :, :R]
    table, cache, at = np.full((B, max(held)), -7), [], 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
        cache.append(rows_of(gen, rows[b], "cuda"))
        u = torch.arange(rows[b], device="cuda")
        pool[torch.tensor(table[b], device="cuda")[u // bs], u % bs] = cache[b]
    i32 = dict(dtype=torch.int32, device="cuda")
    q = (torch.randn((B, T, H, R), generator=gen, device="cuda") * 0.25).to(torch.bfloat16)
    w_uv = (torch.randn((H, D_V, R), generator=gen, device="cuda") * 0.05).to(torch.bfloat16)
    gate = (torch.randn((B, T, H * D_V), generator=gen, device="cuda") * 2).to(torch.bfloat16) if kw.get("gate") else None
    parents = trees(rng, B, T) if kw.get("tree") else None
    before = lca.mla_kernel_launches()
    got = lca.mla_latent_attend_paged(q, pool, torch.tensor(table, **i32), torch.tensor(lens, **i32), w_uv, gate=gate, scale=scale,
                                      counts=None if counts is None else torch.tensor(counts, **i32), window=window, sinks=sinks,
                                      parents=None if parents is None else torch.tensor(parents, **i32))
    if torch.cuda.get_device_properties(0).multi_processor_count == 152:
        assert lca.mla_kernel_launches() - before == kernels
    assert lca.mla_get_device_error() == 0
    got = got.view(B, T, H, D_V)
    heads = sorted(rng.choice(H, min(H, kw.get("heads", 4)), replace=False).tolist())
    for b in range(B):
        c = T if counts is None else counts[b]
        assert bool((got[b, c:] == 0).all())
        # every tile of a short run, some 24 tokens of a longer one
        tokens = list(range(c)) if c <= 40 else sorted({0, c - 1, *rng.choice(c, 22, replace=False).tolist()})
        seen = visible(tokens, lens[b], window, sinks, None if parents is None else parents[b])
        used = seen.any(0)
        at = used.nonzero().flatten().cuda()
        pick = lambda x: x[b][tokens][:, heads].double()   # noqa: E731
        y, x = exact(cache[b][at].double(), pick(q), w_uv[heads].double(),
                     None if gate is None else pick(gate.view(B, T, H, D_V)), seen[:, used].cuda(), scale)
        tile = (torch.tensor(tokens)[:, None] * H + torch.tensor(heads)) // TILE
        share = share_of_allowed(pick(got), y, x, tile.cuda())
        assert share <= 1, f"sequence {b}: {share:.2f} of what a tile's error may be"
