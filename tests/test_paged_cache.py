"""GPU tests of the paged latent cache's bookkeeping and writes: block tables, slot maps and the free stack against a
one-by-one restatement on the host, rows against the slots they go to (all exact)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

BOUNDS = -9


@pytest.fixture(scope="module")
def env():
    import torch

    import latent_compressed_attention_gb300 as lca
    lca.build()
    lca.mla_get_device_error()
    return torch, lca


def one_by_one(lens, counts, T, table, held, free, left, bs):
    """What mla_reserve_latent_blocks does, a block at a time; the state is changed in place, slots are returned."""
    need = [-(-(n + c) // bs) for n, c in zip(lens, counts)]
    stack = list(free[:left])
    given = [table[b][j] for b in range(len(lens)) for j in range(need[b], held[b])]
    stack += reversed(given)
    for b in range(len(lens)):
        for j in range(held[b], need[b]):
            table[b][j] = stack.pop()
    held[:] = need
    free[:len(stack)] = stack
    slots = np.full((len(lens), T), -1)
    for b, (n, c) in enumerate(zip(lens, counts)):
        for t in range(c):
            slots[b, t] = table[b][(n + t) // bs] * bs + (n + t) % bs
    return slots, len(stack)


class Cache:
    """The state on the GPU and its copy on the host."""

    def __init__(self, env, B, wide, blocks, capacity, bs, seed, ld=None):
        self.torch, self.lca, self.bs, self.B = *env, bs, B
        self.rng = np.random.default_rng(seed)
        self.table, self.held = np.full((B, wide), -3), np.zeros(B, int)
        self.free, self.left = np.full(capacity, -5), blocks
        self.free[:blocks] = self.rng.permutation(blocks)
        i32 = dict(dtype=self.torch.int32, device="cuda")
        self.g_table = self.torch.tensor(np.full((B, ld or wide), -3), **i32)[:, :wide]
        self.g_held, self.g_free = self.torch.tensor(self.held, **i32), self.torch.tensor(self.free, **i32)
        self.g_left = self.torch.tensor([blocks], **i32)

    def call(self, lens, counts, T):
        i32 = dict(dtype=self.torch.int32, device="cuda")
        return self.lca.mla_reserve_latent_blocks(self.torch.tensor(lens, **i32), self.torch.tensor(counts, **i32), T,
                                                  self.g_table, self.g_held, self.g_free, self.g_left, self.bs)

    def state(self):
        return [x.cpu().numpy() for x in (self.g_table, self.g_held, self.g_free, self.g_left)]

    def step(self, lens, counts, T):
        got = self.call(lens, counts, T)
        slots, self.left = one_by_one(list(lens), list(counts), T, self.table, self.held, self.free, self.left, self.bs)
        if T:
            np.testing.assert_array_equal(got.cpu().numpy(), slots)
        else:
            assert got is None
        table, held, free, left = self.state()
        np.testing.assert_array_equal(held, self.held)
        np.testing.assert_array_equal(table, self.table)
        np.testing.assert_array_equal(free, self.free)
        assert left[0] == self.left


@pytest.mark.parametrize("B,T,bs,longest,ld", [
    (1, 1, 64, 200, None), (3, 5, 64, 300, 17), (64, 8, 128, 2000, None), (7, 2000, 1, 50, 2100), (1000, 9, 16, 64, None),
    (1025, 3, 64, 500, None), (5, 4097, 64, 100, None), (513, 64, 192, 700, 30), (33, 250, 7, 90, None)])
def test_reserve_steps(env, B, T, bs, longest, ld):
    """Sequences grow, shrink, end and start again, several ways in one call; counts of zero and of T among them."""
    wide = -(-(longest + T) // bs)
    cache = Cache(env, B, wide, B * wide, B * wide + 3, bs, seed=B, ld=ld)
    rng = cache.rng
    for i in range(5):
        lens = rng.integers(0, longest + 1, B)
        counts = rng.integers(0, T + 1, B)
        lens[rng.random(B) < 0.2] = 0
        counts[rng.random(B) < 0.3] = 0
        counts[rng.integers(B)] = T
        cache.step(lens, counts, T)
    cache.step(np.zeros(B, int), np.zeros(B, int), 0)
    assert cache.left == B * wide
    assert env[1].mla_get_device_error() == 0


def test_growth_and_shrinking_restore_the_stack(env):
    cache = Cache(env, 40, 20, 500, 500, 64, seed=1)
    lens = cache.rng.integers(0, 600, 40)
    cache.step(lens, np.zeros(40, int), 0)
    free, left = cache.free[:cache.left].copy(), cache.left
    cache.step(lens, np.full(40, 300), 300)
    cache.step(lens, np.zeros(40, int), 4)
    assert cache.left == left and np.array_equal(cache.free[:left], free)


def test_most_sequences(env):
    """The largest number of sequences, and one more."""
    torch, lca = env
    B = 16384
    cache = Cache(env, B, 2, 2 * B, 2 * B, 64, seed=2)
    cache.step(cache.rng.integers(0, 100, B), np.ones(B, int), 1)
    one = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    with pytest.raises(lca.MLAError, match="not supported"):
        lca.mla_reserve_latent_blocks(one, one, 1, one[:, None].repeat(1, 2), one, one, one[:1], 64)


@pytest.mark.parametrize("T", [4, 4000])
@pytest.mark.parametrize("what", ["blocks", "wide", "count", "negative len", "negative count", "held", "left", "overflow"])
def test_what_does_not_fit_changes_nothing(env, what, T):
    cache = Cache(env, 5, 70, 90, 400, 64, seed=3)
    cache.step(np.array([100, 0, 64, 65, 1]), np.array([4, 4, 4, 4, 4]), T)
    lens, counts = np.array([100, 0, 64, 65, 1]), np.full(5, 4)
    if what == "blocks":
        lens[:] = 2000
    elif what == "wide":
        lens[2] = 70 * 64 - 3
    elif what == "count":
        counts[3] = T + 1
    elif what == "negative len":
        lens[4] = -1
    elif what == "negative count":
        counts[0] = -2
    elif what == "overflow":
        lens[1] = 2**31 - 1
    elif what == "held":
        cache.g_held[1] = 71
    else:
        cache.g_left[0] = 401
    before = cache.state()
    slots = cache.call(lens, counts, T)
    assert bool((slots == -1).all())
    for a, b in zip(before, cache.state()):
        np.testing.assert_array_equal(a, b)
    assert env[1].mla_get_device_error() == BOUNDS


def test_blocks_past_the_last_row_number(env):
    torch, lca = env
    i32 = dict(dtype=torch.int32, device="cuda")
    slots = lca.mla_reserve_latent_blocks(torch.tensor([0], **i32), torch.tensor([2], **i32), 2, torch.zeros(1, 1, **i32),
                                          torch.zeros(1, **i32), torch.tensor([2**30], **i32), torch.ones(1, **i32), 64)
    assert slots.tolist() == [[-1, -1]] and lca.mla_get_device_error() == BOUNDS


def test_reserve_in_a_graph(env):
    """A captured call, replayed, goes on from the state that it finds."""
    torch, lca = env
    cache = Cache(env, 6, 30, 180, 180, 64, seed=4)
    i32 = dict(dtype=torch.int32, device="cuda")
    lens, counts, slots = torch.zeros(6, **i32), torch.full((6,), 3, **i32), torch.zeros(6, 3, **i32)
    args = (lens, counts, 3, cache.g_table, cache.g_held, cache.g_free, cache.g_left, 64)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lca.mla_reserve_latent_blocks(*args, slots=slots)
    for i in range(4):
        now = cache.rng.integers(0, 1000, 6)
        lens.copy_(torch.tensor(now, **i32))
        graph.replay()
        want, cache.left = one_by_one(list(now), [3] * 6, 3, cache.table, cache.held, cache.free, cache.left, 64)
        np.testing.assert_array_equal(slots.cpu().numpy(), want)
        np.testing.assert_array_equal(cache.state()[2], cache.free)
    assert lca.mla_get_device_error() == 0


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("shape,bs,r,ld", [
    ((1, 1), 64, 512, 512), ((3, 5), 64, 512, 576), ((64, 9), 128, 512, 512), ((700,), 16, 40, 48), ((5, 1000), 1, 8, 8),
    ((2, 3, 7), 192, 1000, 1000), ((9, 1001), 64, 512, 520), ((1, 40001), 64, 64, 64)])
def test_append(env, shape, bs, r, ld, dtype):
    torch, lca = env
    gen = torch.Generator(device="cuda").manual_seed(5)
    n = int(np.prod(shape))
    blocks = -(-n // bs) + 2
    records = torch.randn((blocks, bs, ld), generator=gen, device="cuda").to(torch.bfloat16)
    slots = torch.randperm(blocks * bs, generator=gen, device="cuda")[:n].int()
    slots[torch.rand(n, generator=gen, device="cuda") < 0.1] = -1
    c = torch.randn((*shape, r), generator=gen, device="cuda").to(getattr(torch, dtype))
    want = records.clone()
    there = slots >= 0
    at = slots[there].long()
    want[at // bs, at % bs, :r] = c.reshape(n, r)[there].to(torch.bfloat16)
    pool = records[:, :, :r]
    assert lca.mla_append_latent_paged(c, pool, slots.view(shape)) is pool
    assert torch.equal(records.view(torch.int16), want.view(torch.int16))
    assert lca.mla_get_device_error() == 0


def test_append_values_as_they_are(env):
    """NaN, infinities, zeros of either sign and values next to a rounding border of an fp32 row."""
    torch, lca = env
    x = torch.tensor([float("nan"), float("inf"), -float("inf"), 0.0, -0.0, 1 + 2**-8, 1 + 2**-8 + 2**-20, 1 + 3 * 2**-8,
                      3.4e38, 1e-40, -1e-45, 65504.0, 1.0, -1.0, 2.0**-126, 2.0**-133], device="cuda")
    pool = torch.zeros(1, 64, 16, dtype=torch.bfloat16, device="cuda")
    lca.mla_append_latent_paged(x[None], pool, torch.tensor([7], dtype=torch.int32, device="cuda"))
    want = x.to(torch.bfloat16)
    assert torch.equal(pool[0, 7].isnan(), want.isnan())
    assert torch.equal(pool[0, 7, 1:].view(torch.int16), want[1:].view(torch.int16))


@pytest.mark.parametrize("bad", [-2, 128, 2**31 - 1, -2**31])
def test_append_outside_the_pool(env, bad):
    torch, lca = env
    pool = torch.zeros(3, 64, 512, dtype=torch.bfloat16, device="cuda")
    lca.mla_append_latent_paged(torch.ones(2, 512, dtype=torch.bfloat16, device="cuda"), pool[:2],
                                torch.tensor([bad, 127], dtype=torch.int32, device="cuda"))
    assert lca.mla_get_device_error() == BOUNDS
    assert float(pool.float().sum()) == 512 and float(pool[1, 63].float().sum()) == 512


def test_append_far_rows(env):
    """Element offsets past 2^32 (the last rows of a 9 GB pool)."""
    torch, lca = env
    pool = torch.empty(137000, 64, 512, dtype=torch.bfloat16, device="cuda")
    last = 137000 * 64 - 1
    assert last * 512 > 2**32
    c = torch.randn(2, 512, device="cuda")
    pool[-2:].zero_()
    lca.mla_append_latent_paged(c, pool, torch.tensor([last, last - 64], dtype=torch.int32, device="cuda"))
    assert torch.equal(pool[-1, -1], c[0].to(torch.bfloat16)) and torch.equal(pool[-2, -1], c[1].to(torch.bfloat16))
    assert int((pool[-2:] != 0).sum()) == int((c.to(torch.bfloat16) != 0).sum())


def test_refusals(env):
    torch, lca = env
    pool = torch.zeros(2, 64, 512, dtype=torch.bfloat16, device="cuda")
    c = torch.zeros(2, 512, dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(2, dtype=torch.int32, device="cuda")
    for bad in (dict(c=c.half()), dict(c=c.cpu()), dict(c=c[:, ::2]), dict(pool=pool.float()), dict(pool=pool[:, :32]),
                dict(pool=pool[0]), dict(pool=pool[:, :, :256]), dict(slots=slots.long()), dict(slots=slots[:1])):
        with pytest.raises((TypeError, ValueError)):
            lca.mla_append_latent_paged(**(dict(c=c, pool=pool, slots=slots) | bad))
    good = dict(lens=slots, counts=slots, T=1, block_table=slots[:, None].clone(), held=slots.clone(),
                free_blocks=slots.clone(), free_count=slots[:1].clone(), block_size=64)
    lca.mla_reserve_latent_blocks(**good)
    for bad in (dict(counts=slots[:1]), dict(counts=slots.long()), dict(block_table=slots), dict(held=slots.cpu()),
                dict(block_table=torch.zeros(2, 4, dtype=torch.int32, device="cuda")[:, ::2]),
                dict(block_table=slots[:1, None].expand(2, 3)), dict(free_count=slots), dict(T=-1), dict(T=2**31),
                dict(free_blocks=slots[:, None]), dict(slots=slots)):
        with pytest.raises((TypeError, ValueError)):
            lca.mla_reserve_latent_blocks(**(good | bad))
    with pytest.raises(lca.MLAError):
        lca.mla_reserve_latent_blocks(**(good | dict(block_size=0)))
