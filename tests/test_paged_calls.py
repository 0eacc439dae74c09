"""GPU tests of calls of the paged latent cache as programs make them: from several threads at once, with states at the
edge of their ranges or outside them, step after step."""
import threading

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


def test_reserve_from_two_threads(env):
    """Calls whose numbers of sequences ask for different amounts of shared memory, at the same time."""
    torch, lca = env
    lib, status, state, go = lca.library(), {}, {}, threading.Event()

    def calls(B, n):
        i32 = dict(dtype=torch.int32, device="cuda")
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            lens, table, free = torch.full((B,), 70, **i32), torch.zeros(B, 2, **i32), torch.randperm(2 * B, device="cuda").int()
            held, left, counts = torch.zeros(B, **i32), torch.tensor([2 * B], **i32), torch.zeros(B, **i32)
        stream.synchronize()
        args = (lens.data_ptr(), counts.data_ptr(), table.data_ptr(), 2, held.data_ptr(), free.data_ptr(), left.data_ptr(), None,
                B, 0, 2, 2 * B, 64, stream.cuda_stream)
        go.wait()
        status[B] = [lib.mla_reserve_latent_blocks(*args) for _ in range(n)]
        stream.synchronize()
        state[B] = left, held

    threads = [threading.Thread(target=calls, args=(B, 3000)) for B in (16384, 3400, 9000)]
    for t in threads:
        t.start()
    go.set()
    for t in threads:
        t.join()
    assert {B: sum(rc != 0 for rc in rcs) for B, rcs in status.items()} == {16384: 0, 3400: 0, 9000: 0}
    for left, held in state.values():
        assert int(left) == 0 and bool((held == 2).all())
    assert len(state) == 3
    assert lca.mla_get_device_error() == 0


def test_more_blocks_than_an_int_counts(env):
    """Half of the sequences give up all their blocks and the others take as many, 2^31."""
    torch, lca = env
    B, wide, i32 = 16384, 2**18, dict(dtype=torch.int32, device="cuda")
    table = torch.empty((B, wide), **i32)
    table[:, :2] = 5
    held = torch.full((B,), wide, **i32)
    held[1::2] = 0
    lens = wide - held
    free, left, none = torch.full((4,), -5, **i32), torch.zeros(1, **i32), torch.zeros(B, **i32)
    before = [x.clone() for x in (held, free, left, table[:, :2])]
    lca.mla_reserve_latent_blocks(lens, none, 0, table, held, free, left, 1)
    assert lca.mla_get_device_error() == BOUNDS
    assert all(torch.equal(a, b) for a, b in zip(before, (held, free, left, table[:, :2])))


@pytest.mark.parametrize("T", [4, 4000])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("where", ["given up, to the stack", "given up, taken", "stack"])
def test_what_is_no_block_is_not_moved(env, where, many, T):
    """A number below 0 among those given up or taken refuses the call; where it stays it does not count."""
    torch, lca = env
    i32 = dict(dtype=torch.int32, device="cuda")
    wide, bs = (6000, 1) if many else (6, 64)   # up to 12000 blocks moved, more than one each thread's turn, or 12
    gen = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randperm(4 * wide, generator=gen, device="cuda").int()
    table = torch.full((5, wide), -3, **i32)
    table[:3] = ids[:3 * wide].view(3, wide)
    held, left = torch.tensor([wide, wide, wide, 0, 0], **i32), torch.tensor([wide], **i32)
    free = torch.cat([ids[3 * wide:], torch.full((3 * wide,), -5, **i32)])
    lens, counts = torch.tensor([wide * bs, 0, 0, 0, 0], **i32), torch.zeros(5, **i32)
    if where != "given up, to the stack":   # those that two give up go to the others, or some of the stack too
        lens[3] = lens[4] = wide * bs
    if where == "stack":
        lens[2] = wide * bs
        free[wide // 2] = -1
    else:
        table[2 if many else 1, wide // 3] = -1
    table[0, 1] = -2   # of a sequence that keeps its blocks
    before = [x.clone() for x in (table[:3], held, free[:wide], left)]
    slots = lca.mla_reserve_latent_blocks(lens, counts, T, table, held, free, left, bs)
    assert lca.mla_get_device_error() == BOUNDS and bool((slots == -1).all())
    assert all(torch.equal(a, b) for a, b in zip(before, (table[:3], held, free[:wide], left)))
    if where == "stack":
        free[wide // 2] = 4 * wide
    else:
        table[2 if many else 1, wide // 3] = 4 * wide
    lca.mla_reserve_latent_blocks(lens, counts, T, table, held, free, left, bs)
    assert lca.mla_get_device_error() == 0
    assert held.tolist() == [-(-n // bs) for n in lens.tolist()]
    now = torch.cat([table[b, :n] for b, n in enumerate(held.tolist())] + [free[:int(left)]])
    then = torch.cat([before[0].flatten(), before[2]])
    for n in (-1, -2):   # a block each, in one place
        then, now = then[then != n], now[now != n]
    assert sorted(now.tolist()) == sorted(then.tolist() + [4 * wide])


def test_kept_paths_of_drafted_trees(env):
    """Rounds of drafting as the header tells them: of each sequence's tree a path is kept, and all paths' latents are
    appended again in one call.  Every sequence's rows are its kept tokens, and the attention's outputs those over the same
    rows in blocks of their own, bit by bit."""
    torch, lca = env
    i32, bf16 = dict(dtype=torch.int32, device="cuda"), torch.bfloat16
    gen = torch.Generator(device="cuda").manual_seed(3)
    rng = np.random.default_rng(3)
    B, T, H, bs, wide, r = 5, 9, 16, 64, 4, 512
    pool = torch.full((B * wide, bs, r), float("nan"), dtype=bf16, device="cuda")
    table, held = torch.full((B, wide), -1, **i32), torch.zeros(B, **i32)
    free, left = torch.randperm(B * wide, generator=gen, device="cuda").int(), torch.tensor([B * wide], **i32)
    w_uv = (torch.randn((H, 128, r), generator=gen, device="cuda") * 0.05).to(bf16)
    lens, past = torch.tensor([0, 61, 5, 63, 120], **i32), []
    c = torch.randn((B, 120, r), generator=gen, device="cuda").to(bf16)   # prompts
    slots = lca.mla_reserve_latent_blocks(torch.zeros_like(lens), lens, 120, table, held, free, left, bs)
    lca.mla_append_latent_paged(c, pool, slots)
    past = [c[b, :n] for b, n in enumerate(lens.tolist())]

    def rows(b, n):
        u = torch.arange(n, device="cuda")
        return pool[table[b].long()[u // bs], u % bs]

    moved = 0
    for _ in range(8):
        counts = torch.full((B,), T, **i32)
        parents = np.array([[rng.integers(-1, t) if t else -1 for t in range(T)] for _ in range(B)])
        c = torch.randn((B, T, r), generator=gen, device="cuda")   # fp32, as a norm leaves them
        slots = lca.mla_reserve_latent_blocks(lens, counts, T, table, held, free, left, bs)
        lca.mla_append_latent_paged(c, pool, slots)
        q = torch.randn((B, T, H, r), generator=gen, device="cuda").to(bf16)
        out = lca.mla_latent_attend_paged(q, pool, table, lens, w_uv, parents=torch.tensor(parents, **i32), scale=0.05)
        alone = torch.zeros((B, wide * bs, r), dtype=bf16, device="cuda")
        for b in range(B):
            alone[b, :len(past[b]) + T] = torch.cat([past[b], c[b].to(bf16)])
        own = torch.arange(B * wide, **i32).view(B, wide)
        want = lca.mla_latent_attend_paged(q, alone.view(B * wide, bs, r), own, lens, w_uv,
                                           parents=torch.tensor(parents, **i32), scale=0.05)
        assert bool(out.isfinite().all()) and torch.equal(out, want)
        path = np.full((B, T), -1)
        for b in range(B):
            line, a = [], rng.integers(-1, T)   # -1: none is kept
            while a >= 0:
                line.insert(0, a)
                a = parents[b, a]
            path[b, :len(line)] = line
            moved += line != list(range(len(line)))
        path = torch.tensor(path, device="cuda")
        kept = (path >= 0).sum(1).int()
        lca.mla_append_latent_paged(c.gather(1, path.clamp(min=0)[:, :, None].expand(B, T, r)), pool,
                                    torch.where(path >= 0, slots, -1))
        lens = lens + kept
        for b in range(B):
            past[b] = torch.cat([past[b], c[b, path[b, :int(kept[b])]].to(bf16)])
            assert torch.equal(rows(b, int(lens[b])), past[b])
    assert moved > B and lca.mla_get_device_error() == 0


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("more", [-1, 0, 1])
def test_append_at_a_wave_of_threads(env, more, dtype):
    """Just fewer and just more rows than a thread each of the GPU has a piece of 8 elements for."""
    torch, lca = env
    rows = torch.cuda.get_device_properties(0).multi_processor_count * 2048 // 64 + more
    gen = torch.Generator(device="cuda").manual_seed(rows)
    c = torch.randn((rows, 512), generator=gen, device="cuda").to(getattr(torch, dtype))
    pool = torch.zeros((-(-rows // 64) + 1, 64, 512), dtype=torch.bfloat16, device="cuda")
    slots = torch.randperm(len(pool) * 64, generator=gen, device="cuda")[:rows].int()
    want = pool.view(-1, 512).clone()
    want[slots.long()] = c.to(torch.bfloat16)
    lca.mla_append_latent_paged(c, pool, slots)
    assert torch.equal(pool.view(-1, 512), want) and lca.mla_get_device_error() == 0


def test_attention_calls_at_once(env):
    """Calls of all three endings on four streams at the same time, and a captured one without a workspace of its own between
    eager calls: each gives the bits that it gives alone."""
    torch, lca = env
    from tests.test_paged_attend import attend, problem
    calls = [problem(env, 1, 8, [300, 1], window=100, sinks=2, seed=1), problem(env, 64, 96, [900, 20], tree="mixed", seed=2),
             problem(env, 16, 96, [5000, 70, 2000], tree="chain", seed=3), problem(env, 300, 30, [2000], seed=4)]
    want = [attend(env, d) for d in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[] for _ in calls]
    for _ in range(12):
        for d, s, g in zip(calls, streams, got):
            with torch.cuda.stream(s):
                g.append(attend(env, d))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w, x) for x in g)
    outs, graphs = [torch.zeros_like(w) for w in want], []
    for d, o in zip(calls, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            attend(env, d, out=o)
            attend(env, d, out=o)
    for _ in range(3):
        for graph, d, o, w in zip(graphs, calls[1:] + calls[:1], outs, want):
            junk = torch.full((2**22,), float("nan"), device="cuda")
            graph.replay()
            other = attend(env, d)
            del junk
            assert torch.equal(o, w) and bool(other.isfinite().all())
            o.zero_()
    assert lca.mla_get_device_error() == 0
