"""GPU tests of mla_latent_attend_paged where its calls end with two kernels (parts joined, then W_UV and the gate), that is
with more than 2 CTAs of (head, 32 tokens) per SM; each test sees to it that its calls are such.  Inputs, reference and bound
are those of tests/test_paged_attend.py."""
import pytest

from tests.test_paged_attend import BOUNDS, D_V, R, attend, check, env, problem  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture
def three(env):  # noqa: F811
    """Counts the kernels of a call: the pair kernel, the join, the product."""
    torch, lca = env

    def call(d, **more):
        B, T, H = d["q_abs"].shape[:3]
        assert -(-B * T // 32) * H > 2 * torch.cuda.get_device_properties(0).multi_processor_count
        before = lca.mla_kernel_launches()
        out = attend(env, d, **more)
        assert lca.mla_kernel_launches() - before == 3
        return out

    return call


def sevens(env, d):  # noqa: F811
    B, T, H = d["q_abs"].shape[:3]
    return env[0].full((B, T, H * D_V), 7.0, dtype=env[0].bfloat16, device="cuda")


@pytest.mark.parametrize("T,H,lens,kw", [
    (130, 64, [200, 31, 1000], dict(counts=[130, 0, 7])),
    (130, 64, [200, 31, 1000], dict(counts=[0, 130, 129], window=50, sinks=4, bs=128)),
    (64, 96, [300, 0, 77, 1000], dict(counts=[64, 13, 0, 40], tree="mixed")),
    (64, 96, [300, 0], dict(tree="star", window=100, sinks=3, gate=False)),
    (64, 70, [500, 2, 65], dict(tree="mixed", window=7, sinks=300, counts=[1, 64, 63])),
    (40, 128, [127, 64, 0], dict(ld=520, scale=-0.1)),
    (90, 101, [3, 700], dict(bs=192, scale=0.0)),
    (350, 33, [65], dict(scale=3.0)),
    # rows that see nothing of a part: windows that end inside a tile's units
    (1100, 9, [0, 130], dict(window=1)),
    (1100, 9, [60, 5], dict(window=5, sinks=1, counts=[1100, 1003])),
    (1100, 9, [500, 1], dict(window=64, sinks=130, gate=False))])
def test_shapes(env, three, T, H, lens, kw):  # noqa: F811
    d = problem(env, T, H, lens, **kw)
    check(env, d, three(d, out=sevens(env, d)))


def test_no_tokens(env, three):  # noqa: F811
    d = problem(env, 200, 80, [10, 20, 30], counts=[0, 0, 0])
    assert bool((three(d, out=sevens(env, d)) == 7.0).all())
    assert bool((three(d) == 0).all())
    assert env[1].mla_get_device_error() == 0


def test_hidden_rows_have_no_effect(env, three):  # noqa: F811
    torch, _ = env
    for bad in (float("nan"), float("inf"), -float("inf")):
        d = problem(env, 64, 96, [200, 90], tree="star", seed=9, gate=False)
        clean = three(d)
        d["pool"][int(d["block_table"][0, 203 // 64]), 203 % 64, 17] = bad
        got = three(d)
        rest = [t for t in range(64) if t != 3]
        assert bool(got[0, 3].isnan().all())
        assert torch.equal(got[0, rest], clean[0, rest]) and torch.equal(got[1], clean[1])
        d = problem(env, 200, 60, [200], window=30, sinks=3, seed=10)
        clean = three(d)
        for row in (1, 171 + 40, 398):     # a sink, one that tokens 11 .. 40 see, one that 198 and 199 see
            c = d["pool"][int(d["block_table"][0, row // 64]), row % 64]
            kept = c.clone()
            c[400] = bad
            got = three(d)
            hit = [t for t in range(200) if row < 3 or row <= 200 + t < row + 30]
            rest = [t for t in range(200) if t not in hit]
            assert bool(got[0, hit].isnan().all()) and torch.equal(got[0, rest], clean[0, rest])
            c.copy_(kept)
    assert env[1].mla_get_device_error() == 0


def test_queries_that_are_no_tokens(env, three):  # noqa: F811
    torch, _ = env
    d = problem(env, 60, 90, [300, 70, 10], counts=[4, 60, 0], window=90, sinks=2)
    want = three(d)
    for bad in (float("nan"), float("inf"), 3e38):
        for b, c in enumerate((4, 60, 0)):
            d["q_abs"][b, c:] = bad
            d["gate"][b, c:] = bad
        assert torch.equal(three(d), want)
    assert env[1].mla_get_device_error() == 0


@pytest.mark.parametrize("byte", [0, 255, 0x7F, 0xC3])
def test_whatever_the_workspace_holds(env, three, byte):  # noqa: F811
    torch, lca = env
    d = problem(env, 130, 64, [900, 31, 1000], counts=[130, 0, 7], window=500, sinks=4)
    want = check(env, d)
    B, T, H = d["q_abs"].shape[:3]
    ws = torch.full((lca.mla_latent_attend_paged_workspace_size(B, T, H, R),), byte, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        assert torch.equal(three(d, workspace=ws, out=sevens(env, d)), want)
    assert lca.mla_get_device_error() == 0


def test_streams_and_graphs_that_share_a_workspace(env, three):  # noqa: F811
    """A large call and a short one: on another stream, and as two graphs replayed in turn, with lengths that change."""
    torch, lca = env
    one = problem(env, 60, 96, [3000, 100, 900], tree="mixed", seed=1)
    two = problem(env, 1, 40, [9000, 20], window=2000, sinks=5, seed=2)
    need = max(lca.mla_latent_attend_paged_workspace_size(*d["q_abs"].shape) for d in (one, two))
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    want = [check(env, d) for d in (one, two)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert torch.equal(three(one, workspace=ws), want[0])
    side.synchronize()
    got = three(one, stream=side)
    side.synchronize()
    assert torch.equal(got, want[0])
    outs, graphs = [torch.zeros_like(w) for w in want], []
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
    one["lens"].copy_(torch.tensor([2900, 90, 800], dtype=torch.int32, device="cuda"))
    outs[0].fill_(7.0)
    graphs[0].replay()
    check(env, one, outs[0])
    assert lca.mla_get_device_error() == 0


def test_least_alignment(env, three):  # noqa: F811
    torch, lca = env

    def moved(t, by):
        flat = torch.empty(t.numel() + 64, dtype=t.dtype, device="cuda")
        at = next(i for i in range(64) if (flat.data_ptr() + i * t.element_size()) % 64 == by)
        return flat[at:at + t.numel()].view(t.shape).copy_(t)

    d = problem(env, 40, 128, [100, 300, 7], counts=[40, 39, 2], tree="mixed", window=50, sinks=3)
    want = check(env, d)
    for key in d:
        if isinstance(d[key], torch.Tensor):
            d[key] = moved(d[key], 16 if d[key].dtype == torch.bfloat16 else 4)
    ws = torch.empty(lca.mla_latent_attend_paged_workspace_size(3, 40, 128, R) + 64, dtype=torch.uint8, device="cuda")
    ws = ws[next(i for i in range(64) if (ws.data_ptr() + i) % 64 == 16):]
    got = three(d, out=moved(sevens(env, d), 16), workspace=ws[:lca.mla_latent_attend_paged_workspace_size(3, 40, 128, R)])
    assert got.data_ptr() % 32 == 16 and torch.equal(got, want)


def test_reports(env, three):  # noqa: F811
    torch, lca = env
    for key, value in (("lens", -1), ("lens", 2**31 - 1), ("counts", -1), ("counts", 61)):
        d = problem(env, 60, 96, [100, 130, 150], counts=[60, 2, 3])
        # as without the sequence: what it takes of the axis decides where the others' tiles are cut
        want = check(env, dict(d, counts=torch.tensor([60, 0, 3], dtype=torch.int32, device="cuda")))
        d[key][1] = value
        got = three(d, out=sevens(env, d))
        assert lca.mla_get_device_error() == BOUNDS and torch.equal(got, want)
    d = problem(env, 60, 96, [100, 200])
    d["block_table"][0, 1] = 10**6
    got = three(d)
    assert lca.mla_get_device_error() == BOUNDS
    spare = problem(env, 60, 96, [100, 200])
    spare["pool"][int(spare["block_table"][0, 1])] = 0
    assert torch.equal(got, three(spare))
