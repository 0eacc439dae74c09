"""GPU tests of the fp4 latent cache at its edges, with the helpers and the elementwise bounds of test_parity_fp4.py:
heads whose running maxima move together, weights and groups far below the largest, the sizes and arguments that the
other file leaves out."""
import numpy as np
import pytest

from latent_compressed_attention_gb300 import workloads as W
from tests.test_parity_fp4 import R, check, decode, decode_case, env, latent  # noqa: F401 (env: the fixture)

pytestmark = pytest.mark.gpu


def counted_rows(u, seed):
    """Latent rows that hold a number each, u = sum of 7^k digit_k < 6 * 7^4, its digits in columns 32 (k + 1) as values
    that e2m1 has: digit - 3, the last one less 1; columns 32 .. 191 are zero otherwise."""
    c, u = latent(np.random.default_rng(seed), (len(u), R)), np.asarray(u)
    c[:, 32:192] = 0.0
    for k in range(5):
        c[:, 32 * (k + 1)] = u // 7**k % 7 - 3.0 if k < 4 else u // 7**4 - 1.0
    return c


def query_of_numbers(H, step):
    """q_abs [1, H, r] whose scores are step[h] times the rows' numbers (and a constant)."""
    q = np.zeros((1, H, R))
    for k in range(5):
        q[0, :, 32 * (k + 1)] = W.round_bf16(step * 7.0**k)
    return q


@pytest.mark.parametrize("H", [16, 31, 48, 49, 64, 96])
def test_heads_whose_maxima_move_together(env, H):  # noqa: F811
    """Scores rise from row to row, in neighbouring heads by different steps: the running maxima of heads that share
    columns of the accumulator move in the same unit, each by an amount of its own."""
    n = 2050
    d = decode_case(H, [n], n, seed=51)
    d["rows"][0] = W.encode_fp4(counted_rows(np.arange(n), 52))
    d["q_abs"] = query_of_numbers(H, 0.01 * (1 + np.arange(H) % 5))
    got = decode(env, d)
    check(env, d, got)
    for _ in range(5):
        assert np.array_equal(decode(env, d), got)


def many_light_rows(torch, lca, H, light, heavy_at, n, seed):
    """len(heavy_at) sequences of n rows: n - 1 equal light ones and the heavy one at heavy_at[b].  The heavy row lies in
    the lower half of the latent and the light ones in the upper; a head's light rows weigh about light[b, h] of its
    heavy one, and the first half of each head's outputs comes from the upper half alone.  Returns the call's arguments
    and per (b, h, v): the exact output, the sum of the rows' shares without regard to their signs, that sum over single
    latent values (A of test_parity_fp4.py), and the share of one light row as heavy as the heavy one."""
    rng = np.random.default_rng([seed, H])
    B = len(heavy_at)
    heavy, dim = np.zeros(R), np.zeros(R)
    heavy[:256], dim[256:] = 1.0, np.where(np.arange(256) % 2 == 0, 1.0, -1.0)
    cache = torch.tensor(W.encode_fp4(dim[None]), device="cuda").repeat(B, n, 1)
    cache[torch.arange(B), torch.tensor(heavy_at)] = torch.tensor(W.encode_fp4(heavy[None]), device="cuda")
    q = np.zeros((B, H, R))
    rest = -np.log(light) / 4   # by which the heavy row's score is higher: in three bf16 parts, on four columns each
    for k in range(3):
        q[:, :, 4 * k : 4 * k + 4] = W.round_bf16(rest)[..., None]
        rest = rest - q[:, :, 4 * k]
    w_uv = W.round_bf16(rng.standard_normal((H, 128, R)) * 0.02)
    w_uv[:, :64, :256] = 0.0
    w = np.exp(-(q @ heavy))[..., None]
    total = 1.0 + (n - 1) * w
    y = (w_uv @ heavy + (n - 1) * w * (w_uv @ dim)) / total
    rows = (np.abs(w_uv @ heavy) + (n - 1) * w * np.abs(w_uv @ dim)) / total
    A = (np.abs(w_uv) @ heavy + (n - 1) * w * (np.abs(w_uv) @ np.abs(dim))) / total
    args = [torch.tensor(x, dtype=torch.bfloat16, device="cuda") for x in (q, w_uv)]
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    return (args[0], cache, lens, args[1]), y, rows, A, np.abs(w_uv @ dim) / total


@pytest.mark.parametrize("H", [16, 48, 64, 96])
def test_light_rows_far_below_a_heavy_one(env, H):  # noqa: F811
    """32767 equal rows at 2^-8 .. 2^-21 of a heavy one, 2^-16 * 1.125 and both sides of 2^-21 among them: together they
    count for their weight wherever the heavy row lies.  A row's weight is held within 2^-8 of itself up to 48 heads, 2^-7
    above, and, of the heavy one, 2^-21 in its window of 4096 rows, 2^-24 in the next and so on: 4096 * 2^-21 * 8/7
    of it in all.  The error of a weight is a factor of its whole row, so it counts by |c . W_UV|.  q_abs's smaller parts lie below 2^-9 of its largest
    (3.7 at most) and are off by at most 2^-17 of it on four columns each: 2^-12 of a weight; 2^-10 covers that and the
    exponential.  Sums in fp32 and the merge's o_lat (2^-17) are within 2^-15 of A."""
    torch, lca, _ = env
    n, B = 32768, 64
    rng = np.random.default_rng(H)
    light = np.exp2(-rng.uniform(8, 21, (B, H)))
    light[:, 0], light[:, 1], light[:, 2] = 1.125 * 2.0**-16, 2.0**-20.99, 2.0**-21.01
    light[:, 3:6] = 2.0**-17 * np.array([1.125, 1.375, 1.875])
    heavy_at = rng.integers(0, n, B)
    heavy_at[:4] = 0, n - 1, 4095, 127
    args, y, rows, A, one = many_light_rows(torch, lca, H, light, heavy_at, n, 53)
    got = lca.mla_latent_decode_fp4(*args).double().cpu().numpy().reshape(y.shape)
    assert lca.mla_get_device_error() == 0
    weights = 2.0**-8 if H <= 48 else 2.0**-7
    bound = 2.0**-8 * np.abs(y) + (weights + 2.0**-10) * rows + 4096 * 2.0**-21 * 8 / 7 * one + 2.0**-15 * A
    worst = np.unravel_index(np.argmax(np.abs(got - y) / bound), y.shape)
    assert np.all(np.abs(got - y) <= bound), (worst, light[worst[:2]], got[worst], y[worst], bound[worst])


@pytest.mark.parametrize("H", [16, 48, 49, 96])
def test_maxima_that_fall_and_rise_in_long_runs(env, H):  # noqa: F811
    """Scores that fall (in other heads rise) over thousands of rows and turn: the maxima are set lower and higher again
    by anything from a fraction of a binade to far more than the accumulators could follow."""
    torch, lca, _ = env
    n, B = 14000, 140
    u = np.abs(np.arange(n) - 9000) + 100
    rows = W.encode_fp4(counted_rows(u, 54))
    q = query_of_numbers(H, 0.02 * (-1.0) ** np.arange(H) * 2.0 ** (-(np.arange(H) // 2 % 6)))
    w_uv = W.round_bf16(np.random.default_rng(55).standard_normal((H, 128, R)) * 0.02)
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    got = lca.mla_latent_decode_fp4(torch.tensor(q, **bf16).repeat(B, 1, 1), torch.tensor(rows, device="cuda").repeat(B, 1, 1),
                                    torch.full((B,), n, dtype=torch.int32, device="cuda"), torch.tensor(w_uv, **bf16))
    assert lca.mla_get_device_error() == 0
    one = dict(q_abs=q, w_uv=w_uv, gate=None, lens=np.array([n], np.int32), rows=rows[None])
    for b in (0, 61, B - 1):
        check(env, one, got[b : b + 1].double().cpu().numpy())


def apart(rng, n, least, most):
    """Latent rows whose sixteen groups lie 2^least to 2^most below the row's largest, the even ones (group 0 holds the
    largest) by half of that at most."""
    far = np.where(np.arange(R // 32) % 2 == 0, rng.integers(0, least // 2 + 1, (n, R // 32)),
                   rng.integers(least, most + 1, (n, R // 32)))
    far[:, 0] = 0
    return latent(rng, (n, R)) * np.exp2(-far.astype(np.float64)).repeat(32, -1)


@pytest.mark.parametrize("H,lens,max_len", [(8, [300, 129, 1], 300), (48, [1000], 1024), (60, [257, 0, 640], 640),
                                            (96, [200] * 5, 256), (96, [40, 300] + [90] * 38, 300), (3, [40000], 40000)])
def test_groups_far_below_their_row_s_largest(env, H, lens, max_len):  # noqa: F811
    """Groups 2^15 to 2^70 below their row's largest: scores and half of the outputs that come from such groups alone."""
    d = decode_case(H, lens, max_len, seed=61)
    rng = np.random.default_rng(62)
    odd = (np.arange(R) // 32 % 2 == 1)
    rows = d["rows"].reshape(-1, d["rows"].shape[-1])
    for b, (least, most) in zip(range(len(lens)), [(15, 19), (19, 22), (25, 35), (15, 70)] * len(lens)):
        c = apart(rng, max_len, least, most)
        if b % 2 == 1:   # only some of the rows, in the middle
            c[: max_len // 3], c[max_len // 2 :] = latent(rng, (max_len // 3, R)), latent(rng, (max_len - max_len // 2, R))
        c *= 2.0 ** (least // 2)   # all within the scale bytes' range
        rows[b * max_len : (b + 1) * max_len] = W.encode_fp4(c)
        scale = np.abs(c[: max(lens[b], 1), odd]).max()
        d["q_abs"][b][:, ~odd] = 0.0
        d["q_abs"][b] = W.round_bf16(d["q_abs"][b] * np.exp2(-np.round(np.log2(scale))))
    d["w_uv"][:, :64, ~odd] = 0.0
    check(env, d, decode(env, d))


@pytest.mark.parametrize("H", [20, 96])
def test_scale_bytes_of_groups_of_zeros(env, H):  # noqa: F811
    """Groups of zeros under any scale byte, the largest and NaN's among them, beside ordinary ones."""
    d = decode_case(H, [700, 300], 700, seed=63)
    rng = np.random.default_rng(64)
    rows = d["rows"]
    zero = rng.random((2, 700, R // 32)) < 0.3
    zero[:, :, 0] = False
    codes = rows[..., : R // 2].reshape(2, 700, R // 32, 16)
    codes[zero] = rng.choice(np.array([0x00, 0x80, 0x08, 0x88], np.uint8), (zero.sum(), 16))
    rows[..., R // 2 : 272][zero] = rng.choice([0, 87, 90, 120, 140, 150, 167, 200], zero.sum())
    got = decode(env, d)
    check(env, d, got)
    rows[1, 299, R // 2 + 7], rows[1, 299, R // 2 + 8] = 255, 167
    again = decode(env, d)
    assert np.array_equal(again[0], got[0]) and np.all(np.isnan(again[1]))


def test_more_sequences_than_a_grid_has_rows(env):  # noqa: F811
    """32 * 65535 sequences and one more: each of one row (or none), whose output is its values times W_UV."""
    torch, lca, _ = env
    B = 32 * 65535 + 1
    gen = torch.Generator(device="cuda").manual_seed(71)
    cache = lca.mla_quantize_latent_fp4(torch.randn((B, R), generator=gen, device="cuda", dtype=torch.bfloat16))
    q = torch.zeros((B, 1, R), dtype=torch.bfloat16, device="cuda")
    w_uv = (torch.randn((1, 128, R), generator=gen, device="cuda") * 0.02).bfloat16()
    lens = torch.ones(B, dtype=torch.int32, device="cuda")
    lens[5] = lens[B - 2] = 0
    got = lca.mla_latent_decode_fp4(q, cache.view(B, 1, -1), lens, w_uv)
    assert lca.mla_get_device_error() == 0
    for at in (0, 1 << 20, B - 64):
        c = W.decode_fp4(cache[at : at + 64].cpu().numpy(), R) * lens[at : at + 64].double().cpu().numpy()[:, None]
        w = w_uv[0].double().cpu().numpy()
        err, A = np.abs(got[at : at + 64].double().cpu().numpy() - c @ w.T), np.abs(c) @ np.abs(w).T
        assert np.all(err <= 2.0**-8 * np.abs(c @ w.T) + (2.0**-8 + 2.0**-10) * A)


@pytest.mark.parametrize("gate", [False, True])
def test_empty_caches_and_batches(env, gate):  # noqa: F811
    """Caches without rows give zeros, batches without sequences nothing: as the writers and the reader take them."""
    torch, lca, _ = env
    for B in (3, 0):
        empty = torch.empty((B, 0, 272), dtype=torch.uint8, device="cuda")
        q = torch.ones((B, 20, R), dtype=torch.bfloat16, device="cuda")
        w_uv = torch.ones((20, 128, R), dtype=torch.bfloat16, device="cuda")
        g = torch.ones((B, 20 * 128), dtype=torch.bfloat16, device="cuda") if gate else None
        lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        out = torch.full((B, 20 * 128), 7.0, dtype=torch.bfloat16, device="cuda")
        assert lca.mla_latent_decode_fp4(q, empty, lens, w_uv, g, out=out) is out and not bool(out.any())
        assert lca.mla_latent_decode_fp4(q, empty, lens, w_uv, g).shape == (B, 20 * 128)
        assert lca.mla_dequantize_latent_fp4(empty, R).shape == (B, 0, R)
    assert lca.mla_append_latent_fp4(torch.empty((0, 1, R), device="cuda"), empty, lens) is empty
    assert lca.mla_get_device_error() == 0


@pytest.mark.parametrize("view", ["middle", "unsqueezed"])
def test_one_row_caches_at_any_stride(env, view):  # noqa: F811
    """A cache of one row per sequence that lies in a larger one: appended to, read back and attended to in place."""
    torch, lca, _ = env
    d = decode_case(9, [1, 1, 0, 1], 1, seed=81, gate=True)
    c = latent(np.random.default_rng(82), (4, 1, R))
    d["rows"][..., :272] = W.encode_fp4(c)
    base = torch.full((4, 9, 320), 7, dtype=torch.uint8, device="cuda")
    cache = base[:, 5:6, :272] if view == "middle" else base[:, 5, :272].unsqueeze(1)
    bf16 = lambda x: torch.tensor(x, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    assert lca.mla_append_latent_fp4(bf16(c), cache, torch.zeros(4, dtype=torch.int32, device="cuda")) is cache
    want = np.full((4, 9, 320), 7, np.uint8)
    want[:, 5, :272] = d["rows"][:, 0, :272]
    assert np.array_equal(base.cpu().numpy(), want)
    back = lca.mla_dequantize_latent_fp4(cache, R)
    assert np.array_equal(back.double().cpu().numpy(), W.decode_fp4(want[:, 5:6, :272], R))
    lens = torch.tensor(d["lens"], device="cuda")
    got = lca.mla_latent_decode_fp4(bf16(d["q_abs"]), cache, lens, bf16(d["w_uv"]), bf16(d["gate"]))
    check(env, d, got.double().cpu().numpy())
    assert lca.mla_get_device_error() == 0


def test_workspaces_that_are_none(env):  # noqa: F811
    """Tensors that do not stand for as much memory of the device as they have elements are refused on the host."""
    torch, lca, _ = env
    d = decode_case(8, [30, 5], 30, seed=91)
    n = lca.mla_latent_decode_fp4_workspace_size(2, 8, R, 30)
    for workspace in (torch.empty(n, dtype=torch.uint8), torch.empty(1, dtype=torch.uint8, device="cuda").expand(n),
                      torch.empty((n, 2), dtype=torch.uint8, device="cuda")[:, 0]):
        with pytest.raises(ValueError, match="workspace"):
            decode(env, d, workspace=workspace)
    with pytest.raises(lca.MLAError):
        decode(env, d, workspace=torch.empty(n - 1, dtype=torch.uint8, device="cuda"))
    check(env, d, decode(env, d, workspace=torch.empty(n, dtype=torch.uint8, device="cuda")))


def test_calls_on_a_given_stream(env):  # noqa: F811
    """The stream argument of every call: the same results as on the current stream, in order on that one."""
    torch, lca, _ = env
    d = decode_case(40, [0, 300], 400, seed=92)
    c = latent(np.random.default_rng(93), (2, 1, R))
    bf16 = lambda x: torch.tensor(x, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    q, w_uv, new = bf16(d["q_abs"]), bf16(d["w_uv"]), bf16(c)
    cache, lens = torch.tensor(d["rows"], device="cuda"), torch.tensor(d["lens"], device="cuda")
    after, side = lens + 1, torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    lca.mla_append_latent_fp4(new, cache, lens, stream=side)
    got = lca.mla_latent_decode_fp4(q, cache, after, w_uv, stream=side)
    back = lca.mla_dequantize_latent_fp4(cache, R, stream=side)
    rows = lca.mla_quantize_latent_fp4(new, stream=side)
    side.synchronize()
    for b, n in enumerate((0, 300)):
        d["rows"][b, n] = W.encode_fp4(c[b, 0])
    d["lens"] = d["lens"] + 1
    check(env, d, got.double().cpu().numpy())
    assert np.array_equal(back.double().cpu().numpy(), W.decode_fp4(d["rows"], R))
    assert np.array_equal(rows.cpu().numpy(), W.encode_fp4(c)) and lca.mla_get_device_error() == 0


@pytest.mark.parametrize("gone", ["_cuda_getCurrentRawStream", "_cuda_cudaCachingAllocator_raw_alloc",
                                  "_cuda_cudaCachingAllocator_raw_delete"])
def test_without_torch_s_inner_names(env, gone, monkeypatch):  # noqa: F811
    """The names inside torch that save host time may go: the calls then take torch's public ones."""
    torch, lca, _ = env
    d = decode_case(8, [30, 5], 30, seed=94)
    want = decode(env, d)
    monkeypatch.delattr(torch._C, gone)
    with torch.cuda.stream(torch.cuda.Stream()):
        got = decode(env, d)
    assert np.array_equal(got, want)


@pytest.mark.parametrize("B,T,max_len,r,ld", [(1, 1, 1, 512, 272), (5, 1, 300, 512, 320), (3, 700, 900, 512, 272),
                                              (4, 3, 9, 96, 64), (2, 5000, 5003, 32, 32)])
@pytest.mark.parametrize("with_counts", [False, True])
def test_append_of_fp32_rows(env, B, T, max_len, r, ld, with_counts):  # noqa: F811
    """fp32 rows with more bits than bf16 has: the bytes of the rows from lens[b] on, and no other byte of the cache."""
    torch, lca, _ = env
    rng = np.random.default_rng(B * T + r)
    row, used = W.fp4_row_bytes(r), r // 2 + r // 32
    c = (latent(rng, (B, T, r), spread=5) * (1 + 2.0**-12 * rng.integers(-8, 9, (B, T, r)))).astype(np.float32)
    c[0, 0, 3] = np.nan
    lens = rng.integers(0, max_len - T + 1, B).astype(np.int32)
    counts = rng.integers(0, T + 1, B).astype(np.int32) if with_counts else np.full(B, T, np.int32)
    counts[0] = T
    want = rng.integers(0, 256, (B, max_len, ld)).astype(np.uint8)
    cache = torch.tensor(want, device="cuda")
    lca.mla_append_latent_fp4(torch.tensor(c, device="cuda"), cache[:, :, :row], torch.tensor(lens, device="cuda"),
                              torch.tensor(counts, device="cuda") if with_counts else None)
    for b in range(B):
        want[b, lens[b] : lens[b] + counts[b], :used] = W.encode_fp4(c[b, : counts[b]])[:, :used]
    assert np.array_equal(cache.cpu().numpy(), want) and lca.mla_get_device_error() == 0


@pytest.mark.parametrize("H", [16, 48, 64, 96])
def test_query_elements_far_below_the_largest(env, H):  # noqa: F811
    """Queries whose larger elements lie on a group of small values and the smaller ones, 2^10 to 2^13 below, on the rest:
    a smaller element is off by at most 2^-21 of its head's largest (2^-17 above 48 heads), so a score by at most that
    times the sum of the row's other values, and the weights by twice its exponential's change."""
    d = decode_case(H, [900, 40], 900, seed=95)
    rng = np.random.default_rng(96)
    c = latent(rng, (2, 900, R))
    c[..., :32] *= 2.0**-9
    d["rows"][..., :272] = W.encode_fp4(c)
    q = rng.standard_normal((2, H, R)) * np.exp2(-rng.integers(10, 14, (2, H, R)).astype(float)) * 64
    q[..., :32] = rng.standard_normal((2, H, 32)) * 64
    d["q_abs"] = W.round_bf16(q)
    got = decode(env, d)
    part = 2.0**-21 if H <= 48 else 2.0**-17
    for b, n in enumerate(d["lens"]):
        c = W.decode_fp4(d["rows"][b, :n, :272], R)
        s = d["q_abs"][b] @ c.T
        p = np.exp(s - s.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        y = np.einsum("hr,hvr->hv", p @ c, d["w_uv"]).reshape(-1)
        A = np.einsum("hr,hvr->hv", p @ np.abs(c), np.abs(d["w_uv"]))
        off = 2 * np.expm1(part * np.abs(d["q_abs"][b]).max(-1) * np.abs(c[:, 32:]).sum(-1).max())
        weights = 2.0**-8 if H <= 48 else 2.0**-7
        bound = 2.0**-8 * np.abs(y) + ((weights + 2.0**-9 + 2.0**-10 + off[:, None]) * A).reshape(-1)
        assert np.all(np.abs(got[b] - y) <= bound)
