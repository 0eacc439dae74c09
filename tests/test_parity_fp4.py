"""GPU tests of the fp4 latent cache: the writers (mla_quantize_latent_fp4, mla_append_latent_fp4), the reader
(mla_dequantize_latent_fp4) and the decode over it (mla_latent_decode_fp4), through the C ABI.

Writers and reader are integer-valued work: bit-exact against the host codec (workloads.encode_fp4 / decode_fp4, pinned
in test_fp4_codec.py).  The decode is compared with the fp64 oracle on the values that the cache holds.  Its error has
two parts, each an elementwise bound, with A = sum_u p_u |c_u| |W_UV| sigma:
  the output's rounding to bf16                                   2^-8 |y|
  the softmax weights, held as e4m3 hi + lo.  hi is off by at most 2^-4 of the weight.
    up to 48 heads: lo = e4m3(16 rest), 2^-4 of the rest, and never less than half its step, 2^-9 / 16 / 2 = 2^-14, where
    a running maximum is set so that the largest weight is 2^7 or more    (2^-8 + n 2^-21) A
    above:          lo = e5m2(rest), 2^-3 of the rest, half a step is 2^-17, the largest weight 2^5 or more
                                                                          (2^-7 + n 2^-22) A
q_abs is held as e4m3 hi + lo too: the 8 bits of a bf16 value are the 4 of hi and the 4 of the rest, so both together are
exact but for elements below 2^-9 of the head's largest; sums are fp32; 2^-10 A covers both at |score| <= 100.  The
rounding errors are independent, so over a whole output they are far smaller than the sum of bounds: the 2-norm is held
to 2^-8 |y| for the rounding and as much again for everything else.
"""
import numpy as np
import pytest

from latent_compressed_attention_gb300 import workloads as W
from tests.conftest import gpu_available

pytestmark = pytest.mark.gpu
R, ROW = 512, 272


@pytest.fixture(scope="module")
def env():
    if not gpu_available():
        pytest.skip("no CUDA device")
    import torch

    import latent_compressed_attention_gb300 as lca
    import oracle
    from latent_compressed_attention_gb300 import _build
    _build.build()
    oracle.build()
    return torch, lca, oracle


def dev(torch, a, dtype=None):
    return torch.tensor(np.asarray(a), dtype=dtype, device="cuda")


def bf(torch, a):
    return dev(torch, np.asarray(a, np.float32)).to(torch.bfloat16)


def latent(rng, shape, spread=0):
    c = rng.standard_normal(shape)
    c /= np.sqrt(np.mean(c * c, -1, keepdims=True))
    return W.round_bf16(c * np.exp2(rng.integers(-spread, spread + 1, (*shape[:-1], 1))))


def special(c):
    """Groups of a [n >= 8, r >= 32] array with ties, saturation, zeros, subnormals, infinities and NaN."""
    c = c.copy()
    c[0, :16] = 2.0**-3 * np.array([7, -7, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -5, -0.25, 6, 4, 0, -0.0, 0.5])
    c[0, 16:32] = 0
    c[1, :32] = 0
    c[2, :32] = 2.0**-130
    c[3, :32] *= 2.0**60
    c[4, 3], c[5, 31], c[6, 0] = np.nan, np.inf, -np.inf
    c[7, :32] *= 2.0**-44
    return W.round_bf16(c)


# ------------------------------------------------------------------------------------------------ writers and reader
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("rows,r", [(8, 32), (9, 96), (300, 512), (17, 2080)])
def test_write_and_read_back_exact(env, dtype, rows, r):
    torch, lca, _ = env
    rng = np.random.default_rng(rows)
    c = special(latent(rng, (rows, r), spread=6))
    if dtype == "float32":   # bits that bf16 does not have
        c = np.where(np.isfinite(c), (c * (1 + 2.0**-12 * rng.integers(-8, 9, c.shape))).astype(np.float32), c)
    t = dev(torch, c.astype(np.float32)).to(getattr(torch, dtype))
    rows4 = lca.mla_quantize_latent_fp4(t)
    want = W.encode_fp4(c)
    used = r // 2 + r // 32
    assert rows4.shape == want.shape
    assert np.array_equal(rows4.cpu().numpy()[:, :used], want[:, :used])
    back = lca.mla_dequantize_latent_fp4(rows4, r, dtype=t.dtype)
    assert back.dtype == t.dtype
    assert np.array_equal(back.double().cpu().numpy(), W.decode_fp4(want, r), equal_nan=True)


def test_strided_rows_at_the_c_abi(env):
    """Row strides wider than the rows on both sides; nothing between the rows is touched."""
    torch, lca, _ = env
    rng = np.random.default_rng(1)
    c = latent(rng, (37, 96))
    wide = torch.full((37, 104), 9.0, dtype=torch.bfloat16, device="cuda")
    wide[:, :96] = bf(torch, c)
    c4 = torch.full((37, 80), 0xAB, dtype=torch.uint8, device="cuda")
    lib = lca.library()
    s = torch.cuda.current_stream().cuda_stream
    assert lib.mla_quantize_latent_fp4(wide.data_ptr(), 104, c4.data_ptr(), 80, 37, 96, 0, s) == 0
    want = W.encode_fp4(c)
    assert np.array_equal(c4.cpu().numpy()[:, :51], want[:, :51]) and bool((c4[:, 51:] == 0xAB).all())
    back = torch.full((37, 104), 9.0, dtype=torch.bfloat16, device="cuda")
    assert lib.mla_dequantize_latent_fp4(c4.data_ptr(), 80, 0, None, back.data_ptr(), 104, 1, 37, 96, 0, s) == 0
    assert np.array_equal(back[:, :96].double().cpu().numpy(), W.decode_fp4(want, 96)) and bool((back[:, 96:] == 9).all())


@pytest.mark.parametrize("B,T,max_len,r,ld", [(1, 1, 1, 512, 272), (5, 1, 300, 512, 320), (3, 70, 200, 512, 272),
                                              (4, 3, 9, 96, 64)])
@pytest.mark.parametrize("with_counts", [False, True])
def test_append(env, B, T, max_len, r, ld, with_counts):
    """Rows lens[b] .. of each sequence, and no other byte of the cache; rows past its end and bad counts are reported."""
    torch, lca, _ = env
    rng = np.random.default_rng(B * T)
    row, used = W.fp4_row_bytes(r), r // 2 + r // 32
    c = latent(rng, (B, T, r))
    lens = rng.integers(0, max_len - T + 1, B)
    counts = rng.integers(0, T + 1, B) if with_counts else np.full(B, T)
    counts[0] = T
    buf = rng.integers(0, 256, (B, max_len, ld)).astype(np.uint8)
    cache = dev(torch, buf)
    got = lca.mla_append_latent_fp4(bf(torch, c), cache[:, :, :row], dev(torch, lens, torch.int32),
                                    dev(torch, counts, torch.int32) if with_counts else None)
    assert got.data_ptr() == cache.data_ptr() and lca.mla_get_device_error() == 0
    want = buf.copy()
    for b in range(B):
        want[b, lens[b] : lens[b] + counts[b], :used] = W.encode_fp4(c[b, : counts[b]])[:, :used]
    assert np.array_equal(cache.cpu().numpy(), want)


def test_long_runs(env):
    """Runs long enough for several pieces per thread: written, appended with counts, read back with lengths."""
    torch, lca, _ = env
    rng = np.random.default_rng(41)
    B, T, max_len = 3, 8003, 8100
    c = latent(rng, (B, T, R))
    want = W.encode_fp4(c)
    assert np.array_equal(lca.mla_quantize_latent_fp4(bf(torch, c)).cpu().numpy(), want)
    f32 = dev(torch, c.astype(np.float32))
    assert np.array_equal(lca.mla_quantize_latent_fp4(f32.view(B * T, R)).cpu().numpy(), want.reshape(B * T, ROW))
    lens, counts = [97, 0, 5], [8003, 1, 4111]
    cache = torch.full((B, max_len, ROW), 3, dtype=torch.uint8, device="cuda")
    lca.mla_append_latent_fp4(bf(torch, c), cache, dev(torch, lens, torch.int32), dev(torch, counts, torch.int32))
    full = np.full((B, max_len, ROW), 3, np.uint8)
    for b in range(B):
        full[b, lens[b] : lens[b] + counts[b]] = want[b, : counts[b]]
    assert np.array_equal(cache.cpu().numpy(), full)
    values = W.decode_fp4(full, R)
    for dtype in (torch.bfloat16, torch.float32):
        out = torch.full((B, max_len, R), 5.0, dtype=dtype, device="cuda")
        upto = [8100, 0, 6001]
        lca.mla_dequantize_latent_fp4(cache, R, lens=dev(torch, upto, torch.int32), out=out)
        expect = np.full((B, max_len, R), 5.0)
        for b in range(B):
            expect[b, : upto[b]] = values[b, : upto[b]]
        assert np.array_equal(out.double().cpu().numpy(), expect)
    assert lca.mla_get_device_error() == 0


def test_append_out_of_range_is_reported_and_not_written(env):
    torch, lca, _ = env
    rng = np.random.default_rng(2)
    c = latent(rng, (4, 3, 512))
    for lens, counts in (([2, 4, 5, 2**31 - 1], None), ([-1, -3, 0, -(2**31)], None), ([0, 1, 2, 2], [3, 4, -1, 0])):
        cache = torch.full((4, 5, ROW), 7, dtype=torch.uint8, device="cuda")
        lca.mla_append_latent_fp4(bf(torch, c), cache, dev(torch, lens, torch.int32),
                                  None if counts is None else dev(torch, counts, torch.int32))
        assert lca.mla_get_device_error() == -9
        want = np.full((4, 5, ROW), 7, np.uint8)
        for b in range(4):
            for t in range(3 if counts is None else min(max(counts[b], 0), 3)):
                if 0 <= lens[b] + t < 5:
                    want[b, lens[b] + t] = W.encode_fp4(c[b, t])
        assert np.array_equal(cache.cpu().numpy(), want)


def test_read_back_lengths_views_and_scale_bytes(env):
    torch, lca, _ = env
    rng = np.random.default_rng(4)
    rows = rng.integers(0, 256, (4, 50, 288)).astype(np.uint8)   # every code, every scale byte
    cache = dev(torch, rows)[:, :, :ROW]
    want = W.decode_fp4(rows[..., :ROW], 512)
    for dtype in (torch.bfloat16, torch.float32):
        got = lca.mla_dequantize_latent_fp4(cache, 512, dtype=dtype)
        assert np.array_equal(got.double().cpu().numpy(), want, equal_nan=True)
    part = lca.mla_dequantize_latent_fp4(cache[:, 7:20], 512)
    assert np.array_equal(part.double().cpu().numpy(), want[:, 7:20], equal_nan=True)
    one = lca.mla_dequantize_latent_fp4(cache[2, 3:9], 512)
    assert np.array_equal(one.double().cpu().numpy(), want[2, 3:9], equal_nan=True)
    out = torch.full((4, 50, 512), 5.0, dtype=torch.bfloat16, device="cuda")
    lens = [0, 50, 70, 13]
    assert lca.mla_dequantize_latent_fp4(cache, 512, lens=dev(torch, lens, torch.int32), out=out) is out
    expect = np.full((4, 50, 512), 5.0)
    for b, n in enumerate(lens):
        expect[b, :n] = want[b, :n]
    assert np.array_equal(out.double().cpu().numpy(), expect, equal_nan=True) and lca.mla_get_device_error() == 0
    lca.mla_dequantize_latent_fp4(cache, 512, lens=dev(torch, [-1, 1, 1, 1], torch.int32))
    assert lca.mla_get_device_error() == -9
    assert lca.mla_dequantize_latent_fp4(cache[:, :0], 512).shape == (4, 0, 512)
    assert lca.mla_quantize_latent_fp4(torch.zeros((0, 512), device="cuda")).shape == (0, ROW)


# ------------------------------------------------------------------------------------------------ decode
def decode_case(H, lens, max_len, seed=0, gate=False, q_mul=1.0, spread=0, ld=ROW):
    rng = np.random.default_rng([seed, H, len(lens)])
    B = len(lens)
    d = W.draw_decode(W.K3_DECODE_BF16, seed=seed, B=B, lens=np.clip(lens, 0, max_len), gate=gate, H=H)
    d["q_abs"] = W.round_bf16(d["q_abs"] * q_mul)
    d["lens"] = np.asarray(lens, np.int32)
    d["rows"] = np.zeros((B, max_len, ld), np.uint8)
    d["rows"][..., :ROW] = W.encode_fp4(latent(rng, (B, max_len, R), spread))
    return d


def decode(env, d, scale=1.0, **kw):
    torch, lca, _ = env
    out = lca.mla_latent_decode_fp4(bf(torch, d["q_abs"]), dev(torch, d["rows"])[..., :ROW], dev(torch, d["lens"]),
                                    bf(torch, d["w_uv"]), None if d["gate"] is None else bf(torch, d["gate"]), scale, **kw)
    torch.cuda.synchronize()
    assert lca.mla_get_device_error() == 0
    return out.double().cpu().numpy()


def check(env, d, got, scale=1.0):
    oracle = env[2]
    B, H = d["q_abs"].shape[:2]
    c = W.decode_fp4(d["rows"][..., :ROW], R)
    for b in range(B):
        c[b, d["lens"][b]:] = 0.0
    ref = oracle.decode(d["q_abs"], c, d["lens"], d["w_uv"], d["gate"], scale)
    assert np.all(np.isfinite(got))
    for b in range(B):
        n = int(d["lens"][b])
        if n == 0:
            assert np.all(got[b] == 0.0)
            continue
        s = scale * d["q_abs"][b] @ c[b, :n].T
        p = np.exp(s - s.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        A = np.einsum("hr,hvr->hv", p @ np.abs(c[b, :n]), np.abs(d["w_uv"])).reshape(-1)
        if d["gate"] is not None:
            A = A / (1 + np.exp(-d["gate"][b]))
        err = np.abs(got[b] - ref[b])
        weights = 2.0**-8 + n * 2.0**-21 if H <= 48 else 2.0**-7 + n * 2.0**-22
        assert np.all(err <= 2.0**-8 * np.abs(ref[b]) + (weights + 2.0**-10) * A)
        assert np.linalg.norm(err) <= 2.0**-7 * np.linalg.norm(ref[b])


@pytest.mark.parametrize("H,lens,max_len", [
    (1, [1], 1),
    (8, [1, 130, 300], 300),
    (96, [1, 2, 127, 128, 129, 255, 256, 257], 300),
    (96, [0, 700, 0, 1500], 1600),
    (16, [513, 1000, 64, 1999, 5], 2048),
    (37, [300, 280, 1], 300),
    (48, [640, 17], 640),
    (49, [333, 0, 128], 400),
    (64, [1000], 1000),
    (17, [3] * 40, 3),
    (65, [900, 1, 0, 257], 900),
    (80, [40] * 33 + [0, 500], 500),
    (3, [0] * 31 + [200, 0, 5, 0, 129], 256),
    (2, [0, 0], 7),
])
@pytest.mark.parametrize("gate", [False, True])
def test_decode_shapes(env, H, lens, max_len, gate):
    d = decode_case(H, lens, max_len, seed=len(lens) + H, gate=gate)
    check(env, d, decode(env, d))


def test_decode_poisoned_tail_row_stride_and_workspace(env):
    """Rows at or past lens[b], the bytes between rows and the workspace hold NaN patterns: none reaches the result."""
    torch, lca, _ = env
    d = decode_case(96, [5, 200, 129, 1], 256, seed=3, ld=320)
    for b, n in enumerate(d["lens"]):
        d["rows"][b, n:] = 255
    d["rows"][..., ROW:] = 255
    need = lca.mla_latent_decode_fp4_workspace_size(4, 96, 512, 256)
    ws = torch.full((need // 4 + 4,), float("nan"), dtype=torch.float32, device="cuda").view(torch.uint8)
    check(env, d, decode(env, d, workspace=ws))


@pytest.mark.parametrize("q_mul,scale", [(4.0, 1.0), (1.0, 0.5), (20.0, 0.25), (0.0, 1.0), (1.0, -1.0)])
def test_decode_score_spreads(env, q_mul, scale):
    d = decode_case(32, [600, 50, 3000], 3000, seed=5, q_mul=q_mul)
    check(env, d, decode(env, d, scale), scale)


@pytest.mark.parametrize("H,lens,max_len", [(5, [32768, 32769, 70001], 70001), (70, [33000, 3, 65536], 65536)])
def test_decode_past_a_chunk(env, H, lens, max_len):
    """Sequences whose rows are split into chunks with maxima of their own, in the middle of shares and at their ends."""
    d = decode_case(H, lens, max_len, seed=21)
    check(env, d, decode(env, d))


@pytest.mark.parametrize("H", [24, 80])
def test_decode_rows_of_other_magnitudes(env, H):
    """Rows and groups far apart in magnitude: row scales 2^-12 .. 2^12 in one sequence, a sequence of rows near 2^-30
    with one zero row, and groups of one row 2^10 apart."""
    d = decode_case(H, [400, 300, 260], 400, seed=6, spread=12, q_mul=2.0**-12)
    rng = np.random.default_rng(8)
    small = latent(rng, (300, R)) * 2.0**-30
    small[7] = 0.0
    d["rows"][1, :300, :ROW] = W.encode_fp4(small)
    mixed = latent(rng, (260, R)) * np.exp2(rng.integers(-5, 6, (260, R // 32))).repeat(32, -1)
    d["rows"][2, :260, :ROW] = W.encode_fp4(mixed)
    check(env, d, decode(env, d))


@pytest.mark.parametrize("H", [16, 64, 96])
def test_decode_one_heavy_row_among_many_light_ones(env, H):
    """One row takes about half of the weight and thousands of equal light rows share the rest: the light rows, 2^-14 of
    the heavy one each, count in full."""
    n = 16384
    d = decode_case(H, [n], n, seed=7)
    row = np.ones(R)
    light = np.where(np.arange(R) % 2 == 0, 1.0, -1.0)
    rows = np.tile(light, (n, 1))
    rows[5] = row
    d["rows"][0, :, :ROW] = W.encode_fp4(rows)
    d["q_abs"][:] = 0.0
    d["q_abs"][0, :, :8] = W.round_bf16(np.where(np.arange(8) % 2 == 0, 0.0, np.log(n) / 8))[None]   # heavy - light = ln n
    check(env, d, decode(env, d))


@pytest.mark.parametrize("H", [40, 96])
def test_decode_maxima_that_keep_rising(env, H):
    """Every row's score above the one before, by little and by much: each unit moves the running maxima of all heads."""
    for step in (0.02, 0.5):
        n = 700
        d = decode_case(H, [n], n, seed=22)
        c = latent(np.random.default_rng(23), (n, R))
        c[:, 32:64] = 0.0
        c[:, 32] = np.arange(n) % 7 - 3.0       # integers that e2m1 holds, the score's small part
        c[:, 64:96] = (np.arange(n) // 7 % 7 - 3.0)[:, None] * (np.arange(32) == 0)
        c[:, 96:128] = (np.arange(n) // 49 % 7 - 3.0)[:, None] * (np.arange(32) == 0)
        c[:, 128:160] = (np.arange(n) // 343 - 1.0)[:, None] * (np.arange(32) == 0)
        d["rows"][0, :, :ROW] = W.encode_fp4(c)
        d["q_abs"][:] = 0.0
        for k, at in enumerate((32, 64, 96, 128)):
            d["q_abs"][0, :, at] = W.round_bf16(np.array(step * 7.0**k))
        check(env, d, decode(env, d))


@pytest.mark.parametrize("H", [40, 96])
def test_decode_nan_row_stays_in_its_sequence(env, H):
    torch, lca, _ = env
    d = decode_case(H, [300, 300, 300], 300, seed=9)
    clean = decode(env, d)
    d["rows"][1, 222, 256 + 3] = 255
    got = decode(env, d)
    assert np.all(np.isnan(got[1])) and np.array_equal(got[[0, 2]], clean[[0, 2]])


def test_decode_full_workload_sampled(env):
    """The K3 decode workload (B = 64, lengths U[1024, 32768], H = 96) over an fp4 cache written on the device."""
    torch, lca, _ = env
    w = W.K3_DECODE_BF16
    d = W.draw_decode(w, seed=0)
    cache = torch.zeros((w.B, w.max_len, ROW), dtype=torch.uint8, device="cuda")
    for b in range(w.B):
        gen = torch.Generator(device="cuda").manual_seed(b)
        c = torch.randn((1, int(d["lens"][b]), R), generator=gen, device="cuda")
        lca.mla_append_latent_fp4(c, cache[b : b + 1], torch.zeros(1, dtype=torch.int32, device="cuda"))
    out = lca.mla_latent_decode_fp4(bf(torch, d["q_abs"]), cache, dev(torch, d["lens"]), bf(torch, d["w_uv"]))
    torch.cuda.synchronize()
    assert lca.mla_get_device_error() == 0
    got = out.double().cpu().numpy()
    for b in sorted({int(np.argmax(d["lens"])), int(np.argmin(d["lens"])), 17}):
        one = {k: d[k][b : b + 1] for k in ("q_abs", "lens")}
        check(env, dict(one, w_uv=d["w_uv"], gate=None, rows=cache[b : b + 1].cpu().numpy()), got[b : b + 1])


def test_prompt_steps_and_read_back_together(env):
    """As a server uses them: prompts written, three decode steps that append and attend, the context read back."""
    torch, lca, _ = env
    rng = np.random.default_rng(11)
    B, H, max_len, P = 3, 20, 160, [100, 0, 127]
    c = latent(rng, (B, max_len, R))
    cache = torch.zeros((B, max_len, ROW), dtype=torch.uint8, device="cuda")
    lens = dev(torch, P, torch.int32)
    lca.mla_append_latent_fp4(bf(torch, c[:, :130]), cache, torch.zeros_like(lens), counts=lens)
    for step in range(3):
        new = np.stack([c[b, P[b] + step] for b in range(B)])[:, None]
        lca.mla_append_latent_fp4(bf(torch, new), cache, lens)
        lens += 1
        d = decode_case(H, [p + step + 1 for p in P], max_len, seed=step, gate=True)
        d["rows"][..., :ROW] = W.encode_fp4(c)
        got = lca.mla_latent_decode_fp4(bf(torch, d["q_abs"]), cache, lens, bf(torch, d["w_uv"]), bf(torch, d["gate"]))
        check(env, d, got.double().cpu().numpy())
    back = lca.mla_dequantize_latent_fp4(cache, R, lens=lens)
    for b in range(B):
        n = P[b] + 3
        assert np.array_equal(back[b, :n].double().cpu().numpy(), W.decode_fp4(W.encode_fp4(c[b, :n]), R))
        assert not bool(back[b, n:].any())
    assert lca.mla_get_device_error() == 0


def test_captured_step_on_a_side_stream(env):
    """Append and decode captured into a graph on a stream of their own, replayed with other inputs."""
    torch, lca, _ = env
    d = [decode_case(50, [130, 77], 256, seed=s) for s in (1, 2)]
    rng = np.random.default_rng(12)
    new = [latent(rng, (2, 1, R)) for _ in d]
    q, cache, w_uv = bf(torch, d[0]["q_abs"]), dev(torch, d[0]["rows"]), bf(torch, d[0]["w_uv"])
    tok, lens = bf(torch, new[0]), dev(torch, [130, 77], torch.int32)
    ws = torch.empty(lca.mla_latent_decode_fp4_workspace_size(2, 50, R, 256), dtype=torch.uint8, device="cuda")
    out, after = torch.empty((2, 50 * 128), dtype=torch.bfloat16, device="cuda"), lens + 1

    def step():
        lca.mla_append_latent_fp4(tok, cache, lens)
        lca.mla_latent_decode_fp4(q, cache, after, w_uv, out=out, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            step()
    for k in (1, 0):
        q.copy_(bf(torch, d[k]["q_abs"]))
        cache.copy_(dev(torch, d[k]["rows"]))
        tok.copy_(bf(torch, new[k]))
        w_uv.copy_(bf(torch, d[k]["w_uv"]))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        one = dict(d[k], lens=np.array([131, 78], np.int32), rows=d[k]["rows"].copy())
        for b, n in enumerate((130, 77)):
            one["rows"][b, n, :ROW] = W.encode_fp4(new[k][b, 0])
        check(env, one, out.double().cpu().numpy())
    assert lca.mla_get_device_error() == 0


def test_two_graphs_one_workspace_and_two_streams(env):
    """Two captured decodes that share a workspace, replayed in turn; two decodes at once on streams and workspaces of
    their own: the same bits as one after the other."""
    torch, lca, _ = env
    cases = [decode_case(20, [900, 130], 1000, seed=31), decode_case(70, [400, 0, 777], 800, seed=32)]
    want = [decode(env, d) for d in cases]
    args = [(bf(torch, d["q_abs"]), dev(torch, d["rows"]), dev(torch, d["lens"]), bf(torch, d["w_uv"])) for d in cases]
    need = [lca.mla_latent_decode_fp4_workspace_size(*d["q_abs"].shape, d["rows"].shape[1]) for d in cases]
    outs = [torch.empty(w.shape, dtype=torch.bfloat16, device="cuda") for w in want]
    shared = torch.empty(max(need), dtype=torch.uint8, device="cuda")
    side, graphs = torch.cuda.Stream(), []
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for a, o in zip(args, outs):
            lca.mla_latent_decode_fp4(*a, out=o, workspace=shared)
        side.synchronize()
        for a, o in zip(args, outs):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=side):
                lca.mla_latent_decode_fp4(*a, out=o, workspace=shared)
        for o in outs:
            o.fill_(7.0)
        for k in (0, 1, 1, 0, 1):
            graphs[k].replay()
    side.synchronize()
    for o, w in zip(outs, want):
        assert np.array_equal(o.double().cpu().numpy(), w)
        o.fill_(7.0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        for s, a, o in zip(streams, args, outs):
            with torch.cuda.stream(s):
                lca.mla_latent_decode_fp4(*a, out=o)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert np.array_equal(o.double().cpu().numpy(), w)
    assert lca.mla_get_device_error() == 0


def test_captured_between_copies_and_branches(env):
    """A graph in which the calls follow copies, memsets and two joined branches, and other kernels follow them: each
    launch is a programmatic dependent, whatever kind of node comes before it."""
    torch, lca, _ = env
    d = decode_case(33, [300, 129], 400, seed=41)
    want = decode(env, d)
    src = [bf(torch, d["q_abs"]), bf(torch, W.decode_fp4(d["rows"], R)), dev(torch, d["lens"])]
    q, c, lens = (torch.empty_like(x) for x in src)
    cache = torch.empty((2, 400, ROW), dtype=torch.uint8, device="cuda")
    w_uv, zeros = bf(torch, d["w_uv"]), torch.zeros(2, dtype=torch.int32, device="cuda")
    twice, back = torch.empty(want.shape, dtype=torch.bfloat16, device="cuda"), torch.empty_like(c)
    side, other, graph = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()

    def work():
        c.copy_(src[1])
        cache.zero_()
        lca.mla_append_latent_fp4(c, cache, zeros)
        other.wait_stream(side)
        with torch.cuda.stream(other):
            q.copy_(src[0])
            lens.copy_(src[2])
        lca.mla_dequantize_latent_fp4(cache, R, out=back)
        side.wait_stream(other)
        out = lca.mla_latent_decode_fp4(q, cache, lens, w_uv)
        twice.copy_(out + out)
        lens.zero_()

    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            work()
        for _ in range(20):
            for x in (q, c, back, twice):
                x.fill_(3.0)
            graph.replay()
    side.synchronize()
    assert np.array_equal(twice.double().cpu().numpy(), 2 * want)
    assert np.array_equal(back.double().cpu().numpy(), W.decode_fp4(d["rows"], R)) and not bool(lens.any())
    assert lca.mla_get_device_error() == 0


def test_same_inputs_same_bits(env):
    d = decode_case(96, [3000, 1, 777], 3000, seed=13)
    assert np.array_equal(decode(env, d), decode(env, d))


@pytest.mark.parametrize("H", [16, 32, 48, 64, 96])
def test_same_bits_over_long_shares(env, H):
    """Many units per CTA, every buffer reused many times: flat softmaxes, so that each row counts."""
    torch, lca, oracle = env
    B, n = 16, 12000
    gen = torch.Generator(device="cuda").manual_seed(H)
    cache = torch.empty((B, n, ROW), dtype=torch.uint8, device="cuda")
    for b in range(B):
        lca.mla_quantize_latent_fp4(torch.randn((n, R), generator=gen, device="cuda"), out=cache[b])
    q = (torch.randn((B, H, R), generator=gen, device="cuda") * 0.05).bfloat16()
    w_uv = (torch.randn((H, 128, R), generator=gen, device="cuda") * 0.02).bfloat16()
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    runs = [lca.mla_latent_decode_fp4(q, cache, lens, w_uv) for _ in range(4)]
    torch.cuda.synchronize()
    assert lca.mla_get_device_error() == 0 and all(torch.equal(runs[0], x) for x in runs[1:])
    one = dict(q_abs=q[3:4].double().cpu().numpy(), lens=np.array([n], np.int32), gate=None,
               w_uv=w_uv.double().cpu().numpy(), rows=cache[3:4].cpu().numpy())
    check(env, one, runs[0][3:4].double().cpu().numpy())


def test_decode_length_outside_the_cache_is_clamped_and_reported(env):
    torch, lca, _ = env
    d = decode_case(8, [300, 50], 300, seed=14)
    want = decode(env, d)
    args = (bf(torch, d["q_abs"]), dev(torch, d["rows"]))
    for lens in ([301, 50], [2**31 - 1, 50]):
        got = lca.mla_latent_decode_fp4(*args, dev(torch, lens, torch.int32), bf(torch, d["w_uv"]))
        assert np.array_equal(got.double().cpu().numpy(), want) and lca.mla_get_device_error() == -9
    got = lca.mla_latent_decode_fp4(*args, dev(torch, [-5, 50], torch.int32), bf(torch, d["w_uv"]))
    assert not bool(got[0].any()) and np.array_equal(got[1].double().cpu().numpy(), want[1])
    assert lca.mla_get_device_error() == -9
