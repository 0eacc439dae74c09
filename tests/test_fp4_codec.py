"""The host codec of the fp4 latent cache (workloads.encode_fp4 / decode_fp4), the oracle side of its GPU tests,
against a brute-force search over the format's definition, and the refusals of the entry points that take such a cache."""
import math

import numpy as np
import pytest

from latent_compressed_attention_gb300 import workloads as W


def nearest(x, e):
    """The e2m1 value nearest to x * 2^-e (of two, the one with the even index), times 2^e, by search."""
    m = abs(x) * 2.0**-e
    best = min(range(8), key=lambda k: (abs(m - W.E2M1[k]), k % 2))
    return math.copysign(W.E2M1[best] * 2.0**e, x)


@pytest.mark.parametrize("r", [32, 96, 512])
def test_values_are_the_nearest_ones(r):
    rng = np.random.default_rng(r)
    c = W.round_bf16(rng.standard_normal((6, r)) * np.exp2(rng.integers(-45, 45, (6, 1))))
    c[0, :16] = 2.0 ** -3 * np.array([7, -7, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -5, -0.25, 6, 4, 0, -0.0, 0.5])
    c[0, 16:32] = 0
    c[1, :32] = 0
    got = W.decode_fp4(W.encode_fp4(c), r)
    for i in range(6):
        for g in range(r // 32):
            x = c[i, 32 * g : 32 * g + 32]
            e = next((e for e in range(-40, 41) if np.abs(x).max() <= 7 * 2.0**e), 40)
            assert np.array_equal(got[i, 32 * g : 32 * g + 32], [nearest(v, e) for v in x]), (i, g, e)


def test_rounding_bound_and_layout():
    """Within a group no value is off by more than its exponent's unit (half the widest step, 4 to 6, and the
    saturation from 7 to 6), and the row is r / 2 code bytes, r / 32 scale bytes and zeros up to 16."""
    rng = np.random.default_rng(3)
    c = rng.standard_normal((50, 96))
    rows = W.encode_fp4(c)
    assert rows.shape == (50, 64) and W.fp4_row_bytes(512) == 272 and W.fp4_row_bytes(32) == 32
    assert not rows[:, 51:].any()
    unit = np.exp2(rows[:, 48:51].astype(np.float64) - 127).repeat(32, -1)
    assert np.all(np.abs(W.decode_fp4(rows, 96) - c) <= unit)
    top = np.abs(c.reshape(50, 3, 32)).max(-1).repeat(32, -1)
    assert np.all(top <= 7 * unit) and np.all(top > 3.5 * unit)


def test_nan_groups_and_scale_range():
    c = np.ones((3, 64))
    c[0, 5], c[1, 40] = np.nan, -np.inf
    v = W.decode_fp4(W.encode_fp4(c), 64)
    assert np.isnan(v[0, :32]).all() and np.all(v[0, 32:] == 1)
    assert np.isnan(v[1, 32:]).all() and np.all(v[1, :32] == 1) and np.all(v[2] == 1)
    rows = W.encode_fp4(np.full((1, 32), 6.0))
    for X, e in ((0, -40), (86, -40), (87, -40), (127, 0), (167, 40), (168, 40), (254, 40)):
        rows[0, 16] = X
        assert np.all(W.decode_fp4(rows, 32) == W.decode_fp4(rows, 32)[0, 0]) and W.decode_fp4(rows, 32)[0, 0] > 0
        ratio = W.decode_fp4(rows, 32)[0, 0] / 2.0**e
        assert ratio in W.E2M1


# ------------------------------------------------------------------------- refusals of the entry points (host only)
OK, NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, UNSUPPORTED = 0, -1, -2, -3, -4, -5, -6
FAKE = 0x10000   # an aligned address that is never dereferenced: the checks fail first


@pytest.fixture(scope="module")
def lib():
    import latent_compressed_attention_gb300 as lca
    from latent_compressed_attention_gb300 import _build
    _build.build()
    return lca.library()


def test_row_bytes(lib):
    for r in (32, 64, 96, 512, 65536):
        assert lib.mla_latent_fp4_row_bytes(r) == W.fp4_row_bytes(r)
    for r in (0, -32, 31, 48, 65568):
        assert lib.mla_latent_fp4_row_bytes(r) == 0


def quantize(lib, c=FAKE, ld_c=512, c4=FAKE, ld=272, rows=4, r=512, dtype=0):
    return lib.mla_quantize_latent_fp4(c, ld_c, c4, ld, rows, r, dtype, None)


def append(lib, c=FAKE, ld_c=512, c4=FAKE, ld=272, lens=FAKE, counts=None, max_len=9, B=2, T=1, r=512, dtype=0):
    return lib.mla_append_latent_fp4(c, ld_c, c4, ld, lens, counts, max_len, B, T, r, dtype, None)


def dequantize(lib, c=FAKE, ld_c=512, c4=FAKE, ld=272, batch=2720, lens=None, B=2, rows=9, r=512, dtype=0):
    return lib.mla_dequantize_latent_fp4(c4, ld, batch, lens, c, ld_c, B, rows, r, dtype, None)


@pytest.mark.parametrize("call", [quantize, append, dequantize])
def test_rows_refusals(lib, call):
    for bad, status in ((dict(c=None), NULL), (dict(c4=None), NULL), (dict(dtype=2), DTYPE), (dict(r=0), SHAPE),
                        (dict(r=48), UNSUPPORTED), (dict(r=65568, ld_c=65568, ld=65568), UNSUPPORTED),
                        (dict(ld_c=511), SHAPE), (dict(ld=256), SHAPE), (dict(ld=280), ALIGN), (dict(ld_c=516), ALIGN),
                        (dict(ld_c=514, dtype=1), ALIGN), (dict(c=FAKE + 8), ALIGN), (dict(c4=FAKE + 4), ALIGN),
                        (dict(ld_c=2**62), SHAPE), (dict(ld=2**62), SHAPE)):
        assert call(lib, **bad) == status, bad
    if call is quantize:
        assert call(lib, rows=-1) == SHAPE and call(lib, rows=0, c=None, c4=None) == OK
        return
    assert call(lib, B=-1) == SHAPE and call(lib, B=0, c=None, c4=None) == OK
    assert call(lib, lens=FAKE + 4) == ALIGN
    if call is append:
        assert call(lib, T=-1) == SHAPE and call(lib, T=0) == OK and call(lib, max_len=-1) == SHAPE
        assert call(lib, lens=None) == NULL and call(lib, counts=FAKE + 8) == ALIGN
    else:
        assert call(lib, rows=-1) == SHAPE and call(lib, rows=0) == OK
        assert call(lib, batch=-16) == SHAPE and call(lib, batch=2721) == ALIGN and call(lib, batch=2**62) == SHAPE


def test_decode_refusals(lib):
    def call(q=FAKE, c4=FAKE, ld=272, lens=FAKE, max_len=100, w_uv=FAKE, gate=None, out=FAKE, B=2, H=96, d_v=128, r=512):
        return lib.mla_latent_decode_fp4(q, c4, ld, lens, max_len, w_uv, gate, 1.0, out, B, H, d_v, r, None, 0, None)

    for name in ("q", "c4", "lens", "w_uv", "out"):
        assert call(**{name: None}) == NULL and call(**{name: FAKE + 8}) == ALIGN
    for bad, status in ((dict(gate=FAKE + 2), ALIGN), (dict(ld=256), SHAPE), (dict(ld=280), ALIGN), (dict(H=97), UNSUPPORTED),
                        (dict(H=0), SHAPE), (dict(d_v=64), UNSUPPORTED), (dict(r=256), UNSUPPORTED), (dict(B=-1), SHAPE),
                        (dict(max_len=-1), SHAPE), (dict(ld=2**60), SHAPE)):
        assert call(**bad) == status, bad
    assert call(B=0) == OK
    assert lib.mla_latent_decode_fp4_workspace_size(2, 97, 512, 100) == 0
    assert lib.mla_latent_decode_fp4_workspace_size(0, 96, 512, 100) == 0


def test_binding_refuses_host_tensors():
    import torch

    import latent_compressed_attention_gb300 as lca
    with pytest.raises(ValueError):
        lca.mla_quantize_latent_fp4(torch.zeros(4, 512))
    with pytest.raises(ValueError):
        lca.mla_append_latent_fp4(torch.zeros(1, 1, 512), torch.zeros(1, 4, 272, dtype=torch.uint8), torch.zeros(1))
    with pytest.raises(TypeError):
        lca.mla_dequantize_latent_fp4(torch.zeros(1, 4, 272, dtype=torch.uint8), 512)
    with pytest.raises(ValueError):
        lca.mla_latent_decode_fp4(torch.zeros(1, 4, 512), torch.zeros(1, 4, 272, dtype=torch.uint8), torch.zeros(1),
                                  torch.zeros(4, 128, 512))
