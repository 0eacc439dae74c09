"""GPU tests of the fp4 latent cache at its edges, with the helpers and the elementwise bounds of test_parity_fp4.py:
heads whose running maxima move together, weights and groups far below the largest, the sizes and arguments that the
other file leaves out."""
import numpy as np
import pytest

from latent_compressed_attention_gb300 import workloads as W
from tests.test_parity_fp4 import R, check, decode, decode_case, env, latent  # noqa: F401 (env: the fixture)

pytestmark = pytest.mark.gpu


def counted_rows(n, seed):
    """Latent rows that hold their own number u = d0 + 7 d1 + 49 d2 + 343 d3 in columns 32, 64, 96 and 128, as values
    that e2m1 has: d0 .. d2 less 3, d3 less 1 (n < 343 * 6); columns 32 .. 159 are zero otherwise."""
    c, u = latent(np.random.default_rng(seed), (n, R)), np.arange(n)
    c[:, 32:160] = 0.0
    c[:, 32], c[:, 64], c[:, 96], c[:, 128] = u % 7 - 3.0, u // 7 % 7 - 3.0, u // 49 % 7 - 3.0, u // 343 - 1.0
    return c


@pytest.mark.parametrize("H", [16, 31, 48, 49, 64, 96])
def test_heads_whose_maxima_move_together(env, H):  # noqa: F811
    """Scores rise from row to row, in neighbouring heads by different steps: the running maxima of heads that share
    columns of the accumulator move in the same unit, each by an amount of its own."""
    n = 2050
    d = decode_case(H, [n], n, seed=51)
    d["rows"][0] = W.encode_fp4(counted_rows(n, 52))
    d["q_abs"][:] = 0.0
    step = 0.01 * (1 + np.arange(H) % 5)
    for k, at in enumerate((32, 64, 96, 128)):
        d["q_abs"][0, :, at] = W.round_bf16(step * 7.0**k)
    got = decode(env, d)
    check(env, d, got)
    for _ in range(5):
        assert np.array_equal(decode(env, d), got)
