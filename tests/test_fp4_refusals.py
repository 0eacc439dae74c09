"""What the entry points of the fp4 latent cache refuse or take without a GPU, beside test_fp4_codec.py: empty calls,
streams of another device."""
import pytest

from tests.test_fp4_codec import FAKE, NULL, OK, lib  # noqa: F401 (lib: the fixture)


def test_decode_of_nothing(lib):  # noqa: F811
    """No sequences: nothing to read or write, whatever the pointers; a cache without rows needs no address."""
    args = dict(q=None, c4=None, lens=None, w_uv=None, out=None)

    def call(B, q, c4, lens, w_uv, out, max_len=0):
        return lib.mla_latent_decode_fp4(q, c4, 272, lens, max_len, w_uv, None, 1.0, out, B, 96, 128, 512, None, 0, None)

    assert call(0, **args) == OK and call(0, **args, max_len=9) == OK
    assert call(2, **dict.fromkeys(args, FAKE) | {"c4": None}, max_len=9) == NULL
    assert call(2, **dict.fromkeys(args, FAKE) | {"c4": None}) not in (OK, NULL)   # goes on to the workspace


def test_stream_of_another_device():
    import torch

    import latent_compressed_attention_gb300 as lca

    class Stream:
        device = torch.device("cuda", 1)

    with pytest.raises(ValueError, match="cuda:1"):
        lca._on(Stream(), torch.device("cuda", 0))
