"""What the entry points of the paged latent cache refuse or take without a GPU: host-side validation comes before any
launch (CPU)."""
import pytest
import torch

import latent_compressed_attention_gb300 as lca
from tests.test_abi import ERR_ALIGN, ERR_DTYPE, ERR_NULL, ERR_SHAPE, ERR_UNSUPPORTED, FAKE, OK, lib  # noqa: F401

BIG = 2**31 - 1


def reserve(lib, **kw):  # noqa: F811
    a = dict(lens=FAKE, counts=FAKE, table=FAKE, ld=8, held=FAKE, free=FAKE, free_count=FAKE, slots=FAKE, B=2, T=4, wide=8,
             capacity=16, bs=64) | kw
    return lib.mla_reserve_latent_blocks(*a.values(), None)


def append(lib, **kw):  # noqa: F811
    a = dict(c=FAKE, ld_c=512, pool=FAKE, ld_pool=512, pool_rows=640, slots=FAKE, rows=4, r=512, dtype=0) | kw
    return lib.mla_append_latent_paged(*a.values(), None)


def attend(lib, **kw):  # noqa: F811
    a = dict(q=FAKE, pool=FAKE, ld_pool=512, table=FAKE, ld_table=8, lens=FAKE, counts=FAKE, parents=FAKE, w_uv=FAKE,
             gate=FAKE, scale=1.0, window=0, sinks=0, out=FAKE, B=2, T=4, H=96, d_v=128, r=512, blocks=10, bs=64, wide=8,
             ws=None, ws_bytes=0) | kw
    return lib.mla_latent_attend_paged(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), ERR_SHAPE), (dict(T=-1), ERR_SHAPE), (dict(wide=-1), ERR_SHAPE), (dict(capacity=-1), ERR_SHAPE),
    (dict(bs=0), ERR_SHAPE), (dict(ld=7), ERR_SHAPE), (dict(wide=2**25, ld=2**25, bs=64), ERR_SHAPE),
    (dict(B=16385), ERR_UNSUPPORTED), (dict(lens=None), ERR_NULL), (dict(counts=None), ERR_NULL),
    (dict(table=None), ERR_NULL), (dict(held=None), ERR_NULL), (dict(free=None), ERR_NULL),
    (dict(free_count=None), ERR_NULL), (dict(slots=None), ERR_NULL), (dict(lens=FAKE + 2), ERR_ALIGN),
    (dict(slots=FAKE + 4), ERR_ALIGN), (dict(B=0, lens=None, slots=None), OK)])
def test_reserve(lib, kw, want):  # noqa: F811
    assert reserve(lib, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), ERR_DTYPE), (dict(rows=-1), ERR_SHAPE), (dict(r=0), ERR_SHAPE), (dict(r=12), ERR_SHAPE),
    (dict(ld_c=504), ERR_SHAPE), (dict(ld_pool=504), ERR_SHAPE), (dict(pool_rows=2**31), ERR_SHAPE),
    (dict(pool_rows=-1), ERR_SHAPE), (dict(c=None), ERR_NULL), (dict(pool=None), ERR_NULL), (dict(slots=None), ERR_NULL),
    (dict(c=FAKE + 8), ERR_ALIGN), (dict(ld_pool=516), ERR_ALIGN), (dict(ld_c=516), ERR_ALIGN),
    (dict(slots=FAKE + 1), ERR_ALIGN), (dict(rows=0, c=None, slots=None), OK)])
def test_append(lib, kw, want):  # noqa: F811
    assert append(lib, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), ERR_SHAPE), (dict(T=-1), ERR_SHAPE), (dict(H=0), ERR_SHAPE), (dict(window=-1), ERR_SHAPE),
    (dict(sinks=-1), ERR_SHAPE), (dict(bs=0), ERR_SHAPE), (dict(blocks=-1), ERR_SHAPE), (dict(wide=-1), ERR_SHAPE),
    (dict(ld_pool=511), ERR_SHAPE), (dict(ld_table=7), ERR_SHAPE), (dict(blocks=2**25), ERR_SHAPE),
    (dict(wide=2**25, ld_table=2**25), ERR_SHAPE), (dict(B=BIG, T=64), ERR_SHAPE), (dict(H=129), ERR_UNSUPPORTED),
    (dict(r=256), ERR_UNSUPPORTED), (dict(d_v=64), ERR_UNSUPPORTED), (dict(bs=32), ERR_UNSUPPORTED),
    (dict(bs=96), ERR_UNSUPPORTED), (dict(T=65), ERR_UNSUPPORTED), (dict(q=None), ERR_NULL), (dict(pool=None), ERR_NULL),
    (dict(table=None), ERR_NULL), (dict(lens=None), ERR_NULL), (dict(w_uv=None), ERR_NULL), (dict(out=None), ERR_NULL),
    (dict(q=FAKE + 8), ERR_ALIGN), (dict(gate=FAKE + 8), ERR_ALIGN), (dict(ld_pool=516), ERR_ALIGN),
    (dict(lens=FAKE + 2), ERR_ALIGN), (dict(B=0, q=None), OK), (dict(T=0, q=None), OK)])
def test_attend(lib, kw, want):  # noqa: F811
    assert attend(lib, **kw) == want


def test_attend_workspace_of_unsupported_sizes(lib):  # noqa: F811
    size = lca.mla_latent_attend_paged_workspace_size
    assert size(0, 1, 96, 512) == size(1, 0, 96, 512) == size(1, 1, 129, 512) == size(1, 1, 96, 256) == 0
    assert size(BIG, 64, 96, 512) == 0


def test_tensors_of_the_host(lib):  # noqa: F811
    i32 = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        lca.mla_reserve_latent_blocks(i32, i32, 1, i32.view(2, 1), i32, i32, i32[:1], 64)
    c, pool = torch.zeros(2, 512, dtype=torch.bfloat16), torch.zeros(1, 64, 512, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        lca.mla_append_latent_paged(c, pool, i32)
    with pytest.raises(ValueError, match="CUDA"):
        lca.mla_latent_attend_paged(c.view(1, 2, 1, 512), pool, i32.view(1, 2), i32[:1], c.new_zeros(1, 128, 512))
    with pytest.raises(ValueError, match="32 bits"):
        lca._count(2**31, "window")
