"""Row transforms that the other tests of the operators leave out: parts that are switched off while their ranges and
parameters stay set, and in the paged append layer norms, offsets and rotations by halves, in reach of the wide body
and out of it."""
import dataclasses

import numpy as np
import pytest
import torch

import cross_layer_latent_b200 as li
from oracle import attention as A
from tests.test_gpu_attention import BF, DEV, F32, Pool, check_rows, f64, make_tf, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = li.Context(0)
    yield c
    c.close()


def appended(ctx, x, tf, page=8):
    """The rows of x [1, T, dim] as they stand in the cache."""
    _, T, dim = x.shape
    pool = Pool([0], T, page, dim, x.dtype)
    pool.cache.page_table.copy_(torch.arange(pool.table_cpu.numel(), dtype=torch.int32).view(1, -1))
    ws = li.attention_workspace(ctx, 1, 1)
    li.li_append_paged(ctx, pool.cache, x, ws, tf=tf)
    assert li.li_device_status(ctx, ws) == "LI_OK" and pool.cache.lengths.tolist() == [T]
    return pool.cache.data.view(-1, dim)[:T]


def normed(ctx, x, tf):
    out = torch.full_like(x, float("nan"))
    pos = torch.arange(x.shape[1], dtype=torch.int32, device=DEV)
    rows = [li.HeadRows(t.transpose(0, 1), tf, o.transpose(0, 1)) for t, o in ((x, out),)]
    li.li_norm_rope(ctx, rows, pos)
    return out[0]


@pytest.mark.parametrize("op", [appended, normed])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("dim", [48, 96, 192, 576, 1024, 20], ids=lambda d: f"d{d}")
def test_a_norm_that_is_off_does_nothing(ctx, op, dim, dt):
    """Neither its range nor gamma, beta or an eps that no norm would take; the same for a rotation of size 0."""
    if dim * dt.itemsize % 16:
        pytest.skip("rows of this type are not whole 16-byte pieces")
    rope = 16 if dim >= 48 else 4
    x = rand(1, 9, dim, dtype=dt, seed=dim).to(DEV)
    on = make_tf(dim, "rms", rope, False, 4, ndim=dim - rope, beta=True)
    for off in (dataclasses.replace(on, norm="none"), dataclasses.replace(on, norm="none", eps=float("nan"))):
        got = op(ctx, x, off)
        assert torch.equal(got[:, :dim - rope], x[0, :, :dim - rope]), "rows of a norm that is off changed"
        tf = li.RowTransform(rope_offset=dim - rope, rope_dim=rope, inv_freq=on.inv_freq)
        check_rows(got, x[0], tf, np.arange(9), "rotation alone")
    still = dataclasses.replace(on, norm="none", rope_dim=0)
    assert torch.equal(op(ctx, x, still), x[0])
    check_rows(op(ctx, x, dataclasses.replace(on, rope_dim=0)), x[0], dataclasses.replace(on, rope_dim=0), np.arange(9), "norm alone")


TF = [  # dim, norm, rope, halves, options
    (576, "layer", 64, False, dict(ndim=512)), (576, "layer", 64, True, dict(ndim=512, beta=True)),
    (576, "rms", 64, True, dict(ndim=512)), (576, "rms", 64, False, dict(ndim=512, beta=True)), (576, "none", 64, True, {}),
    (192, "layer", 64, False, {}), (48, "rms", 16, True, dict(ndim=32, beta=True)),
    # by halves across the wide body's 16 lanes of 8 elements, and with partners in another register
    (192, "rms", 64, True, dict(roff=96)), (384, "layer", 384, True, dict(roff=0, beta=True)), (320, "rms", 256, True, dict(roff=0)),
    # the body of odd sizes and of rows past 640
    (40, "layer", 12, True, dict(noff=3, ndim=30, roff=5, beta=True)), (1024, "layer", 128, True, dict(beta=True)),
    (704, "none", 64, True, {}), (104, "layer", 30, False, dict(ndim=74)),
]


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", TF, ids=[f"d{c[0]}-{c[1]}-{c[2]}{'h' if c[3] else 'p'}" for c in TF])
def test_append_paged_transforms(ctx, case, dt):
    dim, norm, rope, halves, opt = case
    tf = make_tf(dim, norm, rope, halves, 7, **opt)
    x = rand(1, 37, dim, dtype=dt, seed=dim).to(DEV)
    check_rows(appended(ctx, x, tf), x[0], tf, np.arange(37), "append")
