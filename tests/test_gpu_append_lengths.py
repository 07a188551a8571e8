"""The paged append where starts or numbers of rows are the lengths themselves: every row reads them before they
advance."""
import pytest
import torch

import cross_layer_latent_b200 as li
from tests.test_gpu_attention import BF, DEV, F32, rand, refused

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = li.Context(0)
    yield c
    c.close()


def cache(batch, per, page, dim, lens, dt=BF):
    table = torch.randperm(batch * per, generator=torch.Generator().manual_seed(3)).to(torch.int32).view(batch, per).to(DEV)
    return li.PagedCache(torch.zeros(batch * per, page, dim, dtype=dt, device=DEV), table, torch.tensor(lens, dtype=torch.int32, device=DEV))


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(3, 5, 4, 64), (40, 700, 16, 64), (5, 333, 7, 1024)], ids=["small", "many", "odd"])
@pytest.mark.parametrize("starts", ["other", "lengths", "none"])
def test_append_as_many_rows_as_there_are(ctx, shape, starts, dt):
    batch, T, page, dim = shape
    lens = [(T * 5 * b // batch + 3) % T + 1 if b % 4 else 0 for b in range(batch)]
    start = [(7 * b) % 11 for b in range(batch)]
    c = cache(batch, (2 * T + 12) // page + 1, page, dim, lens, dt)
    x = rand(batch, T, dim, dtype=dt, seed=1).to(DEV)
    ws = li.attention_workspace(ctx, 1, 1)
    s = {"other": torch.tensor(start, dtype=torch.int32, device=DEV), "lengths": c.lengths, "none": None}[starts]
    if starts != "other":
        start = lens
    li.li_append_paged(ctx, c, x, ws, start=s, n_new=c.lengths)
    assert li.li_device_status(ctx, ws) == "LI_OK"
    assert c.lengths.tolist() == [a + n for a, n in zip(start, lens)]
    want = torch.zeros_like(c.data).view(-1, dim)
    for b in range(batch):
        at = start[b] + torch.arange(lens[b])
        want[c.page_table[b].cpu().long()[at // page].mul(page).add(at % page).to(DEV)] = x[b, :lens[b]]
    assert torch.equal(c.data.view(-1, dim), want)


def test_append_refuses_numbers_that_overlap_the_lengths(ctx):
    buf = torch.zeros(8, dtype=torch.int32, device=DEV)
    c = li.PagedCache(torch.zeros(4, 8, 64, dtype=BF, device=DEV), torch.zeros(3, 1, dtype=torch.int32, device=DEV), buf[2:5])
    x, ws = rand(3, 1, 64, dtype=BF).to(DEV), li.attention_workspace(ctx, 1, 1)
    for other in (buf[0:3], buf[1:4], buf[3:6], buf[4:7]):
        refused("LI_ERR_ARG", li.li_append_paged, ctx, c, x, ws, start=other)
        refused("LI_ERR_ARG", li.li_append_paged, ctx, c, x, ws, start=buf[5:8], n_new=other)
    li.li_append_paged(ctx, c, x[:, :1], ws, start=buf[5:8], n_new=buf[5:8])
    assert li.li_device_status(ctx, ws) == "LI_OK"
