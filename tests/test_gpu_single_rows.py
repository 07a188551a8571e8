"""Operands of one token, one head or one row, whose strides over that dimension are whatever the view left: no call
steps by them."""
import pytest
import torch

import cross_layer_latent_b200 as li
from tests.test_gpu_attention import BF, DEV, F32, check_prompt, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = li.Context(0)
    yield c
    c.close()


def odd(t, dims):
    """The tensor with strides over `dims`, of size 1, that no row alignment fits."""
    assert all(t.shape[d] == 1 for d in dims)
    return t.as_strided(t.shape, [(13, 7)[d] if d in dims else s for d, s in enumerate(t.stride())])


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("nq, nk, H", [(1, 1, 1), (1, 1, 3), (5, 9, 1), (1, 40, 2)])
def test_prompt_of_one_token_or_head(ctx, nq, nk, H, dt):
    dn, dr, dv = 64, 32, 64
    q, kn, v, kr = (rand(*s, dtype=dt, seed=i).to(DEV) for i, s in enumerate(((nq, H, dn + dr), (nk, H, dn), (nk, H, dv), (nk, dr))))
    ones = lambda n: [d for d, c in enumerate((n, H)) if c == 1]  # noqa: E731
    cu = lambda n: torch.tensor([0, n], dtype=torch.int32, device=DEV)  # noqa: E731
    out, lse = torch.empty(nq, H, dv, dtype=dt, device=DEV), torch.empty(nq, H, device=DEV)
    ws = li.attention_workspace(ctx, H, dv)
    li.li_prompt_attention(ctx, odd(q, ones(nq)), odd(kn, ones(nk)), odd(kr, [0] if nk == 1 else []), odd(v, ones(nk)), cu(nq), cu(nk),
                           nq, 0.1, out, ws, lse=lse)
    assert li.li_device_status(ctx, ws) == "LI_OK"
    check_prompt(q, kn, kr, v, [0, nq], [0, nk], 0.1, True, out, lse)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_append_of_one_row(ctx, dt):
    c = li.PagedCache(torch.zeros(2, 4, 64, dtype=dt, device=DEV), torch.tensor([[1, 0]], dtype=torch.int32, device=DEV),
                      torch.tensor([5], dtype=torch.int32, device=DEV))
    x, ws = rand(1, 1, 64, dtype=dt).to(DEV), li.attention_workspace(ctx, 1, 1)
    li.li_append_paged(ctx, c, odd(x, [0, 1]), ws)
    assert li.li_device_status(ctx, ws) == "LI_OK" and c.lengths.tolist() == [6]
    assert torch.equal(c.data[0, 1], x[0, 0]) and (c.data.view(-1, 64)[[0, 2, 3, 4, 5, 6, 7]] == 0).all()
