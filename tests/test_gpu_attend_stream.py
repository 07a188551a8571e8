"""GroupIndexer.attend on a stream of the caller's while the current stream is busy: the workspace that its first call
makes is ready on that stream before the kernels use it."""
import pytest
import torch

import cross_layer_latent_b200 as li

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


@pytest.mark.parametrize("as_int", [False, True], ids=["stream", "handle"])
def test_first_attend_on_another_stream(as_int):
    ctx = li.Context(0)
    try:
        n, H, d_v = 400, 16, 64
        G = li.GroupIndexer(ctx, batch=1, capacity=512, d_c=64, H=8, d_k=64, G=1, k=300)
        sel = torch.arange(300, dtype=torch.int32, device=DEV)
        sel[7] = n                               # past the prefix: the call's status word says so
        G.idx[0].copy_(sel.view(1, 1, -1))
        data = torch.randn(8, 64, 576, generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
        cache = li.PagedCache(data, torch.arange(8, dtype=torch.int32, device=DEV)[None].contiguous(),
                              torch.tensor([n], dtype=torch.int32, device=DEV))
        q = torch.randn(1, 1, H, 576, generator=torch.Generator().manual_seed(2)).to(BF).to(DEV)
        out = torch.zeros(1, 1, H, d_v, dtype=BF, device=DEV)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        torch.cuda._sleep(200_000_000)           # about a tenth of a second on the current stream
        G.attend(0, cache, q, d_v, 0.04, out, stream=side.cuda_stream if as_int else side)
        side.synchronize()
        first = out.clone()
        torch.cuda.synchronize()
        assert li.li_device_status(ctx, G.ws_attn) == "LI_ERR_INDEX", "the workspace was cleared after the call"
        # on the current stream, and a wider one's first call with the default stream's handle
        G.attend(0, cache, q, d_v, 0.04, out)
        wide = torch.zeros(1, 1, H, 512, dtype=BF, device=DEV)
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)
            G.attend(0, cache, q, 512, 0.04, wide, stream=0)
        torch.cuda.synchronize()
        assert torch.equal(out, first) and (first != 0).any()
        assert li.li_device_status(ctx, G.ws_attn) == "LI_ERR_INDEX"
    finally:
        ctx.close()
