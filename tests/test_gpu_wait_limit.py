"""Bounded waits: with a wait limit of 0 every wait of the scan that is not
already satisfied gives up (the first wait for copied data always is not);
the kernel records LI_ERR_DEVICE_TIMEOUT, lets its own copies land, frees
its tensor memory and returns, and the context stays usable."""
import numpy as np
import pytest
import torch

import cross_layer_latent_b200 as li
from oracle import indexer
from tests.gpu_setup import build_group
from workloads import generate, shrunk, workload

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_wait_that_runs_out_is_reported_and_the_context_recovers():
    ctx = li.Context(0)
    try:
        wl = shrunk(workload(1), capacity=3000, queries=1)
        inp = generate(wl)
        g = build_group(ctx, inp, dsa=False)
        assert li.li_device_status(ctx, g.ws) == "LI_OK"
        li.li_set_wait_limit(ctx, 0)
        try:
            g.score_topk(0)
            st = li.li_device_status(ctx, g.ws)
        finally:
            li.li_set_wait_limit(ctx, 2_000_000_000)
        assert st == "LI_ERR_DEVICE_TIMEOUT"
        dump = torch.full((wl.batch, 1, wl.capacity), float("nan"), device=DEV)
        g.score_topk(0, dump=dump)
        assert li.li_device_status(ctx, g.ws) == "LI_OK"
        d, idx = dump.cpu().numpy(), g.idx[0].cpu().numpy()
        n = int(inp.lengths[0])
        e, _ = indexer.topk(d[0, 0, :n], wl.k, n)
        assert np.array_equal(idx[0, 0], e)
        assert np.isfinite(d[0, 0, :n]).all()
    finally:
        ctx.close()


def test_follower_gather_wait_that_runs_out_is_reported_and_the_context_recovers():
    """The same for the row-gather scan, whose two loader warps hand each
    stage over through a barrier of their own."""
    ctx = li.Context(0)
    try:
        wl = shrunk(workload(1), capacity=3000, queries=1)
        inp = generate(wl)
        g = build_group(ctx, inp, dsa=False)
        g.hs_anchor(0)
        torch.cuda.synchronize()
        assert li.li_device_status(ctx, g.ws) == "LI_OK"
        li.li_set_wait_limit(ctx, 0)
        try:
            g.hs_follower(1)
            st = li.li_device_status(ctx, g.ws)
        finally:
            li.li_set_wait_limit(ctx, 2_000_000_000)
        assert st == "LI_ERR_DEVICE_TIMEOUT"
        g.hs_anchor(0)                     # fresh candidates (li_device_status cleared the status)
        fdump = torch.full((wl.batch, 1, wl.B), float("nan"), device=DEV)
        g.hs_follower(1, dump=fdump)
        assert li.li_device_status(ctx, g.ws) == "LI_OK"
        fd, fidx = fdump.cpu().numpy(), g.idx[1].cpu().numpy()
        cand, cand_n = g.cand.cpu().numpy(), g.cand_n.cpu().numpy()
        cn = int(cand_n[0, 0])
        ef, _ = indexer.hs_follower(fd[0, 0, :cn], cand[0, 0], cn, wl.k)
        assert np.array_equal(fidx[0, 0], ef)
        assert np.isfinite(fd[0, 0, :cn]).all()
    finally:
        ctx.close()


@pytest.mark.parametrize("case", [([300] * 3, 1), ([20000], 1), ([200, 4000], 5)], ids=["groups", "split", "queries"])
def test_latent_attention_wait_that_runs_out_is_reported_and_the_context_recovers(case):
    """The attention kernels; the call before leaves the workspace with entries of other sizes."""
    lens, T = case
    ctx = li.Context(0)
    try:
        ws = li.attention_workspace(ctx, 16, 512)
        rng = torch.Generator().manual_seed(5)

        def call(lens, T):
            b, pages = len(lens), (max(lens) + 63) // 64
            data = torch.randn(b * pages, 64, 576, generator=rng).bfloat16().to(DEV)
            table = torch.arange(b * pages, dtype=torch.int32, device=DEV).view(b, pages)
            cache = li.PagedCache(data, table, torch.tensor(lens, dtype=torch.int32, device=DEV))
            q = torch.randn(b, T, 16, 576, generator=rng).bfloat16().to(DEV)
            out = torch.zeros(b, T, 16, 512, dtype=torch.bfloat16, device=DEV)
            return out, lambda: li.li_latent_attention(ctx, cache, q, 512, 0.04, out, ws)

        _, large = call([700] * 40, 3)
        out, run = call(lens, T)
        run()
        good = out.clone()
        large()
        li.li_set_wait_limit(ctx, 0)
        try:
            run()
            st = li.li_device_status(ctx, ws)
        finally:
            li.li_set_wait_limit(ctx, 2_000_000_000)
        assert st == "LI_ERR_DEVICE_TIMEOUT"
        run()
        assert li.li_device_status(ctx, ws) == "LI_OK"
        assert torch.equal(out, good) and torch.isfinite(out).all()
    finally:
        ctx.close()


@pytest.mark.parametrize("nq", [[300, 40], [2200, 5]], ids=["single", "pair"])
def test_prompt_attention_wait_that_runs_out_is_reported_and_the_context_recovers(nq):
    ctx = li.Context(0)
    try:
        n, H = sum(nq), 4
        rng = torch.Generator().manual_seed(6)
        q, kn, v, kr = (torch.randn(*s, generator=rng).bfloat16().to(DEV) for s in ((n, H, 192), (n, H, 128), (n, H, 128), (n, 64)))
        cu = torch.tensor([0, nq[0], n], dtype=torch.int32, device=DEV)
        ws = li.attention_workspace(ctx, H, 128)
        out = torch.zeros(n, H, 128, dtype=torch.bfloat16, device=DEV)
        run = lambda: li.li_prompt_attention(ctx, q, kn, kr, v, cu, cu, max(nq), 0.07, out, ws)  # noqa: E731
        run()
        good = out.clone()
        li.li_set_wait_limit(ctx, 0)
        try:
            run()
            st = li.li_device_status(ctx, ws)
        finally:
            li.li_set_wait_limit(ctx, 2_000_000_000)
        assert st == "LI_ERR_DEVICE_TIMEOUT"
        for _ in range(2):
            out.zero_()
            run()
            assert li.li_device_status(ctx, ws) == "LI_OK"
            assert torch.equal(out, good)
    finally:
        ctx.close()
