"""The attention operators where addresses and order matter: elements past 2^31 of
a tensor, two streams, and captured graphs, each with its own workspace.  Results
are compared with the same call at an ordinary place, bit for bit (no result
depends on where its operands lie or on what runs beside it)."""
import weakref

import pytest
import torch

import cross_layer_latent_b200 as li

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


@pytest.fixture(scope="module")
def ctx():
    c = li.Context(0)
    yield c
    c.close()


def rand(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(BF).to(DEV)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("page", [64, 7], ids=["boxes", "rows"])
def test_pages_far_into_a_pool(ctx, page):
    """Rows near the end of a pool of 9.7 GB, written and read, selected and not."""
    dim, H, d_v, n = 576, 16, 512, 150
    n_pages = 8_400_000 // page
    used = (n + page - 1) // page
    x = rand(2, n, dim, seed=1)
    q = rand(2, 1, H, dim, seed=2)
    sel = i32([list(range(0, n, 3)) + [-1] * 2, list(range(1, n, 3)) + [-1] * 2]).view(2, 1, -1)
    ws = li.attention_workspace(ctx, H, d_v)
    results = []
    for first, pages in ((0, 2 * used), (n_pages - 2 * used, n_pages)):
        data = torch.empty(pages, page, dim, dtype=BF, device=DEV)
        table = (first + torch.arange(2 * used, dtype=torch.int32).flip(0).view(2, used)).to(DEV)
        cache = li.PagedCache(data, table, i32([0, 0]))
        li.li_append_paged(ctx, cache, x, ws)
        out = [torch.empty(2, 1, H, d_v, dtype=BF, device=DEV) for _ in range(2)]
        li.li_latent_attention(ctx, cache, q, d_v, 0.04, out[0], ws)
        li.li_latent_attention(ctx, cache, q, d_v, 0.04, out[1], ws, sel=sel)
        assert li.li_device_status(ctx, ws) == "LI_OK"
        results.append(out)
        last = data.view(-1, dim)[(first + 2 * used - 1) * page]
        assert torch.equal(last, x[0, 0])
        del data, cache, last
    for near, far in zip(*results):
        assert torch.isfinite(near).all() and torch.equal(near, far)


def test_strides_past_32_bits(ctx):
    """Head rows and prompt operands whose tokens lie more than 2^31 elements apart."""
    step = 2 ** 31 + 16
    big = torch.empty(step + 4096, dtype=BF, device=DEV)
    x = big.as_strided((2, 3, 64), (step, 64, 1))
    x.copy_(rand(2, 3, 64, seed=3))
    tf = li.RowTransform(norm="rms", norm_dim=64)
    near, far = x.contiguous(), torch.empty(2, 3, 64, dtype=BF, device=DEV)
    li.li_norm_rope(ctx, [li.HeadRows(x, tf, far)], None)
    li.li_norm_rope(ctx, [li.HeadRows(near, tf, near)], None)
    assert torch.equal(near, far)
    k = big.as_strided((2, 1, 64), (step, 64, 1))
    v = big.as_strided((2, 1, 64), (step, 64, 1), 128)
    v.copy_(rand(2, 1, 64, seed=4))
    q = rand(2, 1, 64, seed=5)
    ws = li.attention_workspace(ctx, 1, 64)
    out = [torch.empty(2, 1, 64, dtype=BF, device=DEV) for _ in range(2)]
    li.li_prompt_attention(ctx, q, k, None, v, i32([0, 2]), i32([0, 2]), 2, 0.125, out[0], ws)
    li.li_prompt_attention(ctx, q, k.contiguous(), None, v.contiguous(), i32([0, 2]), i32([0, 2]), 2, 0.125, out[1], ws)
    assert li.li_device_status(ctx, ws) == "LI_OK"
    assert torch.equal(out[0], out[1]) and torch.isfinite(out[0]).all()


def calls(ctx, seed):
    """A prompt by single CTAs, one by pairs, and a cut latent group, on a workspace of their own."""
    H, n = 4, 2300
    q, kn, v, kr = (rand(*s, seed=seed + i) for i, s in enumerate(((n, H, 192), (n, H, 128), (n, H, 128), (n, 64))))
    data, table = rand(n // 64 + 1, 64, 576, seed=seed + 4), torch.arange(n // 64 + 1, dtype=torch.int32, device=DEV)[None]
    cache = li.PagedCache(data, table.contiguous(), i32([n]))
    ql = rand(1, 1, 64, 576, seed=seed + 5)
    ws = li.attention_workspace(ctx, 64, 512)
    cu = [i32([0, 2200, n]), i32([0, 1100, n])]
    outs = [torch.zeros(n, H, 128, dtype=BF, device=DEV) for _ in cu] + [torch.zeros(1, 1, 64, 512, dtype=BF, device=DEV)]

    def run(stream=None):
        for c, m, o in zip(cu, (2200, 1200), outs):
            li.li_prompt_attention(ctx, q, kn, kr, v, c, c, m, 0.07, o, ws, stream=stream)
        li.li_latent_attention(ctx, cache, ql, 512, 0.04, outs[2], ws, stream=stream)

    return run, outs, ws


def test_two_streams_with_a_workspace_each(ctx):
    pairs = [calls(ctx, 10), calls(ctx, 20)]
    for run, _, _ in pairs:
        run()
    torch.cuda.synchronize()
    good = [[o.clone() for o in outs] for _, outs, _ in pairs]
    streams = [torch.cuda.Stream() for _ in pairs]
    for _, outs, _ in pairs:
        for o in outs:
            o.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for (run, _, _), s in zip(pairs, streams):
            run(s.cuda_stream)
    torch.cuda.synchronize()
    for (_, outs, ws), g in zip(pairs, good):
        assert li.li_device_status(ctx, ws) == "LI_OK"
        assert all(torch.equal(a, b) for a, b in zip(outs, g))


def test_two_graphs_with_a_workspace_each(ctx):
    pairs = [calls(ctx, 30), calls(ctx, 40)]
    graphs, good = [], []
    for run, outs, _ in pairs:
        run()
        torch.cuda.synchronize()
        good.append([o.clone() for o in outs])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        graphs.append(g)
        for o in outs:
            o.zero_()
    streams = [torch.cuda.Stream() for _ in pairs]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (_, outs, ws), g in zip(pairs, good):
        assert li.li_device_status(ctx, ws) == "LI_OK"
        assert all(torch.equal(a, b) for a, b in zip(outs, g))


def test_a_captured_attend_outlives_a_wider_one(ctx):
    """A graph of the group's attention keeps its workspace when a later call needs a larger one."""
    G = li.GroupIndexer(ctx, batch=1, capacity=512, d_c=64, H=8, d_k=64, G=1, k=300)
    G.idx[0].copy_(i32(list(range(300))).view(1, 1, -1))
    n = 400
    data = rand(8, 64, 576, seed=50)
    cache = li.PagedCache(data, torch.arange(8, dtype=torch.int32, device=DEV)[None].contiguous(), i32([n]))
    q = rand(1, 1, 16, 576, seed=51)
    out = torch.empty(1, 1, 16, 64, dtype=BF, device=DEV)
    G.attend(0, cache, q, 64, 0.04, out)
    torch.cuda.synchronize()
    good, held = out.clone(), weakref.ref(G.ws_attn)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        G.attend(0, cache, q, 64, 0.04, out)
    G.attend(0, cache, q, 512, 0.04, torch.empty(1, 1, 16, 512, dtype=BF, device=DEV))
    assert held() is not None
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, good)
