"""The attention operators against the fp64 oracle: head norms with rotation,
paged append, latent attention (absorbed) and prompt attention (expanded).

Tolerances count roundings.  An output rounded once to type t is off by at most
half a step, H = eps(t) / 2, of its value.  A dot product of d terms in fp32 is
off by at most d 2^-23 of the sum of its terms' absolute values (one rounding
a product and one a sum), which moves a softmax weight relatively by twice the
scaled amount; bf16 weights are rounded by H(bf16) more; exp2 and the scaling add
2^-20.  All of that weighs on sum p |v|, which `attend` returns.
"""
import dataclasses

import numpy as np
import pytest
import torch

import cross_layer_latent_b200 as li
from oracle import attention as A

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ctx():
    c = li.Context(0)
    yield c
    c.close()


def half(dt):
    return torch.finfo(dt).eps / 2


def rand(*shape, dtype=F32, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


def close(got, ref, tol, what):
    got = f64(got)
    assert got.shape == ref.shape
    fin = np.isfinite(ref)
    assert np.array_equal(got[~fin], ref[~fin]), what
    bad = np.abs(got - np.where(fin, ref, 0.0))[fin] > np.broadcast_to(tol, ref.shape)[fin]
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, worst {np.abs(got - ref)[fin].max():.3g}"


# ------------------------------------------------------------------ head norms with rotation

def transform_tol(x, kw):
    """Bound of a transformed row's error before its last rounding: sums of n terms in the norm, two products in the
    rotation, each term at most the row's largest."""
    y = np.abs(x)
    n = max(kw["norm_dim"], 1)
    r = slice(kw["norm_offset"], kw["norm_offset"] + n)
    beta = 0.0 if kw["beta"] is None else np.abs(kw["beta"]).max()
    gamma = 1.0 if kw["gamma"] is None else np.abs(kw["gamma"])
    if kw["kind"] == "rms":
        y[..., r] = np.abs(A.norm(x[..., r], "rms", gamma, None, kw["eps"])) + beta
    elif kw["kind"] == "layer":
        # the mean is off by n 2^-24 of the largest |x|, which the deviation then divides
        s = x[..., r]
        y[..., r] = 2 * np.abs(s).max(-1, keepdims=True) / np.sqrt(s.var(-1, keepdims=True) + kw["eps"]) * gamma + beta
    return (n + 16) * 2.0 ** -23 * y.max(-1, keepdims=True)


def oracle_kw(tf):
    g = lambda t: None if t is None else f64(t)  # noqa: E731
    return dict(kind=tf.norm, norm_offset=tf.norm_offset, norm_dim=tf.norm_dim, gamma=g(tf.gamma), beta=g(tf.beta),
                eps=float(np.float32(tf.eps)), rope_offset=tf.rope_offset, rope_dim=tf.rope_dim, inv_freq=g(tf.inv_freq),
                halves=tf.rope_halves)


def check_rows(got, x, tf, pos, what):
    kw = oracle_kw(tf)
    ref = A.transform(f64(x), pos, **kw)
    tol = transform_tol(f64(x), kw)
    close(got, ref, half(x.dtype) * np.abs(ref) + tol * (1 + half(x.dtype)), what)


def make_tf(dim, norm, rope, halves, seed, noff=0, ndim=None, roff=None, beta=False):
    ndim = dim - noff if ndim is None else ndim
    roff = dim - rope if roff is None else roff
    f = (10000.0 ** (-torch.arange(0, rope, 2, dtype=torch.float64) / max(rope, 1))).float().to(DEV) if rope else None
    return li.RowTransform(norm=norm, norm_offset=noff, norm_dim=ndim if norm != "none" else 0,
                           gamma=(1 + 0.3 * rand(ndim, seed=seed)).to(DEV) if norm != "none" else None,
                           beta=(0.5 * rand(ndim, seed=seed + 1)).to(DEV) if beta and norm != "none" else None, eps=1e-5,
                           rope_offset=roff if rope else 0, rope_dim=rope, rope_halves=halves, inv_freq=f)


NR = [  # n_tok, H, dim, norm, rope, halves, options
    (1, 1, 128, "rms", 64, False, {}), (3, 64, 128, "rms", 64, True, {}), (5, 7, 192, "rms", 64, True, {}),
    (700, 3, 64, "layer", 32, False, dict(beta=True)), (2, 5, 256, "none", 256, True, {}), (4, 2, 96, "rms", 0, False, {}),
    (3, 3, 576, "rms", 64, False, dict(ndim=512)), (2, 3, 1024, "layer", 128, False, dict(beta=True)),
    (2, 3, 1000, "rms", 30, True, {}), (3, 4, 7, "rms", 4, False, {}), (2, 9, 33, "layer", 10, True, dict(noff=3, roff=5)),
    (2, 2, 320, "rms", 64, True, {}), (1, 1, 1, "rms", 0, False, {}), (600, 66, 128, "rms", 128, True, {}),
    (2, 40, 40, "rms", 16, False, dict(noff=8, ndim=24, roff=0)),
]


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", NR, ids=[f"{c[0]}x{c[1]}x{c[2]}-{c[3]}-{c[4]}{'h' if c[5] else 'p'}" for c in NR])
def test_norm_rope(ctx, case, dt):
    n, H, dim, norm, rope, halves, opt = case
    tf = make_tf(dim, norm, rope, halves, 3, **opt)
    x = rand(n, H, dim, dtype=dt, seed=5).to(DEV)
    pos = torch.randint(0, 1 << 20, (n,), generator=torch.Generator().manual_seed(1)).to(torch.int32).to(DEV)
    out = torch.full_like(x, float("nan"))
    li.li_norm_rope(ctx, [li.HeadRows(x, tf, out)], pos if rope else None)
    check_rows(out, x, tf, f64(pos)[:, None], "norm_rope")
    # the same rows alone, in place, through other strides
    buf = torch.full((n, 2 * H + 1, dim + 8), 7.0, dtype=dt, device=DEV)
    view = buf[:, 1::2, :dim]
    view.copy_(x)
    li.li_norm_rope(ctx, [li.HeadRows(view, tf, view)], pos if rope else None)
    check_rows(view, x, tf, f64(pos)[:, None], "norm_rope in place")
    assert (buf[:, 0::2] == 7).all() and (buf[:, :, dim:] == 7).all()


def test_norm_rope_several_sets(ctx):
    n = 37
    pos = torch.arange(n, dtype=torch.int32, device=DEV) * 3001
    fused = rand(n, (8 + 2 + 1) * 128, dtype=BF, seed=2).to(DEV)
    q, k, ix = fused[:, :1024].unflatten(1, (8, 128)), fused[:, 1024:1280].unflatten(1, (2, 128)), fused[:, 1280:].unflatten(1, (2, 64))
    tfs = [make_tf(128, "rms", 64, False, 1), make_tf(128, "layer", 64, True, 2, beta=True), make_tf(64, "none", 64, False, 3)]
    tfs[1] = dataclasses.replace(tfs[1], inv_freq=tfs[0].inv_freq)          # shared frequencies
    outs = [torch.empty(t.shape, dtype=BF, device=DEV) for t in (q, k, ix)]
    li.li_norm_rope(ctx, [li.HeadRows(x, tf, o) for x, tf, o in zip((q, k, ix), tfs, outs)], pos)
    for x, tf, o in zip((q, k, ix), tfs, outs):
        check_rows(o, x, tf, f64(pos)[:, None], "several sets")


def test_norm_rope_far_and_negative_positions(ctx):
    pos = torch.tensor([0, -5, 2 ** 31 - 1, 123456789, -(2 ** 31)], dtype=torch.int32, device=DEV)
    tf = make_tf(64, "none", 64, False, 1)
    x = rand(5, 2, 64, seed=4).to(DEV)
    out = torch.empty_like(x)
    li.li_norm_rope(ctx, [li.HeadRows(x, tf, out)], pos)
    # the angle in double is off by 2^31 2^-52 at the farthest position
    ref = A.transform(f64(x), f64(pos)[:, None], **oracle_kw(tf))
    close(out, ref, 2.0 ** -20 * np.abs(ref) + 24 * 2.0 ** -23 * np.abs(f64(x)).max(), "far positions")


# ------------------------------------------------------------------ paged pools

class Pool:
    """Sequences of given lengths in shuffled pages; what no sequence holds is NaN."""

    def __init__(self, lens, cap, page, dim, dt, seed=0):
        g = torch.Generator().manual_seed(seed)
        per = max((cap + page - 1) // page, 1)
        self.n_pages, self.page = len(lens) * per + 2, page
        table = torch.randperm(self.n_pages, generator=g)[:len(lens) * per].reshape(len(lens), per).to(torch.int32)
        data = torch.full((self.n_pages, page, dim), float("nan"), dtype=dt)
        flat = data.view(-1, dim)
        for b, n in enumerate(lens):
            if n:
                flat[torch.from_numpy(A.page_rows(table[b], np.arange(n), page))] = rand(n, dim, dtype=dt, seed=seed + 10 + b)
        # pages past a sequence's length are never looked up: entries there may be anything
        for b, n in enumerate(lens):
            table[b, (n + page - 1) // page:] = 2 ** 30 if b % 2 else -7
        self.table_cpu, self.data_cpu = table, data
        self.cache = li.PagedCache(data.to(DEV), table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV))

    def rows(self, b, positions):
        if len(positions) == 0:
            return np.zeros((0, self.data_cpu.shape[-1]))
        return f64(self.data_cpu.view(-1, self.data_cpu.shape[-1]))[A.page_rows(self.table_cpu[b], positions, self.page)]


AP = [  # batch, T, dim, page, norm over, rope, lens, n_new
    (1, 1, 576, 64, 512, 64, [0], None), (3, 5, 576, 64, 512, 64, [0, 62, 130], [5, 0, 3]),
    (2, 33, 192, 1, 128, 64, [0, 7], None), (4, 2, 48, 17, 32, 16, [16, 17, 33, 0], [2, 1, 9, -3]),
    (2, 700, 576, 16, 512, 64, [5, 1000], [700, 699]), (2, 3, 1024, 8, 1024, 0, [1, 2], None),
    (2, 3, 20, 4, 9, 6, [1, 2], None),
]


@pytest.mark.parametrize("with_start", [False, True])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", AP, ids=[f"b{c[0]}t{c[1]}d{c[2]}p{c[3]}" for c in AP])
def test_append_paged(ctx, case, dt, with_start):
    b, T, dim, page, nd, rope, lens, n_new = case
    if dim * dt.itemsize % 16:
        pytest.skip("rows of this type are not whole 16-byte pieces")
    pool = Pool(lens, max(lens) + T, page, dim, dt, seed=3)
    pool.table_cpu = torch.randperm(pool.n_pages, generator=torch.Generator().manual_seed(9))[:pool.table_cpu.numel()].reshape(
        pool.table_cpu.shape).to(torch.int32)
    pool.cache.page_table.copy_(pool.table_cpu)
    tf = make_tf(dim, "rms", rope, False, 4, ndim=nd)
    x = rand(b, T, dim + 16, dtype=dt, seed=6).to(DEV)[..., :dim]
    ws = li.attention_workspace(ctx, 1, 1)
    start = torch.tensor(lens, dtype=torch.int32, device=DEV) if with_start else None
    nn = None if n_new is None else torch.tensor(n_new, dtype=torch.int32, device=DEV)
    before = pool.cache.data.clone()
    if with_start:
        pool.cache.lengths.fill_(12345)
    li.li_append_paged(ctx, pool.cache, x, ws, tf=tf, start=start, n_new=nn)
    counts = [T] * b if n_new is None else [min(max(v, 0), T) for v in n_new]
    assert li.li_device_status(ctx, ws) == "LI_OK"
    assert pool.cache.lengths.tolist() == [n + c for n, c in zip(lens, counts)]
    flat, flat0 = pool.cache.data.view(-1, dim), before.view(-1, dim)
    touched = torch.zeros(flat.shape[0], dtype=torch.bool)
    for i in range(b):
        if counts[i]:
            rows = torch.from_numpy(A.page_rows(pool.table_cpu[i], lens[i] + np.arange(counts[i]), page))
            touched[rows] = True
            check_rows(flat[rows.to(DEV)], x[i, :counts[i]], tf, lens[i] + np.arange(counts[i]), f"sequence {i}")
    same = (flat0.view(torch.uint8) == flat.view(torch.uint8)).view(flat.shape[0], -1).all(1).cpu()
    assert same[~touched].all(), "a row outside the appended ones changed"


def test_append_paged_reports_what_does_not_fit(ctx):
    pool = Pool([6, 2, 3], 8, 4, 64, BF)
    t = pool.cache.page_table
    t[:] = torch.tensor([[0, 1], [2, 3], [4, 99]], dtype=torch.int32)
    before = pool.cache.data.clone()
    ws = li.attention_workspace(ctx, 1, 1)
    x = rand(3, 3, 64, dtype=BF).to(DEV)
    li.li_append_paged(ctx, pool.cache, x, ws)
    # sequence 0 would need a ninth position; sequence 2's second page is not in the pool
    assert li.li_device_status(ctx, ws) in ("LI_ERR_CAPACITY", "LI_ERR_INDEX")
    assert li.li_device_status(ctx, ws) == "LI_OK"
    assert pool.cache.lengths.tolist() == [6, 5, 6]
    flat, old = pool.cache.data.view(-1, 64), before.view(-1, 64)
    assert torch.equal(flat[0:8].view(torch.int16), old[0:8].view(torch.int16))
    assert torch.equal(flat[8 + 2:8 + 5], x[1]) and torch.equal(flat[16 + 3], x[2, 0])
    start = torch.tensor([-1, 0, 6], dtype=torch.int32, device=DEV)
    li.li_append_paged(ctx, pool.cache, x, ws, start=start)
    assert li.li_device_status(ctx, ws) == "LI_ERR_CAPACITY"
    assert pool.cache.lengths.tolist() == [6, 3, 6] and torch.equal(flat[8:11], x[1])


def test_append_paged_repeats_in_a_graph(ctx):
    pool = Pool([0, 3], 64, 4, 64, BF)
    pool.cache.page_table.copy_(torch.arange(32, dtype=torch.int32).view(2, 16))
    ws = li.attention_workspace(ctx, 1, 1)
    x = rand(2, 2, 64, dtype=BF).to(DEV)
    li.li_append_paged(ctx, pool.cache, x, ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        li.li_append_paged(ctx, pool.cache, x, ws)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert pool.cache.lengths.tolist() == [8, 11]
    flat = pool.cache.data.view(-1, 64)
    assert torch.equal(flat[0:8], x[0].repeat(4, 1)) and torch.equal(flat[64 + 3:64 + 11], x[1].repeat(4, 1))


# ------------------------------------------------------------------ latent attention

def check_attention(out, lse, ref, d, n, dt, what):
    """ref = attend()'s four results for H heads; d terms a score, n keys."""
    o, l, pv, zabs = ref
    dz = (d * 2.0 ** -23 * zabs + 2.0 ** -20)[:, None]
    h = half(dt)
    weights = (half(BF) if dt == BF else 0.0) + 2 * dz + (n + 64) * 2.0 ** -24 + 2.0 ** -20
    close(out, o, h * np.abs(o) + weights * pv * (1 + h) + 1e-30, what + " out")
    if lse is not None:
        close(lse, l, dz[:, 0] + (n + 64) * 2.0 ** -24 + 2.0 ** -22 * np.where(np.isfinite(l), np.abs(l), 0) + 2.0 ** -20, what + " lse")


def run_latent(ctx, pool, q, d_v, scale, sel=None, q_pos=None, ws=None, stream=None):
    b, T, H, _ = q.shape
    ws = li.attention_workspace(ctx, H, d_v) if ws is None else ws
    out = torch.full((b, T, H, d_v), float("nan"), dtype=q.dtype, device=DEV)
    lse = torch.full((b, T, H), float("nan"), device=DEV)
    li.li_latent_attention(ctx, pool.cache, q, d_v, scale, out, ws, lse=lse, sel=sel, q_pos=q_pos, stream=stream)
    return out, lse, ws


def check_latent(pool, lens, q, d_v, scale, out, lse, sel=None, q_pos=None):
    b, T, H, dim = q.shape
    for i in range(b):
        for t in range(T):
            n = lens[i] if q_pos is None else min(lens[i], int(q_pos[i, t]) + 1)
            at = np.arange(max(n, 0))
            if sel is not None:
                s = sel[i, t].cpu().numpy()
                at = s[(s >= 0) & (s < n)]
            c = pool.rows(i, at)
            check_attention(out[i, t], lse[i, t], A.attend(f64(q[i, t]), c, c[:, :d_v], scale), dim, len(at), q.dtype, f"row {i},{t}")


LA = [  # lens, T, H, dim, d_v, page
    ([0], 1, 1, 576, 512, 64), ([1], 1, 16, 576, 512, 64), ([127, 128, 129], 1, 64, 576, 512, 64),
    ([300, 0, 700], 1, 128, 576, 512, 16), ([515], 1, 20, 192, 128, 1), ([60, 260], 3, 8, 256, 256, 17),
    ([1000], 1, 65, 320, 256, 64), ([200, 33], 5, 16, 96, 64, 8), ([150], 2, 3, 48, 32, 5), ([140], 1, 40, 64, 64, 32),
    ([2500], 1, 32, 576, 512, 128), ([400], 1, 130, 64, 8, 3), ([333], 1, 9, 128, 120, 4), ([260], 1, 64, 512, 512, 64),
    ([200], 1, 16, 8, 8, 64), ([385], 1, 33, 200, 136, 64),
]


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", LA, ids=[f"n{max(c[0])}b{len(c[0])}t{c[1]}h{c[2]}d{c[3]}v{c[4]}p{c[5]}" for c in LA])
def test_latent_attention_dense(ctx, case, dt):
    lens, T, H, dim, d_v, page = case
    pool = Pool(lens, max(max(lens), 1), page, dim, dt, seed=1)
    q = rand(len(lens), T, H, dim, dtype=dt, seed=2, scale=2.0).to(DEV)
    out, lse, ws = run_latent(ctx, pool, q, d_v, dim ** -0.5)
    assert li.li_device_status(ctx, ws) == "LI_OK"
    check_latent(pool, lens, q, d_v, dim ** -0.5, out, lse)
    # causal: the T queries are the last T positions, some before the start
    q_pos = torch.tensor([[n - T + t for t in range(T)] for n in lens], dtype=torch.int32, device=DEV)
    out, lse, ws = run_latent(ctx, pool, q, d_v, dim ** -0.5, q_pos=q_pos, ws=ws)
    check_latent(pool, lens, q, d_v, dim ** -0.5, out, lse, q_pos=q_pos)


def selection(lens, T, k, seed, q_pos=None):
    g = np.random.default_rng(seed)
    sel = np.full((len(lens), T, k), -1, np.int32)
    for b, n in enumerate(lens):
        for t in range(T):
            m = n if q_pos is None else max(min(n, int(q_pos[b, t]) + 1), 0)
            s = np.sort(g.permutation(m)[:k])
            sel[b, t, :len(s)] = s
    return torch.from_numpy(sel).to(DEV)


LS = [  # lens, T, H, dim, d_v, page, k
    ([8192], 1, 64, 576, 512, 64, 2048), ([300, 5, 0], 1, 16, 576, 512, 16, 64), ([1000, 2000], 3, 32, 576, 512, 64, 300),
    ([700], 1, 128, 192, 128, 1, 129), ([64], 2, 8, 96, 64, 17, 1), ([5000], 4, 3, 48, 32, 64, 640), ([900], 1, 1, 576, 512, 64, 128),
]


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", LS, ids=[f"n{max(c[0])}b{len(c[0])}t{c[1]}h{c[2]}d{c[3]}k{c[6]}" for c in LS])
def test_latent_attention_selected(ctx, case, dt):
    lens, T, H, dim, d_v, page, k = case
    pool = Pool(lens, max(lens), page, dim, dt, seed=5)
    q = rand(len(lens), T, H, dim, dtype=dt, seed=6, scale=2.0).to(DEV)
    sel = selection(lens, T, k, 7)
    out, lse, ws = run_latent(ctx, pool, q, d_v, dim ** -0.5, sel=sel)
    assert li.li_device_status(ctx, ws) == "LI_OK"
    check_latent(pool, lens, q, d_v, dim ** -0.5, out, lse, sel=sel)
    # any order, holes, one position twice; q_pos hides some
    g = torch.Generator().manual_seed(8)
    sel = sel[..., torch.randperm(k, generator=g).to(DEV)].contiguous()
    sel[..., -1] = sel[..., 0]
    q_pos = torch.tensor([[n - T + t for t in range(T)] for n in lens], dtype=torch.int32, device=DEV)
    sel = torch.where(sel <= q_pos[..., None], sel, -3).contiguous()
    out, lse, ws = run_latent(ctx, pool, q, d_v, dim ** -0.5, sel=sel, q_pos=q_pos, ws=ws)
    assert li.li_device_status(ctx, ws) == "LI_OK"
    check_latent(pool, lens, q, d_v, dim ** -0.5, out, lse, sel=sel, q_pos=q_pos)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_latent_attention_skips_and_reports_bad_entries(ctx, dt):
    lens, H, dim, d_v = [300, 200], 16, 192, 128
    pool = Pool(lens, 300, 16, dim, dt)
    q = rand(2, 1, H, dim, dtype=dt, seed=1).to(DEV)
    sel = selection(lens, 1, 150, 2)
    good = sel.clone()
    sel[0, 0, 140], sel[1, 0, 3] = 300, 2 ** 31 - 1       # past the prefix
    good[0, 0, 140], good[1, 0, 3] = -1, -1
    out, lse, ws = run_latent(ctx, pool, q, d_v, 0.1, sel=sel)
    assert li.li_device_status(ctx, ws) == "LI_ERR_INDEX"
    check_latent(pool, lens, q, d_v, 0.1, out, lse, sel=good)
    # pages outside the pool: their positions are skipped
    for bad in (pool.n_pages, -1, 2 ** 31 - 1):
        table = pool.table_cpu.clone()
        table[0, 3] = bad
        pool.cache.page_table.copy_(table)
        out, lse, ws = run_latent(ctx, pool, q, d_v, 0.1, ws=ws)
        assert li.li_device_status(ctx, ws) == "LI_ERR_INDEX"
        keep = torch.arange(300)
        keep = torch.where((keep >= 48) & (keep < 64), -1, keep).to(torch.int32)
        sel = torch.stack([keep, torch.where(keep < 0, 48 + torch.arange(300) % 16, keep).to(torch.int32)])[:, None].contiguous()
        sel[1, 0, :] = torch.arange(300, dtype=torch.int32)
        check_latent(pool, lens, q, d_v, 0.1, out, lse, sel=torch.where(sel < torch.tensor(lens)[:, None, None], sel, -1))


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_latent_attention_large_and_lopsided_scores(ctx, dt):
    """Scores far apart, late maxima, all equal, and lengths that are clamped."""
    lens, H, dim, d_v = [600], 16, 64, 64
    pool = Pool(lens, 600, 64, dim, dt)
    q = rand(1, 1, H, dim, dtype=dt, seed=3, scale=60.0).to(DEV)
    q[0, 0, 0] = 0
    out, lse, ws = run_latent(ctx, pool, q, d_v, 1.0)
    check_latent(pool, lens, q, d_v, 1.0, out, lse)
    out, lse, _ = run_latent(ctx, pool, q, d_v, -1.0, ws=ws)
    check_latent(pool, lens, q, d_v, -1.0, out, lse)
    out, lse, _ = run_latent(ctx, pool, q, d_v, 0.0, ws=ws)
    check_latent(pool, lens, q, d_v, 0.0, out, lse)
    pool.cache.lengths.fill_(-5)
    out, lse, _ = run_latent(ctx, pool, q, d_v, 1.0, ws=ws)
    assert (out == 0).all() and torch.isneginf(lse).all()


def test_latent_attention_long_rows_and_split_order(ctx):
    """A prefix long enough to be split over the GPU: the same answer every time, on another stream and in a graph."""
    lens, H, dim, d_v = [20000, 33, 9000], 64, 576, 512
    pool = Pool(lens, 20000, 64, dim, BF)
    q = rand(3, 1, H, dim, dtype=BF, seed=3, scale=2.0).to(DEV)
    out, lse, ws = run_latent(ctx, pool, q, d_v, dim ** -0.5)
    check_latent(pool, lens, q, d_v, dim ** -0.5, out, lse)
    for _ in range(3):
        again, l2, _ = run_latent(ctx, pool, q, d_v, dim ** -0.5, ws=ws)
        assert torch.equal(again, out) and torch.equal(l2, lse)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again, l2, _ = run_latent(ctx, pool, q, d_v, dim ** -0.5, ws=ws)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(again, out) and torch.equal(l2, lse)
    o3, l3 = torch.zeros_like(out), torch.zeros_like(lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        li.li_latent_attention(ctx, pool.cache, q, d_v, dim ** -0.5, o3, ws, lse=l3)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o3, out) and torch.equal(l3, lse)
    # new lengths and queries in the captured buffers
    pool.cache.lengths.copy_(torch.tensor([700, 33, 0], dtype=torch.int32))
    q.copy_(rand(3, 1, H, dim, dtype=BF, seed=9, scale=2.0))
    g.replay()
    torch.cuda.synchronize()
    check_latent(pool, [700, 33, 0], q, d_v, dim ** -0.5, o3, l3)


def test_latent_attention_many_sequences(ctx):
    lens = [(37 * i) % 200 for i in range(300)]
    pool = Pool(lens, 200, 16, 64, BF)
    q = rand(300, 1, 4, 64, dtype=BF, seed=3, scale=2.0).to(DEV)
    out, lse, _ = run_latent(ctx, pool, q, 32, 0.125)
    check_latent(pool, lens, q, 32, 0.125, out, lse)


# ------------------------------------------------------------------ prompt attention

def check_prompt(q, kn, kr, v, cu_q, cu_k, scale, causal, out, lse):
    H = q.shape[1]
    for b in range(len(cu_q) - 1):
        q0, q1, k0, k1 = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        nq, nk = q1 - q0, k1 - k0
        kk = f64(kn[k0:k1]).transpose(1, 0, 2)
        if kr is not None:
            kk = np.concatenate([kk, np.broadcast_to(f64(kr[k0:k1]), (H,) + tuple(kr[k0:k1].shape))], -1)
        vv = f64(v[k0:k1]).transpose(1, 0, 2)
        qq = f64(q[q0:q1])
        rows = range(nq) if nq <= 40 else sorted(set(list(range(0, nq, max(nq // 23, 1))) + [0, 1, nq - 1, min(127, nq - 1), min(128, nq - 1), min(255, nq - 1), min(256, nq - 1)]))
        for i in rows:
            n = min(max(i + 1 + nk - nq, 0), nk) if causal else nk
            check_attention(out[q0 + i], lse[q0 + i], A.attend(qq[i], kk[:, :n], vv[:, :n], scale), kk.shape[-1], n, q.dtype,
                            f"sequence {b} query {i}")


def run_prompt(ctx, nq, nk, H, dn, dr, dv, dt, causal=True, seed=0, pad=3, check=True, max_q=None):
    tq, tk = sum(nq) + pad, sum(nk) + pad
    q = rand(tq, H, dn + dr, dtype=dt, seed=seed, scale=2.0).to(DEV)
    kv = rand(tk, H, dn + dv, dtype=dt, seed=seed + 1).to(DEV)
    kn, v = kv[..., :dn], kv[..., dn:]
    kr = rand(tk, dr, dtype=dt, seed=seed + 2).to(DEV) if dr else None
    cu_q, cu_k = np.concatenate([[0], np.cumsum(nq)]), np.concatenate([[0], np.cumsum(nk)])
    # keys and values behind the last sequence are nobody's
    kv[cu_k[-1]:] = float("nan")
    if dr:
        kr[cu_k[-1]:] = float("nan")
    i32 = lambda a: torch.tensor(a.tolist(), dtype=torch.int32, device=DEV)  # noqa: E731
    out = torch.full((tq, H, dv), 3.0, dtype=dt, device=DEV)
    lse = torch.full((tq, H), 3.0, device=DEV)
    ws = li.attention_workspace(ctx, H, dv)
    scale = (dn + dr) ** -0.5
    li.li_prompt_attention(ctx, q, kn, kr, v, i32(cu_q), i32(cu_k), max_q or max(max(nq), 1), scale, out, ws, lse=lse, causal=causal)
    assert li.li_device_status(ctx, ws) == "LI_OK"
    assert (out[cu_q[-1]:] == 3).all() and (lse[cu_q[-1]:] == 3).all(), "rows behind the last sequence changed"
    if check:
        check_prompt(q, kn, kr, v, cu_q, cu_k, scale, causal, out, lse)
    return out, lse


PA = [  # nq, nk, H, d_nope, d_rope, d_v, causal
    ([1], [1], 1, 128, 64, 128, True), ([5, 0, 130], [5, 0, 130], 4, 128, 64, 128, True),
    ([257], [257], 2, 128, 64, 128, True), ([256, 1, 128], [256, 1, 128], 3, 64, 32, 64, True),
    ([100, 20], [333, 20], 2, 128, 64, 128, True), ([40, 7], [13, 3], 2, 64, 0, 128, True),   # more queries than keys
    ([70, 300], [129, 40], 2, 128, 0, 64, False), ([3, 9], [0, 500], 2, 128, 64, 128, False),
    ([600], [600], 5, 72, 8, 40, True), ([1, 1, 1, 1], [400, 1, 0, 128], 8, 128, 64, 128, True),
    ([700], [700], 1, 16, 16, 16, True),
]


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", PA, ids=[f"q{max(c[0])}k{max(c[1])}b{len(c[0])}h{c[2]}d{c[3]}r{c[4]}v{c[5]}{'c' if c[6] else 'f'}" for c in PA])
def test_prompt_attention(ctx, case, dt):
    nq, nk, H, dn, dr, dv, causal = case
    run_prompt(ctx, nq, nk, H, dn, dr, dv, dt, causal)


def test_prompt_attention_long(ctx):
    run_prompt(ctx, [1500, 3, 2100], [1500, 700, 2100], 2, 128, 64, 128, BF)


@pytest.mark.parametrize("case", PA, ids=[f"q{max(c[0])}k{max(c[1])}b{len(c[0])}h{c[2]}d{c[3]}r{c[4]}v{c[5]}{'c' if c[6] else 'f'}" for c in PA])
def test_prompt_attention_small_sequences_by_pairs(ctx, case):
    """max_q above every sequence's queries: short sequences by the kernel for long ones."""
    nq, nk, H, dn, dr, dv, causal = case
    run_prompt(ctx, nq, nk, H, dn, dr, dv, BF, causal, pad=2100, max_q=2100)


@pytest.mark.parametrize("n", [2048, 2049, 2561], ids=lambda n: f"n{n}")
def test_prompt_attention_where_the_kernel_changes(ctx, n):
    run_prompt(ctx, [n, 1], [n + 77, 2], 2, 128, 64, 128, BF)


def test_prompt_attention_many_short_sequences(ctx):
    nq = [(7 * i) % 5 for i in range(150)]
    run_prompt(ctx, nq, [n + i % 3 for i, n in enumerate(nq)], 2, 64, 32, 64, BF)
    run_prompt(ctx, nq, [n + i % 3 for i, n in enumerate(nq)], 2, 64, 32, 64, BF, pad=2100, max_q=2100)


def test_prompt_attention_clamps_offsets(ctx):
    """Offsets past the tensors are clamped to them; max_q bounds the rows that are written."""
    q, kn, v = (rand(10, 2, 64, dtype=BF, seed=s).to(DEV) for s in (1, 2, 3))
    out = torch.full((10, 2, 64), 3.0, dtype=BF, device=DEV)
    lse = torch.full((10, 2), 3.0, device=DEV)
    ws = li.attention_workspace(ctx, 2, 64)
    cu = torch.tensor([0, 4, 1000], dtype=torch.int32, device=DEV)
    li.li_prompt_attention(ctx, q, kn, None, v, cu, cu, 10, 0.125, out, ws, lse=lse)
    check_prompt(q, kn, None, v, [0, 4, 10], [0, 4, 10], 0.125, True, out, lse)
    out.fill_(3.0)
    li.li_prompt_attention(ctx, q, kn, None, v, cu, cu, 4, 0.125, out, ws, lse=lse)
    assert (out[8:] == 3).all() and (out[:8] != 3).any()


def test_prompt_attention_in_a_graph(ctx):
    a, la = run_prompt(ctx, [300, 20], [300, 20], 4, 128, 64, 128, BF, check=False)
    q = rand(323, 4, 192, dtype=BF, seed=0, scale=2.0).to(DEV)
    kv = rand(323, 4, 256, dtype=BF, seed=1).to(DEV)
    kr = rand(323, 64, dtype=BF, seed=2).to(DEV)
    cu = torch.tensor([0, 300, 320], dtype=torch.int32, device=DEV)
    out, lse = torch.zeros_like(a), torch.zeros_like(la)
    ws = li.attention_workspace(ctx, 4, 128)
    args = (q, kv[..., :128], kr, kv[..., 128:], cu, cu, 300, 192 ** -0.5, out, ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        li.li_prompt_attention(ctx, *args, lse=lse)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[:320], a[:320]) and torch.equal(lse[:320], la[:320])


# ------------------------------------------------------------------ refusals

def refused(status, fn, *a, **kw):
    with pytest.raises(li.LiError) as e:
        fn(*a, **kw)
    assert e.value.name == status, str(e.value)


def refusals(ctx, dev, stream):
    """Every call here is turned down on the host: nothing is launched."""
    z = lambda *s, dtype=BF: torch.zeros(*s, dtype=dtype, device=dev)  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev)  # noqa: E731
    ws = z(4096, dtype=torch.uint8)
    ws_big = z(li.li_attention_workspace_bytes(ctx, 8, 512), dtype=torch.uint8)
    assert li.li_attention_workspace_bytes(ctx, 0, 1) == 0 and li.li_attention_workspace_bytes(None, 1, 1) == 0
    tf = lambda **k: li.RowTransform(**k)  # noqa: E731
    f = z(32, dtype=F32)
    nr = lambda x, t, o=None, pos=i(2): li.li_norm_rope(ctx, [li.HeadRows(x, t, x if o is None else o)], pos, stream=stream)  # noqa: E731
    x = z(2, 3, 64)
    refused("LI_ERR_ARG", li.li_norm_rope, ctx, [], i(2), stream=stream)
    refused("LI_ERR_DTYPE", li.HeadRows, z(2, 3, 64, dtype=torch.float16), tf(), z(2, 3, 64, dtype=torch.float16))
    refused("LI_ERR_SHAPE", nr, x, tf(norm="rms", norm_offset=1, norm_dim=64))
    refused("LI_ERR_SHAPE", nr, x, tf(norm="rms"))
    refused("LI_ERR_ARG", nr, x, tf(norm="rms", norm_dim=64, eps=float("nan")))
    refused("LI_ERR_ARG", tf, norm="batch", norm_dim=64)
    refused("LI_ERR_SHAPE", nr, x, tf(rope_dim=63, inv_freq=z(31, dtype=F32)))
    refused("LI_ERR_SHAPE", tf, rope_dim=64, inv_freq=z(31, dtype=F32))
    refused("LI_ERR_SHAPE", nr, x, tf(rope_offset=2, rope_dim=64, inv_freq=f))
    refused("LI_ERR_ARG", nr, x, tf(rope_dim=64))
    refused("LI_ERR_ARG", nr, x, tf(rope_dim=64, inv_freq=f), None, None)
    refused("LI_ERR_SHAPE", nr, z(2, 1, 1025), tf())
    refused("LI_ERR_SHAPE", li.HeadRows, x, tf(), z(2, 3, 32))
    cache = lambda d=z(4, 8, 64), t=i(2, 2), n=i(2): li.PagedCache(d, t, n)  # noqa: E731
    ap = lambda c, x, w=ws, **k: li.li_append_paged(ctx, c, x, w, stream=stream, **k)  # noqa: E731
    refused("LI_ERR_SHAPE", ap, cache(), z(2, 0, 64))
    refused("LI_ERR_SHAPE", ap, cache(), z(3, 1, 64))
    refused("LI_ERR_DTYPE", ap, cache(), z(2, 1, 64, dtype=F32))
    refused("LI_ERR_SHAPE", ap, cache(z(4, 8, 4), i(2, 2)), z(2, 1, 4))
    refused("LI_ERR_SHAPE", ap, cache(z(4, 8, 1032), i(2, 2)), z(2, 1, 1032))
    refused("LI_ERR_SHAPE", ap, cache(), z(2, 1, 64), n_new=i(3))
    refused("LI_ERR_WORKSPACE", ap, cache(), z(2, 1, 64), ws[:128])
    refused("LI_ERR_WORKSPACE", ap, cache(), z(2, 1, 64), ws[16:])
    refused("LI_ERR_ARG", ap, cache(), z(3, 2, 64)[::2])
    refused("LI_ERR_ALIGN", ap, cache(), z(2, 1, 68)[..., 1:65])
    la = lambda c, q, d_v=32, scale=1.0, out=None, w=ws_big, **k: li.li_latent_attention(  # noqa: E731
        ctx, c, q, d_v, scale, z(*q.shape[:3], d_v) if out is None else out, w, stream=stream, **k)
    q = z(2, 1, 4, 64)
    refused("LI_ERR_SHAPE", la, cache(), z(2, 1, 4, 32))
    refused("LI_ERR_SHAPE", la, cache(), q, 65)
    refused("LI_ERR_SHAPE", la, cache(), q, 0)
    refused("LI_ERR_SHAPE", la, cache(z(4, 8, 584), i(2, 2)), z(2, 1, 4, 584))
    refused("LI_ERR_SHAPE", la, cache(), z(2, 0, 4, 64))
    refused("LI_ERR_SHAPE", la, cache(), q, sel=i(2, 1, 0))
    refused("LI_ERR_SHAPE", la, cache(), q, sel=i(2, 2, 8))
    refused("LI_ERR_ARG", la, cache(), q, 32, float("inf"))
    refused("LI_ERR_DTYPE", la, cache(), q, out=z(2, 1, 4, 32, dtype=F32))
    refused("LI_ERR_DTYPE", cache, z(4, 8, 64, dtype=torch.uint8))
    refused("LI_ERR_SHAPE", cache, z(4, 8, 64), i(2, 2), i(3))
    refused("LI_ERR_ARG", la, cache(), z(2, 1, 4, 128)[..., :64])
    refused("LI_ERR_WORKSPACE", la, cache(), q, w=ws_big[:128])
    pa = lambda q, kn, kr, v, cq=i(3), ck=i(3), out=None, w=ws_big, scale=1.0, m=4: li.li_prompt_attention(  # noqa: E731
        ctx, q, kn, kr, v, cq, ck, m, scale, z(*q.shape[:2], v.shape[-1]) if out is None else out, w, stream=stream)
    q, kn, kr, v = z(5, 2, 96), z(6, 2, 64), z(6, 32), z(6, 2, 64)
    refused("LI_ERR_SHAPE", pa, q, kn, None, v)
    refused("LI_ERR_SHAPE", pa, q, kn, kr[:5], v)
    refused("LI_ERR_SHAPE", pa, z(5, 2, 136), z(6, 2, 136), None, v)
    refused("LI_ERR_SHAPE", pa, z(5, 2, 60), z(6, 2, 60), None, v)
    refused("LI_ERR_SHAPE", pa, z(5, 2, 64), kn, None, z(6, 2, 136))
    refused("LI_ERR_SHAPE", pa, q, kn, kr, v, m=-1)
    refused("LI_ERR_ARG", pa, q, kn, kr, v, scale=float("nan"))
    refused("LI_ERR_ALIGN", pa, z(5, 2, 100)[..., 2:98], kn, kr, v)
    refused("LI_ERR_WORKSPACE", pa, q, kn, kr, v, w=ws_big[16:])
    refused("LI_ERR_DTYPE", pa, q, kn, kr, v.float())


def test_refusals(ctx):
    refusals(ctx, DEV, None)


# ------------------------------------------------------------------ the run of them together

def test_decode_step_with_selection_and_attention(ctx):
    """One layer's decode step as a serving program makes it: norms and rotation of the heads, the new latent into the
    paged cache, the indexer's selection, and the attention over the selected tokens."""
    b, n, H, d_c, d_r, k, page = 2, 700, 16, 512, 64, 128, 64
    dim = d_c + d_r
    pool = Pool([n, 0], n + 8, page, dim, BF, seed=11)
    pool.table_cpu = torch.arange(pool.table_cpu.numel(), dtype=torch.int32).view(pool.table_cpu.shape)
    pool.cache.page_table.copy_(pool.table_cpu)
    pool.cache.lengths.zero_()
    ws = li.attention_workspace(ctx, H, d_c)
    tf = make_tf(dim, "rms", d_r, False, 1, ndim=d_c)
    kv = rand(b, n, dim, dtype=BF, seed=1).to(DEV)
    li.li_append_paged(ctx, pool.cache, kv, ws, tf=tf, n_new=torch.tensor([n, 300], dtype=torch.int32, device=DEV))
    new = rand(b, 1, dim, dtype=BF, seed=2).to(DEV)
    li.li_append_paged(ctx, pool.cache, new, ws, tf=tf)
    lens = [n + 1, 301]
    assert pool.cache.lengths.tolist() == lens
    # rotated queries: [q_nope absorbed, q_rope]
    q = rand(b, H, dim, dtype=BF, seed=3, scale=2.0).to(DEV)
    pos = torch.tensor([n, 300], dtype=torch.int32, device=DEV)
    qtf = li.RowTransform(rope_offset=d_c, rope_dim=d_r, inv_freq=tf.inv_freq)
    li.li_norm_rope(ctx, [li.HeadRows(q, qtf, q)], pos)
    # the indexer selects on its own latent
    G = li.GroupIndexer(ctx, batch=b, capacity=1024, d_c=192, H=8, d_k=64, G=1, k=k)
    G.load(lens, [rand(64, 192, seed=4) / 14], [rand(b, 1, 8, 64, seed=5)], [rand(b, 1, 8, seed=6)], latent=rand(b, 1024, 192, seed=7))
    G.score_topk(0)
    out = torch.empty(b, 1, H, d_c, dtype=BF, device=DEV)
    lse = torch.empty(b, 1, H, device=DEV)
    G.attend(0, pool.cache, q[:, None].contiguous(), d_c, dim ** -0.5, out, lse=lse)
    torch.cuda.synchronize()
    assert li.li_device_status(ctx, G.ws_attn) == "LI_OK"
    pool.data_cpu = pool.cache.data.cpu()
    sel = G.idx[0]
    assert (sel >= 0).sum() == 2 * k
    check_latent(pool, lens, q[:, None], d_c, dim ** -0.5, out, lse, sel=sel)


def test_prompt_then_decode_agree(ctx):
    """The expanded form over a prompt and the absorbed form over the cached latent give the same answer for its last token."""
    n, H, d_c, dn, dr, dv = 150, 8, 128, 64, 32, 64
    c, kr = rand(n, d_c, dtype=BF, seed=1).to(DEV), rand(n, dr, dtype=BF, seed=2).to(DEV)
    W_K, W_V = (rand(H, d, d_c, seed=s, scale=d_c ** -0.5).to(DEV) for d, s in ((dn, 3), (dv, 4)))
    q = rand(n, H, dn + dr, dtype=BF, seed=5, scale=2.0).to(DEV)
    kn, v = (torch.einsum("nc,hdc->nhd", c.float(), W).to(BF) for W in (W_K, W_V))
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    out = torch.empty(n, H, dv, dtype=BF, device=DEV)
    ws = li.attention_workspace(ctx, H, d_c)
    scale = (dn + dr) ** -0.5
    li.li_prompt_attention(ctx, q, kn, kr, v, cu, cu, n, scale, out, ws)
    pool = Pool([0], n, 16, d_c + dr, BF)
    pool.cache.page_table.copy_(torch.arange(pool.table_cpu.numel(), dtype=torch.int32).view(1, -1))
    li.li_append_paged(ctx, pool.cache, torch.cat([c, kr], -1)[None].contiguous(), ws)
    qa = torch.cat([torch.einsum("hd,hdc->hc", q[-1, :, :dn].float(), W_K).to(BF), q[-1, :, dn:]], -1)
    o = torch.empty(1, 1, H, d_c, dtype=BF, device=DEV)
    li.li_latent_attention(ctx, pool.cache, qa[None, None].contiguous(), d_c, scale, o, ws)
    got = torch.einsum("hc,hdc->hd", o[0, 0].float(), W_V)
    # both sides round keys, queries and weights to bf16: scores differ by sqrt(dn + d_c) of 2^-8 times a term of size 2
    torch.testing.assert_close(got, out[-1].float(), rtol=0.1, atol=0.1)
