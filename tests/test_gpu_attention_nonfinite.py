"""Attention where a query is not finite, in every kernel.

A query whose scores hold a NaN, or +inf, has no softmax: out and lse are NaN, for that query and head alone.  One
whose scores are all -inf gives its keys no weight: out = 0 and lse = -inf = log(sum exp z), as one that attends
nothing, which stays so whatever it holds."""
import numpy as np
import pytest
import torch

import cross_layer_latent_b200 as li
from oracle import attention as A
from tests.test_gpu_attention import BF, DEV, F32, Pool, check_attention, f64, rand, run_latent, selection

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def ctx():
    c = li.Context(0)
    yield c
    c.close()


# what is put into element 0 of the queries of heads 0 .. 3; the keys' element 0 is positive
MARKS = (NAN, INF, -INF, -INF)


def expect(out, lse, head, attends, what):
    """Results of the marked heads; head 3 has a key whose element 0 is zero among the attended, so a NaN score."""
    if not attends or head == 2:
        assert (out == 0).all() and torch.isneginf(lse), f"{what} head {head}: {out[:4]} {lse}"
    else:
        assert torch.isnan(out).all() and torch.isnan(lse), f"{what} head {head}: {out[:4]} {lse}"


LATENT = [  # lens, T, H, dim, d_v, page, k
    ([300, 0, 1], 1, 16, 576, 512, 64, 0), ([20000, 70], 1, 64, 576, 512, 64, 0), ([130], 3, 8, 96, 64, 16, 0),
    ([400, 30], 2, 8, 96, 64, 16, 70), ([9000], 1, 64, 576, 512, 64, 2048),
]


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", LATENT, ids=[f"n{max(c[0])}t{c[1]}h{c[2]}k{c[6]}" for c in LATENT])
def test_latent_attention_of_queries_that_are_not_finite(ctx, case, dt):
    lens, T, H, dim, d_v, page, k = case
    pool = Pool(lens, max(lens), page, dim, dt, seed=1)
    # element 0 positive, but zero at position 0 for head 3 alone: a second element takes its place there
    pool.data_cpu[..., 0] = pool.data_cpu[..., 0].abs() + 0.5
    pool.data_cpu[..., 1] = pool.data_cpu[..., 1].abs() + 0.5
    for b, n in enumerate(lens):
        if n:
            pool.data_cpu.view(-1, dim)[A.page_rows(pool.table_cpu[b], [0], page)[0], 1] = 0.0
    pool.cache.data.copy_(pool.data_cpu)
    q = rand(len(lens), T, H, dim, dtype=dt, seed=2, scale=2.0)
    for h, x in enumerate(MARKS):
        q[:, T - 1, h, 1 if h == 3 else 0] = x
    sel = None
    if k:
        sel = selection(lens, T, k, 3)
        sel[..., 0] = 0                          # position 0 among the selected
        sel[..., 1:] = torch.where(sel[..., 1:] == 0, -1, sel[..., 1:])
    out, lse, ws = run_latent(ctx, pool, q.to(DEV), d_v, dim ** -0.5, sel=sel)
    assert li.li_device_status(ctx, ws) == "LI_OK"
    for b, n in enumerate(lens):
        for t in range(T):
            at = np.arange(n) if sel is None else sel[b, t][sel[b, t] >= 0].cpu().numpy()
            c = pool.rows(b, at)
            marked = len(MARKS) if t == T - 1 else 0
            for h in range(marked):
                expect(out[b, t, h], lse[b, t, h], h, len(at), f"row {b},{t}")
            check_attention(out[b, t, marked:], lse[b, t, marked:], A.attend(f64(q[b, t, marked:]), c, c[:, :d_v], dim ** -0.5), dim,
                            len(at), dt, f"row {b},{t}")


PROMPT = [  # nq, nk, causal
    ([300, 5, 4], [300, 40, 0], True), ([130, 1], [7, 600], False), ([270, 30], [20, 33], True),
]


@pytest.mark.parametrize("kernel", ["single", "pair", "f32"])
@pytest.mark.parametrize("case", PROMPT, ids=[f"q{max(c[0])}k{max(c[1])}{'c' if c[2] else 'f'}" for c in PROMPT])
@pytest.mark.parametrize("zero_key", [0, 6])
def test_prompt_attention_of_queries_that_are_not_finite(ctx, case, kernel, zero_key):
    nq, nk, causal = case
    H, dn, dr, dv = 6, 64, 32, 64
    dt = F32 if kernel == "f32" else BF
    tq, tk = sum(nq), sum(nk)
    pad = 2100 if kernel == "pair" else 0        # max_q above 2048 takes the kernel for long prompts
    q = rand(tq + pad, H, dn + dr, dtype=dt, seed=1, scale=2.0)
    kn, v, kr = (rand(tk, *s, dtype=dt, seed=4 + i) for i, s in enumerate(((H, dn), (H, dv), (dr,))))
    kn[..., 0] = kn[..., 0].abs() + 0.5
    kn[:, 4, 0] *= -1                            # head 4: one key with a score of +inf among ones of -inf
    cu_q, cu_k = np.concatenate([[0], np.cumsum(nq)]), np.concatenate([[0], np.cumsum(nk)])
    for b, n in enumerate(nk):
        if n > zero_key:
            kn[cu_k[b] + zero_key, 3, 0] = 0.0
            kn[cu_k[b] + zero_key, 4, 0] = 1.0
    at_q = [int(cu_q[b]) + i for b, n in enumerate(nq) for i in {0, n // 2, n - 1}]
    for i in at_q:
        for h, x in enumerate(MARKS + (INF,)):
            q[i, h, 0] = x
    i32 = lambda a: torch.tensor(a.tolist(), dtype=torch.int32, device=DEV)  # noqa: E731
    out = torch.full((tq + pad, H, dv), 3.0, dtype=dt, device=DEV)
    lse = torch.full((tq + pad, H), 3.0, device=DEV)
    ws = li.attention_workspace(ctx, H, dv)
    scale = (dn + dr) ** -0.5
    li.li_prompt_attention(ctx, q.to(DEV), kn.to(DEV), kr.to(DEV), v.to(DEV), i32(cu_q), i32(cu_k), 2100 if pad else max(nq), scale,
                           out, ws, lse=lse, causal=causal)
    assert li.li_device_status(ctx, ws) == "LI_OK"
    assert (out[tq:] == 3).all() and (lse[tq:] == 3).all()
    for b in range(len(nq)):
        ks = np.concatenate([f64(kn[cu_k[b]:cu_k[b + 1]]).transpose(1, 0, 2),
                             np.broadcast_to(f64(kr[cu_k[b]:cu_k[b + 1]]), (H, nk[b], dr))], -1)
        vs = f64(v[cu_k[b]:cu_k[b + 1]]).transpose(1, 0, 2)
        for i in sorted({0, 1, nq[b] // 2, nq[b] - 2, nq[b] - 1} & set(range(nq[b]))):
            n = min(max(i + 1 + nk[b] - nq[b], 0), nk[b]) if causal else nk[b]
            r = int(cu_q[b]) + i
            marked = len(MARKS) + 1 if r in at_q else 0
            for h in range(marked):
                # heads 3 and 4 without their own key among the attended: all scores are -inf
                kind = 2 if h >= 3 and n <= zero_key else h
                expect(out[r, h], lse[r, h], kind, n, f"sequence {b} query {i}")
            check_attention(out[r, marked:], lse[r, marked:], A.attend(f64(q[r, marked:]), ks[marked:, :n], vs[marked:, :n], scale), dn + dr,
                            n, dt, f"sequence {b} query {i}")
