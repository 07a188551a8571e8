"""Prompt attention over many units that take next to no time: sequences without keys, whose units do no work but their
zeros, between ones with a few, in the kernel of pairs of CTAs.  Every CTA reads a unit's record, and the records have
two places, so a reader that is not waited for would see a later unit."""
import pytest
import torch

import cross_layer_latent_b200 as li
from tests.test_gpu_attention import BF, DEV, check_attention, f64, rand
from oracle import attention as A

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("every", [0, 7, 2], ids=["no keys", "some keys", "half of them with keys"])
def test_units_without_keys(every):
    ctx = li.Context(0)
    try:
        n_seq, H, d = 1500, 16, 64
        nq = [1 + (37 * i) % 3 for i in range(n_seq)]
        nk = [(i % 5 + 1) if every and i % every == 0 else 0 for i in range(n_seq)]
        cu_q, cu_k = ([0] + torch.tensor(n).cumsum(0).tolist() for n in (nq, nk))
        tq, tk = cu_q[-1], max(cu_k[-1], 1)
        q, k, v = rand(tq, H, d, dtype=BF, seed=1).to(DEV), rand(tk, H, d, dtype=BF, seed=2).to(DEV), rand(tk, H, d, dtype=BF, seed=3).to(DEV)
        i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
        out, lse = torch.empty(tq, H, d, dtype=BF, device=DEV), torch.empty(tq, H, device=DEV)
        ws = li.attention_workspace(ctx, H, d)
        first = None
        for _ in range(20):
            out.fill_(3.0)
            lse.fill_(3.0)
            li.li_prompt_attention(ctx, q, k, None, v, i32(cu_q), i32(cu_k), 2100, 0.125, out, ws, lse=lse, causal=False)
            assert li.li_device_status(ctx, ws) == "LI_OK"
            if first is None:
                first = out.clone(), lse.clone()
            assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
        for b in range(n_seq):
            rows = slice(cu_q[b], cu_q[b + 1])
            if nk[b] == 0:
                assert (out[rows] == 0).all() and torch.isneginf(lse[rows]).all(), b
            elif b % 29 == 0:
                kk, vv = (f64(t[cu_k[b]:cu_k[b + 1]]).transpose(1, 0, 2) for t in (k, v))
                for r in range(cu_q[b], cu_q[b + 1]):
                    check_attention(out[r], lse[r], A.attend(f64(q[r]), kk, vv, 0.125), d, nk[b], BF, f"sequence {b}")
        assert every == 0 or (lse > -1e30).any()
    finally:
        ctx.close()
