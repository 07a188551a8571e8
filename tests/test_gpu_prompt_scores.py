"""Prompt attention where the kept maximum moves after the first tile of keys, by tens and by little, up and down the
sequence, with a positive, a negative and no scale; both bf16 kernels and fp32."""
import numpy as np
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


# score of key j of n, in units of the query's own factor
RAMPS = {
    "up": lambda j, n: j / 8, "down": lambda j, n: (n - j) / 8, "steps": lambda j, n: j // 128 * 7.0,
    "peaks": lambda j, n: np.where(j % 150 == 149, 3.0 * (j // 150), -20.0), "low": lambda j, n: -300.0 + j / 16,
}


@pytest.mark.parametrize("kernel", ["single", "pair", "f32"])
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("scale", [1.0, -1.0, 0.0])
@pytest.mark.parametrize("ramp", list(RAMPS))
def test_prompt_attention_moves_its_maximum(ctx, ramp, scale, causal, kernel):
    nq, nk, H, dn, dr, dv = [290, 3], [700, 390], 3, 64, 32, 64
    dt = F32 if kernel == "f32" else BF
    pad = 2100 if kernel == "pair" else 2        # max_q above 2048 takes the kernel for long prompts
    cu_q, cu_k = np.concatenate([[0], np.cumsum(nq)]), np.concatenate([[0], np.cumsum(nk)])
    q = rand(sum(nq) + pad, H, dn + dr, seed=1, scale=0.3)
    kn, v, kr = (rand(sum(nk), *s, seed=4 + i, scale=0.3) for i, s in enumerate(((H, dn), (H, dv), (dr,))))
    # heads 0, 1 and 2 see the ramp by factors of 1, 1/2 and, the other way round, -1
    q[..., 0] = torch.tensor([1.0, 0.5, -1.0])
    for b, n in enumerate(nk):
        kn[cu_k[b]:cu_k[b + 1], :, 0] = torch.from_numpy(RAMPS[ramp](np.arange(n), n)).float()[:, None]
    q, kn, v, kr = (t.to(dt).to(DEV) for t in (q, kn, v, kr))
    i32 = lambda a: torch.tensor(a.tolist(), dtype=torch.int32, device=DEV)  # noqa: E731
    out = torch.full((q.shape[0], H, dv), 3.0, dtype=dt, device=DEV)
    lse = torch.full((q.shape[0], H), 3.0, device=DEV)
    ws = li.attention_workspace(ctx, H, dv)
    li.li_prompt_attention(ctx, q, kn, kr, v, i32(cu_q), i32(cu_k), 2100 if kernel == "pair" else max(nq), scale, out, ws, lse=lse,
                           causal=causal)
    assert li.li_device_status(ctx, ws) == "LI_OK"
    check_prompt(q, kn, kr, v, cu_q, cu_k, scale, causal, out, lse)
    assert (out[sum(nq):] == 3).all() and (lse[sum(nq):] == 3).all()
