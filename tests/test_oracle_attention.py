"""The attention oracle against other forms of the same definitions (CPU)."""
import numpy as np
import pytest

from oracle import attention as A

rng = np.random.default_rng(7)


def test_absorbed_form_equals_expanded_form():
    H, n, d_c, d_nope, d_rope, d_v = 3, 11, 16, 8, 4, 6
    c, kr = rng.standard_normal((n, d_c)), rng.standard_normal((n, d_rope))
    W_K, W_V = rng.standard_normal((H, d_nope, d_c)), rng.standard_normal((H, d_v, d_c))
    qn, qr = rng.standard_normal((H, d_nope)), rng.standard_normal((H, d_rope))
    k = np.concatenate([np.einsum("hdc,nc->hnd", W_K, c), np.broadcast_to(kr, (H, n, d_rope))], -1)
    v = np.einsum("hdc,nc->hnd", W_V, c)
    out, lse, _, _ = A.attend(np.concatenate([qn, qr], -1), k, v, 0.3)
    qa = np.concatenate([np.einsum("hdc,hd->hc", W_K, qn), qr], -1)
    o, lse2, _, _ = A.attend(qa, np.concatenate([c, kr], -1), c, 0.3)
    np.testing.assert_allclose(np.einsum("hdc,hc->hd", W_V, o), out, rtol=1e-11)
    np.testing.assert_allclose(lse2, lse, rtol=1e-11)


@pytest.mark.parametrize("halves", [False, True])
def test_rotation_keeps_lengths_and_depends_on_distance_alone(halves):
    f = 10000.0 ** (-np.arange(4) / 4)
    q, k = rng.standard_normal(8), rng.standard_normal(8)
    turn = lambda x, p: A.rotate(x, np.float64(p), f, halves)  # noqa: E731
    assert np.isclose(np.linalg.norm(turn(q, 123456)), np.linalg.norm(q), rtol=1e-12)
    assert np.isclose(turn(q, 1007) @ turn(k, 1000), turn(q, 7) @ turn(k, 0), rtol=1e-9)
    first = turn(np.eye(8)[0], 1)      # slot 0 turns by one radian
    other = 4 if halves else 1
    assert np.isclose(first[0], np.cos(1)) and np.isclose(first[other], np.sin(1))


def test_norms():
    x = rng.standard_normal((5, 12)) + 3
    y = A.norm(x, "rms")
    np.testing.assert_allclose((y * y).mean(-1), 1, rtol=1e-12)
    z = A.norm(x, "layer")
    np.testing.assert_allclose(z.mean(-1), 0, atol=1e-12)
    np.testing.assert_allclose(z.std(-1), 1, rtol=1e-12)


def test_nothing_attended():
    out, lse, _, _ = A.attend(rng.standard_normal((2, 4)), np.zeros((0, 4)), np.zeros((0, 3)), 1.0)
    assert (out == 0).all() and np.isneginf(lse).all()


def test_page_rows():
    assert A.page_rows([5, 2], [0, 2, 3, 5], 3).tolist() == [15, 17, 6, 8]
