"""Plain fp64 attention over latents and the row transforms around it, from the
usual definitions (test infrastructure; no code shared with the GPU path)."""
import numpy as np


def norm(x, kind, gamma=None, beta=None, eps=0.0):
    """RMS or layer norm of the last axis."""
    x = np.asarray(x, np.float64)
    if kind == "none":
        return x
    if kind == "layer":
        x = x - x.mean(-1, keepdims=True)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return y * (1.0 if gamma is None else np.asarray(gamma, np.float64)) + (0.0 if beta is None else np.asarray(beta, np.float64))


def rotate(x, pos, inv_freq, halves):
    """Rotary slots of the last axis, turned by pos * inv_freq (pos broadcasts over the leading axes)."""
    x = np.asarray(x, np.float64)
    half = x.shape[-1] // 2
    a, b = (x[..., :half], x[..., half:]) if halves else (x[..., 0::2], x[..., 1::2])
    z = (a + 1j * b) * np.exp(1j * np.asarray(pos, np.float64)[..., None] * np.asarray(inv_freq, np.float64))
    out = np.empty_like(x)
    if halves:
        out[..., :half], out[..., half:] = z.real, z.imag
    else:
        out[..., 0::2], out[..., 1::2] = z.real, z.imag
    return out


def transform(x, pos, *, kind="none", norm_offset=0, norm_dim=0, gamma=None, beta=None, eps=0.0, rope_offset=0, rope_dim=0,
              inv_freq=None, halves=False):
    """A row transform: the norm of one range, then the rotation of another."""
    y = np.array(x, np.float64)
    if kind != "none":
        r = slice(norm_offset, norm_offset + norm_dim)
        y[..., r] = norm(y[..., r], kind, gamma, beta, eps)
    if rope_dim:
        r = slice(rope_offset, rope_offset + rope_dim)
        y[..., r] = rotate(y[..., r], pos, inv_freq, halves)
    return y


def attend(q, k, v, scale):
    """q [H, d], k [n, d] or [H, n, d], v likewise -> out [H, d_v], lse [H], and
    sum p |v| and sum |q_i k_i| maximised over keys (the scales of the
    rounding errors)."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    H, n = q.shape[0], k.shape[-2]
    if n == 0:
        z = np.zeros((H, v.shape[-1]))
        return z, np.full(H, -np.inf), z, np.zeros(H)
    kk = k if k.ndim == 3 else k[None]
    vv = v if v.ndim == 3 else v[None]
    z = scale * (kk @ q[:, :, None])[..., 0]
    m = z.max(-1, keepdims=True)
    p = np.exp(z - m)
    l = p.sum(-1, keepdims=True)
    p = (p / l)[:, None]
    zabs = abs(scale) * (np.abs(kk) @ np.abs(q)[:, :, None])[..., 0].max(-1)
    return (p @ vv)[:, 0], (m + np.log(l))[:, 0], (p @ np.abs(vv))[:, 0], zabs


def page_rows(page_table_row, positions, page_size):
    """Pool row of each position of one sequence."""
    positions = np.asarray(positions, np.int64)
    return np.asarray(page_table_row, np.int64)[positions // page_size] * page_size + positions % page_size
