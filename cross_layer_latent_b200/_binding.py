"""ctypes binding of libli (include/li.h): argument marshalling only.

Every function here has the name of the C entry point it calls and forwards
device pointers taken from torch tensors; all arithmetic runs in the
library's CUDA kernels.  Importing fails loudly when libli.so is missing:
there is no fallback path.
"""
import ctypes
import os
from dataclasses import dataclass
from typing import List, Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libli.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -m cross_layer_latent_b200.build`")
_lib = ctypes.CDLL(LIB_PATH)

# li_status / li_dtype values (include/li.h)
LI_OK = 0
STATUS_NAMES = {0: "LI_OK", 1: "LI_ERR_ARG", 2: "LI_ERR_SHAPE", 3: "LI_ERR_DTYPE", 4: "LI_ERR_ALIGN",
                5: "LI_ERR_WORKSPACE", 6: "LI_ERR_CAPACITY", 7: "LI_ERR_CUDA",
                8: "LI_ERR_DEVICE_TIMEOUT", 9: "LI_ERR_UNSUPPORTED", 10: "LI_ERR_INDEX"}
STATUS = {v: k for k, v in STATUS_NAMES.items()}
LI_F32, LI_BF16, LI_E4M3 = 0, 1, 2
_DTYPE_CODE = {torch.float32: LI_F32, torch.bfloat16: LI_BF16, torch.float8_e4m3fn: LI_E4M3,
               torch.uint8: LI_E4M3}


class LiError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status
        self.name = STATUS_NAMES.get(status, str(status))


class c_li_cache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("lengths", ctypes.c_void_p),
                ("batch", ctypes.c_int32), ("capacity", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("dtype", ctypes.c_int), ("scale_split", ctypes.c_int32)]


class c_li_latent_transform(ctypes.Structure):
    _fields_ = [("rope_offset", ctypes.c_int32), ("rope_dim", ctypes.c_int32), ("rope_sources", ctypes.c_int32),
                ("inv_freq", ctypes.c_void_p), ("norm_offset", ctypes.c_int32), ("norm_dim", ctypes.c_int32),
                ("norm_gamma", ctypes.c_void_p), ("norm_beta", ctypes.c_void_p), ("norm_eps", ctypes.c_float)]


class c_li_query(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("dtype", ctypes.c_int), ("q_scale", ctypes.c_void_p),
                ("beta", ctypes.c_void_p), ("w", ctypes.c_void_p), ("T", ctypes.c_int32),
                ("H", ctypes.c_int32), ("q_pos", ctypes.c_void_p)]


class c_li_row_transform(ctypes.Structure):
    _fields_ = [("norm", ctypes.c_int), ("norm_offset", ctypes.c_int32), ("norm_dim", ctypes.c_int32),
                ("gamma", ctypes.c_void_p), ("beta", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("rope_offset", ctypes.c_int32), ("rope_dim", ctypes.c_int32), ("rope_halves", ctypes.c_int32),
                ("inv_freq", ctypes.c_void_p)]


class c_li_head_rows(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("out", ctypes.c_void_p), ("H", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("tok_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("out_tok_stride", ctypes.c_int64),
                ("out_head_stride", ctypes.c_int64), ("tf", c_li_row_transform)]


class c_li_paged_cache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("page_table", ctypes.c_void_p), ("lengths", ctypes.c_void_p),
                ("batch", ctypes.c_int32), ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("dim", ctypes.c_int32), ("dtype", ctypes.c_int)]


class c_li_prompt(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k_nope", ctypes.c_void_p), ("k_rope", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("dtype", ctypes.c_int), ("H", ctypes.c_int32), ("d_nope", ctypes.c_int32),
                ("d_rope", ctypes.c_int32), ("d_v", ctypes.c_int32), ("total_q", ctypes.c_int32),
                ("total_k", ctypes.c_int32), ("batch", ctypes.c_int32), ("max_q", ctypes.c_int32),
                ("q_tok_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64), ("k_tok_stride", ctypes.c_int64),
                ("k_head_stride", ctypes.c_int64), ("kr_tok_stride", ctypes.c_int64), ("v_tok_stride", ctypes.c_int64),
                ("v_head_stride", ctypes.c_int64), ("cu_q", ctypes.c_void_p), ("cu_k", ctypes.c_void_p),
                ("scale", ctypes.c_float), ("causal", ctypes.c_int32)]


class c_li_profile_record(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_char * 48), ("ms", ctypes.c_float), ("grid", ctypes.c_int32),
                ("block", ctypes.c_int32), ("smem", ctypes.c_int32)]


_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_sigs = {
    "li_create": (_I, [ctypes.POINTER(_P), _I]),
    "li_destroy": (_I, [_P]),
    "li_last_error": (ctypes.c_char_p, [_P]),
    "li_status_string": (ctypes.c_char_p, [_I]),
    "li_workspace_bytes": (_SZ, [_P, _I, _I, _I, _I, _I, _I]),
    "li_device_status": (_I, [_P, _P, _P, ctypes.POINTER(_I)]),
    "li_set_wait_limit": (_I, [_P, ctypes.c_uint64]),
    "li_append_latent": (_I, [_P, ctypes.POINTER(c_li_cache), _P, _I, _I, _P, _I, _P, _SZ, _P]),
    "li_append_latent_ex": (_I, [_P, ctypes.POINTER(c_li_cache), _P, _I, _I, _P, _I,
                                 ctypes.POINTER(c_li_latent_transform), _P, _SZ, _P]),
    "li_absorb_query_group": (_I, [_P, _P, _I, _I, _I, _I, _I, ctypes.POINTER(_P), _I, _I, _P, _P, _P]),
    "li_absorb_query": (_I, [_P, _P, _I, _I, _I, _I, _P, _I64, _P, _I64, _I, _I, _P, _P, _P, _P]),
    "li_score_topk": (_I, [_P, ctypes.POINTER(c_li_cache), ctypes.POINTER(c_li_query), _I, _P, _P, _P, _P,
                           _SZ, _P]),
    "li_score_topk_static": (_I, [_P, ctypes.POINTER(c_li_cache), ctypes.POINTER(c_li_query), _I, _P, _P, _P,
                                  _P]),
    "li_hs_anchor_candidates": (_I, [_P, ctypes.POINTER(c_li_cache), ctypes.POINTER(c_li_query), _I, _I, _P,
                                     _P, _P, _P, _P, _P, _SZ, _P]),
    "li_hs_follower_refine": (_I, [_P, ctypes.POINTER(c_li_cache), ctypes.POINTER(c_li_query), _P, _P, _I, _I,
                                   _P, _P, _P, _P, _SZ, _P]),
    "li_dsa_score_topk": (_I, [_P, ctypes.POINTER(c_li_cache), ctypes.POINTER(c_li_query), _I, _P, _P, _P, _P,
                               _SZ, _P]),
    "li_topk": (_I, [_P, _P, _I, _I, _I64, _P, _I, _P, _P, _P, _SZ, _P]),
    "li_recall_workspace_bytes": (_SZ, [_P, _I, _I, _I, _I]),
    "li_attention_recall": (_I, [_P, _P, _I, _I, _I, _P, _P, _I, _I, _P, _P, _P, _SZ, _P]),
    "li_attention_workspace_bytes": (_SZ, [_P, _I, _I]),
    "li_norm_rope": (_I, [_P, ctypes.POINTER(c_li_head_rows), _I, _I, _I64, _P, _P]),
    "li_append_paged": (_I, [_P, ctypes.POINTER(c_li_paged_cache), _P, _I, _I64, ctypes.POINTER(c_li_row_transform), _P,
                             _P, _P, _SZ, _P]),
    "li_latent_attention": (_I, [_P, ctypes.POINTER(c_li_paged_cache), _P, _I, _I, _I, ctypes.c_float, _P, _P, _I, _P,
                                 _P, _P, _SZ, _P]),
    "li_prompt_attention": (_I, [_P, ctypes.POINTER(c_li_prompt), _P, _P, _P, _SZ, _P]),
    "li_set_trace": (_I, [_P, _P, _SZ]),
    "li_profile_enable": (_I, [_P, _I]),
    "li_profile_read": (_I, [_P, ctypes.POINTER(c_li_profile_record), _I, ctypes.POINTER(_I)]),
    "li_profile_reset": (_I, [_P]),
}
for _name, (_res, _args) in _sigs.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args

EXPORTED = tuple(_sigs)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _dtype(t: torch.Tensor) -> int:
    return _DTYPE_CODE[t.dtype]


class Context:
    """Owns one li_ctx (host state only)."""

    def __init__(self, device: int = 0):
        h = ctypes.c_void_p()
        st = _lib.li_create(ctypes.byref(h), int(device))
        if st != LI_OK:
            raise LiError(st, f"li_create(device={device}) failed")
        self.handle = h
        self.device = device

    def check(self, status: int):
        if status != LI_OK:
            msg = _lib.li_last_error(self.handle)
            raise LiError(status, msg.decode() if msg else "")

    def close(self):
        if self.handle:
            _lib.li_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


@dataclass
class Cache:
    """A latent or key cache: data [batch, capacity, dim] (float32, bfloat16 or
    uint8 e4m3 codes), scale [batch, capacity] float32 (e4m3 only; with
    segmented fp8, scale_split > 0, [batch, capacity, 2]), lengths [batch]
    int32."""
    data: torch.Tensor
    lengths: torch.Tensor
    scale: Optional[torch.Tensor] = None
    dtype: Optional[int] = None
    scale_split: int = 0

    def c(self) -> c_li_cache:
        b, cap, dim = self.data.shape
        dt = self.dtype if self.dtype is not None else _dtype(self.data)
        return c_li_cache(_ptr(self.data), _ptr(self.scale), _ptr(self.lengths), b, cap, dim, dt,
                          int(self.scale_split))


@dataclass
class LatentTransform:
    """The two-branch latent's row transforms (li_latent_transform): rotary
    range [rope_offset, rope_offset + rope_dim) with inv_freq [rope_dim /
    (2 rope_sources)] float32, LayerNorm range [norm_offset, norm_offset +
    norm_dim) with optional gamma / beta [norm_dim] float32."""
    rope_offset: int = 0
    rope_dim: int = 0
    rope_sources: int = 1
    inv_freq: Optional[torch.Tensor] = None
    norm_offset: int = 0
    norm_dim: int = 0
    gamma: Optional[torch.Tensor] = None
    beta: Optional[torch.Tensor] = None
    eps: float = 1e-6

    def c(self) -> c_li_latent_transform:
        return c_li_latent_transform(self.rope_offset, self.rope_dim, self.rope_sources, _ptr(self.inv_freq),
                                     self.norm_offset, self.norm_dim, _ptr(self.gamma), _ptr(self.beta),
                                     float(self.eps))


@dataclass
class Query:
    """Queries of one layer: q [batch, T, H, dim], w [batch, T, H] float32,
    optional q_scale / beta [batch, T, H] float32 and q_pos [batch, T] int32."""
    q: torch.Tensor
    w: torch.Tensor
    q_scale: Optional[torch.Tensor] = None
    beta: Optional[torch.Tensor] = None
    q_pos: Optional[torch.Tensor] = None
    dtype: Optional[int] = None

    def c(self) -> c_li_query:
        b, T, H, dim = self.q.shape
        dt = self.dtype if self.dtype is not None else _dtype(self.q)
        return c_li_query(_ptr(self.q), dt, _ptr(self.q_scale), _ptr(self.beta), _ptr(self.w), T, H,
                          _ptr(self.q_pos))


def li_create(device: int = 0) -> Context:
    return Context(device)


def li_destroy(ctx: Context):
    ctx.close()


def li_status_string(status: int) -> str:
    return _lib.li_status_string(int(status)).decode()


def li_workspace_bytes(ctx: Optional[Context], batch: int, T: int, capacity: int, H: int, k: int, B: int) -> int:
    return int(_lib.li_workspace_bytes(ctx.handle if ctx else None, batch, T, capacity, H, k, B))


def workspace(ctx: Context, batch: int, T: int, capacity: int, H: int, k: int, B: int = 0,
              device=None) -> torch.Tensor:
    """A zero-filled workspace of li_workspace_bytes(...) bytes (256-byte aligned)."""
    n = li_workspace_bytes(ctx, batch, T, capacity, H, k, B)
    ws = torch.zeros(n, dtype=torch.uint8, device=device or f"cuda:{ctx.device}")
    assert ws.data_ptr() % 256 == 0
    return ws


def li_device_status(ctx: Context, ws: torch.Tensor, stream=None) -> str:
    out = ctypes.c_int(0)
    ctx.check(_lib.li_device_status(ctx.handle, _ptr(ws), _stream(stream), ctypes.byref(out)))
    return STATUS_NAMES.get(out.value, str(out.value))


def li_set_wait_limit(ctx: Context, ns: int):
    ctx.check(_lib.li_set_wait_limit(ctx.handle, int(ns)))


def li_append_latent(ctx: Context, cache: Cache, h: torch.Tensor, W_down: Optional[torch.Tensor], T: int,
                     ws: torch.Tensor, stream=None):
    d_model = h.shape[-1]
    cc = cache.c()
    ctx.check(_lib.li_append_latent(ctx.handle, ctypes.byref(cc), _ptr(h), _dtype(h), d_model, _ptr(W_down),
                                    int(T), _ptr(ws), ws.numel(), _stream(stream)))


def li_append_latent_ex(ctx: Context, cache: Cache, h: torch.Tensor, W_down: Optional[torch.Tensor], T: int,
                        tf: Optional[LatentTransform], ws: torch.Tensor, stream=None):
    d_model = h.shape[-1]
    cc = cache.c()
    ct = tf.c() if tf is not None else None
    ctx.check(_lib.li_append_latent_ex(ctx.handle, ctypes.byref(cc), _ptr(h), _dtype(h), d_model, _ptr(W_down),
                                       int(T), ctypes.byref(ct) if ct is not None else None, _ptr(ws), ws.numel(),
                                       _stream(stream)))


def li_absorb_query(ctx: Context, q: torch.Tensor, W_K: Optional[torch.Tensor], d_c: int, out_dtype: int,
                    q_abs: torch.Tensor, q_abs_scale: Optional[torch.Tensor] = None,
                    b_K: Optional[torch.Tensor] = None, beta: Optional[torch.Tensor] = None,
                    W_K_head_stride: int = 0, b_K_head_stride: int = 0, stream=None):
    """q [..., H, d_k] -> q_abs [..., H, d_c] (n_tok = product of the leading dims)."""
    H, d_k = q.shape[-2], q.shape[-1]
    n_tok = q.numel() // (H * d_k)
    ctx.check(_lib.li_absorb_query(ctx.handle, _ptr(q), _dtype(q), n_tok, H, d_k, _ptr(W_K), int(W_K_head_stride),
                                   _ptr(b_K), int(b_K_head_stride), int(d_c), int(out_dtype), _ptr(q_abs),
                                   _ptr(q_abs_scale), _ptr(beta), _stream(stream)))


def li_score_topk(ctx: Context, cache: Cache, query: Query, k: int, out_idx: torch.Tensor,
                  out_score: Optional[torch.Tensor], scores_dump: Optional[torch.Tensor], ws: torch.Tensor,
                  stream=None):
    cc, qq = cache.c(), query.c()
    ctx.check(_lib.li_score_topk(ctx.handle, ctypes.byref(cc), ctypes.byref(qq), int(k), _ptr(out_idx),
                                 _ptr(out_score), _ptr(scores_dump), _ptr(ws), ws.numel(), _stream(stream)))


def li_score_topk_static(ctx: Context, cache: Cache, query: Query, k: int, out_idx: torch.Tensor,
                         out_score: Optional[torch.Tensor] = None, device_status: Optional[torch.Tensor] = None,
                         stream=None):
    """li_score_topk with the library's fixed internal scratch instead of a workspace."""
    cc, qq = cache.c(), query.c()
    ctx.check(_lib.li_score_topk_static(ctx.handle, ctypes.byref(cc), ctypes.byref(qq), int(k), _ptr(out_idx),
                                        _ptr(out_score), _ptr(device_status), _stream(stream)))


def li_dsa_score_topk(ctx: Context, key_cache: Cache, query: Query, k: int, out_idx: torch.Tensor,
                      out_score: Optional[torch.Tensor], scores_dump: Optional[torch.Tensor], ws: torch.Tensor,
                      stream=None):
    cc, qq = key_cache.c(), query.c()
    ctx.check(_lib.li_dsa_score_topk(ctx.handle, ctypes.byref(cc), ctypes.byref(qq), int(k), _ptr(out_idx),
                                     _ptr(out_score), _ptr(scores_dump), _ptr(ws), ws.numel(), _stream(stream)))


def li_hs_anchor_candidates(ctx: Context, cache: Cache, query: Query, B: int, k: int, cand: torch.Tensor,
                            cand_n: torch.Tensor, anchor_idx: torch.Tensor, anchor_score: Optional[torch.Tensor],
                            scores_dump: Optional[torch.Tensor], ws: torch.Tensor, stream=None):
    cc, qq = cache.c(), query.c()
    ctx.check(_lib.li_hs_anchor_candidates(ctx.handle, ctypes.byref(cc), ctypes.byref(qq), int(B), int(k),
                                           _ptr(cand), _ptr(cand_n), _ptr(anchor_idx), _ptr(anchor_score),
                                           _ptr(scores_dump), _ptr(ws), ws.numel(), _stream(stream)))


def li_hs_follower_refine(ctx: Context, cache: Cache, query: Query, cand: torch.Tensor, cand_n: torch.Tensor,
                          B: int, k: int, out_idx: torch.Tensor, out_score: Optional[torch.Tensor],
                          scores_dump: Optional[torch.Tensor], ws: torch.Tensor, stream=None):
    cc, qq = cache.c(), query.c()
    ctx.check(_lib.li_hs_follower_refine(ctx.handle, ctypes.byref(cc), ctypes.byref(qq), _ptr(cand),
                                         _ptr(cand_n), int(B), int(k), _ptr(out_idx), _ptr(out_score),
                                         _ptr(scores_dump), _ptr(ws), ws.numel(), _stream(stream)))


def li_absorb_query_group(ctx: Context, q: torch.Tensor, W_K: List[torch.Tensor], d_c: int, out_dtype: int,
                          q_abs: torch.Tensor, q_abs_scale: Optional[torch.Tensor] = None, stream=None):
    """q [batch, G, H, d_k] (f32 or bf16), W_K: G decoders [d_k, d_c] of q's
    dtype -> q_abs [batch, G, H, d_c] (and q_abs_scale [batch, G, H] for e4m3)."""
    batch, G, H, d_k = q.shape
    ptrs = (_P * G)(*[W.data_ptr() for W in W_K])
    ctx.check(_lib.li_absorb_query_group(ctx.handle, _ptr(q), _dtype(q), batch, G, H, d_k, ptrs, int(d_c),
                                         int(out_dtype), _ptr(q_abs), _ptr(q_abs_scale), _stream(stream)))


def li_topk(ctx: Context, scores: torch.Tensor, k: int, out_idx: torch.Tensor, out_score: Optional[torch.Tensor],
            ws: torch.Tensor, lengths: Optional[torch.Tensor] = None, n: Optional[int] = None, stream=None):
    """scores [rows, stride] float32; row r selects among its first n (or lengths[r]) entries."""
    rows, stride = scores.shape
    n = stride if n is None else n
    ctx.check(_lib.li_topk(ctx.handle, _ptr(scores), rows, int(n), int(scores.stride(0)), _ptr(lengths), int(k),
                           _ptr(out_idx), _ptr(out_score), _ptr(ws), ws.numel(), _stream(stream)))


def li_attention_recall(ctx: Context, probs: torch.Tensor, sel: torch.Tensor, K: int,
                        lengths: Optional[torch.Tensor] = None, mean: bool = True, ws: Optional[torch.Tensor] = None,
                        stream=None):
    """probs [rows, H, N] float32, sel [rows, k] int32 (-1 padded).  Returns
    (recall [rows, H], mean_recall [rows] or None) as device tensors."""
    rows, H, N = probs.shape
    k = sel.shape[-1]
    need = int(_lib.li_recall_workspace_bytes(ctx.handle, rows, H, N, int(K)))
    if ws is None or ws.numel() < need:
        ws = torch.zeros(need, dtype=torch.uint8, device=probs.device)
    rec = torch.empty(rows, H, device=probs.device)
    mrec = torch.empty(rows, device=probs.device) if mean else None
    ctx.check(_lib.li_attention_recall(ctx.handle, _ptr(probs), rows, H, N, _ptr(lengths), _ptr(sel), int(k), int(K),
                                       _ptr(rec), _ptr(mrec), _ptr(ws), ws.numel(), _stream(stream)))
    return rec, mrec


# ---------------------------------------------------------------- attention over the selected tokens

_NORM = {"none": 0, "rms": 1, "layer": 2}
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else None


def _need(ok: bool, status: str, message: str):
    """Shape and type checks of the tensors behind the pointers, which the C entry points cannot see."""
    if not ok:
        raise LiError(STATUS[status], message)


def _check_tensor(name: str, t: torch.Tensor, shape, dtype, device: int, contiguous: bool = True):
    """Explains what is wrong with a tensor (calls are made once per launch, so the passing path is kept short)."""
    _need(t.shape == shape, "LI_ERR_SHAPE", f"{name} is {tuple(t.shape)}, expected {tuple(shape)}")
    _need(t.dtype is dtype, "LI_ERR_DTYPE", f"{name} is {t.dtype}, expected {dtype}")
    _need(t.get_device() == device, "LI_ERR_ARG", f"{name} is on {t.device}, expected device {device}")
    _need(t.is_contiguous() if contiguous else t.shape[-1] <= 1 or t.stride(-1) == 1, "LI_ERR_ARG",
          f"{name} must be contiguous" if contiguous else f"rows of {name} must be contiguous")


def _in(name: str, t: Optional[torch.Tensor], shape, dtype, device: int):
    """Address of a contiguous tensor of this shape and type (None: NULL)."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or not t.is_contiguous() or t.get_device() != device:
        _check_tensor(name, t, shape, dtype, device)
    return t.data_ptr()


def _current_stream(ctx, stream):
    if stream is None and _raw_stream is not None:
        return _raw_stream(ctx.device)
    return _stream(stream)


def _attn_dtype(t: torch.Tensor) -> int:
    _need(t.dtype in (torch.float32, torch.bfloat16), "LI_ERR_DTYPE", f"float32 or bfloat16 only (got {t.dtype})")
    return _DTYPE_CODE[t.dtype]


@dataclass(frozen=True)
class RowTransform:
    """Transforms of one row (li_row_transform): a norm ("none", "rms" or
    "layer") of elements [norm_offset, norm_offset + norm_dim) with optional
    gamma / beta [norm_dim] float32, then the rotation of [rope_offset,
    rope_offset + rope_dim) by inv_freq [rope_dim / 2] float32, slots being
    adjacent pairs or, with rope_halves, element p and p + rope_dim / 2.  The C
    record is made here, once: build a new one to change anything."""
    norm: str = "none"
    norm_offset: int = 0
    norm_dim: int = 0
    gamma: Optional[torch.Tensor] = None
    beta: Optional[torch.Tensor] = None
    eps: float = 1e-6
    rope_offset: int = 0
    rope_dim: int = 0
    rope_halves: bool = False
    inv_freq: Optional[torch.Tensor] = None

    def __post_init__(self):
        _need(self.norm in _NORM, "LI_ERR_ARG", f"unknown norm {self.norm!r}")
        tensors = [t for t in (self.gamma, self.beta, self.inv_freq if self.rope_dim else None) if t is not None]
        device = tensors[0].get_device() if tensors else None
        g, b = (_in(n, t, (self.norm_dim,), torch.float32, device) for n, t in (("gamma", self.gamma), ("beta", self.beta)))
        f = _in("inv_freq", self.inv_freq, (self.rope_dim // 2,), torch.float32, device) if self.rope_dim else None
        object.__setattr__(self, "device", device)
        object.__setattr__(self, "c", c_li_row_transform(_NORM[self.norm], self.norm_offset, self.norm_dim, g, b,
                                                         float(self.eps), self.rope_offset, self.rope_dim,
                                                         1 if self.rope_halves else 0, f))


@dataclass(frozen=True)
class HeadRows:
    """The heads of every token in one tensor (li_head_rows): x [n_tok, H,
    dim] and out of the same shape, any strides over tokens and heads; out
    may be x.  The C record is made here, once."""
    x: torch.Tensor
    tf: RowTransform
    out: torch.Tensor

    def __post_init__(self):
        x, out = self.x, self.out
        _need(x.dim() == 3, "LI_ERR_SHAPE", f"x is {tuple(x.shape)}, expected [n_tok, H, dim]")
        device = x.get_device()
        _check_tensor("x", x, x.shape, x.dtype, device, contiguous=False)
        _check_tensor("out", out, x.shape, x.dtype, device, contiguous=False)
        _need(self.tf.device in (None, device), "LI_ERR_ARG", f"the transform is on device {self.tf.device}, x on {device}")
        object.__setattr__(self, "dtype", _attn_dtype(x))
        object.__setattr__(self, "device", device)
        object.__setattr__(self, "n", x.shape[0])
        object.__setattr__(self, "c", c_li_head_rows(x.data_ptr(), out.data_ptr(), x.shape[1], x.shape[2], x.stride(0),
                                                     x.stride(1), out.stride(0), out.stride(1), self.tf.c))


_HEAD_ROWS = {n: c_li_head_rows * n for n in (1, 2, 3, 4)}


@dataclass(frozen=True)
class PagedCache:
    """A paged cache of attention latents (li_paged_cache): data [n_pages,
    page_size, dim] float32 or bfloat16, page_table [batch, max_pages] int32,
    lengths [batch] int32.  The C record is made here, once."""
    data: torch.Tensor
    page_table: torch.Tensor
    lengths: torch.Tensor

    def __post_init__(self):
        _need(self.data.dim() == 3 and self.page_table.dim() == 2, "LI_ERR_SHAPE",
              "data must be [n_pages, page_size, dim] and page_table [batch, max_pages]")
        (n_pages, page, dim), (batch, max_pages) = self.data.shape, self.page_table.shape
        device = self.data.get_device()
        c = c_li_paged_cache(_in("data", self.data, self.data.shape, self.data.dtype, device),
                             _in("page_table", self.page_table, (batch, max_pages), torch.int32, device),
                             _in("lengths", self.lengths, (batch,), torch.int32, device), batch, n_pages, page, max_pages,
                             dim, _attn_dtype(self.data))
        for name, v in (("c", c), ("ref", ctypes.byref(c)), ("device", device), ("batch", batch), ("dim", dim)):
            object.__setattr__(self, name, v)


def li_attention_workspace_bytes(ctx: Optional[Context], H: int, d_v: int) -> int:
    return int(_lib.li_attention_workspace_bytes(ctx.handle if ctx else None, int(H), int(d_v)))


def attention_workspace(ctx: Context, H: int, d_v: int, device=None) -> torch.Tensor:
    """A zero-filled workspace of li_attention_workspace_bytes(...) bytes: for
    li_append_paged, li_latent_attention and li_prompt_attention of up to H
    heads of d_v values."""
    return torch.zeros(li_attention_workspace_bytes(ctx, H, d_v), dtype=torch.uint8, device=device or f"cuda:{ctx.device}")


def _workspace(ctx: Context, ws: torch.Tensor):
    _need(ws.get_device() == ctx.device and ws.dtype is torch.uint8 and ws.is_contiguous(), "LI_ERR_WORKSPACE",
          f"the workspace must be contiguous uint8 on device {ctx.device}")
    return ws.data_ptr(), ws.numel()


def li_norm_rope(ctx: Context, sets: List[HeadRows], pos: Optional[torch.Tensor] = None, stream=None):
    """Norms and rotation of the heads in every tensor of `sets` (1 to 4, the
    same tokens and type), pos [n_tok] int32, in one launch."""
    _need(1 <= len(sets) <= 4, "LI_ERR_ARG", f"need 1 to 4 tensors (got {len(sets)})")
    n, dtype = sets[0].n, sets[0].dtype
    for s in sets:
        _need(s.n == n and s.dtype == dtype, "LI_ERR_SHAPE", "the tensors differ in tokens or type")
        _need(s.device == ctx.device, "LI_ERR_ARG", f"a tensor is on device {s.device}, the context on {ctx.device}")
    ctx.check(_lib.li_norm_rope(ctx.handle, _HEAD_ROWS[len(sets)](*[s.c for s in sets]), len(sets), dtype, n,
                                _in("pos", pos, (n,), torch.int32, ctx.device), _current_stream(ctx, stream)))


def li_append_paged(ctx: Context, cache: PagedCache, x: torch.Tensor, ws: torch.Tensor, tf: Optional[RowTransform] = None,
                    start: Optional[torch.Tensor] = None, n_new: Optional[torch.Tensor] = None, stream=None):
    """x [batch, T, dim] (rows at one stride) into the cache, transformed, at
    positions start[b] (or lengths[b]) onwards; n_new [batch]: rows of each
    sequence."""
    dev, batch = ctx.device, cache.batch
    _need(cache.device == dev and (tf is None or tf.device in (None, dev)), "LI_ERR_ARG",
          f"the cache or the transform is not on the context's device {dev}")
    _need(x.dim() == 3, "LI_ERR_SHAPE", f"x is {tuple(x.shape)}, expected [batch, T, dim]")
    T = x.shape[1]
    if x.shape != (batch, T, cache.dim) or x.dtype is not cache.data.dtype or x.get_device() != dev or x.stride(2) != 1:
        _check_tensor("x", x, (batch, T, cache.dim), cache.data.dtype, dev, contiguous=False)
    stride = x.stride(1) if T > 1 else x.stride(0)
    _need(batch == 1 or T == 0 or x.stride(0) == T * stride, "LI_ERR_ARG", "the rows of x must lie at one stride")
    p, n = _workspace(ctx, ws)
    ctx.check(_lib.li_append_paged(ctx.handle, cache.ref, x.data_ptr(), T, stride, tf.c if tf is not None else None,
                                   _in("start", start, (batch,), torch.int32, dev),
                                   _in("n_new", n_new, (batch,), torch.int32, dev), p, n, _current_stream(ctx, stream)))


def li_latent_attention(ctx: Context, cache: PagedCache, q: torch.Tensor, d_v: int, scale: float, out: torch.Tensor,
                        ws: torch.Tensor, lse: Optional[torch.Tensor] = None, sel: Optional[torch.Tensor] = None,
                        q_pos: Optional[torch.Tensor] = None, stream=None):
    """Absorbed queries q [batch, T, H, dim] over the cached latents: the
    positions of sel [batch, T, k] (a selection output), or the whole prefix.
    out [batch, T, H, d_v], lse [batch, T, H] float32, q_pos [batch, T]."""
    dev, b = ctx.device, cache.batch
    _need(cache.device == dev, "LI_ERR_ARG", f"the cache is on device {cache.device}, the context on {dev}")
    _need(q.dim() == 4, "LI_ERR_SHAPE", f"q is {tuple(q.shape)}, expected [batch, T, H, dim]")
    _, T, H, _ = q.shape
    dt = cache.data.dtype
    k, sel_ptr = 0, None
    if sel is not None:
        k = sel.shape[-1]
        _need(k >= 1, "LI_ERR_SHAPE", "k must be >= 1 with sel")
        sel_ptr = _in("sel", sel, (b, T, k), torch.int32, dev)
    p, n = _workspace(ctx, ws)
    ctx.check(_lib.li_latent_attention(ctx.handle, cache.ref, _in("q", q, (b, T, H, cache.dim), dt, dev), T, H, d_v, scale,
                                       _in("q_pos", q_pos, (b, T), torch.int32, dev), sel_ptr, k,
                                       _in("out", out, (b, T, H, d_v), dt, dev),
                                       _in("lse", lse, (b, T, H), torch.float32, dev), p, n, _current_stream(ctx, stream)))


def li_prompt_attention(ctx: Context, q: torch.Tensor, k_nope: torch.Tensor, k_rope: Optional[torch.Tensor],
                        v: torch.Tensor, cu_q: torch.Tensor, cu_k: torch.Tensor, max_q: int, scale: float,
                        out: torch.Tensor, ws: torch.Tensor, lse: Optional[torch.Tensor] = None, causal: bool = True,
                        stream=None):
    """Expanded attention of a ragged batch of prompts: q [total_q, H, d_nope +
    d_rope], k_nope [total_k, H, d_nope], k_rope [total_k, d_rope] (shared by
    the heads) or None, v [total_k, H, d_v], any positive strides over tokens
    and heads; cu_q, cu_k [batch + 1] int32; out [total_q, H, d_v], lse
    [total_q, H] float32."""
    _need(q.dim() == 3 and k_nope.dim() == 3 and v.dim() == 3, "LI_ERR_SHAPE", "q, k_nope and v must be [tokens, H, dim]")
    (tq, H, dq), (tk, _, dn), dv, dt, dev = q.shape, k_nope.shape, v.shape[-1], q.dtype, ctx.device
    dr = 0 if k_rope is None else k_rope.shape[-1]
    for name, t, shape in (("q", q, (tq, H, dn + dr)), ("k_nope", k_nope, (tk, H, dn)), ("v", v, (tk, H, dv)),
                           ("k_rope", k_rope, (tk, dr))):
        if t is not None and (t.shape != shape or t.dtype is not dt or t.get_device() != dev or t.stride(-1) != 1):
            _check_tensor(name, t, shape, dt, dev, contiguous=False)
    qs, ks, vs = q.stride(), k_nope.stride(), v.stride()
    batch = cu_q.shape[0] - 1
    rec = c_li_prompt(q.data_ptr(), k_nope.data_ptr(), None if k_rope is None else k_rope.data_ptr(), v.data_ptr(),
                      _attn_dtype(q), H, dn, dr, dv, tq, tk, batch, max_q, qs[0], qs[1], ks[0], ks[1],
                      0 if k_rope is None else k_rope.stride(0), vs[0], vs[1],
                      _in("cu_q", cu_q, (batch + 1,), torch.int32, dev), _in("cu_k", cu_k, (batch + 1,), torch.int32, dev),
                      scale, 1 if causal else 0)
    p, n = _workspace(ctx, ws)
    ctx.check(_lib.li_prompt_attention(ctx.handle, rec, _in("out", out, (tq, H, dv), dt, dev),
                                       _in("lse", lse, (tq, H), torch.float32, dev), p, n, _current_stream(ctx, stream)))


def li_set_trace(ctx: Context, buf: Optional[torch.Tensor]):
    """Diagnostic per-tile trace of the scoring kernels into buf (uint8/int64
    device tensor of >= 32768 bytes, viewed as [8, 64, 8] int64), or None."""
    ctx.check(_lib.li_set_trace(ctx.handle, _ptr(buf), 0 if buf is None else buf.numel() * buf.element_size()))


def li_profile_enable(ctx: Context, enable: bool = True):
    ctx.check(_lib.li_profile_enable(ctx.handle, 1 if enable else 0))


def li_profile_read(ctx: Context):
    count = ctypes.c_int(0)
    ctx.check(_lib.li_profile_read(ctx.handle, None, 0, ctypes.byref(count)))
    n = count.value
    recs = (c_li_profile_record * max(n, 1))()
    ctx.check(_lib.li_profile_read(ctx.handle, recs, n, ctypes.byref(count)))
    return [dict(kernel=recs[i].kernel.decode(), ms=recs[i].ms, grid=recs[i].grid, block=recs[i].block,
                 smem=recs[i].smem) for i in range(n)]


def li_profile_reset(ctx: Context):
    ctx.check(_lib.li_profile_reset(ctx.handle))
