"""Binding of the operators between a decode step's projections (``include/sgemm_decode.h``):

- :func:`sgemm_bf16_add_rmsnorm`, :func:`sgemm_bf16_add_rmsnorm_e4m3`: residual add and RMS norm,
- :func:`sgemm_bf16_latent_append`: append to a paged latent cache, rotating on the way,
- :func:`sgemm_bf16_latent_attention`: attention over that cache (absorbed form).

As in the rest of the package, the functions check and marshal their arguments; every step of
the computation runs in the library's CUDA kernels.  Each takes preallocated outputs (allocating
nothing then), launch flags and a stream, and can be captured into a CUDA graph.  All tensors are on
the current device.  Outputs and scratch that a call is not given come from the allocator's blocks
of the stream it runs on; the caller orders what it does with the outputs behind that stream, as
with any work there.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import struct
import warnings

import torch

from . import SgemmError, _empty, load
from .build import marshal_path

__all__ = [
    "sgemm_bf16_add_rmsnorm", "sgemm_bf16_add_rmsnorm_e4m3", "sgemm_bf16_latent_append",
    "sgemm_bf16_latent_attention", "sgemm_latent_attention_workspace",
    "SGEMM_NORM_BF16", "SGEMM_NORM_E4M3_ROW", "SGEMM_NORM_E4M3_GROUP128", "LATENT_WORKSPACE_MAX",
]

SGEMM_NORM_BF16 = 0
SGEMM_NORM_E4M3_ROW = 1
SGEMM_NORM_E4M3_GROUP128 = 2
LATENT_WORKSPACE_MAX = 64 << 20

# the argument structures of the header, field by field (natural alignment, no padding)
_NORM = struct.Struct("<6Q6qiifI")        # sgemm_add_rmsnorm_t
_APPEND = struct.Struct("<8Q11q5ifIi")    # sgemm_latent_append_t
_ATTN = struct.Struct("<8Q11q7ifIi")      # sgemm_latent_attention_t

_BF16 = torch.bfloat16
_fns: dict = {}


class _None:
    """In place of ``_marshal`` where there is none for this Python and torch: the checks below look
    at every call, which takes longer and is the same call."""

    def add_rmsnorm(self, *args):
        return -1

    latent_append = latent_attention = add_rmsnorm


class _Unbound:
    """Stands in for ``_marshal`` until the first call has loaded the library."""

    def _first(self, name, args):
        global _short
        lib = load()
        try:
            loader = importlib.machinery.ExtensionFileLoader("_marshal", marshal_path())
            module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_marshal", loader))
            loader.exec_module(module)
            module.bind(*(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value for f in (
                "sgemm_bf16_add_rmsnorm", "sgemm_bf16_latent_append", "sgemm_bf16_latent_attention")))
        except ImportError as e:
            warnings.warn(f"calls take longer than they need: {e}; build the module for this torch with "
                          "python -c 'import __graft_entry__ as g; g.build()'", RuntimeWarning, stacklevel=4)
            module = _None()
        _short = module
        return getattr(module, name)(*args)

    def add_rmsnorm(self, *args):
        return self._first("add_rmsnorm", args)

    def latent_append(self, *args):
        return self._first("latent_append", args)

    def latent_attention(self, *args):
        return self._first("latent_attention", args)


# The short way of a well-formed call with all its buffers given (native/marshal.cpp): it returns
# the call's status, or -1 for what the checks below have to look at.
_short = _Unbound()


def _fn(name: str):
    f = _fns.get(name)
    if f is None:
        f = getattr(load(), name)
        f.argtypes = [ctypes.c_char_p, ctypes.c_void_p]
        f.restype = ctypes.c_int
        _fns[name] = f
    return f


def _raw(stream):
    """A torch stream's handle; a handle, or None for the current stream, as it is."""
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else stream


def _call(name: str, args: bytes, t: torch.Tensor, stream) -> None:
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(t.get_device())
    elif isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    status = (_fns.get(name) or _fn(name))(args, stream)
    if status:
        raise SgemmError(status, name)


def _on_current_device(**tensors) -> None:
    """The library launches on the current device, so that every tensor has to be there."""
    here = torch.cuda.current_device()
    for name, t in tensors.items():
        if t is not None and t.get_device() != here:
            raise ValueError(f"{name} is on cuda:{t.get_device()}, the current device is cuda:{here}")


def _refuse(t, name: str, dtype, shape):
    """What is wrong with a tensor; its strides if nothing is (a last dimension of one element has
    a stride of no account)."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.dim() != len(shape):
        raise TypeError(f"{name} must be a {len(shape)}-D {dtype} tensor")
    if not t.is_cuda:
        raise TypeError(f"{name} must be on a CUDA device")
    for n, want in zip(t.shape, shape):
        if want is not None and n != want:
            raise ValueError(f"{name} must be {['any' if w is None else w for w in shape]}, got {list(t.shape)}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")
    return t.stride()


def _strides(t, name: str, dtype, shape):
    """The strides of a CUDA tensor of this type and shape whose last dimension has unit stride
    (one pass over its attributes: a step's calls are short)."""
    try:
        if t.dtype is dtype and t.is_cuda and t.shape == shape:
            s = t.stride()
            if s[-1] == 1:
                return s
    except AttributeError:
        pass
    return _refuse(t, name, dtype, shape)


def _shape(t, name: str, dtype, dim: int):
    """The shape of a tensor that has any of this rank."""
    try:
        if t.dtype is dtype and len(t.shape) == dim:
            return t.shape
    except AttributeError:
        pass
    _refuse(t, name, dtype, (None,) * dim)


# ----------------------------------------------------------------------------- residual RMS norm
def _norm(x, weight, residual, eps, form, y, y_dtype, scales, residual_out, flags, stream):
    shape = _shape(x, "x", _BF16, 2)
    T, D = shape
    ldx = _strides(x, "x", _BF16, shape)[0]
    _strides(weight, "weight", _BF16, (D,))
    ldr = ldro = D
    pr = pro = ps = lds = 0
    if residual is not None:
        ldr = _strides(residual, "residual", _BF16, shape)[0]
        pr = residual.data_ptr()
        if residual_out is None:
            residual_out = _empty(shape, _BF16, x.device, stream)
    if residual_out is not None:
        ldro = _strides(residual_out, "residual_out", _BF16, shape)[0]
        pro = residual_out.data_ptr()
    if y is None:
        y = _empty(shape, y_dtype, x.device, stream)
    named = "y" if form == SGEMM_NORM_BF16 else "q"
    ldy = _strides(y, named, y_dtype, shape)[0]
    if form != SGEMM_NORM_BF16:
        groups = -(-D // 128) if form == SGEMM_NORM_E4M3_GROUP128 else 1
        if scales is None:
            scales = _empty((T, groups), torch.float32, x.device, stream)
        lds = _strides(scales, "scales", torch.float32, (T, groups))[0]
        ps = scales.data_ptr()
    _on_current_device(x=x, weight=weight, residual=residual, **{named: y}, scales=scales, residual_out=residual_out)
    if T <= 1:
        if T == 0:
            return y, scales, residual_out
        ldx = ldr = ldro = ldy = lds = D  # the row stride of a single row is of no account
    _call("sgemm_bf16_add_rmsnorm", _NORM.pack(
        x.data_ptr(), pr, weight.data_ptr(), pro, y.data_ptr(), ps, ldx, ldr, ldro, ldy, lds, T, D, form, eps, flags),
        x, stream)
    return y, scales, residual_out


def sgemm_bf16_add_rmsnorm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None,
                           eps: float = 1e-6, y: torch.Tensor | None = None,
                           residual_out: torch.Tensor | None = None, flags: int = 0, stream=None):
    """``h = x + residual``, ``y = bf16(h * rsqrt(mean(h**2) + eps) * weight)``; returns
    ``(y, residual_out)`` with ``residual_out = bf16(h)`` (None where neither a residual nor a
    buffer for it is given).  x, residual: BF16 [T, D], rows of any stride; weight: BF16 [D].
    ``residual_out`` may be ``residual`` or ``x``, and ``y`` may be ``x``: in place."""
    status = _short.add_rmsnorm(x, weight, residual, eps, SGEMM_NORM_BF16, y, None, residual_out, flags, _raw(stream))
    if status == 0:
        return y, residual_out
    if status > 0:
        raise SgemmError(status, "sgemm_bf16_add_rmsnorm")
    y, _, residual_out = _norm(x, weight, residual, eps, SGEMM_NORM_BF16, y, _BF16, None, residual_out, flags, stream)
    return y, residual_out


def sgemm_bf16_add_rmsnorm_e4m3(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None,
                                eps: float = 1e-6, group: int = 128, q: torch.Tensor | None = None,
                                scales: torch.Tensor | None = None,
                                residual_out: torch.Tensor | None = None, flags: int = 0, stream=None):
    """:func:`sgemm_bf16_add_rmsnorm` with y in 8 bits: returns ``(q, scales, residual_out)``,
    ``q = e4m3(y / scale)`` (torch.float8_e4m3fn [T, D]) and FP32 scales ``max|y| / 448``
    (1 where that is 0) per 128 columns (``group=128``: [T, ceil(D / 128)]) or per row
    (``group=0``: [T, 1])."""
    if group not in (0, 128):
        raise ValueError(f"group must be 128 (columns a scale) or 0 (one scale a row), got {group}")
    form = SGEMM_NORM_E4M3_GROUP128 if group else SGEMM_NORM_E4M3_ROW
    status = _short.add_rmsnorm(x, weight, residual, eps, form, q, scales, residual_out, flags, _raw(stream))
    if status == 0:
        return q, scales, residual_out
    if status > 0:
        raise SgemmError(status, "sgemm_bf16_add_rmsnorm")
    return _norm(x, weight, residual, eps, form, q, torch.float8_e4m3fn, scales,
                 residual_out, flags, stream)


# ---------------------------------------------------------------------------------- cache append
def sgemm_bf16_latent_append(kv: torch.Tensor, cache: torch.Tensor, slots: torch.Tensor,
                             positions: torch.Tensor, cos_sin: torch.Tensor,
                             weight: torch.Tensor | None = None, eps: float = 1e-6,
                             q: torch.Tensor | None = None, q_out: torch.Tensor | None = None,
                             interleaved: bool = True, flags: int = 0, stream=None):
    """Write each token's row into the paged latent cache; returns ``(cache, q_out)``.

    kv: BF16 [T, R + E], the latent vector and the E elements to rotate; cache: BF16
    [pages, page_size, R + E] (pages and rows of any stride); slots, positions: int64 [T], the
    row ``page * page_size + i`` each token goes to (negative: none) and its position; cos_sin:
    FP32 [positions, E], cosines then sines.  With ``weight`` (BF16 [R]) the latent vector is
    RMS-normalised on the way.  q, q_out: BF16 [T, H, E] views, the part of each head's query
    that is rotated and where it goes (may be the same).  ``interleaved``: the rotated pairs are
    (2i, 2i + 1), else (i, E / 2 + i)."""
    status = _short.latent_append(kv, cache, slots, positions, cos_sin, weight, eps, q, q_out, interleaved, flags,
                                  _raw(stream))
    if status == 0:
        return cache, q_out
    if status > 0:
        raise SgemmError(status, "sgemm_bf16_latent_append")
    T, W = shape = _shape(kv, "kv", _BF16, 2)
    pages, page_size, width = _shape(cache, "cache", _BF16, 3)
    limit, E = _shape(cos_sin, "cos_sin", torch.float32, 2)
    R = W - E
    if width != W:
        raise ValueError(f"cache rows must be as wide as kv's ({W}), got {width}")
    if R < 1:
        raise ValueError(f"kv rows ({W}) must be wider than cos_sin's ({E})")
    ldkv = _strides(kv, "kv", _BF16, shape)[0]
    page_stride, row_stride, _ = _strides(cache, "cache", _BF16, (pages, page_size, W))
    ldcs = _strides(cos_sin, "cos_sin", torch.float32, (limit, E))[0]
    _strides(slots, "slots", torch.int64, (T,))
    _strides(positions, "positions", torch.int64, (T,))
    H = pq = pqo = pw = q_token = q_head = qo_token = qo_head = 0
    if weight is not None:
        _strides(weight, "weight", _BF16, (R,))
        pw = weight.data_ptr()
    if q is not None:
        H = _shape(q, "q", _BF16, 3)[1]
        q_token, q_head, _ = _strides(q, "q", _BF16, (T, H, E))
        if q_out is None:
            q_out = _empty((T, H, E), _BF16, kv.device, stream)
        qo_token, qo_head, _ = _strides(q_out, "q_out", _BF16, (T, H, E))
        if H:
            pq, pqo = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    _on_current_device(kv=kv, cache=cache, slots=slots, positions=positions, cos_sin=cos_sin, weight=weight, q=q, q_out=q_out)
    if T == 0:
        return cache, q_out
    # strides along dimensions of one element are of no account
    if T == 1:
        ldkv = W
    if limit == 1:
        ldcs = E
    if page_size == 1:
        row_stride = W
    if pages == 1:
        page_stride = page_size * row_stride
    _call("sgemm_bf16_latent_append", _APPEND.pack(
        kv.data_ptr(), pw, cos_sin.data_ptr(), positions.data_ptr(), slots.data_ptr(), cache.data_ptr(), pq, pqo,
        ldkv, ldcs, row_stride, page_stride, q_token, q_head, qo_token, qo_head,
        T, limit, pages, page_size, R, E, H, 1 if interleaved else 0, eps, flags, 0), kv, stream)
    return cache, q_out


# ------------------------------------------------------------------------------ latent attention
def sgemm_latent_attention_workspace(batch: int, heads: int, rank: int, rope: int, page_size: int,
                                     table_width: int, max_q: int = 1) -> int:
    """Bytes of scratch :func:`sgemm_bf16_latent_attention` needs for such a call
    (at most ``LATENT_WORKSPACE_MAX``)."""
    n = ctypes.c_longlong(0)
    f = _fn("sgemm_latent_attention_workspace")
    # one token: how many there are does not matter, and sequences of max_q each may be too many
    args = _ATTN.pack(*([0] * 16), 1, 0, min(batch * max_q, 1), page_size, table_width, batch, heads, rank, rope, max_q,
                      1.0, 0, 0)
    status = f(args, ctypes.addressof(n))
    if status:
        raise SgemmError(status, "sgemm_latent_attention_workspace")
    return n.value


def sgemm_bf16_latent_attention(q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor,
                                seq_lens: torch.Tensor, rank: int, scale: float,
                                cu_q: torch.Tensor | None = None, max_q: int = 1,
                                out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                                workspace: torch.Tensor | None = None, flags: int = 0, stream=None):
    """Attention over a paged latent cache, absorbed form; returns ``(out, lse)``.

    q: BF16 [total_q, H, rank + E]; cache: BF16 [pages, page_size, rank + E], whose first ``rank``
    elements are also the values; block_table: int32 [B, width]; seq_lens: int32 [B], cached rows
    of each sequence, its new tokens' among them.  ``cu_q``: int32 [B + 1], where each sequence's
    query tokens begin, at most ``max_q`` each (None: ``max_q`` each).  Token i of a sequence's n
    sees its first ``seq_lens - n + i + 1`` rows; one that sees none gets zeros (and -inf).
    out: BF16 [total_q, H, rank]; lse: FP32 [total_q, H] or None (not written).  ``workspace``:
    scratch on the device (:func:`sgemm_latent_attention_workspace` bytes; allocated for the call
    where None)."""
    status = _short.latent_attention(q, cache, block_table, seq_lens, rank, scale, cu_q, max_q, out, lse, workspace, flags,
                                     _raw(stream))
    if status == 0:
        return out, lse
    if status > 0:
        raise SgemmError(status, "sgemm_bf16_latent_attention")
    total, H, W = shape = _shape(q, "q", _BF16, 3)
    pages, page_size, width = _shape(cache, "cache", _BF16, 3)
    B, table_width = _shape(block_table, "block_table", torch.int32, 2)
    if width != W:
        raise ValueError(f"cache rows must be as wide as q's ({W}), got {width}")
    q_token, q_head, _ = _strides(q, "q", _BF16, shape)
    page_stride, row_stride, _ = _strides(cache, "cache", _BF16, (pages, page_size, W))
    ldt = _strides(block_table, "block_table", torch.int32, (B, table_width))[0]
    _strides(seq_lens, "seq_lens", torch.int32, (B,))
    pcu = plse = lse_token = 0
    if cu_q is not None:
        _strides(cu_q, "cu_q", torch.int32, (B + 1,))
        pcu = cu_q.data_ptr()
    elif total != B * max_q:
        raise ValueError(f"q must hold {B} x {max_q} tokens without cu_q, got {total}")
    if out is None:
        out = _empty((total, H, rank), _BF16, q.device, stream)
    out_token, out_head, _ = _strides(out, "out", _BF16, (total, H, rank))
    if lse is not None:
        lse_token = _strides(lse, "lse", torch.float32, (total, H))[0]
        plse = lse.data_ptr()
    _on_current_device(q=q, cache=cache, block_table=block_table, seq_lens=seq_lens, cu_q=cu_q, out=out, lse=lse)
    if total == 0 or B == 0:
        return out, lse
    if workspace is None:
        need = sgemm_latent_attention_workspace(B, H, rank, W - rank, page_size, table_width, max_q)
        workspace = _empty((need,), torch.uint8, q.device, stream, returned=False)
    elif not workspace.is_cuda or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous CUDA tensor")
    else:
        _on_current_device(workspace=workspace)
    # strides along dimensions of one element are of no account
    if page_size == 1:
        row_stride = W
    if pages == 1:
        page_stride = page_size * row_stride
    if B == 1:
        ldt = table_width
    _call("sgemm_bf16_latent_attention", _ATTN.pack(
        q.data_ptr(), cache.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(), pcu, out.data_ptr(),
        plse, workspace.data_ptr(), q_token, q_head, row_stride, page_stride, ldt, out_token, out_head, lse_token,
        pages, workspace.nbytes, total, page_size, table_width, B, H, rank, W - rank, max_q, scale, flags, 0), q, stream)
    return out, lse
