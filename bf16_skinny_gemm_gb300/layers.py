"""Binding of the operators that make whole layers of a step (``include/sgemm_layers.h``):

- :func:`sgemm_bf16_moe_route`, :func:`sgemm_bf16_moe_experts`: a mixture of experts for a few tokens,
- :func:`sgemm_bf16_latent_tree_attention`: latent attention for a tree of drafted tokens,
- :func:`sgemm_bf16_linear_step`, :func:`sgemm_bf16_linear_attention`: linear attention with a decay
  for each head, one token a sequence and whole prompts.

As in ``decode``: the functions check and marshal, every step of the computation runs in the
library's CUDA kernels, outputs and scratch may be given (nothing is allocated then), tensors are
on the current device, and the calls can be captured into a CUDA graph.
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
from .decode import _ATTN, _fn, _on_current_device, _raw, _shape, _strides

__all__ = [
    "sgemm_bf16_moe_route", "sgemm_bf16_moe_experts", "sgemm_moe_experts_workspace",
    "sgemm_bf16_latent_tree_attention", "sgemm_latent_tree_attention_workspace", "sgemm_bf16_linear_step", "sgemm_bf16_linear_attention",
    "sgemm_linear_attention_workspace", "SGEMM_ROUTE_SOFTMAX", "SGEMM_ROUTE_SIGMOID", "MOE_MAX_TOKENS",
]

SGEMM_ROUTE_SOFTMAX = 0
SGEMM_ROUTE_SIGMOID = 1
MOE_MAX_TOKENS = 128

# the argument structures of the header, field by field (natural alignment, no padding)
_ROUTE = struct.Struct("<5Q5q5ifIi")     # sgemm_moe_route_t
_EXPERTS = struct.Struct("<7Q9q5iI")     # sgemm_moe_experts_t
_STEP = struct.Struct("<7Q14q4ifI")      # sgemm_linear_step_t
_LINEAR = struct.Struct("<10Q16q4ifI")   # sgemm_linear_attention_t

_BF16 = torch.bfloat16
_SCORING = {"softmax": SGEMM_ROUTE_SOFTMAX, "sigmoid": SGEMM_ROUTE_SIGMOID}


class _None:
    """In place of the native module where there is none for this Python and torch."""

    def moe_route(self, *args):
        return -1

    moe_experts = latent_tree_attention = linear_step = linear_attention = moe_route


class _Unbound:
    """Stands in for it until the first call has loaded the library."""

    def _first(self, name, args):
        global _short
        lib = load()
        try:
            loader = importlib.machinery.ExtensionFileLoader("_marshal", marshal_path())
            module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_marshal", loader))
            loader.exec_module(module)
            module.bind_layers(*(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value for f in (
                "sgemm_bf16_moe_route", "sgemm_bf16_moe_experts", "sgemm_bf16_latent_tree_attention",
                "sgemm_bf16_linear_step", "sgemm_bf16_linear_attention")))
        except (ImportError, AttributeError) as e:
            warnings.warn(f"calls take longer than they need: {e}; build the module for this torch with "
                          "python -c 'import __graft_entry__ as g; g.build()'", RuntimeWarning, stacklevel=4)
            module = _None()
        _short = module
        return getattr(module, name)(*args)

    def moe_route(self, *args):
        return self._first("moe_route", args)

    def moe_experts(self, *args):
        return self._first("moe_experts", args)

    def latent_tree_attention(self, *args):
        return self._first("latent_tree_attention", args)

    def linear_step(self, *args):
        return self._first("linear_step", args)

    def linear_attention(self, *args):
        return self._first("linear_attention", args)


# The short way of a well-formed call with all its buffers given (native/marshal.cpp), as in decode:
# the call's status, or -1 for what the checks below have to look at.
_short = _Unbound()


def _call(name: str, args: bytes, t: torch.Tensor, stream, *more) -> None:
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(t.get_device())
    elif isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    status = _fn(name)(args, *more, ctypes.c_void_p(stream))
    if status:
        raise SgemmError(status, name)


def _scratch(workspace, need: int, device, stream):
    """The scratch of a call: (tensor, pointer, bytes)."""
    if workspace is None:
        workspace = _empty((need,), torch.uint8, device, stream, returned=False)
    elif not isinstance(workspace, torch.Tensor) or not workspace.is_cuda or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous CUDA tensor")
    else:
        _on_current_device(workspace=workspace)
    return workspace, workspace.data_ptr(), workspace.nbytes


# ------------------------------------------------------------------------------ mixture of experts
def sgemm_bf16_moe_route(x: torch.Tensor, w: torch.Tensor, k: int, bias: torch.Tensor | None = None,
                         scoring: str = "softmax", renormalize: bool = True, scale: float = 1.0,
                         ids: torch.Tensor | None = None, weights: torch.Tensor | None = None,
                         flags: int = 0, stream=None):
    """The ``k`` experts of each token and their weights; returns ``(ids, weights)``.

    x: BF16 [T, D]; w: BF16 [E, D], the router's rows; the scores are the softmax over all experts or
    the sigmoid (``scoring``) of ``x @ w.T`` (FP32).  Chosen are the experts of the largest score
    (plus ``bias``, FP32 [E], which counts for the choice only), the largest first, the lower index
    of equal ones.  ids: int32 [T, k]; weights: FP32 [T, k], the chosen scores (divided by their sum
    with ``renormalize``) times ``scale``.  Both may be columns of wider arrays."""
    status = _short.moe_route(x, w, k, bias, _SCORING.get(scoring), renormalize, scale, ids, weights, flags, _raw(stream))
    if status == 0:
        return ids, weights
    if status > 0:
        raise SgemmError(status, "sgemm_bf16_moe_route")
    T, D = _shape(x, "x", _BF16, 2)
    E = _shape(w, "w", _BF16, 2)[0]
    if scoring not in _SCORING:
        raise ValueError(f"scoring must be 'softmax' or 'sigmoid', got {scoring!r}")
    ldx = _strides(x, "x", _BF16, (T, D))[0]
    ldw = _strides(w, "w", _BF16, (E, D))[0]
    pb = 0
    if bias is not None:
        _strides(bias, "bias", torch.float32, (E,))
        pb = bias.data_ptr()
    if ids is None:
        ids = _empty((T, k), torch.int32, x.device, stream)
    if weights is None:
        weights = _empty((T, k), torch.float32, x.device, stream)
    ldi = _strides(ids, "ids", torch.int32, (T, k))[0]
    ldwt = _strides(weights, "weights", torch.float32, (T, k))[0]
    _on_current_device(x=x, w=w, bias=bias, ids=ids, weights=weights)
    if T <= 1:
        if T == 0:
            return ids, weights
        ldx, ldi, ldwt = -(-D // 8) * 8, k, k  # the row stride of a single row is of no account
    if E == 1:
        ldw = -(-D // 8) * 8
    _call("sgemm_bf16_moe_route", _ROUTE.pack(
        x.data_ptr(), w.data_ptr(), pb, ids.data_ptr(), weights.data_ptr(), ldx, ldw, ldi, ldwt, T, D, E, k,
        _SCORING[scoring], 1 if renormalize else 0, scale, flags, 0), x, stream)
    return ids, weights


def sgemm_moe_experts_workspace(tokens: int, experts: int, k: int, hidden: int, width: int) -> int:
    """Bytes of scratch :func:`sgemm_bf16_moe_experts` needs for ``tokens`` tokens of ``hidden``
    elements, ``k`` entries each, and ``experts`` experts of ``width`` elements."""
    n = ctypes.c_longlong(0)
    args = _EXPERTS.pack(*([0] * 16), tokens, hidden, width, experts, k, 0)
    status = _fn("sgemm_moe_experts_workspace")(args, ctypes.addressof(n))
    if status:
        raise SgemmError(status, "sgemm_moe_experts_workspace")
    return n.value


def sgemm_bf16_moe_experts(x: torch.Tensor, w_gate_up: torch.Tensor, w_down: torch.Tensor, ids: torch.Tensor,
                           weights: torch.Tensor, y: torch.Tensor | None = None,
                           workspace: torch.Tensor | None = None, flags: int = 0, stream=None) -> torch.Tensor:
    """``y[t] = sum_j weights[t, j] * (silu(x[t] @ g.T) * (x[t] @ u.T)) @ d.T`` with the gate, up and
    down matrices g, u, d of expert ``ids[t, j]`` (a negative id: none); returns y.

    x, y: BF16 [T, D], T <= ``MOE_MAX_TOKENS``; w_gate_up: BF16 [E, 2 F, D], a gate's rows before its
    up rows; w_down: BF16 [E, D, F]; ids: int32 [T, k]; weights: FP32 [T, k].  ``workspace``: scratch
    on the device (:func:`sgemm_moe_experts_workspace` bytes; allocated for the call where None)."""
    status = _short.moe_experts(x, w_gate_up, w_down, ids, weights, y, workspace, flags, _raw(stream))
    if status == 0:
        return y
    if status > 0:
        raise SgemmError(status, "sgemm_bf16_moe_experts")
    T, D = _shape(x, "x", _BF16, 2)
    E, F2, _ = _shape(w_gate_up, "w_gate_up", _BF16, 3)
    k = _shape(ids, "ids", torch.int32, 2)[1]
    if F2 % 2:
        raise ValueError(f"w_gate_up must have an even number of rows (gate, up), got {F2}")
    F = F2 // 2
    ldx = _strides(x, "x", _BF16, (T, D))[0]
    gu_expert, gu_row, _ = _strides(w_gate_up, "w_gate_up", _BF16, (E, F2, D))
    dn_expert, dn_row, _ = _strides(w_down, "w_down", _BF16, (E, D, F))
    ldi = _strides(ids, "ids", torch.int32, (T, k))[0]
    ldwt = _strides(weights, "weights", torch.float32, (T, k))[0]
    if y is None:
        y = _empty((T, D), _BF16, x.device, stream)
    ldy = _strides(y, "y", _BF16, (T, D))[0]
    _on_current_device(x=x, w_gate_up=w_gate_up, w_down=w_down, ids=ids, weights=weights, y=y)
    if T == 0:
        return y
    # strides along dimensions of one element are of no account
    if T == 1:
        ldx, ldi, ldwt, ldy = -(-D // 8) * 8, k, k, D
    if E == 1:
        gu_expert, dn_expert = F2 * gu_row, D * dn_row
    need = 0 if workspace is not None else sgemm_moe_experts_workspace(T, E, k, D, F)
    workspace, pws, nws = _scratch(workspace, need, x.device, stream)
    _call("sgemm_bf16_moe_experts", _EXPERTS.pack(
        x.data_ptr(), w_gate_up.data_ptr(), w_down.data_ptr(), ids.data_ptr(), weights.data_ptr(), y.data_ptr(), pws,
        ldx, gu_expert, gu_row, dn_expert, dn_row, ldi, ldwt, ldy, nws, T, D, F, E, k, flags), x, stream)
    return y


# -------------------------------------------------------------------- attention for drafted tokens
def sgemm_latent_tree_attention_workspace(batch: int, heads: int, rank: int, rope: int, page_size: int,
                                          table_width: int, max_q: int = 1) -> int:
    """Bytes of scratch :func:`sgemm_bf16_latent_tree_attention` needs for such a call (at most
    ``LATENT_WORKSPACE_MAX``)."""
    n = ctypes.c_longlong(0)
    args = _ATTN.pack(*([0] * 16), 1, 0, min(batch * max_q, 1), page_size, table_width, batch, heads, rank, rope, max_q,
                      1.0, 0, 0)
    status = _fn("sgemm_latent_tree_attention_workspace")(args, ctypes.addressof(n))
    if status:
        raise SgemmError(status, "sgemm_latent_tree_attention_workspace")
    return n.value


def sgemm_bf16_latent_tree_attention(q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor,
                                     seq_lens: torch.Tensor, rank: int, scale: float, tree: torch.Tensor,
                                     cu_q: torch.Tensor | None = None, max_q: int = 1,
                                     out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                                     workspace: torch.Tensor | None = None, flags: int = 0, stream=None):
    """:func:`sgemm_bf16_latent_attention` whose new tokens are drafts that see one another by a mask;
    returns ``(out, lse)``.

    ``tree``: int64 [total_q, words], a token's mask in words of 64 bits: token i of a sequence's n
    new ones sees the ``seq_lens - n`` rows before them, and new token j's row where bit ``j % 64`` of
    word ``j // 64`` is set (for a tree: its ancestors and itself).  At most 64 * words new tokens a
    sequence.  A token that sees nothing gets zeros (and -inf).  All else is as there."""
    status = _short.latent_tree_attention(q, cache, block_table, seq_lens, rank, scale, cu_q, max_q, out, lse, workspace, flags,
                                          _raw(stream), tree)
    if status == 0:
        return out, lse
    if status > 0:
        raise SgemmError(status, "sgemm_bf16_latent_tree_attention")
    total, H, W = shape = _shape(q, "q", _BF16, 3)
    pages, page_size, width = _shape(cache, "cache", _BF16, 3)
    B, table_width = _shape(block_table, "block_table", torch.int32, 2)
    words = _shape(tree, "tree", torch.int64, 2)[1]
    if width != W:
        raise ValueError(f"cache rows must be as wide as q's ({W}), got {width}")
    q_token, q_head, _ = _strides(q, "q", _BF16, shape)
    page_stride, row_stride, _ = _strides(cache, "cache", _BF16, (pages, page_size, W))
    ldt = _strides(block_table, "block_table", torch.int32, (B, table_width))[0]
    _strides(seq_lens, "seq_lens", torch.int32, (B,))
    ld_tree = _strides(tree, "tree", torch.int64, (total, words))[0]
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
    _on_current_device(q=q, cache=cache, block_table=block_table, seq_lens=seq_lens, tree=tree, cu_q=cu_q, out=out, lse=lse)
    if total == 0 or B == 0:
        return out, lse
    need = 0 if workspace is not None else sgemm_latent_tree_attention_workspace(B, H, rank, W - rank, page_size, table_width, max_q)
    workspace, pws, nws = _scratch(workspace, need, q.device, stream)
    # strides along dimensions of one element are of no account
    if page_size == 1:
        row_stride = W
    if pages == 1:
        page_stride = page_size * row_stride
    if B == 1:
        ldt = table_width
    if total == 1:
        ld_tree = words
    _call("sgemm_bf16_latent_tree_attention", _ATTN.pack(
        q.data_ptr(), cache.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(), pcu, out.data_ptr(), plse, pws,
        q_token, q_head, row_stride, page_stride, ldt, out_token, out_head, lse_token,
        pages, nws, total, page_size, table_width, B, H, rank, W - rank, max_q, scale, flags, 0), q, stream,
        ctypes.c_void_p(tree.data_ptr()), ctypes.c_longlong(ld_tree), ctypes.c_int(words))
    return out, lse


# -------------------------------------------------------------------------------- linear attention
def _linear(q, k, v, g, state, out, stream):
    """Checks that both forms share: (sizes, pointers' tensors, strides, out)."""
    N, Hk, Dk = _shape(q, "q", _BF16, 3)
    _, Hv, Dv = _shape(v, "v", _BF16, 3)
    slots = _shape(state, "state", torch.float32, 4)[0]
    s = [*_strides(q, "q", _BF16, (N, Hk, Dk))[:2], *_strides(k, "k", _BF16, (N, Hk, Dk))[:2],
         *_strides(v, "v", _BF16, (N, Hv, Dv))[:2]]
    if tuple(_shape(g, "g", torch.float32, 2)) != (N, Hv) or not g.is_cuda:
        raise ValueError(f"g must be a float32 [{N}, {Hv}] CUDA tensor, got {list(g.shape)}")
    s += g.stride()
    sizes = tuple(state.shape)
    ss = _strides(state, "state", torch.float32, (slots, Hv, Dk, Dv))
    if ss[2] != Dv:
        raise ValueError(f"state must hold dense [{Dk}, {Dv}] matrices, got {sizes} with strides {tuple(ss)}")
    s += ss[:2]
    if out is None:
        out = _empty((N, Hv, Dv), _BF16, q.device, stream)
    s += _strides(out, "out", _BF16, (N, Hv, Dv))[:2]
    # strides along dimensions of one element are of no account
    if N == 1:
        s[0] = s[2] = s[4] = s[6] = s[10] = 0
    if Hk == 1:
        s[1] = s[3] = 0
    if Hv == 1:
        s[5] = s[7] = s[9] = s[11] = 0
    if slots == 1:
        s[8] = 0
    return (N, slots, Hk, Hv, Dk, Dv), s, out


def sgemm_bf16_linear_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, state: torch.Tensor,
                           slots: torch.Tensor, scale: float = 1.0, out: torch.Tensor | None = None,
                           flags: int = 0, stream=None) -> torch.Tensor:
    """One token of each sequence through linear attention with a decay for each head; returns out.

    q, k: BF16 [B, Hk, Dk]; v, out: BF16 [B, Hv, Dv], Hv a multiple of Hk (value head h reads key head
    ``h // (Hv // Hk)``), Dk and Dv 64 or 128; g: FP32 [B, Hv], logarithms of the decays (strides of
    0 allowed); state: FP32 [slots, Hv, Dk, Dv]; slots: int64 [B], each sequence's state (negative:
    a padded sequence, whose out is 0).  In place, ``S = exp(g) S + k v^T``; ``out = scale * q^T S``."""
    status = _short.linear_step(q, k, v, g, state, slots, scale, out, flags, _raw(stream))
    if status == 0:
        return out
    if status > 0:
        raise SgemmError(status, "sgemm_bf16_linear_step")
    (B, pool, Hk, Hv, Dk, Dv), s, out = _linear(q, k, v, g, state, out, stream)
    _strides(slots, "slots", torch.int64, (B,))
    _on_current_device(q=q, k=k, v=v, g=g, state=state, slots=slots, out=out)
    if B == 0:
        return out
    _call("sgemm_bf16_linear_step", _STEP.pack(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), state.data_ptr(), slots.data_ptr(), out.data_ptr(),
        *s, B, pool, Hk, Hv, Dk, Dv, scale, flags), q, stream)
    return out


def sgemm_linear_attention_workspace(tokens: int, batch: int, heads: int, key_width: int, value_width: int) -> int:
    """Bytes of scratch :func:`sgemm_bf16_linear_attention` needs for ``tokens`` tokens in ``batch``
    sequences with ``heads`` value heads."""
    n = ctypes.c_longlong(0)
    args = _LINEAR.pack(*([0] * 22), tokens, batch, 0, 0, 1, heads, key_width, value_width, 1.0, 0)
    status = _fn("sgemm_linear_attention_workspace")(args, ctypes.addressof(n))
    if status:
        raise SgemmError(status, "sgemm_linear_attention_workspace")
    return n.value


def sgemm_bf16_linear_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, state: torch.Tensor,
                                slots: torch.Tensor, cu: torch.Tensor, scale: float = 1.0,
                                fresh: torch.Tensor | None = None, out: torch.Tensor | None = None,
                                workspace: torch.Tensor | None = None, flags: int = 0, stream=None) -> torch.Tensor:
    """Whole sequences through linear attention with a decay for each head, in chunks; returns out.

    q, k: BF16 [N, Hk, Dk]; v, out: BF16 [N, Hv, Dv]; g: FP32 [N, Hv]; state: FP32 [slots, Hv, Dk, Dv],
    as for :func:`sgemm_bf16_linear_step`, whose recurrence this is.  Sequence b has the tokens
    ``cu[b] .. cu[b + 1] - 1`` (cu: int32 [B + 1]), starts from ``state[slots[b]]`` (from zeros where
    ``fresh[b]``, int32 [B], is not 0) and leaves its last state there (slots: int64 [B]; negative:
    from zeros, not kept).  ``workspace``: scratch on the device
    (:func:`sgemm_linear_attention_workspace` bytes; allocated for the call where None)."""
    status = _short.linear_attention(q, k, v, g, state, slots, cu, scale, fresh, out, workspace, flags, _raw(stream))
    if status == 0:
        return out
    if status > 0:
        raise SgemmError(status, "sgemm_bf16_linear_attention")
    (N, pool, Hk, Hv, Dk, Dv), s, out = _linear(q, k, v, g, state, out, stream)
    B = _shape(slots, "slots", torch.int64, 1)[0]
    _strides(slots, "slots", torch.int64, (B,))
    _strides(cu, "cu", torch.int32, (B + 1,))
    pf = 0
    if fresh is not None:
        _strides(fresh, "fresh", torch.int32, (B,))
        pf = fresh.data_ptr()
    _on_current_device(q=q, k=k, v=v, g=g, state=state, slots=slots, cu=cu, fresh=fresh, out=out)
    if B == 0:
        return out
    need = 0 if workspace is not None else sgemm_linear_attention_workspace(N, B, Hv, Dk, Dv)
    workspace, pws, nws = _scratch(workspace, need, q.device, stream)
    _call("sgemm_bf16_linear_attention", _LINEAR.pack(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), state.data_ptr(), slots.data_ptr(), cu.data_ptr(), pf,
        out.data_ptr(), pws, *s, N, B, pool, nws, Hk, Hv, Dk, Dv, scale, flags), q, stream)
    return out
