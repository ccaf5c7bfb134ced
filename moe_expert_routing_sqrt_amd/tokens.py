"""The two ends of a training step on tokens: the embedding lookup with its
gradient, and losses on a vocabulary's logits with theirs (distillation from a
teacher's top logits, the clipped policy loss with a KL term), each one call into
the library."""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Tuple

import torch

from . import MOE_F32, _device_index, _dt, _lib, _stream, _ws_len, lib
from .training import _arg as _sized

_f32, _i32 = torch.float32, torch.int32


def _arg(t: Optional[torch.Tensor], numel: int, name: str, dtype: Optional[torch.dtype] = None) -> int:
    """The pointer of a tensor argument (0 for None): its size, type and layout are
    checked, and that it lives on the current device, whose stream the call uses."""
    p = _sized(t, numel, name, dtype)
    if t is not None and _device_index is not None and t.get_device() != _device_index():
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{_device_index()}")
    return p


# ---------------------------------------------------------------- embedding

def embedding(ids: torch.Tensor, table: torch.Tensor, scale: float = 1.0, out: Optional[torch.Tensor] = None,
              out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """Rows of table [V, d] by token id, times scale: [*ids.shape, d] in out_dtype
    (None: the table's).  Ids (int32) outside [0, V) give zeros."""
    V, d = table.shape
    T = ids.numel()
    i_p, t_p, o_p = _arg(ids, T, "ids", _i32), _arg(table, 0, "table"), _arg(out, T * d, "out")
    if out is None:
        out = table.new_empty((*ids.shape, d), dtype=out_dtype)
        o_p = out.data_ptr()
    st = lib().moe_embedding(T, V, d, i_p, t_p, _dt(table), scale, o_p, _dt(out), _stream())
    _lib.check("moe_embedding", st)
    return out


@functools.lru_cache(maxsize=1024)
def _embedding_ws_bytes(T: int, V: int, d: int) -> int:
    return lib().moe_embedding_backward_workspace_size(T, V, d)


def embedding_backward(d_out: torch.Tensor, ids: torch.Tensor, n_rows: int, scale: float = 1.0,
                       d_table: Optional[torch.Tensor] = None, dtype: torch.dtype = _f32, accumulate: bool = False,
                       ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The table's gradient [n_rows, d] for embedding's d_out [*ids.shape, d].
    accumulate: added to what d_table holds (a tied head's gradient, earlier
    micro-batches), else every row is written, in d_table or a new tensor of dtype."""
    d = d_out.shape[-1]
    T = ids.numel()
    i_p, y_p = _arg(ids, T, "ids", _i32), _arg(d_out, T * d, "d_out")
    t_p = _arg(d_table, n_rows * d, "d_table")
    if d_table is None:
        if accumulate:
            raise ValueError("accumulate needs d_table")
        d_table = d_out.new_empty((n_rows, d), dtype=dtype)
        t_p = d_table.data_ptr()
    if ws is None:
        ws = torch.empty(_embedding_ws_bytes(T, n_rows, d), dtype=torch.uint8, device=d_out.device)
    st = lib().moe_embedding_backward(T, n_rows, d, i_p, y_p, _dt(d_out), scale, t_p, _dt(d_table),
                                      1 if accumulate else 0, _arg(ws, 0, "ws"), _ws_len(ws), _stream())
    _lib.check("moe_embedding_backward", st)
    return d_table


# ---------------------------------------------------------------- losses on logits

def _grad_out(logits, with_grad, dlogits, grad_dtype):
    """(dlogits, its pointer, its type) of a loss that may form the gradient too"""
    n = logits.numel()
    if dlogits is None:
        if not with_grad:
            return None, 0, MOE_F32
        dlogits = torch.empty_like(logits, dtype=grad_dtype)
        return dlogits, dlogits.data_ptr(), _dt(dlogits)
    if grad_dtype is not None and dlogits.dtype is not grad_dtype:
        raise TypeError("dlogits must be of grad_dtype")
    return dlogits, _arg(dlogits, n, "dlogits"), _dt(dlogits)


def _row_outputs(logits, T, loss, row_loss, stats):
    """(tensor, pointer) of a loss's outputs, made where not given"""
    l_p, r_p, s_p = _arg(loss, 1, "loss", _f32), _arg(row_loss, T, "row_loss", _f32), _arg(stats, 2 * T, "stats", _f32)
    if loss is None:  # what is made here needs no check
        loss = logits.new_empty(1, dtype=_f32)
        l_p = loss.data_ptr()
    if row_loss is None:
        row_loss = logits.new_empty(T, dtype=_f32)
        r_p = row_loss.data_ptr()
    if stats is None:
        stats = logits.new_empty((T, 2), dtype=_f32)
        s_p = stats.data_ptr()
    return (loss, l_p), (row_loss, r_p), (stats, s_p)


def _size(logits) -> Tuple[int, int]:
    if logits.dim() < 2:
        raise ValueError("logits must be [..., V]")
    V = logits.shape[-1]
    return (logits.numel() // V if V else 0), V


def distill_loss(logits: torch.Tensor, idx: torch.Tensor, teacher: torch.Tensor, temperature: float = 1.0,
                 weight: Optional[torch.Tensor] = None, with_grad: bool = False,
                 grad_loss: Optional[torch.Tensor] = None, grad_dtype: Optional[torch.dtype] = None,
                 loss: Optional[torch.Tensor] = None, row_loss: Optional[torch.Tensor] = None,
                 stats: Optional[torch.Tensor] = None, dlogits: Optional[torch.Tensor] = None):
    """Distillation from a teacher's top logits: teacher [T, K] at the vocabulary's
    entries idx [T, K] (int32; outside [0, V): no entry), against logits [T, V].
    Returns (loss [1], row_loss [T], stats [T, 2], dlogits): the weighted sum of
    temperature^2 KL(teacher's top || student) over the rows (weight [T] fp32;
    None: their mean), and what distill_loss_backward needs.
    with_grad, or dlogits given (it may be logits itself): the gradient times
    grad_loss ([1] fp32 on the device; None: 1) from the same reading of the
    logits, in grad_dtype (None: the logits').  Else dlogits is None."""
    T, V = _size(logits)
    K = idx.shape[-1]
    x_p, i_p, t_p = _arg(logits, T * V, "logits"), _arg(idx, T * K, "idx", _i32), _arg(teacher, T * K, "teacher")
    w_p, g_p = _arg(weight, T, "weight", _f32), _arg(grad_loss, 1, "grad_loss", _f32)
    dlogits, d_p, d_t = _grad_out(logits, with_grad, dlogits, grad_dtype)
    (loss, l_p), (row_loss, r_p), (stats, s_p) = _row_outputs(logits, T, loss, row_loss, stats)
    st = lib().moe_distill_loss(T, V, K, x_p, _dt(logits), i_p, t_p, _dt(teacher), temperature, w_p, g_p, l_p, r_p, s_p,
                                d_p, d_t, _stream())
    _lib.check("moe_distill_loss", st)
    return loss, row_loss, stats, dlogits


def distill_loss_backward(logits: torch.Tensor, stats: torch.Tensor, idx: torch.Tensor, teacher: torch.Tensor,
                          temperature: float = 1.0, weight: Optional[torch.Tensor] = None,
                          grad_loss: Optional[torch.Tensor] = None, grad_dtype: Optional[torch.dtype] = None,
                          dlogits: Optional[torch.Tensor] = None) -> torch.Tensor:
    """distill_loss's gradient from the logits and its stats (dlogits must not be
    logits)."""
    T, V = _size(logits)
    K = idx.shape[-1]
    dlogits, d_p, d_t = _grad_out(logits, True, dlogits, grad_dtype)
    st = lib().moe_distill_loss_backward(T, V, K, _arg(logits, T * V, "logits"), _dt(logits),
                                         _arg(stats, 2 * T, "stats", _f32), _arg(idx, T * K, "idx", _i32),
                                         _arg(teacher, T * K, "teacher"), _dt(teacher), temperature,
                                         _arg(weight, T, "weight", _f32), _arg(grad_loss, 1, "grad_loss", _f32), d_p,
                                         d_t, _stream())
    _lib.check("moe_distill_loss_backward", st)
    return dlogits


def policy_loss(logits: torch.Tensor, tokens: torch.Tensor, old_logp: torch.Tensor, advantage: torch.Tensor,
                ref_logp: Optional[torch.Tensor] = None, clip: Tuple[float, float] = (0.2, 0.2), kl: float = 0.0,
                temperature: float = 1.0, weight: Optional[torch.Tensor] = None, with_grad: bool = False,
                grad_loss: Optional[torch.Tensor] = None, grad_dtype: Optional[torch.dtype] = None,
                loss: Optional[torch.Tensor] = None, row_loss: Optional[torch.Tensor] = None,
                logp: Optional[torch.Tensor] = None, stats: Optional[torch.Tensor] = None,
                dlogits: Optional[torch.Tensor] = None):
    """The clipped policy loss of tokens [T] (int32) under logits [T, V], with kl
    times the KL estimate exp(d) - d - 1, d = ref_logp - logp.  Returns (loss [1],
    row_loss [T], logp [T], stats [T, 2], dlogits).  clip: the ratio stays within
    [1 - clip[0], 1 + clip[1]].  Rows of weight 0 or with a token outside [0, V) do
    not count.  The rest as distill_loss."""
    T, V = _size(logits)
    x_p, i_p = _arg(logits, T * V, "logits"), _arg(tokens, T, "tokens", _i32)
    o_p, a_p = _arg(old_logp, T, "old_logp", _f32), _arg(advantage, T, "advantage", _f32)
    f_p, w_p = _arg(ref_logp, T, "ref_logp", _f32), _arg(weight, T, "weight", _f32)
    g_p, p_p = _arg(grad_loss, 1, "grad_loss", _f32), _arg(logp, T, "logp", _f32)
    dlogits, d_p, d_t = _grad_out(logits, with_grad, dlogits, grad_dtype)
    (loss, l_p), (row_loss, r_p), (stats, s_p) = _row_outputs(logits, T, loss, row_loss, stats)
    if logp is None:
        logp = logits.new_empty(T, dtype=_f32)
        p_p = logp.data_ptr()
    h = _lib.MoePolicyParams(temperature, clip[0], clip[1], kl)
    st = lib().moe_policy_loss(T, V, x_p, _dt(logits), i_p, o_p, a_p, f_p, ctypes.byref(h), w_p, g_p, l_p, r_p, p_p,
                               s_p, d_p, d_t, _stream())
    _lib.check("moe_policy_loss", st)
    return loss, row_loss, logp, stats, dlogits


def policy_loss_backward(logits: torch.Tensor, stats: torch.Tensor, tokens: torch.Tensor, old_logp: torch.Tensor,
                         advantage: torch.Tensor, ref_logp: Optional[torch.Tensor] = None,
                         clip: Tuple[float, float] = (0.2, 0.2), kl: float = 0.0, temperature: float = 1.0,
                         weight: Optional[torch.Tensor] = None, grad_loss: Optional[torch.Tensor] = None,
                         grad_dtype: Optional[torch.dtype] = None,
                         dlogits: Optional[torch.Tensor] = None) -> torch.Tensor:
    """policy_loss's gradient from the logits and its stats (dlogits must not be
    logits)."""
    T, V = _size(logits)
    dlogits, d_p, d_t = _grad_out(logits, True, dlogits, grad_dtype)
    h = _lib.MoePolicyParams(temperature, clip[0], clip[1], kl)
    st = lib().moe_policy_loss_backward(T, V, _arg(logits, T * V, "logits"), _dt(logits),
                                        _arg(stats, 2 * T, "stats", _f32), _arg(tokens, T, "tokens", _i32),
                                        _arg(old_logp, T, "old_logp", _f32), _arg(advantage, T, "advantage", _f32),
                                        _arg(ref_logp, T, "ref_logp", _f32), ctypes.byref(h),
                                        _arg(weight, T, "weight", _f32), _arg(grad_loss, 1, "grad_loss", _f32), d_p,
                                        d_t, _stream())
    _lib.check("moe_policy_loss_backward", st)
    return dlogits


def token_logp(logits: torch.Tensor, tokens: torch.Tensor, temperature: float = 1.0,
               logp: Optional[torch.Tensor] = None, stats: Optional[torch.Tensor] = None):
    """(logp [T], stats [T, 2]): the log-probabilities of tokens [T] (int32) under
    logits [T, V], 0 for tokens outside [0, V): a policy_loss's old_logp or ref_logp."""
    T, V = _size(logits)
    x_p, i_p = _arg(logits, T * V, "logits"), _arg(tokens, T, "tokens", _i32)
    l_p, s_p = _arg(logp, T, "logp", _f32), _arg(stats, 2 * T, "stats", _f32)
    if logp is None:
        logp = logits.new_empty(T, dtype=_f32)
        l_p = logp.data_ptr()
    if stats is None:
        stats = logits.new_empty((T, 2), dtype=_f32)
        s_p = stats.data_ptr()
    st = lib().moe_token_logp(T, V, x_p, _dt(logits), i_p, temperature, l_p, s_p, _stream())
    _lib.check("moe_token_logp", st)
    return logp, stats
