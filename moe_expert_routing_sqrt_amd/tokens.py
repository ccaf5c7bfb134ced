"""The two ends of a training step on tokens: the embedding lookup with its
gradient, and losses on a vocabulary's logits with theirs (distillation from a
teacher's top logits, the clipped policy loss with a KL term), each one call into
the library; and TokenModel, which runs them around a MoEBlock."""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Tuple

import torch

from . import MOE_F32, MOE_OP_LAYER_NORM_BACKWARD, _device_index, _dt, _lib, _stream, _ws_len, lib, workspace_bytes
from .training import AdamW, MoEBlock, layer_norm, layer_norm_backward
from .training import _arg as _sized

_f32, _i32 = torch.float32, torch.int32


def _arg(t: Optional[torch.Tensor], numel: Optional[int], name: str, dtype: Optional[torch.dtype] = None) -> int:
    """The pointer of a tensor argument (0 for None): its size (exactly numel; None:
    any), type and layout are checked, and that it lives on the current device, whose
    stream the call uses."""
    if t is None:
        return 0
    on = t.get_device()
    if (dtype is None or t.dtype is dtype) and on >= 0 and (numel is None or t.numel() == numel) and t.is_contiguous():
        if _device_index is None or on == _device_index():
            return t.data_ptr()
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{_device_index()}")
    if numel is not None and t.numel() != numel and (dtype is None or t.dtype is dtype):
        raise ValueError(f"{name}: needs {numel} elements, has {t.numel()}")
    return _sized(t, 0, name, dtype)  # raises


# ---------------------------------------------------------------- embedding

def embedding(ids: torch.Tensor, table: torch.Tensor, scale: float = 1.0, out: Optional[torch.Tensor] = None,
              out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """Rows of table [V, d] by token id, times scale: [*ids.shape, d] in out_dtype
    (None: the table's).  Ids (int32) outside [0, V) give zeros."""
    if out is not None and out_dtype is not None and out.dtype is not out_dtype:
        raise TypeError("out must be of out_dtype")
    V, d = table.shape
    T = ids.numel()
    i_p, t_p, o_p = _arg(ids, T, "ids", _i32), _arg(table, None, "table"), _arg(out, T * d, "out")
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
                       d_table: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None,
                       accumulate: bool = False, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The table's gradient [n_rows, d] for embedding's d_out [*ids.shape, d].
    accumulate: added to what d_table holds (a tied head's gradient, earlier
    micro-batches), else every row is written, in d_table or a new tensor of dtype
    (None: fp32)."""
    if d_table is not None and dtype is not None and d_table.dtype is not dtype:
        raise TypeError("d_table must be of dtype")
    if accumulate and d_table is None:
        raise ValueError("accumulate needs d_table")
    d = d_out.shape[-1]
    T = ids.numel()
    i_p, y_p = _arg(ids, T, "ids", _i32), _arg(d_out, T * d, "d_out")
    t_p = _arg(d_table, n_rows * d, "d_table")
    if d_table is None:
        d_table = d_out.new_empty((n_rows, d), dtype=_f32 if dtype is None else dtype)
        t_p = d_table.data_ptr()
    if ws is None:
        ws = torch.empty(_embedding_ws_bytes(T, n_rows, d), dtype=torch.uint8, device=d_out.device)
    st = lib().moe_embedding_backward(T, n_rows, d, i_p, y_p, _dt(d_out), scale, t_p, _dt(d_table),
                                      1 if accumulate else 0, _arg(ws, None, "ws"), _ws_len(ws), _stream())
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


def _row_outputs(logits, T, loss, row_loss, stats, logp=None, want_logp=False):
    """[(tensor, pointer)] of a loss's outputs loss, row_loss, stats and logp, made
    where not given (all of them: in one allocation)"""
    if loss is row_loss is stats is logp is None:
        made = logits.new_empty((4 if want_logp else 3) * T + 1, dtype=_f32)
        at = made.data_ptr()
        if want_logp:
            stats, row_loss, logp, loss = made.split_with_sizes((2 * T, T, T, 1))
        else:
            stats, row_loss, loss = made.split_with_sizes((2 * T, T, 1))
        return (loss, at + (16 if want_logp else 12) * T), (row_loss, at + 8 * T), (stats.view(T, 2), at), \
            (logp, at + 12 * T if want_logp else 0)
    if loss is None:
        loss = logits.new_empty(1, dtype=_f32)
    if row_loss is None:
        row_loss = logits.new_empty(T, dtype=_f32)
    if stats is None:
        stats = logits.new_empty((T, 2), dtype=_f32)
    if logp is None and want_logp:
        logp = logits.new_empty(T, dtype=_f32)
    return (loss, _arg(loss, 1, "loss", _f32)), (row_loss, _arg(row_loss, T, "row_loss", _f32)), \
        (stats, _arg(stats, 2 * T, "stats", _f32)), (logp, _arg(logp, T, "logp", _f32))


def _size(logits) -> Tuple[int, int]:
    if logits.dim() < 2:
        raise ValueError("logits must be [..., V]")
    V = logits.shape[-1]
    return (logits.numel() // V if V else 0), V


def _entries(idx, teacher) -> int:
    """The entries of a row, of which idx and teacher have the same number"""
    K = idx.shape[-1] if idx.dim() else 0
    if teacher.dim() == 0 or teacher.shape[-1] != K:
        raise ValueError(f"teacher: needs rows of {K}, as idx has, has shape {tuple(teacher.shape)}")
    return K


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
    K = _entries(idx, teacher)
    x_p, i_p, t_p = _arg(logits, T * V, "logits"), _arg(idx, T * K, "idx", _i32), _arg(teacher, T * K, "teacher")
    w_p, g_p = _arg(weight, T, "weight", _f32), _arg(grad_loss, 1, "grad_loss", _f32)
    dlogits, d_p, d_t = _grad_out(logits, with_grad, dlogits, grad_dtype)
    (loss, l_p), (row_loss, r_p), (stats, s_p), _ = _row_outputs(logits, T, loss, row_loss, stats)
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
    K = _entries(idx, teacher)
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
    g_p = _arg(grad_loss, 1, "grad_loss", _f32)
    dlogits, d_p, d_t = _grad_out(logits, with_grad, dlogits, grad_dtype)
    (loss, l_p), (row_loss, r_p), (stats, s_p), (logp, p_p) = _row_outputs(logits, T, loss, row_loss, stats, logp, True)
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


# ---------------------------------------------------------------- the model

class TokenModel:
    """Token ids to logits around a MoEBlock, for training:

        stream = scale table[ids],  delta = positions[pos]
        out, stream = block(delta, stream),  y = norm(out + stream)
        logits = y table^T

    The table is tied: its gradient (fp32) is the head's, onto which the lookup's is
    accumulated.  table [V, d] and positions [P, d] are bf16; scale None: sqrt(d).
    forward(ids, pos) returns logits [T, V] (bf16); a loss leaves their gradient
    (dlogits=logits writes it over them); backward(dlogits) leaves every weight's
    gradient; step() is the AdamW step on all of them, the block's included.

    forward keeps copies of ids and pos for backward; seq_offsets and token_mask must
    stay as they are until then.  What forward and backward leave or return are buffers
    of the model (and of the block) that the next call writes again.  The products with the table are plain
    library ones."""

    def __init__(self, block: MoEBlock, table: torch.Tensor, positions: torch.Tensor, norm_w: torch.Tensor,
                 norm_b: torch.Tensor, scale: Optional[float] = None, eps: float = 1e-5, master="block"):
        la = block.layer
        T, d, V, P = la.T, la.d, table.shape[0], positions.shape[0]
        if table.shape[1] != d or positions.shape[1] != d:
            raise ValueError(f"table and positions need rows of {d}")
        self.block, self.table, self.positions, self.norm_w, self.norm_b = block, table, positions, norm_w, norm_b
        self.scale, self.eps = d ** 0.5 if scale is None else scale, eps
        new = lambda *s, dt=torch.bfloat16: torch.empty(s, dtype=dt, device=table.device)  # noqa: E731
        self.stream, self.delta, self.sum, self.y, self.dy, self.dx = (new(T, d) for _ in range(6))
        self.logits = new(T, V)
        self.ids, self.pos = new(T, dt=_i32), new(T, dt=_i32)
        self.mean, self.rstd = new(T, dt=_f32), new(T, dt=_f32)
        self.d_table, self.d_positions = new(V, d, dt=_f32), new(P, d, dt=_f32)
        self.d_norm_w, self.d_norm_b = new(d, dt=_f32), new(d, dt=_f32)
        self.norm_ws = new(max(256, workspace_bytes(MOE_OP_LAYER_NORM_BACKWARD, la.sh)), dt=torch.uint8)
        self.table_ws = new(_embedding_ws_bytes(T, V, d), dt=torch.uint8)
        self.positions_ws = new(_embedding_ws_bytes(T, P, d), dt=torch.uint8)
        self.opt = None
        if isinstance(master, str) and master == "block":  # its list holds the block's weights only
            master = block.master if block.master is None or isinstance(block.master, str) else "new"
        self.master = master

    def forward(self, ids: torch.Tensor, pos: torch.Tensor, seq_offsets: Optional[torch.Tensor] = None,
                token_mask: Optional[torch.Tensor] = None) -> torch.Tensor:
        T = self.block.layer.T
        for name, t, kept in (("ids", ids, self.ids), ("pos", pos, self.pos)):
            _arg(t, T, name, _i32)
            kept.copy_(t.view(T))
        embedding(self.ids, self.table, self.scale, out=self.stream)
        embedding(self.pos, self.positions, out=self.delta)
        out, stream = self.block.forward(self.delta, self.stream, seq_offsets, token_mask)
        layer_norm(out, self.norm_w, self.norm_b, residual=stream, eps=self.eps, y=self.y, sum_out=self.sum,
                   mean=self.mean, rstd=self.rstd)
        return torch.mm(self.y, self.table.t(), out=self.logits)

    def backward(self, dlogits: torch.Tensor, grad_loss: Optional[torch.Tensor] = None) -> None:
        """dlogits [T, V] bf16; grad_loss: the balance loss's factor, as
        MoEBlock.backward's."""
        if dlogits.shape != self.logits.shape or dlogits.dtype != torch.bfloat16:
            raise ValueError(f"dlogits: needs bf16 {tuple(self.logits.shape)}")
        torch.mm(dlogits.t(), self.y, out_dtype=_f32, out=self.d_table)
        torch.mm(dlogits, self.table, out=self.dy)
        layer_norm_backward(self.dy, self.sum, self.norm_w, self.mean, self.rstd, dx=self.dx, dw=self.d_norm_w,
                            db=self.d_norm_b, ws=self.norm_ws)
        dx = self.block.backward(self.dx, self.dx, grad_loss)
        embedding_backward(dx, self.ids, self.table.shape[0], self.scale, d_table=self.d_table, accumulate=True,
                           ws=self.table_ws)
        embedding_backward(dx, self.pos, self.positions.shape[0], d_table=self.d_positions, ws=self.positions_ws)

    def step(self, grad_scale: Optional[torch.Tensor] = None) -> None:
        """AdamW on the table, the positions, the norm and the block; the norm and the
        positions do not decay."""
        if self.opt is None:
            args = dict(self.block.opt_args)
            args["weight_decay"] = [args["weight_decay"], 0.0, 0.0, 0.0]
            self.opt = AdamW([self.table, self.positions, self.norm_w, self.norm_b],
                             [self.d_table, self.d_positions, self.d_norm_w, self.d_norm_b], master=self.master, **args)
        self.opt.step(grad_scale)
        self.block.step(grad_scale)
