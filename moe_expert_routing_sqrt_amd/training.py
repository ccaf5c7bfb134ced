"""What a training step needs around the MoE layer: layer norm, the router's
balance loss and the AdamW step (each one call into the library), and MoEBlock,
which runs them with a MoELayer."""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Sequence, Tuple

import torch

from . import (MOE_E4M3, MOE_F32, MOE_FP8_TILE, MOE_OP_LAYER_NORM_BACKWARD, MoeShape, _dt, _lib, _need, _stream,
               _ws_len, lib, workspace_bytes)
from . import _ptr as _checked_ptr
from .layer import MoELayer

_f32, _i32, _u8 = torch.float32, torch.int32, torch.uint8


def _arg(t: Optional[torch.Tensor], numel: int, name: str, dtype: Optional[torch.dtype] = None) -> int:
    """The pointer of a tensor argument (0 for None) once its size, type, device
    and layout are checked."""
    if t is None:
        return 0
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {str(dtype)[6:]}")
    if t.numel() >= numel and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    _need(t, numel, name)
    return _checked_ptr(t)  # raises


# ---------------------------------------------------------------- layer norm

@functools.lru_cache(maxsize=1024)
def _norm_ws_floats(rows: int, d: int) -> int:
    return workspace_bytes(MOE_OP_LAYER_NORM_BACKWARD, MoeShape(rows, d, 1, 1, 1, 1, 1, 1)) // 4


def layer_norm(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
               residual: Optional[torch.Tensor] = None, eps: float = 1e-5, y_dtype: Optional[torch.dtype] = None,
               y: Optional[torch.Tensor] = None, sum_out: Optional[torch.Tensor] = None,
               mean: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None, keep_stats: bool = True):
    """Layer norm over the last dimension of x + residual.  Returns (y, s, mean,
    rstd): s is the sum (x itself without a residual), mean and rstd [rows] fp32
    what layer_norm_backward needs (None with keep_stats=False)."""
    d = x.shape[-1]
    n = x.numel()
    rows = n // d if d else 0
    dt = x.dtype
    if sum_out is not None and residual is None:
        raise ValueError("sum_out needs a residual")
    r_p, w_p, b_p = _arg(residual, n, "residual", dt), _arg(weight, d, "weight", _f32), _arg(bias, d, "bias", _f32)
    s_p, y_p = _arg(sum_out, n, "sum_out", dt), _arg(y, n, "y")
    m_p, i_p = _arg(mean, rows, "mean", _f32), _arg(rstd, rows, "rstd", _f32)
    if y is None:  # what is made here needs no check
        y = torch.empty_like(x) if y_dtype is None or y_dtype == dt else torch.empty_like(x, dtype=y_dtype)
        y_p = y.data_ptr()
    if residual is not None and sum_out is None:
        sum_out = torch.empty_like(x)
        s_p = sum_out.data_ptr()
    if keep_stats:
        if mean is None:
            mean = weight.new_empty(rows)
            m_p = mean.data_ptr()
        if rstd is None:
            rstd = weight.new_empty(rows)
            i_p = rstd.data_ptr()
    st = lib().moe_layer_norm(rows, d, _arg(x, n, "x"), r_p, _dt(x), w_p, b_p, eps, s_p, y_p, _dt(y), m_p, i_p,
                              _stream())
    _lib.check("moe_layer_norm", st)
    return y, x if residual is None else sum_out, mean, rstd


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, mean: torch.Tensor,
                        rstd: torch.Tensor, d_sum: Optional[torch.Tensor] = None,
                        dx: Optional[torch.Tensor] = None, dx_dtype: Optional[torch.dtype] = None,
                        dw: Optional[torch.Tensor] = None, db: Optional[torch.Tensor] = None,
                        ws: Optional[torch.Tensor] = None, has_bias: bool = True):
    """Gradients of layer_norm for dy: (dx, dw, db).  x: what was normalised
    (layer_norm's s).  d_sum: the gradient reaching s past the norm, added to
    dx, which is then the gradient of both of layer_norm's inputs.
    has_bias=False: no db (returned None)."""
    d = x.shape[-1]
    n = x.numel()
    rows = n // d if d else 0
    dt = x.dtype
    w_p, x_p = _arg(weight, d, "weight", _f32), _arg(x, n, "x")
    dx_p, dw_p, db_p = _arg(dx, n, "dx"), _arg(dw, d, "dw", _f32), _arg(db, d, "db", _f32)
    if dx is None:
        dx = torch.empty_like(x) if dx_dtype is None or dx_dtype == dt else torch.empty_like(x, dtype=dx_dtype)
        dx_p = dx.data_ptr()
    if dw is None:
        dw = torch.empty_like(weight)
        dw_p = dw.data_ptr()
    if db is None and has_bias:
        db = torch.empty_like(weight)
        db_p = db.data_ptr()
    need = 0 if ws is not None else _norm_ws_floats(rows, d)
    if need:
        ws = weight.new_empty(need)
    st = lib().moe_layer_norm_backward(rows, d, _arg(dy, n, "dy"), _dt(dy), x_p, _dt(x), w_p,
                                       _arg(mean, rows, "mean", _f32), _arg(rstd, rows, "rstd", _f32),
                                       _arg(d_sum, n, "d_sum", dt), dx_p, _dt(dx), dw_p, db_p, _arg(ws, 0, "ws"),
                                       _ws_len(ws), _stream())
    _lib.check("moe_layer_norm_backward", st)
    return dx, dw, db


# ---------------------------------------------------------------- balance loss

@functools.lru_cache(maxsize=1024)
def _loss_ws_floats(T: int, E: int, k: int, n: int) -> int:
    sh = MoeShape(T, 1, E, 1, 1, k, 1, 1)
    return lib().moe_balance_loss_workspace_size(ctypes.byref(sh), n) // 4


def _sequences(T: int, seq_offsets, token_mask):
    """(number of sequences, offsets pointer, mask pointer)"""
    if token_mask is not None and token_mask.dtype not in (torch.bool, _u8):
        raise TypeError("token_mask must be bool or uint8")
    n = 1 if seq_offsets is None else seq_offsets.numel() - 1
    return n, _arg(seq_offsets, 2, "seq_offsets", _i32), _arg(token_mask, T, "token_mask")


def balance_loss(sh: MoeShape, logits: torch.Tensor, idx: torch.Tensor, alpha: float,
                 seq_offsets: Optional[torch.Tensor] = None, token_mask: Optional[torch.Tensor] = None,
                 logit_offset: Optional[torch.Tensor] = None, loss: Optional[torch.Tensor] = None,
                 counts: Optional[torch.Tensor] = None, prob: Optional[torch.Tensor] = None,
                 dprob: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None):
    """The router's balance loss over the sequences of seq_offsets (int32 [n+1];
    None: all T tokens are one).  Returns (loss [1], counts [n, E] int32, prob
    [n, E], dprob [n, E]); dprob is what balance_loss_backward needs.
    Tokens outside the sequences or with token_mask 0 do not count."""
    T, E, k = sh.T, sh.E, sh.k
    if idx.dtype != _i32:
        raise TypeError("idx must be int32")
    n, off_p, mask_p = _sequences(T, seq_offsets, token_mask)
    m = n * E
    l_p, i_p = _arg(logits, T * E, "logits", _f32), _arg(idx, T * k, "idx")
    o_p = _arg(logit_offset, E, "logit_offset", _f32)
    loss_p, c_p = _arg(loss, 1, "loss", _f32), _arg(counts, m, "counts", _i32)
    p_p, d_p = _arg(prob, m, "prob", _f32), _arg(dprob, m, "dprob", _f32)
    if loss is None:  # what is made here needs no check
        loss = logits.new_empty(1)
        loss_p = loss.data_ptr()
    if counts is None:
        counts = idx.new_empty((n, E))
        c_p = counts.data_ptr()
    if prob is None:
        prob = logits.new_empty((n, E))
        p_p = prob.data_ptr()
    if dprob is None:
        dprob = torch.empty_like(prob)
        d_p = dprob.data_ptr()
    need = 0 if ws is not None else _loss_ws_floats(T, E, k, n)
    if need:
        ws = logits.new_empty(need)
    st = lib().moe_balance_loss(ctypes.byref(sh), l_p, o_p, i_p, off_p, n, mask_p, alpha, c_p, p_p, d_p, loss_p,
                                _arg(ws, 0, "ws"), _ws_len(ws), _stream())
    _lib.check("moe_balance_loss", st)
    return loss, counts, prob, dprob


def balance_loss_backward(sh: MoeShape, logits: torch.Tensor, dprob: torch.Tensor,
                          seq_offsets: Optional[torch.Tensor] = None, token_mask: Optional[torch.Tensor] = None,
                          logit_offset: Optional[torch.Tensor] = None, grad_loss: Optional[torch.Tensor] = None,
                          d_extra: Optional[torch.Tensor] = None,
                          dlogits: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dlogits [T, E] = d_extra + the balance loss's gradient times grad_loss
    ([1] fp32 on the device; None: 1).  dlogits may be d_extra."""
    T, E = sh.T, sh.E
    n, off_p, mask_p = _sequences(T, seq_offsets, token_mask)
    m = T * E
    out_p = _arg(dlogits, m, "dlogits", _f32)
    if dlogits is None:
        dlogits = logits.new_empty((T, E))
        out_p = dlogits.data_ptr()
    st = lib().moe_balance_loss_backward(ctypes.byref(sh), _arg(logits, m, "logits", _f32),
                                         _arg(logit_offset, E, "logit_offset", _f32), off_p, n, mask_p,
                                         _arg(dprob, n * E, "dprob", _f32), _arg(grad_loss, 1, "grad_loss", _f32),
                                         _arg(d_extra, m, "d_extra", _f32), out_p, _stream())
    _lib.check("moe_balance_loss_backward", st)
    return dlogits


# ---------------------------------------------------------------- AdamW

class AdamW:
    """AdamW over a list of tensors, one library call a step.

    params   fp32 or bf16 tensors, updated in place
    grads    the buffers their gradients are written to (fp32 or bf16); step()
             reads what they then hold
    master   fp32 weights of bf16 params (None per tensor: the param itself is
             the weight); "new": made from the params
    states   "f32", or "e4m3" (8 bits a moment and a scale per 128 elements);
             m, v, m_scale, v_scale given: continue from them
    weight_decay  one value, or one per tensor

    All tensors are held by reference and must stay what they are (pointers are
    taken once); state dicts are the lists m, v, m_scale, v_scale, master and
    step_count."""

    def __init__(self, params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], lr: float,
                 betas: Tuple[float, float] = (0.9, 0.999), eps: float = 1e-8, weight_decay=0.01, states: str = "f32",
                 master=None, m=None, v=None, m_scale=None, v_scale=None, step_count: int = 0):
        n = len(params)
        if len(grads) != n:
            raise ValueError("one gradient per parameter")
        if states not in ("f32", "e4m3"):
            raise ValueError("states must be 'f32' or 'e4m3'")
        if isinstance(master, str):
            if master != "new":
                raise ValueError("master must be 'new' or a list")
            master = [p.to(_f32) if p.dtype == torch.bfloat16 else None for p in params]
        wd = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else [weight_decay] * n

        def state(given, make):
            out = [make(p) for p in params] if given is None else list(given)
            if len(out) != n:
                raise ValueError("one state per parameter")
            return out

        code = torch.uint8 if states == "e4m3" else _f32
        tiles = lambda p: -(-p.numel() // MOE_FP8_TILE)  # noqa: E731
        self.params, self.grads = list(params), list(grads)
        self.master = [None] * n if master is None else list(master)
        self.m = state(m, lambda p: torch.zeros(p.numel(), dtype=code, device=p.device))
        self.v = state(v, lambda p: torch.zeros(p.numel(), dtype=code, device=p.device))
        eight = [_dt(t) == MOE_E4M3 for t in self.m]
        scale = lambda p, e: torch.ones(tiles(p), dtype=_f32, device=p.device) if e else None  # noqa: E731
        self.m_scale = [scale(p, e) for p, e in zip(params, eight)] if m_scale is None else list(m_scale)
        self.v_scale = [scale(p, e) for p, e in zip(params, eight)] if v_scale is None else list(v_scale)
        if not len(self.master) == len(self.m_scale) == len(self.v_scale) == len(wd) == n:
            raise ValueError("one master, scale and weight decay per parameter")
        self.lr, self.betas, self.eps, self.step_count = lr, betas, eps, step_count
        self._items = (_lib.MoeAdamwTensor * max(n, 1))()
        for i, p in enumerate(self.params):
            k = p.numel()
            if _dt(self.m[i]) != _dt(self.v[i]) or _dt(self.m[i]) not in (MOE_F32, MOE_E4M3):
                raise TypeError("m and v must both be fp32 or both 8-bit codes")
            for t, name in ((self.grads[i], "grad"), (self.m[i], "m"), (self.v[i], "v")):
                if t.numel() != k:
                    raise ValueError(f"{name} {i}: needs {k} elements, has {t.numel()}")
            self._items[i] = _lib.MoeAdamwTensor(
                k, _arg(p, k, "param"), _arg(self.grads[i], k, "grad"), _arg(self.master[i], k, "master", _f32),
                _arg(self.m[i], k, "m"), _arg(self.v[i], k, "v"),
                _arg(self.m_scale[i], tiles(p), "m_scale", _f32) if eight[i] else 0,
                _arg(self.v_scale[i], tiles(p), "v_scale", _f32) if eight[i] else 0,
                wd[i], _dt(p), _dt(self.grads[i]), _dt(self.m[i]), 0)

    def step(self, grad_scale: Optional[torch.Tensor] = None, lr: Optional[float] = None) -> None:
        """One step on what the gradient buffers hold, times grad_scale ([1]
        fp32 on the device).  lr: this step's rate (else the constructor's)."""
        h = _lib.MoeAdamwParams(self.lr if lr is None else lr, self.betas[0], self.betas[1], self.eps,
                                self.step_count + 1)
        st = lib().moe_adamw_step(len(self.params), self._items, ctypes.byref(h),
                                  _arg(grad_scale, 1, "grad_scale", _f32), _stream())
        _lib.check("moe_adamw_step", st)
        self.step_count += 1


# ---------------------------------------------------------------- the block

class MoEBlock:
    """A pre-norm MoE block that trains: stream' = stream + delta, h =
    norm(stream'), out = MoE(h), with a balance loss on the router.

    forward(delta, stream) returns (out, stream'): the next block adds them in
    its own norm, so no pass of its own is spent on the residual add.
    backward(d_out, d_stream, grad_loss) leaves the gradients of every weight in
    the block's buffers and returns the gradient of delta and stream.
    step() is the AdamW step on them.

    Whatever forward and backward leave or return (out, stream, loss, counts,
    prob, dprob, grads and the input's gradient) are buffers of the block that
    the next forward and backward write again: read or copy a value that is to
    be kept (losses.append(float(blk.loss)), or blk.loss.clone())."""

    def __init__(self, layer: MoELayer, norm_w: torch.Tensor, norm_b: torch.Tensor, eps: float = 1e-5,
                 alpha: float = 1e-3, lr: float = 3e-4, betas: Tuple[float, float] = (0.9, 0.95),
                 weight_decay: float = 0.1, states: str = "f32", master="new"):
        dev = layer.bias.device
        T, d = layer.T, layer.d
        self.layer, self.norm_w, self.norm_b, self.eps, self.alpha = layer, norm_w, norm_b, eps, alpha
        bf = torch.bfloat16
        self.stream = torch.empty((T, d), dtype=bf, device=dev)
        self.h = torch.empty((T, d), dtype=bf, device=dev)
        self.mean = torch.empty(T, dtype=_f32, device=dev)
        self.rstd = torch.empty(T, dtype=_f32, device=dev)
        self.dx = torch.empty((T, d), dtype=bf, device=dev)
        self.d_norm_w = torch.empty(d, dtype=_f32, device=dev)
        self.d_norm_b = torch.empty(d, dtype=_f32, device=dev)
        sh = layer.sh
        self.norm_ws = torch.empty(max(256, workspace_bytes(MOE_OP_LAYER_NORM_BACKWARD, sh)), dtype=torch.uint8,
                                   device=dev)
        self.opt_args = dict(lr=lr, betas=betas, states=states, weight_decay=weight_decay)
        self.master, self.opt = master, None
        # balance_loss's buffers by the number of sequences they hold, a power of two: what a captured graph
        # writes stays where it is, and there are at most 17 sets of them
        self._loss_bufs = {}

    def forward(self, delta: torch.Tensor, stream: torch.Tensor, seq_offsets: Optional[torch.Tensor] = None,
                token_mask: Optional[torch.Tensor] = None):
        self._rows(delta=delta, stream=stream)
        layer_norm(delta, self.norm_w, self.norm_b, residual=stream, eps=self.eps, y=self.h, sum_out=self.stream,
                   mean=self.mean, rstd=self.rstd)
        out = self.layer.forward(self.h, save_for_backward=True)
        la = self.layer
        self.seqs = (seq_offsets, token_mask)
        n = 1 if seq_offsets is None else seq_offsets.numel() - 1
        self.loss, self.counts, self.prob, self.dprob = balance_loss(
            la.sh, la.logits, la.idx, self.alpha, seq_offsets, token_mask, la.logit_offset, **self._loss_buffers(n))
        return out, self.stream

    def _rows(self, **tensors) -> None:
        """Every tensor has the layer's T rows of d: of fewer, the others would keep
        what an earlier call left in the block's buffers."""
        for name, t in tensors.items():
            if t is not None and t.numel() != self.layer.T * self.layer.d:
                raise ValueError(f"{name}: needs {self.layer.T} rows of {self.layer.d}, has shape {tuple(t.shape)}")

    def _loss_buffers(self, n: int) -> dict:
        if n > _lib.MOE_MAX_SEQUENCES:
            return {}  # refused by the call
        la, room = self.layer, min(1 << max(n - 1, 0).bit_length(), _lib.MOE_MAX_SEQUENCES)
        if room not in self._loss_bufs:
            new = la.logits.new_empty
            self._loss_bufs[room] = dict(loss=new(1), counts=new((room, la.E), dtype=_i32), prob=new((room, la.E)),
                                         dprob=new((room, la.E)),
                                         ws=new(max(1, _loss_ws_floats(la.T, la.E, la.k, room))))
        b = dict(self._loss_bufs[room])
        for name in ("counts", "prob", "dprob"):
            b[name] = b[name][:n]
        return b

    def backward(self, d_out: torch.Tensor, d_stream: Optional[torch.Tensor] = None,
                 grad_loss: Optional[torch.Tensor] = None) -> torch.Tensor:
        """grad_loss ([1] fp32 on the device; None: 1): the gradient of the balance
        loss, that is, the factor that d_out carries (a loss scale) and that
        step()'s grad_scale takes off again."""
        self._rows(d_out=d_out, d_stream=d_stream)
        la = self.layer
        dl = la._bwd_ws(d_out.device)["dlogits"]
        balance_loss_backward(la.sh, la.logits, self.dprob, *self.seqs, la.logit_offset, grad_loss, dlogits=dl)
        self.grads = la.backward(self.h, d_out, add_dlogits=True)
        layer_norm_backward(self.grads["dx"], self.stream, self.norm_w, self.mean, self.rstd, d_sum=d_stream,
                            dx=self.dx, dw=self.d_norm_w, db=self.d_norm_b, ws=self.norm_ws)
        return self.dx

    def step(self, grad_scale: Optional[torch.Tensor] = None) -> None:
        """AdamW on the norm, the router and all experts; the norm's weights do
        not decay.  The optimizer is made at the first step, when the layer's
        gradient buffers exist."""
        if self.opt is None:
            la, g = self.layer, self.grads
            pairs = [(self.norm_w, self.d_norm_w), (self.norm_b, self.d_norm_b), (la.w_gate, g["dw_gate"]),
                     (la.w13, g["dw13"]), (la.w2, g["dw2"])]
            if la.has_shared:
                pairs += [(la.sh_w13, g["dsh_w13"]), (la.sh_w2, g["dsh_w2"])]
            args = dict(self.opt_args)
            args["weight_decay"] = [0.0, 0.0] + [args["weight_decay"]] * (len(pairs) - 2)
            self.opt = AdamW([p for p, _ in pairs], [q for _, q in pairs], master=self.master, **args)
        self.opt.step(grad_scale)
