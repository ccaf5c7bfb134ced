"""What a training step needs around the MoE layer: layer norm, the router's
balance loss and the AdamW step (each one call into the library), and MoEBlock,
which runs them with a MoELayer."""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence, Tuple

import torch

from . import (MOE_E4M3, MOE_F32, MOE_FP8_TILE, MOE_OP_LAYER_NORM_BACKWARD, MoeShape, _dt, _lib, _need, _ptr,
               _stream, _ws_len, lib, workspace_bytes)
from .layer import MoELayer

_f32 = torch.float32


def _need_f32(t: Optional[torch.Tensor], numel: int, name: str):
    if t is not None and t.dtype != _f32:
        raise TypeError(f"{name} must be fp32")
    _need(t, numel, name)


# ---------------------------------------------------------------- layer norm

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
    dev = x.device
    if residual is not None and residual.dtype != x.dtype:
        raise TypeError("residual must have x's dtype")
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype if y_dtype is None else y_dtype, device=dev)
    if residual is not None and sum_out is None:
        sum_out = torch.empty_like(x)
    if sum_out is not None and (residual is None or sum_out.dtype != x.dtype):
        raise ValueError("sum_out needs a residual and x's dtype")
    if keep_stats and mean is None:
        mean = torch.empty(rows, dtype=_f32, device=dev)
    if keep_stats and rstd is None:
        rstd = torch.empty(rows, dtype=_f32, device=dev)
    _need(residual, n, "residual")
    _need(sum_out, n, "sum_out")
    _need(y, n, "y")
    _need_f32(weight, d, "weight")
    _need_f32(bias, d, "bias")
    _need_f32(mean, rows, "mean")
    _need_f32(rstd, rows, "rstd")
    st = lib().moe_layer_norm(rows, d, _ptr(x), _ptr(residual), _dt(x), _ptr(weight), _ptr(bias), eps, _ptr(sum_out),
                              _ptr(y), _dt(y), _ptr(mean), _ptr(rstd), _stream())
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
    dev = x.device
    if d_sum is not None and d_sum.dtype != x.dtype:
        raise TypeError("d_sum must have x's dtype")
    if dx is None:
        dx = torch.empty(x.shape, dtype=x.dtype if dx_dtype is None else dx_dtype, device=dev)
    if dw is None:
        dw = torch.empty(d, dtype=_f32, device=dev)
    if db is None and has_bias:
        db = torch.empty(d, dtype=_f32, device=dev)
    if ws is None and rows > 0:
        sh = MoeShape(rows, d, 1, 1, 1, 1, 1, 1)
        ws = torch.empty(workspace_bytes(MOE_OP_LAYER_NORM_BACKWARD, sh), dtype=torch.uint8, device=dev)
    _need(dy, n, "dy")
    _need(d_sum, n, "d_sum")
    _need(dx, n, "dx")
    _need_f32(weight, d, "weight")
    _need_f32(mean, rows, "mean")
    _need_f32(rstd, rows, "rstd")
    _need_f32(dw, d, "dw")
    _need_f32(db, d, "db")
    st = lib().moe_layer_norm_backward(rows, d, _ptr(dy), _dt(dy), _ptr(x), _dt(x), _ptr(weight), _ptr(mean),
                                       _ptr(rstd), _ptr(d_sum), _ptr(dx), _dt(dx), _ptr(dw), _ptr(db), _ptr(ws),
                                       _ws_len(ws), _stream())
    _lib.check("moe_layer_norm_backward", st)
    return dx, dw, db


# ---------------------------------------------------------------- balance loss

def _sequences(sh: MoeShape, seq_offsets, token_mask) -> int:
    if seq_offsets is not None and seq_offsets.dtype != torch.int32:
        raise TypeError("seq_offsets must be int32")
    if token_mask is not None and token_mask.dtype not in (torch.bool, torch.uint8):
        raise TypeError("token_mask must be bool or uint8")
    _need(token_mask, sh.T, "token_mask")
    return 1 if seq_offsets is None else seq_offsets.numel() - 1


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
    dev = logits.device
    n = _sequences(sh, seq_offsets, token_mask)
    if idx.dtype != torch.int32:
        raise TypeError("idx must be int32")
    if loss is None:
        loss = torch.empty(1, dtype=_f32, device=dev)
    if counts is None:
        counts = torch.empty((n, E), dtype=torch.int32, device=dev)
    if prob is None:
        prob = torch.empty((n, E), dtype=_f32, device=dev)
    if dprob is None:
        dprob = torch.empty((n, E), dtype=_f32, device=dev)
    if ws is None:
        ws = torch.empty(max(256, lib().moe_balance_loss_workspace_size(ctypes.byref(sh), n)), dtype=torch.uint8,
                         device=dev)
    if counts.dtype != torch.int32:
        raise TypeError("counts must be int32")
    _need_f32(logits, T * E, "logits")
    _need(idx, T * k, "idx")
    _need_f32(logit_offset, E, "logit_offset")
    _need_f32(loss, 1, "loss")
    _need(counts, n * E, "counts")
    _need_f32(prob, n * E, "prob")
    _need_f32(dprob, n * E, "dprob")
    st = lib().moe_balance_loss(ctypes.byref(sh), _ptr(logits), _ptr(logit_offset), _ptr(idx), _ptr(seq_offsets), n,
                                _ptr(token_mask), alpha, _ptr(counts), _ptr(prob), _ptr(dprob), _ptr(loss), _ptr(ws),
                                _ws_len(ws), _stream())
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
    n = _sequences(sh, seq_offsets, token_mask)
    if dlogits is None:
        dlogits = torch.empty((T, E), dtype=_f32, device=logits.device)
    _need_f32(logits, T * E, "logits")
    _need_f32(logit_offset, E, "logit_offset")
    _need_f32(dprob, n * E, "dprob")
    _need_f32(grad_loss, 1, "grad_loss")
    _need_f32(d_extra, T * E, "d_extra")
    _need_f32(dlogits, T * E, "dlogits")
    st = lib().moe_balance_loss_backward(ctypes.byref(sh), _ptr(logits), _ptr(logit_offset), _ptr(seq_offsets), n,
                                         _ptr(token_mask), _ptr(dprob), _ptr(grad_loss), _ptr(d_extra),
                                         _ptr(dlogits), _stream())
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
            _need_f32(self.master[i], k, "master")
            if eight[i]:
                _need_f32(self.m_scale[i], tiles(p), "m_scale")
                _need_f32(self.v_scale[i], tiles(p), "v_scale")
            self._items[i] = _lib.MoeAdamwTensor(
                k, _ptr(p), _ptr(self.grads[i]), _ptr(self.master[i]), _ptr(self.m[i]), _ptr(self.v[i]),
                _ptr(self.m_scale[i]), _ptr(self.v_scale[i]), wd[i], _dt(p), _dt(self.grads[i]), _dt(self.m[i]), 0)

    def step(self, grad_scale: Optional[torch.Tensor] = None, lr: Optional[float] = None) -> None:
        """One step on what the gradient buffers hold, times grad_scale ([1]
        fp32 on the device).  lr: this step's rate (else the constructor's)."""
        _need_f32(grad_scale, 1, "grad_scale")
        h = _lib.MoeAdamwParams(self.lr if lr is None else lr, self.betas[0], self.betas[1], self.eps,
                                self.step_count + 1)
        st = lib().moe_adamw_step(len(self.params), self._items, ctypes.byref(h), _ptr(grad_scale), _stream())
        _lib.check("moe_adamw_step", st)
        self.step_count += 1


# ---------------------------------------------------------------- the block

class MoEBlock:
    """A pre-norm MoE block that trains: stream' = stream + delta, h =
    norm(stream'), out = MoE(h), with a balance loss on the router.

    forward(delta, stream) returns (out, stream'): the next block adds them in
    its own norm, so no pass of its own is spent on the residual add.
    backward(d_out, d_stream) leaves the gradients of every weight in the
    block's buffers and returns the gradient of delta and stream.
    step() is the AdamW step on them."""

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

    def forward(self, delta: torch.Tensor, stream: torch.Tensor, seq_offsets: Optional[torch.Tensor] = None,
                token_mask: Optional[torch.Tensor] = None):
        layer_norm(delta, self.norm_w, self.norm_b, residual=stream, eps=self.eps, y=self.h, sum_out=self.stream,
                   mean=self.mean, rstd=self.rstd)
        out = self.layer.forward(self.h, save_for_backward=True)
        la = self.layer
        self.seqs = (seq_offsets, token_mask)
        self.loss, self.counts, self.prob, self.dprob = balance_loss(
            la.sh, la.logits, la.idx, self.alpha, seq_offsets, token_mask, la.logit_offset)
        return out, self.stream

    def backward(self, d_out: torch.Tensor, d_stream: Optional[torch.Tensor] = None) -> torch.Tensor:
        la = self.layer
        dl = la._bwd_ws(d_out.device)["dlogits"]
        balance_loss_backward(la.sh, la.logits, self.dprob, *self.seqs, la.logit_offset, dlogits=dl)
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
