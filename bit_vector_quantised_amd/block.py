"""What stands around the experts of a layer, on top of the C ABI: the norm with the residual's addition, the router with
its choice of experts, and the layer's whole mixture-of-experts block, with their gradients.

Objects, streams, workspaces and gradients are as in dense.py: each call runs on the current stream of the object's device,
the gradients are calls of their own, and calls of one object that may overlap need two objects.
"""
from __future__ import annotations

from typing import Optional, Tuple, Union

import torch

from . import _lib
from .dense import DenseExperts, Linear, Rows8, _device, _need, _OnDevice
from .layer import x_dtype_code

SCORES = {"softmax": _lib.SCORE_SOFTMAX, "sigmoid": _lib.SCORE_SIGMOID}


class RmsNorm(_OnDevice):
    """s = x + residual, y = s / sqrt(mean(s^2) + eps) * gain over rows of len(gain) columns (gain: fp32).  backward: make
    the workspace of the gradients, for up to max_rows rows."""

    def __init__(self, gain: torch.Tensor, eps: float = 1e-6, max_rows: int = 1, backward: bool = False):
        super().__init__(_device(gain.device))
        self.n_cols, self.max_rows, self.eps = gain.numel(), max_rows, float(eps)
        self.gain = gain
        self._gain()
        need = _lib.norm_bytes(max_rows, self.n_cols)
        if need == 0 or not eps > 0:
            raise ValueError("invalid number of rows or columns, or eps")
        self.ws_bytes = need if backward else 0
        self.ws = self._new(need, torch.uint8) if backward else None

    def _gain(self) -> int:
        return _need(self.gain, "gain", (self.n_cols,), torch.float32, self.device)

    def _rows(self, t: torch.Tensor) -> int:
        if t.shape[0] > self.max_rows:
            raise ValueError(f"{t.shape[0]} rows, made for {self.max_rows}")
        return t.shape[0]

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None, s: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, rows8: Optional[Rows8] = None, dense: bool = True) -> Optional[torch.Tensor]:
        """x [M, C] -> y [M, C], bf16 or fp32 (as out; by default as x).  residual [M, C] is added first; s receives the
        sum, in residual's type (it may be residual, or x).  rows8 receives y in 8 bits; with dense=False that is all."""
        M, C = self._rows(x), self.n_cols
        xp = _need(x, "x", (M, C), x.dtype, self.device)
        stream = residual if residual is not None else s if s is not None else x
        r = _need(residual, "residual", (M, C), stream.dtype, self.device) if residual is not None else 0
        sp = _need(s, "s", (M, C), stream.dtype, self.device) if s is not None else 0
        if not dense and out is not None:
            raise ValueError("out without dense")
        if dense and out is None:
            out = torch.empty_like(x)
        y = _need(out, "out", (M, C), out.dtype, self.device) if dense else 0
        q = rows8.desc("rows8", M, C, self.device) if rows8 is not None else None
        self._call(_lib.norm_forward, xp, x_dtype_code(x), r, sp, x_dtype_code(stream), M, C, self._gain(), self.eps, y,
                   x_dtype_code(out) if dense else _lib.F32, q)
        return out

    def backward(self, s: torch.Tensor, dy: torch.Tensor, dy2: Optional[torch.Tensor] = None,
                 ds: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                 dgain: Optional[torch.Tensor] = None) -> None:
        """Gradients from s [M, C] (x, if nothing was added), the gradient dy + dy2 of y and ds, that of s: those of dx
        [M, C] (of x and of residual alike; it may be ds) and dgain [C] (fp32) that are given are written."""
        M, C = self._rows(s), self.n_cols
        if dgain is not None and self.ws is None:
            raise ValueError("made without backward")
        sp = _need(s, "s", (M, C), s.dtype, self.device)
        g = _need(dy, "dy", (M, C), dy.dtype, self.device)
        g2 = _need(dy2, "dy2", (M, C), dy.dtype, self.device) if dy2 is not None else 0
        like = dx if dx is not None else ds if ds is not None else s
        kind = like.dtype
        d = _need(ds, "ds", (M, C), kind, self.device) if ds is not None else 0
        xd = _need(dx, "dx", (M, C), kind, self.device) if dx is not None else 0
        gd = _need(dgain, "dgain", (C,), torch.float32, self.device) if dgain is not None else 0
        self._call(_lib.norm_backward, sp, x_dtype_code(s), M, C, self._gain(), self.eps, g, g2, x_dtype_code(dy), d, xd,
                   x_dtype_code(like), gd, 0 if self.ws is None else self.ws.data_ptr(), self.ws_bytes)


class ExpertChoice(_OnDevice):
    """The experts of each token from the router's logits.  Scores are softmax or sigmoid of the logits; bias (fp32 [E], for
    the experts' balance) is added to them for the choice only.  groups > top_groups: the experts lie in equal groups of
    neighbours, and only those of the top_groups groups with the largest sums of their `best` (1 or 2) largest
    values can be chosen.  Weights are the chosen experts' scores, with renorm divided by their sum, times scale.

    An expert whose logit or bias is -inf or NaN is off; places that no expert is left for have id -1, a dropped pair of
    ExpertRows, and weight 0."""

    def __init__(self, n_experts: int, top_k: int, score: str = "softmax", bias: Optional[torch.Tensor] = None,
                 groups: int = 1, top_groups: Optional[int] = None, best: int = 2, renorm: bool = True, scale: float = 1.0,
                 device="cuda"):
        super().__init__(_device(device))
        if score not in SCORES:
            raise ValueError(f"score must be one of {', '.join(SCORES)}")
        top_groups = groups if top_groups is None else top_groups
        if not (1 <= n_experts <= 1024 and 1 <= groups <= 64 and n_experts % groups == 0 and 1 <= top_groups <= groups
                and best in (1, 2) and 1 <= top_k <= min(32, top_groups * (n_experts // groups))):
            raise ValueError("invalid number of experts, groups or top_k")
        self.n_experts, self.top_k, self.bias = n_experts, top_k, bias
        self.c = _lib.Choice(n_experts, top_k, SCORES[score], groups, top_groups, best, int(bool(renorm)), float(scale), None)
        self._choice()

    def _choice(self) -> _lib.Choice:
        """The description of the choice, with the present address of bias."""
        self.c.bias = _need(self.bias, "bias", (self.n_experts,), torch.float32, self.device) if self.bias is not None else None
        return self.c

    def forward(self, logits: torch.Tensor, ids: Optional[torch.Tensor] = None,
                w: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """logits [T, E] (fp32) -> ids [T, k] (int32) and w [T, k] (fp32), the largest value first."""
        T, k = logits.shape[0], self.top_k
        p = _need(logits, "logits", (T, self.n_experts), torch.float32, self.device)
        ids = torch.empty((T, k), dtype=torch.int32, device=self.device) if ids is None else ids
        w = torch.empty((T, k), dtype=torch.float32, device=self.device) if w is None else w
        i = _need(ids, "ids", (T, k), torch.int32, self.device)
        o = _need(w, "w", (T, k), torch.float32, self.device)
        self._call(_lib.choose, self._choice(), p, T, i, o)
        return ids, w

    def backward(self, logits: torch.Tensor, ids: torch.Tensor, dw: torch.Tensor,
                 dlogits: Optional[torch.Tensor] = None) -> torch.Tensor:
        """dlogits [T, E] (fp32; it may be logits) from dw [T, k], the gradient of the weights at the chosen ids."""
        T, k = logits.shape[0], self.top_k
        p = _need(logits, "logits", (T, self.n_experts), torch.float32, self.device)
        i = _need(ids, "ids", (T, k), torch.int32, self.device)
        d = _need(dw, "dw", (T, k), torch.float32, self.device)
        dlogits = torch.empty_like(logits) if dlogits is None else dlogits
        o = _need(dlogits, "dlogits", (T, self.n_experts), torch.float32, self.device)
        self._call(_lib.choose_backward, self._choice(), p, T, i, d, o)
        return dlogits


class Router(_OnDevice):
    """The router's product and the choice of experts: logits = x w^T (w [E, H], bf16 or fp32; the logits are fp32), then
    ExpertChoice with the further arguments.  backward: make what the gradients need, from x as it is or in 8 bits."""

    def __init__(self, w: torch.Tensor, top_k: int, max_tokens: int, backward: bool = False, **choice):
        super().__init__(_device(w.device))
        E = w.shape[0]
        self.linear = Linear(w, max_rows=max_tokens, backward=backward, kept8=backward)
        self.choice = ExpertChoice(E, top_k, device=w.device, **choice)
        self.logits = self._new((max_tokens, E), torch.float32)
        self.ids = self._new((max_tokens, top_k), torch.int32)
        self.w = self._new((max_tokens, top_k), torch.float32)
        self.dlogits = self._new((max_tokens, E), torch.float32) if backward else None
        self.n_tokens = None  # of the last forward
        self._pass = None     # its mark, for a block that goes back through it

    def forward(self, x: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
        """x [T, H] -> ids [T, k] (int32) and w [T, k] (fp32), valid until the next forward."""
        T = x.shape[0]
        self.n_tokens = self._pass = None
        self._here()  # (the parts' calls use this object's buffers)
        if T > self.linear.max_rows:
            raise ValueError(f"{T} tokens, made for {self.linear.max_rows}")
        self.linear.forward(x, out=self.logits[:T])
        ids, w = self.choice.forward(self.logits[:T], self.ids[:T], self.w[:T])
        self.n_tokens, self._pass = T, object()
        return ids, w

    def backward(self, x: Union[torch.Tensor, Rows8, None], dw: torch.Tensor, dx: Optional[torch.Tensor] = None,
                 dweight: Optional[torch.Tensor] = None) -> None:
        """Gradients of the last forward from dw [T, k]: those of dx [T, H] and dweight (as w) that are given are
        written.  x as it was, or in 8 bits; None without dweight."""
        if self.dlogits is None:
            raise ValueError("made without backward")
        if self.n_tokens is None:
            raise ValueError("no forward to go back through")
        T = self.n_tokens
        self._here()
        dlogits = self.choice.backward(self.logits[:T], self.ids[:T], dw, self.dlogits[:T])
        self.linear.backward(x, dlogits, dx=dx, dw=dweight)


class MoeBlock(_OnDevice):
    """A layer's mixture of experts with the norm before it: s = x + residual, n = norm(s), ids and w = router(n), y =
    sum_i w_i E_i(n).  The next block adds y to s.  After a forward with keep=True, backward gives the gradients; what it
    needs beside s is kept here and in its router and experts (made with kept8 in 8 bits, which the norm then writes), so
    that backward refuses if either has made another pass since, alone or in another block.  work: another block of
    the same sizes whose buffers this one uses (see DenseExperts; both of experts with kept8)."""

    def __init__(self, norm: RmsNorm, router: Router, experts: DenseExperts, work: Optional["MoeBlock"] = None):
        super().__init__(norm.device)
        T, H, k = experts.rows.max_tokens, norm.n_cols, experts.rows.top_k
        w1 = experts.fc1.w
        if router.linear.n_in != H or w1.shape[-1] != H or router.linear.dtype != w1.dtype:
            raise ValueError("norm, router and experts must be of one hidden size, router and experts of one type")
        if router.choice.top_k != k or router.choice.n_experts != experts.rows.n_experts:
            raise ValueError("router and experts must be of one number of experts and top_k")
        if norm.max_rows < T or router.linear.max_rows < T or {norm.device, router.device, experts.rows.device} != {self.device}:
            raise ValueError("norm and router must be made for as many tokens as the experts, on their device")
        if work is not None and not (experts.kept8 and work.experts.kept8 and work.experts.sizes == experts.sizes):
            raise ValueError("work must be a block of the same sizes, both of experts with kept8")
        self.norm, self.router, self.experts = norm, router, experts
        back = experts.z is not None

        def new(name, shape, dtype):
            return self._new(shape, dtype) if work is None else self._share(getattr(work, name))

        self.n = new("n", (T, H), w1.dtype)
        self.dn, self.dn2 = (new("dn", (T, H), w1.dtype), new("dn2", (T, H), w1.dtype)) if back else (None, None)
        self.dw = new("dw", (T, k), torch.float32) if back else None
        self._kept = None

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None, s: Optional[torch.Tensor] = None,
                y: Optional[torch.Tensor] = None, keep: bool = False) -> torch.Tensor:
        """x [T, H] (and residual [T, H], added to it) -> y [T, H], fp32 unless given.  s receives the sum, which
        backward takes."""
        T = x.shape[0]
        self._kept = None
        if T > self.experts.rows.max_tokens:
            raise ValueError(f"{T} tokens, made for {self.experts.rows.max_tokens}")
        if keep and (self.dn is None or self.router.dlogits is None or self.norm.ws is None):
            raise ValueError("made without backward")
        self._here()  # (the parts' calls use this object's buffers)
        kept8 = keep and self.experts.kept8
        if kept8:
            self.experts._kept = None  # (the norm writes x8, even if a call after it is refused)
        self.norm.forward(x, residual, s, self.n[:T], self.experts.x8 if kept8 else None)
        ids, w = self.router.forward(self.n[:T])
        y = self.experts.forward(self.n[:T], ids, w, y, keep=keep, x8_there=kept8)
        if keep:
            self._kept = T, self.router._pass, self.experts._kept[0]
        return y

    def backward(self, s: torch.Tensor, dy: torch.Tensor, ds: Optional[torch.Tensor], dx: torch.Tensor, dgain: torch.Tensor,
                 drouter: torch.Tensor, dw1: torch.Tensor, dw2: torch.Tensor) -> None:
        """Gradients of the last forward(keep=True) from dy [T, H] and ds [T, H], the gradient of s (None: y is all that
        is used): dx [T, H] (of x and of residual alike; it may be ds), dgain, drouter, dw1 and dw2."""
        if self._kept is None:
            raise ValueError("the last forward kept nothing")
        (T, routed, kept), self._kept = self._kept, None
        if self.router._pass is not routed or self.experts._kept is None or self.experts._kept[0] is not kept:
            raise ValueError("the router or the experts have made another pass since")
        self._here()  # (the parts' calls use this object's buffers)
        self.experts.backward(dy, self.dn[:T], self.dw[:T], dw1, dw2)
        self.router.backward(self.experts.x8 if self.experts.kept8 else self.n[:T], self.dw[:T], self.dn2[:T], drouter)
        self.norm.backward(s, self.dn[:T], self.dn2[:T], ds, dx, dgain)
