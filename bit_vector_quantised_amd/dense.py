"""Unquantised experts on top of the C ABI: the routed pairs sorted by expert and back, the
dense product with bias, activation and residual (one matrix, or one per expert over the
sorted rows), and their gradients.  The gradients are calls of their own: nothing here records a graph
for autograd, and outputs carry none even if an input requires a gradient.

As in layer.py, PyTorch provides device memory and the stream; every step of the
computation runs in the HIP library.  An object's workspace serves its calls one after the
other on a stream: calls of one object that may overlap (on two streams, or in two graphs
replayed at once) need two objects.  An object may be dropped while its calls are still under way on
any stream; one whose calls are in a captured graph has to be kept as long as the graph.  As with a
tensor, another stream than the one it was made on waits for that one before its first call.
"""
from __future__ import annotations

from typing import List, Optional, Tuple

import torch

from . import _lib
from .layer import x_dtype_code

ACTS = {"none": _lib.ACT_NONE, "silu": _lib.ACT_SILU, "gelu": _lib.ACT_GELU, "swiglu": _lib.ACT_SWIGLU}


def _need(t: torch.Tensor, what: str, shape, dtype, device) -> int:
    """The address of t, which must be a contiguous tensor of this shape, type and device."""
    if t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{what}: need a contiguous {tuple(shape)} {dtype} tensor on {device}, "
                         f"got {tuple(t.shape)} {t.dtype} on {t.device}")
    return t.data_ptr()


def _device(device) -> torch.device:
    d = torch.device(device)
    return torch.device(d.type, torch.cuda.current_device()) if d.type == "cuda" and d.index is None else d


class _OnDevice:
    """Calls run on the current stream of the object's device, whichever device is current."""

    def __init__(self, device: torch.device):
        if device.type != "cuda":
            raise ValueError(f"need a GPU tensor or device, got {device}")
        self.device = device
        self._buffers: List[torch.Tensor] = []
        self._streams = {torch.cuda.current_stream(device).cuda_stream}  # the buffers' allocator knows of these

    def _new(self, shape, dtype) -> torch.Tensor:
        """A buffer of the object, in use by the streams of its calls."""
        t = torch.empty(shape, dtype=dtype, device=self.device)
        self._buffers.append(t)
        return t

    def _call(self, fn, *args) -> None:
        index = self.device.index
        stream = torch.cuda.current_stream(index)
        if stream.cuda_stream not in self._streams:
            for t in self._buffers:
                t.record_stream(stream)
            self._streams.add(stream.cuda_stream)
        if torch.cuda.current_device() == index:
            fn(*args, stream.cuda_stream)
        else:
            with torch.cuda.device(index):
                fn(*args, stream.cuda_stream)


class ExpertRows(_OnDevice):
    """The pairs of up to max_tokens tokens in the order of their experts.  sort(ids) fills
    expert_start [E + 1], pair_row and row_pair [T*k] (int32, valid until the next sort);
    the other calls use them for the T tokens sorted last."""

    def __init__(self, n_experts: int, top_k: int, max_tokens: int, device="cuda"):
        super().__init__(_device(device))
        self.n_experts, self.top_k, self.max_tokens, self.n_tokens = n_experts, top_k, max_tokens, 0
        self.ws_bytes = _lib.sort_bytes(max_tokens, top_k, n_experts)
        if self.ws_bytes == 0:
            raise ValueError("invalid number of experts, tokens or top_k")
        self.ws = self._new(self.ws_bytes, torch.uint8)
        self.expert_start = self._new(n_experts + 1, torch.int32).zero_()
        self.pair_row = self._new(max_tokens * top_k, torch.int32)
        self.row_pair = self._new(max_tokens * top_k, torch.int32)

    def sort(self, ids: torch.Tensor) -> torch.Tensor:
        """Sort the pairs of ids [T, k] (int32; outside 0..E-1: dropped); returns expert_start."""
        T = ids.shape[0]
        if T > self.max_tokens:
            raise ValueError(f"{T} tokens, made for {self.max_tokens}")
        p = _need(ids, "ids", (T, self.top_k), torch.int32, self.device)
        self._call(_lib.sort_pairs, p, T, self.top_k, self.n_experts, self.expert_start.data_ptr(),
                   self.pair_row.data_ptr(), self.row_pair.data_ptr(), self.ws.data_ptr(), self.ws_bytes)
        self.n_tokens = T
        return self.expert_start

    def gather(self, x: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """x [T, C] -> rows [T*k, C] in the order of the experts (rows of dropped pairs as they were)."""
        T, k = self.n_tokens, self.top_k
        C = x.shape[-1]
        p = _need(x, "x", (T, C), x.dtype, self.device)
        out = torch.empty((T * k, C), dtype=x.dtype, device=self.device) if out is None else out
        o = _need(out, "out", (T * k, C), x.dtype, self.device)
        self._call(_lib.gather_rows, p, x_dtype_code(x), T, k, C, self.pair_row.data_ptr(), o)
        return out

    def gather_backward(self, drows: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """dx [T, C] of gather from drows [T*k, C]."""
        if out is None:
            out = torch.empty((self.n_tokens, drows.shape[-1]), dtype=drows.dtype, device=self.device)
        return self.combine(drows, None, None, out)

    def combine(self, rows: torch.Tensor, w: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """y[t] = residual[t] + sum_i w[t, i] rows[pair_row[t, i]] (w None: all 1).  out: [T, C], bf16
        or fp32 (its type is residual's; fp32 without either); it may be residual."""
        T, k = self.n_tokens, self.top_k
        C = rows.shape[-1]
        r = _need(rows, "rows", (T * k, C), rows.dtype, self.device)
        if out is None:
            out = torch.empty((T, C), dtype=torch.float32 if residual is None else residual.dtype, device=self.device)
        o = _need(out, "out", (T, C), out.dtype, self.device)
        a = _need(residual, "residual", (T, C), out.dtype, self.device) if residual is not None else 0
        wp = _need(w, "w", (T, k), torch.float32, self.device) if w is not None else 0
        self._call(_lib.combine_rows, r, x_dtype_code(rows), T, k, C, self.pair_row.data_ptr(), wp, a, o,
                   x_dtype_code(out))
        return out

    def combine_backward(self, dy: torch.Tensor, w: Optional[torch.Tensor], rows: torch.Tensor,
                         drows: Optional[torch.Tensor] = None,
                         dw: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """(drows, dw) of combine from dy [T, C]; rows are the ones combined.  drows: bf16 or fp32 (by default as
        rows; in another type by a launch of its own)."""
        T, k = self.n_tokens, self.top_k
        C = rows.shape[-1]
        g = _need(dy, "dy", (T, C), dy.dtype, self.device)
        r = _need(rows, "rows", (T * k, C), rows.dtype, self.device)
        drows = torch.empty_like(rows) if drows is None else drows
        dw = torch.empty((T, k), dtype=torch.float32, device=self.device) if dw is None else dw
        d = _need(drows, "drows", (T * k, C), drows.dtype, self.device)
        p = _need(dw, "dw", (T, k), torch.float32, self.device)
        wp = _need(w, "w", (T, k), torch.float32, self.device) if w is not None else 0
        both = drows.dtype == rows.dtype
        if not both:  # (first: dw may be w, and is written by the second)
            self._call(_lib.combine_rows_backward, g, x_dtype_code(dy), T, k, C, self.pair_row.data_ptr(), wp, 0,
                       x_dtype_code(drows), d, 0)
        self._call(_lib.combine_rows_backward, g, x_dtype_code(dy), T, k, C, self.pair_row.data_ptr(), wp, r,
                   x_dtype_code(rows), d if both else 0, p)
        return drows, dw


class Linear(_OnDevice):
    """y = act(x W^T + b) + residual for up to max_rows rows.  w: [R, n_in], or [G, R, n_in] for one
    matrix per group of rows; bf16 or fp32.  R is n_out, or 2 n_out for act "swiglu" (gate rows, then
    up rows; swiglu_limit: its clamp, 0 none).  bias: fp32 [R] or [G, R].  backward: make the
    workspace of the gradients too.  Each call reads w and bias where they are at that time (a
    captured graph where they were when it was captured)."""

    def __init__(self, w: torch.Tensor, bias: Optional[torch.Tensor] = None, act: str = "none",
                 swiglu_limit: float = 0.0, max_rows: int = 1, backward: bool = False):
        super().__init__(_device(w.device))
        if act not in ACTS:
            raise ValueError(f"act must be one of {', '.join(ACTS)}")
        if w.dim() not in (2, 3) or (act == "swiglu" and w.shape[-2] % 2):
            raise ValueError("w must be [R, n_in] or [G, R, n_in], with an even R for swiglu")
        self.w, self.bias, self.max_rows = w, bias, max_rows
        self.grouped = w.dim() == 3
        self.n_groups = w.shape[0] if self.grouped else 1
        self.n_rows_w, self.n_in = w.shape[-2], w.shape[-1]
        self.n_out = self.n_rows_w // 2 if act == "swiglu" else self.n_rows_w
        self.w_shape, self.dtype = w.shape, w.dtype
        self.c = _lib.LinearDesc(self.n_in, self.n_out, self.n_groups, ACTS[act], x_dtype_code(w), float(swiglu_limit))
        self._weights()
        need = [_lib.linear_bytes(self.c, max_rows, b) for b in (False, True)[:2 if backward else 1]]
        if 0 in need:
            raise ValueError("invalid sizes")
        self.ws_bytes = max(need)
        self.ws = self._new(self.ws_bytes, torch.uint8)

    def _weights(self) -> _lib.LinearDesc:
        """The description of the product, with the present addresses of w and bias."""
        self.c.w = _need(self.w, "w", self.w_shape, self.dtype, self.device)
        self.c.bias = _need(self.bias, "bias", self.w_shape[:-1], torch.float32, self.device) if self.bias is not None else None
        return self.c

    def _rows(self, rows: torch.Tensor, group_start: Optional[torch.Tensor]) -> Tuple[int, int]:
        if rows.shape[0] > self.max_rows:
            raise ValueError(f"{rows.shape[0]} rows, made for {self.max_rows}")
        if group_start is None:
            if self.grouped:
                raise ValueError("weights of groups need group_start")
            return rows.shape[0], 0
        return rows.shape[0], _need(group_start, "group_start", (self.n_groups + 1,), torch.int32, self.device)

    def forward(self, x: torch.Tensor, group_start: Optional[torch.Tensor] = None,
                residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                z: Optional[torch.Tensor] = None) -> torch.Tensor:
        """x [M, n_in] -> y [M, n_out].  group_start [G + 1] (int32): the first row of each group; rows
        in no group are neither read nor written.  out: bf16 or fp32 (by default as residual, or as x); it
        may be residual.  z [M, R]: receives the values before the activation, for backward."""
        M, gs = self._rows(x, group_start)
        xp = _need(x, "x", (M, self.n_in), self.dtype, self.device)
        if out is None:
            out = torch.empty((M, self.n_out), dtype=x.dtype if residual is None else residual.dtype, device=self.device)
        y = _need(out, "out", (M, self.n_out), out.dtype, self.device)
        r = _need(residual, "residual", (M, self.n_out), out.dtype, self.device) if residual is not None else 0
        zp = _need(z, "z", (M, self.n_rows_w), self.dtype, self.device) if z is not None else 0
        self._call(_lib.linear_forward, self._weights(), xp, M, gs, r, y, x_dtype_code(out), zp, self.ws.data_ptr(),
                   self.ws_bytes)
        return out

    def backward(self, x: Optional[torch.Tensor], dy: torch.Tensor, z: Optional[torch.Tensor] = None,
                 group_start: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                 dw: Optional[torch.Tensor] = None, dbias: Optional[torch.Tensor] = None) -> None:
        """Gradients from dy [M, n_out] and the z that forward kept (not needed for act "none"): those of dx
        [M, n_in], dw (as w) and dbias (as bias) that are given are written.  x may be None without dw."""
        M, gs = self._rows(dy, group_start)
        if x is None and dw is not None:
            raise ValueError("dw needs x")
        xp = _need(x, "x", (M, self.n_in), self.dtype, self.device) if x is not None else 0
        g = _need(dy, "dy", (M, self.n_out), dy.dtype, self.device)
        zp = _need(z, "z", (M, self.n_rows_w), self.dtype, self.device) if z is not None else 0
        xd = _need(dx, "dx", (M, self.n_in), self.dtype, self.device) if dx is not None else 0
        wd = _need(dw, "dw", self.w_shape, self.dtype, self.device) if dw is not None else 0
        bd = _need(dbias, "dbias", self.w_shape[:-1], torch.float32, self.device) if dbias is not None else 0
        self._call(_lib.linear_backward, self._weights(), xp, M, gs, zp, g, x_dtype_code(dy), xd, wd, bd, self.ws.data_ptr(),
                   self.ws_bytes)


class DenseExperts:
    """The routed-expert step of a layer with unquantised experts: w1 [E, 2I, H] (gate rows, then up
    rows) and w2 [E, H, I], bf16 or fp32.  forward(x, ids, w) computes y = sum_i w_i E_i(x) (+ y
    itself with add=True) from a routing such as Step.route's; after a forward with keep=True,
    backward(dy) gives the gradients of x, the routing weights and the experts.  What backward needs
    of the pass is kept here: x, ids and w may change in between (w1 and w2 may not).

    With bf16 experts h, z and the gradients between the products are held in bf16, which the matrix
    instructions take; an expert's output o is held in fp32 until the weighted sum."""

    def __init__(self, w1: torch.Tensor, w2: torch.Tensor, top_k: int, max_tokens: int, swiglu_limit: float = 0.0,
                 backward: bool = False):
        E, R, H = w1.shape
        if tuple(w2.shape) != (E, H, R // 2) or w2.dtype != w1.dtype or w2.device != w1.device:
            raise ValueError("w1 must be [E, 2I, H] and w2 [E, H, I], of one type and device")
        P = max_tokens * top_k
        self.fc1 = Linear(w1, act="swiglu", swiglu_limit=swiglu_limit, max_rows=P, backward=backward)
        self.fc2 = Linear(w2, max_rows=P, backward=backward)
        self.rows = ExpertRows(E, top_k, max_tokens, device=w1.device)
        # (buffers of rows: each pass of the step calls it, on the pass's stream)
        new = lambda *shape: self.rows._new(shape, w1.dtype)  # noqa: E731
        self.xs, self.h, self.o = new(P, H), new(P, R // 2), self.rows._new((P, H), torch.float32)
        self.z, self.dh, self.do = (new(P, R), new(P, R // 2), new(P, H)) if backward else (None, None, None)
        self.w_kept = self.rows._new((max_tokens, top_k), torch.float32) if backward else None
        self._kept = None

    def forward(self, x: torch.Tensor, ids: torch.Tensor, w: torch.Tensor, y: Optional[torch.Tensor] = None,
                add: bool = False, keep: bool = False) -> torch.Tensor:
        """x [T, H], ids and w [T, k] -> y [T, H] (fp32 unless given)."""
        if keep and self.z is None:
            raise ValueError("made without backward")
        if add and y is None:
            raise ValueError("add needs y")
        self._kept = None  # (from here on the buffers are another pass's, even if a call below is refused)
        P = x.shape[0] * self.rows.top_k
        start = self.rows.sort(ids)
        self.rows.gather(x, self.xs[:P])
        self.fc1.forward(self.xs[:P], start, out=self.h[:P], z=self.z[:P] if keep else None)
        self.fc2.forward(self.h[:P], start, out=self.o[:P])
        out = self.rows.combine(self.o[:P], w, y if add else None, y)
        if keep:
            self._kept = (x, self.w_kept[:x.shape[0]].copy_(w))  # (of x only the number of tokens is used)
        return out

    def backward(self, dy: torch.Tensor, dx: torch.Tensor, dw: torch.Tensor, dw1: torch.Tensor,
                 dw2: torch.Tensor) -> None:
        """Gradients of the last forward(keep=True): dx [T, H], dw [T, k], dw1 and dw2 (as w1 and w2)."""
        if self._kept is None:
            raise ValueError("the last forward kept nothing")
        x, w = self._kept
        self._kept = None
        P = x.shape[0] * self.rows.top_k
        start = self.rows.expert_start
        self.rows.combine_backward(dy, w, self.o[:P], self.do[:P], dw)
        self.fc2.backward(self.h[:P], self.do[:P], group_start=start, dx=self.dh[:P], dw=dw2)
        # (do has been read: it takes the gradient of the gathered rows)
        self.fc1.backward(self.xs[:P], self.dh[:P], self.z[:P], start, dx=self.do[:P], dw=dw1)
        self.rows.gather_backward(self.do[:P], dx)
