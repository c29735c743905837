"""The dense products around the routed experts, as plans of C-ABI calls on
preallocated device buffers (no allocation per step): the router's projection
and a shared expert's gated feed-forward block, forward and backward, and a
layer's training step that joins them to the routed experts.

Operands are bf16; x (and LinearPlan's W) may be a column slice of a wider
buffer.  A plan's outputs are its own buffers, valid until its next call."""

import torch

from . import ops
from .layer import TrainPlan, capture_graph
from .ops import _dense, _Device, launch, rows_of, workspace_bytes

BF16 = torch.bfloat16


def _ptr(t):
    return None if t is None else t.data_ptr()


def _code(table, name, what):
    if name not in table:
        raise ValueError(f"unknown {what} {name!r}: one of {', '.join(table)}")
    return table[name]


class LinearPlan:
    """out = act(x W^T + bias) + residual for x [T, K], W [N, K], and its
    gradients when ``train`` (the argument of act is then kept in bf16).
    bias: the plan also holds a bias gradient."""

    def __init__(self, T, K, N, act="none", out_dtype=BF16, train=False, bias=False, device="cuda"):
        self.T, self.K, self.N, self.train = T, K, N, train
        self.act = _code(ops.ACTS, act, "activation")
        if out_dtype not in (BF16, torch.float32):
            raise TypeError(f"out_dtype: bf16 or fp32, got {out_dtype}")
        self.out_dtype = out_dtype
        self.f32 = ops.SRC_F32 if out_dtype == torch.float32 else ops.SRC_BF16
        dv = self.device = torch.device(device) if torch.device(device).index is not None else torch.device(
            "cuda", torch.cuda.current_device())
        with _Device(dv):
            n = workspace_bytes("moe_linear_workspace", T, N, K)
            if train:
                n = max(n, workspace_bytes("moe_linear_backward_workspace", T, N, K))
        self.ws = torch.empty(max(n, 16), dtype=torch.uint8, device=dv)
        self.out = torch.empty((T, N), dtype=out_dtype, device=dv)
        self.pre = torch.empty((T, N), dtype=BF16, device=dv) if train and self.act else None
        self.dx = torch.empty((T, K), dtype=BF16, device=dv) if train else None
        self.dW = torch.empty((N, K), dtype=BF16, device=dv) if train else None
        self.db = torch.empty(N, dtype=BF16, device=dv) if train and bias else None
        self._out, self._pre, self._ws, self.ws_bytes = self.out.data_ptr(), _ptr(self.pre), _ptr(self.ws), self.ws.numel()
        self._grads = (_ptr(self.dx), _ptr(self.dW), _ptr(self.db))

    def forward(self, x, W, bias=None, residual=None):
        dv, T, K, N = self.device, self.T, self.K, self.N
        ldx = rows_of(x, (T, K), BF16, "x", dv)
        ldw = rows_of(W, (N, K), BF16, "W", dv)
        if bias is not None:
            _dense(bias, (N,), BF16, "bias", dv)
        ldr = N if residual is None else rows_of(residual, (T, N), BF16, "residual", dv)
        launch("moe_linear", dv, x.data_ptr(), ldx, W.data_ptr(), ldw, _ptr(bias), _ptr(residual), ldr, T, N, K, self.act,
               self._out, self.f32, N, self._pre, self._ws, self.ws_bytes)
        return self.out

    def backward(self, dy, x, W, dx_add=None):
        """(dx [T, K] + dx_add, dW [N, K], db [N] or None) of the last forward
        for dy [T, N] of out's type (also the residual's gradient).  dx and dW are
        products of dy * act' rounded to bf16, from fp32 too."""
        if not self.train:
            raise ValueError("the plan was made without train=True")
        dv, T, K, N = self.device, self.T, self.K, self.N
        _dense(dy, (T, N), self.out_dtype, "dy", dv)
        ldx = rows_of(x, (T, K), BF16, "x", dv)
        ldw = rows_of(W, (N, K), BF16, "W", dv)
        if dx_add is not None:
            _dense(dx_add, (T, K), BF16, "dx_add", dv)
        launch("moe_linear_backward", dv, dy.data_ptr(), self.f32, self._pre, x.data_ptr(), ldx, W.data_ptr(), ldw,
               _ptr(dx_add), T, N, K, self.act, *self._grads, self._ws, self.ws_bytes)
        return self.dx, self.dW, self.db

    def capture(self, x, W, bias=None, residual=None, warmup=1):
        """``forward`` over these exact buffers as a HIP graph (see ForwardPlan.capture)."""
        return capture_graph(lambda: self.forward(x, W, bias=bias, residual=residual), warmup, self.device)


class GatedFFNPlan:
    """A shared expert on T tokens: y = (act(x Wg^T + bg) * (x Wu^T + bu)) W2^T
    + b2 + residual with W13 [2f, d] = [Wg; Wu], W2 [d, f].

    save: "none" (inference), "bf16" or "int8" -- how [G, U] is kept for the
    backward (int8: f % 128 == 0, half the bytes).  bias: the plan also holds the
    bias gradients."""

    def __init__(self, T, d, f, act="silu", save="none", bias=False, device="cuda"):
        self.T, self.d, self.f = T, d, f
        self.act = _code(ops.ACTS, act, "activation")
        self.save = _code(ops.SAVES, save, "save mode")
        if save == "int8" and f % 128:
            raise ValueError(f"save='int8' needs f % 128 == 0, got f={f}")
        dv = self.device = torch.device(device) if torch.device(device).index is not None else torch.device(
            "cuda", torch.cuda.current_device())
        train = self.save != 0
        with _Device(dv):
            n = workspace_bytes("moe_gated_ffn_workspace", T, d, f)
            if train:
                n = max(n, workspace_bytes("moe_gated_ffn_backward_workspace", T, d, f))
        e = lambda shape, dt=BF16: torch.empty(shape, dtype=dt, device=dv)
        self.ws = e(max(n, 16), torch.uint8)
        self.h = e((T, f))
        self.y = e((T, d))
        self.gu = self.gu_s = None
        if save == "bf16":
            self.gu = e((T, 2 * f))
        elif save == "int8":
            self.gu = e((T, 2 * f), torch.int8)
            self.gu_s = e((2 * f // 128, T), torch.float32)
        self.dx = e((T, d)) if train else None
        self.dW13 = e((2 * f, d)) if train else None
        self.dW2 = e((d, f)) if train else None
        self.db13 = e(2 * f) if train and bias else None
        self.db2 = e(d) if train and bias else None
        self._h, self._y, self._gu, self._gu_s = _ptr(self.h), _ptr(self.y), _ptr(self.gu), _ptr(self.gu_s)
        self._ws, self.ws_bytes = _ptr(self.ws), self.ws.numel()
        self._grads = tuple(_ptr(t) for t in (self.dx, self.dW13, self.dW2, self.db13, self.db2))

    def _weights(self, W13, W2):
        _dense(W13, (2 * self.f, self.d), BF16, "W13", self.device)
        _dense(W2, (self.d, self.f), BF16, "W2", self.device)

    def forward(self, x, W13, W2, b13=None, b2=None, residual=None):
        dv, T, d, f = self.device, self.T, self.d, self.f
        ldx = rows_of(x, (T, d), BF16, "x", dv)
        self._weights(W13, W2)
        if b13 is not None:
            _dense(b13, (2 * f,), BF16, "b13", dv)
        if b2 is not None:
            _dense(b2, (d,), BF16, "b2", dv)
        if residual is not None:
            _dense(residual, (T, d), BF16, "residual", dv)
        launch("moe_gated_ffn", dv, x.data_ptr(), ldx, W13.data_ptr(), _ptr(b13), W2.data_ptr(), _ptr(b2),
               _ptr(residual), T, d, f, self.act, self._h, self._y, self.save, self._gu, self._gu_s, self._ws,
               self.ws_bytes)
        return self.y

    def backward(self, dy, x, W13, W2, dx_add=None):
        """(dx + dx_add, dW13, dW2, db13, db2) of the last forward for dy [T, d]
        (also the residual's gradient); the bias gradients are None unless the
        plan has them."""
        if not self.save:
            raise ValueError("the plan was made without a save mode")
        dv, T, d, f = self.device, self.T, self.d, self.f
        _dense(dy, (T, d), BF16, "dy", dv)
        ldx = rows_of(x, (T, d), BF16, "x", dv)
        self._weights(W13, W2)
        if dx_add is not None:
            _dense(dx_add, (T, d), BF16, "dx_add", dv)
        launch("moe_gated_ffn_backward", dv, dy.data_ptr(), x.data_ptr(), ldx, W13.data_ptr(), W2.data_ptr(), self.save,
               self._gu, self._gu_s, _ptr(dx_add), T, d, f, self.act, *self._grads, self._ws, self.ws_bytes)
        return self.dx, self.dW13, self.dW2, self.db13, self.db2

    def capture(self, x, W13, W2, b13=None, b2=None, residual=None, warmup=1):
        """``forward`` over these exact buffers as a HIP graph (see ForwardPlan.capture)."""
        return capture_graph(lambda: self.forward(x, W13, W2, b13=b13, b2=b2, residual=residual), warmup, self.device)


class MoELayerPlan:
    """One MoE layer's training step with what surrounds the routed experts:

        logits = x Wr^T + br                     (router, fp32)
        y      = routed experts(x, logits) + shared expert(x)

    on preallocated buffers: a LinearPlan, a TrainPlan and a GatedFFNPlan whose
    sums ride in the products' epilogues (the shared expert adds the routed
    experts' y, the data gradients add up in turn).  act8: x and the shared expert's
    [G, U] are kept in 8 bits for the backward (fs % 128 == 0), 1.03 bytes per
    value.  The router's dWr and the shared expert's dW13s are then products with x
    as restored from them (``xr``, valid after a backward until the next call).
    scoring: experts chosen by scores (see ForwardPlan; ``routed.route_bias`` and
    ``routed.load`` are the balance bias and the experts' load).
    Needs every expert on this GPU (L == E): under expert parallelism d_logits
    has to be summed over the GPUs between the parts."""

    def __init__(self, T, d, f, E, k, fs, act="silu", act8=False, router_bias=False, device="cuda", scoring=None):
        self.T, self.d = T, d
        self.router = LinearPlan(T, d, E, out_dtype=torch.float32, train=True, bias=router_bias, device=device)
        dv = self.router.device
        self.routed = TrainPlan(T, d, f, E, E, k, device=dv, scoring=scoring)
        self.shared = GatedFFNPlan(T, d, fs, act=act, save="int8" if act8 else "bf16", device=dv)
        self.x8 = self.xr = None
        if act8:
            self.x8 = (torch.empty((T, d), dtype=torch.int8, device=dv),
                       torch.empty(((d + 127) // 128, T), dtype=torch.float32, device=dv))
            # x is restored where the routed experts' backward, done by then, had the
            # gradients of its rows (at least T): no memory of its own
            self.xr = self.routed.dX[:T]

    def forward(self, x, Wr, wts, W13s, W2s, br=None, replay=None):
        """y [T, d]; wts from quantize_weights (with its transposed copies where
        ``self.routed.transpose_weights``); replay = (rec, layer, s0) replays
        recorded ids."""
        with _Device(self.router.device):
            if self.x8 is not None:
                ops.act_save(x, out=self.x8)
            logits = self.router.forward(x, Wr, bias=br)
            y = self.routed.forward(x, logits, wts, replay=replay)
            return self.shared.forward(x, W13s, W2s, residual=y)

    def backward(self, dy, x, Wr, wts, W13s, W2s):
        """Gradients of the last forward: dict of dx, dWr, dbr (None without
        router_bias), dW13 and dW2 (routed experts), dW13s and dW2s.  With act8,
        x is not read (None will do)."""
        with _Device(self.router.device):
            # (x is in its own 8-bit copies)
            dx, dW13, dW2, d_logits = self.routed.backward(x, dy, wts, logits=self.router.out)
            if self.x8 is not None:
                x = ops.act_restore(*self.x8, out=self.xr)
            dx, dWr, dbr = self.router.backward(d_logits, x, Wr, dx_add=dx)
            dx, dW13s, dW2s, _, _ = self.shared.backward(dy, x, W13s, W2s, dx_add=dx)
        return dict(dx=dx, dWr=dWr, dbr=dbr, dW13=dW13, dW2=dW2, dW13s=dW13s, dW2s=dW2s)
