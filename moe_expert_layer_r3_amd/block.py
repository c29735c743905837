"""What stands between a model's residual stream and the experts, as plans of
C-ABI calls on preallocated device buffers (no allocation per step): the choice
of experts by scores, the norms in front of and behind the layer, and a layer's
training step from residual stream to residual stream.

A plan's outputs are its own buffers, valid until its next call."""

import torch

from . import ops
from .dense import MoELayerPlan
from .layer import capture_graph
from .ops import _dense, _Device, launch, rows_of, workspace_bytes

BF16, F32 = torch.bfloat16, torch.float32


def _device(device):
    dv = torch.device(device)
    return dv if dv.index is not None else torch.device("cuda", torch.cuda.current_device())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _type(dtype, what):
    if dtype not in ops.SRC_TYPES:
        raise TypeError(f"{what}: bf16 or fp32, got {dtype}")
    return ops.SRC_TYPES[dtype]


class RoutePlan:
    """The choice of k of E experts for T tokens by ``scoring`` (ops.Scoring), or
    its replay from a record, and the gradient of its weights when ``train``.
    ids, w: of the last call; status: the MOE_FLAG_* bits of replays, never
    cleared here."""

    def __init__(self, T, E, k, scoring, logits_dtype=F32, train=False, device="cuda"):
        if logits_dtype not in ops.SRC_TYPES:
            raise TypeError(f"logits_dtype: bf16 or fp32, got {logits_dtype}")
        self.T, self.E, self.k, self.scoring, self.logits_dtype = T, E, k, scoring, logits_dtype
        self.lt = ops.SRC_TYPES[logits_dtype]
        dv = self.device = _device(device)
        self.ids = torch.empty((T, k), dtype=torch.int32, device=dv)
        self.w = torch.empty((T, k), dtype=F32, device=dv)
        self.status = torch.zeros(1, dtype=torch.int32, device=dv)
        self.d_logits = torch.empty((T, E), dtype=logits_dtype, device=dv) if train else None
        self._ids, self._w, self._status, self._d_logits = (_ptr(t) for t in (self.ids, self.w, self.status, self.d_logits))

    def forward(self, logits, bias=None, load=None, capture=None):
        """(ids, w) of logits [T, E]; bias, load and capture as for ops.route_scored."""
        dv, E, c = self.device, self.E, self.scoring
        _dense(logits, (self.T, E), self.logits_dtype, "logits", dv)
        if bias is not None:
            _dense(bias, (E,), F32, "bias", dv)
        if load is not None:
            _dense(load, (E,), torch.int32, "load", dv)
        rec = (None, 0, 0, 0, 0) if capture is None else ops.record_args(*capture, self.k, dv)
        launch("moe_route_scored", dv, logits.data_ptr(), self.lt, self.T, E, self.k, c.code, _ptr(bias), c.groups,
               c.top_groups, c.group_top, c.renorm, c.scale, self._ids, self._w, _ptr(load), *rec)
        return self.ids, self.w

    def replay(self, rec, layer, s0, logits):
        """(ids, w) of tokens s0 .. s0 + T - 1 of a record's layer."""
        dv, c = self.device, self.scoring
        _dense(logits, (self.T, self.E), self.logits_dtype, "logits", dv)
        p, NL, S, layer, s0 = ops.record_args(rec, layer, s0, self.k, dv)
        launch("moe_replay_scored", dv, p, NL, self.k, S, layer, s0, self.T, logits.data_ptr(), self.lt, self.E, c.code,
               c.renorm, c.scale, self._ids, self._w, self._status)
        return self.ids, self.w

    def backward(self, d_w, logits):
        """d_logits [T, E] of the last call's weights for d_w [T, k]."""
        if self.d_logits is None:
            raise ValueError("the plan was made without train=True")
        dv, c = self.device, self.scoring
        _dense(logits, (self.T, self.E), self.logits_dtype, "logits", dv)
        _dense(d_w, (self.T, self.k), F32, "d_w", dv)
        launch("moe_route_scored_backward", dv, d_w.data_ptr(), logits.data_ptr(), self.lt, self._ids, self.T, self.k, self.E,
               c.code, c.renorm, c.scale, self._d_logits)
        return self.d_logits

    def capture(self, logits, bias=None, load=None, warmup=1):
        """``forward`` over these exact buffers as a HIP graph (see ForwardPlan.capture);
        the warm-up calls count into load too."""
        return capture_graph(lambda: self.forward(logits, bias=bias, load=load), warmup, self.device)


class NormPlan:
    """h = x rho w with rho = 1 / sqrt(mean x^2 + eps) for x [T, d] (bf16 or fp32,
    its rows may lie apart), and its gradients when ``train``."""

    def __init__(self, T, d, x_dtype=BF16, w_dtype=BF16, eps=1e-6, train=False, device="cuda"):
        self.T, self.d, self.eps = T, d, eps
        self.x_dtype, self.w_dtype = x_dtype, w_dtype
        self.xt, self.wt = _type(x_dtype, "x_dtype"), _type(w_dtype, "w_dtype")
        dv = self.device = _device(device)
        e = lambda shape, dt: torch.empty(shape, dtype=dt, device=dv)
        self.h = e((T, d), BF16)
        self.rstd = self.dx = self.dw = self.ws = None
        if train:
            with _Device(dv):
                self.ws = e(max(workspace_bytes("moe_norm_backward_workspace", T, d), 16), torch.uint8)
            self.rstd, self.dx, self.dw = e(T, F32), e((T, d), x_dtype), e(d, w_dtype)

    def forward(self, x, w):
        dv, T, d = self.device, self.T, self.d
        ldx = rows_of(x, (T, d), self.x_dtype, "x", dv)
        _dense(w, (d,), self.w_dtype, "w", dv)
        launch("moe_norm", dv, x.data_ptr(), self.xt, ldx, w.data_ptr(), self.wt, T, d, self.eps, self.h.data_ptr(),
               _ptr(self.rstd))
        return self.h

    def backward(self, dh, x, w, dx_add=None):
        """(dx + dx_add, dw) of the last forward for dh [T, d] bf16."""
        if self.ws is None:
            raise ValueError("the plan was made without train=True")
        dv, T, d = self.device, self.T, self.d
        _dense(dh, (T, d), BF16, "dh", dv)
        ldx = rows_of(x, (T, d), self.x_dtype, "x", dv)
        _dense(w, (d,), self.w_dtype, "w", dv)
        if dx_add is not None:
            _dense(dx_add, (T, d), self.x_dtype, "dx_add", dv)
        launch("moe_norm_backward", dv, dh.data_ptr(), x.data_ptr(), self.xt, ldx, w.data_ptr(), self.wt,
               self.rstd.data_ptr(), _ptr(dx_add), T, d, self.dx.data_ptr(), self.dw.data_ptr(), self.ws.data_ptr(),
               self.ws.numel())
        return self.dx, self.dw

    def capture(self, x, w, warmup=1):
        """``forward`` over these exact buffers as a HIP graph (see ForwardPlan.capture)."""
        return capture_graph(lambda: self.forward(x, w), warmup, self.device)


class JoinPlan:
    """What follows a layer's output y [T, d] (bf16), in one pass:

        r_out = r_scale r + y_scale g norm(y; w_post)       h = norm(r_out; w_pre)

    for the residual stream r [T, d] (r_dtype; rows of y and r may lie apart), and
    the gradients of all of it when ``train``.  post / pre: whether the norm behind
    the layer / in front of the next one is there; gate: "none", "channel" [d],
    "token" [T] or "full" [T, d] of gate_dtype, taken through gate_act ("none" or
    "sigmoid")."""

    def __init__(self, T, d, r_dtype=BF16, w_dtype=BF16, post=True, pre=True, gate="none", gate_dtype=BF16, gate_act="none",
                 r_scale=1.0, y_scale=1.0, eps=1e-6, train=False, device="cuda"):
        if gate not in ops.GATES:
            raise ValueError(f"unknown gate {gate!r}: one of {', '.join(ops.GATES)}")
        if gate_act not in ("none", "sigmoid"):
            raise ValueError(f"unknown gate_act {gate_act!r}: none or sigmoid")
        self.T, self.d, self.post, self.pre, self.eps = T, d, post, pre, eps
        self.shape = (T, d)
        self.r_dtype, self.w_dtype, self.gate_dtype = r_dtype, w_dtype, gate_dtype
        self.rt, self.wt = _type(r_dtype, "r_dtype"), _type(w_dtype, "w_dtype")
        self.gate_shape = dict(none=None, channel=(d,), token=(T,), full=(T, d))[gate]
        self.gate_args = (ops.GATES[gate], _type(gate_dtype, "gate_dtype"), ops.ACTS[gate_act], r_scale, y_scale)
        dv = self.device = _device(device)
        e = lambda shape, dt: torch.empty(shape, dtype=dt, device=dv)
        self.r_out = e((T, d), r_dtype)
        self.h = e((T, d), BF16) if pre else None
        self._outs = (self.r_out.data_ptr(), _ptr(self.h))
        self.rstd_post = self.rstd_pre = self.dr = self.dy = self.dw_post = self.dw_pre = self.dgate = self.ws = None
        if train:
            with _Device(dv):
                self.ws = e(max(workspace_bytes("moe_join_backward_workspace", T, d), 16), torch.uint8)
            self.dr, self.dy = e((T, d), r_dtype), e((T, d), BF16)
            if post:
                self.rstd_post, self.dw_post = e(T, F32), e(d, w_dtype)
            if pre:
                self.rstd_pre, self.dw_pre = e(T, F32), e(d, w_dtype)
            if self.gate_shape is not None:
                self.dgate = e(self.gate_shape, gate_dtype)
        self._rstd = (_ptr(self.rstd_post), _ptr(self.rstd_pre))
        self._grads = tuple(_ptr(t) for t in (self.dr, self.dy, self.dw_post, self.dw_pre, self.dgate, self.ws))

    def _weight(self, w, there, name):
        if (w is not None) != there:
            raise ValueError(f"{name}: the plan was made {'with' if there else 'without'} this norm")
        if there:
            _dense(w, (self.d,), self.w_dtype, name, self.device)

    def _operands(self, y, w_post, gate, w_pre):
        dv = self.device
        ldy = rows_of(y, self.shape, BF16, "y", dv)
        self._weight(w_post, self.post, "w_post")
        self._weight(w_pre, self.pre, "w_pre")
        if (gate is not None) != (self.gate_shape is not None):
            raise ValueError("gate: not as the plan was made")
        if gate is not None:
            _dense(gate, self.gate_shape, self.gate_dtype, "gate", dv)
        return ldy

    def forward(self, y, r, w_post=None, gate=None, w_pre=None):
        """(r_out, h); h is None without the norm in front of the next layer."""
        dv, T, d = self.device, self.T, self.d
        ldy = self._operands(y, w_post, gate, w_pre)
        ldr = rows_of(r, (T, d), self.r_dtype, "r", dv)
        launch("moe_join", dv, y.data_ptr(), ldy, r.data_ptr(), self.rt, ldr, _ptr(w_post), _ptr(gate), *self.gate_args,
               _ptr(w_pre), self.wt, T, d, self.eps, *self._outs, *self._rstd)
        return self.r_out, self.h

    def backward(self, d_out, dh, y, w_post=None, gate=None, w_pre=None):
        """Gradients of the last forward for d_out [T, d] of r_dtype (along the
        residual stream; None: zero) and dh [T, d] bf16 (of h; None without it):
        dict of dr, dy, dw_post, dw_pre and dgate (None where there is none)."""
        if self.ws is None:
            raise ValueError("the plan was made without train=True")
        dv, T, d = self.device, self.T, self.d
        ldy = self._operands(y, w_post, gate, w_pre)
        if (dh is not None) != self.pre:
            raise ValueError(f"dh: the plan was made {'with' if self.pre else 'without'} the norm that gives h")
        if d_out is not None:
            _dense(d_out, (T, d), self.r_dtype, "d_out", dv)
        if dh is not None:
            _dense(dh, (T, d), BF16, "dh", dv)
        launch("moe_join_backward", dv, _ptr(d_out), _ptr(dh), y.data_ptr(), ldy, self.r_out.data_ptr(), self.rt,
               _ptr(w_post), _ptr(gate), *self.gate_args, _ptr(w_pre), self.wt, *self._rstd, T, d, *self._grads,
               self.ws.numel())
        return dict(dr=self.dr, dy=self.dy, dw_post=self.dw_post, dw_pre=self.dw_pre, dgate=self.dgate)

    def capture(self, y, r, w_post=None, gate=None, w_pre=None, warmup=1):
        """``forward`` over these exact buffers as a HIP graph (see ForwardPlan.capture)."""
        return capture_graph(lambda: self.forward(y, r, w_post=w_post, gate=gate, w_pre=w_pre), warmup, self.device)


class MoEBlockPlan:
    """One layer's training step on the residual stream: with h = norm(r) from the
    block before (its ``w_next``) or a NormPlan in front of the first,

        y = layer(h)                                      (MoELayerPlan)
        r_out, h_next = join(y, r)                        (JoinPlan)

    on preallocated buffers.  scoring, act, act8 and router_bias as MoELayerPlan
    takes them; r_dtype, w_dtype, post, gate, gate_dtype, gate_act, r_scale,
    y_scale and eps as JoinPlan does; next_norm: whether a block follows."""

    def __init__(self, T, d, f, E, k, fs, scoring=None, act="silu", act8=False, router_bias=False, r_dtype=BF16,
                 w_dtype=BF16, post=False, next_norm=True, gate="none", gate_dtype=BF16, gate_act="none", r_scale=1.0,
                 y_scale=1.0, eps=1e-6, device="cuda"):
        self.layer = MoELayerPlan(T, d, f, E, k, fs, act=act, act8=act8, router_bias=router_bias, scoring=scoring,
                                  device=device)
        self.join = JoinPlan(T, d, r_dtype=r_dtype, w_dtype=w_dtype, post=post, pre=next_norm, gate=gate,
                             gate_dtype=gate_dtype, gate_act=gate_act, r_scale=r_scale, y_scale=y_scale, eps=eps, train=True,
                             device=self.layer.router.device)

    def forward(self, r, h, Wr, wts, W13s, W2s, br=None, w_post=None, gate=None, w_next=None, replay=None):
        """(r_out, h_next) for the stream r [T, d] and its norm h [T, d]; weights as
        MoELayerPlan.forward and JoinPlan.forward take them."""
        y = self.layer.forward(h, Wr, wts, W13s, W2s, br=br, replay=replay)
        return self.join.forward(y, r, w_post=w_post, gate=gate, w_pre=w_next)

    def backward(self, d_r, d_h, h, Wr, wts, W13s, W2s, w_post=None, gate=None, w_next=None):
        """Gradients of the last forward for d_r (of r_out along the stream) and d_h
        (of h_next; None without it): the layer's (dx as ``dh``, of h) and the
        join's (``dr``, of r along the stream; dw_post, dw_next, dgate).  The block
        before takes (dr, dh) as its (d_r, d_h)."""
        g = self.join.backward(d_r, d_h, self.layer.shared.y, w_post=w_post, gate=gate, w_pre=w_next)
        out = self.layer.backward(g["dy"], h, Wr, wts, W13s, W2s)
        out["dh"] = out.pop("dx")
        out.update(dr=g["dr"], dw_post=g["dw_post"], dw_next=g["dw_pre"], dgate=g["dgate"])
        return out
