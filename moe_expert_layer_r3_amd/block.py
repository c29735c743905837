"""What stands between a model's residual stream and the experts, as plans of
C-ABI calls on preallocated device buffers (no allocation per step): the choice
of experts by scores.

A plan's outputs are its own buffers, valid until its next call."""

import torch

from . import ops
from .layer import capture_graph
from .ops import _dense, _Device

BF16, F32 = torch.bfloat16, torch.float32


def _device(device):
    dv = torch.device(device)
    return dv if dv.index is not None else torch.device("cuda", torch.cuda.current_device())


class RoutePlan:
    """The choice of k of E experts for T tokens by ``scoring`` (ops.Scoring), or
    its replay from a record, and the gradient of its weights when ``train``.
    ids, w: of the last call; status: the MOE_FLAG_* bits of replays, never
    cleared here."""

    def __init__(self, T, E, k, scoring, logits_dtype=F32, train=False, device="cuda"):
        if logits_dtype not in ops.SRC_TYPES:
            raise TypeError(f"logits_dtype: bf16 or fp32, got {logits_dtype}")
        self.T, self.E, self.k, self.scoring, self.logits_dtype = T, E, k, scoring, logits_dtype
        dv = self.device = _device(device)
        self.ids = torch.empty((T, k), dtype=torch.int32, device=dv)
        self.w = torch.empty((T, k), dtype=F32, device=dv)
        self.status = torch.zeros(1, dtype=torch.int32, device=dv)
        self.d_logits = torch.empty((T, E), dtype=logits_dtype, device=dv) if train else None

    def _logits(self, logits):
        _dense(logits, (self.T, self.E), self.logits_dtype, "logits", self.device)

    def forward(self, logits, bias=None, load=None, capture=None):
        """(ids, w) of logits [T, E]; bias, load and capture as for ops.route_scored."""
        self._logits(logits)
        return ops.route_scored(logits, self.k, self.scoring, bias=bias, load=load, capture=capture, out=(self.ids, self.w))

    def replay(self, rec, layer, s0, logits):
        """(ids, w) of tokens s0 .. s0 + T - 1 of a record's layer."""
        self._logits(logits)
        if rec.shape[1] != self.k:
            raise ValueError(f"record top_k {rec.shape[1]} differs from the plan's k {self.k}")
        return ops.replay_scored(rec, layer, s0, logits, self.scoring, status=self.status, out=(self.ids, self.w))

    def backward(self, d_w, logits):
        """d_logits [T, E] of the last call's weights for d_w [T, k]."""
        if self.d_logits is None:
            raise ValueError("the plan was made without train=True")
        self._logits(logits)
        return ops.route_scored_backward(d_w, logits, self.ids, self.scoring, out=self.d_logits)

    def capture(self, logits, bias=None, load=None, warmup=1):
        """``forward`` over these exact buffers as a HIP graph (see ForwardPlan.capture);
        the warm-up calls count into load too."""
        return capture_graph(lambda: self.forward(logits, bias=bias, load=load), warmup)
