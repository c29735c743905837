"""Plain 64-bit forms of the dense products and the bounds their bf16 / fp32
kernels have to keep (not collected by pytest).

Bounds, for values v computed from bf16 operands:
  - a sum of K exact products held in fp32, in any order, is off by at most
    (K + 8) 2^-24 sum |a b| (each of its at most K + 7 additions, split pieces
    and bias included, rounds by 2^-24 of a partial sum that sum |a b| bounds);
  - bf16 rounding of the result: 2^-8 |v| (half of eps = 2^-7);
  - the activations' own error: exp2, reciprocal and erf are good to a few
    2^-24; 2^-20 (|z| + 1) covers each with room for the argument's rounding
    (|z| 2^-24 1.44 in the exponent)."""

import math

import torch

U16 = 2.0 ** -8       # bf16 rounding
ACT_ERR = 2.0 ** -20
SLOPE = 1.13          # largest |act'| of silu (1.0998), gelu (1.1290), relu, sigmoid


REF = ["cpu"]         # where the 64-bit forms are computed (large cases: on the GPU)


def d64(t):
    return None if t is None else t.detach().to(REF[0]).double()


def acc_err(K, a, b):
    """Bound of the fp32 accumulation of a @ b (64-bit matrices)."""
    return (K + 8) * 2.0 ** -24 * (a.abs() @ b.abs())


def act(name, z):
    """(value, slope) in 64 bits."""
    if name == "relu":
        return torch.where(z.isnan(), z, z.clamp_min(0)), (z > 0).double()
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    if name == "sigmoid":
        s = torch.sigmoid(z)
        return s, s * (1 - s)
    if name == "gelu":
        c = 0.5 * (1 + torch.erf(z / math.sqrt(2)))
        return z * c, c + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return z, torch.ones_like(z)


def close(got, ref, tol, what):
    """Every element within its bound; the message names the worst."""
    got = d64(got)
    bad = ~((got - ref).abs() <= tol)
    if bool(bad.any()):
        r = ((got - ref).abs() / tol.clamp_min(1e-300))
        i = int(torch.nan_to_num(r, nan=float("inf")).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst at {i}: got "
                             f"{got.flatten()[i]:.6g}, want {ref.flatten()[i]:.6g} +- {tol.flatten()[i]:.3g}")


def keep8(v):
    """(codes, scales [blocks, rows]) of fp32 rows in blocks of 128 columns."""
    rows, cols = v.shape
    nb = (cols + 127) // 128
    p = torch.zeros(rows, nb * 128, dtype=torch.float32)
    p[:, :cols] = v
    p = p.view(rows, nb, 128)
    a = p.abs().amax(2).clamp_min(2.0 ** -100)
    q = torch.round(p * (torch.tensor(127.0) / a)[:, :, None])
    return q.view(rows, nb * 128)[:, :cols], (a / torch.tensor(127.0)).t().contiguous()


def spread(s, cols):
    """Scales [blocks, rows] as one per element [rows, cols]."""
    return s.t().repeat_interleave(128, dim=1)[:, :cols]
