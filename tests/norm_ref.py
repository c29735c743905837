"""Plain 64-bit forms of the norms around the layer and the bounds their kernels
have to keep (not collected by pytest).

u = 2^-24. A sum of n terms held in fp32 in any order is off by at most (n + 8) u
of the sum of their sizes.  Everything a kernel computes from one row is a short
chain of fp32 operations (at most 16 roundings: CHAIN u of the terms' sizes); rho
comes from a sum of d squares, all of one sign, so it is off by at most
((d + 8) u / 2 + 4 u) of itself (RHO).  A result is rounded once to its type:
u in fp32, 2^-8 in bf16 (ROUND), half the smallest step where it is subnormal."""

import torch

U = 2.0 ** -24
CHAIN = 16
ROUND = {torch.float32: U * 1.001, torch.bfloat16: (2.0 ** -8 + U) * 1.001}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -134}


def d64(t):
    return None if t is None else t.detach().cpu().double()


def rho_err(d):
    return ((d + 8) / 2 + 4) * U


def rho_of(v, eps):
    return 1.0 / torch.sqrt((v * v).mean(dim=1, keepdim=True) + eps)


def norm(v, w, eps):
    """(norm, rho)."""
    rho = rho_of(v, eps)
    return v * rho * w, rho


def norm_back(a, v, rho, ea):
    """Gradient of v * rho for the gradient a that is off by at most ea, and its bound."""
    d = v.shape[1]
    vh, e = v * rho, rho_err(d)
    mean = (a * vh).mean(dim=1, keepdim=True)
    big = (a * vh).abs().mean(dim=1, keepdim=True)
    out = rho * (a - vh * mean)
    emean = (ea * vh.abs()).mean(dim=1, keepdim=True) + big * ((d + 8) * U + e + CHAIN * U)
    err = rho * (ea + vh.abs() * emean + (a.abs() + vh.abs() * mean.abs()) * (2 * e + CHAIN * U))
    return out, err


def close(got, ref, err, what):
    """Every element within err, rounded to got's type."""
    t = got.dtype
    tol = err + ROUND[t] * (ref.abs() + err) + TINY[t]
    g = d64(got)
    assert torch.equal(g.isnan(), ref.isnan()), what + ": NaN elsewhere"
    bad = ~((g - ref).abs() <= tol) & ~ref.isnan()
    if bool(bad.any()):
        r = torch.where(bad, (g - ref).abs() / tol, torch.zeros(()).double())
        i = int(r.argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst at {i}: got {g.flatten()[i]:.9g}, "
                             f"want {ref.flatten()[i]:.9g} +- {tol.flatten()[i]:.3g}")


def gate_of(gate, kind, act, T, d):
    """(value, slope) in a shape that broadcasts to [T, d]."""
    if kind == "none":
        one = torch.ones(1, 1, dtype=torch.float64)
        return one, one
    g = d64(gate).reshape(dict(channel=(1, d), token=(T, 1), full=(T, d))[kind])
    if act == "sigmoid":
        return torch.sigmoid(g), torch.sigmoid(g) * torch.sigmoid(-g)
    return g, torch.ones_like(g)


def column(terms, eterms, T):
    """(sum over the tokens, bound): each term off by eterms, T terms added in fp32."""
    return terms.sum(dim=0), eterms.sum(dim=0) + (T + 16) * U * (terms.abs() + eterms).sum(dim=0)
