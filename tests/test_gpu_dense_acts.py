"""The activations of the dense products far into their tails, relative to their
own size.

Bounds, for z exact in bf16 and a weight matrix that is the identity:
  - gelu(z) = z Phi(z): Phi from the complementary error function at |z| / sqrt 2.
    The argument's two roundings (product and constant) move ln Phi by at most
    2^-23 z (z + 1), the function itself by a few 2^-24 (64 are allowed), products 3:
    relative (2 z^2 + 2 |z| + 70) 2^-24
  - its slope Phi + z phi: the same for Phi; the exponent of phi is two products
    and a constant, 1.5 z^2 2^-24 absolute, and 8 2^-24 for exp2 and the products:
    (2 z^2 + 2 |z| + 70) 2^-24 of Phi + |z| phi
  - sigmoid and its slope s(z) s(-z): the exponent's two roundings |z| 2^-23, exp2,
    reciprocal and products 8 2^-24, squared at most: (4 |z| + 16) 2^-24
  - dz is rounded to bf16 for the products: 2^-8 of the slope"""

import math

import pytest
import torch

from dense_ref import U16, close
from gpu_util import DEV
from moe_expert_layer_r3_amd.dense import GatedFFNPlan, LinearPlan

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def grid(lo, hi):
    """Rows of eight values between lo and hi, exact in bf16."""
    return torch.linspace(lo, hi, 320).to(BF).view(40, 8)


def forms(name, z):
    """(value, slope, what the slope's bound is relative to, bound in 2^-24) in 64 bits."""
    z = z.double()
    if name == "gelu":
        c = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        p = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        return z * c, c + z * p, c + z.abs() * p, 2 * z * z + 2 * z.abs() + 70
    s, r = torch.sigmoid(z), torch.sigmoid(-z)
    return s, s * r, s * r, 4 * z.abs() + 16


@pytest.mark.parametrize("name, lo, hi", [("gelu", -12, -3), ("gelu", -3, 3), ("gelu", 3, 12), ("sigmoid", -60, -4),
                                          ("sigmoid", -4, 4), ("sigmoid", 4, 60)])
def test_tails(name, lo, hi):
    z = grid(lo, hi)
    W = torch.eye(8).to(BF).to(DEV)
    p = LinearPlan(40, 8, 8, act=name, out_dtype=torch.float32, train=True, device=DEV)
    out = p.forward(z.to(DEV), W)
    val, slope, mag, e = forms(name, z)
    close(out, val, e * 2.0 ** -24 * val.abs() + 1e-300, "value")
    dx, _, _ = p.backward(torch.ones(40, 8, device=DEV), z.to(DEV), W)
    e = e * 2.0 ** -24 * mag
    close(dx, slope, e + U16 * (slope.abs() + e), "slope")


@pytest.mark.parametrize("name, lo, hi", [("gelu", -12, -3), ("sigmoid", 4, 60)])
@pytest.mark.parametrize("save", ["bf16", "none"])
def test_gated_tails(name, lo, hi, save):
    """h = act(G) U with U = 1 by its bias, and dG = act'(G), dU = act(G) by way of
    dx = [dG, dU] W13 with one of the halves of W13 zero."""
    z = grid(lo, hi)
    W13 = torch.cat([torch.eye(8), torch.zeros(8, 8)]).to(BF).to(DEV)
    b13 = torch.cat([torch.zeros(8), torch.ones(8)]).to(BF).to(DEV)
    W2 = torch.eye(8).to(BF).to(DEV)
    p = GatedFFNPlan(40, 8, 8, act=name, save=save, bias=save != "none", device=DEV)
    y = p.forward(z.to(DEV), W13, W2, b13=b13)
    val, slope, mag, e = forms(name, z)
    e1 = e * 2.0 ** -24 * val.abs()
    close(y, val, e1 + U16 * (val.abs() + e1) + 1e-300, "y")
    if save == "none":
        return
    dx = p.backward(torch.ones(40, 8, dtype=BF, device=DEV), z.to(DEV), W13, W2)[0]
    e = e * 2.0 ** -24 * mag
    close(dx, slope, e + U16 * (slope.abs() + e), "dx")
