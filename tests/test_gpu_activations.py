"""The activations of the products' epilogue far out, relative to their values, in float32.  With
activations of zero z is the bias itself, so what is compared is the function.

Bounds, with u = 2^-24.  sigmoid(x) is one exponential of a rounded product of x and a rounded
constant (2 |x| u), with hardware exponential, sum, reciprocal and product (2, 1, 2 and 1 u, taken
as 8): 8 u + 2 |x| u.  silu: that.  gelu_tanh: its argument v is a sum of two terms of one sign with
five roundings, so 8 u + (2 + 5) |v| u.  gelu: z^2 and its product with a rounded constant (3 u of
z^2 / 2), a polynomial of nine terms in a reciprocal (2 u) whose slopes are below 1 and whose
roundings are below 4 u, the exponential and three products: 10 u + 1.5 z^2 u, taken as 16 u (1 +
z^2).  Below 2^-118 results may be flushed to zero."""
import math

import pytest
import torch

from bit_lifted_gemv_amd import lq

pytestmark = pytest.mark.gpu

U = 2.0**-24


def exact(z, act):
    """Value and relative bound in float64."""
    if act == "silu":
        return z * torch.special.expit(z), (8 + 2 * z.abs()) * U
    if act == "gelu_tanh":
        v = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z**3)
        return z * torch.special.expit(v), (8 + 7 * v.abs()) * U
    if act == "gelu":
        return z * torch.erfc(-z * math.sqrt(0.5)) / 2, 16 * U * (1 + z * z)
    return torch.clamp(z, min=0.0), torch.zeros_like(z)


# few rows in one slice, few rows in slices, many rows, many rows in slices
@pytest.mark.parametrize("B,K", [(1, 128), (5, 65536), (300, 256), (40, 16384)])
@pytest.mark.parametrize("act,far", [("gelu", 13.0), ("silu", 80.0), ("gelu_tanh", 7.0), ("relu", 1e30)])
def test_activations_far_out(act, far, B, K):
    m = 4096
    z = torch.cat([torch.linspace(-far, far, m // 2), torch.logspace(-8, math.log10(far), m // 4),
                   -torch.logspace(-8, math.log10(far), m // 4)]).cuda()
    w = torch.randint(-2**31, 2**31, (m, K // 32)).to(torch.int32).cuda()
    s = torch.rand(m, device="cuda") + 0.5
    out = lq.gemm_ep(w, s, torch.zeros(B, K, dtype=torch.bfloat16, device="cuda"), bias=z, act=act,
                     out_dtype=torch.float32)
    y, near = exact(z.double(), act)
    off = (out.double() - y).abs()
    assert (off <= near * y.abs() + 2.0**-118).all(), float((off / (near * y.abs() + 2.0**-118)).max())
