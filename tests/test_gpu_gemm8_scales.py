"""Scales of lq_gemm8 over their whole range.

Every value times its block's power of two lies within float32's normal range, which
is all that the product asks of exponents.  Sums are exact here: within a block
values are multiples of 1/2 up to 7, products multiples of 1/4 below 2^6; the powers of two
of the two operands cancel but for 2^-2 .. 2^2; so all terms are multiples of 2^-4 and
sums of up to 1280 of them stay below 2^6 2^2 1280 < 2^19: 23 bits, exact in float32 in
any order, and no product lies 2^13 below another of its eight.  Results are the exact
sums, rounded once by a 16-bit output.
"""
import pytest
import torch

from bit_lifted_gemv_amd import lq

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2

# the few-row kernel in one slice and in several, and every tile of the many-row kernel
SIZES = [(384, 1280, 1), (200, 1200, 3), (31, 1100, 15), (384, 1280, 300), (129, 640, 21760), (4096, 512, 2048),
         (4096, 300, 4000)]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"


def held(exps):
    """Exponents whose rows are whole words."""
    rows, blocks = exps.shape
    out = torch.zeros(rows, blocks + -blocks % 4, dtype=torch.uint8)
    out[:, :blocks] = exps
    return out.cuda()[:, :blocks]


def values(rows, K, exps, g):
    """Values that stay normal times 2^(exps - 127) (a byte per row and 128 positions): small
    for large exponents, large for small ones; zeros behind K."""
    width = exps.shape[1] * 128
    v = torch.randint(2, 8, (rows, width), generator=g).float()
    small = torch.randint(0, 2, (rows, width), generator=g) * 0.5 + 1.0                  # 1 or 1.5
    v = torch.where(exps.repeat_interleave(128, 1) > 250, small, v)
    v *= torch.randint(-1, 2, (rows, width), generator=g)
    v[:, K:] = 0.0
    return v


def operands(m, K, B, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    blocks, strips = -(-K // 128), -(-m // 128)
    at = torch.tensor([0, 254, 1, 253, 127, 60, 200, 2, 252, 130])[(torch.arange(blocks) * 3 + seed) % 10]
    we = (at + torch.randint(-1, 2, (strips, blocks), generator=g)).clamp(0, 254)
    ae = (254 - at + torch.randint(-1, 2, (B, blocks), generator=g)).clamp(0, 254)
    w = values(m, K, we.repeat_interleave(128, 0)[:m], g)
    a = values(B, K, ae, g)
    weights = lq.Blocks8(w.to(E4M3).cuda(), held(we))
    rows = lq.Rows8(a.to(dtype).cuda(), held(ae))
    return weights, rows


def exact(w, a):
    """The sums in float64 (2^-127 to 2^127 and back are well inside)."""
    m = w.values.shape[0]
    W = w.values.double() * torch.exp2(w.scales.double() - 127).repeat_interleave(128, 0)[:m].repeat_interleave(128, 1)
    return (a.values.double() * torch.exp2(a.exps.double() - 127).repeat_interleave(128, 1)) @ W.T


@pytest.mark.parametrize("out", [F16, BF16, F32])
@pytest.mark.parametrize("dtype", [E4M3, E5M2])
@pytest.mark.parametrize("m,K,B", SIZES)
def test_exponents_from_end_to_end(m, K, B, dtype, out):
    for seed in (0, 1, 5):
        w, a = operands(m, K, B, dtype, seed)
        want = exact(w, a)
        assert torch.equal(lq.gemm8(w, a, out_dtype=out), want.float().to(out))
