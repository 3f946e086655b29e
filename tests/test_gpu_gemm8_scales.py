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


def one_value(m, K, B, at, w_value, a_value, w_byte, a_byte, w_scale=None):
    """A single position of every row and token that is not zero, in a block of those scales."""
    w, a = torch.zeros(m, K), torch.zeros(B, K)
    w[:, at], a[:, at] = w_value, a_value
    we, ae = torch.full((-(-m // 128), K // 128), 127), torch.full((B, K // 128), 127)
    we[:, at // 128], ae[:, at // 128] = w_byte, a_byte
    scales = held(we)
    if w_scale is not None:
        scales = torch.ones(we.shape, device="cuda")
        scales[:, at // 128] = w_scale
    return lq.Blocks8(w.to(E4M3).cuda(), scales), lq.Rows8(a.to(E4M3).cuda(), held(ae))


@pytest.mark.parametrize("out", [F16, BF16, F32])
@pytest.mark.parametrize("m,B", [(256, 1), (256, 3), (256, 300), (129, 21760), (4096, 2048), (4096, 4000)])
def test_the_byte_255_is_a_nan(m, B, out):
    """In the outputs that read the block, and in no others; also where the block's values are zeros."""
    K = 384
    for value in (1.0, 0.0):
        w, a = one_value(m, K, B, 200, value, value, 127, 127)
        clean = lq.gemm8(w, a, out_dtype=out)
        w.scales[m // 128 - 1, 1] = 255
        got = lq.gemm8(w, a, out_dtype=out)
        lo = (m // 128 - 1) * 128
        hit = (torch.arange(m, device="cuda") >= lo) & (torch.arange(m, device="cuda") < lo + 128)
        assert torch.isnan(got[:, hit]).all() and torch.equal(got[:, ~hit], clean[:, ~hit])
        w.scales[m // 128 - 1, 1] = 127
        a.exps[B - 1, 1] = 255
        got = lq.gemm8(w, a, out_dtype=out)
        assert torch.isnan(got[B - 1]).all() and torch.equal(got[:B - 1], clean[:B - 1])


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("B", [1, 3, 300, 4000])
def test_float32_scales_of_any_size(B, out):
    """Both signs, near the ends of float32, infinities and NaN.  The block's sum before its scale is a float32 number:
    exact here, so one rounding for the scale and one for the output."""
    for scale, value, byte in ((2.0**-120, 3.0, 245), (2.0**120, 3.0, 6), (-3e38, 1.5, 10), (1.2e-38, 448.0, 200), (0.0, 5.0, 127),
                               (1.7e38, 0.001953125, 127), (-1e-30, 448.0, 230)):
        w, a = one_value(256, 384, B, 130, value, 1.0, 127, byte, scale)
        want = torch.tensor(scale).double().item() * value * 2.0**(byte - 127)
        got = lq.gemm8(w, a, out_dtype=out).double()
        assert ((got - want).abs() <= (2.0**-24 + torch.finfo(out).eps / 2 * 1.001) * abs(want)).all()
    w, a = one_value(256, 384, B, 130, 2.0, 1.0, 127, 127, float("inf"))
    assert (lq.gemm8(w, a, out_dtype=out) == float("inf")).all()
    w, a = one_value(256, 384, B, 130, 2.0, 1.0, 127, 127, float("nan"))
    assert torch.isnan(lq.gemm8(w, a, out_dtype=out)).all()
