"""A mixture-of-experts layer held in 8 bits, as it would be used: router, rows
quantized and sorted, products, join, and the gradients back through them."""
import pytest
import torch

from bit_lifted_gemv_amd import lq

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"


def matrix64(values, scales):
    s = scales.double() if scales.dtype == F32 else torch.exp2(scales.double() - 127)
    m = values.shape[0]
    return values.double() * s.repeat_interleave(128, 0)[:m].repeat_interleave(128, 1)


def rows64(a):
    return a.values.double() * torch.exp2(a.exps.double() - 127).repeat_interleave(128, 1)


def layer(T, E, k, n, f, seed, padded=0.1):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, n, generator=g).to(BF16).cuda()
    w1 = lq.quantize8_blocks((torch.randn(E, 2 * f, n, generator=g) * n**-0.5).cuda())
    w2 = lq.quantize8_blocks((torch.randn(E, n, f, generator=g) * f**-0.5).cuda())
    valid = (torch.rand(T, generator=g) >= padded).to(torch.uint8).cuda()
    r = lq.route(torch.randn(T, E, generator=g).cuda(), k, valid=valid)
    return x, w1, w2, r


@pytest.mark.parametrize("T,E,k,n,f", [(1, 8, 2, 256, 200), (24, 16, 4, 300, 128), (333, 8, 2, 256, 392)])
def test_forward(T, E, k, n, f):
    """Against a per-token float64 evaluation of the same quantized numbers."""
    x, w1, w2, r = layer(T, E, k, n, f, T)
    q = lq.quantize8(x)
    h = lq.gemm8_grouped(w1, q, r.offsets, rows=r.rows, act="silu", gated=True, out_dtype=BF16)
    qh = lq.quantize8(h)
    z = lq.gemm8_grouped(w2, qh, r.offsets, out_dtype=F32)
    y = lq.join_rows(z, r.pos, r.weight, residual=x, out_dtype=BF16)
    sorted_h = lq.gemm8_grouped(w1, lq.sort_rows(q, r.rows), r.offsets, act="silu", gated=True, out_dtype=BF16)
    used = int(r.offsets[-1])
    assert torch.equal(sorted_h[:used], h[:used])
    x64, h64 = rows64(q), rows64(qh)
    for t in range(0, T, max(1, T // 7)):
        want = x[t].double()
        size = want.abs()
        for j in range(k):
            e, p = int(r.ids[t, j]), int(r.pos[t, j])
            if e < 0:
                continue
            u = matrix64(w1.values[e], w1.scales[e]) @ x64[t]
            act = u[:f] * torch.special.expit(u[:f]) * u[f:]
            assert ((h[p].double() - act).abs() <= 2.0**-8 * act.abs() + 1e-4).all()
            W2 = matrix64(w2.values[e], w2.scales[e])
            term = r.weight[t, j].double() * (W2 @ h64[p])
            want, size = want + term, size + r.weight[t, j].double() * (W2.abs() @ h64[p].abs())
        assert ((y[t].double() - want).abs() <= 2.0**-8 * want.abs() + 2.0**-18 * size).all()


def test_gradients_of_the_way_out():
    """y = join(z, weight), z = w2 . h per expert, h = the tokens' sorted rows: the gradients of the weights and of the
    tokens, against the formulas in float64 on the numbers that each step is given."""
    T, E, k, n, f = 60, 8, 2, 256, 256
    x, _, w2, r = layer(T, E, k, n, f, 5)
    dy = torch.randn(T, n, device="cuda")
    q = lq.quantize8(x)
    z = lq.gemm8_grouped(w2, q, r.offsets, rows=r.rows, out=torch.zeros(T * k, n, device="cuda"))
    dz, dweight = lq.join_rows_grad(dy, z, r.pos, r.weight, r.rows)
    qz = lq.quantize8(dz, torch.float8_e5m2)
    dh = lq.gemm8_grouped(w2.transposed(), qz, r.offsets, out=torch.zeros(T * k, f, device="cuda"))
    dx = lq.join_rows(dh, r.pos)
    W = [matrix64(w2.values[e], w2.scales[e]) for e in range(E)]
    x64, qz64 = rows64(q), rows64(qz)
    for t in range(T):
        back = torch.zeros(f, dtype=torch.float64, device="cuda")
        size = back.clone()
        for j in range(k):
            e, p = int(r.ids[t, j]), int(r.pos[t, j])
            if e < 0:
                assert dweight[t, j] == 0
                continue
            row = W[e] @ x64[t]
            terms = dy[t].double() * row
            assert abs(dweight[t, j].item() - terms.sum().item()) <= 2.0**-16 * (dy[t].double().abs() @ (W[e].abs() @ x64[t].abs())).item()
            back, size = back + qz64[p] @ W[e], size + qz64[p].abs() @ W[e].abs()
        assert ((dx[t].double() - back).abs() <= 2.0**-19 * size).all()
