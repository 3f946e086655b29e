"""lq_gemm8 and lq_gemm8_grouped on 16-bit activations: the same results, bit for bit, as on
activations that lq_quant8 quantized before (both calls take the same kernel in the
same order), whether the call quantizes them by a launch of its own or, for up to four tokens,
on their way into LDS; also where the positions are split, rows lie apart and no 16-byte
piece of them is aligned, and for runs of one to four rows."""
import pytest
import torch

from bit_lifted_gemv_amd import lq

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"


def weights(m, K, kind, seed, E=0):
    g = torch.Generator().manual_seed(seed)
    q = lq.quantize8_blocks(torch.randn(*((E,) if E else ()), m, K, generator=g).cuda())
    if kind == F32:
        return lq.Blocks8(q.values, torch.exp2(q.scales.float() - 127) * (torch.rand(q.scales.shape, generator=g) + 0.5).cuda())
    return q


def activations(B, K, dtype, seed, pitch=0):
    g = torch.Generator().manual_seed(seed)
    a = torch.randn(B, K + pitch, generator=g) * torch.exp(2 * torch.randn(B, 1, generator=g))
    return a.to(dtype).cuda()[:, :K]


# in LDS: one slice of up to 128 blocks of one token, 64 of two, 32 of four; two slices; the rest is quantized by a launch
FEW = [(31, 20000, 1), (200, 16384, 2), (4096, 4096, 1), (130, 8192, 2), (514, 5000, 3), (2048, 4096, 4), (64, 77, 4),
       (31, 20000, 4), (512, 16400, 1)]
MANY = [(130, 515, 5), (130, 515, 16), (514, 2048, 17), (64, 1000, 300), (1000, 5000, 40), (129, 300, 21760), (4096, 520, 2048), (4096, 520, 4000)]


@pytest.mark.parametrize("kind", [torch.uint8, F32])
@pytest.mark.parametrize("out", [F16, BF16, F32])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("m,K,B", FEW + MANY)
def test_as_quantized_before(m, K, B, dtype, out, kind):
    w = weights(m, K, kind, m + K)
    for pitch in (0, 1, 8):
        a = activations(B, K, dtype, B + pitch, pitch)
        q = lq.quantize8(a.contiguous())
        for gated in (False, True)[:1 + (m % 2 == 0)]:
            assert torch.equal(lq.gemm8(w, a, act="silu", gated=gated, out_dtype=out),
                               lq.gemm8(w, q, act="silu", gated=gated, out_dtype=out))


@pytest.mark.parametrize("kind", [torch.uint8, F32])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("m,K,B", FEW)
def test_few_against_float64(m, K, B, dtype, kind):
    """Float32 results: 2^-19 of the sum of magnitudes for the additions (at most 160 blocks of 128 positions, whose
    sums of four instructions follow one another: sqrt(640) 2^-24 < 2^-19, of errors that add like independent ones)."""
    w, a = weights(m, K, kind, m + K), activations(B, K, dtype, B)
    q = lq.quantize8(a)
    s = w.scales.double() if kind == F32 else torch.exp2(w.scales.double() - 127)
    W = w.values.double() * s.repeat_interleave(128, 0)[:m].repeat_interleave(128, 1)
    A = q.values.double() * torch.exp2(q.exps.double() - 127).repeat_interleave(128, 1)
    assert ((lq.gemm8(w, a, out_dtype=F32).double() - A @ W.T).abs() <= 2.0**-19 * (A.abs() @ W.abs().T)).all()


@pytest.mark.parametrize("kind", [torch.uint8, F32])
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("m,K", [(70, 300), (1000, 4096), (34, 20000), (256, 16384)])
def test_runs_of_up_to_four_rows(m, K, dtype, out, kind):
    """Rows to different experts, gathered, repeated and invalid, and rows behind the last run."""
    E = 5
    w = weights(m, K, kind, 3, E)
    bias = torch.randn(E, m, device="cuda")
    for rows, ends in (([2], [0, 0, 1, 1, 1, 1]), ([1, 0], [0, 1, 1, 2, 2, 2]), ([0, -1, 2], [0, 0, 0, 2, 3, 3]),
                       ([2, 2, 7, 0], [0, 1, 1, 1, 2, 4]), ([1, 1, 0, 2], [0, 4, 4, 4, 4, 4]), ([0, 2, 1, 1], [0, 0, 1, 3, 3, 3]),
                       (None, [0, 1, 1, 2, 2, 3]), (None, [0, 0, 0, 0, 0, 2])):
        a = activations(3, K, dtype, 4)
        q = lq.quantize8(a)
        R = 3 if rows is None else len(rows)
        rows = None if rows is None else torch.tensor(rows, dtype=torch.int32, device="cuda")
        offsets = torch.tensor(ends, dtype=torch.int32, device="cuda")
        for gated in (False, True):
            one, two = (torch.full((R, m // 2 if gated else m), 9.0, dtype=out, device="cuda") for _ in range(2))
            lq.gemm8_grouped(w, a, offsets, rows=rows, bias=bias, act="gelu", gated=gated, out=one)
            lq.gemm8_grouped(w, q, offsets, rows=rows, bias=bias, act="gelu", gated=gated, out=two)
            assert torch.equal(one, two) and (one[ends[-1]:] == 9.0).all()
            if out == F32 and not gated:
                A = q.values.double() * torch.exp2(q.exps.double() - 127).repeat_interleave(128, 1)
                for e in range(E):
                    s = w.scales[e].double() if kind == F32 else torch.exp2(w.scales[e].double() - 127)
                    W = w.values[e].double() * s.repeat_interleave(128, 0)[:m].repeat_interleave(128, 1)
                    for r in range(ends[e], ends[e + 1]):
                        t = r if rows is None else int(rows[r])
                        x = A[t] if 0 <= t < 3 else torch.zeros_like(A[0])
                        z = W @ x + bias[e].double()
                        want = z * torch.special.ndtr(z)
                        bound = 1.13 * (2.0**-19 * (W.abs() @ x.abs()) + 2.0**-23 * (z.abs() + bias[e].double().abs()))
                        assert ((one[r].double() - want).abs() <= bound + 2.0**-20 * (z.abs() + 1.0) + 2.0**-23 * want.abs()).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("R", [1, 5, 40, 700])
def test_gathered_rows_as_quantized_before(R, dtype):
    g = torch.Generator().manual_seed(R)
    w, a = weights(130, 700, torch.uint8, 1, 6), activations(50, 700, dtype, 2)
    rows = torch.randint(-1, 51, (R,), generator=g).int().cuda()
    offsets = torch.tensor([0, R // 7, R // 3, R // 3, R // 2, R, R], dtype=torch.int32, device="cuda")
    for out in (F16, BF16, F32):
        assert torch.equal(lq.gemm8_grouped(w, a, offsets, rows=rows, out_dtype=out),
                           lq.gemm8_grouped(w, lq.quantize8(a), offsets, rows=rows, out_dtype=out))
