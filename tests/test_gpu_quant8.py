"""lq_quant8 and lq_quant8_blocks against the definition in float64: values and
exponents exact (the scale is a power of two and the rounding is one step)."""
import pytest
import torch

from bit_lifted_gemv_amd import lq

pytestmark = pytest.mark.gpu

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TOP = {E4M3: 448.0, E5M2: 57344.0}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"


def exponent(largest, dtype):
    """127 + the smallest e >= -127 with largest <= top 2^e, 127 for zeros; float64 on the CPU."""
    part, e = torch.frexp(largest / TOP[dtype])          # part 2^e, part in [1/2, 1): exact but for the division
    e = torch.where(part == 0.5, e - 1, e)
    up = torch.ldexp(torch.full_like(largest, TOP[dtype]), e) < largest
    e = torch.where(up, e + 1, e)
    return torch.where(largest > 0, e.clamp(min=-127) + 127, torch.full_like(e, 127))


def rounded(y, dtype):
    """float64 to the nearest value of the type, ties to even; infinities to NaN where it has none."""
    bits, low = (3, -6) if dtype == E4M3 else (2, -14)
    _, e = torch.frexp(y)
    unit = torch.ldexp(torch.ones_like(y), (e - 1).clamp(min=low) - bits)
    r = torch.round(y / unit) * unit
    r = torch.where(torch.isfinite(y), r, y)
    return torch.where(torch.isinf(y), torch.full_like(y, float("nan")), r) if dtype == E4M3 else r


def finite_abs(x):
    return torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x))


def plain_rows(x, dtype):
    x = torch.nn.functional.pad(x.double().cpu(), (0, -x.shape[1] % 128))
    g = x.unflatten(1, (-1, 128))
    e = exponent(finite_abs(g).amax(-1), dtype)
    return rounded(torch.ldexp(g, (127 - e).unsqueeze(-1)), dtype).flatten(1), e


def same(q, exps, want, e):
    got = q.float().double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(nan=0.0), want.nan_to_num(nan=0.0))
    assert torch.equal(exps.cpu().long(), e.long())


def inputs(rows, K, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, K, generator=g) * torch.exp(3 * torch.randn(rows, 1, generator=g))
    return (x * torch.where(torch.rand(K, generator=g) < 0.02, 30.0, 1.0)).to(dtype)


@pytest.mark.parametrize("to", [E4M3, E5M2])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 127), (2, 128), (3, 129), (1, 4096), (5, 511), (7, 513),
                                    (33, 1000), (257, 640), (1000, 136)])
def test_rows(rows, K, dtype, to):
    x = inputs(rows, K, dtype, rows * 1000 + K)
    q = lq.quantize8(x.cuda(), to)
    assert q.values.shape == (rows, (K + 127) // 128 * 128) and q.exps.shape == (rows, (K + 127) // 128)
    same(q.values, q.exps, *plain_rows(x, to))


@pytest.mark.parametrize("to", [E4M3, E5M2])
def test_edges_of_the_scale(to):
    """Largest values at, below and above top 2^e; zeros; subnormal and huge ones; ties."""
    top = TOP[to]
    rows = [[top], [top * (1 + 2**-20)], [top * (1 - 2**-20)], [2 * top], [0.0], [2.0**-149], [2.0**-126],
            [2.0**-130, 2.0**-149], [3.4e38], [2.0**127, 1.0], [1.0, -1.0], [1.75, 1.8125, 1.6875, 0.1],
            [448.0, 18.0, 20.0, 22.0, 26.0, -17.0, 2.0**-9, 2.0**-10, 3 * 2.0**-10], [1e-45, 3e-45]]
    x = torch.zeros(len(rows), 200)
    for i, r in enumerate(rows):
        x[i, 3:3 + len(r)] = torch.tensor(r)
        x[i, 150:150 + len(r)] = -torch.tensor(r) / 3
    q = lq.quantize8(x.cuda(), to)
    same(q.values, q.exps, *plain_rows(x, to))


@pytest.mark.parametrize("to", [E4M3, E5M2])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_infinities_and_nan_leave_the_other_values_alone(dtype, to):
    x = inputs(6, 300, dtype, 5)
    x[0, 7], x[1, 140], x[2, 3], x[2, 5] = float("inf"), float("nan"), float("-inf"), float("nan")
    x[3] = float("nan")
    x[4, :128] = float("inf")
    q = lq.quantize8(x.cuda(), to)
    same(q.values, q.exps, *plain_rows(x, to))
    if to == E5M2:
        assert q.values.float()[0, 7].item() == float("inf") and q.values.float()[2, 3].item() == float("-inf")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shift,pitch", [(0, 1), (1, 0), (3, 8), (8, 8), (2, 7)])
def test_rows_apart_and_not_aligned(dtype, shift, pitch):
    K = 391
    held = inputs(1, shift + 9 * (K + pitch), dtype, 9).flatten().cuda()
    x = held[shift:].as_strided((9, K), (K + pitch, 1), shift)
    q = lq.quantize8(x)
    same(q.values, q.exps, *plain_rows(x.cpu(), E4M3))


def test_rows_of_a_wide_buffer_are_left_alone():
    """Through the C call: pitches wider than needed, bytes between the rows stay."""
    x = inputs(5, 200, F16, 1).cuda()
    values = torch.full((5, 320), 0x55, dtype=torch.uint8, device="cuda")
    exps = torch.full((5, 12), 0x66, dtype=torch.uint8, device="cuda")
    lq.check(lq.lib().lq_quant8(x.data_ptr(), lq.LQ_F16, 5, 200, 200, values.data_ptr(), lq.LQ_E4M3, 320,
                                exps.data_ptr(), 12, None))
    torch.cuda.synchronize()
    want, e = plain_rows(x.cpu(), E4M3)
    same(values[:, :256].contiguous().view(E4M3), exps[:, :2], want, e)
    assert (values[:, 256:] == 0x55).all() and (exps[:, 4:] == 0x66).all()


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("E,m,K", [(0, 1, 1), (0, 128, 128), (0, 129, 127), (3, 200, 300), (2, 5, 700), (1, 384, 257)])
def test_blocks(E, m, K, dtype):
    g = torch.Generator().manual_seed(m + K)
    w = (torch.randn(E or 1, m, K, generator=g) * torch.exp(2 * torch.randn(E or 1, m, 1, generator=g))).to(dtype)
    q = lq.quantize8_blocks(w.cuda() if E else w[0].cuda())
    values = q.values if E else q.values[None]
    scales = q.scales if E else q.scales[None]
    for i in range(E or 1):
        x = torch.nn.functional.pad(w[i].double(), (0, -K % 128, 0, -m % 128))
        b = x.unflatten(1, (-1, 128)).unflatten(0, (-1, 128))
        e = exponent(b.abs().amax(-1).amax(1), E4M3)
        want = rounded(torch.ldexp(b, (127 - e)[:, None, :, None]), E4M3).flatten(2).flatten(0, 1)[:m]
        same(values[i], scales[i], want, e)


def test_no_rows():
    q = lq.quantize8(torch.empty(0, 130, device="cuda"))
    assert q.values.shape == (0, 256) and q.exps.shape == (0, 2)


def test_captured_and_on_another_stream():
    x = inputs(40, 1000, BF16, 3).cuda()
    want = lq.quantize8(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = lq.quantize8(x, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got.values.view(torch.uint8), want.values.view(torch.uint8)) and torch.equal(got.exps, want.exps)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = lq.quantize8(x)
    for seed in (11, 12, 13):
        x.copy_(inputs(40, 1000, BF16, seed))
        graph.replay()
        again = lq.quantize8(x)
        torch.cuda.synchronize()
        assert torch.equal(captured.values.view(torch.uint8), again.values.view(torch.uint8))
        assert torch.equal(captured.exps, again.exps)


@pytest.mark.parametrize("to", [torch.float8_e4m3fn, torch.float8_e5m2])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_every_16_bit_value_as_from_float32(dtype, to):
    """All 65536 of them, in order (blocks of one binade) and mixed (blocks of the widest range), in few rows and many."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    mixed = bits[torch.randperm(65536, generator=torch.Generator().manual_seed(1))]
    x = torch.stack([bits, mixed]).view(dtype).reshape(1024, 128).cuda()
    for a in (x, x.reshape(32, 4096).repeat(200, 1)):
        got, want = lq.quantize8(a, to), lq.quantize8(a.float(), to)
        nan = torch.isnan(want.values.float())
        assert torch.equal(got.exps, want.exps) and torch.equal(torch.isnan(got.values.float()), nan)
        assert torch.equal(got.values.view(torch.uint8)[~nan], want.values.view(torch.uint8)[~nan])
