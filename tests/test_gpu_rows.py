"""lq_sort_rows, lq_join_rows and lq_join_rows_grad against float64.

Tolerances.  The sort moves values: exact.  A join of k terms in float32: each
product rounds once and each of the k additions and the residual's once, so
(k + 2) 2^-24 of the sum of magnitudes, plus the output's own half step.  A
dot product of n terms in any order of additions: every term passes at most n + 1
roundings of 2^-24, bounded by (n / 64 + 40) 2^-24 of the sum of magnitudes for the
order used (a thread adds n / 256 + 8 of them, then 6 + 2 steps across threads);
dz: one product, one rounding of the type.
"""
import pytest
import torch

from bit_lifted_gemv_amd import lq

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def routing(T, E, k, seed, padded=0.2):
    g = torch.Generator().manual_seed(seed)
    valid = (torch.rand(T, generator=g) >= padded).to(torch.uint8)
    return lq.route(torch.randn(T, E, generator=g).cuda(), k, valid=valid.cuda())


def values(rows, n, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(rows, n, generator=g).to(dtype).cuda()


def plain_sort(x, rows):
    out = torch.zeros(rows.shape[0], x.shape[1], dtype=x.dtype)
    for r, t in enumerate(rows.tolist()):
        if 0 <= t < x.shape[0]:
            out[r] = x[t]
    return out


SIZES = [(1, 4, 1, 1), (1, 8, 8, 64), (3, 5, 2, 127), (24, 64, 8, 2048), (65, 16, 4, 1001), (300, 7, 3, 520),
         (130, 256, 10, 40), (64, 64, 32, 96), (17, 9, 9, 4100)]


@pytest.mark.parametrize("dtype", [F32, F16, BF16, E4M3, torch.uint8])
@pytest.mark.parametrize("T,E,k,n", SIZES)
def test_sort(T, E, k, n, dtype):
    r = routing(T, E, k, T + n)
    x = (values(T, n, F32, n) * 8).to(dtype) if dtype != torch.uint8 else torch.randint(0, 256, (T, n), dtype=torch.uint8, device="cuda")
    got = lq.sort_rows(x, r.rows)
    bytes_ = (lambda t: t.cpu().contiguous().view(torch.uint8))
    assert torch.equal(bytes_(got), plain_sort(bytes_(x).view(T, -1), r.rows))


def test_offsets_past_32_bits():
    """Rows whose bytes lie past 2^32, and columns wider than a workgroup's pass."""
    n, R = 2**21 + 3, 1100
    x = torch.zeros(2, n, dtype=torch.uint8, device="cuda")
    x[0], x[1] = 3, 5
    rows = torch.zeros(R, dtype=torch.int32, device="cuda")
    rows[-1] = 1
    out = lq.sort_rows(x, rows, out=torch.empty(R, 2**22, dtype=torch.uint8, device="cuda")[:, :n])
    assert (out[-1] == 5).all() and (out[-2] == 3).all() and (out[0] == 3).all()
    z = torch.empty(R, 2**21, dtype=F16, device="cuda")
    z[-1], z[0] = 2.0, 1.0
    pos = torch.tensor([[R - 1, 0]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, 3.0]], device="cuda")
    assert (lq.join_rows(z, pos, w) == 4.0).all()
    dz, dw = lq.join_rows_grad(torch.ones(1, 2**21, dtype=F16, device="cuda"), z, pos, w)
    assert (dz[-1] == 0.5).all() and (dz[0] == 3.0).all() and dw.tolist() == [[2.0**22, 2.0**21]]


def test_sort_of_indices_out_of_range_and_repeated():
    x = values(5, 70, BF16, 1)
    rows = torch.tensor([4, -1, 5, 4, 2**31 - 1, -2**31, 0, 4], dtype=torch.int32)
    assert torch.equal(lq.sort_rows(x, rows.cuda()).cpu(), plain_sort(x.cpu(), rows))


@pytest.mark.parametrize("shift,pitch,n", [(0, 3, 64), (1, 0, 64), (1, 1, 33), (8, 8, 64), (4, 4, 36)])
def test_sort_and_join_of_rows_apart(shift, pitch, n):
    T, k = 20, 4
    r = routing(T, 8, k, 3)
    held = values(1, shift + T * (n + pitch), F16, 2).flatten()
    x = held[shift:].as_strided((T, n), (n + pitch, 1), shift)
    room = torch.full((T * k * (n + pitch) + shift,), 7.0, dtype=F16, device="cuda")
    out = room.as_strided((T * k, n), (n + pitch, 1), shift)
    assert lq.sort_rows(x, r.rows, out=out) is out
    assert torch.equal(out.cpu(), plain_sort(x.cpu(), r.rows.cpu()))
    if pitch:
        assert (room[shift:].view(T * k, n + pitch)[:, n:] == 7.0).all()
    y = lq.join_rows(out, r.pos, r.weight, residual=x)
    check_join(y, out, r.pos, r.weight, x)


def test_sort_of_quantized_rows():
    r = routing(30, 8, 2, 4)
    q = lq.quantize8(values(30, 700, BF16, 5))
    s = lq.sort_rows(q, r.rows)
    t = lq.quantize8(lq.sort_rows(values(30, 700, BF16, 5), r.rows))
    live = (r.rows >= 0).cpu()
    assert torch.equal(s.values.view(torch.uint8), t.values.view(torch.uint8))
    assert torch.equal(s.exps.cpu()[live], t.exps.cpu()[live])


def check_join(got, z, pos, weight, residual):
    zz = torch.cat([z.double().cpu(), torch.zeros(1, z.shape[1], dtype=torch.float64)])
    p = pos.cpu().long()
    p = torch.where((p >= 0) & (p < z.shape[0]), p, torch.full_like(p, z.shape[0]))
    w = torch.ones_like(p, dtype=torch.float64) if weight is None else weight.double().cpu()
    terms = zz[p] * w.unsqueeze(-1)
    add = torch.zeros(()) if residual is None else residual.double().cpu()
    want, size = terms.sum(1) + add, terms.abs().sum(1) + add.abs()
    off = (got.double().cpu() - want).abs()
    assert (off <= (p.shape[1] + 2) * 2.0**-24 * size + half_step(got.dtype) * want.abs() * (1 + 2.0**-10)
            + torch.finfo(got.dtype).smallest_normal * torch.finfo(got.dtype).eps).all(), off.max()


@pytest.mark.parametrize("dtype,out", [(F32, F32), (F16, F16), (BF16, BF16), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("T,E,k,n", SIZES)
def test_join(T, E, k, n, dtype, out):
    r = routing(T, E, k, T + n)
    z = values(T * k, n, dtype, n)
    res = values(T, n, out, n + 1)
    check_join(lq.join_rows(z, r.pos, r.weight, out_dtype=out), z, r.pos, r.weight, None)
    check_join(lq.join_rows(z, r.pos, None, residual=res, out_dtype=out), z, r.pos, None, res)
    got = res.clone()
    assert lq.join_rows(z, r.pos, r.weight, residual=got, out=got) is got
    check_join(got, z, r.pos, r.weight, res)


def test_join_of_positions_out_of_range():
    """Rows that nobody names may hold anything."""
    z = values(6, 50, BF16, 1)
    z[3] = float("nan")
    pos = torch.tensor([[0, 6], [-1, -1], [2**31 - 1, 5], [-2**31, 1]], dtype=torch.int32, device="cuda")
    w = torch.rand(4, 2, device="cuda")
    got = lq.join_rows(z, pos, w)
    assert (got[1] == 0).all()
    check_join(got, torch.where(torch.isnan(z), torch.zeros_like(z), z), pos, w, None)


def check_grad(dy, z, pos, weight, rows, dz, dweight):
    R, n = z.shape
    g, zz, p = dy.double().cpu(), z.double().cpu(), pos.cpu().long()
    want, named = torch.zeros(R, n, dtype=torch.float64), torch.zeros(R, dtype=torch.bool)
    for t in range(p.shape[0]):
        for j in range(p.shape[1]):
            r = p[t, j].item()
            if 0 <= r < R:
                want[r] = weight[t, j].double().item() * g[t]
                named[r] = True
                products = g[t] * zz[r]
                off = abs(dweight[t, j].item() - products.sum().item())
                assert off <= (n / 64 + 40) * 2.0**-24 * products.abs().sum().item(), (t, j, off)
            else:
                assert dweight[t, j].item() == 0.0
    off = (dz.double().cpu() - want).abs()
    named |= torch.tensor([rows is not None and not 0 <= t < p.shape[0] for t in (rows.tolist() if rows is not None else [0] * R)])
    assert named.all() or rows is None
    off = off[named]
    bound = (half_step(z.dtype) + 2.0**-24) * want[named].abs() * (1 + 2.0**-10)
    assert (off <= bound + torch.finfo(z.dtype).smallest_normal * torch.finfo(z.dtype).eps).all()


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("T,E,k,n", SIZES)
def test_grad(T, E, k, n, dtype):
    r = routing(T, E, k, T + n)
    z, dy = values(T * k, n, dtype, n), values(T, n, dtype, n + 7)
    dz, dweight = lq.join_rows_grad(dy, z, r.pos, r.weight, r.rows)
    weight, pos, rows = r.weight.cpu(), r.pos, r.rows.cpu()
    check_grad(dy, z, pos, weight, rows, dz, dweight.cpu())


def test_grad_leaves_rows_alone_without_rows():
    """Through the C call: rows that no pair names stay, between the rows too."""
    z, dy = values(8, 40, F32, 1), values(2, 40, F32, 2)
    pos = torch.tensor([[1, 6], [-1, 3]], dtype=torch.int32, device="cuda")
    w = torch.rand(2, 2, device="cuda")
    dz = torch.full((8, 44), 9.0, device="cuda")
    dw = torch.empty(2, 2, device="cuda")
    lq.check(lq.lib().lq_join_rows_grad(dy.data_ptr(), lq.LQ_F32, 40, z.data_ptr(), 40, 8, 40, pos.data_ptr(),
                                        w.data_ptr(), 2, 2, None, dz.data_ptr(), 44, dw.data_ptr(), None))
    torch.cuda.synchronize()
    assert (dz[:, 40:] == 9.0).all() and (dz[[0, 2, 4, 5, 7]] == 9.0).all()
    check_grad(dy, z, pos, w.cpu(), None, dz[:, :40], dw.cpu())


def test_grad_against_differences():
    """L = sum(c . join(z)): dL/dz and dL/dweight by central differences in float64, which for a bilinear
    function are exact but for the values' rounding; the sort's gradient is the plain join."""
    T, E, k, n = 6, 5, 2, 24
    r = routing(T, E, k, 3, padded=0.0)
    z, c = values(T * k, n, F32, 1), values(T, n, F32, 2)
    dz, dw = lq.join_rows_grad(c, z, r.pos, r.weight, r.rows)
    p, zz, cc, w = r.pos.cpu().long(), z.double().cpu(), c.double().cpu(), r.weight.double().cpu()
    loss = lambda z_, w_: (cc * (z_[p] * w_.unsqueeze(-1)).sum(1)).sum()  # noqa: E731
    for row, col in [(0, 0), (5, 11), (T * k - 1, n - 1)]:
        step = torch.zeros_like(zz)
        step[row, col] = 0.5
        assert abs((loss(zz + step, w) - loss(zz - step, w)).item() - dz[row, col].item()) < 1e-6
    for t, j in [(0, 0), (3, 1), (5, 0)]:
        step = torch.zeros_like(w)
        step[t, j] = 0.5
        assert abs((loss(zz, w + step) - loss(zz, w - step)).item() - dw[t, j].item()) < 1e-5
    x, dxs = values(T, n, F32, 4), values(T * k, n, F32, 5)
    dx = lq.join_rows(dxs, r.pos)
    sorted_loss = lambda x_: (dxs.double().cpu() * x_[r.rows.cpu().long()]).sum()  # noqa: E731
    for t, col in [(0, 0), (4, 9)]:
        step = torch.zeros(T, n, dtype=torch.float64)
        step[t, col] = 0.5
        xx = x.double().cpu()
        assert abs((sorted_loss(xx + step) - sorted_loss(xx - step)).item() - dx[t, col].item()) < 1e-5


def test_no_tokens_and_all_padding():
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    x = values(4, 16, BF16, 1)
    assert lq.sort_rows(x, none).shape == (0, 16)
    assert (lq.sort_rows(torch.empty(0, 16, dtype=BF16, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")) == 0).all()
    empty = torch.empty(0, 2, device="cuda")
    assert lq.join_rows(x, empty.int(), empty).shape == (0, 16)
    pos = torch.full((4, 2), -1, dtype=torch.int32, device="cuda")
    rows = torch.full((8,), -1, dtype=torch.int32, device="cuda")
    assert torch.equal(lq.join_rows(values(8, 16, BF16, 2), pos, pos.float(), residual=x), x)
    dz, dw = lq.join_rows_grad(x, values(8, 16, BF16, 2), pos, pos.float(), rows)
    assert (dz == 0).all() and (dw == 0).all()
    dz, dw = lq.join_rows_grad(x[:0], values(8, 16, BF16, 2), empty.int(), empty, rows)
    assert (dz == 0).all() and dw.shape == (0, 2)


def test_captured_and_replayed():
    T, E, k, n = 50, 8, 4, 320
    r = routing(T, E, k, 8)
    x, res, dy = values(T, n, BF16, 1), values(T, n, BF16, 2), values(T, n, BF16, 3)
    run = lambda: (lambda s: (s, lq.join_rows(s, r.pos, r.weight, residual=res),  # noqa: E731
                              *lq.join_rows_grad(dy, s, r.pos, r.weight, r.rows)))(lq.sort_rows(x, r.rows))
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run()
    for seed in (21, 22, 23):
        x.copy_(values(T, n, BF16, seed))
        dy.copy_(values(T, n, BF16, seed + 9))
        graph.replay()
        eager = run()
        torch.cuda.synchronize()
        for a, b in zip(captured, eager):
            assert torch.equal(a, b)
