"""Where the many-row 8-bit product writes: outputs whose rows lie any number of values apart,
begin at any value and have any width, on the tiles of 256 rows, whose 16-bit outputs pass the
caches by in pieces of four.  The values are those of a dense output, what lies between the
rows stays, and a call that reads the output next finds all of it."""
import pytest
import torch

from bit_lifted_gemv_amd import lq

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"


def integers(*shape, seed):
    """Up to 7: products and sums are exact, so that every result is the exact one rounded once."""
    return torch.randint(-7, 8, shape, generator=torch.Generator().manual_seed(seed)).float().cuda()


def exact(w, a, gated):
    z = (a.double() @ w.double().T).float()
    half = w.shape[0] // 2
    return torch.relu(z[:, :half]) * z[:, half:] if gated else torch.relu(z)


# 128 x 256 tiles and 256 x 256 ones; widths that leave one, two and three values over
@pytest.mark.parametrize("out", [F16, BF16, F32])
@pytest.mark.parametrize("first,behind", [(0, 1), (1, 0), (3, 2), (2, 5), (8, 8)])
@pytest.mark.parametrize("m,B", [(4093, 2000), (4095, 2048), (4094, 4001), (4090, 4000)])
def test_rows_apart(m, B, first, behind, out):
    w, a = integers(m, 384, seed=1), integers(B, 384, seed=2)
    w8, a8 = lq.quantize8_blocks(w), lq.quantize8(a)
    for gated in (False, True)[:1 + (m % 2 == 0)]:
        width = m // 2 if gated else m
        pitch = first + width + behind
        y = exact(w, a, gated)
        res = torch.randn(B, pitch + 1, device="cuda").to(out)[:, 1:1 + width]
        for residual in (None, res):
            held = torch.full((B, pitch), 7.0, dtype=out, device="cuda")
            view = held[:, first:first + width]
            assert lq.gemm8(w8, a8, gated=gated, act="relu", residual=residual, out=view) is view
            assert torch.equal(view, (y if residual is None else y + residual.float()).to(out))
            assert (held[:, :first] == 7.0).all() and (held[:, first + width:] == 7.0).all()
        # in place of the residual, the same pitch
        lq.gemm8(w8, a8, gated=gated, act="relu", residual=res, out=res)
        assert torch.equal(res, view)


@pytest.mark.parametrize("out", [F16, BF16])
@pytest.mark.parametrize("E,R,m", [(2, 4000, 8190), (16, 6000, 1278)])
def test_runs_apart(E, R, m, out):
    """Runs on 256 x 256 and 128 x 256 tiles, some empty, rows outside every run left as they were."""
    K = 256
    w, a = integers(E, m, K, seed=3), integers(500, K, seed=4)
    w8, a8 = lq.quantize8_blocks(w), lq.quantize8(a)
    g = torch.Generator().manual_seed(R)
    rows = torch.randint(-1, 501, (R,), generator=g)
    ends = torch.cat([torch.tensor([5, 5]), torch.randint(6, R - 8, (E - 1,), generator=g).sort().values])
    x = torch.where(((rows >= 0) & (rows < 500))[:, None].cuda(), a[rows.clamp(0, 499).cuda()], 0.0)
    for gated in (False, True):
        width = m // 2 if gated else m
        held = torch.full((R, width + 3), 7.0, dtype=out, device="cuda")
        lq.gemm8_grouped(w8, a8, ends.int().cuda(), rows=rows.int().cuda(), gated=gated, act="relu", out=held[:, 1:1 + width])
        want = torch.full_like(held, 7.0)
        for e in range(E):
            lo, hi = int(ends[e]), int(ends[e + 1])
            want[lo:hi, 1:1 + width] = exact(w[e], x[lo:hi], gated).to(out)
        assert torch.equal(held, want)


@pytest.mark.parametrize("m,B", [(4096, 2048), (8192, 4096)])
def test_the_next_call_reads_all_of_it(m, B):
    w, outs = lq.quantize8_blocks(integers(m, 384, seed=1)), []
    for seed in range(6):
        y = lq.gemm8(w, lq.quantize8(integers(B, 384, seed=seed + 2)), out_dtype=BF16)
        outs.append((y, lq.quantize8(y)))
    for y, q in outs:
        again = lq.quantize8(y.clone())
        assert torch.equal(q.exps, again.exps) and torch.equal(q.values.view(torch.uint8), again.values.view(torch.uint8))
