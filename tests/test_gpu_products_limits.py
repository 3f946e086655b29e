"""lq_gemm_ep, lq_gemm_grouped and lq_gemm_join at the ends of their sizes, against float64.  Values
are whole numbers in [-8, 8], K is small and s is 1, so every sum is exact in float32 and a result is
the exact one, rounded once."""
import pytest
import torch

from bit_lifted_gemv_amd import lq

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def words(gen, *shape):
    *lead, K = shape
    return torch.randint(-2**31, 2**31, (*lead, ((K + 31) // 32 + 3) // 4 * 4), generator=gen).to(torch.int32).cuda()


def signs(w, K):
    bit = (w.long().unsqueeze(-1) >> torch.arange(32, device=w.device)) & 1
    return 2.0 * bit.flatten(-2)[..., :K].double() - 1.0


def whole(gen, rows, K, dtype):
    return torch.randint(-8, 9, (rows, K), generator=gen).to(dtype).cuda()


@pytest.mark.parametrize("B,dtype", [(600, BF16), (600, F32), (25000, F16)])
def test_one_row_of_weights(B, dtype):
    gen = torch.Generator().manual_seed(B)
    K = 4096 if B < 1000 else 264
    w, s = words(gen, 1, K), torch.ones(1, device="cuda")
    a = whole(gen, B, K, BF16)
    z = a.double() @ signs(w, K).T
    assert torch.equal(lq.gemm_ep(w, s, a, out_dtype=dtype), z.to(dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_one_row_of_weights_per_expert(dtype):
    E, K, T, k = 4, 128, 100, 1
    gen = torch.Generator().manual_seed(9)
    w, s = words(gen, E, 1, K), torch.ones(E, 1, device="cuda")
    a = whole(gen, T, K, BF16)
    r = lq.route(torch.randn(T, E, generator=gen).cuda(), k)
    z = torch.stack([a.double() @ signs(w[e], K).T for e in range(E)])      # [E][T][1]
    pick = z[r.ids[:, 0].long(), torch.arange(T, device="cuda")]
    out = lq.gemm_grouped(w, s, a, r.offsets, rows=r.rows, out_dtype=dtype)
    assert torch.equal(out, pick[r.rows.long()].to(dtype))
    own = a[r.rows.long()].contiguous()
    out = lq.gemm_join(w, s, own, r.offsets, r.pos, r.weight, out_dtype=dtype)
    assert torch.equal(out, pick.to(dtype))                                  # k = 1: the weight is 1


def test_most_rows_of_experts():
    """R = 2^31 - 1 gathered rows: more workgroups than one launch takes, runs whose tiles' end lies
    past 2^31, and rows behind the last run, which stay."""
    R, E, K, T = 2**31 - 1, 3, 8, 16
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    gen = torch.Generator().manual_seed(12)
    w, s = words(gen, E, 1, K), torch.ones(E, 1, device="cuda")
    a = whole(gen, T, K, BF16)
    rows = torch.randint(0, T, (R,), dtype=torch.int32, device="cuda")
    ends = [0, 5, 5, R - 2]
    off = torch.tensor(ends, dtype=torch.int32, device="cuda")
    out = torch.full((R, 1), 300.0, dtype=BF16, device="cuda")
    lq.gemm_grouped(w, s, a, off, rows=rows, out=out)
    z = [(a.double() @ signs(w[e], K).T)[:, 0].to(BF16) for e in range(E)]
    for e in range(E):
        for lo in range(ends[e], ends[e + 1], 1 << 28):
            hi = min(lo + (1 << 28), ends[e + 1])
            assert torch.equal(out[lo:hi, 0], z[e][rows[lo:hi]]), (e, lo)
    assert (out[R - 2:] == 300).all()
    off[3] = R                                               # the last run's end is R itself
    lq.gemm_grouped(w, s, a, off, rows=rows, out=out)
    assert torch.equal(out[-1000:, 0], z[2][rows[-1000:]])
    del out, rows
    torch.cuda.empty_cache()


@pytest.mark.parametrize("m,K,B", [(8, 128, 65535 * 16 + 1), (8, 128, 1100000), (1, 512, 2 * 65535 * 16 + 5)])
def test_more_token_tiles_than_a_grid_is_deep(m, K, B):
    """So few signs that the kernel for few rows takes any number of tokens, 16 a tile."""
    gen = torch.Generator().manual_seed(B)
    w, s = words(gen, m, K), torch.ones(m, device="cuda")
    a = torch.randint(-8, 9, (B, K), dtype=torch.int8, device="cuda").to(BF16)
    out = lq.gemm_ep(w, s, a)
    for lo in range(0, B, 1 << 19):
        z = a[lo:lo + (1 << 19)].double() @ signs(w, K).T
        assert torch.equal(out[lo:lo + (1 << 19)], z.to(BF16)), lo
