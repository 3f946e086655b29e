"""How many bits lq_gemm_ep, lq_gemm_grouped and lq_gemm_join keep.

float16 results keep an activation to 2^-19 of the largest one of its 32
positions: behind three float6 parts the remainder is at most 1/16 of a unit of
the third part's scale (2^-12 where the largest value is scaled into [4, 8)),
so 2^14 times it lies below 4, where float6 has steps of at most 1/4, and half
of one is 2^-17, 2^-19 of a largest value of 4.  float32 results keep 2^-24 of it (the
fourth part leaves 1/8 of a unit at 2^-14, 32 times which lies at 4: half a step
of 1/4 at 2^-19 is 2^-22, 2^-24 of 4).
"""
import math

import pytest
import torch

from bit_lifted_gemv_amd import lq

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    lq.load_library()
    return torch.device("cuda:0")


def words(gen, *shape):
    *lead, K = shape
    ldw = ((K + 31) // 32 + 3) // 4 * 4
    return torch.randint(-2**31, 2**31, (*lead, ldw), generator=gen).to(torch.int32)


def signs(w, K):
    bit = (w.long().unsqueeze(-1) >> torch.arange(32, device=w.device)) & 1
    return 2.0 * bit.flatten(-2)[..., :K].double() - 1.0


def beside_large(gen, rows, K, large):
    """float16 values of 11 bits below 1, and one `large` in every block of 32."""
    a = torch.randint(1024, 2048, (rows, K), generator=gen).double() * 2.0**-11
    a *= 2 * torch.randint(0, 2, (rows, K), generator=gen) - 1
    for b in range(0, K, 32):
        a[torch.arange(rows), b + torch.randint(0, min(32, K - b), (rows,), generator=gen)] = large
    return a


def within(out, z, part):
    """Half a step of float16 (2^-25 for its smallest numbers), the parts, and
    float32 sums: 2^-24 of a partial sum below 2^13, six of them at most."""
    off = (out.cpu().double() - z).abs()
    tol = z.abs() * 2.0**-11 + 2.0**-25 + part + 6 * 2.0**-24 * 2.0**13
    assert (off <= tol).all(), (float(off.max()), float((off / tol).max()))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("m,B", [(512, 1), (300, 5), (256, 16), (200, 40), (1024, 200), (8192, 300), (32768, 600)])
def test_float16_result_keeps_small_values_beside_large_ones(dev, m, B, dtype):
    """Where the two large values of a row cancel, the small ones are the result."""
    K, large = 64, 2048.0
    gen = torch.Generator().manual_seed(m + B)
    w = words(gen, m, K)
    a = beside_large(gen, B, K, large).to(dtype)
    z = a.double() @ signs(w, K).T
    out = lq.gemm_ep(w.to(dev), torch.ones(m, device=dev), a.to(dev), out_dtype=F16)
    within(out, z, K * 2.0**-19 * large)


@pytest.mark.parametrize("T", [2, 40, 400])
def test_float16_expert_results_keep_small_values_beside_large_ones(dev, T):
    E, k, m, K, large = 4, 2, 512, 64, 2048.0
    gen = torch.Generator().manual_seed(T)
    w = words(gen, E, m, K)
    s = torch.ones(E, m, device=dev)
    r = lq.route(torch.randn(T, E, generator=gen).to(dev), k)
    off, rows = r.offsets.tolist(), r.rows.long().cpu()
    a = beside_large(gen, T, K, large)
    out = lq.gemm_grouped(w.to(dev), s, a.to(F16).to(dev), r.offsets, rows=r.rows)
    z = torch.cat([a[rows[off[e]:off[e + 1]]] @ signs(w[e], K).T for e in range(E)])
    within(out, z, K * 2.0**-19 * large)
    own = a[rows]
    one = torch.where(torch.arange(k) == 0, 1.0, 0.0).expand(T, k).contiguous().to(dev)
    out = lq.gemm_join(w.to(dev), s, own.to(F16).to(dev), r.offsets, r.pos, one)
    within(out, z[r.pos[:, 0].long().cpu()], K * 2.0**-19 * large)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("B", [3, 16, 300])
def test_float16_results_with_outliers_round_like_the_exact_ones(dev, B, gated):
    """One position in a hundred twenty times the others.  A block's largest value is below
    20 x 5 standard deviations of the others, so a value is off by at most 2^-19 x 100, and uniform,
    by 2^-19 x 100 / sqrt 3 = 1.1e-4 of that deviation in the mean; at most 0.3 of the blocks hold such
    a position, and the root mean square of all values is above 2 deviations: 1.1e-4 sqrt(0.3) / 2 =
    3.0e-5 of the result.  A gate multiplies two of these, one through a slope below 1.13: below
    5e-5.  Rounding the exact result to float16 leaves 2e-4 of it."""
    m, K = 2048, 8192
    gen = torch.Generator().manual_seed(B)
    w = words(gen, m, K).to(dev)
    s = (torch.rand(m, generator=gen) * 0.02 + 0.01).to(dev)
    a = torch.randn(B, K, generator=gen) * torch.where(torch.rand(K, generator=gen) < 0.01, 20.0, 1.0)
    a = a.to(F16).to(dev)
    z = a.double() @ signs(w, K).T * s.double()
    y = z[:, :m // 2] * torch.special.expit(z[:, :m // 2]) * z[:, m // 2:] if gated else z
    out = lq.gemm_ep(w, s, a, act="silu" if gated else "none", gated=gated)
    rms = lambda x: math.sqrt(float((x * x).mean()))  # noqa: E731
    best = rms(y.to(F16).double() - y)
    bound = math.sqrt(best**2 + ((5e-5 if gated else 3e-5) * rms(y))**2)
    assert rms(out.double() - y) <= bound


def sparse_beside_large(gen, rows, K):
    """float16 values of 11 bits below 1 in 2000 positions at most, and 2048 in one: all are multiples
    of 2^-11, and any partial sum lies below 2000 + 2048 < 2^12, so float32 sums are exact."""
    a = torch.randint(1024, 2048, (rows, K), generator=gen).double() * 2.0**-11
    a *= 2 * torch.randint(0, 2, (rows, K), generator=gen) - 1
    if K > 2000:
        a *= torch.zeros(K, dtype=torch.float64).index_fill_(0, torch.randperm(K, generator=gen)[:2000], 1.0)
    a[torch.arange(rows), torch.randint(0, K, (rows,), generator=gen)] = 2048.0
    return a


@pytest.mark.parametrize("m,K,B", [(64, 65536, 1), (512, 16384, 5), (4096, 16384, 16), (300, 32768, 40), (1281, 5128, 777)])
def test_float32_result_is_exact_over_slices(dev, m, K, B):
    gen = torch.Generator().manual_seed(m + K + B)
    w, a = words(gen, m, K), sparse_beside_large(gen, B, K)
    z = a.to(dev) @ signs(w.to(dev), K).T
    out = lq.gemm_ep(w.to(dev), torch.ones(m, device=dev), a.to(F16).to(dev), out_dtype=F32)
    assert torch.equal(out.double(), z)


@pytest.mark.parametrize("E,m,K,T", [(4, 256, 1024, 2), (8, 500, 1024, 300), (2, 320, 32768, 20), (3, 64, 65536, 4)])
def test_float32_expert_results_are_exact(dev, E, m, K, T):
    """Into the experts, and out of them with weights of 1: sums of two rows, below 2^13."""
    k = 2
    gen = torch.Generator().manual_seed(E + m + K + T)
    w, s = words(gen, E, m, K).to(dev), torch.ones(E, m, device=dev)
    r = lq.route(torch.randn(T, E, generator=gen).to(dev), k)
    off, rows = r.offsets.tolist(), r.rows.long()
    a = sparse_beside_large(gen, T, K).to(dev)
    z = torch.cat([a[rows[off[e]:off[e + 1]]] @ signs(w[e], K).T for e in range(E)])
    assert torch.equal(lq.gemm_grouped(w, s, a.to(F16), r.offsets, rows=r.rows, out_dtype=F32).double(), z)
    out = lq.gemm_join(w, s, a[rows].to(F16).contiguous(), r.offsets, r.pos, torch.ones(T, k, device=dev), out_dtype=F32)
    assert torch.equal(out.double(), z[r.pos.long()].sum(1))


# Each tile of the many-row kernel with four parts
@pytest.mark.parametrize("m,K,B", [
    (28672, 264, 1024),                    # 256 x 64 in two workgroups of four waves: 896 tiles of 512 rows
    (28672, 256, 1170),                    # 512 x 64 in eight waves, 19 columns of token tiles
    (8190, 512, 500),                      # 256 x 64 in eight waves
    (262200, 256, 17), (38402, 1024, 60), (28672, 1032, 57), (4100, 8200, 40),
])
@pytest.mark.parametrize("gated", [False, True])
def test_float16_results_of_each_tile(dev, m, K, B, gated):
    """Whole numbers up to 8: sums below 2^17 are exact, and so is the result, rounded once."""
    gen = torch.Generator().manual_seed(m + K + B)
    w, s = words(gen, m, K).to(dev), torch.full((m,), 2.0**-4, device=dev)
    a = torch.randint(-8, 9, (B, K), generator=gen).to(F16).to(dev)
    pick = torch.randperm(m // 2, generator=gen)[:1000].to(dev)
    at = torch.cat([pick, pick + m // 2])
    z = a.double() @ signs(w[at], K).T * 2.0**-4
    out = lq.gemm_ep(w, s, a, act="relu", gated=gated)
    y = torch.relu(z[:, :len(pick)]) * z[:, len(pick):] if gated else torch.relu(z[:, :len(pick)])
    # a gate's product of two exact numbers is rounded to float32 first
    assert torch.equal(out[:, pick], y.float().to(F16))


@pytest.mark.parametrize("E,m,K,T,k", [(64, 1408, 512, 2000, 8), (8, 4096, 8456, 700, 2), (16, 2048, 264, 1500, 4)])
def test_float16_expert_results_of_the_large_tiles(dev, E, m, K, T, k):
    gen = torch.Generator().manual_seed(E + m + K)
    w, s = words(gen, E, m, K).to(dev), torch.full((E, m), 2.0**-4, device=dev)
    r = lq.route(torch.randn(T, E, generator=gen).to(dev), k)
    off, rows = r.offsets.tolist(), r.rows.long()
    a = torch.randint(-8, 9, (T, K), generator=gen).to(F16).to(dev)
    out = lq.gemm_grouped(w, s, a, r.offsets, rows=r.rows)
    z = torch.cat([a[rows[off[e]:off[e + 1]]].double() @ signs(w[e], K).T for e in range(E)]) * 2.0**-4
    assert torch.equal(out, z.to(F16))
