"""lq_gemm8 and lq_gemm8_grouped against the definition in float64.

Tolerances, fixed before the first run.  Products of 8-bit values are exact in
float32 and the powers of two too; a float32 sum of K products in any order is
given 2^-20 of the sum of magnitudes (K <= 8192 here: the matrix cores add 64 or
128 products at a time, so at most 2 K / 64 + 6 <= 262 additions follow one another, each off
by at most 2^-24 of the sum of magnitudes, and errors of this kind add like independent
ones, sqrt(262) = 16 = 2^4; a float32 scale rounds once a block).  So
  dz = 2^-20 sum_k |w_k| |a_k| + 2^-23 (|z| + |bias|)
bounds z; activations have slopes below 1.13 and are evaluated to 2^-20 of
|z| + 1; the output's own rounding adds eps / 2 of the value.

For 16-bit results the 8-bit matrix instructions add one more term, which the
first bound left out: they add the products of eight consecutive positions and
cut each off (toward zero) below 2^-13 of the largest one's power of two.  (Seen
with 2^16 - 2^16 + 2^s: 2^3 comes out whole, 2^2 as 0; 2^16 - 2^16 + 14.0625 as 8.)
Each of the eight loses less than one such unit, so a group is off by less than
8 2^-13 max |w_k a_k| <= 2^-10 max |w_k| max |a_k|: added over the groups.  Float32
results are computed with 16-bit instructions, which keep 24 bits, and are held to
the first bound.
"""
import math

import pytest
import torch

from bit_lifted_gemv_amd import lq

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"


def weights(m, K, kind, seed, E=0):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(E or 1, m, K, generator=g) * torch.exp(torch.randn(E or 1, m, 1, generator=g))
    q = lq.quantize8_blocks((w if E else w[0]).cuda())
    if kind == F32:       # any scale, of either sign
        s = torch.randn(q.scales.shape, generator=g).cuda()
        return lq.Blocks8(q.values, s * 0.37)
    return q


def activations(B, K, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    a = torch.randn(B, K, generator=g) * torch.where(torch.rand(K, generator=g) < 0.01, 20.0, 1.0)
    return lq.quantize8(a.cuda(), dtype) if dtype in (E4M3, E5M2) else a.to(dtype).cuda()


def matrix64(w):
    """[m][K in whole 128] of one matrix."""
    s = w.scales.double() if w.scales.dtype == F32 else torch.exp2(w.scales.double() - 127)
    m, K = w.values.shape
    return w.values.double() * s.repeat_interleave(128, 0)[:m].repeat_interleave(128, 1)


def rows64(a):
    if not isinstance(a, lq.Rows8):
        a = lq.quantize8(a)
    return a.values.double() * torch.exp2(a.exps.double() - 127).repeat_interleave(128, 1)


def act64(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "silu":
        return z * torch.special.expit(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return z * torch.special.expit(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z**3))
    return z


def largest8(x):
    """The largest magnitude of each eight positions."""
    return x.abs().unflatten(1, (-1, 8)).amax(2)


def product64(w, a, bias, act, gated, out_dtype):
    """Outputs before the residual, and the bound of their error."""
    W = matrix64(w)
    z = a @ W.T
    dz = 2.0**-20 * (a.abs() @ W.abs().T)
    if out_dtype != F32:
        dz = dz + 2.0**-10 * (largest8(a) @ largest8(W).T)
    if bias is not None:
        z = z + bias.double()
    dz = dz + 2.0**-23 * (z.abs() + (0.0 if bias is None else bias.double().abs()))
    m = W.shape[0]
    g, dg = (z[:, :m // 2], dz[:, :m // 2]) if gated else (z, dz)
    y = act64(g, act)
    dy = 1.13 * dg + (0.0 if act == "none" else 2.0**-20 * (g.abs() + 1.0))
    if gated:
        u, du = z[:, m // 2:], dz[:, m // 2:]
        dy = dy * (u.abs() + du) + y.abs() * du + 2.0**-23 * (y * u).abs()
        y = y * u
    return y, dy


def near(got, y, dy, residual=None):
    if residual is not None:
        y = y + residual.double()
        dy = dy + 2.0**-23 * y.abs()
    eps = torch.finfo(got.dtype).eps / 2
    off = (got.double() - y).abs()
    bound = dy + eps * (y.abs() + dy) + torch.finfo(got.dtype).smallest_normal * eps
    # past the type's largest value (float16: 65504) the nearest one is an infinity of that sign
    far = torch.isinf(got) & (y * got.sign() + bound > torch.finfo(got.dtype).max)
    off = torch.where(far, torch.zeros_like(off), off)
    assert (off <= bound).all(), ((off / bound).max().item(), off.max().item())


def check(w, a, bias=None, act="none", gated=False, residual=None, out_dtype=F32):
    got = lq.gemm8(w, a, bias=bias, act=act, gated=gated, residual=residual, out_dtype=out_dtype)
    y, dy = product64(w, rows64(a), bias, act, gated, out_dtype)
    near(got, y, dy, residual)
    return got


TYPES = [E4M3, E5M2, F16, BF16]


@pytest.mark.parametrize("kind", [torch.uint8, F32])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,K,B", [(1, 1, 1), (16, 128, 1), (33, 129, 2), (128, 1000, 3), (129, 127, 16), (200, 4096, 15),
                                   (1281, 640, 17), (64, 2049, 33), (300, 513, 64), (512, 256, 65), (257, 384, 130),
                                   (4096, 1024, 1), (1000, 8192, 5), (31, 8192, 1), (640, 896, 300), (1281, 1100, 777)])
def test_product(m, K, B, dtype, kind):
    check(weights(m, K, kind, m + K), activations(B, K, dtype, B + K))


@pytest.mark.parametrize("out", [F16, BF16, F32])
@pytest.mark.parametrize("act", sorted(lq.ACTS))
@pytest.mark.parametrize("m,K,B,dtype,kind", [(202, 300, 1, BF16, F32), (384, 1000, 20, E4M3, torch.uint8),
                                              (1000, 512, 270, E5M2, F32), (514, 700, 513, F16, torch.uint8)])
def test_epilogue(m, K, B, dtype, kind, act, out):
    g = torch.Generator().manual_seed(7)
    w, a = weights(m, K, kind, 1), activations(B, K, dtype, 2)
    w = w if kind == F32 else lq.Blocks8(w.values, (w.scales - 3))
    if kind != F32:
        held = torch.zeros(*w.scales.shape[:-1], w.scales.shape[-1] + -w.scales.shape[-1] % 4, dtype=torch.uint8, device="cuda")
        held[..., :w.scales.shape[-1]] = w.scales
        w = lq.Blocks8(w.values, held[..., :w.scales.shape[-1]])
    a = a if isinstance(a, lq.Rows8) else a / 8
    bias = torch.randn(m, generator=g).cuda()
    for gated in (False, True):
        width = m // 2 if gated else m
        residual = torch.randn(B, width, generator=g).to(out).cuda()
        check(w, a, bias, act, gated, residual, out)
        check(w, a, None, act, gated, None, out)


# one size at least for every tile that the products are computed on, with one and several slices of the positions
TILES = [(4096, 300, 4000), (4096, 300, 2048), (129, 200, 21760), (1000, 260, 2000), (130, 5000, 40), (2048, 700, 260), (31, 20000, 3)]


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("kind", [torch.uint8, F32])
@pytest.mark.parametrize("dtype", [E4M3, E5M2])
@pytest.mark.parametrize("m,K,B", TILES)
def test_every_tile(m, K, B, dtype, kind, out):
    g = torch.Generator().manual_seed(3)
    w, a = weights(m, K, kind, 1), activations(B, K, dtype, 2)
    bias, residual = torch.randn(m, generator=g).cuda(), torch.randn(B, m, generator=g).to(out).cuda()
    check(w, a, bias, "gelu", False, residual, out)
    if m % 2 == 0:
        w = lq.Blocks8(w.values, w.scales / 64) if kind == F32 else w
        check(w, a, bias, "relu", True, residual[:, :m // 2], out)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("B,K", [(1, 512), (3, 1000), (4, 2048), (1, 333), (20, 640), (200, 333)])
def test_the_identity_gives_the_quantized_values(B, K, dtype):
    """Weights of 1 on the diagonal: every output is one activation as it was quantized, bit for bit."""
    eye = lq.quantize8_blocks(torch.eye(K).cuda())
    g = torch.Generator().manual_seed(B + K)
    a = torch.randn(B, K, generator=g) * torch.exp(3 * torch.randn(B, (K + 127) // 128, generator=g)).repeat_interleave(128, 1)[:, :K]
    a[0, :128] *= 2.0**-14 if dtype == F16 else 2.0**-100
    a = a.to(dtype).cuda()
    want = rows64(lq.quantize8(a))[:, :K]
    assert torch.equal(lq.gemm8(eye, a, out_dtype=F32).double(), want)
    a[B - 1, 5] = float("inf")                                   # e4m3 has none: a NaN, and the block's scale is that of the others
    q = lq.quantize8(a)
    clean = torch.where(torch.isnan(q.values.float()), torch.zeros_like(q.values.float()), q.values.float()).to(E4M3)
    rest = torch.arange(B, device="cuda") != B - 1
    got = lq.gemm8(eye, a, out_dtype=F32)
    assert torch.isnan(got[B - 1]).all() and torch.equal(got[rest].double(), rows64(lq.Rows8(clean, q.exps))[rest, :K])


def routing(T, E, k, seed, skew=1.0, padded=0.0):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(T, E, generator=g) + torch.randn(E, generator=g) * skew
    valid = (torch.rand(T, generator=g) >= padded).to(torch.uint8)
    return lq.route(logits.cuda(), k, valid=valid.cuda())


def check_grouped(w, a, offsets, rows=None, bias=None, act="none", gated=False, out_dtype=F32):
    E, m, _ = w.values.shape
    a64 = rows64(a)
    R = a64.shape[0] if rows is None else rows.shape[0]
    width = m // 2 if gated else m
    out = torch.full((R, width), 123.0, dtype=out_dtype, device="cuda")
    assert lq.gemm8_grouped(w, a, offsets, rows=rows, bias=bias, act=act, gated=gated, out=out) is out
    source = torch.arange(R, device="cuda") if rows is None else rows.long()
    live = (source >= 0) & (source < a64.shape[0])
    x = torch.where(live[:, None], a64[source.clamp(0, a64.shape[0] - 1)], 0.0)
    ends = offsets.clamp(0, R).tolist()
    untouched = torch.ones(R, dtype=torch.bool, device="cuda")
    for e in range(E):
        lo, hi = ends[e], ends[e + 1]
        if hi > lo:
            one = lq.Blocks8(w.values[e], w.scales[e])
            near(out[lo:hi], *product64(one, x[lo:hi], None if bias is None else bias[e], act, gated, out_dtype))
            untouched[lo:hi] = False
    assert (out[untouched] == 123.0).all()
    return out


@pytest.mark.parametrize("kind", [torch.uint8, F32])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E,k,T,m,K,gated", [(4, 1, 1, 64, 128, False), (64, 8, 1, 96, 300, True), (8, 2, 24, 200, 1000, False),
                                             (64, 8, 40, 130, 257, True), (3, 2, 300, 384, 640, True), (130, 4, 500, 64, 200, False),
                                             (8, 2, 2000, 256, 512, True), (2, 1, 5, 1000, 4096, False),
                                             (70, 2, 900, 130, 300, True), (2, 1, 4000, 8192, 200, False),
                                             (16, 2, 3000, 640, 1100, True)])
def test_experts(E, k, T, m, K, gated, dtype, kind):
    r = routing(T, E, k, T + E, padded=0.1)
    w = weights(m, K, kind, E + m, E=E)
    bias = torch.randn(E, m, device="cuda")
    check_grouped(w, activations(T, K, dtype, T), r.offsets, r.rows, bias, "silu", gated, BF16)
    check_grouped(w, activations(T * k, K, dtype, T), r.offsets, None, None, "none", gated, F32)


def test_runs_that_are_empty_or_leave_rows():
    w = weights(70, 300, torch.uint8, 1, E=6)
    a = activations(90, 300, E4M3, 2)
    for ends in ([0, 0, 0, 0, 0, 0, 0], [0, 90, 90, 90, 90, 90, 90], [5, 5, 20, 20, 21, 60, 80], [0, 0, 0, 0, 0, 0, 90],
                 [-7, 3, 3, 40, 200, 300, 400]):
        check_grouped(w, a, torch.tensor(ends, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("repeats", [1, 3, 40])
def test_row_indices_out_of_range_are_rows_of_zeros(repeats):
    w = weights(40, 200, F32, 1, E=2)
    a = activations(10, 200, E4M3, 2)
    a.values.view(torch.uint8)[0, 3] = 0x7F                     # a NaN in row 0, which nobody asks for
    rows = torch.tensor([3, -1, 10, 5, 2**31 - 1, -2**31, 9, 1] * repeats, dtype=torch.int32, device="cuda")
    bias = torch.randn(2, 40, device="cuda")
    clean = lq.Rows8(a.values.clone(), a.exps)
    clean.values.view(torch.uint8)[0, 3] = 0
    offsets = torch.tensor([0, 3, 8 * repeats], dtype=torch.int32, device="cuda")
    want = check_grouped(w, clean, offsets, rows, bias)
    assert torch.equal(lq.gemm8_grouped(w, a, offsets, rows=rows, bias=bias, out_dtype=F32), want)


@pytest.mark.parametrize("B", [1, 9, 40, 300])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_16_bit_activations_give_the_quantized_ones_bit_for_bit(B, dtype):
    for m, K in ((130, 515), (513, 2048), (64, 1000)):
        w, a = weights(m, K, torch.uint8, 3), activations(B, K, dtype, 4)
        one = lq.gemm8(w, a, out_dtype=F32)
        two = lq.gemm8(w, lq.quantize8(a), out_dtype=F32)
        assert (one - two).abs().max() <= 2.0**-20 * (rows64(a).abs() @ matrix64(w).abs().T).max()


@pytest.mark.parametrize("B", [1, 5, 70, 300])
def test_sums_that_are_exact_come_out_exact(B):
    """Integers: every sum below 2^24 is exact in whatever order."""
    g = torch.Generator().manual_seed(1)
    K, m = 1500, 200
    w = torch.randint(-7, 8, (m, K), generator=g).float()
    a = torch.randint(-7, 8, (B, K), generator=g).float()
    w[:, ::128], a[:, ::128] = 7.0, 7.0                          # every block's scale the same
    for kind in (torch.uint8, F32):
        q = lq.quantize8_blocks(w.cuda())
        if kind == F32:
            q = lq.Blocks8(q.values, torch.exp2(q.scales.float() - 127))
        for x in (a.half().cuda(), lq.quantize8(a.cuda())):
            assert torch.equal(lq.gemm8(q, x, out_dtype=F32).double(), a.double().cuda() @ w.double().cuda().T)


@pytest.mark.parametrize("B", [2, 40, 300])
@pytest.mark.parametrize("dtype", TYPES)
def test_nan_in_one_token(B, dtype):
    w, a = weights(100, 400, torch.uint8, 1), activations(B, 400, dtype, 2)
    clean = lq.gemm8(w, a, out_dtype=F32)
    if isinstance(a, lq.Rows8):
        a.values.view(torch.uint8)[1, 77] = 0x7F
    else:
        a[1, 77] = float("nan")
    got = lq.gemm8(w, a, out_dtype=F32)
    assert torch.isnan(got[1]).all()
    keep = torch.arange(B, device="cuda") != 1
    assert torch.equal(got[keep], clean[keep])


def test_scales_over_their_range():
    """Exponents from end to end, float32 scales of any size, and a block of zeros."""
    m, K, B = 256, 512, 3
    w, a = weights(m, K, torch.uint8, 1), activations(B, K, E4M3, 2)
    for shift in (-60, 60):
        s = w.scales.clone()
        held = torch.zeros(2, 4, dtype=torch.uint8, device="cuda")
        held[:] = (s.int() + shift).to(torch.uint8)
        far = lq.Blocks8(w.values, held)
        assert torch.equal(lq.gemm8(far, a, out_dtype=F32), torch.ldexp(lq.gemm8(w, a, out_dtype=F32), torch.tensor(shift, device="cuda")))
    zero = lq.Blocks8(w.values, torch.zeros(2, 4, device="cuda"))
    assert (lq.gemm8(zero, a, out_dtype=F32) == 0).all()


@pytest.mark.parametrize("B", [1, 30, 300])
def test_rows_apart(B):
    """Pitches of activations, exponents, residual and outputs; what lies between the rows stays."""
    m, K = 130, 300
    w, a = weights(m, K, F32, 1), activations(B, K, E4M3, 2)
    values = torch.zeros(B, 512, dtype=torch.uint8, device="cuda")
    values[:, :384] = a.values.view(torch.uint8)
    values[:, 384:] = 0x7F
    exps = torch.full((B, 8), 255, dtype=torch.uint8, device="cuda")
    exps[:, :3] = a.exps
    apart = lq.Rows8(values.view(E4M3)[:, :384], exps[:, :3])
    res = torch.randn(B, 200, device="cuda").half()[:, 3:133]
    out = torch.full((B, 150), 5.0, dtype=F16, device="cuda")
    lq.gemm8(w, apart, residual=res, out=out[:, 7:137])
    assert torch.equal(out[:, 7:137], lq.gemm8(w, a, residual=res.contiguous(), out_dtype=F16))
    assert (out[:, :7] == 5).all() and (out[:, 137:] == 5).all()
    wide = torch.randn(B, K + 9, device="cuda").half()
    for x in (wide[:, :K], wide[:, 1:K + 1]):
        assert torch.equal(lq.gemm8(w, x), lq.gemm8(w, x.contiguous()))


def test_gradient_of_the_activations():
    """dL/da of L = sum(c . (a w^T)) through the transposed weights: the product's own definition, and against
    differences of the forward sum in float64, which is linear in a."""
    for kind in (torch.uint8, F32):
        m, K, B = 300, 520, 20
        w, a = weights(m, K, kind, 1), activations(B, K, E4M3, 2)
        dz = lq.quantize8(torch.randn(B, m, device="cuda"), E5M2)
        da = lq.gemm8(w.transposed(), dz, out_dtype=F32)
        assert da.shape == (B, 640)
        W, c = matrix64(w), rows64(dz)[:, :m]
        bound = 2.0**-20 * (c.abs() @ W.abs()) + 2.0**-23 * (c @ W).abs()
        assert ((da.double() - c @ W).abs() <= bound).all()
        x, step = rows64(a), torch.zeros(B, 640, dtype=torch.float64, device="cuda")
        step[3, 17] = 0.5
        slope = ((c * ((x + step) @ W.T)).sum() - (c * ((x - step) @ W.T)).sum()).item()
        assert abs(slope - da[3, 17].item()) <= bound[3, 17].item() + 1e-9 * (c.abs() @ W.abs()).sum().item()


@pytest.mark.parametrize("B", [1, 20, 300])
def test_the_same_twice_and_on_two_streams(B):
    w, a = weights(500, 4096, F32, 1), activations(B, 4096, BF16, 2)
    want = lq.gemm8(w, a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        x, y = lq.gemm8(w, a), lq.gemm8(w, a, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(x, want) and torch.equal(y, want)


@pytest.mark.parametrize("B", [1, 20, 300])
def test_captured_and_replayed(B):
    w, a = weights(500, 4096, F32, 1), activations(B, 4096, BF16, 2)
    we, r = weights(128, 4096, torch.uint8, 3, E=4), routing(B, 4, 2, 1)
    run = lambda: (lq.gemm8(w, a), lq.gemm8_grouped(we, a, r.offsets, rows=r.rows))  # noqa: E731
    run()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run()
        graphs.append((graph, out))
    for seed in (5, 6, 7):
        a.copy_(activations(B, 4096, BF16, seed))
        for graph, _ in graphs:
            graph.replay()
        eager = run()
        torch.cuda.synchronize()
        for _, out in graphs:
            for x, y in zip(out, eager):
                assert torch.equal(x, y)


def test_no_rows():
    w = weights(40, 200, torch.uint8, 1, E=2)
    offsets = torch.zeros(3, dtype=torch.int32, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    for a in (activations(5, 200, E4M3, 1), activations(5, 200, F16, 1)):
        assert lq.gemm8_grouped(w, a, offsets, rows=none).shape == (0, 40)
        out = torch.full((5, 40), 3.0, device="cuda")
        assert (lq.gemm8_grouped(w, a, offsets, out=out) == 3.0).all()      # runs without rows
    assert lq.gemm8_grouped(w, torch.empty(0, 200, dtype=F16, device="cuda"), offsets).shape == (0, 40)
    with pytest.raises(lq.LQError):
        lq.gemm8(lq.Blocks8(w.values[0], w.scales[0]), torch.empty(0, 200, dtype=F16, device="cuda"))


def test_one_expert_takes_all_rows_and_indices_repeat():
    w = weights(96, 300, torch.uint8, 1, E=5)
    a = activations(3, 300, E4M3, 2)
    rows = torch.tensor([2, 2, 0, 2, 1] * 60, dtype=torch.int32, device="cuda")
    for ends in ([0, 0, 300, 300, 300, 300], [0, 300, 300, 300, 300, 300], [0, 0, 0, 0, 0, 300]):
        check_grouped(w, a, torch.tensor(ends, dtype=torch.int32, device="cuda"), rows)


def test_many_rows_of_few_tokens():
    """More rows than a launch has threads for, from three tokens: tiles and offsets stay whole."""
    R = 2**24 + 77
    w = weights(2, 128, torch.uint8, 1, E=1)
    a = activations(3, 128, E4M3, 2)
    rows = (torch.arange(R, device="cuda") % 3).to(torch.int32)
    out = lq.gemm8_grouped(w, a, torch.tensor([0, R], dtype=torch.int32, device="cuda"), rows=rows, out_dtype=F16)
    want = lq.gemm8(lq.Blocks8(w.values[0], w.scales[0]), a, out_dtype=F16)
    assert torch.equal(out, want[rows.long()])
