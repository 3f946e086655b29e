"""lq_gemm_ep, lq_gemm_grouped and lq_gemm_join against the definition in
float64.

Tolerances, fixed before the first run.  A value is carried to 2^-14 of the
largest one of its 32 positions with three parts (16-bit outputs) and to
2^-18 with four (float32 outputs): after p parts the remainder is at most 1/4,
1/8, 1/16, 1/16 of a unit of the last part's scale when the largest value is
scaled into [4, 8) (the few 16-bit values above 7.75 come out exactly), so
1/16 / 256 / 4 and 1/16 / 4096 / 4.  A float32 sum of K products in any order
is given 2^-20 of the sum of magnitudes (K <= 4096 here: at most 3 K / 64 + 1
roundings of 2^-24 each, and the matrix cores' own alignment).  So
  dz = s (parts * sum_k largest(k) + 2^-20 sum_k |a_k|) + 2^-23 (|z| + |bias|)
bounds z; activations have slopes below 1.13 and are evaluated to 2^-20 of
|z| + 1; the output's own rounding adds eps / 2 of the value.
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


def words(gen, *shape, extra=0):
    *lead, K = shape
    ldw = ((K + 31) // 32 + 3) // 4 * 4 + extra
    w = torch.randint(-2**31, 2**31, (*lead, ldw), generator=gen, dtype=torch.int64)
    return w.to(torch.int32).cuda()


def signs(w, K):
    bit = (w.long().unsqueeze(-1) >> torch.arange(32, device=w.device)) & 1
    return (2.0 * bit.flatten(-2)[..., :K].double() - 1.0)


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


def product64(w, s, a, bias, out_dtype):
    """z and the bound of its error."""
    K = a.shape[1]
    a = a.double()
    z = a @ signs(w, K).T * s.double()
    pad = torch.nn.functional.pad(a.abs(), (0, -K % 32)).reshape(a.shape[0], (K + 31) // 32, 32)
    largest = pad.amax(2).sum(1, keepdim=True) * 32
    part = 2.0**-18 if out_dtype == F32 else 2.0**-14
    dz = s.double() * (part * largest + 2.0**-20 * a.abs().sum(1, keepdim=True))
    b = 0.0 if bias is None else bias.double()
    z = z + b
    return z, dz + 2.0**-23 * (z.abs() + (0.0 if bias is None else b.abs()))


def finish64(z, dz, act, gated):
    m = z.shape[1]
    g, dg = (z[:, :m // 2], dz[:, :m // 2]) if gated else (z, dz)
    y = act64(g, act)
    dy = 1.13 * dg + (0.0 if act == "none" else 2.0**-20 * (g.abs() + 1.0))
    if gated:
        u, du = z[:, m // 2:], dz[:, m // 2:]
        dy = dy * (u.abs() + du) + y.abs() * du
        y = y * u
    return y, dy


def check(out, y, dy, residual=None):
    if residual is not None:
        y = y + residual.double()
    tol = dy * (1 + 1e-6) + y.abs() * (torch.finfo(out.dtype).eps / 2 + 2.0**-22) + 1e-30
    if out.dtype == F16:
        tol = tol + 2.0**-25                      # halves of its smallest step
    off = (out.double() - y).abs()
    assert torch.isfinite(out).all()
    bad = off > tol
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} outside, worst "
                           f"{float((off / tol).max()):.3g} times the bound")


def data(dev, seed, m, K, B, dtype, E=None, extra=0, outliers=False):
    gen = torch.Generator().manual_seed(seed)
    lead = (m,) if E is None else (E, m)
    w = words(gen, *lead, K, extra=extra)
    s = (torch.rand(*lead, generator=gen) * 0.02 + 0.01).cuda()
    bias = torch.randn(*lead, generator=gen).cuda()
    a = torch.randn(B, K, generator=gen)
    if outliers:
        a *= torch.where(torch.rand(K, generator=gen) < 0.02, 50.0, 1.0)
    return w, s, bias, a.to(dtype).cuda(), gen


# (m, K, B): one row, one token; sizes below and above every tile; each tile shape of the
# many-token kernel (128, 256 and 512 rows, 32 and 64 tokens) and of the few-token one
SHAPES = [
    (1, 8, 1), (2, 32, 1), (37, 40, 3), (128, 256, 1), (130, 264, 33), (257, 520, 64),
    (512, 1024, 65), (1282, 2056, 100), (2048, 512, 200), (300, 4096, 17), (640, 4000, 5),
    (4100, 1024, 16), (64, 4096, 2), (16400, 520, 1), (16400, 520, 9),
    (28672, 256, 640), (28672, 264, 40), (8192, 256, 500), (65536, 264, 16), (16384, 512, 31),
]


@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (F16, F16), (F16, F32), (BF16, F16)])
@pytest.mark.parametrize("m,K,B", SHAPES)
def test_gemm_ep_shapes(dev, m, K, B, dtype, out_dtype):
    print(m, K, B, dtype, out_dtype, flush=True)
    w, s, bias, a, gen = data(dev, m + K + B, m, K, B, dtype)
    res = torch.randn(B, m, generator=gen).to(out_dtype).cuda()
    out = lq.gemm_ep(w, s, a, bias=bias, act="gelu", residual=res, out_dtype=out_dtype)
    assert out.shape == (B, m) and out.dtype == out_dtype
    check(out, *finish64(*product64(w, s, a, bias, out_dtype), "gelu", False), res)
    if m % 2 == 0:
        res = res[:, :m // 2].contiguous()
        out = lq.gemm_ep(w, s, a, act="silu", gated=True, residual=res, out_dtype=out_dtype)
        check(out, *finish64(*product64(w, s, a, None, out_dtype), "silu", True), res)


@pytest.mark.parametrize("B", [1, 6, 100])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", sorted(lq.ACTS))
def test_gemm_ep_activations(dev, act, gated, B):
    w, s, bias, a, _ = data(dev, 7, 386, 1032, B, BF16)
    bias = bias * 4
    for b in (None, bias):
        out = lq.gemm_ep(w, s, a, bias=b, act=act, gated=gated, out_dtype=F32)
        check(out, *finish64(*product64(w, s, a, b, F32), act, gated))


@pytest.mark.parametrize("B", [1, 4, 16, 70])
def test_gemm_ep_outlying_values(dev, B):
    w, s, bias, a, _ = data(dev, 8, 514, 2048, B, F16, outliers=True)
    for dt in (F16, F32):
        check(lq.gemm_ep(w, s, a, bias=bias, out_dtype=dt),
              *product64(w, s, a, bias, dt))


@pytest.mark.parametrize("B", [1, 5, 16, 40, 130])
def test_gemm_ep_pitches_and_garbage(dev, B):
    """Rows that lie apart, a longer weight pitch with random bits behind K, outputs that no
    wide store fits, the residual in place, and nothing written beside the output."""
    m, K = 262, 1000
    w, s, bias, a, gen = data(dev, 9, m, K, B, BF16, extra=8)
    wide = torch.full((B, K + 56), float("nan"), dtype=BF16, device=dev)
    wide[:, :K] = a
    for gated in (False, True):
        n = m // 2 if gated else m
        buf = torch.full((B, n + 5), 7.0, dtype=BF16, device=dev)
        res = torch.randn(B, n, generator=gen).to(BF16).cuda()
        view = buf[:, 3:3 + n]
        view.copy_(res)
        out = lq.gemm_ep(w, s, wide[:, :K], bias=bias, act="relu", gated=gated, residual=view,
                         out=view)
        assert out is view
        check(view, *finish64(*product64(w, s, a, bias, BF16), "relu", gated), res)
        assert (buf[:, :3] == 7).all() and (buf[:, 3 + n:] == 7).all()
        flat = lq.gemm_ep(w, s, a, bias=bias, act="relu", gated=gated, residual=res)
        assert torch.equal(flat, view)


@pytest.mark.parametrize("B", [1, 3, 16, 64])
def test_gemm_ep_zero_small_and_large_values(dev, B):
    m, K = 200, 768
    w, s, _, a, _ = data(dev, 10, m, K, B, BF16)
    assert (lq.gemm_ep(w, s, torch.zeros_like(a)) == 0).all()
    for scale in (2.0**-90, 2.0**90):
        out = lq.gemm_ep(w, s, (a.float() * scale).to(BF16), out_dtype=BF16)
        ref = lq.gemm_ep(w, s, a)
        assert torch.equal(out.float() * (1 / scale), ref.float())   # powers of two: exactly
    tiny = torch.full_like(a, 2.0**-130)                              # below the least scale: zero or right
    out = lq.gemm_ep(w, s, tiny, out_dtype=F32)
    assert torch.isfinite(out).all() and out.abs().max() <= 2.0**-126


@pytest.mark.parametrize("B", [2, 5, 16, 33, 100])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_gemm_ep_nonfinite_token(dev, bad, B):
    """A token with an infinity or a NaN is all NaN, and the other tokens do not change."""
    m, K = 160, 1024
    w, s, _, a, _ = data(dev, 11, m, K, B, F16)
    clean = lq.gemm_ep(w, s, a)
    a = a.clone()
    a[1, K - 5] = bad
    out = lq.gemm_ep(w, s, a)
    assert torch.isnan(out[1]).all()
    keep = [i for i in range(B) if i != 1]
    assert torch.equal(out[keep], clean[keep])


def test_gemm_ep_largest_matrix(dev):
    """2^30 bytes of signs in one call: offsets past 2^29 words, sampled rows."""
    m, K = 16384, 524288
    w = torch.randint(-2**31, 2**31 - 1, (m, K // 32), dtype=torch.int32, device=dev)
    s = torch.rand(m, device=dev) * 0.02 + 0.01
    pick = torch.tensor([0, 1, 8191, 16000, 16383], device=dev)
    for B in (1, 20):
        a = torch.randn(B, K, device=dev).to(BF16)
        out = lq.gemm_ep(w, s, a)
        z = a.double() @ signs(w[pick], K).T * s[pick].double()
        # Gaussian parts: three-part rounding is at most 2^-14 of about 4 standard deviations
        assert ((out[:, pick].double() - z).abs() <= z.abs() * 2.0**-8 + 0.03 * 2.0**-14 * 4 * K**0.5 * 6).all()


# ---------------------------------------------------------------- experts
def runs_of(gen, E, R, kind):
    if kind == "one":                              # everything to one expert
        n = [0] * E
        n[E // 2] = R
    elif kind == "even":
        n = [R // E + (e < R % E) for e in range(E)]
    else:                                          # random, some empty
        cuts = torch.randint(0, R + 1, (E - 1,), generator=gen).sort().values.tolist()
        n = [b - a for a, b in zip([0] + cuts, cuts + [R])]
    off = torch.tensor([0] + n).cumsum(0)
    return off.to(torch.int32).cuda(), n


def grouped64(w, s, bias, a, rows, off, act, gated, out_dtype):
    ys, ds = [], []
    for e in range(w.shape[0]):
        lo, hi = int(off[e]), int(off[e + 1])
        x = a[rows[lo:hi].long()] if rows is not None else a[lo:hi]
        y, d = finish64(*product64(w[e], s[e], x, None if bias is None else bias[e], out_dtype),
                        act, gated)
        ys.append(y)
        ds.append(d)
    return torch.cat(ys), torch.cat(ds)


GROUPED = [  # (E, m, K, tokens, R, kind)
    (1, 130, 264, 5, 5, "even"), (4, 128, 512, 3, 7, "random"), (8, 386, 1032, 40, 100, "random"),
    (64, 256, 512, 24, 192, "random"), (3, 512, 520, 300, 700, "one"), (70, 130, 256, 9, 30, "random"),
    (16, 2816, 512, 100, 800, "even"), (8, 4096, 264, 700, 1400, "random"), (130, 64, 64, 1, 8, "even"),
    (64, 2816, 256, 1, 8, "even"), (5, 1024, 4096, 2, 4, "even"), (1024, 34, 40, 50, 333, "random"),
    (8, 20000, 256, 300, 600, "even"),
]


@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (F16, F32)])
@pytest.mark.parametrize("E,m,K,T,R,kind", GROUPED)
def test_gemm_grouped(dev, E, m, K, T, R, kind, dtype, out_dtype):
    print(E, m, K, T, R, kind, dtype, out_dtype, flush=True)
    w, s, bias, a, gen = data(dev, E + m + R, m, K, T, dtype, E=E)
    off, _ = runs_of(gen, E, R, kind)
    rows = torch.randint(0, T, (R,), generator=gen).to(torch.int32).cuda()
    out = lq.gemm_grouped(w, s, a, off, rows=rows, bias=bias, act="gelu_tanh", out_dtype=out_dtype)
    check(out, *grouped64(w, s, bias, a, rows, off, "gelu_tanh", False, out_dtype))
    out = lq.gemm_grouped(w, s, a, off, rows=rows, act="silu", gated=True, out_dtype=out_dtype)
    check(out, *grouped64(w, s, None, a, rows, off, "silu", True, out_dtype))
    own = a[rows.long()].contiguous()              # rows in the sorted order, no index
    same = lq.gemm_grouped(w, s, own, off, act="silu", gated=True, out_dtype=out_dtype)
    check(same, *grouped64(w, s, None, own, None, off, "silu", True, out_dtype))


@pytest.mark.parametrize("R", [6, 90, 400])
def test_gemm_grouped_rows_behind_the_last_run_stay(dev, R):
    E, m, K, T = 6, 144, 328, 50
    w, s, _, a, gen = data(dev, 21, m, K, T, BF16, E=E)
    off, _ = runs_of(gen, E, R - 5, "random")
    rows = torch.randint(0, T, (R,), generator=gen).to(torch.int32).cuda()
    buf = torch.full((R, m + 8), 3.0, dtype=BF16, device=dev)
    out = lq.gemm_grouped(w, s, a, off, rows=rows, out=buf[:, :m])
    check(out[:R - 5], *grouped64(w, s, None, a, rows, off, "none", False, BF16))
    assert (buf[R - 5:] == 3).all() and (buf[:, m:] == 3).all()


@pytest.mark.parametrize("R", [5, 60, 300])
def test_gemm_grouped_bad_indices(dev, R):
    """Row indices out of range read zeros; offsets out of order or range write inside [0, R) only."""
    E, m, K, T = 4, 96, 200, 20
    w, s, bias, a, gen = data(dev, 22, m, K, T, F16, E=E)
    rows = torch.randint(0, T, (R,), generator=gen).to(torch.int32).cuda()
    off, _ = runs_of(gen, E, R, "even")
    rows[1], rows[R - 1] = -1, T
    out = lq.gemm_grouped(w, s, a, off, rows=rows, bias=bias)
    padded = torch.cat([a, torch.zeros(1, K, dtype=F16, device=dev)])
    fixed = torch.where((rows < 0) | (rows >= T), torch.full_like(rows, T), rows)
    check(out, *grouped64(w, s, bias, padded, fixed, off, "none", False, F16))
    guard = torch.full((R + 8, m), 5.0, dtype=F16, device=dev)
    for bad in ([0, R, 2, R + 1000, R], [-7, 3, -1, 2**31 - 1, -2**31], [R + 5] * 5, [0, 2, 1, 3, 2]):
        lq.gemm_grouped(w, s, a, torch.tensor(bad, dtype=torch.int32, device=dev), rows=rows,
                        bias=bias, out=guard[:R])
        torch.cuda.synchronize()
        assert (guard[R:] == 5).all()


def test_gemm_grouped_no_rows(dev):
    w, s, _, a, _ = data(dev, 23, 64, 64, 4, BF16, E=3)
    off = torch.zeros(4, dtype=torch.int32, device=dev)
    out = lq.gemm_grouped(w, s, a, off, rows=torch.empty(0, dtype=torch.int32, device=dev))
    assert out.shape == (0, 64)
    out = torch.full((4, 64), 2.0, dtype=BF16, device=dev)
    lq.gemm_grouped(w, s, a, off, out=out)         # rows, but no run
    assert (out == 2).all()


JOINED = [  # (E, m, K, T, k)
    (4, 130, 264, 1, 2), (8, 256, 512, 5, 3), (64, 2048, 256, 24, 8), (6, 386, 1032, 300, 2),
    (64, 512, 512, 1, 8), (8, 4096, 264, 200, 2), (16, 64, 4096, 16, 1), (3, 515, 104, 70, 3),
]


@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (F16, F16), (F16, F32)])
@pytest.mark.parametrize("E,m,K,T,k", JOINED)
def test_gemm_join(dev, E, m, K, T, k, dtype, out_dtype):
    print(E, m, K, T, k, dtype, out_dtype, flush=True)
    R = T * k
    w, s, bias, a, gen = data(dev, E + m + T, m, K, R, dtype, E=E)
    logits = torch.randn(T, E, generator=gen).cuda()
    valid = (torch.rand(T, generator=gen) < 0.9).to(torch.uint8).cuda()
    r = lq.route(logits, k, valid=valid)
    res = torch.randn(T, m, generator=gen).to(out_dtype).cuda()
    out = lq.gemm_join(w, s, a, r.offsets, r.pos, r.weight, bias=bias, residual=res,
                       out_dtype=out_dtype)
    z, dz = grouped64(w, s, bias, a, None, r.offsets, "none", False, out_dtype)
    y = torch.zeros(T, m, device=dev, dtype=torch.float64)
    dy = torch.zeros_like(y)
    for j in range(k):
        p = r.pos[:, j].long()
        live = (p >= 0).double()[:, None]
        if z.shape[0]:
            p = p.clamp(0, z.shape[0] - 1)
            wt = r.weight[:, j:j + 1].double() * live
            y += wt * z[p]
            # z between the product and the sum is held in float32 or to 2^-11 of its own
            # size and 2^-12 of the largest of its tile
            dy += wt * (dz[p] + 2.0**-22 * z[p].abs() + (2.0**-12 * z[p].abs() + 2.0**-23 * z[p].abs().amax(1, keepdim=True) if out_dtype != F32 else 0.0))
    check(out, y, dy, res)
    inplace = res.clone()
    lq.gemm_join(w, s, a, r.offsets, r.pos, r.weight, bias=bias, residual=inplace, out=inplace)
    assert torch.equal(inplace, out)


def test_gemm_join_nothing_chosen(dev):
    w, s, _, a, _ = data(dev, 31, 96, 64, 6, BF16, E=3)
    r = lq.route(torch.full((3, 3), float("-inf"), device=dev), 2)
    res = torch.randn(3, 96, device=dev).to(BF16)
    out = lq.gemm_join(w, s, a, r.offsets, r.pos, r.weight, residual=res)
    assert torch.equal(out, res)
    assert (lq.gemm_join(w, s, a, r.offsets, r.pos, r.weight) == 0).all()
    none = lq.gemm_join(w, s, a, r.offsets, r.pos[:0], r.weight[:0])
    assert none.shape == (0, 96)
    r = lq.route(torch.full((3, 3), float("-inf"), device=dev), 2)
    out = lq.gemm_join(w, s, a[:0], r.offsets, r.pos, r.weight, residual=res)   # no rows at all
    assert torch.equal(out, res)


# ---------------------------------------------------------------- together, streams, graphs
def layer64(x, logits, k, t1, M1, d, D, w1, s1, t2, M2, w2, s2):
    """A mixture-of-experts layer in float64 from the definition, no sorting: every token by itself."""
    def lift64(a, t, M):
        n = a.shape[1]
        u = torch.matmul(t.double(), a.double().reshape(a.shape[0], n // 128, 128, 1)).reshape(a.shape[0], n)
        return (u.reshape(-1, d) @ M.double()).reshape(a.shape[0], -1)
    T, m2 = x.shape[0], w2.shape[1]
    out = torch.zeros(T, m2, dtype=torch.float64, device=x.device)
    la = lift64(x, t1, M1)
    S1, S2 = signs(w1, la.shape[1]), signs(w2, w1.shape[1] // 2 // d * D)
    for t in range(T):
        top = torch.sort(logits[t].double(), descending=True, stable=True)
        p = torch.softmax(top.values[:k], 0)
        for j in range(k):
            e = int(top.indices[j])
            z = S1[e] @ la[t] * s1[e].double()
            h = act64(z[:len(z) // 2], "silu") * z[len(z) // 2:]
            out[t] += p[j] * (S2[e] @ lift64(h[None], t2, M2)[0] * s2[e].double())
    return out


@pytest.mark.parametrize("T", [1, 5, 70])
def test_experts_layer(dev, T):
    """Router, lift, experts in, lift, experts out: 2e-2 of the largest output, the 16-bit
    roundings on the way (lifted values, hidden rows, lifted hidden rows, output: four of
    2^-11 in float16, each at most doubled by the gate) and the float6 parts."""
    E, k, n, f, d, D = 12, 3, 256, 384, 8, 16
    gen = torch.Generator().manual_seed(T)
    x = torch.randn(T, n, generator=gen).to(F16).cuda()
    logits = torch.randn(T, E, generator=gen).cuda()
    orth = lambda q: torch.linalg.qr(torch.randn(q, 128, 128, generator=gen))[0].to(F16).contiguous().cuda()  # noqa: E731
    t1, t2 = orth(n // 128), orth(f // 128)
    M1, M2 = ((torch.randn(d, D, generator=gen) / D**0.5).cuda() for _ in range(2))
    w1, w2 = words(gen, E, 2 * f, n // d * D), words(gen, E, n, f // d * D)
    s1, s2 = (torch.rand(E, r, generator=gen).cuda() * 0.02 + 0.03 for r in (2 * f, n))
    layer = lq.DeviceExperts(w1, s1, t1, M1, w2, s2, t2, M2, d, D, k)
    res = torch.randn(T, n, generator=gen).to(F16).cuda()
    out = layer.forward(x, logits, residual=res)
    ref = layer64(x, logits, k, t1, M1, d, D, w1, s1, t2, M2, w2, s2)
    diff = (out.double() - res.double() - ref).abs().max() / ref.abs().max()
    assert diff <= 2e-2, float(diff)
    assert torch.equal(layer.forward(x, logits, residual=res), out)
    masked = layer.forward(x, logits, residual=res, valid=torch.zeros(T, dtype=torch.bool, device=dev))
    assert torch.equal(masked, res)


def test_two_streams_at_once(dev):
    """Calls on two streams at the same time, each with temporaries of its own."""
    w, s, bias, a, gen = data(dev, 41, 1024, 2048, 200, BF16)
    few = a[:4].contiguous()
    ref = [lq.gemm_ep(w, s, x, bias=bias) for x in (a, few)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for _ in range(8):
        for st, x in zip(streams, (a, few)):
            with torch.cuda.stream(st):
                outs.append(lq.gemm_ep(w, s, x, bias=bias))
    outs2 = [torch.empty_like(ref[0]) for _ in range(4)]
    torch.cuda.synchronize()
    for o, st in zip(outs2, streams * 2):
        lq.gemm_ep(w, s, a, bias=bias, out=o, stream=st)
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, ref[i % 2])
    for o in outs2:
        assert torch.equal(o, ref[0])


@pytest.mark.parametrize("T", [1, 24, 150])
def test_graphs_of_the_experts(dev, T):
    """Two graphs of router + experts in + experts out captured on one stream, replayed in turn and
    three times each with eager calls and new inputs between; each replay equals the eager result."""
    E, k, m, K = 16, 4, 256, 512
    w, s, bias, _, gen = data(dev, 51, m, K, 1, BF16, E=E)
    wj, sj = words(gen, E, 128, 128), torch.rand(E, 128, generator=gen).cuda()
    xs = [torch.randn(T, K, generator=gen).to(BF16).cuda() for _ in range(2)]
    ls = [torch.randn(T, E, generator=gen).cuda() for _ in range(2)]

    def run(x, lg):
        r = lq.route(lg, k)
        h = lq.gemm_grouped(w, s, x, r.offsets, rows=r.rows, bias=bias, act="silu", gated=True)
        return lq.gemm_join(wj, sj, h, r.offsets, r.pos, r.weight)

    st = torch.cuda.Stream()
    graphs, outs = [], []
    with torch.cuda.stream(st):
        for x, lg in zip(xs, ls):
            run(x, lg)
    torch.cuda.synchronize()
    for x, lg in zip(xs, ls):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            outs.append(run(x, lg))
        graphs.append(g)
    for rep in range(3):
        for x, lg in zip(xs, ls):
            x.copy_(torch.randn(T, K, generator=gen).to(BF16))
            lg.copy_(torch.randn(T, E, generator=gen))
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for x, lg, o in zip(xs, ls, outs):
            assert torch.equal(run(x, lg), o), rep


def test_results_do_not_depend_on_timing(dev):
    for B in (1, 16, 300):
        w, s, bias, a, _ = data(dev, 61, 2050, 4096, B, F16)
        ref = lq.gemm_ep(w, s, a, bias=bias, act="gelu")
        for _ in range(5):
            assert torch.equal(lq.gemm_ep(w, s, a, bias=bias, act="gelu"), ref)


def test_the_same_result_as_lq_gemm(dev):
    """Next to lq_gemm on the same operands: float32 outputs within both bounds."""
    w, s, _, a, _ = data(dev, 71, 700, 2048, 130, F16)
    z, dz = product64(w, s, a, None, F32)
    old = lq.gemm(w, s, a)
    new = lq.gemm_ep(w, s, a, out_dtype=F32)
    check(new, z, dz)
    assert ((old - new).abs().double() <= dz + 2.0**-20 * z.abs() + 1e-6 * z.abs().max()).all()


def test_wrapper_refusals(dev):
    w, s, bias, a, _ = data(dev, 81, 64, 128, 4, BF16)
    with pytest.raises(TypeError):
        lq.gemm_ep(w, s, a.float())
    with pytest.raises(ValueError):
        lq.gemm_ep(w, s, a, act="swish")
    with pytest.raises(ValueError):
        lq.gemm_ep(w, s[:63], a)
    with pytest.raises(ValueError):
        lq.gemm_ep(w, s, a.cpu())
    with pytest.raises(ValueError):
        lq.gemm_ep(w, s, a.t())
    with pytest.raises(TypeError):
        lq.gemm_ep(w, s, a, residual=torch.zeros(4, 64, device=dev))
    with pytest.raises(lq.LQError):
        lq.gemm_ep(w, s, a[:, 1:121])              # not 16-byte aligned
    with pytest.raises(lq.LQError):
        lq.gemm_ep(w, s, a[:0])
    with pytest.raises(lq.LQError):
        lq.gemm_ep(w, s, a[:1].expand(4, 128))     # pitch 0
    with pytest.raises(ValueError):
        lq.gemm_grouped(w[None], s[None], a, torch.zeros(3, dtype=torch.int32, device=dev))
    with pytest.raises(lq.LQError):
        lq.route(torch.zeros(2, 4, device=dev), 5)


# Each tile of the many-row kernel, and its slices of the positions: (m, K, B)
MANY = [
    (28672, 256, 641),                     # 512 x 64 in two workgroups of four waves (float32: 256 x 64)
    (8192, 256, 1023),                     # 512 x 64 in eight waves
    (8190, 512, 500),                      # 256 x 64
    (262200, 256, 17),                     # 512 x 32
    (38402, 1024, 60),                     # 256 x 32 in four waves
    (28672, 1032, 57),                     # 256 x 32 in eight
    (4096, 8192, 250), (4100, 8200, 40),   # 128 x 32, one slice and four
    (1000, 65536, 20), (514, 49160, 90),   # sixteen slices and fewer, odd lengths
]


@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (F16, F32)])
@pytest.mark.parametrize("m,K,B", MANY)
def test_gemm_ep_many_rows(dev, m, K, B, dtype, out_dtype):
    print(m, K, B, dtype, out_dtype, flush=True)
    w, s, bias, a, gen = data(dev, m + K + B, m, K, B, dtype)
    s = s * (4096 / K) ** 0.5 if K > 4096 else s       # sums of K terms in the range of the others
    pick = torch.randperm(m // 2, generator=gen)[:min(m // 2, 600)].cuda()
    both = torch.cat([pick, pick + m // 2])            # outputs checked, as gate and up rows
    res = torch.randn(B, m, generator=gen).to(out_dtype).cuda()
    out = lq.gemm_ep(w, s, a, bias=bias, act="silu", residual=res, out_dtype=out_dtype)
    z, dz = product64(w[both], s[both], a, bias[both], out_dtype)
    dz = dz * max(1.0, K / 4096)                       # the bound of the sum grows with its length
    check(out[:, both], *finish64(z, dz, "silu", False), res[:, both])
    half = res[:, :m // 2].contiguous()
    out = lq.gemm_ep(w, s, a, bias=bias, act="gelu", gated=True, residual=half, out_dtype=out_dtype)
    check(out[:, pick], *finish64(z, dz, "gelu", True), half[:, pick])
    assert torch.equal(lq.gemm_ep(w, s, a, bias=bias, act="gelu", gated=True, residual=half.clone(),
                                  out_dtype=out_dtype), out)


LONG_RUNS = [  # (E, m, K, tokens, R): slices of the positions over ragged runs, and short runs of many experts
    (2, 500, 32768, 60, 60), (3, 64, 65536, 5, 12), (1, 96, 40960, 30, 30), (128, 2048, 512, 300, 2048),
    (5, 1000, 16384, 64, 200),
]


@pytest.mark.parametrize("E,m,K,T,R", LONG_RUNS)
def test_experts_long_positions(dev, E, m, K, T, R):
    """Rows in and out of the experts where the positions are split; the last three rows are in no run."""
    print(E, m, K, T, R, flush=True)
    w, s, bias, a, gen = data(dev, E + m + K, m, K, T, BF16, E=E)
    s = s * (4096 / K) ** 0.5 if K > 4096 else s
    off, _ = runs_of(gen, E, R - 3, "random")
    rows = torch.randint(0, T, (R,), generator=gen).to(torch.int32).cuda()
    grow = max(1.0, K / 4096)
    for gated in (False, True):
        out = torch.full((R, m // 2 if gated else m), 9.0, dtype=BF16, device=dev)
        lq.gemm_grouped(w, s, a, off, rows=rows, bias=bias, act="silu", gated=gated, out=out)
        y, dy = grouped64(w, s, bias, a, rows, off, "silu", gated, BF16)
        check(out[:R - 3], y, dy * grow)
        assert (out[R - 3:] == 9).all()
    own = a[rows.long()].contiguous()
    pos = torch.randperm(R - 3, generator=gen)[:(R - 3) // 2 * 2].reshape(-1, 2).to(torch.int32).cuda()
    weight = torch.rand(pos.shape, generator=gen).cuda()
    out = lq.gemm_join(w, s, own, off, pos, weight, bias=bias)
    z, dz = grouped64(w, s, bias, own, None, off, "none", False, BF16)
    y = sum(weight[:, j:j + 1].double() * z[pos[:, j].long()] for j in range(2))
    dy = sum(weight[:, j:j + 1].double() * (grow * dz[pos[:, j].long()] + 2.0**-20 * z[pos[:, j].long()].abs())
             for j in range(2))
    check(out, y, dy)


@pytest.mark.parametrize("B", [40, 250])
def test_many_rows_pitches_and_nonfinite(dev, B):
    """The many-row kernel (B = 40: four slices): rows that lie apart, random bits behind K, outputs
    that no wide store fits, the residual in place, a token with an infinity, zeros and 2^90."""
    m, K = 4098, 8136
    w, s, bias, a, gen = data(dev, 91, m, K, B, F16, extra=8)
    s = s * 0.7
    pick = torch.randperm(m // 2, generator=gen)[:200].cuda()
    wide = torch.full((B, K + 56), float("nan"), dtype=F16, device=dev)
    wide[:, :K] = a
    for gated in (False, True):
        n, at = (m // 2, torch.cat([pick, pick + m // 2])) if gated else (m, pick)
        buf = torch.full((B, n + 5), 7.0, dtype=F16, device=dev)
        res = torch.randn(B, n, generator=gen).to(F16).cuda()
        view = buf[:, 3:3 + n]
        view.copy_(res)
        lq.gemm_ep(w, s, wide[:, :K], bias=bias, act="relu", gated=gated, residual=view, out=view)
        z, dz = product64(w[at], s[at], a, bias[at], F16)
        check(view[:, pick], *finish64(z, 2 * dz, "relu", gated), res[:, pick])
        assert (buf[:, :3] == 7).all() and (buf[:, 3 + n:] == 7).all()
        assert torch.equal(lq.gemm_ep(w, s, a, bias=bias, act="relu", gated=gated, residual=res), view)
    clean = lq.gemm_ep(w, s, a)
    a[1, 77] = float("-inf")
    out = lq.gemm_ep(w, s, a)
    keep = [i for i in range(B) if i != 1]
    assert torch.isnan(out[1]).all() and torch.equal(out[keep], clean[keep])
    assert (lq.gemm_ep(w, s, torch.zeros_like(a)) == 0).all()
    b = torch.randn(B, K, generator=gen).to(BF16).cuda()
    ref, big = lq.gemm_ep(w, s, b), lq.gemm_ep(w, s, (b.float() * 2.0**90).to(BF16))
    assert torch.equal(big.float() * 2.0**-90, ref.float())


@pytest.mark.parametrize("m,K,B", [(4096, 8192, 40), (4096, 8192, 250), (8192, 68096, 5)])
def test_gemm_ep_graphs_and_streams(dev, m, K, B):
    """Two captured graphs (slices, parts image, or both as the sizes give) replayed at the same time
    on two streams, three times with new inputs, each equal to the eager call."""
    w, s, bias, a, gen = data(dev, 95, m, K, B, BF16)
    xs = [a, a.flip(0).contiguous()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    graphs, outs = [], []
    for st, x in zip(streams, xs):
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            outs.append(lq.gemm_ep(w, s, x, bias=bias, act="silu"))
        graphs.append(g)
    for rep in range(3):
        for x in xs:
            x.copy_(torch.randn(B, K, generator=gen).to(BF16))
        torch.cuda.synchronize()
        for st, g in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for x, o in zip(xs, outs):
            assert torch.equal(lq.gemm_ep(w, s, x, bias=bias, act="silu"), o), rep


@pytest.mark.parametrize("B", [1, 20, 200])
def test_layer_with_epilogue(dev, B):
    """DeviceLayer.forward_ep against the float64 layer of the oracle: 2e-3 of each token's largest
    output (the layer bar) for the lifted values' rounding to float16, and the output's own."""
    import numpy as np
    from bit_lifted_gemv_amd import synth
    from oracle import lq_oracle as O
    L = synth.make_layer(m=768, n=1024, d=8, D=19, B=B, seed=B, dtype="bf16")
    layer = lq.DeviceLayer.from_synth(L, device=dev)
    a = lq.to_torch_16(L.a, L.dtype).to(dev)
    ref = torch.from_numpy(np.ascontiguousarray(O.forward(L.packed, L.K, L.M, L.t_inv, L.s, L.a, L.d, L.D, L.dtype))).to(dev)
    bias = torch.randn(768, device=dev)
    res = torch.randn(B, 384, device=dev).to(BF16)
    z = ref.double() + bias.double()
    want = act64(z[:, :384], "silu") * z[:, 384:] + res.double()
    out = layer.forward_ep(a, bias=bias, act="silu", gated=True, residual=res)
    assert out.dtype == BF16 and out.shape == (B, 384)
    bar = 2e-3 * (want.abs().amax(1, keepdim=True) + ref.double().abs().amax(1, keepdim=True) * 2)
    assert ((out.double() - want).abs() <= bar + want.abs() * 2.0**-8).all()
    plain = layer.forward_ep(a, out_dtype=F32)
    assert O.rel_err_colmax(plain.cpu().numpy(), ref.cpu().numpy()) <= 2e-3


@pytest.mark.parametrize("m,B", [(64, 1), (300, 5), (256, 16), (200, 40), (1024, 200), (8192, 300)])
def test_float32_result_keeps_small_values_beside_a_large_one(dev, m, B):
    """float16 values of 11 bits in the block of one 2048 times theirs: all are
    multiples of 2^-11 and every partial sum lies below 2048 + 1024 < 2^12, so
    float32 sums are exact and the result is the exact one."""
    K = 1024
    gen = torch.Generator().manual_seed(m + B)
    w = torch.randint(-2**31, 2**31, (m, K // 32), generator=gen).to(torch.int32)
    steps = torch.randint(1024, 2048, (B, K), generator=gen) * (2 * torch.randint(0, 2, (B, K), generator=gen) - 1)
    a = steps.double() * 2.0**-11
    a[torch.arange(B), torch.randint(0, K, (B,), generator=gen)] = 2048.0
    z = a @ signs(w, K).T
    out = lq.gemm_ep(w.to(dev), torch.ones(m, device=dev), a.to(F16).to(dev), out_dtype=F32)
    assert torch.equal(out.cpu().double(), z)
