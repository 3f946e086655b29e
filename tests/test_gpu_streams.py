"""Calls on a given stream beside calls on the current one, with nothing
between them: each allocates its own workspace and results, and both have to
be right."""
import pytest
import torch

from bit_lifted_gemv_amd import lq

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def words(gen, *shape):
    *lead, K = shape
    return torch.randint(-2**31, 2**31, (*lead, (K // 32 + 3) // 4 * 4), generator=gen).to(torch.int32).cuda()


def case(name, gen):
    """Two inputs of one size, and the call."""
    if name == "route":
        return [torch.randn(16384, 256, generator=gen).cuda() for _ in range(2)], lambda x, **k: lq.route(x, 8, **k)
    if name in ("prompt", "tokens"):
        m, K, B = (4096, 8192, 600) if name == "prompt" else (8192, 20480, 5)      # an image; slices
        w, s = words(gen, m, K), torch.rand(m, generator=gen).cuda()
        return ([torch.randn(B, K, generator=gen).to(BF16).cuda() for _ in range(2)],
                lambda x, **k: lq.gemm_ep(w, s, x, **k))
    E, m, K, T, k = 8, 2048, 2048, 300, 2
    w, s = words(gen, E, m, K), torch.rand(E, m, generator=gen).cuda()
    r = lq.route(torch.randn(T, E, generator=gen).cuda(), k)
    if name == "grouped":
        return ([torch.randn(T, K, generator=gen).to(BF16).cuda() for _ in range(2)],
                lambda x, **o: lq.gemm_grouped(w, s, x, r.offsets, rows=r.rows, act="silu", gated=True, **o))
    return ([torch.randn(T * k, K, generator=gen).to(BF16).cuda() for _ in range(2)],
            lambda x, **o: lq.gemm_join(w, s, x, r.offsets, r.pos, r.weight, **o))


@pytest.mark.parametrize("name", ["prompt", "tokens", "grouped", "join", "route"])
def test_a_call_on_a_stream_beside_one_on_the_current_stream(name):
    (x, y), call = case(name, torch.Generator().manual_seed(3))
    flat = lambda r: r if isinstance(r, tuple) else (r,)  # noqa: E731
    want_x, want_y = flat(call(x)), flat(call(y))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(6):
        got = [(want_x, flat(call(x))), (want_y, flat(call(y, stream=side))), (want_x, flat(call(x))),
               (want_y, flat(call(y, stream=side)))]
        torch.cuda.synchronize()
        for want, have in got:
            assert all(torch.equal(p, q) for p, q in zip(want, have))


def test_results_of_another_stream_can_be_dropped_early():
    """The caller's stream waits for the other one, reads the result and lets go of it, and the
    other stream goes on: what was read is the first result."""
    (x, y), call = case("prompt", torch.Generator().manual_seed(4))
    want = call(x).float()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        out = call(x, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        read = sum(out.float() for _ in range(8)) / 8
        del out
        call(y, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(read, want)


def test_the_other_wrappers_on_a_stream_of_their_own():
    """Lift and GEMV of one and sixteen tokens, the layer on the parts image and M's objective on a
    side stream that makes every workspace for the first time, beside the same on the current one."""
    from bit_lifted_gemv_amd import synth
    gen = torch.Generator().manual_seed(6)
    L = synth.make_layer(m=4096, n=4096, d=8, D=19, B=16, seed=6, dtype="bf16")
    layer = lq.DeviceLayer.from_synth(L, device="cuda")
    a = lq.to_torch_16(L.a, L.dtype).cuda()
    samples = torch.randn(20000, 8, generator=gen).cuda()

    def run(stream=None):
        one = lq.lift(a[:1], layer.t_inv, layer.M, layer.d, layer.D, stream=stream)
        out = [lq.gemv(layer.w, layer.s, one, layer.K, stream=stream)]
        img = lq.lift_parts(a, layer.t_inv, layer.M, layer.d, layer.D, stream=stream)
        out.append(lq.gemv_parts(layer.w, layer.s, img, layer.K, 16, stream=stream))
        return out + list(lq.softmin_grad(samples, layer.M, stream=stream))
    want = run()
    for _ in range(3):
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        here, there = run(), run(side)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) and torch.equal(x, z) for x, y, z in zip(want, here, there))


@pytest.mark.parametrize("name", ["prompt", "tokens", "grouped", "join", "route"])
def test_a_captured_call_on_a_side_stream(name):
    """Inside one graph: a call on a second stream beside one on the captured stream.  Replayed three
    times with new inputs and eager calls between."""
    gen = torch.Generator().manual_seed(8)
    (x, y), call = case(name, gen)
    flat = lambda r: r if isinstance(r, tuple) else (r,)  # noqa: E731
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    call(x), call(y, stream=side)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        there, here = flat(call(y, stream=side)), flat(call(x))
        main.wait_stream(side)
        both = [p.float() + q.float() for p, q in zip(here, there)]
    for _ in range(3):
        for t in (x, y):
            t.copy_(torch.randn(t.shape, generator=gen).to(t.dtype))
        g.replay()
        torch.cuda.synchronize()
        want_x, want_y = flat(call(x)), flat(call(y))
        assert all(torch.equal(p, q) for p, q in zip(want_x, here))
        assert all(torch.equal(p, q) for p, q in zip(want_y, there))
        assert all(torch.equal(p.float() + q.float(), b) for p, q, b in zip(want_x, want_y, both))


def test_join_may_write_over_its_activations():
    """out in the place of a_lift: the sums over experts come last."""
    gen = torch.Generator().manual_seed(9)
    for T in (3, 300):
        E, m, k = 4, 512, 2
        w, s = words(gen, E, m, m), torch.rand(E, m, generator=gen).cuda()
        r = lq.route(torch.randn(T, E, generator=gen).cuda(), k)
        a = torch.randn(T * k, m, generator=gen).to(BF16).cuda()
        want = lq.gemm_join(w, s, a, r.offsets, r.pos, r.weight)
        assert torch.equal(lq.gemm_join(w, s, a, r.offsets, r.pos, r.weight, out=a[:T]), want)


def test_learning_on_a_side_stream():
    """Samples made right before the call and dropped with it."""
    gen = torch.Generator().manual_seed(10)
    M0 = (torch.randn(8, 16, generator=gen) / 4).cuda()
    host = [torch.randn(4096, 8, generator=gen) for _ in range(4)]
    want, losses = lq.learn_m(M0, [x.cuda() for x in host])
    for _ in range(3):
        side = torch.cuda.Stream()
        batches = [x.cuda() for x in host]
        torch.cuda.synchronize()
        M, ls = lq.learn_m(M0, batches, stream=side)
        del batches
        junk = [torch.full((4096, 8), float("nan"), device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        assert torch.equal(M, want) and all(torch.equal(p, q) for p, q in zip(ls, losses))
        del junk
