"""lq_route against a plain sort on the CPU: choices, order and offsets exact,
weights to 2^-20 (exp and a sum of at most 1024 float32 terms, each within a
few 2^-24) of the float64 softmax."""
import numpy as np
import pytest
import torch

from bit_lifted_gemv_amd import lq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"


def plain(logits, k, valid, renorm):
    T, E = logits.shape
    x = logits.double().numpy()
    ids = np.full((T, k), -1, np.int32)
    weight = np.zeros((T, k))
    for t in range(T):
        if valid is not None and not valid[t]:
            continue
        live = [e for e in range(E) if not np.isnan(x[t, e]) and x[t, e] != -np.inf]
        best = sorted(live, key=lambda e: (-x[t, e], e))[:k]
        if not best:
            continue
        top = x[t, best[0]]
        share = lambda e: 1.0 if x[t, e] == top else np.exp(x[t, e] - top)  # noqa: E731
        total = sum(share(e) for e in (best if renorm else live))
        ids[t, :len(best)] = best
        weight[t, :len(best)] = [share(e) / total for e in best]
    flat = ids.reshape(-1)
    pairs = [i for e in range(E) for i in np.flatnonzero(flat == e)]
    rows = np.full(T * k, -1, np.int32)
    pos = np.full(T * k, -1, np.int32)
    rows[:len(pairs)] = [i // k for i in pairs]
    pos[pairs] = np.arange(len(pairs))
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(E)])])
    return ids, weight, pos.reshape(T, k), rows, offsets


def compare(logits, k, valid=None, renorm=True, dev_logits=None):
    r = lq.route(logits.cuda() if dev_logits is None else dev_logits, k,
                 valid=None if valid is None else valid.cuda(), renorm=renorm)
    ids, weight, pos, rows, offsets = plain(logits, k, valid, renorm)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.pos.cpu().numpy(), pos)
    assert np.array_equal(r.rows.cpu().numpy(), rows)
    off = np.abs(r.weight.cpu().double().numpy() - weight)
    assert (off <= 2.0**-20 * weight + 1e-38).all(), off.max()


CASES = [(1, 1, 1), (1, 64, 8), (2, 3, 3), (5, 65, 2), (63, 64, 8), (64, 128, 6), (65, 16, 4),
         (129, 256, 8), (300, 1024, 32), (1000, 7, 2), (517, 200, 10), (2049, 60, 6), (64, 513, 1)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", CASES)
def test_route(T, E, k, dtype):
    gen = torch.Generator().manual_seed(T * 1000 + E)
    logits = (torch.randn(T, E, generator=gen) * 2).to(dtype)
    valid = (torch.rand(T, generator=gen) < 0.8).to(torch.uint8)
    compare(logits, k)
    compare(logits, k, valid=valid, renorm=False)


@pytest.mark.parametrize("T", [3, 200])
def test_route_ties_and_special_values(T):
    gen = torch.Generator().manual_seed(T)
    logits = torch.randint(-2, 3, (T, 70), generator=gen).float()       # many equal ones
    logits[logits == 0] *= -1                                            # -0 among them
    logits[0, ::2] = 0.0
    compare(logits, 9)
    logits[torch.rand(T, 70, generator=gen) < 0.5] = float("-inf")
    logits[torch.rand(T, 70, generator=gen) < 0.3] = float("nan")
    logits[1] = float("-inf")
    logits[2] = float("nan")
    logits[2, 69] = -3e38
    logits[0, 5] = logits[0, 66] = float("inf")
    for renorm in (True, False):
        compare(logits, 20, renorm=renorm)
    compare(torch.zeros(T, 70), 32)


def test_route_masks_and_sizes():
    logits = torch.randn(100, 8)
    compare(logits, 2, valid=torch.zeros(100, dtype=torch.uint8))        # nobody
    compare(logits, 2, valid=torch.ones(100, dtype=torch.bool))
    r = lq.route(torch.empty(0, 8, device="cuda"), 2)
    assert r.ids.shape == (0, 2) and (r.offsets == 0).all() and r.rows.numel() == 0
    wide = torch.randn(130, 40).cuda()                                   # rows that lie apart
    compare(wide[:, 5:28].cpu(), 3, dev_logits=wide[:, 5:28])


def test_route_long():
    """More than 256 runs of 64 tokens: workgroups of several runs."""
    gen = torch.Generator().manual_seed(5)
    T, E, k = 40001, 24, 3
    logits = torch.randn(T, E, generator=gen)
    r = lq.route(logits.cuda(), k)
    top = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(r.ids.cpu().long(), top)
    key, perm = torch.sort(top.reshape(-1), stable=True)
    assert torch.equal(r.rows.cpu().long(), perm // k)
    assert torch.equal(r.pos.cpu().reshape(-1)[perm].long(), torch.arange(T * k))
    assert torch.equal(r.offsets.cpu().long(), torch.searchsorted(key, torch.arange(E + 1)))


def test_route_repeats_and_graph():
    logits = torch.randn(500, 64).cuda()
    ref = lq.route(logits, 8)
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(lq.route(logits, 8), ref))
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        r = lq.route(logits, 8)
    for i in range(3):
        logits.copy_(torch.randn(500, 64))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(r, lq.route(logits, 8))), i


@pytest.mark.parametrize("T,E,k,crowd", [
    (16385, 1021, 4, False),      # two runs a workgroup, words of counts not full
    (49152, 5, 2, True),          # three: every token on one expert, 192 a count
    (49152, 256, 8, False),
    (49153, 7, 3, True),          # four: counts of 16 bits, 256 of them
    (70001, 1024, 1, False),
])
def test_route_runs_per_workgroup(T, E, k, crowd):
    """The oracle of many tokens is a stable sort instead of a loop."""
    gen = torch.Generator().manual_seed(T + E)
    logits = torch.randn(T, E, generator=gen).to(torch.bfloat16)
    if crowd:
        logits[:, 2] = 50.0
    r = lq.route(logits.cuda(), k)
    x = logits.double().numpy()
    ids = np.argsort(-x, axis=1, kind="stable")[:, :k]
    flat = ids.reshape(-1)
    order = np.argsort(flat, kind="stable")
    pos = np.empty(T * k, np.int64)
    pos[order] = np.arange(T * k)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    assert np.array_equal(r.rows.cpu().numpy(), order // k)
    assert np.array_equal(r.pos.cpu().numpy().reshape(-1), pos)
    counts = np.bincount(flat, minlength=E)
    assert np.array_equal(r.offsets.cpu().numpy(), np.concatenate([[0], np.cumsum(counts)]))
    top = np.take_along_axis(x, ids, 1)
    share = np.exp(top - top[:, :1])
    share /= share.sum(1, keepdims=True)
    # d = l - max is rounded to float32, off by up to |d| 2^-24 (a relative half
    # step); exp(d + x) = exp(d) (1 + x + ...) makes that a relative error of
    # |d| 2^-24, beside 2^-20 for exp, the sum and the quotient
    near = 2.0**-20 + np.abs(top - top[:, :1]) * 2.0**-24
    assert (np.abs(r.weight.cpu().double().numpy() - share) <= near * share + 1e-38).all()


def test_route_most_tokens():
    """T = 2^31 - 1: the last workgroup's runs would go on past 2^31.  One expert: every token's
    choice is 0, and order and positions are the tokens' own."""
    T = 2**31 - 1
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB")
    r = lq.route(torch.zeros(T, 1, dtype=torch.bfloat16, device="cuda"), 1)
    assert r.offsets.tolist() == [0, T]
    assert not r.ids.any() and (r.weight == 1).all()
    for lo in range(0, T, 1 << 28):
        own = torch.arange(lo, min(lo + (1 << 28), T), dtype=torch.int32, device="cuda")
        assert torch.equal(r.pos[lo:lo + (1 << 28), 0], own) and torch.equal(r.rows[lo:lo + (1 << 28)], own)
    del r, own
    torch.cuda.empty_cache()
