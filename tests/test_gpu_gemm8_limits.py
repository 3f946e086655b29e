"""The 8-bit layers at the largest sizes of one call: activations of just below 4 GiB,
weights of just below 2 GiB, rows to quantize past 2^32 bytes."""
import pytest
import torch

from bit_lifted_gemv_amd import lq
from test_gpu_gemm8 import near, product64, rows64

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"


def test_quantize_past_4_gib():
    B, K = 2**20 + 5, 4096
    x = torch.zeros(B, K, dtype=BF16, device="cuda")
    x[-300:] = torch.randn(300, K, device="cuda").to(BF16)
    q, want = lq.quantize8(x), lq.quantize8(x[-300:])
    assert torch.equal(q.values[-300:].view(torch.uint8), want.values.view(torch.uint8))
    assert torch.equal(q.exps[-300:], want.exps)
    assert int(q.exps[:-300].min()) == int(q.exps[:-300].max()) == 127


@pytest.mark.parametrize("out", [BF16, F32])
def test_activations_below_4_gib(out):
    B, K, m = 2**20 - 1, 4096, 130
    w = lq.quantize8_blocks(torch.randn(m, K, device="cuda"))
    tail = lq.quantize8(torch.randn(300, K, device="cuda").to(BF16))
    a = lq.Rows8(torch.zeros(B, K, dtype=torch.uint8, device="cuda").view(E4M3),
                 torch.full((B, K // 128), 127, dtype=torch.uint8, device="cuda"))
    a.values.view(torch.uint8)[-300:] = tail.values.view(torch.uint8)
    a.exps[-300:] = tail.exps
    y, dy = product64(w, rows64(tail), None, "none", False, out)
    got = lq.gemm8(w, a, out_dtype=out)
    near(got[-300:], y, dy)
    assert (got[:-300] == 0).all()
    # rows of the end asked for by index: few of them, and many
    one = lq.Blocks8(w.values[None], w.scales[None])
    for n in (3, 300):
        rows = torch.arange(B - n, B, dtype=torch.int32, device="cuda")
        offsets = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        near(lq.gemm8_grouped(one, a, offsets, rows=rows, out_dtype=out), y[-n:], dy[-n:])


@pytest.mark.parametrize("B", [3, 300])
def test_weights_below_2_gib(B):
    m, K = 2**19 - 5, 4096
    tail = lq.quantize8_blocks(torch.randn(123, K, device="cuda"))          # the last, ragged strip
    w = lq.Blocks8(torch.zeros(m, K, dtype=torch.uint8, device="cuda").view(E4M3),
                   torch.full((m // 128 + 1, K // 128), 127, dtype=torch.uint8, device="cuda"))
    w.values.view(torch.uint8)[-123:] = tail.values.view(torch.uint8)
    w.scales[-1:] = tail.scales
    a = lq.quantize8(torch.randn(B, K, device="cuda").to(BF16))
    y, dy = product64(tail, rows64(a), None, "none", False, BF16)
    got = lq.gemm8(w, a)
    near(got[:, -123:], y, dy)
    assert (got[:, :-123] == 0).all()
    both = lq.Blocks8(torch.stack([w.values.view(torch.uint8)] * 2).view(E4M3), torch.stack([w.scales] * 2))
    offsets = torch.tensor([0, 1, B], dtype=torch.int32, device="cuda")
    near(lq.gemm8_grouped(both, a, offsets)[:, -123:], y, dy)
