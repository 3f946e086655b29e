"""DeviceLayer.forward_ep and DeviceExperts.forward at the ends of what they take."""
import numpy as np
import pytest
import torch

from bit_lifted_gemv_amd import lq, synth
from oracle import lq_oracle as O

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.mark.parametrize("B", [1, 20, 200])
def test_values_past_the_range_of_float16(B):
    """Lifted values of 2^40 need bfloat16, which holds each to half a step, 2^-9 of itself: a sum of
    2432 of random signs is off by less than six standard deviations of 2^-9 / sqrt 3 of its root mean
    square, and the largest of 768 outputs is above two of those: 6 x 2^-9 / sqrt 3 / 2 = 3.4e-3."""
    L = synth.make_layer(m=768, n=1024, d=8, D=19, B=B, seed=B, dtype="bf16")
    layer = lq.DeviceLayer.from_synth(L, device="cuda")
    a = (lq.to_torch_16(L.a, L.dtype).float() * 2.0**40).to(BF16).cuda()          # a power of two: exact
    ref = np.ascontiguousarray(O.forward(L.packed, L.K, L.M, L.t_inv, L.s, L.a, L.d, L.D, L.dtype)) * 2.0**40
    out = layer.forward_ep(a, out_dtype=F32, lift_dtype=BF16)
    assert torch.isfinite(out).all()
    assert O.rel_err_colmax(out.cpu().numpy(), ref) <= 3.4e-3


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_experts_of_no_tokens(dtype):
    """A batch of no tokens gives no rows, like the router and the experts' products."""
    E, n, f, d, D = 4, 256, 128, 8, 16
    w1 = torch.zeros(E, 2 * f, n // d * D // 32, dtype=torch.int32, device="cuda")
    w2 = torch.zeros(E, n, f // d * D // 32, dtype=torch.int32, device="cuda")
    eye = lambda q: torch.eye(128, dtype=dtype, device="cuda").expand(q, 128, 128).contiguous()  # noqa: E731
    M = torch.rand(d, D, device="cuda")
    layer = lq.DeviceExperts(w1, torch.ones(E, 2 * f, device="cuda"), eye(n // 128), M, w2,
                             torch.ones(E, n, device="cuda"), eye(f // 128), M, d, D, 2)
    x = torch.empty(0, n, dtype=dtype, device="cuda")
    for res in (None, x):
        out = layer.forward(x, torch.empty(0, E, device="cuda"), residual=res)
        assert out.shape == (0, n) and out.dtype == dtype
    one = torch.ones(1, n, dtype=dtype, device="cuda")
    assert layer.forward(one, torch.zeros(1, E, device="cuda")).shape == (1, n)
