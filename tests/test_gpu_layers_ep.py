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
