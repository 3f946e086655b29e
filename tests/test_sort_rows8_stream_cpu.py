"""sort_rows of Rows8 on a given stream: both of its launches go there, and a stream of
another device is refused as it is for one tensor (no GPU needed; stand-ins for tensors,
streams and the library)."""
import types

import pytest
import torch

from bit_lifted_gemv_amd import lq
from test_products8_cpu import Tensor8, gpu8  # noqa: F401
from test_streams_cpu import gpu  # noqa: F401


def call(**k):
    q = lq.Rows8(Tensor8((40, 512), torch.float8_e4m3fn), Tensor8((40, 4), torch.uint8))
    return lq.sort_rows(q, Tensor8((80,), torch.int32), **k)


def test_both_launches_are_on_the_stream(gpu8):  # noqa: F811
    out = call(stream=gpu8.other)
    assert gpu8.handles == [77, 77] and gpu8.current is gpu8.default
    assert all(t.owner is gpu8.other for t in gpu8.made)
    assert all(gpu8.default.cuda_stream in t.used_on for t in gpu8.made) and len(out) == 2
    call()
    assert gpu8.handles == [77, 77, 0, 0]


def test_stream_of_another_device_is_refused(gpu8):  # noqa: F811
    with pytest.raises(ValueError):
        call(stream=types.SimpleNamespace(cuda_stream=5, device=torch.device("cuda", 1)))
    assert not gpu8.handles
