"""lq_quant8 and lq_quant8_blocks refuse outputs over their input, before any HIP call
(no GPU needed): other workgroups still read it."""
import pytest

from bit_lifted_gemv_amd import lq

P, Q, E = 0x10000000, 0x20000000, 0x30000000          # never dereferenced
F32, E4M3 = 0, 3
UNSUPPORTED = 5


@pytest.mark.parametrize("x,q,e", [(P, P, E), (P, Q, P)])
def test_outputs_over_the_input_are_refused(x, q, e):
    L = lq.load_library()
    assert L.lq_quant8(x, F32, 5, 300, 300, q, E4M3, 384, e, 4, None) == UNSUPPORTED
    assert b"overlaps" in L.lq_last_error()
    assert L.lq_quant8_blocks(x, F32, 1, 200, 300, 300, q, 384, e, 4, None) == UNSUPPORTED
    assert L.lq_quant8(x, F32, 0, 300, 300, q, E4M3, 384, e, 4, None) == 0      # no rows: nothing is written
