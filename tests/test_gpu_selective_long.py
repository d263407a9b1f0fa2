"""Selective scan over rows of several pieces: few rows (four waves share a row's steps), odd and even numbers of modes."""
import pytest

import test_gpu_selective as sel

pytestmark = pytest.mark.gpu

# (B, H, N, S, G, D, gate, bias, softplus, state, lengths); pieces of 4096 steps
LONG = [
    (1, 2, 12301, 1, 1, True, True, True, True, True, None),       # three whole pieces and a rest
    (2, 2, 8209, 5, 2, True, True, True, True, True, [8209, 8192]),
    (1, 1, 20000, 7, 1, True, False, True, True, False, [19999]),
    (1, 3, 8704, 2, 3, True, True, True, True, True, None),
]


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", LONG, ids=sel.ids)
def test_selective_scan_long(io, case):
    """y and the final state."""
    sel.test_selective_scan(io, case)


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", LONG[1:2], ids=sel.ids)
def test_selective_scan_bwd_long(io, case):
    """The gradients, from the states that a shared row's waves saved."""
    sel.test_selective_scan_bwd(io, case)
