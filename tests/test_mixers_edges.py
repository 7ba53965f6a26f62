"""Sizes at the ends of the accepted range, without a GPU: refused by the C
entry points and by the binding before any CUDA call."""
import pytest

import kernelized_sequence_mixing_gb300 as la
from test_mixers_host import (INVALID, LDS, SCAN, UNSUPPORTED, Call, F, T, fails, lib, no_library,  # noqa: F401
                              passes)

MOST = 2 ** 31 - 2 ** 16  # tokens; the rounding of parts and runs stays in 32 bits


@pytest.mark.parametrize("B,L", [(1, MOST), (1, 2 ** 31 - 1), (2, MOST // 2), (MOST, 1), (MOST // 8, 8)])
def test_most_tokens(lib, B, L):
    """At the limit refused, one token a sequence fewer accepted (and then
    refused for a missing input)."""
    sizes = {"B": B, "L": L, "E": 8, "N": 8, "G": 1, **LDS}
    conv = {"B": B, "L": L, "E": 8, "W": 4, "ldx": 0, "silu": 1, "dtype": 1}
    calls = [Call(lib.la_forward_selective, SCAN + " h0 lens y hN", sizes),
             Call(lib.la_backward_selective, SCAN + " h0 dy dhN dx ddt dA dBm dCm dD dz ddt_bias dh0", sizes),
             Call(lib.la_forward_conv, "x w bias state lens y state_out", conv),
             Call(lib.la_backward_conv, "x w bias state dy dx dw dbias dstate", conv)]
    for c in calls:
        assert c(x=None) == UNSUPPORTED
        if B * L == MOST and B * 8 < 2 ** 31:
            assert c(x=None, **({"L": L - 1} if L > 1 else {"B": B - 1})) == INVALID
