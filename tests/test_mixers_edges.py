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


def test_sizes_beyond_a_c_int(no_library):
    """Sizes that a C int cannot hold are refused: passed on, they would be cut
    to their low 32 bits and part of the rows computed."""
    big = 2 ** 32 + 8
    w, A = F(8, 4), F(8, 8)
    for lead in ((1, big), (big, 1)):
        x, m = T(*lead, 8), T(*lead, 1, 8)
        fails(ValueError, la.forward_selective, x=x, dt=x, A=A, Bm=m, Cm=m)
        fails(ValueError, la.backward_selective, x=x, dt=x, A=A, Bm=m, Cm=m, dy=x)
        fails(ValueError, la.forward_conv, x=x, w=w)
        fails(ValueError, la.backward_conv, x=x, w=w, dy=x)
        y = T(lead[0], 1, lead[1], 8)
        fails(ValueError, la.forward_norm_gate, y=y, gate=x)
        fails(ValueError, la.backward_norm_gate, y=y, gate=x, do=x)
    x, m = T(big, 8), T(big, 1, 8)
    fails(ValueError, la.decode_selective, x=x, dt=x, A=A, Bm=m, Cm=m, h=F(big, 8, 8))
    fails(ValueError, la.decode_conv, x=x, w=w, state=T(big, 3, 8))
    passes(la.forward_norm_residual, x=x)                 # rows are 64 bits wide; refused in the library
    x = T(1, big)
    fails(ValueError, la.forward_norm_residual, x=x)
    fails(ValueError, la.backward_norm_residual, r=x, do=x)
    x, m = T(1, 1, big), T(1, 1, 1, 8)
    fails(ValueError, la.forward_selective, x=x, dt=x, A=F(big, 8), Bm=m, Cm=m)
    fails(ValueError, la.forward_conv, x=x, w=F(big, 4))
    fails(ValueError, la.forward_norm_gate, y=T(1, 1, 1, big), gate=x)
    fails(ValueError, la.forward_norm_gate, y=T(1, big, 1, 8), gate=T(1, 1, big * 8))
