"""Refusals of arrays whose spans no address space holds (no GPU needed): the
comparison of spans must not run on sums beyond 64 bits."""
import pytest

from lut_binary_basis_b200 import fluxbin
from test_int8_host import SHAPE, linear, norm, quant, silu

WIDE, MANY = 1 << 39, 1 << 30                 # 2^69 elements apart


@pytest.mark.parametrize("call,kw", [
    (quant, dict(T=MANY, ldx=WIDE)), (quant, dict(T=MANY, ldq=WIDE)), (quant, dict(T=(1 << 31) - 1, ldx=WIDE, ldq=WIDE)),
    (quant, dict(T=(1 << 25) + 1, ldx=WIDE)),         # 2^65 bytes: 0 in 64 bits
    (silu, dict(T=MANY, ldg=WIDE)), (silu, dict(T=MANY, ldu=WIDE)), (silu, dict(T=MANY, ldq=WIDE)),
    (norm, dict(T=MANY, ldh=WIDE)), (norm, dict(T=MANY, ldd=WIDE)), (norm, dict(T=MANY, ldq=WIDE)),
    (norm, dict(T=MANY, o=0xC0000000, ldo=WIDE)), (norm, dict(T=1 << 20, ldh=1 << 36, flags=fluxbin.FLAG_H_FP32)),
    (linear, dict(M=MANY, ldw=WIDE, ldy=MANY)), (linear, dict(T=MANY, ldx=WIDE)), (linear, dict(T=MANY, ldy=WIDE)),
    (linear, dict(T=1 << 20, ldy=1 << 36, flags=fluxbin.FLAG_Y_FP32)),
])
def test_spans_beyond_any_address_space(call, kw):
    assert call(**kw) == SHAPE


def test_pitches_that_say_nothing():
    """One row, or none, at any pitch up to 2^39."""
    assert quant(T=0, ldx=WIDE, ldq=WIDE) == 0 and linear(T=0, ldx=WIDE, ldy=WIDE) == 0
    assert quant(T=1, ldx=WIDE, x=0) == -1 and norm(T=1, ldh=WIDE, h=0) == -1       # on to the next check
