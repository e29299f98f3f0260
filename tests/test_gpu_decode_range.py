"""mx_decode at both ends of its types: exact up to the largest number, Inf past
it, subnormal numbers exact in 32 bits and rounded to nearest in bf16."""
import math

import pytest
import torch

from tensor_scaling_cast_gb300 import fp8q as F

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("a CUDA GPU is required for the gpu tests")
    from tensor_scaling_cast_gb300 import build
    build.build()
    F.load()
    torch.cuda.set_device(0)


#: format, a code, its value, a code one step below it and that value
CODES = [(F.E2M1, 0x77, 6.0, 0x66, 4.0), (F.E4M3, 0x7E, 448.0, 0x7D, 416.0), (F.E5M2, 0x7B, 57344.0, 0x7A, 49152.0)]


def decoded(fmt, byte, e8m0, kind):
    q = torch.full((1, 16 if fmt == F.E2M1 else 32), byte, dtype=torch.uint8, device="cuda")
    out = torch.full((1, 32), 5.0, dtype=kind, device="cuda")
    F.mx_decode(F.MXMatrix(q, torch.full((1, 1), e8m0, dtype=torch.uint8, device="cuda"), fmt), out)
    assert (out == out[0, 0]).all()
    return float(out[0, 0])


@pytest.mark.parametrize("fmt,byte,value,below,lower", CODES)
@pytest.mark.parametrize("kind", [BF, F32])
def test_largest_numbers(fmt, byte, value, below, lower, kind):
    for e in range(235, 255):
        for code, v in ((byte, value), (below, lower)):
            m, x = math.frexp(v)
            want = math.ldexp(m, x + e - 127)        # a Python float holds it
            assert decoded(fmt, code, e, kind) == (want if want < 2.0 ** 128 else math.inf)


@pytest.mark.parametrize("fmt,code,value", [(F.E2M1, 0x33, 1.5), (F.E4M3, 0x01, 2.0 ** -9), (F.E4M3, 0x07, 7 * 2.0 ** -9),
                                            (F.E5M2, 0x03, 3 * 2.0 ** -16)])
def test_smallest_numbers(fmt, code, value):
    for e in range(0, 20):
        want = math.ldexp(value, e - 127)
        assert decoded(fmt, code, e, F32) == want
        near = torch.tensor(want, dtype=torch.float64).to(F32).to(BF)
        assert decoded(fmt, code, e, BF) == float(near)


def test_a_finite_number_can_come_back_as_infinity():
    """4-bit casts with headroom reach 2^127, whose codes from 2 on are past the types' largest."""
    x = torch.full((1, 32), 3e38, device="cuda")
    x[0, 1::2] = 1e38
    m = F.MXMatrix.allocate(1, 32, F.E2M1)
    F.mx_cast_ex(x, F.E2M1, F.MX_FLOOR, 4, F.MX_ROWWISE, m.q, m.e8m0)
    assert int(m.e8m0) == 254 and (m.q == 0x14).all()
    for kind in (BF, F32):
        out = torch.empty(1, 32, dtype=kind, device="cuda")
        F.mx_decode(m, out)
        assert (out[0, ::2] == math.inf).all() and (out[0, 1::2] == 2.0 ** 126).all()
