"""Without a GPU: linear layers of no rows.  A tensor without elements has no
address, so that with no rows a NULL does not say that something was left out."""
import ctypes

import pytest

from tensor_scaling_cast_gb300 import fp8q as F

EINVAL, EDTYPE = -1, -3


@pytest.fixture(scope="module")
def lib():
    from tensor_scaling_cast_gb300 import build
    build.build()
    return F.load()


def empty(cols=128, fmt=F.E4M3, rows=0):
    return F._MXMatrixStruct(None, None, rows, cols, cols // 2 if fmt == F.E2M1 else cols, cols // 32, fmt)


def ref(m):
    return None if m is None else ctypes.addressof(m)


def forward(lib, u_saved=None, z_saved=None, h_mx=None, act=0, dtype=F.BF16, rule=0, cols=128, rows=0):
    return lib.mx_act_forward(act, None, cols, None, cols, dtype, rows, cols, ref(z_saved), ref(u_saved), rule, None, cols,
                              ref(h_mx), None)


def backward(lib, z_saved, u_saved=None, act=0, dtype=F.BF16):
    return lib.mx_act_backward(act, ref(z_saved), ref(u_saved), None, 128, dtype, None, 128, None, 128, None, 128, None)


def test_nothing_to_do(lib):
    z, u, h = empty(), empty(), empty(fmt=F.E2M1)
    assert forward(lib) == 0
    assert forward(lib, u, z) == 0
    assert forward(lib, None, z) == 0
    assert forward(lib, u, z, h) == 0
    assert backward(lib, z) == 0
    assert backward(lib, z, u) == 0


def test_what_is_wrong_without_rows_too(lib):
    z, u = empty(), empty()
    assert forward(lib, u, z, act=3) == EINVAL and forward(lib, u, z, rule=3) == EINVAL
    assert forward(lib, u, z, dtype=7) == EDTYPE
    assert forward(lib, u, z, cols=100) == EINVAL
    assert forward(lib, u, empty(fmt=F.E2M1)) == EDTYPE and forward(lib, empty(fmt=F.E5M2), z) == EDTYPE
    assert forward(lib, u, empty(cols=160)) == EINVAL
    assert backward(lib, None) == EINVAL and backward(lib, z, u, act=-1) == EINVAL
    assert backward(lib, z, u, dtype=7) == EDTYPE and backward(lib, z, empty(fmt=F.E5M2)) == EDTYPE
    assert backward(lib, z, empty(cols=160)) == EINVAL and backward(lib, empty(rows=-1)) == EINVAL


def test_with_rows_what_is_left_out_is_still_refused(lib):
    kept = F._MXMatrixStruct(0x10000, 0x20000, 4, 128, 128, 4, F.E4M3)
    assert forward(lib, rows=4) == EINVAL
    assert forward(lib, kept, kept, rows=4) == EINVAL
    assert backward(lib, kept, kept) == EINVAL
