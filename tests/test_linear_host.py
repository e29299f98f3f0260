"""Linear layers in MX form without a GPU: the host-side refusals of mx_decode,
mx_matmul, mx_act_forward, mx_act_backward and of the 4-bit casts, and the
binding's checks."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import kv

E4M3, E5M2, E2M1 = 0, 1, 2
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def lib():
    from tensor_scaling_cast_gb300 import build
    build.build()
    from tensor_scaling_cast_gb300 import fp8q
    return fp8q.load()


class Matrix(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("e8m0", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("q_stride", ctypes.c_int64), ("e8m0_stride", ctypes.c_int64),
                ("format", ctypes.c_int32)]


def matrix(rows=64, cols=128, fmt=E4M3, **kw):
    d = dict(q=0x10000, e8m0=0x20000, rows=rows, cols=cols, q_stride=cols // 2 if fmt == E2M1 else cols,
             e8m0_stride=cols // 32, format=fmt)
    d.update(kw)
    return Matrix(**d)


def ref(m):
    return None if m is None else ctypes.addressof(m)


def decode(lib, m, out=0x30000, dtype=BF16, stride=128):
    return lib.mx_decode(ref(m), out, dtype, stride, None)


def matmul(lib, a, b, out=0x30000, dtype=BF16, stride=64, add=None, add_stride=64):
    return lib.mx_matmul(ref(a), ref(b), out, dtype, stride, add, add_stride, None)


def forward(lib, act=0, z=0x30000, u=0x40000, zs=128, us=128, dtype=BF16, rows=64, cols=128, z_saved=None, u_saved=None,
            rule=0, h=0x50000, hs=128, h_mx=None):
    return lib.mx_act_forward(act, z, zs, u, us, dtype, rows, cols, ref(z_saved), ref(u_saved), rule, h, hs, ref(h_mx),
                              None)


def backward(lib, z_saved, u_saved, act=0, dh=0x30000, dhs=128, dtype=BF16, dz=0x40000, dzs=128, du=0x50000, dus=128,
             h=None, hs=0):
    return lib.mx_act_backward(act, ref(z_saved), ref(u_saved), dh, dhs, dtype, dz, dzs, du, dus, h, hs, None)


BAD = [(dict(format=3), -3), (dict(format=-1), -3), (dict(rows=-1), -1), (dict(rows=1 << 31), -1), (dict(cols=0), -1),
       (dict(cols=48), -1), (dict(cols=-32), -1), (dict(q=0), -1), (dict(e8m0=0), -1), (dict(q=0x10008), -2),
       (dict(q_stride=136), -2), (dict(q_stride=112), -1), (dict(e8m0_stride=3), -1), (dict(q_stride=-128), -1)]


@pytest.mark.parametrize("kw,status", BAD)
def test_matrix_refusals(lib, kw, status):
    bad, good = matrix(**kw), matrix()
    assert decode(lib, bad) == status
    assert matmul(lib, bad, good) == status
    assert matmul(lib, good, bad) == status
    assert backward(lib, bad, matrix()) == status
    assert backward(lib, matrix(), bad) == status
    assert forward(lib, z_saved=bad, u_saved=matrix()) == status
    assert forward(lib, z_saved=matrix(), u_saved=bad) == status
    assert forward(lib, h_mx=bad) == status


def test_decode_refusals(lib):
    assert decode(lib, None) == -1
    assert decode(lib, matrix(), out=None) == -1
    assert decode(lib, matrix(), dtype=2) == -3
    assert decode(lib, matrix(), out=0x30008) == -2
    assert decode(lib, matrix(), stride=132) == -2
    assert decode(lib, matrix(), stride=96) == -1
    assert decode(lib, matrix(rows=0, q=0, e8m0=0), out=None) == 0


def test_matmul_refusals(lib):
    a, b = matrix(), matrix()
    assert matmul(lib, None, b) == -1
    assert matmul(lib, a, None) == -1
    assert matmul(lib, a, matrix(cols=160)) == -1
    assert matmul(lib, matrix(cols=(1 << 26) + 32), matrix(cols=(1 << 26) + 32)) == -1
    assert matmul(lib, a, matrix(fmt=E2M1)) == -3
    assert matmul(lib, matrix(fmt=E2M1), b) == -3
    assert matmul(lib, a, b, dtype=2) == -3
    assert matmul(lib, a, b, out=None) == -1
    assert matmul(lib, a, b, out=0x30001) == -2
    assert matmul(lib, a, b, out=0x30002, dtype=F32) == -2
    assert matmul(lib, a, b, stride=63) == -1
    assert matmul(lib, a, b, add=0x60001) == -2
    assert matmul(lib, a, b, add=0x60000, add_stride=63) == -1
    assert matmul(lib, matrix(rows=0, q=0, e8m0=0), b, out=None) == 0
    assert matmul(lib, a, matrix(rows=0, q=0, e8m0=0), out=None) == 0


def test_activation_refusals(lib):
    eight, four = matrix(), matrix(fmt=E2M1)
    for act in (-1, 3):
        assert forward(lib, act=act) == -1
        assert backward(lib, eight, matrix(), act=act) == -1
    assert forward(lib, rule=3) == -1
    assert forward(lib, dtype=5) == -3
    assert forward(lib, z=None) == -1
    assert forward(lib, h=None) == -1                              # nothing to write
    assert forward(lib, z=0x30008) == -2
    assert forward(lib, us=132) == -2
    assert forward(lib, zs=96) == -1
    assert forward(lib, cols=100) == -1
    assert forward(lib, rows=-1) == -1
    assert forward(lib, z_saved=eight) == -1                       # u would be lost
    assert forward(lib, u=None, z_saved=eight, u_saved=matrix()) == -1
    assert forward(lib, z_saved=four, u_saved=matrix()) == -3
    assert forward(lib, z_saved=eight, u_saved=matrix(fmt=E5M2)) == -3
    assert forward(lib, z_saved=matrix(rows=63), u_saved=matrix()) == -1
    assert forward(lib, h_mx=matrix(cols=160)) == -1
    assert forward(lib, rows=0, z=None, u=None, h=0x50000) == 0
    assert backward(lib, None, None, du=None) == -1
    assert backward(lib, eight, matrix(), du=None) == -1
    assert backward(lib, eight, None) == -1
    assert backward(lib, four, matrix()) == -3
    assert backward(lib, eight, matrix(fmt=E5M2)) == -3
    assert backward(lib, eight, matrix(rows=32)) == -1
    assert backward(lib, eight, matrix(), dtype=2) == -3
    assert backward(lib, eight, matrix(), dh=None) == -1
    assert backward(lib, eight, matrix(), dz=None) == -1
    assert backward(lib, eight, matrix(), dzs=100) == -2
    assert backward(lib, eight, matrix(), h=0x60004, hs=128) == -2
    assert backward(lib, matrix(rows=0, q=0, e8m0=0), None, dh=None, dz=None, du=None) == 0


def test_4_bit_casts_take_rows_and_the_dual_form(lib):
    assert lib.mx_cast_ex(0x10000, BF16, 64, 64, E2M1, 0, 0, 1, 0x20000, 0x30000, None, None) == -3      # column-wise
    assert lib.mx_cast_ex(0x10000, BF16, 64, 48, E2M1, 0, 0, 0, 0x20000, 0x30000, None, None) == -1
    assert lib.mx_cast_ex(0x10000, BF16, 64, 64, 3, 0, 0, 0, 0x20000, 0x30000, None, None) == -3
    assert lib.mx_cast_ex(0x10000, BF16, 64, 64, E2M1, 0, 5, 0, 0x20000, 0x30000, None, None) == -1
    assert lib.mx_cast_ex(0x10000, BF16, 0, 64, E2M1, 0, 0, 0, None, None, None, None) == 0
    assert lib.mx_cast_dual(0x10000, BF16, 40, 64, E2M1, 0, 0, 1, 1, 1, 1, None, None, None) == -1
    assert lib.mx_cast_dual(0x10000, BF16, 64, 64, E2M1, 0, 0, 0x20008, 1, 0x30000, 1, None, None, None) == -2
    h = ctypes.c_void_p()
    assert lib.fp8q_create(E2M1, 4, 0, 0, ctypes.byref(h)) == -3
    assert lib.mx_error_stats(0x10000, BF16, 64, 64, 0x20000, 0x30000, E2M1, 0x40000, None) == -3


def test_binding_refuses_wrong_tensors():
    from tensor_scaling_cast_gb300 import fp8q as F
    m = F.MXMatrix.allocate(8, 64, E4M3, device="cpu")
    assert m.shape == (8, 64) and F.MXMatrix.allocate(3, 96, E2M1, device="cpu").q.shape == (3, 48)
    half = F.MXMatrix(m.q[:, :32], m.e8m0[:, :1], E4M3)
    assert half.shape == (8, 32) and half._struct.q_stride == 64 and half._struct.e8m0_stride == 2
    for q, e, f in ((m.q, m.e8m0, E2M1), (m.q.int(), m.e8m0, E4M3), (m.q, m.e8m0[:4], E4M3), (m.q[:, ::2], m.e8m0[:, :1], E4M3),
                    (m.q.t(), m.e8m0, E4M3)):
        with pytest.raises(TypeError):
            F.MXMatrix(q, e, f)
    x = torch.zeros(8, 64, dtype=torch.bfloat16)
    out = torch.zeros(8, 8)
    for call in (lambda: F.mx_decode(m, x[:4]), lambda: F.mx_decode(m, x.half()), lambda: F.mx_decode(m, x.t().t()[:, ::2]),
                 lambda: F.mx_matmul(m, m, out[:4]), lambda: F.mx_matmul(m, m, out.t()[:, ::2]),
                 lambda: F.mx_matmul(m, m, out.double()), lambda: F.mx_matmul(m, m, out, add=out.bfloat16()),
                 lambda: F.mx_act_forward(0, x, x.float(), h=x), lambda: F.mx_act_forward(0, x, x[:4], h=x),
                 lambda: F.mx_act_forward(0, x.half(), h=x.half()), lambda: F.mx_act_forward(0, x[0], h=x[0]),
                 lambda: F.mx_act_backward(0, m, None, x, x.float()), lambda: F.mx_act_backward(0, m, None, x[:4], x)):
        with pytest.raises(TypeError):
            call()


def test_binding_refuses_tensors_off_the_gpu():
    from tensor_scaling_cast_gb300 import fp8q as F
    m = F.MXMatrix.allocate(8, 64, E4M3, device="cpu")
    x = torch.zeros(8, 64, dtype=torch.bfloat16)
    for call in (lambda: F.mx_decode(m, x), lambda: F.mx_matmul(m, m, torch.zeros(8, 8)),
                 lambda: F.mx_act_forward(0, x, h=x), lambda: F.mx_act_backward(0, m, None, x, x)):
        with pytest.raises(TypeError, match="cpu"):
            call()


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU answer")
@pytest.mark.parametrize("fmt", [E2M1, E4M3])
def test_no_gpu_is_an_error(lib, fmt):
    for m, n, k in ((1, 64, 64), (20, 300, 2048), (40, 64, 64), (64, 8192, 8192), (300, 300, 2048), (1024, 1024, 64)):
        assert matmul(lib, matrix(m, k, fmt), matrix(n, k, fmt), stride=n) == -4          # FP8Q_ECUDA
        assert matmul(lib, matrix(m, k, fmt), matrix(n, k, fmt), dtype=F32, stride=n, add=0x30000, add_stride=n) == -4
    assert decode(lib, matrix(fmt=fmt)) == -4
    assert forward(lib, z_saved=matrix(), u_saved=matrix()) == -4
    assert backward(lib, matrix(), matrix()) == -4
    for rows, cols in ((32, 32), (8192, 8192)):
        assert lib.mx_cast_dual(0x10000, BF16, rows, cols, fmt, 0, 0, 0x20000, 0x30000, 0x40000, 0x50000, None, None,
                                None) == -4


def test_reference_with_headroom_agrees_with_the_c_oracle(orc):
    x = (np.random.default_rng(3).standard_normal((16, 64)) * 100).astype(np.float32)
    x[3, :32] = 0
    for headroom in (0, 1, 4):
        q, e, _ = orc.mx_cast_ex(x.view(np.uint32), E4M3, 1, headroom, 0)
        code, e8 = kv.encode(x, E4M3, 1, headroom)
        assert np.array_equal(q, code) and np.array_equal(e, e8)
