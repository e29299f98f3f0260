"""Without a GPU: the form that mx_matmul takes by sizes, types and alignment,
and the sizes that tests/test_gpu_matmul_forms.py runs each form at."""
import ctypes
import itertools
import random

import pytest

import matmul_forms as forms
from tensor_scaling_cast_gb300 import fp8q as F


@pytest.fixture(scope="module")
def lib():
    from tensor_scaling_cast_gb300 import build
    build.build()
    return F.load()


def matrix(rows, cols, fmt):
    return F._MXMatrixStruct(0x10000, 0x20000, rows, cols, cols // 2 if fmt == F.E2M1 else cols, cols // 32, fmt)


def plan(lib, m, n, k, fmt, fp32, add, sms=forms.SMS, out=0x30000, stride=None):
    a, b, form = matrix(m, k, fmt), matrix(n, k, fmt), F.MXMatmulForm()
    st = lib.mx_matmul_plan(ctypes.addressof(a), ctypes.addressof(b), out, F.F32 if fp32 else F.BF16, stride or n,
                            0x40000 if add else None, n, sms, ctypes.addressof(form))
    assert st == 0
    return form


@pytest.mark.parametrize("fmt", [F.E2M1, F.E4M3])
@pytest.mark.parametrize("columns,way_out,m,n,kblocks,fp32", forms.PAIRS)
def test_pair_forms(lib, fmt, columns, way_out, m, n, kblocks, fp32):
    f = plan(lib, m, n, forms.elements(fmt == F.E2M1, kblocks), fmt, fp32, way_out >= forms.ADD_BF16)
    assert (f.pair, f.columns, f.way_out, f.splits) == (1, columns, way_out, 1)
    assert f.tiles == -(-m // 256) * -(-n // columns) > forms.SMS          # more than two for some pair


@pytest.mark.parametrize("fmt", [F.E2M1, F.E4M3])
@pytest.mark.parametrize("columns,splits,few,many,kblocks", forms.SPLITS)
def test_split_forms(lib, fmt, columns, splits, few, many, kblocks):
    k = forms.elements(fmt == F.E2M1, kblocks)
    for m, n in ((few, many), (many, few)):
        f = plan(lib, m, n, k, fmt, False, False)
        assert (f.pair, f.columns, f.splits) == (0, columns, splits)


def test_no_other_form_is_taken(lib):
    """Random sizes over the whole range take no form that the lists do not have."""
    known = {(1, c, w, 1) for c, w, *_ in forms.PAIRS} | {(0, c, 0, s) for c, s, *_ in forms.SPLITS}
    assert {(c, w) for c, w, *_ in forms.PAIRS} == set(itertools.product((128, 256), range(5))) | {(224, 0), (224, 4)}
    rng = random.Random(1)
    seen = set()
    for _ in range(40000):
        m, n = (max(1, int(2 ** rng.uniform(0, 14.3))) for _ in range(2))
        if rng.random() < 0.5:
            n = 8 * (n // 8 + 1)
        fmt, fp32, add = rng.choice((F.E2M1, F.E4M3, F.E5M2)), rng.random() < 0.5, rng.random() < 0.5
        f = plan(lib, m, n, 32 * max(1, int(2 ** rng.uniform(0, 9))), fmt, fp32, add, out=0x30000 + rng.choice((0, 4)))
        seen.add((f.pair, f.columns, f.way_out, f.splits))
    assert seen <= known


def test_refusals_and_nothing_to_do(lib):
    a, b, form = matrix(64, 128, F.E4M3), matrix(64, 128, F.E4M3), F.MXMatmulForm()

    def status(x=a, y=b, out=0x30000, dtype=F.BF16, stride=64, sms=152, to=ctypes.addressof(form)):
        return lib.mx_matmul_plan(ctypes.addressof(x), ctypes.addressof(y), out, dtype, stride, None, 0, sms, to)
    assert status() == 0 and form.tiles > 0
    assert status(to=None) == -1 and status(sms=1) == -1 and status(sms=-4) == -1
    assert status(y=matrix(64, 160, F.E4M3)) == -1 and status(y=matrix(64, 128, F.E2M1)) == -3
    assert status(out=None) == -1 and status(out=0x30001) == -2 and status(dtype=2) == -3 and status(stride=63) == -1
    assert status(x=matrix(0, 128, F.E4M3)) == 0 and form.tiles == 0
