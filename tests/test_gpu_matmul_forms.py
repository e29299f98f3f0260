"""Every form of mx_matmul (kernel, tile, way out, CTAs that share a sum), with
several tiles to a pair of SMs, on sums of whole numbers: exact."""
import pytest
import torch

import matmul_forms as forms
from canary import Guards
from tensor_scaling_cast_gb300 import fp8q as F

pytestmark = pytest.mark.gpu

G = Guards(seed=0x23)
BF, F32 = torch.bfloat16, torch.float32
#: codes of 0, 1, 2, -1, -2
CODES = {F.E2M1: (0, 2, 4, 10, 12), F.E4M3: (0, 0x38, 0x40, 0xB8, 0xC0)}
VALUES = (0.0, 1.0, 2.0, -1.0, -2.0)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("a CUDA GPU is required for the gpu tests")
    from tensor_scaling_cast_gb300 import build
    build.build()
    F.load()
    torch.cuda.set_device(0)


@pytest.fixture(autouse=True)
def _guards():
    G.release()
    yield
    G.check_and_release("at the end of the test")
    assert F.fp8q_pipeline_status() == 0


def whole(rows, cols, fmt, seed):
    """A matrix of 0, +-1, +-2 under scales 1, 2 and 4, and its values."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    at = torch.randint(0, 5, (rows, cols), generator=g, device="cuda")
    e = torch.randint(127, 130, (rows, cols // 32), generator=g, device="cuda")
    q = torch.tensor(CODES[fmt], dtype=torch.uint8, device="cuda")[at]
    if fmt == F.E2M1:
        q = q[:, ::2] | q[:, 1::2] << 4
    v = torch.tensor(VALUES, dtype=torch.float64, device="cuda")[at] * torch.exp2(e.double() - 127).repeat_interleave(32, 1)
    return F.MXMatrix(q.contiguous(), e.to(torch.uint8), fmt), v


def check(a, b, want, kind, add=None):
    """Sums below 2^24 are exact in 32 bits, and rounded once."""
    total = want if add is None else want + add.double()
    assert float(total.abs().max()) < 2.0 ** 24
    out = G.full(tuple(want.shape), float("nan"), kind)
    F.mx_matmul(a, b, out, add=add)
    G.check("after mx_matmul")
    assert torch.equal(out, total.to(F32).to(kind))
    return out


def sms():
    n = torch.cuda.get_device_properties(0).multi_processor_count
    if n != forms.SMS:
        pytest.skip(f"the forms are those of {forms.SMS} SMs, here are {n}")


@pytest.mark.parametrize("fmt", [F.E2M1, F.E4M3])
@pytest.mark.parametrize("columns,way_out,m,n,kblocks,fp32", forms.PAIRS)
def test_pair_forms(fmt, columns, way_out, m, n, kblocks, fp32):
    sms()
    k, kind = forms.elements(fmt == F.E2M1, kblocks), F32 if fp32 else BF
    (a, x), (b, y) = whole(m, k, fmt, m + k), whole(n, k, fmt, n + 3 * k)
    want = x @ y.T
    add = None
    if way_out >= forms.ADD_BF16:
        add = torch.randint(-99, 100, (m, n), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(kind)
    f = F.mx_matmul_plan(a, b, torch.empty(m, n, dtype=kind, device="cuda"), add)
    assert (f.pair, f.columns, f.way_out) == (1, columns, way_out)
    out = check(a, b, want, kind, add)
    if add is not None:                              # out itself is added to
        total = want + out.double()
        F.mx_matmul(a, b, out, add=out)
        assert torch.equal(out, total.to(F32).to(kind))


@pytest.mark.parametrize("fmt", [F.E2M1, F.E4M3])
@pytest.mark.parametrize("columns,splits,few,many,kblocks", forms.SPLITS)
def test_split_forms(fmt, columns, splits, few, many, kblocks):
    sms()
    k = forms.elements(fmt == F.E2M1, kblocks)
    for m, n in ((few, many), (many, few)):
        (a, x), (b, y) = whole(m, k, fmt, m + k), whole(n, k, fmt, n + 3 * k)
        want = x @ y.T
        for kind in (BF, F32):
            f = F.mx_matmul_plan(a, b, torch.empty(m, n, dtype=kind, device="cuda"))
            assert (f.pair, f.columns, f.splits) == (0, columns, splits)
            check(a, b, want, kind)
            check(a, b, want, kind, torch.randint(-99, 100, (m, n), device="cuda").to(kind))
