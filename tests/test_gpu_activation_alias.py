"""Outputs of mx_act_forward and mx_act_backward on their inputs, as the header
allows: h on z or u, dz or du on dh.  The same bits as apart."""
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


def inputs(rows, cols, kind):
    """z, u as halves of one tensor, dh with a stride of its own."""
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    both = (torch.randn(rows, 2 * cols, generator=g, device="cuda") * 3).to(kind)
    dh = torch.randn(rows, cols + 64, generator=g, device="cuda").to(kind)[:, 32:32 + cols]
    return both[:, :cols], both[:, cols:], dh


def copies(*tensors):
    """With the same strides, inside larger ones."""
    made = []
    for t in tensors:
        wide = torch.full((t.shape[0], t.stride(0)), 7.0, dtype=t.dtype, device="cuda")
        made.append(wide[:, :t.shape[1]])
        made[-1].copy_(t)
    return made


SIZES = [(1, 32), (5, 2080), (700, 1056), (2048, 4096)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("kind", [BF, F32])
@pytest.mark.parametrize("act", [F.MX_ACT_SILU, F.MX_ACT_GELU, F.MX_ACT_GELU_TANH])
def test_h_on_z_or_u(rows, cols, kind, act):
    z, u, _ = inputs(rows, cols, kind)
    new = F.MXMatrix.allocate

    def run(z, u, h, gated=True):
        kept = new(rows, cols), new(rows, cols) if gated else None, new(rows, cols, F.E2M1)
        F.mx_act_forward(act, z, u if gated else None, z_saved=kept[0], u_saved=kept[1], h=h, h_mx=kept[2], rule=F.MX_CEIL)
        return [t for m in kept if m is not None for t in (m.q, m.e8m0)] + [h.clone()]

    for gated in (True, False):
        apart = run(z, u, torch.empty(rows, cols, dtype=kind, device="cuda"), gated)
        for on in ("z", "u") if gated else ("z",):
            z2, u2 = copies(z, u)
            got = run(z2, u2, z2 if on == "z" else u2, gated)
            assert all(torch.equal(a, b) for a, b in zip(got, apart))
            other, held = (u2, u) if on == "z" else (z2, z)
            assert torch.equal(other, held)
            for t in (z2, u2):                       # what lies between the rows
                wide = t._base
                assert (wide[:, cols:] == 7).all()


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("kind", [BF, F32])
@pytest.mark.parametrize("act", [F.MX_ACT_SILU, F.MX_ACT_GELU, F.MX_ACT_GELU_TANH])
def test_dz_or_du_on_dh(rows, cols, kind, act):
    z, u, dh = inputs(rows, cols, kind)
    zs, us = F.MXMatrix.allocate(rows, cols), F.MXMatrix.allocate(rows, cols)
    F.mx_act_forward(act, z, u, z_saved=zs, u_saved=us)
    apart = [torch.empty(rows, cols, dtype=kind, device="cuda") for _ in range(3)]
    F.mx_act_backward(act, zs, us, dh, apart[0], apart[1], h=apart[2])
    for on in (0, 1):
        (grad,) = copies(dh)
        outs = [torch.empty(rows, cols, dtype=kind, device="cuda") for _ in range(3)]
        outs[on] = grad
        F.mx_act_backward(act, zs, us, grad, outs[0], outs[1], h=outs[2])
        assert all(torch.equal(a, b) for a, b in zip(outs, apart))
        assert (grad._base[:, cols:] == 7).all()
    alone, (grad,) = torch.empty(rows, cols, dtype=kind, device="cuda"), copies(dh)
    F.mx_act_backward(act, zs, None, dh, alone)
    F.mx_act_backward(act, zs, None, grad, grad)
    assert torch.equal(alone, grad)
