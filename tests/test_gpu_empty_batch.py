"""A training step of no tokens through the binding: nothing is written, nothing
is refused."""
import pytest
import torch

from tensor_scaling_cast_gb300 import fp8q as F

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("a CUDA GPU is required for the gpu tests")
    from tensor_scaling_cast_gb300 import build
    build.build()
    F.load()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gated", [True, False])
def test_a_step_of_no_tokens(kind, gated):
    ffn, hidden, dev = 128, 64, "cuda"
    both = torch.empty(0, 2 * ffn, dtype=kind, device=dev)
    z, u = both[:, :ffn], both[:, ffn:] if gated else None
    new = F.MXMatrix.allocate
    zs, us, h4 = new(0, ffn), new(0, ffn) if gated else None, new(0, ffn, F.E2M1)
    w4, wt, dy = new(hidden, ffn, F.E2M1), new(ffn, hidden), new(0, hidden, F.E5M2)
    h, dh, dz, du = (torch.empty(0, ffn, dtype=kind, device=dev) for _ in range(4))
    y = torch.empty(0, hidden, dtype=kind, device=dev)
    launches = F.launch_count()
    F.mx_act_forward(F.MX_ACT_SILU, z, u, z_saved=zs, u_saved=us, h=h, h_mx=h4)
    F.mx_act_forward(F.MX_ACT_GELU, z, u, h=h)
    F.mx_matmul(h4, w4, y)
    F.mx_matmul(w4, h4, torch.empty(hidden, 0, dtype=kind, device=dev))
    F.mx_cast_ex(y, F.E5M2, F.MX_CEIL, 0, F.MX_ROWWISE, dy.q, dy.e8m0)
    dyt = new(hidden, 0, F.E5M2)
    F.mx_cast_dual(y, F.E5M2, F.MX_CEIL, 0, dy.q, dy.e8m0, dyt.q, dyt.e8m0)
    F.mx_matmul(dy, wt, dh, add=dh)
    F.mx_act_backward(F.MX_ACT_SILU, zs, us, dh, dz, du if gated else None, h=h)
    F.mx_act_backward(F.MX_ACT_SILU, zs, us, dh, dh, du if gated else None)
    F.mx_decode(h4, h)
    torch.cuda.synchronize()
    assert F.launch_count() == launches
