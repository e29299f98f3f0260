"""mx_act_forward and mx_act_backward over every bf16 z and over every code
under every scale, against 64 bits: within the errors that the header gives."""
import math

import pytest
import torch

from oracle import kv
from tensor_scaling_cast_gb300 import fp8q as F

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
ACTS = [F.MX_ACT_SILU, F.MX_ACT_GELU, F.MX_ACT_GELU_TANH]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("a CUDA GPU is required for the gpu tests")
    from tensor_scaling_cast_gb300 import build
    build.build()
    F.load()
    torch.cuda.set_device(0)


def parts(act, z):
    """In 64 bits f, the two terms of f' and w; z s' is 0 where s or 1 - s is."""
    if act == F.MX_ACT_GELU:
        s = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * s, s, z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi), z * z / 2
    y, dy = z, torch.ones_like(z)
    if act == F.MX_ACT_GELU_TANH:
        c = 2 * math.sqrt(2 / math.pi)
        y, dy = c * (z + 0.044715 * z ** 3), c * (1 + 3 * 0.044715 * z * z)
    s = torch.sigmoid(y)
    t = s * torch.sigmoid(-y)
    return z * s, s, torch.where(t == 0, t, z * t * dy), y.abs()


def check(got, want, size, w, slope, factor, where):
    """Off by (24 + slope w) 2^-24 of size, by what may be 0, and by the rounding to got's type."""
    bound = (24 + slope * w.clamp(max=200)) * 2.0 ** -24 * size + 2.0 ** -118 * factor.abs() \
        + torch.finfo(got.dtype).eps / 2 * want.abs()
    where = where & (want.abs() < torch.finfo(got.dtype).max / 2)
    assert torch.isfinite(got[where]).all() and int(where.sum()) > 1000
    worst = torch.where(where, (got.double() - want).abs() / bound, 0.0)
    at = int(worst.argmax())
    assert float(worst.flatten()[at]) <= 1, f"{float(worst.flatten()[at])} of the bound at {at}"


def factors(shape, kind, seed):
    """Significands of every kind, between 1 and 2."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (1 + torch.rand(shape, generator=g, device="cuda")).to(kind)


def every_z(kind):
    if kind is BF:
        z = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(BF)
    else:                                            # every sign and exponent, and random significands
        g = torch.Generator(device="cuda").manual_seed(9)
        z = torch.randint(-2 ** 31, 2 ** 31, (1 << 20,), generator=g, device="cuda").to(torch.int32).view(F32)
        near = torch.linspace(-100, 100, 1 << 18, device="cuda")
        z = torch.cat([z, near])
    z = torch.where(torch.isfinite(z), z, torch.zeros_like(z))
    return z.view(-1, 64).contiguous()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("kind", [BF, F32])
def test_forward_over_every_z(act, kind):
    z = every_z(kind)
    f, _, _, w = parts(act, z.double())
    everywhere = torch.ones_like(z, dtype=torch.bool)
    h = torch.empty_like(z)
    F.mx_act_forward(act, z, h=h)
    check(h, f, f.abs(), w, 8, torch.ones_like(f), everywhere)
    for seed in range(40):
        u = factors(z.shape, kind, seed)
        F.mx_act_forward(act, z, u, h=h)
        want = f * u.double()
        check(h, want, want.abs(), w, 8, u.double(), everywhere)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("fmt", [F.E4M3, F.E5M2])
@pytest.mark.parametrize("kind", [BF, F32])
@pytest.mark.parametrize("gated", [False, True])
def test_backward_over_every_code_and_scale(act, fmt, kind, gated):
    """h again, dz and du from z as its blocks hold it."""
    m = F.MXMatrix.allocate(256, 256, fmt)
    m.q.copy_(torch.arange(256, dtype=torch.uint8)[None])
    m.e8m0.copy_(torch.arange(256, dtype=torch.uint8)[:, None])
    z = torch.from_numpy(kv.decode(m.q.cpu().numpy(), m.e8m0.cpu().numpy(), fmt)).cuda()
    where = torch.isfinite(z) & (z.abs() < torch.finfo(F32).max / 2)
    z = torch.where(where, z, torch.zeros_like(z))
    f, s, t, w = parts(act, z)
    one = torch.ones_like(z)
    gate = None
    if gated:                                        # 1, 1.125, ... or 1, 1.25, ...
        gate = F.MXMatrix.allocate(256, 256, fmt)
        g = torch.Generator().manual_seed(3)
        top = 8 if fmt == F.E4M3 else 4
        gate.q.copy_((0x38 if fmt == F.E4M3 else 0x3C) + torch.randint(0, top, (256, 256), generator=g, dtype=torch.uint8))
        gate.e8m0.fill_(127)
    u = torch.from_numpy(kv.decode(gate.q.cpu().numpy(), gate.e8m0.cpu().numpy(), fmt)).cuda() if gated else one
    dz, du, h = (torch.empty(256, 256, dtype=kind, device="cuda") for _ in range(3))
    for seed in range(40):
        dh = factors(z.shape, kind, seed)
        F.mx_act_backward(act, m, gate, dh, dz, du if gated else None, h=h)
        g = dh.double()
        check(dz, g * u * (s + t), g * u * (s + t.abs()), w, 17, g * u, where)
        check(h, f * u, (f * u).abs(), w, 8, u, where)
        if gated:
            check(du, g * f, (g * f).abs(), w, 8, g, where)
