"""E8M0 rows that start and end anywhere within 32-byte sectors of memory: the
bytes around them, which mx_matmul reads along, do not reach its results."""
import pytest
import torch

from tensor_scaling_cast_gb300 import fp8q as F

pytestmark = pytest.mark.gpu

F32 = torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("a CUDA GPU is required for the gpu tests")
    from tensor_scaling_cast_gb300 import build
    build.build()
    F.load()
    torch.cuda.set_device(0)


def surrounded(rows, blocks, before, pitch, fmt, seed):
    """Whole numbers under scales 1 and 2, from block `before` on of rows of `pitch`
    blocks whose other scales and codes are NaN; and the values."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    at = torch.randint(0, 5, (rows, 32 * blocks), generator=g, device="cuda")
    e = torch.randint(127, 129, (rows, blocks), generator=g, device="cuda")
    codes = (0, 2, 4, 10, 12) if fmt == F.E2M1 else (0, 0x38, 0x40, 0xB8, 0xC0)
    q = torch.tensor(codes, dtype=torch.uint8, device="cuda")[at]
    if fmt == F.E2M1:
        q = q[:, ::2] | q[:, 1::2] << 4
    per = 16 if fmt == F.E2M1 else 32
    wide_q = torch.full((rows, per * pitch), 0x7F, dtype=torch.uint8, device="cuda")
    wide_e = torch.full((rows, pitch), 255, dtype=torch.uint8, device="cuda")
    part_q, part_e = wide_q[:, per * before:per * (before + blocks)], wide_e[:, before:before + blocks]
    part_q.copy_(q), part_e.copy_(e)
    values = torch.tensor((0.0, 1.0, 2.0, -1.0, -2.0), dtype=torch.float64, device="cuda")[at]
    return F.MXMatrix(part_q, part_e, fmt), values * torch.exp2(e.double() - 127).repeat_interleave(32, 1)


@pytest.mark.parametrize("fmt", [F.E2M1, F.E4M3])
@pytest.mark.parametrize("m,n", [(3, 200), (40, 300), (700, 900)])
@pytest.mark.parametrize("blocks", [1, 31, 37, 64])
def test_neighbours_do_not_count(fmt, m, n, blocks):
    for before in (0, 1, 2, 5, 15, 16, 27, 31, 32):
        for pitch in (blocks + before, blocks + before + 1, 32 * ((blocks + before) // 32 + 1)):
            a, x = surrounded(m, blocks, before, pitch, fmt, 1)
            b, y = surrounded(n, blocks, before, pitch + 3, fmt, 2)
            out = torch.full((m, n), float("nan"), dtype=F32, device="cuda")
            F.mx_matmul(a, b, out)
            assert torch.equal(out.double(), x @ y.T), (before, pitch)
