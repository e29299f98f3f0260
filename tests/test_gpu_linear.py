"""Linear layers in MX form on a GPU against plain 64-bit references: 4-bit
casts and decoding bit for bit, products and activations within bounds derived
from their roundings."""
import math

import numpy as np
import pytest
import torch

from canary import Guards
from oracle import kv
from tensor_scaling_cast_gb300 import fp8q as F

pytestmark = pytest.mark.gpu

G = Guards(seed=0x11)
BF, F32 = torch.bfloat16, torch.float32


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


def guarded(rows, cols, fmt):
    """A matrix in guarded arrays."""
    return F.MXMatrix(G.empty((rows, cols // 2 if fmt == F.E2M1 else cols)), G.empty((rows, cols // 32)), fmt)


def same(a, b):
    """Equal values, NaN for NaN, zeros by sign."""
    a, b = np.asarray(a), np.asarray(b)
    return np.array_equal(a, b, equal_nan=True) and np.array_equal(np.signbit(a)[~np.isnan(a)], np.signbit(b)[~np.isnan(b)])


def odd_values(rows, cols, seed, specials=True):
    """Rows of very different sizes, with blocks of zeros, NaN, Inf and subnormals among them."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-30, 30, (rows, 1), generator=g).float())
    if specials:
        flat = x.view(-1, 32)
        for i, v in enumerate((0.0, -0.0, float("inf"), float("nan"), 1e-40, 3e38, -6.0, 2.0 ** -126, 7.0)):
            if 5 * i < flat.shape[0]:
                flat[5 * i, : 3 if v != v or math.isinf(v) else 32] = v
    return x


# ---- 4-bit casts ---------------------------------------------------------------

def clipped(x, e8m0):
    """Elements whose scaled value rounds past 6."""
    e = e8m0.astype(np.float64) - 127
    with np.errstate(invalid="ignore", over="ignore"):
        v = np.abs(x.astype(np.float64)) * np.repeat(np.exp2(-e), 32, axis=-1)
    return int(((v >= 7) & (np.repeat(e8m0, 32, axis=-1) != 255)).sum())


ROWS = [(1, 32, BF), (1, 2048, BF), (3, 96, F32), (37, 160, BF), (1001, 1056, F32), (64, 8192, BF), (513, 32, BF)]


@pytest.mark.parametrize("rows,cols,dtype", ROWS)
@pytest.mark.parametrize("rule,headroom", [(0, 0), (1, 0), (2, 0), (0, 1), (2, 4)])
def test_4_bit_rows_are_exact(rows, cols, dtype, rule, headroom):
    x = odd_values(rows, cols, rows + cols).to(dtype)
    m = guarded(rows, cols, F.E2M1)
    count = G.full((1,), -1, torch.int64)
    F.mx_cast_ex(x.cuda(), F.E2M1, rule, headroom, F.MX_ROWWISE, m.q, m.e8m0, count)
    G.check("after mx_cast_ex")
    code, e8 = kv.encode(x.float().numpy(), kv.E2M1, rule, headroom)
    assert np.array_equal(m.e8m0.cpu().numpy(), e8)
    assert np.array_equal(m.q.cpu().numpy(), kv.pack(code, kv.E2M1))
    assert int(count) == clipped(x.float().numpy(), e8)


DUAL = [(32, 32, BF), (32, 64, F32), (64, 32, BF), (96, 96, BF), (96, 160, F32), (128, 64, BF), (160, 2048, BF),
        (2048, 96, BF), (1024, 1056, F32), (416, 4096, BF), (4128, 32, F32)]


@pytest.mark.parametrize("rows,cols,dtype", DUAL)
@pytest.mark.parametrize("rule,headroom", [(0, 0), (1, 0), (2, 2)])
def test_4_bit_dual_is_exact(rows, cols, dtype, rule, headroom):
    x = odd_values(rows, cols, rows * 3 + cols).to(dtype)
    r, c = guarded(rows, cols, F.E2M1), guarded(cols, rows, F.E2M1)
    counts = G.full((2,), -1, torch.int64)
    F.mx_cast_dual(x.cuda(), F.E2M1, rule, headroom, r.q, r.e8m0, c.q, c.e8m0, counts[:1], counts[1:])
    G.check("after mx_cast_dual")
    for k, (m, v) in enumerate(((r, x.float().numpy()), (c, np.ascontiguousarray(x.float().numpy().T)))):
        code, e8 = kv.encode(v, kv.E2M1, rule, headroom)
        assert np.array_equal(m.e8m0.cpu().numpy(), e8)
        assert np.array_equal(m.q.cpu().numpy(), kv.pack(code, kv.E2M1))
        assert int(counts[k]) == clipped(v, e8)


@pytest.mark.parametrize("fmt", [kv.E2M1, kv.E4M3, kv.E5M2])
@pytest.mark.parametrize("rows,cols,dtype", [(2080, 8320, BF), (4128, 8224, BF), (2592, 8192, BF), (16416, 4160, BF),
                                             (2080, 4128, F32), (8224, 4160, F32)])
@pytest.mark.parametrize("rule,counted", [(0, True), (0, False), (1, True)])
def test_dual_of_every_shape_is_both_row_wise_casts(rows, cols, dtype, fmt, rule, counted):
    """From part of a round of the kernels' grids to several: the same bytes as
    the row-wise casts of x and of its transpose."""
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    x = (x * torch.exp(6 * torch.randn(1, cols, generator=gen, device="cuda"))).to(dtype)
    r, c = guarded(rows, cols, fmt), guarded(cols, rows, fmt)
    counts = G.full((4,), -1, torch.int64)
    F.mx_cast_dual(x, fmt, rule, 0, r.q, r.e8m0, c.q, c.e8m0, *((counts[:1], counts[1:2]) if counted else (None, None)))
    G.check("after mx_cast_dual")
    for k, (m, v) in enumerate(((r, x), (c, x.t().contiguous()))):
        want = F.MXMatrix.allocate(*v.shape, fmt)
        F.mx_cast_ex(v, fmt, rule, 0, F.MX_ROWWISE, want.q, want.e8m0, counts[2 + k:3 + k])
        assert torch.equal(m.e8m0, want.e8m0) and torch.equal(m.q, want.q)
        assert int(counts[k]) == (int(counts[2 + k]) if counted else -1)


@pytest.mark.parametrize("fmt", [kv.E2M1, kv.E4M3])
@pytest.mark.parametrize("rows,cols", [(64, 96), (2080, 4160)])
def test_calls_one_after_the_other_in_a_graph(rows, cols, fmt):
    """An activation, the dual cast of what it wrote (with its counts cleared
    before), decoding of both, and the buffer written anew by the next round:
    replayed with new inputs each gives what the calls by themselves give."""
    z = torch.empty(rows, cols, dtype=BF, device="cuda")
    h = torch.empty_like(z)
    r, c = guarded(rows, cols, fmt), guarded(cols, rows, fmt)
    counts = G.full((2,), -1, torch.int64)
    out, out_t = torch.empty_like(h), torch.empty(cols, rows, dtype=BF, device="cuda")
    twice = torch.empty_like(h)

    def calls(wait=lambda: None):
        for act, dst in ((0, out), (2, twice)):
            F.mx_act_forward(act, z, h=h)
            wait()
            F.mx_cast_dual(h, fmt, 0, 0, r.q, r.e8m0, c.q, c.e8m0, counts[:1], counts[1:])
            wait()
            F.mx_decode(r, dst)
            wait()
        F.mx_decode(c, out_t)
        wait()

    z.normal_()
    calls(torch.cuda.synchronize)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for seed in range(4):
        z.copy_(torch.randn(rows, cols, generator=torch.Generator().manual_seed(seed)) * 8)
        calls(torch.cuda.synchronize)
        want = [t.clone() for t in (out, out_t, twice, counts, r.q, c.q, r.e8m0, c.e8m0)]
        for t in (out, out_t, twice):
            t.zero_()
        counts.fill_(-1)
        graph.replay()
        G.check("after the replay")
        for t, w in zip((out, out_t, twice, counts, r.q, c.q, r.e8m0, c.e8m0), want):
            assert torch.equal(t, w)


def test_4_bit_largest_exponent_under_headroom():
    """E = 127 takes its factor 2^-127 as a subnormal number."""
    x = torch.full((1, 32), 3e38)
    x[0, 3] = -1e38
    m = guarded(1, 32, F.E2M1)
    F.mx_cast_ex(x.cuda(), F.E2M1, 0, 4, F.MX_ROWWISE, m.q, m.e8m0)
    code, e8 = kv.encode(x.numpy(), kv.E2M1, 0, 4)
    assert e8[0, 0] == 254 and np.array_equal(m.e8m0.cpu().numpy(), e8)
    assert np.array_equal(m.q.cpu().numpy(), kv.pack(code, kv.E2M1))


# ---- decode ----------------------------------------------------------------------

@pytest.mark.parametrize("fmt", [kv.E2M1, kv.E4M3, kv.E5M2])
@pytest.mark.parametrize("kind", [BF, F32])
def test_decode_every_byte_and_scale(fmt, kind):
    row = 128 if fmt == kv.E2M1 else 256
    m = guarded(256, 256, fmt)
    m.q.copy_(torch.arange(256, dtype=torch.uint8)[:row].expand(256, row) if fmt != kv.E2M1 else
              torch.arange(256, dtype=torch.uint8).view(2, 128).repeat(128, 1))
    m.e8m0.copy_(torch.arange(256, dtype=torch.uint8)[:, None].expand(256, 8))
    out = G.empty((256, 256), kind)
    F.mx_decode(m, out)
    with np.errstate(over="ignore"):
        want = torch.from_numpy(kv.decode(m.q.cpu().numpy(), m.e8m0.cpu().numpy(), fmt)).float().to(kind).float().numpy()
    assert same(out.float().cpu().numpy(), want)


@pytest.mark.parametrize("rows,cols", [(1, 32), (7, 96), (513, 2080), (129, 8192)])
@pytest.mark.parametrize("fmt", [kv.E2M1, kv.E4M3])
def test_decode_of_slices(rows, cols, fmt):
    """Columns of a wider matrix, into columns of a wider tensor whose other values stay."""
    wide = F.MXMatrix.allocate(rows, cols + 96, fmt)
    wide.q.copy_(torch.randint(0, 100, wide.q.shape, dtype=torch.uint8))
    wide.e8m0.copy_(torch.randint(100, 140, wide.e8m0.shape, dtype=torch.uint8))
    per = 2 if fmt == kv.E2M1 else 1
    m = F.MXMatrix(wide.q[:, 64 // per:(64 + cols) // per], wide.e8m0[:, 2:2 + cols // 32], fmt)
    out = G.full((rows, cols + 64), 5.0, BF)
    F.mx_decode(m, out[:, 32:32 + cols])
    want = kv.decode(m.q.cpu().numpy(), m.e8m0.cpu().numpy(), fmt)
    assert np.array_equal(out[:, 32:32 + cols].float().cpu().numpy(), want.astype(np.float32))
    assert (out[:, :32] == 5).all() and (out[:, 32 + cols:] == 5).all()


def test_more_units_than_31_bits():
    """Past 2^31 units of eight elements: every row of a tall matrix lands in its place."""
    rows, cols = (1 << 29) + 5, 32
    if torch.cuda.mem_get_info()[0] < 70 << 30:
        pytest.skip("70 GB of free memory")
    q = torch.zeros(rows, 16, dtype=torch.uint8, device="cuda")
    e = torch.full((rows, 1), 127, dtype=torch.uint8, device="cuda")
    at = torch.tensor([0, 1, 1 << 20, (1 << 29) - 1, 1 << 29, rows - 1], device="cuda")
    q[at] = torch.arange(1, 7, dtype=torch.uint8, device="cuda")[:, None]
    out = torch.empty(rows, cols, dtype=BF, device="cuda")
    F.mx_decode(F.MXMatrix(q, e, kv.E2M1), out)
    want = torch.from_numpy(kv.decode(q[at].cpu().numpy(), e[at].cpu().numpy(), kv.E2M1)).to(BF)
    assert torch.equal(out[at].cpu(), want)
    assert int(out.view(torch.int32).count_nonzero()) == int(want.view(torch.int32).count_nonzero())


# ---- products --------------------------------------------------------------------

def random_mx(rows, cols, fmt, seed, lo=110, hi=135, wide=0):
    """Codes of finite values (no NaN, no Inf) under random scales; wide: extra columns on both sides of a slice."""
    g = torch.Generator().manual_seed(seed)
    top = {kv.E2M1: 256, kv.E4M3: 0x7F, kv.E5M2: 0x7C}[fmt]
    full = cols + 2 * wide
    q = torch.randint(0, top, (rows, full // 2 if fmt == kv.E2M1 else full), generator=g, dtype=torch.uint8)
    if fmt != kv.E2M1:
        q |= torch.randint(0, 2, q.shape, generator=g, dtype=torch.uint8) << 7
    e = torch.randint(lo, hi, (rows, full // 32), generator=g, dtype=torch.uint8)
    per = 2 if fmt == kv.E2M1 else 1
    q, e = q.cuda(), e.cuda()
    if wide:
        q, e = q[:, wide // per:(wide + cols) // per], e[:, wide // 32:(wide + cols) // 32]
    return F.MXMatrix(q, e, fmt)


def values(m):
    return torch.from_numpy(kv.decode(m.q.cpu().numpy(), m.e8m0.cpu().numpy(), m.fmt)).cuda()


def check_product(a, b, out, add=None):
    """Within the documented roundings: each of the K / 32 additions of partial
    sums may cut 2^-23 of the terms' magnitude, one more for the alignment
    within a partial sum, then the result (and add) is rounded to 24 bits and to
    its type by at most half a step."""
    x, y = values(a), values(b)
    want, size = x @ y.T, x.abs() @ y.abs().T
    if add is not None:
        want, size = want + add.double(), size + add.double().abs()
    steps = a.shape[1] // 32 + 3
    bound = steps * 2.0 ** -23 * size + torch.finfo(out.dtype).eps / 2 * want.abs()
    off = (out.double() - want).abs()
    worst = float((off / bound.clamp(min=1e-300)).max())
    assert worst <= 1, f"{worst} of the bound"


SHAPES = [(1, 1, 32), (1, 8192, 2048), (2, 130, 64), (3, 7, 96), (16, 2048, 8192), (17, 300, 352), (31, 129, 1056),
          (33, 128, 256), (64, 2048, 4096), (65, 257, 512), (128, 128, 128), (129, 4100, 288), (200, 200, 4096),
          (1001, 1055, 2080), (1024, 40, 32), (4097, 3, 160), (300, 9000, 96), (777, 1300, 8224), (2500, 2100, 224), (9000, 5000, 32),
          (5120, 4096, 1024), (4100, 2060, 8224)]
PAIRS = [(kv.E2M1, kv.E2M1), (kv.E4M3, kv.E4M3), (kv.E5M2, kv.E4M3), (kv.E4M3, kv.E5M2), (kv.E5M2, kv.E5M2)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("fmts", PAIRS[:3])
def test_products(m, n, k, fmts):
    a, b = random_mx(m, k, fmts[0], m + k), random_mx(n, k, fmts[1], n + 7 * k)
    for kind in (BF, F32):
        out = G.empty((m, n), kind)
        F.mx_matmul(a, b, out)
        G.check("after mx_matmul")
        check_product(a, b, out)


@pytest.mark.parametrize("fmts", PAIRS)
@pytest.mark.parametrize("m,n,k", [(5, 333, 416), (300, 257, 608), (1300, 1500, 1056), (2100, 2601, 800), (6000, 600, 4640)])
def test_products_of_slices_with_add(m, n, k, fmts):
    """Slices as operands, out and add rows inside wider ones whose other
    values stay; add of its own, and out itself."""
    a, b = random_mx(m, k, fmts[0], m + k, wide=64), random_mx(n, k, fmts[1], n + 7 * k, wide=32)
    for kind in (BF, F32):
        base = torch.randn(m, n + 10, generator=torch.Generator().manual_seed(1)).to(kind).cuda() * 2.0 ** 12
        out = G.full((m, n + 5), 3.0, kind)
        F.mx_matmul(a, b, out[:, 2:2 + n], add=base[:, 7:7 + n])
        check_product(a, b, out[:, 2:2 + n], base[:, 7:7 + n])
        assert (out[:, :2] == 3).all() and (out[:, 2 + n:] == 3).all()
        held = base[:, 7:7 + n].clone()
        F.mx_matmul(a, b, base[:, 7:7 + n], add=base[:, 7:7 + n])
        check_product(a, b, base[:, 7:7 + n], held)


@pytest.mark.parametrize("m,n,k,fmt,kind,with_add", [
    (5120, 4096, 2048, kv.E2M1, BF, False), (2048, 8192, 2048, kv.E4M3, F32, True), (2048, 8192, 2048, kv.E4M3, BF, True),
    (9001, 2048, 512, kv.E2M1, F32, False), (5120, 4096, 2048, kv.E5M2, F32, False), (1000, 2050, 256, kv.E2M1, F32, True),
    (1000, 2048, 4096, kv.E2M1, F32, True), (258, 696, 13408, kv.E2M1, BF, True), (205, 1394, 9984, kv.E4M3, F32, True)])
def test_products_of_every_way_out(m, n, k, fmt, kind, with_add):
    """Tiles of each width, out by TMA and from registers, added to and not, sums
    split over three, five and more CTAs."""
    a, b = random_mx(m, k, fmt, 1), random_mx(n, k, fmt, 2)
    add = torch.randn(m, n, generator=torch.Generator().manual_seed(1)).to(kind).cuda() * 2.0 ** 12 if with_add else None
    out = G.empty((m, n), kind)
    F.mx_matmul(a, b, out, add=add)
    G.check("after mx_matmul")
    check_product(a, b, out, add)


@pytest.mark.parametrize("fmt", [kv.E2M1, kv.E4M3])
@pytest.mark.parametrize("m,n,k", [(1, 200, 1024), (40, 300, 2048), (150, 140, 1024), (600, 1100, 544), (2100, 2300, 1024)])
def test_products_of_whole_numbers_are_exact(fmt, m, n, k):
    """Values 0, +-1, +-2 under scales 1, 2 and 4: every sum is a whole number below 2^24."""
    codes = {kv.E2M1: (0, 2, 4, 10, 12), kv.E4M3: (0, 0x38, 0x40, 0xB8, 0xC0)}[fmt]
    g = torch.Generator().manual_seed(k)
    ms = []
    for rows in (m, n):
        c = torch.tensor(codes, dtype=torch.uint8)[torch.randint(0, 5, (rows, k), generator=g)]
        q = torch.from_numpy(kv.pack(c.numpy(), fmt))
        e = torch.randint(127, 130, (rows, k // 32), generator=g, dtype=torch.uint8)
        ms.append(F.MXMatrix(q.cuda(), e.cuda(), fmt))
    out = G.empty((m, n), F32)
    F.mx_matmul(*ms, out)
    want = values(ms[0]) @ values(ms[1]).T
    assert torch.equal(out.double(), want)


@pytest.mark.parametrize("kind", [BF, F32])
@pytest.mark.parametrize("start", [0, 1, 3, 6])
def test_out_starts_and_ends_anywhere(kind, start):
    """Tiles of the larger kernel whose rows start at any multiple of an element
    and whose last columns are any number: whole numbers up to 2^8, exactly."""
    m, k = 2100, 64
    gen = torch.Generator().manual_seed(start)
    a = torch.randint(-2, 3, (m, k), generator=gen).float()
    b = torch.randint(-1, 2, (1200, k), generator=gen).float()
    a[:, 32:] = 0                                    # at most 64 in magnitude
    am, bm = guarded(m, k, F.E2M1), guarded(1200, k, F.E2M1)
    for x, q in ((a, am), (b, bm)):
        F.mx_cast_ex(x.cuda(), F.E2M1, 0, 0, F.MX_ROWWISE, q.q, q.e8m0)
    want = (a @ b.t()).to(kind).cuda()
    for n in [1024 + c for c in range(1, 41)] + [1119, 1136, 1199]:
        flat = G.empty((m * (n + start) + 16,), kind)
        flat.fill_(-7)
        out = flat[start:start + m * (n + start)].view(m, n + start)[:, :n]
        F.mx_matmul(am, F.MXMatrix(bm.q[:n], bm.e8m0[:n], F.E2M1), out)
        G.check(f"{n} columns")
        assert torch.equal(out, want[:, :n]), n
        assert bool((flat[:start] == -7).all()) and bool((flat[start:start + m * (n + start)].view(m, n + start)[:, n:] == -7).all())
        assert bool((flat[start + m * (n + start):] == -7).all())


def test_one_scale_and_one_element_at_a_time():
    """Each block and each element of K reaches the sum with its own scale: a
    single one is not zero."""
    k = 608
    for fmt, one in ((kv.E2M1, 2), (kv.E4M3, 0x38)):
        c = torch.zeros(k, k, dtype=torch.uint8)
        c.fill_diagonal_(one)
        e = torch.arange(k // 32, dtype=torch.uint8).expand(k, k // 32) + 120
        a = F.MXMatrix(torch.from_numpy(kv.pack(c.numpy(), fmt)).cuda(), e.contiguous().cuda(), fmt)
        b = random_mx(70, k, fmt, 3)
        for x, y in ((a, b), (b, a)):
            out = G.empty((x.shape[0], y.shape[0]), F32)
            F.mx_matmul(x, y, out)
            assert torch.equal(out.double(), values(x) @ values(y).T)


@pytest.mark.parametrize("fmt", [kv.E2M1, kv.E4M3])
@pytest.mark.parametrize("m,n", [(3, 130), (70, 200), (2100, 2300)])
def test_products_over_the_range_of_scales(fmt, m, n):
    """Scales from 2^-126 to 2^127 on one side and their reciprocals on the
    other, block by block; and sums up to 2^120."""
    k = 512
    a, b = random_mx(m, k, fmt, 1), random_mx(n, k, fmt, 2)
    e = torch.randint(1, 254, (k // 32,), generator=torch.Generator().manual_seed(3))
    a.e8m0.copy_(e.to(torch.uint8).expand(m, -1))
    b.e8m0.copy_((254 - e).to(torch.uint8).expand(n, -1))
    out = G.empty((m, n), F32)
    F.mx_matmul(a, b, out)
    check_product(a, b, out)
    a.e8m0.fill_(127 + 50)
    b.e8m0.fill_(127 + 50)
    F.mx_matmul(a, b, out)
    check_product(a, b, out)


def test_products_of_infinities():
    """E5M2's Inf: against positive values Inf, against zeros NaN, in its row alone."""
    a, b = random_mx(5, 64, kv.E5M2, 1), random_mx(200, 64, kv.E5M2, 2)
    a.q[2, 7] = 0x7C
    b.q[:, 7] = 0x3C
    b.q[11, 7] = 0
    out = G.empty((5, 200), F32)
    F.mx_matmul(a, b, out)
    assert out[2, 11].isnan() and (out[2, :11] == math.inf).all() and (out[2, 12:] == math.inf).all()
    assert torch.isfinite(out[[0, 1, 3, 4]]).all()


@pytest.mark.parametrize("m,n", [(3, 200), (300, 500), (1200, 1400), (2300, 2400)])
def test_products_pass_nan_on_to_their_rows_only(m, n):
    a, b = random_mx(m, 256, kv.E4M3, 1), random_mx(n, 256, kv.E4M3, 2)
    a.e8m0[1, 3] = 255
    b.q[17, 40] = 0x7F
    out = G.empty((m, n), BF)
    F.mx_matmul(a, b, out)
    nan = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    nan[1], nan[:, 17] = True, True
    assert torch.equal(out.isnan(), nan)
    a, b = random_mx(m, 256, kv.E2M1, 1), random_mx(n, 256, kv.E2M1, 2)
    b.e8m0[n - 1, 7] = 255
    F.mx_matmul(a, b, out)
    nan.zero_()
    nan[:, n - 1] = True
    assert torch.equal(out.isnan(), nan)


@pytest.mark.parametrize("m,n,k", [(4, 500, 4096), (700, 900, 2048), (2600, 2400, 1024)])
def test_products_repeat_and_replay(m, n, k):
    """The same bits from call to call, on another stream and from a graph whose inputs change."""
    a, b = random_mx(m, k, kv.E2M1, 1), random_mx(n, k, kv.E2M1, 2)
    first, out = G.empty((m, n), F32), G.empty((m, n), F32)
    F.mx_matmul(a, b, first)
    for _ in range(3):
        F.mx_matmul(a, b, out)
        assert torch.equal(first, out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out.zero_()
        F.mx_matmul(a, b, out)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        F.mx_matmul(a, b, out)
        F.mx_matmul(a, b, out, add=out)
    a.q.copy_(random_mx(m, k, kv.E2M1, 5).q)
    graph.replay()
    F.mx_matmul(a, b, first)
    assert torch.equal(out, 2 * first)


def test_two_products_at_once():
    """Calls on two streams share nothing."""
    pairs = [(random_mx(40, 4096, kv.E2M1, s), random_mx(600, 4096, kv.E2M1, s + 9)) for s in (1, 2)]
    outs = [[G.empty((40, 600), F32) for _ in range(8)] for _ in pairs]
    streams = [torch.cuda.Stream() for _ in pairs]
    torch.cuda.synchronize()
    for i in range(8):
        for (a, b), o, s in zip(pairs, outs, streams):
            with torch.cuda.stream(s):
                F.mx_matmul(a, b, o[i])
    torch.cuda.synchronize()
    for (a, b), o in zip(pairs, outs):
        check_product(a, b, o[0])
        assert all(torch.equal(o[0], x) for x in o[1:])


def test_both_kernels_and_attention_at_once():
    """Large and split products, an activation and attention over a cache on four
    streams: they share tensor memory and shared memory of the same SMs, and nothing else."""
    a, b = random_mx(2300, 1024, kv.E4M3, 1), random_mx(2500, 1024, kv.E4M3, 2)
    c, d = random_mx(9, 4096, kv.E2M1, 3), random_mx(2000, 4096, kv.E2M1, 4)
    big, small = G.empty((2300, 2500), BF), G.empty((9, 2000), BF)
    z = torch.randn(500, 2048, device="cuda").bfloat16()
    h, want_h = torch.empty_like(z), torch.empty_like(z)
    cache = F.MXKVCache.allocate(64, 16, 4, 128)
    for t in (cache.k_q, cache.v_q):
        t.copy_(torch.randint(0, 256, t.shape, dtype=torch.uint8))
    cache.k_e8m0.fill_(120), cache.v_e8m0.fill_(120)
    table = torch.arange(64, dtype=torch.int32, device="cuda")[None]
    lens, cu = torch.tensor([1000], dtype=torch.int32, device="cuda"), torch.tensor([0, 300], dtype=torch.int32, device="cuda")
    q = torch.randn(300, 8, 128, device="cuda").bfloat16()
    out, want_out = torch.empty_like(q), torch.empty_like(q)
    ws = F.mx_kv_attention_workspace(cache, q, table, max_q=300)

    def calls(o, hh):
        return (lambda: F.mx_matmul(a, b, big), lambda: F.mx_matmul(c, d, small), lambda: F.mx_act_forward(1, z, h=hh),
                lambda: F.mx_kv_attention(cache, q, o, table, lens, cu_q=cu, max_q=300, workspace=ws))
    for f in calls(want_out, want_h):
        f()
    want = big.clone(), small.clone()
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    for _ in range(20):
        for f, s in zip(calls(out, h), streams):
            with torch.cuda.stream(s):
                f()
    torch.cuda.synchronize()
    assert torch.equal(big, want[0]) and torch.equal(small, want[1]) and torch.equal(h, want_h) and torch.equal(out, want_out)


# ---- activations -------------------------------------------------------------------

def activation64(act, z):
    """f(z), f'(z), and the magnitudes of the terms that f' is a sum of."""
    if act == F.MX_ACT_SILU:
        s = torch.sigmoid(z)
        t = z * s * torch.sigmoid(-z)
        return z * s, s + t, s + t.abs()
    if act == F.MX_ACT_GELU:
        p = 0.5 * torch.erfc(-z / math.sqrt(2))
        t = z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        return z * p, p + t, p + t.abs()
    y, dy = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3), 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z ** 2)
    s = torch.sigmoid(y)
    t = z * s * torch.sigmoid(-y) * dy
    return z * s, s + t, s + t.abs()


def check_close(got, want, terms, z, act, gate):
    """Roundings: the exponent's argument (z, z^2 / 2 or y, some roundings of
    2^-24 each) moves the result by as many times its own size; the exponential,
    the reciprocal and the products add some more.  Values below 2^-118 may be
    flushed with the reciprocal of a number past 2^126."""
    arg = {F.MX_ACT_SILU: z.abs(), F.MX_ACT_GELU: z * z / 2, F.MX_ACT_GELU_TANH: 1.6 * (z.abs() + 0.045 * z.abs() ** 3)}[act]
    bound = (24 + 4 * arg.clamp(max=130)) * 2.0 ** -24 * terms + torch.finfo(got.dtype).eps / 2 * want.abs() \
        + 2.0 ** -118 * gate.abs().clamp(min=1)
    off = (got.double() - want).abs()
    assert torch.isfinite(got).all()
    worst = float((off / bound).max())
    assert worst <= 1, f"{worst} of the bound"


ACTS = [(1, 32), (5, 2080), (37, 96), (130, 1056), (1000, 352), (64, 8192)]


def act_inputs(rows, cols, dtype, gated, seed=0):
    g = torch.Generator().manual_seed(rows * 7 + cols + seed)
    both = torch.randn(rows, 2 * cols if gated else cols, generator=g) * torch.exp2(
        torch.randint(-12, 6, (rows, 1), generator=g).float())
    both = both.clamp(-85, 85).to(dtype).cuda()
    return both[:, :cols], (both[:, cols:] if gated else None), \
        (torch.randn(rows, cols, generator=g) * 1e-3).to(dtype).cuda()


@pytest.mark.parametrize("rows,cols", ACTS)
@pytest.mark.parametrize("act", [0, 1, 2])
@pytest.mark.parametrize("dtype,gated,fmt,rule", [(BF, True, kv.E4M3, 1), (BF, False, kv.E5M2, 0), (F32, True, kv.E5M2, 2),
                                                  (F32, False, kv.E4M3, 1)])
def test_activation_forward_and_backward(rows, cols, act, dtype, gated, fmt, rule):
    z, u, dh = act_inputs(rows, cols, dtype, gated)
    zs, us = guarded(rows, cols, fmt), guarded(rows, cols, fmt) if gated else None
    h = G.full((rows, cols + 32), 9.0, dtype)
    F.mx_act_forward(act, z, u, z_saved=zs, u_saved=us, h=h[:, 16:16 + cols], rule=rule)
    G.check("after mx_act_forward")
    assert (h[:, :16] == 9).all() and (h[:, 16 + cols:] == 9).all()
    for m, x in ((zs, z), (us, u)):
        if m is not None:
            code, e8 = kv.encode(x.float().cpu().numpy(), fmt, rule)
            assert np.array_equal(m.q.cpu().numpy(), code) and np.array_equal(m.e8m0.cpu().numpy(), e8)
    one = torch.ones((), dtype=torch.float64, device="cuda")
    f, _, _ = activation64(act, z.double())
    gate = u.double() if gated else one
    check_close(h[:, 16:16 + cols], f * gate, (f * gate).abs(), z.double(), act, gate)

    dz, du, h2 = (G.empty((rows, cols), dtype) for _ in range(3))
    F.mx_act_backward(act, zs, us, dh, dz, du if gated else None, h=h2)
    G.check("after mx_act_backward")
    z8 = values(zs)
    gate = values(us) if gated else one
    f, d, terms = activation64(act, z8)
    g = dh.double()
    check_close(dz, g * gate * d, (g * gate).abs() * terms, z8, act, g * gate)
    check_close(h2, f * gate, (f * gate).abs(), z8, act, gate)
    if gated:
        check_close(du, g * f, (g * f).abs(), z8, act, g)
    # the same without h, in place on dh
    dz2 = dh.clone()
    F.mx_act_backward(act, zs, us, dz2, dz2, du if gated else None)
    assert torch.equal(dz2, dz)


@pytest.mark.parametrize("act", [0, 1, 2])
def test_gradients_against_differences(act):
    """f' from f at two places, both from the library, in 32 bits."""
    z = torch.linspace(-6, 6, 32 * 64).view(64, 32).cuda()
    m = guarded(64, 32, kv.E4M3)
    F.mx_act_forward(act, z, z_saved=m, rule=1)
    z8 = values(m)
    dz, f = torch.empty_like(z), []
    F.mx_act_backward(act, m, None, torch.ones_like(z), dz)
    step = 2.0 ** -7
    for s in (step, -step):
        h = torch.empty_like(z)
        F.mx_act_forward(act, (z8 + s).float(), h=h)
        f.append(h.double())
    # third derivatives stay below 2, values below 8 and their roundings below 2^-20
    assert float(((f[0] - f[1]) / (2 * step) - dz.double()).abs().max()) < step ** 2 + 2 * 2.0 ** -20 / (2 * step)


@pytest.mark.parametrize("fmt", [kv.E2M1, kv.E4M3, kv.E5M2])
@pytest.mark.parametrize("dtype,gated", [(BF, True), (F32, False)])
@pytest.mark.parametrize("rule", [0, 1, 2])
def test_h_in_blocks(fmt, dtype, gated, rule):
    """h's codes are nearest under their scale, and the scale follows the rule,
    but for values within the activation's own error of a border."""
    rows, cols = 133, 1056
    z, u, _ = act_inputs(rows, cols, dtype, gated, seed=1)
    hm = guarded(rows, cols, fmt)
    F.mx_act_forward(0, z, u, h_mx=hm, rule=rule)
    G.check("after mx_act_forward")
    f, _, _ = activation64(0, z.double())
    h = (f * u.double() if gated else f).cpu().numpy()
    code, e8 = kv.encode(h, fmt, rule)
    got_e = hm.e8m0.cpu().numpy()
    assert (np.abs(got_e.astype(int) - e8) <= 1).all() and (got_e != e8).mean() < 1e-3
    equal = np.repeat(got_e == e8, 32, axis=-1)
    got = kv.unpack(hm.q.cpu().numpy(), fmt)
    # flush of results below 2^-118 moves no code: a block's smallest step is far larger here
    wrong = equal & (got != code)
    assert wrong.mean() < 1e-3
    if wrong.any():
        g = kv.decode(kv.pack(code, fmt), e8, fmt)
        v = kv.decode(hm.q.cpu().numpy(), got_e, fmt)
        mid = (g + v) / 2
        assert (np.abs(h - mid)[wrong] <= (400 * 2.0 ** -24 * np.abs(h))[wrong]).all()


def test_activation_into_slices():
    """z and u kept in the two halves of one matrix, h's blocks within a wider one
    whose other bytes stay."""
    rows, cols = 70, 160
    z, u, dh = act_inputs(rows, cols, BF, True)
    both, wide = guarded(rows, 2 * cols, kv.E4M3), guarded(rows, cols + 128, kv.E2M1)
    before = wide.q.clone(), wide.e8m0.clone()
    zs, us = (F.MXMatrix(both.q[:, i * cols:(i + 1) * cols], both.e8m0[:, i * 5:(i + 1) * 5], kv.E4M3) for i in (0, 1))
    hm = F.MXMatrix(wide.q[:, 32:32 + cols // 2], wide.e8m0[:, 2:7], kv.E2M1)
    F.mx_act_forward(0, z, u, z_saved=zs, u_saved=us, h_mx=hm, rule=1)
    G.check("after mx_act_forward")
    alone = F.MXMatrix.allocate(rows, cols, kv.E2M1)
    F.mx_act_forward(0, z, u, h_mx=alone, rule=1)
    assert torch.equal(hm.q, alone.q) and torch.equal(hm.e8m0, alone.e8m0)
    hm.q.copy_(before[0][:, 32:32 + cols // 2]), hm.e8m0.copy_(before[1][:, 2:7])
    assert torch.equal(wide.q, before[0]) and torch.equal(wide.e8m0, before[1])
    for m, x in ((zs, z), (us, u)):
        code, e8 = kv.encode(x.float().cpu().numpy(), kv.E4M3, 1)
        assert np.array_equal(m.q.cpu().numpy(), code) and np.array_equal(m.e8m0.cpu().numpy(), e8)
    dz, du = G.empty((rows, cols), BF), G.empty((rows, cols), BF)
    F.mx_act_backward(0, zs, us, dh, dz, du)
    f, d, terms = activation64(0, values(zs))
    g, gate = dh.double(), values(us)
    check_close(dz, g * gate * d, (g * gate).abs() * terms, values(zs), 0, g * gate)
    check_close(du, g * f, (g * f).abs(), values(zs), 0, g)


def test_activation_of_nan_and_inf():
    z = torch.randn(4, 64, device="cuda").bfloat16()
    u = torch.randn(4, 64, device="cuda").bfloat16()
    z[0, 3], z[1, 40], u[2, 5] = float("nan"), float("inf"), float("-inf")
    zs, us, hm = guarded(4, 64, kv.E4M3), guarded(4, 64, kv.E4M3), guarded(4, 64, kv.E2M1)
    h, dz, du = (G.empty((4, 64), BF) for _ in range(3))
    F.mx_act_forward(0, z, u, z_saved=zs, u_saved=us, h=h, h_mx=hm)
    bad = torch.zeros(4, 64, dtype=torch.bool, device="cuda")
    bad[0, 3] = bad[1, 40] = bad[2, 5] = True
    assert torch.equal(~torch.isfinite(h), bad)
    blocks = bad.view(4, 2, 32).any(-1)
    assert torch.equal(hm.e8m0 == 255, blocks)
    F.mx_act_backward(0, zs, us, torch.ones_like(z), dz, du)
    zbad = torch.zeros(4, 2, dtype=torch.bool, device="cuda")
    zbad[0, 0] = zbad[1, 1] = True
    assert torch.equal(du.isnan(), zbad.repeat_interleave(32, 1))
    zbad[2, 0] = True
    assert torch.equal(dz.isnan(), zbad.repeat_interleave(32, 1))


@pytest.mark.parametrize("act", [0, 1, 2])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_activation_far_out(act, dtype):
    """Where f is z or 0: values and derivatives stay finite up to the type's largest."""
    z = torch.tensor([300.0, -300.0, 1e6, -1e6, 1e18, -1e18, 1e25, -1e25, 2e38, -2e38, 0.0, -0.0] + [0.0] * 20)
    z = z.repeat_interleave(32).view(-1, 32).to(dtype).cuda()
    m = guarded(*z.shape, kv.E5M2)
    h, dz = G.empty(z.shape, dtype), G.empty(z.shape, dtype)
    F.mx_act_forward(act, z, z_saved=m, h=h, rule=1)
    assert torch.equal(h, torch.where(z > 0, z, torch.zeros_like(z)))
    F.mx_act_backward(act, m, None, torch.ones_like(z), dz)
    want = torch.where(z > 0, 1.0, torch.where(z < 0, 0.0, 0.5)).to(dtype)
    assert torch.equal(dz, want)


# ---- together ------------------------------------------------------------------------

@pytest.mark.parametrize("tokens,ffn,hidden,gated,h_fmt", [(96, 416, 160, True, kv.E4M3), (32, 1056, 288, False, kv.E2M1),
                                                           (544, 2048, 512, True, kv.E2M1)])
def test_half_an_mlp_step(tokens, ffn, hidden, gated, h_fmt):
    """Forward and backward of h = f(z) u, y = h w^T from z and u to the
    gradients of z, u and w, as a training step runs them (captured and replayed
    too); each product and activation against 64 bits from what the step before
    it left."""
    z, u, _ = act_inputs(tokens, ffn, BF, gated)
    g = torch.Generator().manual_seed(4)
    w = (torch.randn(hidden, ffn, generator=g) * 0.02).bfloat16().cuda()
    dy = (torch.randn(tokens, hidden, generator=g) * 1e-3).bfloat16().cuda()
    new = F.MXMatrix.allocate
    w_mx, h_mx = new(hidden, ffn, h_fmt), new(tokens, ffn, h_fmt)
    w8, wt = new(hidden, ffn, kv.E4M3), new(ffn, hidden, kv.E4M3)
    zs, us = new(tokens, ffn, kv.E4M3), new(tokens, ffn, kv.E4M3) if gated else None
    dy_mx, dyt, h8, ht = new(tokens, hidden, kv.E5M2), new(hidden, tokens, kv.E5M2), new(tokens, ffn, kv.E4M3), \
        new(ffn, tokens, kv.E4M3)
    y, dh, h = G.empty((tokens, hidden), BF), G.empty((tokens, ffn), BF), G.empty((tokens, ffn), BF)
    dz, du, dw = G.empty((tokens, ffn), BF), G.empty((tokens, ffn), BF), G.full((hidden, ffn), 0.0, F32)

    def step():
        F.mx_cast_ex(w, h_fmt, 1, 0, F.MX_ROWWISE, w_mx.q, w_mx.e8m0)
        F.mx_cast_dual(w, kv.E4M3, 1, 0, w8.q, w8.e8m0, wt.q, wt.e8m0)
        F.mx_act_forward(0, z, u, z_saved=zs, u_saved=us, h_mx=h_mx, rule=1)
        F.mx_matmul(h_mx, w_mx, y)
        F.mx_cast_dual(dy, kv.E5M2, 1, 0, dy_mx.q, dy_mx.e8m0, dyt.q, dyt.e8m0)
        F.mx_matmul(dy_mx, wt, dh)
        F.mx_act_backward(0, zs, us, dh, dz, du if gated else None, h=h)
        F.mx_cast_dual(h, kv.E4M3, 1, 0, h8.q, h8.e8m0, ht.q, ht.e8m0)
        F.mx_matmul(dyt, ht, dw, add=dw)

    step()
    G.check("after the step")
    check_product(h_mx, w_mx, y)
    check_product(dy_mx, wt, dh)
    check_product(dyt, ht, dw)
    z8, gate = values(zs), values(us) if gated else torch.ones((), dtype=torch.float64, device="cuda")
    f, d, terms = activation64(0, z8)
    check_close(dz, dh.double() * gate * d, (dh.double() * gate).abs() * terms, z8, 0, dh.double() * gate)
    # the whole against the layer in 64 bits without any cast: E4M3 and E5M2 keep
    # values to 2^-4 and 2^-3, E2M1 to 2^-2, of a block's largest at worst
    f, d, _ = activation64(0, z.double())
    hh = f * u.double() if gated else f
    keep = {kv.E4M3: 2.0 ** -4, kv.E2M1: 2.0 ** -2}[h_fmt]
    for got, want, most in ((y, hh @ w.double().T, 2 * keep), (dw, dy.double().T @ hh, 2.0 ** -3 + 2 * 2.0 ** -4)):
        assert float((got.double() - want).norm() / want.norm()) < most
    kept = [t.clone() for t in (y, dh, dz, du, dw)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (y, dh, dz, du, dw):
        t.zero_()
    graph.replay()
    for t, k in zip((y, dh, dz, du, dw), kept):
        if t is not du or gated:
            assert torch.equal(t, k)


def test_the_example_runs_and_its_gradients_are_near():
    """Against the step in 32 bits without casts: what the formats keep of a
    block's largest element (E2M1 2^-2, E4M3 2^-4, E5M2 2^-3), for two operands."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mx_mlp_step.py")
    spec = importlib.util.spec_from_file_location("mx_mlp_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    off = m.main(tokens=160, ffn=576, hidden=224, quiet=True)
    assert off["y"] < 2 * 2.0 ** -2
    assert all(off[k] < 2.0 ** -3 + 3 * 2.0 ** -4 for k in ("dz", "du", "dw"))


def test_tensors_of_a_call_are_on_the_current_gpu():
    m = F.MXMatrix.allocate(8, 64, F.E4M3)
    cpu = F.MXMatrix.allocate(8, 64, F.E4M3, device="cpu")
    x = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(8, 8, device="cuda")
    with pytest.raises(TypeError, match="cpu"):
        F.MXMatrix(m.q, cpu.e8m0, F.E4M3)
    for call in (lambda: F.mx_decode(m, x.cpu()), lambda: F.mx_decode(cpu, x), lambda: F.mx_matmul(m, m, out.cpu()),
                 lambda: F.mx_matmul(m, cpu, out), lambda: F.mx_matmul(m, m, out, add=out.cpu()),
                 lambda: F.mx_act_forward(0, x, h=x.cpu()), lambda: F.mx_act_forward(0, x, x.cpu(), h=x),
                 lambda: F.mx_act_forward(0, x, z_saved=cpu), lambda: F.mx_act_forward(0, x, h_mx=cpu),
                 lambda: F.mx_act_backward(0, m, None, x, x.cpu()), lambda: F.mx_act_backward(0, m, cpu, x, x, x),
                 lambda: F.mx_act_backward(0, cpu, None, x, x)):
        with pytest.raises(TypeError, match="cpu"):
            call()
