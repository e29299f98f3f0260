"""Products of both kernels, an activation and attention over a cache at once, on
streams of their own: every call writes an output of its own, whole, with the
bits that it has by itself."""
import pytest
import torch

from canary import Guards
from tensor_scaling_cast_gb300 import fp8q as F

pytestmark = pytest.mark.gpu

G = Guards(seed=0x31)
BF, F32 = torch.bfloat16, torch.float32
ROUNDS = 10


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
    """0, +-1, +-2 under the scale 1, and the values: sums are exact."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    at = torch.randint(0, 5, (rows, cols), generator=g, device="cuda")
    codes = (0, 2, 4, 10, 12) if fmt == F.E2M1 else (0, 0x38, 0x40, 0xB8, 0xC0)
    q = torch.tensor(codes, dtype=torch.uint8, device="cuda")[at]
    if fmt == F.E2M1:
        q = q[:, ::2] | q[:, 1::2] << 4
    e = torch.full((rows, cols // 32), 127, dtype=torch.uint8, device="cuda")
    return F.MXMatrix(q.contiguous(), e, fmt), torch.tensor((0.0, 1.0, 2.0, -1.0, -2.0), device="cuda", dtype=torch.float64)[at]


def product(m, n, k, fmt, kind, seed, form, with_add=False):
    """(call(out), the values that it writes)."""
    (a, x), (b, y) = whole(m, k, fmt, seed), whole(n, k, fmt, seed + 1)
    want = x @ y.T
    add = None
    if with_add:
        add = torch.randint(-99, 100, (m, n), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(kind)
        want = want + add.double()
    f = F.mx_matmul_plan(a, b, torch.empty(m, n, dtype=kind, device="cuda"), add)
    assert (f.pair, f.columns) == form
    return lambda out: F.mx_matmul(a, b, out, add=add), want.to(F32).to(kind)


def activation():
    z = torch.randn(500, 2048, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda").bfloat16()
    want = torch.empty_like(z)
    F.mx_act_forward(F.MX_ACT_GELU, z, h=want)
    return lambda out: F.mx_act_forward(F.MX_ACT_GELU, z, h=out), want


def attention():
    g = torch.Generator(device="cuda").manual_seed(6)
    cache = F.MXKVCache.allocate(64, 16, 4, 128)
    for t in (cache.k_q, cache.v_q):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, device="cuda"))
    cache.k_e8m0.fill_(120), cache.v_e8m0.fill_(120)
    table = torch.arange(64, dtype=torch.int32, device="cuda")[None]
    lens, cu = torch.tensor([1000], dtype=torch.int32, device="cuda"), torch.tensor([0, 300], dtype=torch.int32, device="cuda")
    q = torch.randn(300, 8, 128, generator=g, device="cuda").bfloat16()
    ws = F.mx_kv_attention_workspace(cache, q, table, max_q=300)
    want = torch.empty_like(q)

    def call(out):
        F.mx_kv_attention(cache, q, out, table, lens, cu_q=cu, max_q=300, workspace=ws)
    call(want)
    return call, want


def test_everything_at_once():
    jobs = [product(5700, 2048, 512, F.E4M3, BF, 1, (1, 256)), product(5700, 2048, 1536, F.E2M1, F32, 3, (1, 256)),
            product(5700, 2048, 1024, F.E2M1, F32, 5, (1, 256), True), product(2600, 3001, 128, F.E4M3, F32, 7, (1, 224), True),
            product(9, 2000, 4096, F.E2M1, BF, 9, (0, 16)), product(40, 300, 4352, F.E2M1, F32, 11, (0, 64)),
            product(20, 900, 2048, F.E4M3, BF, 13, (0, 32)), activation(), attention()]
    outs = [[G.full(tuple(want.shape), float("nan"), want.dtype) for _ in range(ROUNDS)] for _, want in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for i in range(ROUNDS):
        # another job first each time
        for j in [(i + k) % len(jobs) for k in range(len(jobs))]:
            with torch.cuda.stream(streams[j]):
                jobs[j][0](outs[j][i])
    torch.cuda.synchronize()
    G.check("after the calls")
    for j, (_, want) in enumerate(jobs):
        for i in range(ROUNDS):
            assert torch.equal(outs[j][i], want), (j, i)


def test_a_replayed_graph_beside_calls():
    """Branches of one graph, replayed while the same products are called on another stream."""
    jobs = [product(5700, 2048, 512, F.E4M3, BF, 1, (1, 256)), product(9, 2000, 4096, F.E2M1, BF, 9, (0, 16)),
            product(5700, 2048, 1024, F.E2M1, F32, 5, (1, 256), True)]
    inside = [G.full(tuple(want.shape), float("nan"), want.dtype) for _, want in jobs]
    beside = [[G.full(tuple(want.shape), float("nan"), want.dtype) for _ in range(ROUNDS)] for _, want in jobs]
    for (call, _), out in zip(jobs, inside):
        call(out)
    torch.cuda.synchronize()
    graph, branches = torch.cuda.CUDAGraph(), [torch.cuda.Stream() for _ in jobs]
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        for s, (call, _), out in zip(branches, jobs, inside):
            s.wait_stream(here)
            with torch.cuda.stream(s):
                call(out)
            here.wait_stream(s)
    side = torch.cuda.Stream()
    for i in range(ROUNDS):
        for out in inside:
            out.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            for (call, _), out in zip(jobs, beside):
                call(out[i])
        torch.cuda.synchronize()
        for (_, want), out, b in zip(jobs, inside, beside):
            assert torch.equal(out, want) and torch.equal(b[i], want), i
