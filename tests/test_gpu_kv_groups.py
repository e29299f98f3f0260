"""Attention over the 4-bit cache where neighbouring groups of 32 tokens have
different scales, and where a CTA goes from one (sequence, head) to the next:
every row and column against the formula in 64 bits, within a bound per column
that follows from the kernels' roundings."""
import numpy as np
import pytest
import torch

from canary import Guards
from tensor_scaling_cast_gb300 import fp8q as F

pytestmark = pytest.mark.gpu

G = Guards(seed=0x47)
GROUP = 32                                # tokens whose largest value scale is R
MIN_R, MAX_R = -80, 126                   # where R is held


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


def values(codes, e8):
    """E2M1 codes [.., D / 2] and E8M0 bytes [.., D / 32] -> 64-bit values."""
    one = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=codes.device)
    table = torch.cat([one, -one])
    v = torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], -1).flatten(-2)
    scale = torch.exp2(e8.double() - 127).masked_fill(e8 == 255, torch.nan)
    return v * scale.repeat_interleave(32, -1)


class Batch:
    """Sequences of random codes in the pages of one cache.  Scales are 2^(a
    whole number up to `apart` either way) per sequence, head and group of 32
    tokens, times 2^(up to 1 either way) per block, and the values' x-th block
    times 2^v_blocks[x]; everything that belongs to no sequence holds 0xFF bytes."""

    def __init__(self, lens, heads, dim, page, seed, k_apart=1, v_apart=6, v_blocks=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.heads, self.dim, self.page = lens, heads, dim, page
        per = [-(-n // page) for n in lens]
        pages, width = sum(per) + 2, max(1, max(per))
        shape, scales = (pages, heads, page, dim // 2), (pages, heads, page, dim // 32)
        arrays = [torch.full(s, 255, dtype=torch.uint8, device="cuda") for s in (shape, scales, shape, scales)]
        order = torch.randperm(pages, generator=g, device="cuda").int()
        self.table = torch.full((len(lens), width), -7, dtype=torch.int32, device="cuda")
        self.rows, at = [], 0
        for b, n in enumerate(lens):
            self.table[b, :per[b]] = order[at:at + per[b]]
            at += per[b]
            one = []
            for a, apart in enumerate((k_apart, v_apart)):
                codes = torch.randint(0, 256, (n, heads, dim // 2), generator=g, device="cuda", dtype=torch.uint8)
                e8 = torch.randint(-1, 2, (n, heads, dim // 32), generator=g, device="cuda") + 127 - 2
                if a and v_blocks:
                    e8 += torch.tensor(v_blocks, device="cuda")
                shift = torch.randint(-apart, apart + 1, (-(-n // GROUP), heads, 1), generator=g, device="cuda")
                one += [codes, (e8 + shift.repeat_interleave(GROUP, 0)[:n]).to(torch.uint8)]
            self.rows.append(one)
        self.arrays, self.pages = arrays, pages
        self.lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.hidden = [torch.zeros(n, dtype=torch.bool, device="cuda") for n in lens]
        self.gen = g
        self.store()

    def store(self):
        """Bring the arrays in line with `rows`."""
        for b, n in enumerate(self.lens):
            t = torch.arange(n, device="cuda")
            page = self.table[b, t // self.page].long() if n else t
            for array, x in zip(self.arrays, self.rows[b]):
                array[page, :, t % self.page] = x

    def hide(self, b, p):
        """Send page p of sequence b out of the cache (once stored)."""
        self.table[b, p] = (-1, self.pages, 2 ** 31 - 1)[b % 3]
        self.hidden[b][p * self.page:(p + 1) * self.page] = True

    def attend(self, q, nqs, window=0, lse=None, scale=None):
        cache = F.MXKVCache(*self.arrays, fmt=F.E2M1)
        cu = torch.tensor(np.concatenate([[0], np.cumsum(nqs)]), dtype=torch.int32, device="cuda")
        out = G.empty(q.shape, torch.bfloat16)
        ws = F.mx_kv_attention_workspace(cache, q, self.table, max_q=max(nqs))
        F.mx_kv_attention(cache, q, out, self.table, self.lens_t, cu_q=cu, max_q=max(nqs), window=window, lse=lse,
                          scale=scale, workspace=ws)
        return out

    def check(self, nqs, group, window=0, q=None, scale=None):
        dim, total, scale = self.dim, sum(nqs), self.dim ** -0.5 if scale is None else scale
        if q is None:
            q = torch.randn(total, self.heads * group, dim, generator=self.gen, device="cuda").bfloat16()
        lse = G.full((total, self.heads * group), 77.0, torch.float32)
        out = self.attend(q, nqs, window, lse, scale)
        again = self.attend(q, nqs, window, scale=scale)
        assert torch.equal(out.view(torch.int16), again.view(torch.int16))
        at = 0
        for b, n in enumerate(nqs):
            rows, at = slice(at, at + n), at + n
            if not n:
                continue
            kc, ke, vc, ve = self.rows[b]
            for h in range(self.heads):
                heads = slice(h * group, (h + 1) * group)
                self._check_head(out[rows, heads].double(), lse[rows, heads].double(), q[rows, heads].double(),
                                 values(kc[:, h], ke[:, h]), vc[:, h], ve[:, h], self.hidden[b], window, scale, (b, h))

    def _check_head(self, got, got_lse, q, k, v_codes, v_e8, hidden, window, scale, where):
        n, length = q.shape[0], k.shape[0]
        v = values(v_codes, v_e8)
        nan = v.isnan()
        v = v.nan_to_num(0.0)
        key = torch.arange(length, device="cuda")
        pos = torch.arange(length - n, length, device="cuda")[:, None]
        seen = (key <= pos) & ~hidden
        if window:
            seen &= key > pos - window
        seen = seen[:, None].expand(n, q.shape[1], length)
        s = (q @ k.T) * scale
        s = s.masked_fill(~seen, -torch.inf)
        none = ~seen.any(-1, keepdim=True)
        zero = torch.zeros(*q.shape[:2], 1, dtype=torch.float64, device="cuda")
        top = s.amax(-1, keepdim=True).masked_fill(none, 0.0) if length else zero
        p = torch.exp(s - top)
        total = p.sum(-1, keepdim=True).masked_fill(none, 1.0)
        want = p @ v / total
        size = p @ v.abs() / total
        # The bound.  The output's rounding: half a bf16 step, up to 2^-8.  Weights: 11 bits, 2^-11 of their
        # share.  Scores: D products summed by the tensor cores in steps of 16 (at most 8 of them, each off by 2^-23
        # of sum |q k|), so 2^-20 of it in a weight, doubled for the scaling around them; sums over keys: 2^-23
        # for every 16 keys.  A weight times 2^R is held in f16 next to the row's largest such product, so that
        # below 2^-14 of that it is off by up to 2^-25 of it.
        r = v_e8.double().masked_fill((v_e8 == 255) | hidden[:, None], 0).amax(-1) - 127
        r = torch.nn.functional.pad(r, (0, -length % GROUP), value=-127.0).view(-1, GROUP).amax(-1)
        r = r.clamp(MIN_R, MAX_R).repeat_interleave(GROUP)[:length]
        most = (q.abs() @ k.abs().T * scale).masked_fill(~seen, 0.0).amax(-1, keepdim=True) if length else zero
        largest = (p * torch.exp2(r)).amax(-1, keepdim=True) if length else zero
        lost = 2 ** -25 * largest * (seen.double() @ (v.abs() * torch.exp2(-r)[:, None])) / total
        tol = 2 ** -8 * 1.01 * want.abs() + (2 ** -11 + 2 ** -19 * most + 2 ** -27 * length) * size + 1.01 * lost
        spoilt = (seen.double() @ nan.double()) > 0
        assert torch.equal(got.isnan(), spoilt), where
        bad = ((got - want).abs() > tol) & ~spoilt
        assert not bad.any(), (where, bad.sum().item(), bad.nonzero()[:4].tolist(), got[bad][:4], want[bad][:4], tol[bad][:4])
        want_lse = (top + torch.log(total)).masked_fill(none, -torch.inf)[..., 0]
        assert torch.equal(got_lse.isinf(), want_lse.isinf()), where
        off = (got_lse - want_lse).abs().nan_to_num(0.0)
        assert (off <= (2 ** -19 * most + 2 ** -16)[..., 0] + 2 ** -22 * want_lse.abs().nan_to_num(posinf=0.0)).all(), where


# ---- prompt chunks: row counts that leave 1 to 128 modulo 256, so that half of
# the prompt kernel has no rows in some item, and many such items per CTA

CHUNKS = [  # lens, queries, kv_heads, group, head_dim, page
    ([2560] * 32, [80] * 32, 8, 4, 128, 64),
    ([2048] * 16, [300] * 16, 8, 1, 128, 16),
    ([1056] * 8, [1056] * 8, 8, 4, 64, 32),
    ([4096, 2742, 1300, 33], [4096, 2742, 1300, 33], 8, 2, 64, 64),
]


@pytest.mark.parametrize("lens,nqs,heads,group,dim,page", CHUNKS)
def test_chunks_with_a_remainder_of_rows(lens, nqs, heads, group, dim, page):
    Batch(lens, heads, dim, page, seed=sum(nqs)).check(nqs, group)


@pytest.mark.parametrize("lens,nqs,heads,group,dim,page", CHUNKS[:2])
def test_chunks_with_a_remainder_of_rows_and_a_hidden_first_page(lens, nqs, heads, group, dim, page):
    batch = Batch(lens, heads, dim, page, seed=1 + sum(nqs))
    for b in range(1, len(lens), 2):
        batch.hide(b, 0)
    batch.check(nqs, group)


@pytest.mark.parametrize("lens,nqs,heads,group,dim,page", CHUNKS[:2])
def test_chunks_with_a_remainder_of_rows_and_nan_among_the_first_keys(lens, nqs, heads, group, dim, page):
    batch = Batch(lens, heads, dim, page, seed=2 + sum(nqs))
    for b in range(len(lens)):
        for h in range(heads):
            if (b + h) % 3 == 0:                   # one block of values
                batch.rows[b][3][7 * b % 128, h, h % (dim // 32)] = 255
    batch.store()
    batch.check(nqs, group)


# ---- blocks of values far smaller than the others of their tokens, under
# weights of which a few are thousands of times the rest

@pytest.mark.parametrize("rows", [8, 16, 24, 32, 100])
@pytest.mark.parametrize("dim,blocks", [(128, (0, -10, -14, -4)), (64, (-12, 0))])
def test_small_value_blocks_keep_their_bits(rows, dim, blocks):
    nq = rows // 4
    batch = Batch([8192, 1000, 33], 2, dim, 16, seed=rows, v_apart=1, v_blocks=blocks)
    batch.check([nq] * 3, 4, scale=4 * dim ** -0.5)


# ---- few query rows: batches of more (sequence, head)s than CTAs, so that a
# CTA ends one, joins it and goes on to the next, whole ones and parts in turn

@pytest.mark.parametrize("rows", [3, 8, 16, 24, 32])
@pytest.mark.parametrize("dim,page", [(128, 64), (64, 16)])
def test_many_sequences_and_heads_of_few_rows(rows, dim, page):
    group, nq = (3, 1) if rows == 3 else (8, rows // 8)
    batch = Batch([1 + 37 * i % 2000 for i in range(64)], 8, dim, page, seed=rows + dim)
    batch.check([nq] * 64, group)


@pytest.mark.parametrize("nq", [1, 2, 3, 4])
def test_many_short_sequences_some_without_keys_or_queries(nq):
    lens = [53 * i % 230 for i in range(300)]
    batch = Batch(lens, 6, 128, 32, seed=nq)
    batch.hide(4, 0)
    batch.check([nq if i % 6 else 0 for i in range(300)], 8)
    batch.check([nq if i % 5 else 1 for i in range(300)], 8, window=70)


# ---- the workspace's tickets

@pytest.mark.parametrize("nq", [1, 5, 70])
def test_a_part_that_was_given_up_does_not_outlive_the_call(nq):
    """Tickets as a CTA that gave up leaves them: with its mark.  Rows joined
    over one stay unwritten, and the next call finds the tickets zero."""
    batch = Batch([6000, 5000, 40], 2, 128, 16, seed=nq)
    cache = F.MXKVCache(*batch.arrays, fmt=F.E2M1)
    q = torch.randn(3 * nq, 8, 128, generator=batch.gen, device="cuda").bfloat16()
    cu = torch.arange(4, dtype=torch.int32, device="cuda") * nq
    ws = F.mx_kv_attention_workspace(cache, q, batch.table, max_q=nq)
    tickets = ws[:F.WORKSPACE_ZEROED].view(torch.int32)

    def call():
        out = G.full(q.shape, 77.0, torch.bfloat16)
        F.mx_kv_attention(cache, q, out, batch.table, batch.lens_t, cu_q=cu, max_q=nq, workspace=ws)
        return out
    want = call()
    assert (tickets == 0).all() and not (want == 77).any()
    tickets.fill_(1 << 16)
    marked = call()
    left = (marked == 77).all(-1)
    assert left.any() and torch.equal(marked[~left], want[~left])
    assert (tickets == 0).any()
    assert ((tickets == 0) | (tickets == 1 << 16)).all()
    assert torch.equal(call(), want)
    tickets.zero_()
    batch.check([nq] * 3, 4, q=q)


# ---- slots from the kernel just before

def test_slots_written_just_before_the_call():
    """Each step's slots come from a kernel queued right before its write and
    read, into the array that the step before used."""
    tokens, heads, dim, page, steps = 700, 2, 64, 16, 40
    cache = F.MXKVCache.allocate(64, page, heads, dim, fmt=F.E4M3)
    g = torch.Generator(device="cuda").manual_seed(3)
    orders = torch.stack([torch.randperm(64 * page, generator=g, device="cuda")[:tokens] for _ in range(steps)])
    x = torch.randint(-8, 9, (steps, tokens, heads, dim), generator=g, device="cuda").float()      # exact in E4M3
    slots = torch.zeros(tokens, dtype=torch.int64, device="cuda")
    k, v = G.empty((steps, tokens, heads, dim), torch.float32), G.empty((steps, tokens, heads, dim), torch.float32)
    for i in range(steps):
        torch.add(orders[i], 0, out=slots)
        F.mx_kv_write(cache, x[i], -x[i], slots)
        F.mx_kv_read(cache, slots, k[i], v[i])
    assert torch.equal(k, x) and torch.equal(v, -x)


# ---- bounds left out

@pytest.mark.parametrize("nqs", [[1, 1], [2, 0], [9, 3], [150, 70]])
def test_workspace_and_call_without_a_bound(nqs):
    batch = Batch([9000, 300], 2, 128, 16, seed=sum(nqs))
    cache = F.MXKVCache(*batch.arrays, fmt=F.E2M1)
    q = torch.randn(sum(nqs), 8, 128, generator=batch.gen, device="cuda").bfloat16()
    cu = torch.tensor([0, nqs[0], sum(nqs)], dtype=torch.int32, device="cuda")
    out = G.empty(q.shape, torch.bfloat16)
    ws = F.mx_kv_attention_workspace(cache, q, batch.table)
    F.mx_kv_attention(cache, q, out, batch.table, batch.lens_t, cu_q=cu, workspace=ws)
    bounded = G.empty(q.shape, torch.bfloat16)
    F.mx_kv_attention(cache, q, bounded, batch.table, batch.lens_t, cu_q=cu, max_q=max(nqs), workspace=ws)
    batch.check(nqs, 4, q=q)
    # both are right to a rounding or two of bf16
    assert (out.float() - bounded.float()).abs().max() <= 2 ** -6 * bounded.float().abs().max()


# ---- what the documented roundings and ranges say

@pytest.mark.parametrize("rows", [4, 20, 280])
@pytest.mark.parametrize("dim", [64, 128])
def test_one_block_of_large_values_costs_the_other_columns_no_more_than_documented(rows, dim):
    batch = Batch([3000, 700], 2, dim, 16, seed=rows, v_apart=1)
    batch.rows[0][3][1234, :, 1] += 20
    batch.rows[1][3][5, 0, 0] += 24
    batch.store()
    batch.check([rows // 4] * 2, 4)


RANGES = [  # key scales, queries, value scales: times 2^this
    (80, -80, 0), (-100, 98, 0), (0, 0, -72), (0, 0, 110), (40, -40, 20), (0, -60, 0)]


@pytest.mark.parametrize("k_up,q_up,v_up", RANGES)
@pytest.mark.parametrize("rows", [8, 24, 160])
def test_ends_of_the_ranges(rows, k_up, q_up, v_up):
    """And with tokens whose values are all zero (E8M0 byte 0), where they are in range."""
    batch = Batch([1500, 90], 2, 128, 32, seed=rows, v_apart=2)
    for one in batch.rows:
        one[1] += k_up % 256
        one[3] += v_up % 256
        if v_up <= 20:
            one[2][32:80] = 0
            one[3][32:80] = 0
    batch.store()
    nq = rows // 4
    q = torch.randn(2 * nq, 8, 128, generator=batch.gen, device="cuda") * 2.0 ** q_up
    batch.check([nq] * 2, 4, q=q.bfloat16())
