"""The quantised key/value cache: what is timed, and the operators' plain forms.

Three operators over one paged cache whose keys and values are held as MX
blocks (32 consecutive elements of a head's row share an E8M0 power of two) in
4 bits (E2M1) or 8 bits (E4M3, E5M2):

  write   new keys and values are quantised into given cache slots, then the
          same slots are read back as 32-bit or bf16 values
  read    given cache slots are read back as bf16 or 32-bit values
  attend  softmax(scale * q k^T) v of query tokens over the 4-bit cache of
          their sequences: one token per sequence (decoding), a few (checking
          drafted tokens) or a whole prompt chunk; causal, optionally windowed

Cache arrays: codes [pages, kv_heads, page_size, row bytes] and E8M0 bytes
[pages, kv_heads, page_size, head_dim / 32], for keys and for values; slot
page * page_size + offset is one token.
"""
import math

import torch

own = False

E4M3, E5M2, E2M1 = 0, 1, 2
FLOOR, CEIL, NEAREST = 0, 1, 2
BLOCK = 32
#: format: (exponent bits, mantissa bits, bias, largest finite value, exponent of it)
FORMATS = {E4M3: (4, 3, 7, 448.0, 8), E5M2: (5, 2, 15, 57344.0, 15), E2M1: (2, 1, 1, 6.0, 2)}


# ---- cases -----------------------------------------------------------------

def listed():
    return [
        # one new token of one sequence: a decode step's cache write, all latency
        dict(name="write_one_token", op="write", tokens=1, kv_heads=8, head_dim=128, page=16, fmt=E2M1,
             rule=FLOOR, fp32=False, skip=0.0),
        # one new token of each of 128 sequences, scattered over the pool, 8-bit cache
        dict(name="write_step_128", op="write", tokens=128, kv_heads=8, head_dim=128, page=16, fmt=E4M3,
             rule=FLOOR, fp32=False, skip=0.0),
        # an odd fp32 batch with padding tokens that go nowhere, 5-bit exponents, scales rounded up
        dict(name="write_odd_fp32", op="write", tokens=1001, kv_heads=5, head_dim=96, page=32, fmt=E5M2,
             rule=CEIL, fp32=True, skip=0.1),
        # a prompt of 16384 tokens (the decoder workload's token count) into the 4-bit cache
        dict(name="write_prompt", op="write", tokens=16384, kv_heads=8, head_dim=128, page=64, fmt=E2M1,
             rule=CEIL, fp32=False, skip=0.0),
        # a short 8-bit context handed on to a 16-bit consumer
        dict(name="read_short", op="read", tokens=777, kv_heads=4, head_dim=64, page=16, fmt=E4M3, fp32=False),
        # a long 4-bit context read back whole
        dict(name="read_long", op="read", tokens=131072, kv_heads=8, head_dim=128, page=16, fmt=E2M1, fp32=False),
        # one sequence, one token, a short context: the smallest decode call
        dict(name="decode_one_short", op="attend", batch=1, longest=1000, shortest=1000, new=1, q_heads=16,
             kv_heads=4, head_dim=64, page=16, window=0),
        # a serving batch of uneven contexts, one padding entry among them
        dict(name="decode_batch_ragged", op="attend", batch=64, longest=8192, shortest=0, new=1, q_heads=32,
             kv_heads=4, head_dim=128, page=16, window=0),
        # few sequences with very long contexts
        dict(name="decode_long", op="attend", batch=8, longest=131072, shortest=131072, new=1, q_heads=32,
             kv_heads=8, head_dim=128, page=64, window=0),
        # five drafted tokens per sequence checked at once, sliding window
        dict(name="verify_window", op="attend", batch=16, longest=32768, shortest=100, new=5, q_heads=16,
             kv_heads=4, head_dim=128, page=32, window=4096),
        # a prompt chunk of 2048 tokens after 14336 cached ones
        dict(name="chunk_2048", op="attend", batch=1, longest=16384, shortest=16384, new=2048, q_heads=32,
             kv_heads=8, head_dim=128, page=64, window=0),
        # uneven prompts from their first token on
        dict(name="prompts_ragged", op="attend", batch=4, longest=4096, shortest=33, new=4096, q_heads=32,
             kv_heads=8, head_dim=128, page=16, window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["write", "read", "decode", "decode", "verify", "prompt"])
    page = rng.choice([1, 4, 16, 32, 64, 128])
    if kind in ("write", "read"):
        case = dict(op=kind, tokens=_log(rng, 1, 16384 if kind == "write" else 131072),
                    kv_heads=rng.choice([1, 2, 3, 4, 5, 8]), head_dim=rng.choice([32, 64, 96, 128]), page=page,
                    fmt=rng.choice([E2M1, E2M1, E4M3, E5M2]), fp32=rng.random() < 0.25)
        if kind == "write":
            case.update(rule=rng.choice([FLOOR, CEIL, NEAREST]), skip=rng.choice([0.0, 0.0, 0.2]))
        elif case["fp32"]:
            case["tokens"] = max(1, case["tokens"] // 2)
        return case
    kv_heads = rng.choice([1, 2, 4, 8])
    case = dict(op="attend", kv_heads=kv_heads, head_dim=rng.choice([64, 128]), page=page,
                window=rng.choice([0, 0, _log(rng, 1, 8192)]))
    if kind == "prompt":
        new = _log(rng, 17, 4096)
        longest = max(new, _log(rng, new, 16384))
        batch = max(1, min(rng.randint(1, 8), (2048 * 16384) // (new * longest)))
        group = rng.choice([1, 2, 4, 5, 8]) if kv_heads <= 4 else rng.choice([1, 2, 4])
        case.update(new=new, shortest=rng.choice([longest, max(1, longest // 9)]))
    else:
        new = 1 if kind == "decode" else rng.randint(2, 8)
        longest = _log(rng, 20, 131072)
        most = max(1, min(128, 8 * 131072 * 8 // (longest * kv_heads * 2)))
        batch = _log(rng, 1, most)
        group = rng.choice([1, 2, 3, 4, 7, 8, 16])
        case.update(new=new, shortest=rng.choice([longest, 0, longest // 7]))
    case.update(batch=batch, longest=longest, q_heads=group * kv_heads)
    return case


def _row_bytes(fmt, head_dim):
    return head_dim // 2 if fmt == E2M1 else head_dim


def _lengths(case):
    """Context and query lengths of an attend case's sequences: spread evenly, the longest first."""
    n, hi, lo = case["batch"], case["longest"], case["shortest"]
    kv = [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]
    return kv, [min(case["new"], k) if case["new"] > 8 else case["new"] for k in kv]


def _pairs(case):
    """(query, key) pairs that the masks leave, over all sequences."""
    kv, nq = _lengths(case)
    w, total = case["window"], 0
    for k, n in zip(kv, nq):
        for i in range(n):
            seen = max(0, k - n + i + 1)
            total += min(seen, w) if w else seen
    return total


def work(case):
    if case["op"] == "attend":
        kv, nq = _lengths(case)
        w, d, row = case["window"], case["head_dim"], case["head_dim"] // 2 + case["head_dim"] // BLOCK
        keys = sum((min(k, w + n - 1) if w else k) if n else 0 for k, n in zip(kv, nq))
        qo = 2 * 2 * sum(nq) * case["q_heads"] * d
        return {"bytes": 2 * keys * case["kv_heads"] * row + qo, "flops": 4 * _pairs(case) * case["q_heads"] * d}
    n = 2 * case["tokens"] * case["kv_heads"] * case["head_dim"]
    cached = n * (0.5 if case["fmt"] == E2M1 else 1) + n // BLOCK
    plain = n * (4 if case["fp32"] else 2)
    if case["op"] == "read":
        return {"bytes": cached + plain + 8 * case["tokens"], "flops": n}
    # read the new rows, write the cache, read it back, write the values
    return {"bytes": 2 * plain + 2 * cached + 16 * case["tokens"], "flops": 6 * n}


# ---- formats, in elementary operations -------------------------------------

def _quantise(x, fmt, rule):
    """x [..., D] in 32 bits -> (codes int32 [..., D], E8M0 uint8 [..., D / 32])."""
    _, mbits, bias, top, etop = FORMATS[fmt]
    x = x.unflatten(-1, (-1, BLOCK))
    amax = x.abs().amax(-1)
    mant, exp = torch.frexp(amax)                    # amax = mant * 2^exp, mant in [0.5, 1)
    e = exp - 1 - etop
    mu, most = 2 * mant, top / 2.0 ** etop           # significands of amax and of the format's largest value
    if rule == CEIL:
        e = e + (mu > most).int()
    elif rule == NEAREST:                            # nearest in the logarithm: mu against most / sqrt(2)
        e = e - (mu.double().square() < most * most / 2).int()
    e = torch.where(amax == 0, torch.full_like(e, -127), e.clamp(-127, 127))
    v = torch.ldexp(x, -e[..., None]).abs()
    g = (torch.frexp(v)[1] - 1).clamp(min=1 - bias) - mbits          # grid 2^g around v
    v = torch.ldexp(torch.round(torch.ldexp(v, -g)), g).clamp(max=top)
    h = (torch.frexp(v)[1] - 1).clamp(min=1 - bias)
    whole = torch.ldexp(v, mbits - h).int()          # significand as a whole number
    code = torch.where(whole < (1 << mbits), whole, ((h + bias) << mbits) + whole - (1 << mbits))
    code = code | (torch.signbit(x).int() << (7 if fmt != E2M1 else 3))
    return code.flatten(-2), (e + 127).to(torch.uint8)


def _pack(code, fmt):
    if fmt != E2M1:
        return code.to(torch.uint8)
    pair = code.unflatten(-1, (-1, 2))               # the even element in the low half
    return (pair[..., 0] | (pair[..., 1] << 4)).to(torch.uint8)


def _values(packed, e8m0, fmt):
    """Packed codes and E8M0 bytes -> values in 32 bits."""
    ebits, mbits, bias, _, _ = FORMATS[fmt]
    dev = packed.device
    n = 1 << (ebits + mbits)
    whole, field = torch.arange(n, device=dev) % (1 << mbits), torch.arange(n, device=dev) >> mbits
    one = torch.where(field > 0, whole + (1 << mbits), whole).float()
    table = torch.ldexp(one, field.clamp(min=1) - bias - mbits)
    table = torch.cat([table, -table])
    if fmt == E2M1:
        code = torch.stack([packed & 15, packed >> 4], -1).flatten(-2)
    else:
        code = packed
    v = table[code.int()].unflatten(-1, (-1, BLOCK))
    return torch.ldexp(v, e8m0.int()[..., None] - 127).flatten(-2)


# ---- inputs ----------------------------------------------------------------

def _keys(shape, gen, dev):
    """Activations as a projection leaves them: a few channels of every head far larger than the rest."""
    x = torch.randn(shape, generator=gen, device=dev)
    x[..., 5::37] *= 8
    return x


def _fill(pool_shape, fmt, gen, dev):
    """A cache's codes and E8M0 bytes for random rows, quantised page group by page group."""
    pages, heads, page, d = pool_shape
    codes = torch.empty(pages, heads, page, _row_bytes(fmt, d), dtype=torch.uint8, device=dev)
    scales = torch.empty(pages, heads, page, d // BLOCK, dtype=torch.uint8, device=dev)
    step = max(1, (1 << 26) // (heads * page * d))
    for a in range(0, pages, step):
        x = _keys((min(step, pages - a), heads, page, d), gen, dev).bfloat16().float()
        code, e = _quantise(x, fmt, CEIL)
        codes[a:a + step], scales[a:a + step] = _pack(code, fmt), e
    return codes, scales


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    heads, d, page = case["kv_heads"], case["head_dim"], case["page"]
    st = {"case": case}
    if case["op"] == "attend":
        kv, nq = _lengths(case)
        fmt = E2M1
        per = [-(-k // page) for k in kv]
        pages = sum(per) + 3
        order = torch.randperm(pages, generator=gen, device=dev).int()
        table = torch.zeros(len(kv), max(1, max(per)), dtype=torch.int32, device=dev)
        at = 0
        for i, p in enumerate(per):
            table[i, :p] = order[at:at + p]
            at += p
        cu = [0]
        for n in nq:
            cu.append(cu[-1] + n)
        x = torch.randn(cu[-1], case["q_heads"], d, generator=gen, device=dev)
        st.update(table=table, lens=torch.tensor(kv, dtype=torch.int32, device=dev), q=x.bfloat16(),
                  cu=None if max(nq) == min(nq) == 1 else torch.tensor(cu, dtype=torch.int32, device=dev),
                  max_q=max(nq), scale=d ** -0.5)
    else:
        fmt = case["fmt"]
        pages = -(-case["tokens"] // page) + 2
        slots = torch.randperm(pages * page, generator=gen, device=dev)[:case["tokens"]]
        if case["op"] == "read" or case["tokens"] > 4 * page:        # whole pages in any order, as sequences lie
            order = torch.randperm(pages, generator=gen, device=dev)
            slots = (order[:, None] * page + torch.arange(page, device=dev)).flatten()[:case["tokens"]]
        if case["op"] == "write":
            if case["skip"]:
                drop = torch.rand(case["tokens"], generator=gen, device=dev) < case["skip"]
                slots = torch.where(drop, torch.full_like(slots, -1), slots)
            # keys and values are parts of one projection's output: rows with a stride
            both = _keys((case["tokens"], 3 * heads, d), gen, dev)
            both = both if case["fp32"] else both.bfloat16()
            st.update(k=both[:, heads:2 * heads], v=both[:, 2 * heads:])
        st["slots"] = slots.contiguous()
    if case["op"] == "write":
        shape = (pages, heads, page, _row_bytes(fmt, d))
        eshape = (pages, heads, page, d // BLOCK)
        st["pools"] = tuple(torch.zeros(s, dtype=torch.uint8, device=dev) for s in (shape, eshape, shape, eshape))
    else:
        st["pools"] = _fill((pages, heads, page, d), fmt, gen, dev) + _fill((pages, heads, page, d), fmt, gen, dev)
    if own:
        from tensor_scaling_cast_gb300 import fp8q as F
        st["cache"] = F.MXKVCache(*st["pools"], fmt=fmt)
        if case["op"] == "attend":
            st["out"] = torch.empty_like(st["q"])
            st["workspace"] = F.mx_kv_attention_workspace(st["cache"], st["q"], st["table"], max_q=st["max_q"])
        else:
            kind = torch.float32 if case["fp32"] else torch.bfloat16
            st["k_out"] = torch.empty(case["tokens"], heads, d, dtype=kind, device=dev)
            st["v_out"] = torch.empty_like(st["k_out"])
    return st


# ---- one pass --------------------------------------------------------------

def run(st):
    case = st["case"]
    if own:
        from tensor_scaling_cast_gb300 import fp8q as F
        if case["op"] == "attend":
            F.mx_kv_attention(st["cache"], st["q"], st["out"], st["table"], st["lens"], cu_q=st["cu"],
                              max_q=st["max_q"], scale=st["scale"], window=case["window"],
                              workspace=st["workspace"])
            return st["out"]
        if case["op"] == "write":
            F.mx_kv_write(st["cache"], st["k"], st["v"], st["slots"], rule=case["rule"])
        F.mx_kv_read(st["cache"], st["slots"], st["k_out"], st["v_out"])
        return {"k": st["k_out"], "v": st["v_out"]}
    if case["op"] == "attend":
        return _attend(st)
    if case["op"] == "write":
        _write(st)
    return _read(st)


def _write(st):
    fmt, slots = st["case"]["fmt"], st["slots"]
    page = st["case"]["page"]
    keep = slots >= 0
    at, off = slots[keep] // page, slots[keep] % page
    k_q, k_e, v_q, v_e = st["pools"]
    for x, q, e in ((st["k"], k_q, k_e), (st["v"], v_q, v_e)):
        code, scale = _quantise(x[keep].float(), fmt, st["case"]["rule"])
        q[at, :, off] = _pack(code, fmt)
        e[at, :, off] = scale


def _read(st):
    case, slots = st["case"], st["slots"]
    keep, at = slots >= 0, slots.clamp(min=0)
    kind = torch.float32 if case["fp32"] else torch.bfloat16
    k_q, k_e, v_q, v_e = st["pools"]
    out = {}
    for name, q, e in (("k", k_q, k_e), ("v", v_q, v_e)):
        x = _values(q[at // case["page"], :, at % case["page"]], e[at // case["page"], :, at % case["page"]], case["fmt"])
        out[name] = torch.where(keep[:, None, None], x, torch.zeros_like(x)).to(kind)
    return out


def _rows(pool_q, pool_e, table):
    """The cached rows of every sequence, padded to the table's width: [batch, kv_heads, tokens, D]."""
    x = _values(pool_q[table.long()], pool_e[table.long()], E2M1)    # [B, pages, H, page, D]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _attend(st):
    case, table, lens, q = st["case"], st["table"], st["lens"].long(), st["q"].float()
    dev, batch, heads = q.device, table.shape[0], case["kv_heads"]
    k_q, k_e, v_q, v_e = st["pools"]
    cu = st["cu"].long() if st["cu"] is not None else torch.arange(batch + 1, device=dev)
    nq, most = cu[1:] - cu[:-1], st["max_q"]
    step = torch.arange(most, device=dev)
    at = (cu[:-1, None] + step).clamp(max=q.shape[0] - 1)
    # [B, H, tokens * group, D]
    x = q[at].unflatten(2, (heads, -1)).permute(0, 2, 1, 3, 4)
    group = x.shape[3]
    x = x.flatten(2, 3)
    k = _rows(k_q, k_e, table)
    s = torch.matmul(x, k.transpose(-1, -2)) * st["scale"]
    del k
    pos = (lens - nq)[:, None] + step                                # a query's own position
    key = torch.arange(s.shape[-1], device=dev)
    seen = (key <= pos[..., None]) & (key < lens[:, None, None]) & (step < nq[:, None])[..., None]
    if case["window"]:
        seen &= key > pos[..., None] - case["window"]
    s = s.unflatten(2, (most, group)).masked_fill_(~seen[:, None, :, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)))
    del s
    total = p.sum(-1, keepdim=True)
    v = _rows(v_q, v_e, table)
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, (most, group))
    o = torch.where(total > 0, o / total, torch.zeros_like(o))       # [B, H, tokens, group, D]
    o = o.permute(0, 2, 1, 3, 4).flatten(2, 3)
    return o[step < nq[:, None]].bfloat16()


# ---- the definition in 64 bits, apart from the forms above -----------------

def _grid(fmt):
    """The format's magnitudes in code order, in 64 bits."""
    ebits, mbits, bias, top, _ = FORMATS[fmt]
    got = []
    for c in range(1 << (ebits + mbits)):
        f, m = divmod(c, 1 << mbits)
        got.append(math.ldexp(m, 1 - bias - mbits) if f == 0 else math.ldexp(m + (1 << mbits), f - bias - mbits))
    return [g for g in got if g <= top]


def _nearest64(x, fmt, rule):
    """x [..., D] -> the values that its MX form stands for, in 64 bits."""
    top = FORMATS[fmt][3]
    grid = torch.tensor(_grid(fmt), dtype=torch.float64, device=x.device)
    mids = (grid[1:] + grid[:-1]) / 2
    b = x.double().unflatten(-1, (-1, BLOCK))
    amax = b.abs().amax(-1, keepdim=True)
    safe = torch.where(amax > 0, amax, torch.ones_like(amax))
    if rule == CEIL:       # the smallest power that keeps the largest value within the format
        e = torch.ceil(torch.log2(safe / top))
        e = torch.where(safe <= top * torch.exp2(e - 1), e - 1, e)
        e = torch.where(safe > top * torch.exp2(e), e + 1, e)
    elif rule == NEAREST:
        e = torch.round(torch.log2(safe / top))
    else:
        low = torch.floor(torch.log2(safe))
        low = torch.where(safe < torch.exp2(low), low - 1, low)
        low = torch.where(safe >= torch.exp2(low + 1), low + 1, low)
        e = low - FORMATS[fmt][4]
    scale = torch.exp2(e.clamp(-127, 127))
    m = (b.abs() / scale).contiguous()
    low = torch.bucketize(m, mids)                   # a value on a middle gives the lower neighbour
    tie = (low < len(mids)) & (m == mids[low.clamp(max=len(mids) - 1)])
    i = low + (tie & (low % 2 == 1)).long()          # ties go to the even code
    return (torch.sign(b) * grid[i] * scale).flatten(-2)


def _decode64(packed, e8m0, fmt):
    grid = _grid(fmt)
    n = 1 << sum(FORMATS[fmt][:2])
    grid = grid + [math.nan] * (n - len(grid))
    both = torch.tensor(grid + [-g for g in grid], dtype=torch.float64, device=packed.device)
    if fmt == E2M1:
        code = torch.empty(*packed.shape[:-1], 2 * packed.shape[-1], dtype=torch.long, device=packed.device)
        code[..., 0::2], code[..., 1::2] = packed % 16, packed // 16
    else:
        code = packed.long()
    return both[code] * torch.exp2(e8m0.double() - 127).repeat_interleave(BLOCK, -1)


def exact(case, seed):
    st = prepare(case, seed)
    k_q, k_e, v_q, v_e = st["pools"]
    page, heads = case["page"], case["kv_heads"]
    if case["op"] != "attend":
        out = {}
        for name, q, e in (("k", k_q, k_e), ("v", v_q, v_e)):
            if case["op"] == "write":
                x = _nearest64(st[name], case["fmt"], case["rule"])
                x[st["slots"] < 0] = 0
            else:
                at = st["slots"]
                x = torch.cat([_decode64(q[s // page, :, s % page], e[s // page, :, s % page], case["fmt"])
                               for s in at.split(8192)])
            out[name] = x
        return out
    kv, nq = _lengths(case)
    group, d = case["q_heads"] // heads, case["head_dim"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    at = 0
    for b, (n_kv, n_q) in enumerate(zip(kv, nq)):
        rows, at = slice(at, at + n_q), at + n_q
        if not n_kv or not n_q:
            continue
        ids = st["table"][b, :-(-n_kv // page)].long()
        pos = torch.arange(n_kv - n_q, n_kv, device=ids.device)[:, None]
        key = torch.arange(n_kv, device=ids.device)
        seen = key <= pos
        if case["window"]:
            seen &= key + case["window"] > pos
        for h in range(heads):
            k = _decode64(k_q[ids, h].flatten(0, 1)[:n_kv], k_e[ids, h].flatten(0, 1)[:n_kv], E2M1)
            v = _decode64(v_q[ids, h].flatten(0, 1)[:n_kv], v_e[ids, h].flatten(0, 1)[:n_kv], E2M1)
            for g in range(h * group, (h + 1) * group):
                s = (st["q"][rows, g].double() @ k.T) * st["scale"]
                p = torch.softmax(s.masked_fill(~seen, -math.inf), -1)
                out[rows, g] = torch.nan_to_num(p, nan=0.0) @ v
    return out
