"""Linear layers in MX form: what is timed, and the operators' plain forms.

MX blocks are 32 consecutive elements of a row that share an E8M0 power of two;
their codes have 4 bits (E2M1, two to a byte) or 8 (E4M3, E5M2).

  cast    a tensor is quantised to E2M1, row by row or (dual) its transpose as
          well from the same read, and the codes are decoded again
  matmul  out = a b^T (+ add) of two matrices held in MX blocks along the
          summed dimension, sums in 32 bits, out in bf16 or 32 bits
  act     h = f(z) * u of a gated MLP, or f(z): the forward pass keeps z and u
          as 8-bit MX blocks, the backward pass takes them from there
  mlp     these together, as the second half of an MLP's training step: h to
          MX and its product with the weights, then the gradients of z, u and
          the weights from the 8-bit checkpoint
"""
import math

import torch

own = False

E4M3, E5M2, E2M1 = 0, 1, 2
FLOOR, CEIL, NEAREST = 0, 1, 2
SILU, GELU, GELU_TANH = 0, 1, 2
BLOCK = 32
#: format: (exponent bits, mantissa bits, bias, largest finite value, exponent of it)
FORMATS = {E4M3: (4, 3, 7, 448.0, 8), E5M2: (5, 2, 15, 57344.0, 15), E2M1: (2, 1, 1, 6.0, 2)}


# ---- cases -----------------------------------------------------------------

def listed():
    return [
        # one token's activations on the way into a 4-bit layer: all latency
        dict(name="cast_one_token", op="cast", rows=1, cols=2048, fp32=False, rule=FLOOR, dual=False),
        # an odd fp32 batch, scales rounded up
        dict(name="cast_odd_fp32", op="cast", rows=1001, cols=1056, fp32=True, rule=CEIL, dual=False),
        # a training step's widest activation, both ways for the backward products
        dict(name="cast_dual_layer", op="cast", rows=16384, cols=8192, fp32=False, rule=CEIL, dual=True),
        # a decode step of one sequence through the up projection, 4-bit weights
        dict(name="matmul_one_token", op="matmul", m=1, n=8192, k=2048, a_fmt=E2M1, b_fmt=E2M1, fp32=False, add=False),
        # a decode batch through the down projection
        dict(name="matmul_batch_64", op="matmul", m=64, n=2048, k=8192, a_fmt=E2M1, b_fmt=E2M1, fp32=False, add=False),
        # odd sizes in 8 bits, a gradient against weights
        dict(name="matmul_odd_8bit", op="matmul", m=1001, n=1055, k=2080, a_fmt=E5M2, b_fmt=E4M3, fp32=False, add=False),
        # the training step's tokens through the up projection in 4 bits
        dict(name="matmul_tokens", op="matmul", m=16384, n=8192, k=2048, a_fmt=E2M1, b_fmt=E2M1, fp32=False, add=False),
        # the down projection's weight gradient in 8 bits, added to a 32-bit sum
        dict(name="matmul_weight_grad", op="matmul", m=2048, n=8192, k=16384, a_fmt=E5M2, b_fmt=E4M3, fp32=True, add=True),
        # a few tokens in 32 bits, without a gate
        dict(name="act_few_fp32", op="act", rows=5, cols=2080, fp32=True, act=GELU, gated=False, fmt=E5M2, rule=FLOOR),
        # the training step's gated activation, forward and backward
        dict(name="act_layer", op="act", rows=16384, cols=8192, fp32=False, act=SILU, gated=True, fmt=E4M3, rule=CEIL),
        # half an MLP's training step at a small batch, h in 8 bits
        dict(name="mlp_step", op="mlp", rows=2048, ffn=8192, hidden=2048, act=SILU, gated=True, h_fmt=E4M3),
        # an uneven batch with h in 4 bits, no gate
        dict(name="mlp_step_4bit", op="mlp", rows=416, ffn=4096, hidden=1024, act=GELU_TANH, gated=False, h_fmt=E2M1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _multiple(rng, lo, hi, of):
    return of * max(1, _log(rng, lo, hi) // of)


def draw(rng):
    op = rng.choice(["cast", "cast", "matmul", "matmul", "matmul", "act", "act", "mlp"])
    if op == "cast":
        dual = rng.random() < 0.5
        rows, cols = _log(rng, 1, 16384), _multiple(rng, 32, 8192, 32)
        return dict(op=op, rows=-(-rows // 32) * 32 if dual else rows, cols=cols, dual=dual,
                    fp32=rng.random() < 0.3 and rows * cols < 1 << 26, rule=rng.choice([FLOOR, CEIL, NEAREST]))
    if op == "matmul":
        m, n, k = _log(rng, 1, 16384), _log(rng, 1, 16384), _multiple(rng, 32, 16384, 32)
        while m * n * k > 16384 * 8192 * 2048 or m * n > 1 << 27:
            m, n = m // 2, n // 2
        a, b = rng.choice([(E2M1, E2M1), (E2M1, E2M1), (E4M3, E4M3), (E5M2, E4M3), (E4M3, E5M2)])
        return dict(op=op, m=m, n=n, k=k, a_fmt=a, b_fmt=b, fp32=rng.random() < 0.3, add=rng.random() < 0.3)
    if op == "act":
        rows, cols = _log(rng, 1, 16384), _multiple(rng, 32, 8192, 32)
        return dict(op=op, rows=rows, cols=cols, fp32=rng.random() < 0.25 and rows * cols < 1 << 25,
                    act=rng.choice([SILU, GELU, GELU_TANH]), gated=rng.random() < 0.6,
                    fmt=rng.choice([E4M3, E4M3, E5M2]), rule=rng.choice([FLOOR, CEIL, NEAREST]))
    return dict(op=op, rows=_multiple(rng, 32, 2048, 32), ffn=_multiple(rng, 64, 8192, 32),
                hidden=_multiple(rng, 64, 2048, 32), act=rng.choice([SILU, GELU, GELU_TANH]),
                gated=rng.random() < 0.6, h_fmt=rng.choice([E4M3, E2M1]))


def _held(n, fmt):
    """Bytes of n elements in MX blocks."""
    return n * (0.5 if fmt == E2M1 else 1) + n / BLOCK


def work(case):
    if case["op"] == "cast":
        n, size = case["rows"] * case["cols"], 4 if case["fp32"] else 2
        ways = 2 if case["dual"] else 1
        return {"bytes": n * size + ways * (2 * _held(n, E2M1) + n * size), "flops": 4 * ways * n}
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        size = 4 if case["fp32"] else 2
        return {"bytes": _held(m * k, case["a_fmt"]) + _held(n * k, case["b_fmt"]) + m * n * size * (2 if case["add"] else 1),
                "flops": 2 * m * n * k}
    if case["op"] == "act":
        # forward: z, u in, h and the 8-bit z, u out; backward: those and dh in, dz, du out
        n, size, ins = case["rows"] * case["cols"], 4 if case["fp32"] else 2, 2 if case["gated"] else 1
        return {"bytes": n * size * (2 * ins + 2) + 2 * ins * _held(n, case["fmt"]), "flops": 20 * ins * n}
    t, f, d = case["rows"], case["ffn"], case["hidden"]
    ins, h = 2 if case["gated"] else 1, case["h_fmt"]
    n = t * f
    act = 2 * n * 2 * ins + 2 * ins * _held(n, E4M3) + 2 * n
    products = (_held(n, h) + _held(f * d, h) + 2 * t * d) + (_held(t * d, E5M2) + _held(f * d, E4M3) + 2 * n) \
        + (_held(n, E4M3) + _held(t * d, E5M2) + 4 * f * d)
    return {"bytes": act + products + 2 * t * d, "flops": 3 * 2 * t * f * d}


# ---- MX blocks in elementary operations ------------------------------------

def _ldexp(x, n):
    """x * 2^n, exactly: in 64 bits torch.ldexp's power of two is a rounded one."""
    if x.dtype != torch.float64:
        return torch.ldexp(x, n)
    return x * ((n.long() + 1023) << 52).view(torch.float64)


def _quantise(x, fmt, rule):
    """x [rows, cols] -> (one code per element, int32; E8M0 uint8 [rows, cols / 32]); blocks of a row."""
    _, mbits, bias, top, etop = FORMATS[fmt]
    wide = x.dtype if x.dtype == torch.float64 else torch.float32
    x = x.to(wide).unflatten(-1, (-1, BLOCK))
    amax = x.abs().amax(-1)
    mant, exp = torch.frexp(amax)                    # amax = mant * 2^exp, mant in [0.5, 1)
    e = exp - 1 - etop
    mu, most = 2 * mant, top / 2.0 ** etop           # significands of amax and of the format's largest value
    if rule == CEIL:
        e = e + (mu > most).int()
    elif rule == NEAREST:                            # nearest in the logarithm: mu against most / sqrt(2)
        e = e - (mu.double().square() < most * most / 2).int()
    e = torch.where(amax == 0, torch.full_like(e, -127), e.clamp(-127, 127))
    v = _ldexp(x, -e[..., None]).abs()
    g = (torch.frexp(v)[1] - 1).clamp(min=1 - bias) - mbits          # grid 2^g around v
    v = _ldexp(torch.round(_ldexp(v, -g)), g).clamp(max=top)
    h = (torch.frexp(v)[1] - 1).clamp(min=1 - bias)
    whole = _ldexp(v, mbits - h).int()          # significand as a whole number
    code = torch.where(whole < (1 << mbits), whole, ((h + bias) << mbits) + whole - (1 << mbits))
    code = code | (torch.signbit(x).int() << (7 if fmt != E2M1 else 3))
    return code.flatten(-2), (e + 127).to(torch.uint8)


def _pack(code, fmt):
    if fmt != E2M1:
        return code.to(torch.uint8)
    pair = code.unflatten(-1, (-1, 2))               # the even element in the low half
    return (pair[..., 0] | (pair[..., 1] << 4)).to(torch.uint8)


def _values(packed, e8m0, fmt, kind=torch.float32):
    """Packed codes and E8M0 bytes -> the values that they stand for."""
    ebits, mbits, bias, _, _ = FORMATS[fmt]
    n = 1 << (ebits + mbits)
    at = torch.arange(n, device=packed.device)
    whole, field = at % (1 << mbits), at >> mbits
    one = torch.where(field > 0, whole + (1 << mbits), whole).to(kind)
    table = _ldexp(one, field.clamp(min=1) - bias - mbits)
    table = torch.cat([table, -table])
    code = torch.stack([packed & 15, packed >> 4], -1).flatten(-2) if fmt == E2M1 else packed
    v = table[code.int()].unflatten(-1, (-1, BLOCK))
    return _ldexp(v, e8m0.int()[..., None] - 127).flatten(-2)


def _held_values(x, fmt, rule):
    """x as its MX blocks hold it, in x's own width."""
    code, e = _quantise(x, fmt, rule)
    return _values(_pack(code, fmt), e, fmt, x.dtype)


# ---- inputs ----------------------------------------------------------------

def _activations(shape, gen, dev):
    """Activations: a few entries far larger than the rest."""
    x = torch.randn(shape, generator=gen, device=dev)
    x.view(-1)[::9973] *= 20
    return x


def _mx(rows, cols, fmt, size, gen, dev):
    """A matrix in MX blocks, quantised some rows at a time."""
    q = torch.empty(rows, cols // 2 if fmt == E2M1 else cols, dtype=torch.uint8, device=dev)
    e = torch.empty(rows, cols // BLOCK, dtype=torch.uint8, device=dev)
    step = max(1, (1 << 25) // cols)
    for a in range(0, rows, step):
        x = torch.randn(min(step, rows - a), cols, generator=gen, device=dev).mul_(size).bfloat16().float()
        code, e[a:a + step] = _quantise(x, fmt, CEIL)
        q[a:a + step] = _pack(code, fmt)
    return q, e


def _act_inputs(case, gen, dev, st, rows, cols, kind):
    # z and u are halves of one projection's output: rows with a stride
    both = _activations((rows, 2 * cols if case["gated"] else cols), gen, dev).to(kind)
    st["z"], st["u"] = both[:, :cols], both[:, cols:] if case["gated"] else None


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    st = {"case": case}
    if case["op"] == "cast":
        kind = torch.float32 if case["fp32"] else torch.bfloat16
        st["x"] = _activations((case["rows"], case["cols"]), gen, dev).to(kind)
    elif case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        st["a"] = _mx(m, k, case["a_fmt"], 1e-3 if case["a_fmt"] == E5M2 else 1.0, gen, dev)
        st["b"] = _mx(n, k, case["b_fmt"], 0.02, gen, dev)
        kind = torch.float32 if case["fp32"] else torch.bfloat16
        st["add"] = torch.randn(m, n, generator=gen, device=dev).mul_(0.1).to(kind) if case["add"] else None
    elif case["op"] == "act":
        kind = torch.float32 if case["fp32"] else torch.bfloat16
        _act_inputs(case, gen, dev, st, case["rows"], case["cols"], kind)
        st["dh"] = torch.randn(case["rows"], case["cols"], generator=gen, device=dev).mul_(1e-3).to(kind)
    else:
        t, f, d = case["rows"], case["ffn"], case["hidden"]
        _act_inputs(case, gen, dev, st, t, f, torch.bfloat16)
        w = torch.randn(d, f, generator=gen, device=dev).mul_(0.02).bfloat16().float()
        st["w"] = tuple(_packed(w, case["h_fmt"]))            # [hidden, ffn], for the forward product
        st["wt"] = tuple(_packed(w.T.contiguous(), E4M3))     # [ffn, hidden], for dh
        st["dy"] = torch.randn(t, d, generator=gen, device=dev).mul_(1e-3).bfloat16()
    if own:
        _prepare_own(st)
    return st


def _packed(x, fmt):
    code, e = _quantise(x, fmt, CEIL)
    return _pack(code, fmt), e


def _prepare_own(st):
    """The buffers that a program keeps for these calls."""
    from tensor_scaling_cast_gb300 import fp8q as F
    case, dev = st["case"], torch.device("cuda")
    if case["op"] == "cast":
        r, c, kind = case["rows"], case["cols"], st["x"].dtype
        st["row"] = F.MXMatrix.allocate(r, c, E2M1)
        st["out"] = torch.empty(r, c, dtype=kind, device=dev)
        if case["dual"]:
            st["col"] = F.MXMatrix.allocate(c, r, E2M1)
            st["out_t"] = torch.empty(c, r, dtype=kind, device=dev)
    elif case["op"] == "matmul":
        st["a"] = F.MXMatrix(*st["a"], case["a_fmt"])
        st["b"] = F.MXMatrix(*st["b"], case["b_fmt"])
        st["out"] = torch.empty(case["m"], case["n"], dtype=torch.float32 if case["fp32"] else torch.bfloat16, device=dev)
    else:
        z, gated = st["z"], case["gated"]
        rows, cols = z.shape
        fmt = case["fmt"] if case["op"] == "act" else E4M3
        st["z_mx"] = F.MXMatrix.allocate(rows, cols, fmt)
        st["u_mx"] = F.MXMatrix.allocate(rows, cols, fmt) if gated else None
        st["h"] = torch.empty(rows, cols, dtype=z.dtype, device=dev)
        st["dz"] = torch.empty_like(st["h"])
        st["du"] = torch.empty_like(st["h"]) if gated else None
        if case["op"] == "mlp":
            t, f, d = case["rows"], case["ffn"], case["hidden"]
            st["w"], st["wt"] = F.MXMatrix(*st["w"], case["h_fmt"]), F.MXMatrix(*st["wt"], E4M3)
            st["h_mx"] = F.MXMatrix.allocate(t, f, case["h_fmt"])
            st["y"] = torch.empty(t, d, dtype=torch.bfloat16, device=dev)
            st["dy_mx"], st["dyt_mx"] = F.MXMatrix.allocate(t, d, E5M2), F.MXMatrix.allocate(d, t, E5M2)
            st["h8_mx"], st["ht_mx"] = F.MXMatrix.allocate(t, f, E4M3), F.MXMatrix.allocate(f, t, E4M3)
            st["dh"] = torch.empty(t, f, dtype=torch.bfloat16, device=dev)
            st["dw"] = torch.empty(d, f, dtype=torch.float32, device=dev)


# ---- one pass --------------------------------------------------------------

def run(st):
    op = st["case"]["op"]
    if own:
        return {"cast": _cast_own, "matmul": _matmul_own, "act": _act_own, "mlp": _mlp_own}[op](st)
    return {"cast": _cast, "matmul": _matmul, "act": _act, "mlp": _mlp}[op](st)


def _cast_own(st):
    from tensor_scaling_cast_gb300 import fp8q as F
    case, row = st["case"], st["row"]
    if not case["dual"]:
        F.mx_cast_ex(st["x"], E2M1, case["rule"], 0, F.MX_ROWWISE, row.q, row.e8m0)
        F.mx_decode(row, st["out"])
        return st["out"]
    col = st["col"]
    F.mx_cast_dual(st["x"], E2M1, case["rule"], 0, row.q, row.e8m0, col.q, col.e8m0)
    F.mx_decode(row, st["out"])
    F.mx_decode(col, st["out_t"])
    return [st["out"], st["out_t"]]


def _matmul_own(st):
    from tensor_scaling_cast_gb300 import fp8q as F
    F.mx_matmul(st["a"], st["b"], st["out"], add=st["add"])
    return st["out"]


def _act_own(st):
    from tensor_scaling_cast_gb300 import fp8q as F
    case = st["case"]
    F.mx_act_forward(case["act"], st["z"], st["u"], z_saved=st["z_mx"], u_saved=st["u_mx"], h=st["h"], rule=case["rule"])
    F.mx_act_backward(case["act"], st["z_mx"], st["u_mx"], st["dh"], st["dz"], st["du"])
    return {"h": st["h"], "dz": st["dz"], "du": st["du"]}


def _mlp_own(st):
    from tensor_scaling_cast_gb300 import fp8q as F
    act = st["case"]["act"]
    F.mx_act_forward(act, st["z"], st["u"], z_saved=st["z_mx"], u_saved=st["u_mx"], h_mx=st["h_mx"], rule=CEIL)
    F.mx_matmul(st["h_mx"], st["w"], st["y"])
    dy, dyt, h8, ht = st["dy_mx"], st["dyt_mx"], st["h8_mx"], st["ht_mx"]
    F.mx_cast_dual(st["dy"], E5M2, CEIL, 0, dy.q, dy.e8m0, dyt.q, dyt.e8m0)
    F.mx_matmul(dy, st["wt"], st["dh"])
    F.mx_act_backward(act, st["z_mx"], st["u_mx"], st["dh"], st["dz"], st["du"], h=st["h"])
    F.mx_cast_dual(st["h"], E4M3, CEIL, 0, h8.q, h8.e8m0, ht.q, ht.e8m0)
    F.mx_matmul(dyt, ht, st["dw"])
    return {"y": st["y"], "dz": st["dz"], "du": st["du"], "dw": st["dw"]}


def _cast(st):
    case, x = st["case"], st["x"]
    out = _held_values(x.float(), E2M1, case["rule"]).to(x.dtype)
    if not case["dual"]:
        return out
    return [out, _held_values(x.T.float(), E2M1, case["rule"]).to(x.dtype)]


def _matmul(st):
    case = st["case"]
    out = _values(*st["a"], case["a_fmt"]) @ _values(*st["b"], case["b_fmt"]).T
    if st["add"] is not None:
        out += st["add"].float()
    return out if case["fp32"] else out.bfloat16()


def _f(act, z):
    """f(z) and its derivative."""
    if act == SILU:
        s = 1 / (1 + torch.exp(-z))
        return z * s, s * (1 + z * (1 - s))
    if act == GELU:
        phi = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return z * phi, phi + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    c, b = math.sqrt(2 / math.pi), 0.044715
    t = torch.tanh(c * (z + b * z * z * z))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * b * z * z)


def _forward(act, z, u):
    return _f(act, z)[0] if u is None else _f(act, z)[0] * u


def _backward(act, z, u, dh):
    f, df = _f(act, z)
    return (dh * df, None) if u is None else (dh * u * df, dh * f)


def _rounded(d, kind):
    return {k: v.to(kind) for k, v in d.items() if v is not None}


def _act(st):
    case, z, u = st["case"], st["z"].float(), None if st["u"] is None else st["u"].float()
    h = _forward(case["act"], z, u)
    z = _held_values(z, case["fmt"], case["rule"])
    u = None if u is None else _held_values(u, case["fmt"], case["rule"])
    dz, du = _backward(case["act"], z, u, st["dh"].float())
    return _rounded(dict(h=h, dz=dz, du=du), st["z"].dtype)


def _mlp(st):
    case, act = st["case"], st["case"]["act"]
    z, u = st["z"].float(), None if st["u"] is None else st["u"].float()
    # in 64 bits up to the codes of h: values next to a border between two codes
    h = _forward(act, z.double(), None if u is None else u.double())
    y = _held_values(h, case["h_fmt"], CEIL).float() @ _values(*st["w"], case["h_fmt"]).T
    z = _held_values(z, E4M3, CEIL)
    u = None if u is None else _held_values(u, E4M3, CEIL)
    dy = st["dy"].float()
    dh = (_held_values(dy, E5M2, CEIL) @ _values(*st["wt"], E4M3).T).bfloat16().float()
    dz, du = _backward(act, z, u, dh)
    h = _forward(act, z.double(), None if u is None else u.double()).bfloat16().float()
    dw = _held_values(dy.T.contiguous(), E5M2, CEIL) @ _held_values(h.T.contiguous(), E4M3, CEIL).T
    return {**_rounded(dict(y=y, dz=dz, du=du), torch.bfloat16), "dw": dw}


# ---- the definition in 64 bits, apart from the forms above -----------------

def _grid(fmt):
    """The format's finite magnitudes in code order, in 64 bits."""
    ebits, mbits, bias, top, _ = FORMATS[fmt]
    got = []
    for c in range(1 << (ebits + mbits)):
        f, m = divmod(c, 1 << mbits)
        got.append(math.ldexp(m, 1 - bias - mbits) if f == 0 else math.ldexp(m + (1 << mbits), f - bias - mbits))
    return [g for g in got if g <= top]


def _nearest64(x, fmt, rule):
    """x [rows, cols] -> the values that its MX form stands for, in 64 bits, some rows at a time."""
    top = FORMATS[fmt][3]
    grid = torch.tensor(_grid(fmt), dtype=torch.float64, device=x.device)
    mids = (grid[1:] + grid[:-1]) / 2
    parts = []
    for part in x.split(max(1, (1 << 24) // x.shape[1])):
        b = part.double().unflatten(-1, (-1, BLOCK))
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
        low = torch.bucketize(m, mids)               # a value on a middle gives the lower neighbour
        tie = (low < len(mids)) & (m == mids[low.clamp(max=len(mids) - 1)])
        i = low + (tie & (low % 2 == 1)).long()      # ties go to the even code
        parts.append((torch.sign(b) * grid[i] * scale).flatten(-2))
    return torch.cat(parts)


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


def _f64(act, z):
    """The activation and, by the chain rule through its own pieces, its derivative."""
    if act == SILU:
        s = torch.sigmoid(z)
        return z * s, s + z * s * torch.sigmoid(-z)
    if act == GELU:
        return 0.5 * z * torch.erfc(-z / math.sqrt(2)), \
            0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    # tanh(x) = 2 sigmoid(2x) - 1
    x2, dx2 = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3), 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z ** 2)
    s = torch.sigmoid(x2)
    return z * s, s + z * s * torch.sigmoid(-x2) * dx2


def exact(case, seed):
    global own
    was, own = own, False
    st = prepare(case, seed)
    own = was
    if case["op"] == "cast":
        out = _nearest64(st["x"], E2M1, case["rule"])
        return [out, _nearest64(st["x"].T, E2M1, case["rule"])] if case["dual"] else out
    if case["op"] == "matmul":
        if 2 * case["m"] * case["n"] * case["k"] > 4e12:
            return None
        out = _decode64(*st["a"], case["a_fmt"]) @ _decode64(*st["b"], case["b_fmt"]).T
        return out if st["add"] is None else out + st["add"].double()
    act = case["act"]
    z, u = st["z"].double(), None if st["u"] is None else st["u"].double()
    fmt, rule = (case["fmt"], case["rule"]) if case["op"] == "act" else (E4M3, CEIL)
    h = _f64(act, z)[0] if u is None else _f64(act, z)[0] * u
    z8, u8 = _nearest64(st["z"], fmt, rule), None if u is None else _nearest64(st["u"], fmt, rule)
    f, df = _f64(act, z8)
    if case["op"] == "act":
        dh = st["dh"].double()
        return {"h": h, "dz": dh * df, "du": None} if u is None else {"h": h, "dz": dh * u8 * df, "du": dh * f}
    y = _nearest64(h, case["h_fmt"], CEIL) @ _decode64(*st["w"], case["h_fmt"]).T
    # what the step rounds to 16 bits on its way is rounded here too
    dh = (_nearest64(st["dy"], E5M2, CEIL) @ _decode64(*st["wt"], E4M3).T).bfloat16().double()
    h8 = (f if u is None else f * u8).bfloat16()
    dw = _nearest64(st["dy"].T, E5M2, CEIL) @ _nearest64(h8.T, E4M3, CEIL).T
    return {"y": y, "dz": dh * df if u is None else dh * u8 * df, "du": None if u is None else dh * f, "dw": dw}
