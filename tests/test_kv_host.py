"""The key/value cache without a GPU: the plain reference against the plain-C
oracle, and the host-side refusals of the mx_kv_* entry points."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import kv


@pytest.fixture(scope="module")
def lib():
    from tensor_scaling_cast_gb300 import build
    build.build()
    from tensor_scaling_cast_gb300 import fp8q
    return fp8q.load()


@pytest.mark.parametrize("fmt", [kv.E4M3, kv.E5M2])
@pytest.mark.parametrize("rule", [kv.FLOOR, kv.CEIL, kv.NEAREST])
def test_reference_agrees_with_the_c_oracle_in_8_bits(orc, fmt, rule):
    rng = np.random.default_rng(5)
    x = (rng.standard_normal((64, 96)) * np.exp2(rng.integers(-40, 40, (64, 1)))).astype(np.float32)
    x[0], x[1, 3], x[2, 40], x[3, :32] = 0, np.nan, -np.inf, -0.0
    q, e, _ = orc.mx_cast_ex(x.view(np.uint32), fmt, rule, 0, 0)
    code, e8 = kv.encode(x, fmt, rule)
    assert np.array_equal(q, code) and np.array_equal(e, e8)


def test_every_e2m1_code_survives_the_round_trip():
    codes = np.arange(16, dtype=np.uint8).repeat(2)[None]
    for e in (1, 60, 127, 200, 252):
        e8 = np.array([[e]], dtype=np.uint8)
        v = kv.decode(kv.pack(codes, kv.E2M1), e8, kv.E2M1)
        again, e2 = kv.encode(v, kv.E2M1, kv.FLOOR)
        assert np.array_equal(again, codes) and np.array_equal(e2, e8)


def test_e2m1_rounding_and_rules():
    x = np.zeros((1, 32))
    x[0, :12] = [4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, -0.2, -0.25, 7.99]
    code, e = kv.encode(x, kv.E2M1, kv.FLOOR)
    assert e[0, 0] == 127                                # 7.99 = 1.9975 * 2^2: it clips to 6
    assert list(code[0, :12]) == [6, 0, 2, 2, 4, 4, 6, 6, 7, 8, 8, 7]
    assert kv.encode(x, kv.E2M1, kv.CEIL)[1][0, 0] == 128
    for amax, rule, want in ((6.0, kv.CEIL, 127), (6.0000001, kv.CEIL, 128), (4.2426, kv.NEAREST, 126),
                             (4.2427, kv.NEAREST, 127), (8.0, kv.NEAREST, 127), (8.49, kv.NEAREST, 128),
                             (8.48, kv.NEAREST, 127)):
        x = np.full((1, 32), amax)
        assert kv.encode(x, kv.E2M1, rule)[1][0, 0] == want, (amax, rule)


class Cache(ctypes.Structure):
    _fields_ = [("k_q", ctypes.c_void_p), ("k_e8m0", ctypes.c_void_p), ("v_q", ctypes.c_void_p),
                ("v_e8m0", ctypes.c_void_p), ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("format", ctypes.c_int32)]


def _cache(**kw):
    d = dict(k_q=0x1000, k_e8m0=0x2000, v_q=0x3000, v_e8m0=0x4000, num_pages=4, page_size=16, kv_heads=2,
             head_dim=64, format=2)
    d.update(kw)
    return Cache(**d)


def _write(lib, c, x=0x10000, dtype=1, tokens=4, strides=(128, 64, 128, 64), slots=0x20000, rule=0):
    return lib.mx_kv_write(None if c is None else ctypes.addressof(c), x, x, dtype, tokens, *strides, slots, rule, None)


def _read(lib, c, x=0x10000, dtype=1, tokens=4, strides=(128, 64, 128, 64), slots=0x20000):
    return lib.mx_kv_read(None if c is None else ctypes.addressof(c), slots, tokens, x, x, dtype, *strides, None)


BAD_CACHE = [(dict(format=3), -3), (dict(page_size=0), -1), (dict(page_size=24), -1), (dict(kv_heads=0), -1),
             (dict(kv_heads=5000), -1), (dict(head_dim=48), -1), (dict(head_dim=288), -1), (dict(head_dim=0), -1),
             (dict(num_pages=-1), -1), (dict(k_q=0), -1), (dict(v_e8m0=0), -1), (dict(v_q=0x3008), -2),
             (dict(k_e8m0=0x2001), -2)]


@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_cache_refusals(lib, kw, status):
    c = _cache(**kw)
    assert _write(lib, c) == status
    assert _read(lib, c) == status
    assert lib.mx_kv_attention_workspace(ctypes.addressof(c), 1, 2, 1, 1, 1) == status


def test_write_and_read_refusals(lib):
    c = _cache()
    for call in (_write, _read):
        assert call(lib, None) == -1
        assert call(lib, c, dtype=2) == -3
        assert call(lib, c, tokens=-1) == -1
        assert call(lib, c, x=None) == -1
        assert call(lib, c, slots=None) == -1
        assert call(lib, c, x=0x10008) == -2
        assert call(lib, c, strides=(132, 64, 128, 64)) == -2
        assert call(lib, c, strides=(128, 64, 128, 36)) == -2
        assert call(lib, c, tokens=0, x=None, slots=None) == 0
    assert _write(lib, c, rule=3) == -1
    assert _write(lib, c, rule=-1) == -1


def _attend(lib, c, q=0x10000, dtype=1, total=3, heads=4, strides=(256, 64), out=0x20000, cu=None, lens=0x30000,
            table=0x40000, stride=8, width=8, batch=3, max_q=1, scale=0.125, window=0, ws=0x50000, ws_bytes=1 << 40):
    return lib.mx_kv_attention(None if c is None else ctypes.addressof(c), q, dtype, total, heads, *strides, out,
                               *strides, None, cu, lens, table, stride, width, batch, max_q, scale, window, ws,
                               ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=0), -3), (dict(dtype=7), -3), (dict(q=None), -1), (dict(out=None), -1), (dict(lens=None), -1),
    (dict(table=None), -1), (dict(q=0x10004), -2), (dict(out=0x20008), -2), (dict(strides=(252, 64)), -2),
    (dict(heads=3), -1), (dict(heads=0), -1), (dict(total=-1), -1), (dict(batch=-1), -1), (dict(batch=70000), -1),
    (dict(max_q=0), -1), (dict(width=0), -1), (dict(stride=7), -1), (dict(scale=0.0), -1),
    (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(window=-1), -1), (dict(total=4), -1),
    (dict(max_q=2), -1), (dict(width=1 << 28, stride=1 << 28), -1), (dict(ws_bytes=-1), -1)])
def test_attention_refusals(lib, kw, status):
    assert _attend(lib, _cache(), **kw) == status


def test_attention_takes_the_4_bit_cache_and_its_head_sizes(lib):
    assert _attend(lib, None) == -1
    assert _attend(lib, _cache(format=0)) == -3
    assert _attend(lib, _cache(head_dim=96), strides=(384, 96)) == -1
    assert _attend(lib, _cache(), total=0, batch=0, q=None, out=None) == 0


def test_binding_refuses_wrong_tensors():
    from tensor_scaling_cast_gb300 import fp8q as F
    cache = F.MXKVCache.allocate(2, 16, 2, 64, device="cpu")
    assert cache.k_q.shape == (2, 2, 16, 32) and cache.k_e8m0.shape == (2, 2, 16, 2)
    x, slots = torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int64)
    for k, v, s in ((x[:2], x, slots), (x, x[..., :32], slots), (x, x, slots.int()), (x, x.bfloat16(), slots),
                    (x.transpose(1, 2), x, slots), (x, x, slots[:2])):
        with pytest.raises(TypeError):
            F.mx_kv_write(cache, k, v, s)
        with pytest.raises(TypeError):
            F.mx_kv_read(cache, s, k, v)
    with pytest.raises(TypeError):
        F.mx_kv_write(cache, x.half(), x.half(), slots)
    with pytest.raises(TypeError):
        F.MXKVCache(cache.k_q, cache.k_e8m0, cache.v_q[..., :16], cache.v_e8m0)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(3, 1, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    for bad in (dict(q=q.float()), dict(out=q[:2]), dict(table=table.long()), dict(lens=lens[:2]),
                dict(cu_q=lens), dict(lse=torch.zeros(3, 3))):
        a = dict(q=q, out=q.clone(), table=table, lens=lens)
        a.update({k: v for k, v in bad.items() if k in a})
        with pytest.raises(TypeError):
            F.mx_kv_attention(cache, a["q"], a["out"], a["table"], a["lens"], cu_q=bad.get("cu_q"),
                              lse=bad.get("lse"))


def test_a_workspace_without_a_bound_serves_every_plan(monkeypatch):
    """max_q left out: the largest of the plans that any max_q can get, and
    refusals are passed on."""
    from tensor_scaling_cast_gb300 import fp8q as F
    cache = F.MXKVCache.allocate(2, 16, 2, 64, device="cpu")
    asked = []

    class Fake:
        sizes = {1: 20000, 2: 60000, 4: 50000, 8: 70000, 90: 65536}

        def mx_kv_attention_workspace(self, ref, total, heads, batch, max_q, width):
            asked.append((total, heads, batch, max_q, width))
            return self.sizes.get(max_q, 0)
    monkeypatch.setattr(F, "_lib", Fake())
    q, table = torch.zeros(90, 8, 64, dtype=torch.bfloat16), torch.zeros(5, 3, dtype=torch.int32)
    ws = F.mx_kv_attention_workspace(cache, q, table)
    assert ws.numel() == 70000 and not ws[:F.WORKSPACE_ZEROED].any()
    assert {a[3] for a in asked} == {2, 4, 6, 8, 90}           # rows: 8, 16, 24, 32 and all, four per query
    assert {a[:3] + a[4:] for a in asked} == {(90, 8, 5, 3)}
    assert F.mx_kv_attention_workspace(cache, q, table, max_q=1).numel() == 20000
    assert F.mx_kv_attention_workspace(cache, q, table, max_q=3) is None
    Fake.sizes = {90: -3, 8: 70000}
    with pytest.raises(F.Fp8qError) as e:
        F.mx_kv_attention_workspace(cache, q, table)
    assert e.value.status == -3
