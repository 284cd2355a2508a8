"""The cache in 8 bits and the rotary positions without a GPU: refusals on the host before anything
is enqueued, the definition's own pieces, and the frequencies."""
import builtins
import ctypes
import math
import os
import sys
import warnings

import numpy as np
import pytest
import torch

import kv_cache_eviction_gb300 as kv
from kv_cache_eviction_gb300 import _build
from tests.quant import E4M3, nearest, numbers, put, scale_for


@pytest.fixture(scope="module")
def L():
    _build.build()
    return kv.lib()


P = ctypes.c_void_p(0x1000)
ODD4, ODD2 = ctypes.c_void_p(0x1004), ctypes.c_void_p(0x1002)
BIG = 1 << 40
INV, FAR, OK = kv.KV_ERR_INVALID_ARG, kv.KV_ERR_UNSUPPORTED, kv.KV_OK


def shape(**kw):
    base = dict(seqs=4, hq=32, hkv=8, d=128, tables=1, page=16, max_pages=64, dtype="bf16",
                num_pages=1000)
    base.update(kw)
    return kv.KvPagedShape.of(**base)


def call_write(L, s, fmt=0, k=P, v=P, stride=0, slots=P, rows=10, n_rows=None, kp=P, vp=P, ks=P,
               vs=P, ws=P, n=BIG):
    return L.kv_quant_write(ctypes.byref(s) if s else None, fmt, k, v, stride, slots, rows, n_rows,
                            kp, vp, ks, vs, ws, n, None)


def call_read(L, s, fmt=0, k=P, v=P, stride=0, slots=P, rows=10, n_rows=None, kp=P, vp=P, ks=P,
              vs=P, ws=P, n=BIG):
    return L.kv_quant_read(ctypes.byref(s) if s else None, fmt, kp, vp, ks, vs, slots, rows, n_rows,
                           k, v, stride, ws, n, None)


def call_decode(L, s, fmt=0, q=P, kn=P, vn=P, cu=P, slots=P, cap=10, kp=P, vp=P, ks=P, vs=P,
                table=P, lens=P, scale=0.1, out=P, ws=P, n=BIG):
    return L.quant_decode_attn(ctypes.byref(s) if s else None, fmt, q, kn, vn, cu, slots, cap, kp,
                               vp, ks, vs, table, lens, scale, out, ws, n, None)


ROWS = ((call_write, kv.KV_OP_QUANT_WRITE), (call_read, kv.KV_OP_QUANT_READ))


@pytest.mark.parametrize("bad", [
    dict(seqs=-1), dict(hq=30), dict(hq=0), dict(d=100), dict(d=0), dict(tables=2), dict(page=0),
    dict(max_pages=0), dict(num_pages=0), dict(dtype=7), dict(page_stride=8 * 16 * 128 - 16),
    dict(page_stride=8 * 16 * 128 + 8), dict(page_stride=-16)])
def test_invalid_shapes(L, bad):
    for call, op in ROWS + ((call_decode, kv.KV_OP_QUANT_DECODE),):
        assert call(L, shape(**bad)) == INV
        assert kv.kv_paged_workspace_size(op, shape(**bad)) == 0


@pytest.mark.parametrize("far", [
    dict(hq=128), dict(d=136), dict(d=72), dict(d=8), dict(hq=512, hkv=512), dict(page=8),
    dict(page=24), dict(page=512), dict(max_pages=1 << 28), dict(num_pages=1 << 31),
    dict(page_stride=1 << 40), dict(seqs=1 << 29)])
def test_unsupported_shapes(L, far):
    for call, op in ROWS + ((call_decode, kv.KV_OP_QUANT_DECODE),):
        assert call(L, shape(**far)) == FAR
        assert kv.kv_paged_workspace_size(op, shape(**far)) == 0


def test_page_stride_is_in_bytes(L):
    """A stride of 16 bytes more than dense pages is a legal one for either row type."""
    for dtype in ("bf16", "f32"):
        s = shape(dtype=dtype, page_stride=8 * 16 * 128 + 16)
        for call, op in ROWS + ((call_decode, kv.KV_OP_QUANT_DECODE),):
            assert call(L, s, n=0) == kv.KV_ERR_WORKSPACE


def test_row_arguments(L):
    s = shape()
    for call, op in ROWS:
        assert call(L, None) == INV
        for fmt in (-1, 2):
            assert call(L, s, fmt=fmt) == INV
        for arg in ("k", "v", "slots", "kp", "vp", "ks", "vs", "ws"):
            assert call(L, s, **{arg: None}) == INV
            assert call(L, s, **{arg: ODD2}) == INV
        for arg in ("k", "v", "slots", "kp", "vp", "ws", "n_rows"):
            assert call(L, s, **{arg: ODD4}) == INV
        assert call(L, s, rows=-1) == INV
        assert call(L, s, rows=1 << 31) == INV
        for stride in (-8, 8 * 128 - 8, 8 * 128 + 4, 1 << 33):
            assert call(L, s, stride=stride) == INV
        n = kv.kv_paged_workspace_size(op, s)
        assert n >= 256 and call(L, s, n=n - 1) == kv.KV_ERR_WORKSPACE
        assert call(L, s, ks=ODD4, vs=ODD4, n=n - 1) == kv.KV_ERR_WORKSPACE   # 4 bytes suffice
        # nothing to do
        assert call(L, s, 0, None, None, 0, None, 0, None, None, None, None, None) == OK
        assert call(L, shape(seqs=0), 0, None, None, 0, None, 10, None, None, None, None,
                    None) == OK
        assert call(L, shape(seqs=0), rows=-1) == INV


def test_decode_arguments(L):
    s = shape()
    assert call_decode(L, None) == INV
    for fmt in (-1, 2):
        assert call_decode(L, s, fmt=fmt) == INV
    for arg in ("q", "kp", "vp", "ks", "vs", "table", "lens", "out", "ws"):
        assert call_decode(L, s, **{arg: None}) == INV
        assert call_decode(L, s, **{arg: ODD2}) == INV
    for arg in ("q", "kp", "vp", "kn", "vn", "out", "cu", "slots"):
        assert call_decode(L, s, **{arg: ODD4}) == INV
    for arg in ("kn", "vn", "cu", "slots"):
        assert call_decode(L, s, **{arg: None}) == INV
    assert call_decode(L, s, cap=-1) == INV
    for scale in (math.inf, math.nan, 2.0 ** 127, -2.0 ** 127):
        assert call_decode(L, s, scale=scale) == INV
    n = kv.kv_paged_workspace_size(kv.KV_OP_QUANT_DECODE, s)
    assert call_decode(L, s, n=n - 1) == kv.KV_ERR_WORKSPACE
    assert call_decode(L, s, scale=-1.7e38, n=n - 1) == kv.KV_ERR_WORKSPACE
    assert call_decode(L, shape(seqs=1 << 11, max_pages=1 << 16)) == FAR     # 2^31 tiles of 8 rows
    far = shape(seqs=kv.KV_PAGED_DECODE_MAX_TABLES + 1, max_pages=1, hkv=1, hq=1)
    assert call_decode(L, far) == FAR
    assert call_decode(L, shape(seqs=0), 0, None, None, None, None, None, 0, None, None, None, None,
                       None, None, 0.1, None) == OK


def rotary_shape(**kw):
    base = dict(hq=32, hkv=8, d=128, rot=128, layout=kv.KV_ROTARY_HALF, dtype="bf16")
    base.update(kw)
    return kv.KvRotaryShape.of(**base)


A, B, C, D = (ctypes.c_void_p(x << 32) for x in (1, 2, 3, 4))


def call_rotary(L, s, back=0, q=A, qs=0, k=B, ks=0, pos=P, freq=P, rows=10, n_rows=None, qo=C,
                qos=0, ko=D, kos=0):
    return L.kv_rotary(ctypes.byref(s) if s else None, back, q, qs, k, ks, pos, freq, rows, n_rows,
                       qo, qos, ko, kos, None)


def test_rotary_refusals(L):
    s = rotary_shape()
    assert call_rotary(L, None) == INV
    for bad in (dict(hq=-1), dict(hkv=-1), dict(hq=0, hkv=0), dict(d=0), dict(d=100), dict(rot=0),
                dict(rot=136), dict(rot=7), dict(layout=2), dict(layout=-1), dict(dtype=5),
                dict(magnitude=math.inf), dict(magnitude=math.nan)):
        assert call_rotary(L, rotary_shape(**bad)) == INV, bad
    for far in (dict(d=264, rot=64), dict(rot=12), dict(hq=4097), dict(hkv=4097)):
        assert call_rotary(L, rotary_shape(**far)) == FAR, far
    for arg in ("q", "k", "qo", "ko", "pos", "freq"):
        assert call_rotary(L, s, **{arg: None}) == INV
        assert call_rotary(L, s, **{arg: ODD2}) == INV
    for arg in ("q", "k", "qo", "ko", "freq", "n_rows"):
        assert call_rotary(L, s, **{arg: ODD4}) == INV
    assert call_rotary(L, s, rows=-1) == INV
    assert call_rotary(L, s, rows=1 << 31) == INV
    for arg, heads in (("qs", 32), ("ks", 8), ("qos", 32), ("kos", 8)):
        for stride in (-8, heads * 128 - 8, heads * 128 + 4, 1 << 33):
            assert call_rotary(L, s, **{arg: stride}) == INV
    # an output over a part of its input, or in place with another stride
    at = lambda p, n: ctypes.c_void_p(p.value + n)
    for far in (16, 2 * 32 * 128, 10 * 2 * 32 * 128 - 16):
        assert call_rotary(L, s, qo=at(A, far)) == INV
        assert call_rotary(L, s, qo=at(A, -far)) == INV
    assert call_rotary(L, s, ko=at(B, 16)) == INV
    assert call_rotary(L, s, qo=A, qos=32 * 128 + 8) == INV
    # ranges of 2^62 elements are no overflow
    big = dict(rows=(1 << 31) - 1, qs=1 << 31, qos=1 << 31)
    assert call_rotary(L, s, qo=at(A, 1 << 60), **big) == INV
    assert call_rotary(L, s, qo=at(A, 16), **big) == INV
    # nothing to do; no k, no q
    assert call_rotary(L, s, 0, None, 0, None, 0, None, None, 0, None, None, 0, None, 0) == OK
    assert call_rotary(L, rotary_shape(hkv=0), k=None, ko=None, rows=0) == OK
    assert call_rotary(L, rotary_shape(hkv=0), q=None, k=None, ko=None) == INV


def test_binding_refuses_host_tensors(L):
    s = shape(seqs=1)
    i = torch.zeros(2000, dtype=torch.int64)
    t = torch.zeros(1000, 8, 16, 128, dtype=torch.int8)
    f, r = torch.zeros(8000), torch.zeros(10, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        kv.kv_quant_write(s, kv.KV_INT8, r, r, i, None, t, t, f, f, i)
    with pytest.raises(ValueError):
        kv.kv_quant_read(s, kv.KV_INT8, t, t, f, f, i, None, r, r, i)
    with pytest.raises(ValueError):
        kv.quant_decode_attn(s, kv.KV_INT8, r, None, None, None, None, t, t, f, f, i.int(), i.int(),
                             0.1, r, i)
    with pytest.raises(ValueError):
        kv.kv_rotary(rotary_shape(), r, r, i.int(), f.double(), r, r)


def test_binding_code_types():
    """Pools come as the format's own type, or for e4m3 as bytes; any other raises."""
    kv._CODES.update({kv.KV_E4M3: (torch.float8_e4m3fn, torch.uint8), kv.KV_INT8: (torch.int8,)})
    u = torch.zeros(4, 2, 16, 32, dtype=torch.uint8)
    ok = lambda t, fmt: kv._code_pool(t, fmt, 2 * 16 * 32, 4, 2 * 16 * 32, -1, "k_pages")
    assert ok(u, kv.KV_E4M3) == u.data_ptr() == ok(u.view(torch.float8_e4m3fn), kv.KV_E4M3)
    assert ok(u.view(torch.int8), kv.KV_INT8) == u.data_ptr()
    for t, fmt in ((u.view(torch.int8), kv.KV_E4M3), (u, kv.KV_INT8),
                   (u.view(torch.float8_e5m2), kv.KV_E4M3), (u, 2), (u[:3], kv.KV_E4M3),
                   (u.view(torch.float8_e4m3fn), kv.KV_INT8), (u.float(), kv.KV_E4M3)):
        with pytest.raises(ValueError):
            ok(t, fmt)


def test_the_definitions_own_pieces():
    """The tests' codes: e4m3's numbers are torch's, nearest() is the nearest of all, and a scale
    is the least that holds the values."""
    c = torch.arange(256, dtype=torch.uint8)
    t = c.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(E4M3, t, equal_nan=True)
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.normal(size=500) * np.exp(rng.uniform(-8, 6, 500)),
                        np.arange(-40, 40) / 512])
    fine = np.unique(E4M3[~np.isnan(E4M3)])
    for all_, fmt in ((fine, "e4m3"), (np.arange(-127.0, 128), "int8")):
        y = nearest(x, fmt)
        best = np.abs(all_[None] - np.clip(x, all_[0], all_[-1])[:, None]).min(1)
        assert np.isin(y, all_).all()
        assert np.allclose(np.abs(y - np.clip(x, all_[0], all_[-1])), best, rtol=0, atol=0)
    z = torch.tensor(x).float()
    assert np.array_equal(nearest(z.double().numpy(), "e4m3"),
                          z.clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy())
    assert scale_for([448.0], "e4m3") == 1 and scale_for([448.1], "e4m3") == 2
    assert scale_for([127.0], "int8") == 1 and scale_for([-127.1, np.nan, np.inf], "int8") == 2
    assert scale_for([0.0], "e4m3") == scale_for([np.nan], "int8") == 2.0 ** -96
    # rows of a block in one call, or held ones moved to a larger scale
    num, sc = np.zeros((1, 1, 16, 2)), np.full((1, 1, 1), np.nan)
    put(num, sc, np.array([[[3.0, 1]], [[100, -7]]]), [0, 1], "int8")
    assert sc[0, 0, 0] == 1 and (num[0, 0, :2] == [[3, 1], [100, -7]]).all()
    put(num, sc, np.array([[[508.0, 2]]]), [2], "int8")
    assert sc[0, 0, 0] == 4 and (num[0, 0, :3] == [[1, 0], [25, -2], [127, 0]]).all()
    assert numbers(torch.tensor([1, 255], dtype=torch.uint8), "int8").tolist() == [1, -1]


def test_rotary_frequencies():
    f, m = kv.kv_rotary_inv_freq(64, 10000.0)
    assert f.dtype == torch.float64 and m == 1.0 and len(f) == 32
    assert torch.allclose(f, torch.tensor([10000.0 ** (-2 * i / 64) for i in range(32)],
                                          dtype=torch.float64), rtol=1e-14)
    lin = kv.kv_rotary_inv_freq(64, 10000.0, "linear", 8.0)[0]
    assert torch.allclose(lin * 8, f, rtol=1e-15)
    b = kv.kv_rotary_inv_freq(64, 10000.0, "base", 8.0)[0]
    assert float(b[0]) == 1.0 and abs(float(b[-1] * 8 / f[-1]) - 1) < 1e-12
    turns = 8192 * f / (2 * math.pi)
    for kind in ("bands", "yarn"):
        y, m = kv.kv_rotary_inv_freq(64, 10000.0, kind, 8.0, trained=8192, slow=1.0, fast=32.0)
        assert torch.equal(y[turns > 40], f[turns > 40])
        assert torch.allclose(y[turns < 0.7], lin[turns < 0.7], rtol=1e-15)
        between = (turns > 2) & (turns < 20)
        assert bool(((y > lin) & (y < f))[between].all())
        assert bool((y[1:] < y[:-1]).all())
        assert m == (0.1 * math.log(8.0) + 1 if kind == "yarn" else 1.0)
    # a pair of the middle, by hand: 2048 positions, slow 1, fast 4
    y = kv.kv_rotary_inv_freq(4, 1024.0, "bands", 2.0, trained=2048, slow=1.0, fast=100.0)[0]
    n = 2048 / 32 / (2 * math.pi)
    w = (n - 1) / 99
    assert abs(float(y[1]) - (w + (1 - w) / 2) / 32) < 1e-15 and float(y[0]) == 1.0
    for bad in (dict(rot=0), dict(rot=7), dict(base=1.0), dict(factor=0.5), dict(scaling="other"),
                dict(slow=2.0, fast=2.0), dict(trained=0), dict(rot=2, scaling="base")):
        with pytest.raises(ValueError):
            kv.kv_rotary_inv_freq(**{"rot": 64, **bad})


@pytest.mark.parametrize("what", ["torch", "python", "no stamp"])
def test_fast_module_for_another_torch_is_not_loaded(L, monkeypatch, tmp_path, what):
    """_fast.so reads tensors by their layout: with another torch or Python than it was built for,
    or where that is not known, calls go through ctypes, with a warning."""
    if not os.path.exists(_build.FAST):
        pytest.skip("no _fast.so")
    with monkeypatch.context() as m:
        m.setattr(kv, "_quick", None)
        if what == "torch":
            m.setattr(torch, "__version__", "1.0.0")
        elif what == "python":
            m.setattr(sys, "version", "3.99")
        else:
            m.setattr(_build, "STAMP", str(tmp_path / "none.txt"), raising=False)
        with pytest.warns(UserWarning, match="_fast.so"):
            kv._init_fast()
        assert kv._quick is None
    with monkeypatch.context() as m, warnings.catch_warnings():
        warnings.simplefilter("error")
        m.setattr(kv, "_quick", None)
        kv._init_fast()
        assert kv._quick is not None


@pytest.mark.parametrize("error", [ImportError, OSError, RuntimeError])
def test_build_with_a_torch_that_does_not_load(monkeypatch, tmp_path, capsys, error):
    """The library is built without torch; one that fails to load is said, not raised."""
    real = builtins.__import__

    def fails(name, *args, **kw):
        if name == "torch":
            raise error("libtorch_cpu.so: cannot open")
        return real(name, *args, **kw)

    monkeypatch.setattr(_build, "FAST", str(tmp_path / "_fast.so"))
    monkeypatch.setattr(builtins, "__import__", fails)
    _build._build_fast()
    monkeypatch.undo()
    said = "cannot open" in capsys.readouterr().err
    assert said == (error is not ImportError)


def test_yarn_where_every_pair_makes_a_turn():
    """The ramp ends at the pair of `slow` turns also where that lies behind the last one, as for long
    trained lengths on a small base: here pair(turns) = 64 ln(131072 / (2 pi turns)) / ln(10000) is 69.1
    for one turn and 45.03 for 32, so the ramp is from 45 to 70 and pair i is (i - 45) / 25 of the way."""
    f = kv.kv_rotary_inv_freq(128, 10000.0)[0]
    y = kv.kv_rotary_inv_freq(128, 10000.0, "yarn", 4.0, trained=131072)[0]
    i = torch.arange(64, dtype=torch.float64)
    w = ((i - 45) / 25).clamp(0, 1)
    assert torch.allclose(y, f * (1 - w) + f / 4 * w, rtol=1e-14)
    # before the first pair it does not begin: no pair of 200 positions makes 32 turns but the first
    y = kv.kv_rotary_inv_freq(8, 10000.0, "yarn", 4.0, trained=128, slow=1.0, fast=32.0)[0]
    f = kv.kv_rotary_inv_freq(8, 10000.0)[0]
    w = (torch.arange(4, dtype=torch.float64) / 2).clamp(0, 1)   # pair(32) = -0.2, pair(1) = 1.3
    assert torch.allclose(y, f * (1 - w) + f / 4 * w, rtol=1e-14)
