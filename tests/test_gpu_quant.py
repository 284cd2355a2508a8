"""The cache in 8 bits on the GPU: rows written and read back, against the definition in 64 bits,
code by code and scale by scale."""
import numpy as np
import pytest
import torch

import kv_cache_eviction_gb300 as kv
from tests.paged import ERR_ID, ceil_div, workspace
from tests.quant import BLOCK, FORMATS, Pool, nearest, scale_for

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kv_cache_eviction_gb300 import _build
    _build.build()
    kv.lib()
    kv._init_torch()


def i64(x):
    return torch.tensor(np.asarray(x), dtype=torch.int64, device="cuda")


def shape_of(pool, dtype, tables=1, hkv=None):
    num, heads, page, d = pool.size
    hkv = heads * tables if hkv is None else hkv
    return kv.KvPagedShape.of(1, hkv, hkv, d, tables, page, num, dtype, num, pool.page_stride)


def runs(rng, num, page, rows):
    """Slots of runs of all lengths at random places: every page is one table's."""
    slots, pages = [], list(rng.permutation(num))
    while len(slots) < rows and pages:
        n = int(rng.integers(1, 3 * page + 2)) if rng.random() < 0.6 else 1
        at = int(rng.integers(0, page))
        while n > 0 and pages:
            p, m = int(pages.pop()), min(n, page - at)
            slots += range(p * page + at, p * page + at + m)
            n, at = n - m, 0
        if rng.random() < 0.3:
            slots.append(-1)
    return np.array(slots[:rows])


def rows_of(seed, n, heads, d, dtype):
    g = torch.Generator().manual_seed(seed)
    size = lambda: torch.exp(2 * torch.randn(2, n, 1, 1, generator=g))
    return (torch.randn(2, n, heads, d, generator=g) * size()).to(DT[dtype])


def write(pool, shape, k, v, slots, n_rows=None, ws=None, stream=None):
    ws = workspace(kv.KV_OP_QUANT_WRITE, shape) if ws is None else ws
    kv.kv_quant_write(shape, FORMATS[pool.fmt], k, v, i64(slots), n_rows, *pool.args(), ws, stream)
    return ws


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,heads,tables,d,page,fused,extra", [
    (1, 8, 1, 128, 16, True, 0), (77, 2, 1, 48, 16, False, 64), (600, 1, 8, 128, 64, False, 0),
    (513, 3, 1, 16, 256, True, 128), (2050, 4, 1, 96, 32, True, 0), (3001, 1, 2, 64, 16, False, 16),
    (9, 8, 1, 80, 128, False, 0), (300, 5, 1, 112, 32, True, 4096), (5000, 8, 1, 32, 16, True, 0)])
def test_write(fmt, dtype, rows, heads, tables, d, page, fused, extra):
    rng = np.random.default_rng(rows + d)
    num = ceil_div(2 * rows, page) + 3
    slots = runs(rng, num, page, rows)
    n = len(slots)
    x = rows_of(rows, n, heads, d, dtype)
    if fused:
        wide = torch.zeros(n, 3 * heads, d, dtype=DT[dtype], device="cuda")
        wide[:, heads:2 * heads], wide[:, 2 * heads:] = x[0].cuda(), x[1].cuda()
        k, v = wide[:, heads:2 * heads], wide[:, 2 * heads:]
    else:
        k, v = x[0].cuda(), x[1].cuda()
    for limit in (None, 0, n // 2, n + 5, -4):
        pool = Pool(num, heads, page, d, fmt, rows, extra)
        s = shape_of(pool, dtype, tables)
        ws = write(pool, s, k, v, slots, None if limit is None else i64([limit]))
        m = n if limit is None else max(0, min(n, limit))
        pool.put(*x[:, :m].double().numpy(), slots[:m])
        pool.check()
        assert kv.kv_check_device_status(ws) == 0


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_row_by_row(fmt, dtype):
    """Rows that come one by one: a block's scale only rises, its rows are rounded to it, and a
    block begun anew forgets what it had (a scale of NaN too)."""
    pool = Pool(6, 2, 32, 64, fmt, 3, scales=float("nan"))
    s = shape_of(pool, dtype)
    x = rows_of(5, 150, 2, 64, dtype)
    x[:, 40:80] *= torch.exp2(torch.arange(-20, 20)).view(1, -1, 1, 1).to(x.dtype)
    ws = workspace(kv.KV_OP_QUANT_WRITE, s)
    slots = np.concatenate([np.arange(64, 144), np.arange(64, 110), np.arange(0, 24)])
    for i, slot in enumerate(slots):
        write(pool, s, x[0, i:i + 1].cuda(), x[1, i:i + 1].cuda(), [slot], ws=ws)
        pool.put(*x[:, i:i + 1].double().numpy(), [slot])
    pool.check()
    assert kv.kv_check_device_status(ws) == 0


def special_rows(dtype):
    """Rows that try the borders of scales and codes."""
    d = 64
    top = 2.0 ** 126
    rows = [np.zeros(d), np.full(d, np.inf), np.full(d, np.nan), np.full(d, 1e-45),
            np.full(d, 2.0 ** -96 * 448), np.full(d, 2.0 ** -105), np.full(d, -top),
            np.linspace(-1, 1, d), 448.0 * 2.0 ** (np.arange(d) - 60.0),
            127.0 * 2.0 ** (np.arange(d) - 60.0), 2.0 ** (np.arange(d) - 63.0) * 1.75,
            np.where(np.arange(d) % 3 == 0, -np.inf, np.arange(d) / 7),
            np.where(np.arange(d) % 5 == 0, np.nan, np.arange(d) - 20.0),
            # halves between neighbouring codes of both formats, odd and even
            np.concatenate([np.arange(31) + 0.5, [127.0], (np.arange(32) + 8.5) / 16])]
    rows += [np.concatenate([[m], np.full(d - 1, 0.5)]) for m in
             (447, 448, 448.5, 449, 450, 127, 127.25, 127.5, 128, 1.75, 1.7578125, 1.984375,
              1.9921875)]
    return torch.tensor(np.array(rows)).to(DT[dtype])


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_write_specials(fmt, dtype):
    """Zeros, infinities, NaN, the smallest and the largest values, borders between scales and
    halves between codes: each row in a block of its own, then all in common blocks."""
    x = special_rows(dtype)
    n = len(x)
    for slots in (np.arange(n) * BLOCK, np.arange(n), np.arange(n) + 11):
        pool = Pool(ceil_div(n * BLOCK, 32) + 1, 1, 32, 64, fmt, 4)
        s = shape_of(pool, dtype)
        k, v = x.view(n, 1, 64), x.flip(0).view(n, 1, 64)
        ws = write(pool, s, k.cuda(), v.cuda(), slots)
        pool.put(k.double().numpy(), v.double().numpy(), slots)
        pool.check()
        assert kv.kv_check_device_status(ws) == 0


def test_error_of_a_value():
    """What a value is off by, as the header states it."""
    rng = np.random.default_rng(2)
    x = rng.normal(size=(400, 16, 32)) * np.exp(3 * rng.normal(size=(400, 1, 1)))
    for fmt in ("e4m3", "int8"):
        for block in x:
            s = scale_for(block, fmt)
            off = np.abs(nearest(block / s, fmt) * s - block)
            if fmt == "e4m3":
                assert (off <= np.maximum(2.0 ** -4 * np.abs(block), 2.0 ** -10 * s)).all()
            else:
                assert (off <= s / 2).all() and s / 2 < 2.0 ** -6 * np.abs(block).max()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_write_bad_slots(fmt):
    """Slots outside the pool are skipped and reported; the rows around them are stored."""
    pool = Pool(4, 2, 16, 64, fmt, 5)
    s = shape_of(pool, "bf16")
    x = rows_of(1, 8, 2, 64, "bf16")
    slots = [3, 64, -2, 1 << 62, -(1 << 62), 62, 63, 64]
    ws = write(pool, s, x[0].cuda(), x[1].cuda(), slots)
    assert kv.kv_check_device_status(ws) == ERR_ID
    assert kv.kv_check_device_status(ws) == 0
    pool.put(*x.double().numpy(), slots)
    pool.check()


@pytest.mark.parametrize("many", [1, 400])
def test_write_slots_astray(many):
    """A row whose neighbour is of its block but not the row before it there (a gap, a step back,
    the same slot again) is skipped with what follows on from it, and reported; the rest is stored."""
    one = [5, 7, 8, 40, 39, 70, 70, 71, 100, 101, 103, 112, 160, 175, 176, 177, 200, 199, 200, 201]
    kept = [0, 3, 5, 8, 9, 11, 12, 14, 15, 16]
    slots = np.concatenate([np.array(one) + 256 * i for i in range(many)])
    keep = np.concatenate([np.array(kept) + len(one) * i for i in range(many)])
    pool = Pool(16 * many, 2, 16, 64, "int8", 7)
    s = shape_of(pool, "bf16")
    x = rows_of(2, len(slots), 2, 64, "bf16")
    ws = write(pool, s, x[0].cuda(), x[1].cuda(), slots)
    assert kv.kv_check_device_status(ws) == ERR_ID
    left = np.full(len(slots), -1)
    left[keep] = slots[keep]
    pool.put(*x.double().numpy(), left)
    pool.check()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,heads,tables,d,page,fused,extra", [
    (1, 8, 1, 128, 16, True, 0), (77, 2, 1, 48, 16, False, 64), (600, 1, 8, 128, 64, False, 0),
    (513, 3, 1, 16, 256, True, 128), (2050, 4, 1, 96, 32, True, 0), (700, 8, 1, 112, 32, False, 0)])
def test_read(fmt, dtype, rows, heads, tables, d, page, fused, extra):
    """Any slots, repeated ones and -1 among them; rows behind the last and around a destination
    that is part of wider rows are left as they were.  Values are exact."""
    rng = np.random.default_rng(rows)
    num = ceil_div(rows, page) + 2
    pool = Pool(num, heads, page, d, fmt, rows, extra)
    s = shape_of(pool, dtype, tables)
    slots = rng.integers(0, num * page, rows)
    slots[rng.random(rows) < 0.1] = -1
    p, r = slots // page, slots % page
    want = [torch.tensor(pool.values(name)[p, :, r]).to(DT[dtype]) for name in ("k", "v")]
    for limit in (None, 0, rows // 2, rows + 5, -4):
        wide = torch.full((rows, 3 if fused else 2, heads, d), 7.0, dtype=DT[dtype], device="cuda")
        k, v = (wide[:, 1], wide[:, 2]) if fused else (wide[:, 0].clone(), wide[:, 1].clone())
        ws = workspace(kv.KV_OP_QUANT_READ, s)
        kv.kv_quant_read(s, FORMATS[fmt], *pool.args(), i64(slots),
                         None if limit is None else i64([limit]), k, v, ws)
        m = rows if limit is None else max(0, min(rows, limit))
        keep = torch.tensor((slots >= 0) & (np.arange(rows) < m))
        for got, x in zip((k, v), want):
            ref = torch.full_like(x, 7.0)
            ref[keep] = x[keep]
            assert torch.equal(got.cpu(), ref)
        if fused:
            assert bool((wide[:, 0] == 7.0).all())
        assert kv.kv_check_device_status(ws) == 0
        pool.check()


def test_read_bad_slots():
    pool = Pool(4, 2, 16, 64, "e4m3", 5)
    s = shape_of(pool, "f32")
    out = torch.full((2, 6, 2, 64), 7.0, device="cuda")
    ws = workspace(kv.KV_OP_QUANT_READ, s)
    kv.kv_quant_read(s, kv.KV_E4M3, *pool.args(), i64([63, 64, -2, 1 << 62, -(1 << 62), 0]), None,
                     out[0], out[1], ws)
    assert kv.kv_check_device_status(ws) == ERR_ID
    for got, name in zip(out.cpu().double().numpy(), ("k", "v")):
        x = pool.values(name)
        assert np.array_equal(got[0], x[3, :, 15]) and np.array_equal(got[5], x[0, :, 0])
        assert (got[1:5] == 7.0).all()


def test_read_nan_and_the_range_of_scales():
    """A NaN code is a NaN; the largest and the smallest scale keep every code exact."""
    pool = Pool(2, 1, 16, 16, "e4m3", 6)
    pool.dev["k"].view(torch.uint8)[0, 0, 3, 5] = 127
    pool.dev["k"].view(torch.uint8)[0, 0, 3, 6] = 255
    pool.scale_dev["v"][0, 0, 0], pool.scale_dev["v"][1, 0, 0] = 2.0 ** -96, 2.0 ** 118
    s = shape_of(pool, "bf16")
    out = torch.zeros(2, 32, 1, 16, dtype=torch.bfloat16, device="cuda")
    kv.kv_quant_read(s, kv.KV_E4M3, *pool.args(), i64(np.arange(32)), None, out[0], out[1],
                     workspace(kv.KV_OP_QUANT_READ, s))
    k = out[0].cpu().view(2, 16, 16)
    assert bool(torch.isnan(k[0, 3, 5:7]).all()) and int(torch.isnan(k).sum()) == 2
    want = pool.num["v"][:, 0] * np.array([2.0 ** -96, 2.0 ** 118])[:, None, None]
    assert np.array_equal(out[1].cpu().double().numpy().reshape(2, 16, 16), want)


def test_far_pages():
    """Bytes past 2^32 of a pool, and slots past 2^32."""
    num, heads, page, d = 1200, 128, 256, 128
    assert num * heads * page * d > 1 << 32
    kp = torch.zeros(num, heads, page, d, dtype=torch.int8, device="cuda")
    vp = torch.zeros_like(kp)
    ks, vs = (torch.zeros(num, heads, page // 16, device="cuda") for _ in range(2))
    s = kv.KvPagedShape.of(1, heads, heads, d, 1, page, num, "bf16", num)
    x = rows_of(8, 4, heads, d, "bf16").cuda()
    at = [0, num * page - 1, (num - 2) * page + 5, 17 * page]
    ws = workspace(kv.KV_OP_QUANT_WRITE, s)
    kv.kv_quant_write(s, kv.KV_INT8, x[0], x[1], i64(at), None, kp, vp, ks, vs, ws)
    out = torch.zeros_like(x)
    kv.kv_quant_read(s, kv.KV_INT8, kp, vp, ks, vs, i64(at), None, out[0], out[1], ws)
    assert kv.kv_check_device_status(ws) == 0
    for t in range(2):
        for i in range(4):
            for h in (0, heads - 1):
                r = x[t, i, h].double().cpu().numpy()
                sc = scale_for(r, "int8")
                assert np.array_equal(out[t, i, h].double().cpu().numpy(),
                                      nearest(r / sc, "int8") * sc)
    for pool in (kp, vp):
        for a in at:
            assert bool(pool[a // page, :, a % page].any())
            pool[a // page, :, a % page] = 0
        assert not bool(pool.view(torch.int64).any())


def test_captured_on_another_stream():
    """A captured write and read-back, replayed with other rows and slots."""
    pool = Pool(9, 2, 32, 64, "e4m3", 9)
    s = shape_of(pool, "bf16")
    side = torch.cuda.Stream()
    x = torch.zeros(2, 40, 2, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(x)
    slots, n = i64(np.full(40, -1)), i64([40])
    ws = workspace(kv.KV_OP_QUANT_WRITE, s)

    def step(stream=None):
        kv.kv_quant_write(s, kv.KV_E4M3, x[0], x[1], slots, n, *pool.args(), ws, stream)
        kv.kv_quant_read(s, kv.KV_E4M3, *pool.args(), slots, n, out[0], out[1], ws, stream)

    side.wait_stream(torch.cuda.current_stream())
    step(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step()
    rng = np.random.default_rng(3)
    for i in range(4):
        y, at, m = rows_of(i, 40, 2, 64, "bf16"), runs(rng, 9, 32, 40), 40 - 7 * i
        at = np.concatenate([at, np.full(40 - len(at), -1)])
        x.copy_(y)
        slots.copy_(i64(at))
        n.fill_(m)
        g.replay()
        torch.cuda.synchronize()
        pool.put(*y[:, :m].double().numpy(), at[:m])
        pool.check()
        for got, name in zip(out.cpu().double().numpy(), ("k", "v")):
            for j in range(m):
                if at[j] >= 0:
                    assert np.array_equal(got[j], pool.values(name)[at[j] // 32, :, at[j] % 32])
    assert kv.kv_check_device_status(ws) == 0


def test_compacted_rows_of_head_tables():
    """kv_page_map's slots for tables of a head each, with rows laid out as kv_compact leaves
    them: written in two steps, the second from the middle of blocks on."""
    hkv, page, d, cols = 8, 32, 64, 12
    rng = np.random.default_rng(11)
    num = hkv * cols
    pool = Pool(num, 1, page, d, "int8", 12)
    s = kv.KvPagedShape.of(1, hkv, hkv, d, hkv, page, cols, "bf16", num)
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")
    lens, ring, state = i32(np.zeros(hkv)), i32(rng.permutation(num)), i64([0, num])
    table, cu = i32(np.zeros((hkv, cols))), i64(np.zeros(hkv + 1))
    wm = workspace(kv.KV_OP_PAGE_MAP, s)
    for step in range(2):
        add = rng.integers(0, 150, hkv)
        n = int(add.sum())
        slots = i64(np.full(n, -1))
        kv.kv_page_map(s, lens, i32(add), ring, state, table, lens, state, cu, slots, wm)
        x = rows_of(20 + step, n, 1, d, "bf16")
        write(pool, s, x[0].cuda(), x[1].cuda(), slots.cpu().numpy(), cu[hkv:], ws=wm)
        assert kv.kv_check_device_status(wm) == 0
        pool.put(*x.double().numpy(), slots.cpu().numpy())
        pool.check()


def each_call(fmt="int8", dtype="bf16"):
    """The four calls on small tensors: name, function and arguments."""
    pool = Pool(6, 2, 16, 32, fmt, 30)
    s = shape_of(pool, dtype)
    s.seqs, s.max_pages = 3, 2
    x = rows_of(31, 9, 2, 32, dtype).cuda()
    ws = workspace(kv.KV_OP_QUANT_DECODE, s)
    table = torch.tensor([[0, 1], [2, 3], [4, 5]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([20, 1, 32], dtype=torch.int32, device="cuda")
    cu, slots = i64([0, 1, 2, 3]), i64([19, 32, 95])
    rot = kv.KvRotaryShape.of(2, 2, 32, 16, kv.KV_ROTARY_HALF, dtype)
    freq = kv.kv_rotary_inv_freq(16)[0].cuda()
    f = FORMATS[fmt]
    out = lambda n: torch.zeros(n, 2, 32, dtype=DT[dtype], device="cuda")
    return [("kv_quant_write", kv.kv_quant_write,
             [s, f, x[0], x[1], i64(np.arange(9) + 20), None, *pool.args(), ws]),
            ("kv_quant_read", kv.kv_quant_read,
             [s, f, *pool.args(), i64(np.arange(9)), i64([8]), out(9), out(9), ws]),
            ("quant_decode_attn", kv.quant_decode_attn,
             [s, f, x[0, :3].clone(), x[0, 3:6].clone(), x[1, :3].clone(), cu, slots, *pool.args(),
              table, lens, 0.3, out(3), ws]),
            ("kv_rotary", kv.kv_rotary,
             [rot, x[0], x[1], torch.arange(9, dtype=torch.int32, device="cuda"), freq, out(9),
              out(9)])]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_both_ways_of_the_binding(monkeypatch, fmt, dtype):
    """The binding's common case in C++ and its Python code do the same."""
    if kv._quick is None:
        pytest.skip("_fast.so is not built")
    got = []
    for quick in (kv._quick, None):
        monkeypatch.setattr(kv, "_quick", quick)
        side = torch.cuda.Stream()
        for stream in (None, side, side.cuda_stream):
            side.wait_stream(torch.cuda.current_stream())
            calls = each_call(fmt, dtype)
            torch.cuda.synchronize()
            for name, call, args in calls:
                call(*args, stream=stream)
            torch.cuda.synchronize()
            got.append([t.view(torch.uint8).cpu() for _, _, args in calls for t in args
                        if isinstance(t, torch.Tensor)])
    for other in got[1:]:
        assert len(other) == len(got[0])
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


def test_binding_refuses_wrong_tensors(monkeypatch):
    """Types, sizes, strides and host tensors: refused alike both ways, and nothing is run."""
    quick = kv._quick
    for way in (quick, None):
        monkeypatch.setattr(kv, "_quick", way)
        for name, call, args in each_call():
            tensors = [i for i, t in enumerate(args) if isinstance(t, torch.Tensor)]
            before = kv.kv_kernel_launches()
            for i in tensors:
                t = args[i]
                wrong = [t.cpu(), t.to(torch.float16)]
                if t.numel() > 1 and not (name == "quant_decode_attn" and i == 6):
                    wrong.append(t[:-1])      # (a shorter slot_map is a legal one there)
                if t.numel() > 1 and t.dim() == 1 and not (name == "quant_decode_attn" and i == 6):
                    wrong.append(torch.cat([t, t])[::2])
                for w in wrong:
                    if i == len(args) - 1 and name != "kv_rotary" and w.is_cuda:
                        continue              # (ws may be of any type; its size is C's to check)
                    with pytest.raises((ValueError, kv.KvError)):
                        call(*args[:i], w, *args[i + 1:])
            assert kv.kv_kernel_launches() == before
            # what the C function refuses: a workspace too small, no frequencies; and a format
            # that there is none of
            bad = list(args)
            bad[-1 if name != "kv_rotary" else 4] = args[-1][:100] if name != "kv_rotary" else None
            with pytest.raises(kv.KvError):
                call(*bad)
            if name != "kv_rotary":
                with pytest.raises((ValueError, kv.KvError)):
                    call(args[0], 7, *args[2:])
            assert kv.kv_kernel_launches() == before
    torch.cuda.synchronize()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_rows_added_to_a_scale_that_is_no_number(fmt, dtype, bad):
    """Rows written behind rows of a block whose scale was never set: they are stored with a scale of
    their own, and read back as any others; the rows held stay NaN and infinities as far as the
    format has those (int8: zeros and the largest codes)."""
    heads, d, page = 2, 48, 32
    pool = Pool(3, heads, page, d, fmt, 7, scales=bad)
    s = shape_of(pool, dtype)
    runs_of = ((0, 5, 4), (1, 16 + 15, 1), (2, 1, 15), (2, 16 + 8, 8))   # page, first row, rows
    slots = np.concatenate([p * page + r + np.arange(n) for p, r, n in runs_of])
    x = rows_of(11, len(slots), heads, d, dtype)
    ws = write(pool, s, x[0].cuda(), x[1].cuda(), slots)
    for name, rows in (("k", x[0].double().numpy()), ("v", x[1].double().numpy())):
        at = 0
        for p, r, n in runs_of:
            b, new = r // BLOCK, rows[at:at + n]
            at += n
            for h in range(heads):
                now = scale_for(new[:, h], fmt)
                held = pool.num[name][p, h, b * BLOCK:r]
                with np.errstate(invalid="ignore"):
                    pool.num[name][p, h, b * BLOCK:r] = nearest(held * bad, fmt)
                pool.num[name][p, h, r:r + n] = nearest(new[:, h] / now, fmt)
                pool.scale[name][p, h, b] = now
    pool.check()
    k, v = (torch.zeros(len(slots), heads, d, dtype=DT[dtype], device="cuda") for _ in range(2))
    kv.kv_quant_read(s, FORMATS[fmt], *pool.args(), i64(slots), None, k, v, ws)
    for name, got in (("k", k), ("v", v)):
        with np.errstate(invalid="ignore"):     # (blocks that got no row)
            values = pool.values(name)
        want = np.stack([values[i // page, :, i % page] for i in slots])
        assert np.isfinite(want).all() and np.array_equal(got.double().cpu().numpy(), want)
    assert kv.kv_check_device_status(ws) == 0
