"""The paged cache on the GPU: kv_page_map against its definition, kv_paged_write, and
paged_decode_attn against 64 bits, each where it can go wrong, and the three together."""
import math

import numpy as np
import pytest
import torch

import kv_cache_eviction_gb300 as kv
from tests.paged import (ERR_ID, ERR_PAGES, ERR_RING, ERR_SLOTS, ERR_TABLE, Cache, ceil_div,
                         page_map_ref, workspace)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kv_cache_eviction_gb300 import _build
    _build.build()
    kv.lib()


def dev(x, dtype):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


# ------------------------------------------------------------------------------- page map

class Map:
    """Buffers of one kv_page_map call, and its check against the definition."""

    def __init__(self, seqs, tables, page, cols, num, lens, add, cap, state=None, ring=None,
                 seed=0):
        rng = np.random.default_rng(seed)
        U = seqs * tables
        self.page, self.num, self.cap = page, num, cap
        self.shape = kv.KvPagedShape.of(seqs, tables, tables, 64, tables, page, cols, "bf16", num)
        used = [max(0, min(cols, ceil_div(int(n), page))) for n in lens]
        order = rng.permutation(num)
        self.table = rng.integers(0, num, (U, cols))
        at = 0
        for u, n in enumerate(used):
            self.table[u, :n] = order[at:at + n]
            at += n
        free = order[at:]
        start = int(rng.integers(0, 3 * num))
        self.ring = np.full(num, -5)
        self.ring[(start + np.arange(len(free))) % num] = free
        self.state = np.array([start, start + len(free)])
        if state is not None:
            self.state = np.array(state)
        if ring is not None:
            self.ring = np.array(ring)
        self.lens, self.add = np.array(lens), np.array(add)
        self.slots = np.full(cap, -7)

    def run(self, in_place=False, stream=None, ws=None):
        i32, i64 = torch.int32, torch.int64
        lens, add, state = dev(self.lens, i32), dev(self.add, i32), dev(self.state, i64)
        # guards around every output
        pad = 64

        def guarded(x, dtype):
            buf = torch.full((len(x) + 2 * pad,), -99, dtype=dtype, device="cuda")
            buf[pad:pad + len(x)] = dev(x, dtype)
            return buf

        ring, table = guarded(self.ring, i32), guarded(self.table.reshape(-1), i32)
        slots, cu = guarded(self.slots, i64), guarded(np.zeros(len(self.lens) + 1), i64)
        lo = guarded(self.lens if in_place else np.full(len(self.lens), -3), i32)
        so = guarded(self.state if in_place else np.full(2, -3), i64)
        v = [b[pad:len(b) - pad] for b in (ring, table, slots, cu, lo, so)]
        ws = workspace(kv.KV_OP_PAGE_MAP, self.shape) if ws is None else ws
        kv.kv_page_map(self.shape, v[4] if in_place else lens, add, v[0],
                       v[5] if in_place else state, v[1], v[4], v[5], v[3], v[2], ws, stream)
        torch.cuda.synchronize()
        code = kv.kv_check_device_status(ws)
        for b in (ring, table, slots, cu, lo, so):
            assert bool((b[:pad] == -99).all()) and bool((b[len(b) - pad:] == -99).all())
        return [x.cpu().numpy() for x in v] + [code]

    def check(self, want_codes=(), **kw):
        ring, table, slots, cu, lens, state, code = self.run(**kw)
        r = page_map_ref(self.lens, self.add, self.ring, self.state, self.cap, self.table,
                         self.slots, self.page, self.num)
        assert r[6] == set(want_codes), r[6]
        for name, got, ref in (("ring", ring, r[0]), ("state", state, r[1]),
                               ("table", table.reshape(self.table.shape), r[2]),
                               ("lens", lens, r[3]), ("cu", cu, r[4]), ("slots", slots, r[5])):
            assert np.array_equal(got, ref), name
        assert code in r[6] if r[6] else code == 0
        return r


def fitting(seqs, tables, page, seed, kind, mean=100):
    rng = np.random.default_rng(seed)
    U = seqs * tables
    lens = rng.integers(0, 2 * mean, U)
    lens[rng.random(U) < 0.1] = 0
    add = {"one": np.ones(U, int), "idle": (rng.random(U) < 0.5).astype(int),
           "mixed": rng.integers(-2 * mean, 2 * mean, U), "none": np.zeros(U, int),
           "drop": -rng.integers(0, 3 * mean, U)}[kind]
    new = np.maximum(lens + add, 0)
    cols = int(max(1, ceil_div(max(lens.max(), new.max()), page)))
    used = sum(ceil_div(int(n), page) for n in lens)
    need = sum(max(0, ceil_div(int(b), page) - ceil_div(int(a), page)) for a, b in zip(lens, new))
    return Map(seqs, tables, page, cols, used + need + 1, lens, add,
               int(np.maximum(add, 0).sum()) + 5, seed=seed)


@pytest.mark.parametrize("kind", ["one", "idle", "mixed", "none", "drop"])
@pytest.mark.parametrize("seqs,tables,page", [(1, 1, 16), (5, 1, 8), (33, 8, 32), (513, 1, 128),
                                              (700, 4, 16), (3, 8, 256)])
def test_map(kind, seqs, tables, page):
    fitting(seqs, tables, page, seqs + page, kind).check()


def test_map_long_prompts():
    """Many slots (many CTAs), in place: lengths and ring state updated where they are read."""
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 9000, 40)
    add = rng.integers(-9000, 60000, 40)
    new = np.maximum(lens + add, 0)
    cols = int(ceil_div(new.max(), 16))
    num = int(sum(ceil_div(int(n), 16) for n in lens) + sum(ceil_div(int(n), 16) for n in new))
    m = Map(40, 1, 16, cols, num, lens, add, int(np.maximum(add, 0).sum()) + 1000, seed=9)
    m.check()
    m.check(in_place=True)


def test_map_most_tables():
    U = kv.KV_PAGE_MAP_MAX_TABLES
    rng = np.random.default_rng(4)
    lens = rng.integers(0, 64, U)
    add = rng.integers(-3, 20, U)
    m = Map(U // 8, 8, 8, 16, 12 * U, lens, add, int(np.maximum(add, 0).sum()), seed=2)
    m.check(in_place=True)


def test_map_refusals():
    """Each refusal: the tables that cannot be served keep their length and pages, the others
    are served."""
    # a length out of its table's range, growth past the table, a shrink past zero
    m = Map(6, 1, 8, 4, 40, [-1, 33, 30, 10, 5, 32], [3, 2, 3, 4, -100, 0], 40)
    m.check({ERR_TABLE})
    m = Map(2, 1, 8, 4, 40, [10, 2**31 - 1], [2**31 - 1, 2**31 - 1], 40)
    m.check({ERR_TABLE, ERR_SLOTS})
    m = Map(2, 1, 8, 4, 40, [10, -2**31], [-2**31, -2**31], 40)
    m.check({ERR_TABLE})
    # no pages left: refused from the first table that does not fit, except rows that fit
    lens, add = [8, 8, 9, 8, 8, 15], [9, 9, 2, 1, -8, 1]
    m = Map(6, 1, 8, 4, 7 + 3, lens, add, 100)
    assert m.state[1] - m.state[0] == 2
    r = m.check({ERR_PAGES})
    assert list(r[3]) == [17, 8, 11, 8, 0, 16]
    # rows past the slot map's end
    m = Map(4, 1, 8, 4, 30, [1, 2, 3, 4], [5, 5, 5, 0], 12)
    r = m.check({ERR_SLOTS})
    assert list(r[3]) == [6, 7, 3, 4]
    m = Map(2, 1, 8, 4, 30, [1, 2], [5, 5], 0)
    m.check({ERR_SLOTS})


@pytest.mark.parametrize("state", [(-1, 5), (6, 5), (0, 31), (2**62, 2**62 + 3)])
def test_map_bad_ring_state(state):
    m = Map(3, 1, 8, 4, 30, [8, 20, 3], [5, -10, 2], 20, state=state)
    ring, table, slots, cu, lens, st, code = m.run()
    assert code in (ERR_RING, ERR_PAGES)
    assert list(lens) == [8, 20, 5] and list(st) == list(state)
    assert np.array_equal(ring, m.ring)
    assert np.array_equal(table.reshape(m.table.shape), m.table)
    assert (slots[:5] == -1).all() and (slots[5:7] >= 0).all() and (slots[7:] == -7).all()


def test_map_more_returned_than_the_ring_holds():
    m = Map(2, 1, 8, 4, 5, [8, 20], [8, -20], 20, state=(3, 6), ring=range(5))
    m.check({ERR_RING})


def test_map_bad_page_numbers():
    m = Map(3, 1, 8, 4, 30, [8, 20, 4], [3, -20, 2], 20)
    m.ring[m.state[0] % 30] = 30
    m.table[1, 1] = -4
    m.table[2, 0] = 1 << 30
    m.check({ERR_ID})


def test_map_captured_steps():
    """A captured one-token step replayed in place: the lengths walk through page ends."""
    seqs, page, cols = 9, 8, 12
    rng = np.random.default_rng(6)
    lens = rng.integers(0, 60, seqs)
    m = Map(seqs, 1, page, cols, 120, lens, np.ones(seqs, int), seqs)
    i32, i64 = torch.int32, torch.int64
    d = dict(lens=dev(m.lens, i32), add=dev(m.add, i32), ring=dev(m.ring, i32),
             state=dev(m.state, i64), table=dev(m.table, i32), cu=dev(np.zeros(seqs + 1), i64),
             slots=dev(m.slots, i64))
    ws = workspace(kv.KV_OP_PAGE_MAP, m.shape)

    def step():
        kv.kv_page_map(m.shape, d["lens"], d["add"], d["ring"], d["state"], d["table"], d["lens"],
                       d["state"], d["cu"], d["slots"], ws)

    ref = (m.ring, m.state, m.table, m.lens, None, m.slots)
    step()
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        step()
    for i in range(20):
        if i:
            g.replay()
        ref = page_map_ref(ref[3], m.add, ref[0], ref[1], m.cap, ref[2], ref[5], page, m.num)
        assert not ref[6]
        torch.cuda.synchronize()
        for got, want in ((d["ring"], ref[0]), (d["state"], ref[1]), (d["table"], ref[2]),
                          (d["lens"], ref[3]), (d["cu"], ref[4]), (d["slots"], ref[5])):
            assert np.array_equal(got.cpu().numpy(), want)
    assert kv.kv_check_device_status(ws) == 0


# ------------------------------------------------------------------------------- row write

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,hkv,tables,d,page,fused,extra", [
    (1, 8, 1, 128, 16, True, 0), (77, 2, 1, 72, 8, False, 64), (1000, 8, 8, 128, 64, False, 0),
    (513, 3, 1, 8, 256, True, 128), (4099, 4, 1, 96, 32, True, 0), (20001, 8, 8, 64, 16, False, 8),
    (9, 8, 1, 40, 128, False, 0)])
def test_write(dtype, rows, hkv, tables, d, page, fused, extra):
    gen = torch.Generator(device="cuda").manual_seed(rows)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    hp = hkv // tables
    num = ceil_div(rows, page) + 3
    inner = hp * page * d
    s = kv.KvPagedShape.of(1, hkv, hkv, d, tables, page, num, dtype, num,
                           inner + extra if extra else 0)
    width = 4 * hp * d if fused else hp * d
    src = torch.randn(2, rows, width, generator=gen, device="cuda").to(dt)
    k = src[0, :, hp * d:2 * hp * d] if fused else src[0].view(rows, hp, d)
    v = src[1, :, 2 * hp * d:3 * hp * d] if fused else src[1].view(rows, hp, d)
    slots = torch.randperm(num * page, generator=gen, device="cuda")[:rows]
    slots[torch.rand(rows, generator=gen, device="cuda") < 0.1] = -1
    for n in (None, 0, rows // 2, rows + 5, -4):
        pools = []
        for _ in range(2):
            flat = torch.full((num * (inner + extra) + 64,), 7.0, dtype=dt, device="cuda")
            pools.append((flat, flat[:num * (inner + extra)].as_strided(
                (num, hp, page, d), (inner + extra, page * d, d, 1))))
        ws = workspace(kv.KV_OP_PAGED_WRITE, s)
        kv.kv_paged_write(s, k, v, slots, None if n is None else dev([n], torch.int64),
                          pools[0][1], pools[1][1], ws)
        m = rows if n is None else max(0, min(rows, n))
        at = slots[:m]
        keep = at >= 0
        for (flat, pool), x in zip(pools, (k, v)):
            want = torch.full_like(flat, 7.0)
            w = want[:num * (inner + extra)].as_strided(pool.shape, pool.stride())
            w[at[keep] // page, :, at[keep] % page] = x[:m].reshape(m, hp, d)[keep]
            assert torch.equal(flat, want)
        assert kv.kv_check_device_status(ws) == 0


def test_write_bad_slots():
    """Slots outside the pool are skipped and reported; the rows around them are stored."""
    s = kv.KvPagedShape.of(1, 2, 2, 64, 1, 8, 4, "bf16", 4)
    k = torch.randn(6, 2, 64, device="cuda").bfloat16()
    flat = torch.zeros(2, 4 * 2 * 8 * 64 + 4096, dtype=torch.bfloat16, device="cuda")
    kp, vp = (flat[i, 2048:2048 + 4 * 2 * 8 * 64].view(4, 2, 8, 64) for i in range(2))
    ws = workspace(kv.KV_OP_PAGED_WRITE, s)
    slots = dev([3, 32, -2, 1 << 62, -(1 << 62), 31], torch.int64)
    kv.kv_paged_write(s, k, k, slots, None, kp, vp, ws)
    assert kv.kv_check_device_status(ws) == ERR_ID
    assert kv.kv_check_device_status(ws) == 0
    want = torch.zeros_like(flat)
    for i in range(2):
        w = want[i, 2048:2048 + 4 * 2 * 8 * 64].view(4, 2, 8, 64)
        w[0, :, 3] = k[0]
        w[3, :, 7] = k[5]
    assert torch.equal(flat, want)


def test_far_slots():
    """Slots past 2^32 rows' worth of pages in the map, and bytes past 2^32 in the pool."""
    num, page = 1 << 25, 256
    s = kv.KvPagedShape.of(2, 1, 1, 64, 1, page, 4, "bf16", num)
    i32, i64 = torch.int32, torch.int64
    ring = torch.full((num,), -1, dtype=i32, device="cuda")
    ring[:3] = dev([num - 1, 1 << 24, num - 2], i32)
    lens, state = dev([0, 0], i32), dev([0, 3], i64)
    table = torch.full((2, 4), -1, dtype=i32, device="cuda")
    cu, slots = torch.zeros(3, dtype=i64, device="cuda"), torch.zeros(300, dtype=i64, device="cuda")
    ws = workspace(kv.KV_OP_PAGE_MAP, s)
    kv.kv_page_map(s, lens, dev([257, 2], i32), ring, state, table, lens, state, cu, slots, ws)
    assert kv.kv_check_device_status(ws) == 0
    want = [(num - 1) * page + i for i in range(256)] + [(1 << 24) * page] + \
           [(num - 2) * page, (num - 2) * page + 1]
    assert slots[:259].tolist() == want and max(want) > 1 << 32

    num, heads, d = 9000, 8, 128
    s = kv.KvPagedShape.of(1, heads, heads, d, 1, page, num, "bf16", num)
    kp = torch.zeros(num, heads, page, d, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    assert kp.numel() > 1 << 31
    k, v = (torch.randn(4, heads, d, device="cuda").bfloat16() for _ in range(2))
    at = [0, num * page - 1, (num - 2) * page + 5, 17 * page]
    ws = workspace(kv.KV_OP_PAGED_WRITE, s)
    kv.kv_paged_write(s, k, v, dev(at, i64), None, kp, vp, ws)
    assert kv.kv_check_device_status(ws) == 0
    for pool, rows in ((kp, k), (vp, v)):
        for i, x in enumerate(at):
            assert torch.equal(pool[x // page, :, x % page], rows[i])
            pool[x // page, :, x % page] = 0
        assert not bool(pool.any())


# ------------------------------------------------------------------------------- decode

LENS = {"one": [1], "few": [3, 1, 2], "empty": [0, 5, 0, 0, 17, 0], "none": [0, 0],
        "ends": [15, 16, 17, 31, 32, 33, 127, 128, 129], "long": [5000, 1, 0, 2047],
        "ragged": [700, 3, 64, 0, 1500, 260, 8, 90], "big": [20011]}


def lens_for(kind, U):
    base = LENS[kind]
    return [base[i % len(base)] if i < 40 * len(base) else 9 for i in range(max(U, 1))]


@pytest.mark.parametrize("kind", list(LENS))
@pytest.mark.parametrize("dtype,d,G,page,tables", [
    ("bf16", 128, 4, 16, 1), ("bf16", 128, 8, 64, 1), ("bf16", 64, 1, 8, 1), ("f32", 128, 2, 16, 1),
    ("bf16", 128, 4, 32, 4), ("f32", 72, 3, 8, 4), ("bf16", 80, 5, 256, 1), ("bf16", 8, 7, 16, 1),
    ("f32", 64, 8, 128, 1), ("bf16", 104, 6, 128, 4)])
def test_decode(kind, dtype, d, G, page, tables):
    hkv = 4
    seqs = len(LENS[kind])
    c = Cache(seqs, hkv, G, d, tables, page, lens_for(kind, seqs * tables), dtype,
              seed=d + G + page)
    out, ws = c.run()
    torch.cuda.synchronize()
    assert kv.kv_check_device_status(ws) == 0
    c.check(out)
    c.check_pools()
    # the same workspace and rows again: the same bits, and the row stored by the first call
    # read back from the pool gives them too
    again, _ = c.run(ws=ws)
    assert torch.equal(out, again)
    assert torch.equal(out, c.run(with_new=False, ws=ws)[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_idle_sequences_and_many(dtype):
    """Sequences that got no row attend over what they hold; many short ones and few long."""
    rng = np.random.default_rng(8)
    lens = rng.integers(0, 40, 300)
    lens[[5, 77, 200]] = [3000, 1500, 900]
    c = Cache(300, 2, 4, 128, 1, 16, lens, dtype, 3, new=rng.random(300) < 0.5)
    out, ws = c.run()
    torch.cuda.synchronize()
    assert kv.kv_check_device_status(ws) == 0
    c.check(out)
    c.check_pools()


def test_decode_head_tables_skewed():
    """A table per head with lengths from none to thousands, as head-adaptive budgets give."""
    rng = np.random.default_rng(9)
    lens = np.minimum(np.exp(rng.normal(4.5, 1.5, 24 * 8)), 6000).astype(int)
    lens[::11] = 0
    c = Cache(24, 8, 4, 128, 8, 16, lens, "bf16", 4, new=rng.random(24 * 8) < 0.8)
    out, ws = c.run()
    torch.cuda.synchronize()
    assert kv.kv_check_device_status(ws) == 0
    c.check(out)
    c.check_pools()


@pytest.mark.parametrize("lens", [[30000, 9000, 100, 26001], [1] * 50 + [20000, 45000],
                                  [65001]])
@pytest.mark.parametrize("dtype,d,G", [("bf16", 128, 1), ("bf16", 64, 3), ("f32", 40, 1)])
def test_decode_many_tiles_a_warp(dtype, d, G, lens):
    """Calls large enough that CTAs take further segments and a warp has over 32 tiles."""
    c = Cache(len(lens), 8, G, d, 1, 64, lens, dtype, 12)
    out, ws = c.run()
    torch.cuda.synchronize()
    assert kv.kv_check_device_status(ws) == 0
    c.check(out)
    c.check_pools()
    for _ in range(5):
        assert torch.equal(out, c.run(ws=ws)[0])


@pytest.mark.parametrize("extra", [8, 64, 4096])
def test_decode_page_stride(extra):
    c = Cache(3, 2, 4, 128, 1, 16, [100, 0, 333], "bf16", 5, page_stride=2 * 16 * 128 + extra)
    out, ws = c.run()
    assert kv.kv_check_device_status(ws) == 0
    c.check(out)
    c.check_pools()


def test_decode_far_pages():
    """Rows past 2^32 bytes and 2^31 elements of the pool."""
    c = Cache(2, 8, 4, 128, 1, 256, [300, 1000], "bf16", 6, first_page=9000)
    assert c.num_pages * 256 * 8 * 128 > 1 << 31
    out, ws = c.run()
    assert kv.kv_check_device_status(ws) == 0
    c.check(out)


def test_decode_bad_pages_slots_and_lengths():
    """Pages outside the pool are left out of the sums, slots outside it are not written,
    lengths outside the table are cut to it; each is reported."""
    c = Cache(3, 2, 4, 128, 1, 16, [100, 40, 64], "bf16", 7, new=[0, 0, 0])
    c.table[0, 2] = c.num_pages
    c.table[1, 0] = -1
    c.table[2, 3] = 1 << 30
    out, ws = c.run()
    assert kv.kv_check_device_status(ws) == ERR_ID
    c.check(out, skip=[(0, 2), (1, 0), (2, 3)])
    c.check_pools(stored=False)
    # every page bad: zeros
    c.table[:] = -7
    out, ws = c.run(ws=ws)
    assert kv.kv_check_device_status(ws) == ERR_ID
    assert bool((out == 0).all())
    for slot in (-2, 1 << 40, -(1 << 50)):
        c = Cache(2, 2, 4, 128, 1, 16, [100, 40], "bf16", 8, new=[1, 0])
        want, _ = c.run()
        c = Cache(2, 2, 4, 128, 1, 16, [100, 40], "bf16", 8, new=[0, 0])
        c.cu[1:] = 1
        c.slots = dev([slot], torch.int64)
        out, ws = c.run()
        assert kv.kv_check_device_status(ws) == ERR_ID
        c.check(out)
        c.check_pools(stored=False)
    c = Cache(3, 2, 4, 128, 1, 16, [64, 64, 64], "bf16", 9, new=[0, 0, 0])
    c.lens_t = dev([-5, 65, 2**31 - 1], torch.int32)
    out, ws = c.run()
    assert kv.kv_check_device_status(ws) == ERR_TABLE
    c.lens[0] = 0
    c.check(out)


@pytest.mark.parametrize("page", [8, 16])
@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 72), ("bf16", 96), ("f32", 32),
                                     ("f32", 72), ("f32", 80), ("f32", 96), ("f32", 128)])
def test_decode_bad_pages_of_every_width(dtype, d, page):
    """Pages outside the pool, either half of a tile's rows, in rows of every width of a stage."""
    c = Cache(3, 2, 5, d, 1, page, [101, 40, 64], dtype, 17, new=[1, 0, 1])
    bad = [(0, 0), (0, 3), (1, 1), (2, 0), (2, 1), (2, 2)]
    for u, col in bad:
        c.table[u, col] = c.num_pages + u if col & 1 else -1 - u
    out, ws = c.run()
    assert kv.kv_check_device_status(ws) == ERR_ID
    c.check(out, skip=bad)
    c.check_pools()


def test_decode_refused_table_keeps_its_rows():
    """A table that asked for a row and got no page (slot -1): nothing is stored, it attends over
    the rows it holds."""
    c = Cache(3, 2, 4, 128, 1, 16, [32, 20, 7], "bf16", 10, new=[0, 1, 1])
    c.cu = dev([0, 1, 2, 3], torch.int64)
    c.slots = dev([-1] + c.slots_host, torch.int64)
    out, ws = c.run()
    assert kv.kv_check_device_status(ws) == 0
    c.check(out)
    c.check_pools()


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_decode_scale(scale):
    c = Cache(3, 2, 4, 128, 1, 16, [100, 1, 333], "bf16", 11)
    c.scale = scale
    out, ws = c.run()
    c.check(out)


def test_decode_captured_and_on_streams():
    """A captured call replayed, and two calls at once on two streams with workspaces of their
    own: the bits of a call on its own."""
    caches = [Cache(16, 8, 4, 128, 1, 16, np.random.default_rng(i).integers(0, 4000, 16), "bf16",
                    20 + i) for i in range(2)]
    want = [c.run()[0].clone() for c in caches]
    streams = [torch.cuda.Stream() for _ in caches]
    wss = [workspace(kv.KV_OP_PAGED_DECODE, c.shape) for c in caches]
    outs = [torch.zeros_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s, w, o in zip(caches, streams, wss, outs):
            c.run(ws=w, out=o, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
    # two captured graphs that share a workspace, replayed in turn on one stream
    graphs = []
    for c, o in zip(caches, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[0]):
            c.run(ws=wss[0], out=o, stream=streams[0])
        graphs.append(g)
    for _ in range(3):
        for o in outs:
            o.fill_(float("nan"))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
    for w in wss:
        assert kv.kv_check_device_status(w) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_every_head_dim(dtype):
    """Every head dim from 8 to 128 and every group size, over lengths around a tile's end."""
    for i, d in enumerate(range(8, 129, 8)):
        c = Cache(3, 2, 1 + i % 8, d, 1, 8 << (i % 6), [16 + i, 7, 40], dtype, 30 + i)
        out, ws = c.run()
        assert kv.kv_check_device_status(ws) == 0
        c.check(out)
        c.check_pools()


def test_decode_thousands_of_tables():
    """Far more tables than threads, most of them empty, runs of empty ones, one long."""
    rng = np.random.default_rng(11)
    lens = np.where(rng.random(6000) < 0.05, rng.integers(1, 60, 6000), 0)
    lens[100:4000] = 0
    lens[[0, 4001, 5999]] = [3, 2500, 17]
    c = Cache(1500, 4, 2, 64, 4, 16, lens, "bf16", 12, new=rng.random(6000) < 0.5)
    out, ws = c.run()
    assert kv.kv_check_device_status(ws) == 0
    c.check(out)
    c.check_pools()
    assert torch.equal(out, c.run(ws=ws)[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_nan_in_a_row_that_counts(dtype):
    """A NaN in K or V of a row that counts reaches its head's outputs, and no other's."""
    for name, long in (("kp", 40), ("vp", 40), ("kp", 3000), ("vp", 3000)):
        c = Cache(3, 2, 4, 64, 1, 16, [30, long, 50], dtype, 13)
        pool = getattr(c, name)
        pool[int(c.table_host[1, 1]), 1, 3, 5] = float("nan")
        out, ws = c.run()
        hit = torch.isnan(out.float())
        assert bool(hit[1, 4:, 5 if name == "vp" else slice(None)].all())
        assert not bool(hit[1, :4].any()) and not bool(hit[[0, 2]].any())
        if name == "vp":
            assert int(hit.sum()) == 4


def test_binding_refuses_wrong_tensors():
    """Types, sizes and strides that the calls cannot take are refused before anything runs."""
    c = Cache(2, 2, 2, 64, 1, 16, [20, 30], "bf16", 14)
    ws = workspace(kv.KV_OP_PAGED_DECODE, c.shape)
    out = torch.empty_like(c.qd)

    def decode(**kw):
        x = dict(q=c.qd, k_new=c.knd, v_new=c.vnd, cu_add=c.cu, slot_map=c.slots, k_pages=c.kp,
                 v_pages=c.vp, block_table=c.table, lens=c.lens_t, softmax_scale=0.1, out=out,
                 ws=ws)
        x.update(kw)
        kv.paged_decode_attn(c.shape, **x)

    decode()
    for kw in (dict(q=c.qd.float()), dict(q=c.qd[:1]), dict(lens=c.lens_t.long()),
               dict(cu_add=c.cu[:2]), dict(block_table=c.table.t().contiguous().t()),
               dict(k_pages=c.kp[:-1]), dict(k_pages=c.kp.transpose(1, 2)),
               dict(v_pages=c.vp.float()), dict(out=out.cpu()), dict(slot_map=c.slots.int()),
               dict(k_new=c.knd.transpose(0, 1))):
        with pytest.raises(ValueError):
            decode(**kw)
    with pytest.raises(kv.KvError):
        decode(ws=ws[:1024])
    with pytest.raises(kv.KvError):
        decode(k_new=None)
    wsw = workspace(kv.KV_OP_PAGED_WRITE, c.shape)
    rows = torch.zeros(5, 2, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(5, dtype=torch.int64, device="cuda")
    for k, v, sl in ((rows[:, :1], rows, slots), (rows.float(), rows, slots), (rows, rows, slots[:4]),
                     (rows, rows[:4], slots), (rows.transpose(1, 2), rows, slots),
                     (rows[::2], rows[:3], slots), (rows, rows, slots.int())):
        with pytest.raises(ValueError):
            kv.kv_paged_write(c.shape, k, v, sl, None, c.kp, c.vp, wsw)
    m = fitting(4, 1, 16, 3, "one")
    wm = workspace(kv.KV_OP_PAGE_MAP, m.shape)
    i32, i64 = torch.int32, torch.int64
    good = dict(lens=dev(m.lens, i32), add=dev(m.add, i32), free_ring=dev(m.ring, i32),
                free_state=dev(m.state, i64), block_table=dev(m.table, i32),
                lens_out=dev(m.lens, i32), free_out=dev(m.state, i64),
                cu_add=dev(np.zeros(5), i64), slot_map=dev(m.slots, i64))
    kv.kv_page_map(m.shape, ws=wm, **good)
    for kw in (dict(lens=dev(m.lens, i64)), dict(add=dev(m.add[:3], i32)),
               dict(free_ring=dev(m.ring[:-1], i32)), dict(block_table=dev(m.table[:3], i32)),
               dict(cu_add=dev(np.zeros(4), i64)), dict(slot_map=dev(m.slots, i32))):
        with pytest.raises(ValueError):
            kv.kv_page_map(m.shape, ws=wm, **{**good, **kw})


# ------------------------------------------------------------------------------- together

def test_captured_serving_step():
    """One decode step -- tables and lengths in place, then attention that stores the new rows --
    captured once and replayed for 40 tokens without a host round trip: outputs of the last step
    against 64 bits over every row the replays stored."""
    seqs, hkv, G, d, page, steps = 5, 2, 4, 64, 8, 40
    c = Cache(seqs, hkv, G, d, 1, page, [1, 30, 8, 15, 100], "f32", 15, new=[0] * seqs)
    cols = ceil_div(100 + steps, page)
    num = c.num_pages + seqs * ceil_div(steps, page) + 5
    s = kv.KvPagedShape.of(seqs, hkv * G, hkv, d, 1, page, cols, "f32", num)
    i32, i64 = torch.int32, torch.int64
    table = torch.full((seqs, cols), -1, dtype=i32, device="cuda")
    table[:, :c.max_pages] = c.table
    kp = torch.full((num, hkv, page, d), float("nan"), device="cuda")
    vp = kp.clone()
    kp[:c.num_pages], vp[:c.num_pages] = c.kp, c.vp
    used = {int(c.table_host[u, j]) for u in range(seqs) for j in range(ceil_div(c.lens[u], page))}
    free = [p for p in range(num) if p not in used]
    ring = dev(free + [-1] * (num - len(free)), i32)
    state = dev([0, len(free)], i64)
    lens, one = c.lens_t.clone(), torch.ones(seqs, dtype=i32, device="cuda")
    cu = torch.zeros(seqs + 1, dtype=i64, device="cuda")
    slots = torch.full((seqs,), -1, dtype=i64, device="cuda")
    ws = [workspace(op, s) for op in (kv.KV_OP_PAGE_MAP, kv.KV_OP_PAGED_DECODE)]
    gen = torch.Generator(device="cuda").manual_seed(2)
    tokens = [torch.randn(3, steps, seqs, hkv * G, d, generator=gen, device="cuda")]
    q = torch.empty(seqs, hkv * G, d, device="cuda")
    kn, vn = (torch.empty(seqs, hkv, d, device="cuda") for _ in range(2))
    out = torch.empty_like(q)

    def step():
        kv.kv_page_map(s, lens, one, ring, state, table, lens, state, cu, slots, ws[0])
        kv.paged_decode_attn(s, q, kn, vn, cu, slots, kp, vp, table, lens, c.scale, out, ws[1])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    saved = lens.clone(), state.clone(), table.clone()
    q.zero_(), kn.zero_(), vn.zero_()
    step()                                   # (the one-time set-up of the kernels)
    torch.cuda.synchronize()
    for x, y in zip((lens, state, table), saved):
        x.copy_(y)
    with torch.cuda.graph(g, stream=side):
        step()
    for t in range(steps):
        q.copy_(tokens[0][0, t])
        kn.copy_(tokens[0][1, t, :, :hkv])
        vn.copy_(tokens[0][2, t, :, :hkv])
        g.replay()
    torch.cuda.synchronize()
    for w in ws:
        assert kv.kv_check_device_status(w) == 0
    assert lens.tolist() == [n + steps for n in c.lens]
    for name, i in (("k", 1), ("v", 2)):
        fresh = tokens[0][i, :, :, :hkv].cpu()            # [steps][seqs][hkv][d]
        c.rows[name] = [torch.cat([r, fresh[:, u].transpose(0, 1)], 1)
                        for u, r in enumerate(c.rows[name])]
    c.q = tokens[0][0, steps - 1].cpu()
    c.lens = lens.tolist()
    c.check(out)

def test_eviction_into_pages_and_decode():
    """Scores, budgets and compaction of an evicted prefix, its rows into a paged cache with a
    table per head, then decode steps that walk through page ends: each against 64 bits over the
    same rows, and equal in effect to the flat cache's decode (both within their bounds)."""
    import oracle as O
    from kv_cache_eviction_gb300 import workloads as W
    from tests.kvpath import np64, run_allocate, run_compact, run_score

    wl = W.WORKLOADS["llama8b_16k_layer"].with_(n=2048, head_budget_frac=0.1, layers=2, reserve=0,
                                                temp=(0.5, 4.0))
    shape = kv.KvShape.from_workload(wl)
    inp = W.make_batch(wl, device="cuda")
    budgets = wl.budgets()
    scores, _ = run_score(wl, shape, inp)
    _, hb = run_allocate(wl, shape, scores, budgets)
    cap = int(budgets.sum())
    flat = run_compact(wl, shape, inp, scores, None, hb, cap)

    seqs, hkv, d, page, steps = wl.batch * wl.layers, wl.hkv, wl.d, 16, 20
    U = seqs * hkv
    cols = ceil_div(int(flat["lens"].max()) + steps, page)
    num = sum(ceil_div(int(n) + steps, page) for n in flat["lens"].flatten().cpu())
    ps = kv.KvPagedShape.of(seqs, wl.hq, hkv, d, hkv, page, cols, "bf16", num)
    i32, i64 = torch.int32, torch.int64
    lens = torch.zeros(U, dtype=i32, device="cuda")
    ring = torch.randperm(num, device="cuda").to(i32)
    state = dev([0, num], i64)
    table = torch.full((U, cols), -1, dtype=i32, device="cuda")
    cu = torch.zeros(U + 1, dtype=i64, device="cuda")
    slots = torch.full((cap,), -1, dtype=i64, device="cuda")
    kp = torch.full((num, 1, page, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vp = kp.clone()
    wm, ww, wd = (workspace(op, ps) for op in (kv.KV_OP_PAGE_MAP, kv.KV_OP_PAGED_WRITE,
                                               kv.KV_OP_PAGED_DECODE))
    kv.kv_page_map(ps, lens, flat["lens"].flatten(), ring, state, table, lens, state, cu, slots,
                   wm)
    kv.kv_paged_write(ps, flat["kf"], flat["vf"], slots, cu[U:], kp, vp, ww)
    assert torch.equal(lens, flat["lens"].flatten())
    assert int(cu[U]) == cap

    one = torch.ones(U, dtype=i32, device="cuda")
    rows = {"k": [], "v": []}
    fcu = flat["cu"].reshape(seqs, hkv + 1)[:, :hkv].reshape(-1).cpu()
    for u in range(U):
        a, n = int(fcu[u]), int(flat["lens"].flatten()[u])
        rows["k"].append(flat["kf"][a:a + n].cpu())
        rows["v"].append(flat["vf"][a:a + n].cpu())
    ref = Cache.__new__(Cache)
    ref.seqs, ref.hkv, ref.G, ref.d, ref.tables, ref.page = seqs, hkv, wl.group_size, d, hkv, page
    ref.dtype, ref.dt, ref.scale = "bf16", torch.bfloat16, 1 / math.sqrt(d)
    for step in range(steps):
        dec = W.make_decode_batch(wl, step, inp["tau"], device="cuda")
        q = dec["q"].reshape(seqs, wl.hq, d)
        kn, vn = (dec[x].reshape(seqs, hkv, d) for x in ("k_new", "v_new"))
        out = torch.empty_like(q)
        kv.kv_page_map(ps, lens, one, ring, state, table, lens, state, cu, slots, wm)
        kv.paged_decode_attn(ps, q, kn, vn, cu, slots, kp, vp, table, lens, ref.scale, out, wd)
        for u in range(U):
            for name, x in (("k", kn), ("v", vn)):
                rows[name][u] = torch.cat([rows[name][u], x.reshape(U, d)[u:u + 1].cpu()])
        if step % 5 == 0 or step == steps - 1:
            ref.q = q.cpu()
            ref.rows = {n: [r[None] for r in rows[n]] for n in rows}
            ref.lens = [len(r) for r in rows["k"]]
            ref.check(out)
    for w in (wm, ww, wd):
        assert kv.kv_check_device_status(w) == 0

    # re-eviction: every head gives up its last 40 rows, whose pages go back and serve the next
    before = int(state[1] - state[0])
    less = torch.full((U,), -40, dtype=i32, device="cuda")
    want = [max(0, int(n) - 40) for n in lens]
    back = sum(ceil_div(int(n), page) - ceil_div(w, page) for n, w in zip(lens, want))
    kv.kv_page_map(ps, lens, less, ring, state, table, lens, state, cu, slots, wm)
    out = torch.empty_like(q)
    kv.paged_decode_attn(ps, q, None, None, None, None, kp, vp, table, lens, ref.scale, out, wd)
    assert int(state[1] - state[0]) == before + back
    ref.rows = {n: [r[None, :w] for r, w in zip(rows[n], want)] for n in rows}
    ref.lens = want
    ref.check(out)
    assert kv.kv_check_device_status(wm) == 0 and kv.kv_check_device_status(wd) == 0


def test_serving_loop_with_shared_tables():
    """Prompts admitted in pieces, decode steps, a sequence that ends and one that takes its
    pages: rows and outputs against a plain list of rows."""
    seqs, hkv, G, d, page, cols, num = 4, 2, 4, 64, 8, 40, 60
    gen = torch.Generator(device="cuda").manual_seed(1)
    s = kv.KvPagedShape.of(seqs, hkv * G, hkv, d, 1, page, cols, "f32", num)
    i32, i64 = torch.int32, torch.int64
    lens = torch.zeros(seqs, dtype=i32, device="cuda")
    ring = torch.arange(num, dtype=i32, device="cuda")
    state = dev([0, num], i64)
    table = torch.full((seqs, cols), -1, dtype=i32, device="cuda")
    cu = torch.zeros(seqs + 1, dtype=i64, device="cuda")
    slots = torch.full((400,), -1, dtype=i64, device="cuda")
    kp = torch.full((num, hkv, page, d), float("nan"), device="cuda")
    vp = kp.clone()
    ws = [workspace(op, s) for op in (kv.KV_OP_PAGE_MAP, kv.KV_OP_PAGED_WRITE,
                                      kv.KV_OP_PAGED_DECODE)]
    held = {n: [torch.zeros(0, hkv, d) for _ in range(seqs)] for n in "kv"}
    ref = Cache.__new__(Cache)
    ref.seqs, ref.hkv, ref.G, ref.d, ref.tables, ref.page = seqs, hkv, G, d, 1, page
    ref.dtype, ref.dt, ref.scale = "f32", torch.float32, 1 / math.sqrt(d)
    script = [("rows", [100, 30, 0, 1])] + [("one", [1, 1, 0, 1])] * 9 + \
             [("rows", [20, 0, 77, 0]), ("one", [1, 1, 1, 1]), ("rows", [-500, 0, 0, -5]),
              ("rows", [0, 0, 0, 200])] + [("one", [0, 1, 1, 1])] * 9
    for kind, add in script:
        kv.kv_page_map(s, lens, dev(add, i32), ring, state, table, lens, state, cu, slots, ws[0])
        n = sum(max(a, 0) for a in add)
        q = torch.randn(seqs, hkv * G, d, generator=gen, device="cuda")
        out = torch.empty_like(q)
        if kind == "rows":
            k, v = (torch.randn(n + 3, hkv, d, generator=gen, device="cuda") for _ in range(2))
            if n:
                kv.kv_paged_write(s, k, v, slots, cu[seqs:], kp, vp, ws[1])
            kv.paged_decode_attn(s, q, None, None, None, None, kp, vp, table, lens, ref.scale,
                                 out, ws[2])
            at = 0
            fresh = {"k": k.cpu(), "v": v.cpu()}
        else:
            k, v = (torch.randn(seqs, hkv, d, generator=gen, device="cuda") for _ in range(2))
            kv.paged_decode_attn(s, q, k, v, cu, slots, kp, vp, table, lens, ref.scale, out,
                                 ws[2])
            fresh = {"k": k.cpu(), "v": v.cpu()}
        for name in "kv":
            at = 0
            for b, a in enumerate(add):
                r = held[name][b]
                if a < 0:
                    held[name][b] = r[:max(0, len(r) + a)]
                elif kind == "rows":
                    held[name][b] = torch.cat([r, fresh[name][at:at + a]])
                    at += a
                elif a:
                    held[name][b] = torch.cat([r, fresh[name][b:b + 1]])
        assert lens.tolist() == [len(r) for r in held["k"]]
        ref.q = q.cpu()
        ref.lens = lens.tolist()
        ref.rows = {n: [r.transpose(0, 1) for r in held[n]] for n in held}
        ref.check(out)
    for w in ws:
        assert kv.kv_check_device_status(w) == 0
