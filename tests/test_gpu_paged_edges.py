"""paged_decode_attn and kv_page_map on the GPU at the edges of what their arguments may hold."""
import numpy as np
import pytest
import torch

import kv_cache_eviction_gb300 as kv
from tests.paged import Cache, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kv_cache_eviction_gb300 import _build
    _build.build()
    kv.lib()


# ------------------------------------------------------------------------------- NaN

def poison_rows(c, u, head, first, count):
    """NaN in K of rows first .. first + count - 1 of table u, one head."""
    for r in range(first, first + count):
        c.kp[int(c.table_host[u, r // c.page]), head, r % c.page, 2] = float("nan")


# 16 rows are one tile, so one warp's; 64 are split between a CTA's warps; the others cross CTAs
SPLITS = [16, 64, 500, 3000]


@pytest.mark.parametrize("dtype,d,G,page", [("bf16", 128, 4, 16), ("bf16", 72, 8, 8),
                                            ("f32", 128, 3, 16), ("f32", 64, 4, 32)])
def test_decode_nan_query(dtype, d, G, page):
    """A NaN in a query reaches all of its outputs, and no other query's, however its head's rows
    are split."""
    c = Cache(4, 2, G, d, 1, page, SPLITS, dtype, 41, new=[0] * 4)
    want, ws = c.run()
    for b in range(4):
        c.qd[b, 2 * G - 2, (5 * b) % d] = float("nan")
    out, _ = c.run(ws=ws)
    bad = torch.isnan(out.float())
    assert bool(bad[:, 2 * G - 2].all())
    keep = [g for g in range(2 * G) if g != 2 * G - 2]
    assert torch.equal(out[:, keep], want[:, keep])
    assert kv.kv_check_device_status(ws) == 0


@pytest.mark.parametrize("dtype,d,G", [("bf16", 128, 4), ("bf16", 64, 1), ("f32", 128, 2),
                                       ("f32", 72, 4)])
@pytest.mark.parametrize("lens,u,first,count", [
    ([16], 0, 0, 16), ([64], 0, 0, 64), ([64], 0, 16, 32), ([512], 0, 0, 512), ([512], 0, 0, 64),
    ([512], 0, 64, 64), ([512], 0, 448, 64), ([500], 0, 100, 200), ([3000, 40], 0, 0, 1500),
    ([3000, 40], 0, 1400, 900), ([40, 9000], 1, 0, 9000), ([40, 9000], 1, 4000, 2000)])
def test_decode_nan_rows(dtype, d, G, lens, u, first, count):
    """A run of NaN keys as long as what a warp or a CTA takes of a head, or all of them: every
    output of that head is NaN, the other head's and sequence's are untouched."""
    c = Cache(len(lens), 2, G, d, 1, 16, lens, dtype, 42, new=[0] * len(lens))
    want, ws = c.run()
    poison_rows(c, u, 1, first, count)
    out, _ = c.run(ws=ws)
    assert bool(torch.isnan(out[u, G:].float()).all())
    assert torch.equal(out[u, :G], want[u, :G])
    for b in range(len(lens)):
        if b != u:
            assert torch.equal(out[b], want[b])


# ------------------------------------------------------------------------------- scores

U23 = 2.0 ** -23


def place(c, name):
    """c.rows[name] into the device pool, whole rows (none is left to k_new / v_new)."""
    pool = c.kp if name == "k" else c.vp
    for u, n in enumerate(c.lens):
        x = c.rows[name][u].cuda()
        pages = c.table_host[u, :-(-n // c.page)].cuda()
        r = torch.arange(n, device="cuda")
        pool[pages[r // c.page], :, r % c.page] = x.transpose(0, 1)


def check_exact_scores(c, out):
    """Against 64 bits where every score is a float32 number whatever the order of its sum, so
    that only what follows the scores can be off: the exponent (z - max) * scale, rounded twice, with
    a factor rounded once, 2^-22 of itself; exp2 and the rescaling by it, 2^-22 at a time, at most 64
    of those; the weights' bits (2^-16 of bf16's, 2^-21 of fp32's factors); sums of as many
    terms as the head has tiles; the output's rounding."""
    t_p = 2.0 ** -16 if c.dtype == "bf16" else 2.0 ** -20
    half = torch.finfo(c.dt).eps / 2
    got = out.double().cpu().numpy()
    q = c.q.double().numpy()
    for u, n in enumerate(c.lens):
        for h in range(c.hkv):
            k, v = (c.rows[x][u][h].double().numpy() for x in "kv")
            for g in range(c.G):
                z = k @ q[u, h * c.G + g]
                assert np.array_equal(z, z.astype(np.float32))
                x = (z - z.max()) * c.scale
                p = np.exp(x)
                p /= p.sum()
                want, mag = p @ v, p @ np.abs(v)
                e = np.abs(x) * 2.0 ** -22 + 64 * 2.0 ** -22
                tol = ((p * e) @ np.abs(v) + (p @ e) * mag +
                       ((2 * n / 8 + 64) * U23 + t_p) * mag + half * np.abs(want))
                off = np.abs(got[u, h * c.G + g] - want)
                assert bool((off <= tol).all()), (u, h, g, float((off / tol).max()))


@pytest.mark.parametrize("lens", [[16], [64, 16], [500, 40], [3000, 16, 700], [9000]])
@pytest.mark.parametrize("dtype,d,G", [("bf16", 128, 4), ("bf16", 72, 2), ("f32", 128, 2),
                                       ("f32", 64, 3)])
@pytest.mark.parametrize("power,up", [(24, 1), (24, -1), (40, 1)])
def test_decode_far_scores(dtype, d, G, lens, power, up):
    """Scores around 2^24 (where one rounding of score * scale moves an exponent by a half) and
    2^40 (by thousands), rising or falling over the rows: the softmax goes by their differences."""
    c = Cache(len(lens), 2, G, d, 1, 16, lens, dtype, 43, new=[0] * len(lens))
    step = 2.0 ** (power - 23)                    # one step of float32 at 2^power
    c.q.zero_()
    c.q[:, :, 0] = 2.0 ** (power // 2)
    c.q[:, :, 9] = step
    for u, n in enumerate(lens):
        k = c.rows["k"][u]
        k.zero_()
        k[:, :, 0] = 2.0 ** (power - power // 2)
        r = torch.arange(n).float()
        # 0..127 over the rows, so that the maximum moves from tile to tile; every value many times
        k[:, :, 9] = ((r if up > 0 else n - 1 - r) * 128 / n).floor().to(c.dt)
    place(c, "k")
    place(c, "v")
    c.qd.copy_(c.q)
    c.scale = 0.125
    out, ws = c.run(with_new=False)
    assert kv.kv_check_device_status(ws) == 0
    check_exact_scores(c, out)


# ------------------------------------------------------------------------------- page map

@pytest.mark.parametrize("first,second", [(2**31 - 3, 100), (2**31 - 2, 100), (2**31 - 5, 1000),
                                          (2**31 - 5, 3)])
def test_map_sums_of_gains_past_32_bits(first, second):
    """A garbage gain just under 2^31 and a table behind it: both are refused, and every length is
    written."""
    i32, i64 = torch.int32, torch.int64
    s = kv.KvPagedShape.of(4, 1, 1, 64, 1, 8, 4, "bf16", 30)
    lens = torch.tensor([10, 7, 5, 9], dtype=i32, device="cuda")
    add = torch.tensor([first, second, 0, -9], dtype=i32, device="cuda")
    ring = torch.arange(30, dtype=i32, device="cuda")
    state = torch.tensor([6, 30], device="cuda")
    table = torch.arange(16, dtype=i32, device="cuda").view(4, 4) % 6
    out, state_out = torch.full((4,), -3, dtype=i32, device="cuda"), torch.zeros(2, dtype=i64,
                                                                                 device="cuda")
    cu, slots = torch.zeros(5, dtype=i64, device="cuda"), torch.full((6,), -7, device="cuda")
    ws = workspace(kv.KV_OP_PAGE_MAP, s)
    kv.kv_page_map(s, lens, add, ring, state, table, out, state_out, cu, slots, ws)
    assert kv.kv_check_device_status(ws) in (7, 9)
    assert out.tolist() == [10, 7, 5, 0]
    assert state_out.tolist() == [6, 32]
    assert cu.tolist() == [0, first, first + second, first + second, first + second]
    assert slots.tolist() == [-1] * 6


# ------------------------------------------------------------------------------- long sums

class Many:
    """A paged cache built and checked on the device, for calls with many tiles.  Scores are exact:
    q and K are whole numbers, or (whole=False) every score is 0 but each 128th row's, which is
    0.7 more.  V is positive."""

    def __init__(self, seqs, hkv, G, d, page, lens, dtype, seed, whole=True):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.hkv, self.G, self.d, self.page, self.lens = hkv, G, d, page, lens
        self.dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.dtype, self.scale = dtype, 2.0 ** -6
        used = [-(-n // page) for n in lens]
        num, cols = sum(used) + 2, max(used)
        order = torch.randperm(num, generator=gen, device="cuda")
        self.table = torch.zeros(seqs, cols, dtype=torch.int32, device="cuda")
        at = 0
        for u, n in enumerate(used):
            self.table[u, :n] = order[at:at + n]
            at += n
        self.shape = kv.KvPagedShape.of(seqs, hkv * G, hkv, d, 1, page, cols, dtype, num)

        def ints(most, *size):
            return torch.randint(-most, most + 1, size, generator=gen, device="cuda",
                                 dtype=torch.int8).to(self.dt)

        if whole:
            self.q, self.kp = ints(3, seqs, hkv * G, d), ints(2, num, hkv, page, d)
        else:
            self.q = torch.zeros(seqs, hkv * G, d, dtype=self.dt, device="cuda")
            self.kp = torch.zeros(num, hkv, page, d, dtype=self.dt, device="cuda")
            self.q[..., 3], self.scale = 1, 0.7
            for u, n in enumerate(used):
                self.kp[self.table[u, :n:128 // page].long(), :, 0, 3] = 1
        self.vp = self.v_all = torch.rand(num, hkv, page, d, generator=gen, device="cuda").add_(0.5).to(self.dt)
        self.lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def rows(self, pool, u, h):
        n = self.lens[u]
        pages = self.table[u, :-(-n // self.page)].long()
        return pool[pages, h].flatten(0, 1)[:n]

    def mark_blocks(self, i, m):
        """V of block b (8 rows) of a head is left in column b % d, and only where b / d % m = i."""
        v = self.v_all
        for u, n in enumerate(self.lens):
            pages = self.table[u, :-(-n // self.page)].long()
            b = torch.arange(len(pages) * self.page, device="cuda").view(-1, 1, self.page, 1) // 8
            col = torch.arange(self.d, device="cuda")
            for x in range(0, len(pages), 4096):
                y = b[x:x + 4096]
                self.vp[pages[x:x + 4096]] = v[pages[x:x + 4096]] * (
                    (y % self.d == col) & (y // self.d % m == i))

    def run(self):
        out = torch.full((len(self.lens), self.hkv * self.G, self.d), float("nan"), dtype=self.dt,
                         device="cuda")
        ws = workspace(kv.KV_OP_PAGED_DECODE, self.shape)
        kv.paged_decode_attn(self.shape, self.q, None, None, None, None, self.kp, self.vp,
                             self.table, self.lens_t, self.scale, out, ws)
        assert kv.kv_check_device_status(ws) == 0
        return out.double()

    def expected(self):
        """64 bits, and the largest distance of a score to its maximum, times scale."""
        out = torch.zeros(len(self.lens), self.hkv * self.G, self.d, dtype=torch.float64,
                          device="cuda")
        far = 0.0
        for u in range(len(self.lens)):
            for h in range(self.hkv):
                g = slice(h * self.G, (h + 1) * self.G)
                z = self.q[u, g].double() @ self.rows(self.kp, u, h).double().T * self.scale
                z -= z.amax(1, keepdim=True)
                far = max(far, float(-z.amin()))
                p = z.exp()
                out[u, g] = (p / p.sum(1, keepdim=True)) @ self.rows(self.vp, u, h).double()
        return out, far

    def tiles_of_a_warp(self):
        """At most: an even share of the tiles, and what a boundary moves by."""
        rt = 8 if self.dtype == "f32" and self.d > 80 else 16
        tiles = sum(-(-n // rt) for n in self.lens) * self.hkv
        warps = 8 * torch.cuda.get_device_properties(0).multi_processor_count
        return tiles // warps + 25


@pytest.mark.parametrize("seqs,hkv,G,d,lens", [
    (1, 1, 2, 8, [6000001]), (3, 4, 4, 64, [90001, 250000, 17]), (1, 8, 4, 128, [131072]),
    (40, 2, 1, 72, [20000 + 37 * i for i in range(40)]), (2, 8, 8, 96, [40000, 9]),
    (64, 8, 4, 64, [8000] * 64), (16, 8, 2, 128, [24000] * 16)])
def test_decode_fp32_sums_over_many_tiles(seqs, hkv, G, d, lens):
    """Two weights, 1 and exp(-0.7), and positive values: all that can be off is what is kept of
    weights and values and their sums.  (An error that all rows of one weight share moves the output
    by its part times the difference of the two kinds' means.)  V and the weights count to 22 bits
    of the half that has all rows, 2^-22 each at most.  What the matrix instruction adds by itself is
    4 tiles, 32 sums at most, each cut off by up to 2^-23; that 64, and as much as half of it again for
    the merges, in units of 2^-24.  All else is rounded to the nearest: of D errors of at most
    2^-24 with no sign of their own, in the output and in the sum of the weights, 8 sqrt(D) is more
    than ten standard deviations (2^-24 / sqrt(3) each).  Sums that are cut off over all D tiles
    lean to one side, by 2^-24 and more a tile."""
    c = Many(seqs, hkv, G, d, 64, lens, "f32", 51, whole=False)
    want, _ = c.expected()
    D = c.tiles_of_a_warp()
    tol = (2 * 2.0 ** -22 + (16 * D ** 0.5 + 96) * 2.0 ** -24) * want
    off = (c.run() - want).abs()
    assert bool((off <= tol).all()), (D, float((off / want).max() * 2 ** 24))


@pytest.mark.parametrize("dtype,seqs,hkv,G,d,lens", [
    ("bf16", 1, 8, 1, 128, [65001]), ("bf16", 1, 4, 4, 128, [20011]),
    ("bf16", 4, 8, 3, 64, [30000, 9000, 100, 26001]), ("bf16", 1, 1, 8, 64, [100000]),
    ("bf16", 51, 8, 2, 128, [3] * 49 + [20000, 45000]), ("bf16", 1, 2, 4, 8, [20001]),
    ("f32", 1, 8, 1, 40, [65001]), ("f32", 52, 4, 1, 40, [1] * 50 + [20000, 45000]),
    ("f32", 1, 8, 2, 128, [65001]), ("f32", 7, 2, 5, 72, [20011, 8, 7, 16, 40000, 33, 1000]),
    ("bf16", 200, 8, 4, 128, [900 + 13 * i for i in range(200)]),
    # (33 to 38 tables: more than a warp holds, and CTAs of eight warps)
    ("bf16", 36, 1, 4, 128, [9000 - 250 * i for i in range(36)]),
    ("f32", 34, 1, 3, 72, [4, 8000] * 17), ("f32", 37, 1, 8, 128, [100 * i for i in range(1, 38)])])
def test_decode_no_tile_of_a_long_head_is_lost(dtype, seqs, hkv, G, d, lens):
    """Warps with more than 32 tiles, units that cross many CTAs: every 8 rows count in one column
    of V alone (a call for every m-th part of them), so a tile that is left out, taken twice or from
    a wrong page moves that column by about 8 d m / n of itself, and by a fifth of that where its
    weights are small: more than four times the bound.  That is the weights' errors (2^-22 for
    exp2, the exponent's rounding, and each of at most 64 rescalings), their bits, sums of D tiles,
    the output's rounding; scores are exact and all values positive.  One such loss is put into the
    expected values of the longest head, on the CPU, and has to be past the bound."""
    c = Many(seqs, hkv, G, d, 32, lens, dtype, 52)
    c.vp = c.v_all.clone()
    t_p = 2.0 ** -16 if dtype == "bf16" else 2.0 ** -20
    m = -(-max(lens) // (80 * d))
    for i in range(m):
        c.mark_blocks(i, m)
        want, far = c.expected()
        rel = (2 * (64 + far) * 2.0 ** -22 + t_p + (2 * c.tiles_of_a_warp() + 64) * U23 +
               torch.finfo(c.dt).eps / 2)
        assert 4 * rel < 0.2 * 8 * d * m / max(lens)      # (what the test rests on)
        off = (c.run() - want).abs()
        assert bool((off <= rel * want.abs() + 1e-37).all()), (i, float((off / want).nan_to_num().max()))
        if i == 0:
            u = lens.index(max(lens))
            k, v = (c.rows(pool, u, 0).double().cpu() for pool in (c.kp, c.vp))
            p = (c.q[u, :G].double().cpu() @ k.T * c.scale).exp()
            p /= p.sum(1, keepdim=True)
            assert torch.allclose(p @ v, want[u, :G].cpu(), rtol=1e-9)
            for first in (0, 32, 48):            # blocks of part 0: its first d
                lost = p.clone()
                lost[:, first:first + 8] = 0
                lost /= lost.sum(1, keepdim=True)
                moved = (lost @ v - p @ v).abs() > rel * (p @ v)
                assert bool(moved.any(1).all())


# ------------------------------------------------------------------------------- capacity

@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 72), ("f32", 64), ("f32", 128)])
@pytest.mark.parametrize("lens", [[500], [1, 0, 17], [3001, 40], [5] * 40 + [700]])
def test_decode_short_rows_in_long_tables(dtype, d, lens):
    """Block tables sized for 131072 rows a sequence, as a server sizes them, and few rows held: the
    host goes by the capacity, the kernel by the lengths."""
    c = Cache(len(lens), 2, 4, d, 1, 16, lens, dtype, 44)
    far = torch.full((len(lens), 131072 // 16), -1, dtype=torch.int32, device="cuda")
    far[:, :c.max_pages] = c.table
    c.table = far
    c.shape = kv.KvPagedShape.of(len(lens), 8, 2, d, 1, 16, far.shape[1], dtype, c.num_pages)
    out, ws = c.run()
    assert kv.kv_check_device_status(ws) == 0
    c.check(out)
    c.check_pools()


def test_calls_of_several_shapes_share_a_workspace():
    """One workspace for maps, writes and decodes of several shapes, one after the other on a stream:
    the results of workspaces of their own."""
    caches = [Cache(len(n), 2, G, d, t, 16, n * t, dtype, 45 + d, new=[0] * len(n) * t)
              for n, G, d, t, dtype in (([3000, 5, 700], 4, 128, 1, "bf16"), ([9000], 2, 72, 1, "f32"),
                                        ([40] * 60, 1, 64, 2, "bf16"), ([20000, 16], 8, 96, 1, "bf16"))]
    want = [c.run()[0] for c in caches]
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")
    i32 = torch.int32
    s = kv.KvPagedShape.of(40, 1, 1, 64, 1, 8, 2000, "bf16", 40000)
    lens, add = torch.zeros(40, dtype=i32, device="cuda"), torch.full((40,), 900, dtype=i32,
                                                                      device="cuda")
    ring = torch.arange(40000, dtype=i32, device="cuda")
    state = torch.tensor([0, 40000], device="cuda")
    table = torch.full((40, 2000), -1, dtype=i32, device="cuda")
    cu, slots = torch.zeros(41, dtype=torch.int64, device="cuda"), torch.zeros(
        36000, dtype=torch.int64, device="cuda")
    rows = torch.randn(36000, 1, 64, device="cuda").bfloat16()
    kp, vp = (torch.zeros(40000, 1, 8, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for step in range(6):
        kv.kv_page_map(s, lens, add, ring, state, table, lens, state, cu, slots, ws)
        kv.kv_paged_write(s, rows, rows, slots, cu[40:], kp, vp, ws)
        for c, w in zip(caches, want):
            assert torch.equal(c.run(ws=ws)[0], w)
        assert lens.tolist() == [900 * (step + 1)] * 40
        assert bool((kp[slots // 8, 0, slots % 8] == rows[:, 0]).all())
    assert kv.kv_check_device_status(ws) == 0
    # (a page that is never given back: 900 rows six times are 675 pages a table)
    assert state.tolist() == [40 * 675, 40000]


# ------------------------------------------------------------------------------- binding

@pytest.mark.parametrize("slots", [None, "empty"])
def test_map_that_only_gives_pages_back_has_no_slot_map(slots):
    """slot_map NULL with a capacity of 0, as the header allows it: None, or an empty tensor."""
    i32, i64 = torch.int32, torch.int64
    s = kv.KvPagedShape.of(3, 1, 1, 64, 1, 8, 4, "bf16", 12)
    lens = torch.tensor([30, 8, 17], dtype=i32, device="cuda")
    add = torch.tensor([-30, 0, -9], dtype=i32, device="cuda")
    ring = torch.arange(12, dtype=i32, device="cuda")
    state = torch.tensor([8, 12], device="cuda")
    table = torch.tensor([[0, 1, 2, 3], [4, -1, -1, -1], [5, 6, 7, -1]], dtype=i32, device="cuda")
    cu = torch.zeros(4, dtype=i64, device="cuda")
    ws = workspace(kv.KV_OP_PAGE_MAP, s)
    kv.kv_page_map(s, lens, add, ring, state, table, lens, state, cu,
                   None if slots is None else torch.zeros(0, dtype=i64, device="cuda"), ws)
    assert kv.kv_check_device_status(ws) == 0
    assert lens.tolist() == [0, 8, 8] and state.tolist() == [8, 18] and cu.tolist() == [0] * 4
    assert [ring[i % 12].item() for i in range(8, 18)] == [8, 9, 10, 11, 0, 1, 2, 3, 6, 7]


def test_binding_refuses_missing_tensors():
    """None where a call needs a tensor is an error of the library or a ValueError, as elsewhere."""
    c = Cache(2, 2, 2, 64, 1, 16, [20, 30], "bf16", 14)
    ws = workspace(kv.KV_OP_PAGED_DECODE, c.shape)
    out = torch.empty_like(c.qd)
    args = [c.qd, c.knd, c.vnd, c.cu, c.slots, c.kp, c.vp, c.table, c.lens_t, 0.1, out, ws]
    for i in (0, 1, 2, 3, 5, 6, 7, 8, 10, 11):     # (slot_map may be None: no slots)
        with pytest.raises((kv.KvError, ValueError)):
            kv.paged_decode_attn(c.shape, *[None if j == i else x for j, x in enumerate(args)])
    rows = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    args = [rows, rows, c.slots, None, c.kp, c.vp, ws]
    for i in (0, 1, 2, 4, 5, 6):
        with pytest.raises((kv.KvError, ValueError)):
            kv.kv_paged_write(c.shape, *[None if j == i else x for j, x in enumerate(args)])
    ring = torch.zeros(c.num_pages, dtype=torch.int32, device="cuda")
    state = torch.zeros(2, dtype=torch.int64, device="cuda")
    args = [c.lens_t, c.lens_t.clone(), ring, state, c.table, c.lens_t, state, c.cu, c.slots, ws]
    for i in (0, 1, 2, 3, 4, 5, 6, 7, 9):
        with pytest.raises((kv.KvError, ValueError)):
            kv.kv_page_map(c.shape, *[None if j == i else x for j, x in enumerate(args)])
