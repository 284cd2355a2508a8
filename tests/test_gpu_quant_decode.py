"""quant_decode_attn on the GPU against 64 bits, each where it can go wrong, and the calls of a
serving step together."""
import numpy as np
import pytest
import torch

import kv_cache_eviction_gb300 as kv
from tests.paged import ERR_ID, ERR_TABLE, ceil_div, workspace
from tests.quant import BLOCK, FORMATS, QuantCache, put

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kv_cache_eviction_gb300 import _build
    _build.build()
    kv.lib()


LENS = {"one": [1], "few": [3, 1, 2], "empty": [0, 5, 0, 0, 17, 0], "none": [0, 0],
        "ends": [15, 16, 17, 31, 32, 33, 127, 128, 129], "long": [5000, 1, 0, 2047],
        "ragged": [700, 3, 64, 0, 1500, 260, 8, 90], "big": [20011]}


def finish(c, out, ws):
    torch.cuda.synchronize()
    assert kv.kv_check_device_status(ws) == 0
    c.put()
    c.check(out)
    c.check_pools()


@pytest.mark.parametrize("kind", list(LENS))
@pytest.mark.parametrize("fmt,dtype,d,G,page,tables", [
    ("e4m3", "bf16", 128, 4, 16, 1), ("int8", "bf16", 128, 8, 64, 1),
    ("e4m3", "bf16", 64, 1, 16, 1), ("int8", "f32", 128, 2, 16, 1), ("e4m3", "bf16", 128, 4, 32, 4), ("e4m3", "f32", 80, 3, 16, 4),
    ("int8", "bf16", 80, 5, 256, 1), ("e4m3", "bf16", 16, 7, 16, 1), ("e4m3", "f32", 64, 8, 128, 1),
    ("int8", "f32", 32, 6, 128, 4), ("int8", "bf16", 48, 3, 32, 4), ("e4m3", "f32", 112, 4, 64, 1)])
def test_decode(kind, fmt, dtype, d, G, page, tables):
    hkv, base = 4, LENS[kind]
    lens = [base[i % len(base)] for i in range(len(base) * tables)]
    c = QuantCache(len(base), hkv, G, d, tables, page, lens, dtype, fmt, seed=d + G + page)
    out, ws = c.run()
    finish(c, out, ws)
    # the same workspace and rows again: the same bits, and the row that the first call stored,
    # read from the pool, gives them too
    again, _ = c.run(ws=ws)
    assert torch.equal(out, again)
    assert torch.equal(out, c.run(with_new=False, ws=ws)[0])
    c.check_pools()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_idle_sequences_and_many(dtype, fmt):
    """Sequences that got no row attend over what they hold; many short ones and few long."""
    rng = np.random.default_rng(8)
    lens = rng.integers(0, 40, 300)
    lens[[5, 77, 200]] = [3000, 1500, 900]
    c = QuantCache(300, 2, 4, 128, 1, 16, lens, dtype, fmt, 3, new=rng.random(300) < 0.5)
    out, ws = c.run()
    finish(c, out, ws)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_head_tables_skewed(fmt):
    """A table per head with lengths from none to thousands, as head-adaptive budgets give."""
    rng = np.random.default_rng(9)
    lens = np.minimum(np.exp(rng.normal(4.5, 1.5, 24 * 8)), 6000).astype(int)
    lens[::11] = 0
    c = QuantCache(24, 8, 4, 128, 8, 16, lens, "bf16", fmt, 4, new=rng.random(24 * 8) < 0.8)
    out, ws = c.run()
    finish(c, out, ws)


@pytest.mark.parametrize("lens", [[30000, 9000, 100, 26001], [1] * 50 + [20000, 45000], [65001]])
@pytest.mark.parametrize("fmt,dtype,d,G", [("e4m3", "bf16", 128, 1), ("int8", "bf16", 64, 3),
                                           ("e4m3", "f32", 48, 1), ("int8", "f32", 128, 2)])
def test_many_tiles_a_warp(fmt, dtype, d, G, lens):
    """Warps with over 32 tiles, units cut many times, CTAs of four and of eight warps."""
    c = QuantCache(len(lens), 2, G, d, 1, 64, lens, dtype, fmt, 12)
    out, ws = c.run()
    finish(c, out, ws)
    for _ in range(5):
        assert torch.equal(out, c.run(ws=ws)[0])


@pytest.mark.parametrize("G", [1, 3, 5, 6, 7, 8])
@pytest.mark.parametrize("d", [16, 32, 48, 64, 80, 96, 112, 128])
def test_every_width_over_many_ctas(d, G):
    """Units whose parts go through the workspace, at every width and group size: few long units on
    CTAs of eight warps, and more, with shorter tables, on CTAs of four."""
    fmt, dtype = ("e4m3", "int8")[G % 2], ("bf16", "f32")[d // 16 % 2]
    for hkv, lens in ((1, [40001]), (8, [3001, 17, 900, 0, 2500, 1200])):
        c = QuantCache(len(lens), hkv, G, d, 1, 32, lens, dtype, fmt, d + G)
        out, ws = c.run()
        finish(c, out, ws)


def test_thousands_of_tables():
    """More tables than a CTA has threads: strips of tables, windows that move on."""
    rng = np.random.default_rng(7)
    lens = rng.integers(0, 30, 5000)
    lens[[3, 2500, 4990]] = [2000, 900, 40]
    c = QuantCache(1250, 4, 2, 32, 4, 16, lens, "bf16", "e4m3", 8, new=rng.random(5000) < 0.7)
    out, ws = c.run()
    finish(c, out, ws)


@pytest.mark.parametrize("d,G,dtype", [(16, 1, "f32"), (80, 7, "bf16"), (128, 8, "f32"),
                                       (64, 5, "bf16")])
def test_nothing_around_the_outputs(d, G, dtype):
    """Sentinels before and behind the output and the workspace stay, and so do all inputs."""
    for lens in ([9000, 0, 33], [5] * 300):
        c = QuantCache(len(lens), 2, G, d, 1, 32, lens, dtype, "int8", d)
        n, pad = c.seqs * c.hkv * G * d, 256
        buf = torch.full((n + 2 * pad,), 3.0, dtype=c.dt, device="cuda")
        out = buf[pad:pad + n].view(c.seqs, c.hkv * G, d)
        m = kv.kv_paged_workspace_size(kv.KV_OP_QUANT_DECODE, c.shape)
        wbuf = torch.full((m + 512,), 77, dtype=torch.uint8, device="cuda")
        wbuf[256:256 + m] = 0
        ins = [c.qd, c.knd, c.vnd, c.cu, c.slots, c.table, c.lens_t]
        was = [t.clone() for t in ins]
        c.run(ws=wbuf[256:256 + m], out=out)
        torch.cuda.synchronize()
        assert bool((buf[:pad] == 3.0).all()) and bool((buf[pad + n:] == 3.0).all())
        assert bool((wbuf[:256] == 77).all()) and bool((wbuf[256 + m:] == 77).all())
        assert all(torch.equal(a, b) for a, b in zip(ins, was))
        # what the calls that share the workspace need at zero: the error word and the tickets
        assert not bool(wbuf[256:256 + 256 + 2048].any())
        c.put()
        c.check(out)
        c.check_pools()


@pytest.mark.parametrize("hkv,G,d,lens", [(2, 8, 96, [2061, 2500]), (1, 8, 128, [1500] * 40),
                                          (8, 5, 128, [4000]), (4, 8, 112, [900, 2000, 5100, 333]),
                                          (3, 7, 48, [3100, 1250, 7000])])
def test_same_bits_whoever_is_last(hkv, G, d, lens):
    """Units of many parts, cut in the middle of CTAs: which CTA ends last, and whether it then has
    one unit to merge or two, changes from run to run, with other work on the GPU; the bits do not."""
    noise = torch.randn(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    for seed in range(3):
        c = QuantCache(len(lens), hkv, G, d, 1, 64, lens, "f32", ("e4m3", "int8")[seed % 2], seed)
        out, ws = c.run()
        for i in range(40):
            if i % 4 == 1:
                side.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(side):
                    noise @ noise if i % 8 == 1 else noise.add_(1)
            assert torch.equal(out, c.run(ws=ws)[0])
        finish(c, out, ws)


@pytest.mark.parametrize("extra", [16, 128, 4096])
def test_page_stride(extra):
    c = QuantCache(3, 2, 4, 128, 1, 16, [100, 0, 333], "bf16", "e4m3", 5, extra=extra)
    out, ws = c.run()
    finish(c, out, ws)


def test_far_pages():
    """Rows past 2^32 bytes of the pool, at a stride of 4 MB."""
    c = QuantCache(2, 2, 4, 128, 1, 256, [300, 1000], "bf16", "int8", 6, first_page=1200,
                   extra=(1 << 22) - 2 * 256 * 128)
    assert c.num_pages * c.apart > 1 << 32
    out, ws = c.run()
    finish(c, out, ws)


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0, 1e-30, 1e20])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_softmax_scales(dtype, scale):
    """Zero, negative, sharp and extreme scales; the bound follows the scores' size."""
    c = QuantCache(3, 2, 4, 64, 1, 16, [40, 0, 700], dtype, "e4m3", 7)
    c.softmax_scale = scale
    out, ws = c.run()
    torch.cuda.synchronize()
    assert kv.kv_check_device_status(ws) == 0
    c.put()
    if scale == 1e20:     # the largest score alone
        for b, n in ((0, 40), (2, 700)):
            for g in range(8):
                k, v = c.rows(b, "k")[g // 4], c.rows(b, "v")[g // 4]
                z = k @ c.q[b, g].double().numpy()
                top = np.sort(z)
                if top[-1] - top[-2] > 1e-4 * np.abs(top[-1]):
                    got = out[b, g].double().cpu().numpy()
                    assert (np.abs(got - v[z.argmax()]) <= 2.0 ** -8 * np.abs(got) + 1e-30).all()
    else:
        c.check(out)


@pytest.mark.parametrize("q_exp,k_exp", [(100, -90), (-100, 80), (60, -96), (-20, -96), (0, 110)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_far_magnitudes(dtype, q_exp, k_exp):
    """Queries and scales at the ends of their ranges, with scores of ordinary size (or none)."""
    c = QuantCache(2, 2, 3, 80, 1, 16, [50, 300], dtype, "int8", 8, new=[0, 0], spread=0.0)
    c.q = (c.q.float() * 2.0 ** q_exp).to(c.dt)
    c.qd = c.q.cuda()
    held = np.isfinite(c.scale["k"])
    c.scale["k"][held] = 2.0 ** (k_exp - 6)
    c.scale["v"][held] = 2.0 ** min(k_exp - 6, 110)
    if k_exp - 6 < -96:
        c.scale["k"][held], c.scale["v"][held] = 2.0 ** -96, 2.0 ** -96
    for n in ("k", "v"):
        c.scale_dev[n].copy_(torch.tensor(c.scale[n]))
    if q_exp + k_exp > 20:
        c.softmax_scale = 2.0 ** -(q_exp + k_exp) / 9
    out, ws = c.run()
    torch.cuda.synchronize()
    assert kv.kv_check_device_status(ws) == 0
    c.check(out)


def test_growing_rows():
    """A sequence step by step, with rows whose size jumps: every step's block, scale and output."""
    c = QuantCache(2, 2, 4, 64, 1, 32, [1, 14], "bf16", "int8", 9)
    pages = c.num_pages
    table = np.array([[0, 2], [1, 3]])
    c.table_host = table
    c.table.fill_(0)
    c.max_pages = 2
    c.shape.max_pages = 2
    c.table = torch.tensor(table, dtype=torch.int32, device="cuda")
    ws = workspace(kv.KV_OP_QUANT_DECODE, c.shape)
    assert pages >= 4
    rng = np.random.default_rng(3)
    for name in ("k", "v"):      # rows 0..12 of the second table's first page
        c.num[name][1, :, :13] = rng.integers(-127, 128, (2, 13, 64))
        c.scale[name][1, :, 0] = 2.0 ** -7
        c.pool[name][1].copy_(torch.tensor(c.num[name]).to(torch.int8))
        c.scale_dev[name].copy_(torch.tensor(c.scale[name]))
    for step in range(45):
        c.lens = [1 + step, 14 + step]
        c.lens_t.copy_(torch.tensor(c.lens))
        size = 2.0 ** rng.integers(-6, 9)
        c.k_new = (torch.tensor(rng.normal(size=(2, 2, 64))) * min(size, 2.0)).bfloat16()
        c.v_new = (torch.tensor(rng.normal(size=(2, 2, 64))) * size).bfloat16()
        c.knd.copy_(c.k_new)
        c.vnd.copy_(c.v_new)
        c.slots_host = [int(table[u, (n - 1) // 32]) * 32 + (n - 1) % 32
                        for u, n in enumerate(c.lens)]
        c.slots.copy_(torch.tensor(c.slots_host))
        out, _ = c.run(ws=ws)
        finish(c, out, ws)


def test_bad_pages_slots_and_lengths():
    """Pages outside the pool are left out of the sums, lengths outside the table are cut to it;
    each is reported, and nothing is stored."""
    c = QuantCache(3, 2, 4, 128, 1, 16, [100, 40, 64], "bf16", "e4m3", 7, new=[0, 0, 0])
    c.table[0, 2] = c.num_pages
    c.table[1, 0] = -1
    c.table[2, 3] = 1 << 30
    out, ws = c.run()
    assert kv.kv_check_device_status(ws) == ERR_ID
    c.check(out, skip={(0, 2), (1, 0), (2, 3)})
    c.check_pools()
    c = QuantCache(3, 2, 4, 64, 1, 16, [48, 5, 7], "bf16", "int8", 8, new=[0, 0, 0])
    c.lens_t.copy_(torch.tensor([4000, -3, 7]))
    out, ws = c.run()
    assert kv.kv_check_device_status(ws) == ERR_TABLE
    c.lens = [48, 0, 7]
    c.check(out)
    c.check_pools()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_slots_elsewhere(fmt):
    """A new row is stored at its table's own place only: slots that are -1 leave the table as it
    is (its last row is the pool's), others out of place are reported."""
    for slot, code in ((-1, 0), (-2, ERR_ID), (10 ** 9, ERR_ID), (1 << 62, ERR_ID),
                       ("next", ERR_ID), ("block", ERR_ID)):
        c = QuantCache(3, 2, 4, 64, 1, 32, [50, 40, 37], "bf16", fmt, 9, new=[0, 0, 0], spare=2)
        own = [int(c.table_host[u, (n - 1) // 32]) * 32 + (n - 1) % 32
               for u, n in enumerate(c.lens)]
        if slot == "next":
            slot = own[1] + 1
        if slot == "block":
            slot = own[1] - 16 if own[1] % 32 >= 16 else own[1] + 16
        c.cu.copy_(torch.tensor([0, 1, 2, 3]))
        c.slots = torch.tensor([own[0], slot, own[2]], device="cuda")
        out, ws = c.run()
        torch.cuda.synchronize()
        assert kv.kv_check_device_status(ws) == code
        c.new, c.slots_host = [1, 0, 1], [own[0], own[2]]
        c.put()
        c.check(out)
        c.check_pools()


def test_new_row_whose_page_is_outside_the_pool():
    """A table whose last page is no page of the pool: its new row is stored nowhere, whatever its
    slot says."""
    for page in (-1, 1 << 20):
        c = QuantCache(2, 2, 4, 64, 1, 16, [20, 40], "bf16", "int8", 10)
        bad = int(c.table_host[0, 1])
        c.table[0, 1] = page
        c.slots[0] = 3                      # a row of page 0
        assert bad != page
        out, ws = c.run()
        assert kv.kv_check_device_status(ws) == ERR_ID
        c.put(skip={0})
        c.check(out, skip={(0, 1)})
        c.check_pools()


@pytest.mark.parametrize("where", ["q", "k", "v", "k_new", "v_new"])
@pytest.mark.parametrize("n", [1, 40, 9000])
def test_nan_reaches_the_outputs(where, n):
    """A NaN query, or a NaN in a row that counts, is one in the outputs it reaches, and nowhere
    else."""
    c = QuantCache(3, 2, 2, 64, 1, 16, [33, n, 70], "bf16", "e4m3", 11)
    r = 0 if "new" not in where and n > 1 else n - 1
    if where == "q":
        c.qd[1, 1, 5] = float("nan")
    elif "new" in where:
        (c.knd if where == "k_new" else c.vnd)[1, 0, 7] = float("nan")
    elif n == 1:
        return                              # (its only row is the new one)
    else:
        c.pool[where][1].view(torch.uint8)[c.table_host[1, r // 16], 0, r % 16, 7] = 127
    out, ws = c.run()
    torch.cuda.synchronize()
    assert kv.kv_check_device_status(ws) == 0
    nan = torch.isnan(out.cpu().float())
    want = torch.zeros_like(nan)
    if where == "q":
        want[1, 1] = True
    elif where in ("v", "v_new"):
        want[1, :2, 7] = True
    else:
        want[1, :2] = True
    assert torch.equal(nan, want)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_as_write_then_attend(fmt, dtype):
    """Storing the new rows with kv_quant_write first gives the same pools and the same bits; and
    the rows read back give what the attention saw."""
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 90, 40)
    a, b = (QuantCache(10, 4, 2, 96, 4, 32, lens, dtype, fmt, 6) for _ in range(2))
    x, ws = a.run()
    rows = lambda t: t.reshape(-1, 1, 96)[torch.tensor(b.new)].contiguous().cuda()
    kv.kv_quant_write(b.shape, FORMATS[fmt], rows(b.k_new), rows(b.v_new), b.slots, None, *b.args(),
                      ws)
    y, _ = b.run(with_new=False, ws=ws)
    assert torch.equal(x, y)
    for c in (a, b):
        c.put()
        c.check_pools()
    a.check(x)
    u = int(np.argmax(lens))
    r = np.arange(lens[u])
    slots = torch.tensor(a.table_host[u, r // 32] * 32 + r % 32, device="cuda")
    k, v = (torch.zeros(len(r), 1, 96, dtype=a.dt, device="cuda") for _ in range(2))
    kv.kv_quant_read(a.shape, FORMATS[fmt], *a.args(), slots, None, k, v, ws)
    for t, name in ((k, "k"), (v, "v")):
        assert np.array_equal(t[:, 0].double().cpu().numpy(), a.rows(u, name)[0])
    assert kv.kv_check_device_status(ws) == 0


def test_serving_steps_captured():
    """Page map, rotation, row write and decode as a serving program runs them: two prompts, then
    a captured step replayed through the ends of blocks and pages, against 64 bits."""
    seqs, hq, hkv, d, page, cols, fmt = 3, 8, 2, 64, 32, 6, "e4m3"
    rng = np.random.default_rng(4)
    num = seqs * cols
    shape = kv.KvPagedShape.of(seqs, hq, hkv, d, 1, page, cols, "bf16", num)
    dev = lambda x, t: torch.tensor(np.asarray(x), dtype=t, device="cuda")
    i32, i64 = torch.int32, torch.int64
    lens, add, ring = dev([0] * seqs, i32), dev([0] * seqs, i32), dev(rng.permutation(num), i32)
    state, table = dev([0, num], i64), dev(np.zeros((seqs, cols)), i32)
    cu = dev([0] * (seqs + 1), i64)
    kp, vp = (torch.zeros(num, hkv, page, d, dtype=torch.float8_e4m3fn, device="cuda")
              for _ in range(2))
    ks, vs = (torch.full((num, hkv, page // 16), float("nan"), device="cuda") for _ in range(2))
    ws = workspace(kv.KV_OP_QUANT_DECODE, shape)
    freq = kv.kv_rotary_inv_freq(d)[0]
    rot = kv.KvRotaryShape.of(hq, hkv, d, d, kv.KV_ROTARY_HALF, "bf16")
    fd = freq.cuda()
    host = {n: (np.zeros((num, hkv, page, d)), np.full((num, hkv, page // 16), np.nan))
            for n in ("k", "v")}

    # prompts of 45 and 20 rows; the third sequence starts empty
    n = [45, 20, 0]
    add.copy_(dev(n, i32))
    slots = dev([-1] * 65, i64)
    kv.kv_page_map(shape, lens, add, ring, state, table, lens, state, cu, slots, ws)
    qkv = torch.randn(65, hq + 2 * hkv, d, generator=torch.Generator().manual_seed(1)).bfloat16()
    x = qkv.cuda()
    pos = dev(np.concatenate([np.arange(m) for m in n]), i32)
    kv.kv_rotary(rot, x[:, :hq], x[:, hq:hq + hkv], pos, fd, x[:, :hq], x[:, hq:hq + hkv])
    kv.kv_quant_write(shape, kv.KV_E4M3, x[:, hq:hq + hkv], x[:, hq + hkv:], slots, cu[seqs:],
                      kp, vp, ks, vs, ws)
    s = slots.cpu().numpy()
    for name, rows in (("k", x[:, hq:hq + hkv]), ("v", x[:, hq + hkv:])):
        put(*host[name], rows.double().cpu().numpy(), s, fmt)

    # one token of each
    new = torch.zeros(seqs, hq + 2 * hkv, d, dtype=torch.bfloat16, device="cuda")
    q, kn, vn = (torch.zeros(seqs, h, d, dtype=torch.bfloat16, device="cuda")
                 for h in (hq, hkv, hkv))
    out = torch.zeros_like(q)
    slots = dev([-1] * seqs, i64)
    add.fill_(1)
    where = dev([0] * seqs, i32)

    def step():
        where.copy_(lens)
        kv.kv_page_map(shape, lens, add, ring, state, table, lens, state, cu, slots, ws)
        kv.kv_rotary(rot, new[:, :hq], new[:, hq:hq + hkv], where, fd, q, kn)
        vn.copy_(new[:, hq + hkv:])
        kv.quant_decode_attn(shape, kv.KV_E4M3, q, kn, vn, cu, slots, kp, vp, ks, vs, table, lens,
                             d ** -0.5, out, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step()
    g = torch.Generator().manual_seed(2)
    held = np.array(n)
    for i in range(60):
        new.copy_(torch.randn(seqs, hq + 2 * hkv, d, generator=g) * (1 + i % 7))
        graph.replay()
        torch.cuda.synchronize()
        held += 1
        assert lens.tolist() == held.tolist()
        for name, rows in (("k", kn), ("v", vn)):
            r = rows.double().cpu().numpy()
            for u, slot in enumerate(slots.tolist()):
                put(*host[name], r[u:u + 1], [slot], fmt)
        for name, pool, sc in (("k", kp, ks), ("v", vp, vs)):
            assert np.array_equal(pool.double().cpu().numpy(), host[name][0])
            assert np.array_equal(sc.double().cpu().numpy(), host[name][1], equal_nan=True)
        # rotation: angles in 64 bits, bf16's rounding and 2^-20 for float32
        y = new.double().cpu().numpy()
        t = (held - 1)[:, None, None] * freq.numpy()
        a, b = y[..., :d // 2], y[..., d // 2:]
        turned = np.concatenate([a * np.cos(t) - b * np.sin(t), a * np.sin(t) + b * np.cos(t)], 2)
        lim = 2.0 ** -8 * np.abs(turned) + 2.0 ** -20 * (np.abs(y).max() + 1)
        assert (np.abs(q.double().cpu().numpy() - turned[:, :hq]) <= lim[:, :hq]).all()
        assert (np.abs(kn.double().cpu().numpy() - turned[:, hq:hq + hkv])
                <= lim[:, hq:hq + hkv]).all()
        if i % 10 == 9 or i < 3:
            tb = table.cpu().numpy()
            for u in range(seqs):
                at = tb[u, :ceil_div(held[u], page)]
                k, v = ((host[m][0][at] * np.repeat(host[m][1][at], BLOCK, 2)[..., None])
                        .transpose(1, 0, 2, 3).reshape(hkv, -1, d)[:, :held[u]] for m in ("k", "v"))
                for h in range(hq):
                    z = k[h // 4] @ q[u, h].double().cpu().numpy() * d ** -0.5
                    p = np.exp(z - z.max())
                    p /= p.sum()
                    want, mag = p @ v[h // 4], p @ np.abs(v[h // 4])
                    # fp32 sums of d products of scores up to |z| and of held weights, then
                    # bf16's rounding: half of its step, 2^-7 of the value
                    tol = (2.0 ** -8 * np.abs(want) + mag * 2.0 ** -23 * (
                        4 * (d + 10) * (1 + np.abs(z).max() * 8) + 3 * len(z)))
                    assert (np.abs(out[u, h].double().cpu().numpy() - want) <= tol).all()
    assert kv.kv_check_device_status(ws) == 0


def test_shared_workspace_two_graphs_and_streams():
    """Two captured calls of different shapes that share a workspace, replayed in turn on one
    stream, and a third on another stream with its own."""
    a = QuantCache(2, 2, 4, 128, 1, 16, [9000, 400], "bf16", "e4m3", 1)
    b = QuantCache(40, 4, 2, 64, 4, 32, [97] * 160, "f32", "int8", 2)
    big = max(kv.kv_paged_workspace_size(kv.KV_OP_QUANT_DECODE, c.shape) for c in (a, b))
    ws = torch.zeros(big, dtype=torch.uint8, device="cuda")
    side, graphs, outs = torch.cuda.Stream(), [], []
    side.wait_stream(torch.cuda.current_stream())
    for c in (a, b):
        out = torch.zeros(c.seqs, c.hkv * c.G, c.d, dtype=c.dt, device="cuda")
        c.run(ws=ws, out=out)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            c.run(ws=ws, out=out)
        graphs.append(g)
        outs.append(out)
        c.put()
    for _ in range(5):
        for g, out in zip(graphs, outs):
            out.zero_()
            g.replay()
    side.wait_stream(torch.cuda.current_stream())
    third, _ = a.run(stream=side)
    torch.cuda.synchronize()
    assert kv.kv_check_device_status(ws) == 0
    for c, out in zip((a, b), outs):
        c.check(out)
        c.check_pools()
    assert torch.equal(third, outs[0])


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_evicted_cache_into_8_bits(fmt):
    """kv_compact_streaming's rows, their keys turned to positions within the cache, stored as
    codes in head tables and attended to: against 64 bits at each step."""
    from kv_cache_eviction_gb300 import workloads as W
    layers, hq, hkv, d, n, page = 2, 8, 2, 128, 700, 32
    wl = W.Workload(name="evicted", batch=1, layers=layers, hq=hq, hkv=hkv, d=d, n=n, w=32, pool=7,
                    dtype="bf16", temp=(0.5, 8.0), seed=23)
    shape = kv.KvShape.from_workload(wl)
    inp = W.make_batch(wl, device="cuda")
    budget = torch.tensor([[[150, 333], [32, 408]]], dtype=torch.int32, device="cuda")
    cap = int(budget.sum())
    kept = torch.full((cap,), -7, dtype=torch.int32, device="cuda")
    cu = torch.empty(1, layers, hkv + 1, dtype=torch.int64, device="cuda")
    lens = torch.empty(1, layers, hkv, dtype=torch.int32, device="cuda")
    kf, vf = (torch.zeros(cap, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    kv.kv_compact_streaming(shape, inp["k"], inp["v"], 4, budget, 0, kept, cu, lens, kf, vf, cap, ws)
    assert kv.kv_check_device_status(ws) == 0

    # keys from their positions in the text to those in the cache
    rows = lens.flatten().tolist()
    new = np.concatenate([np.arange(m) for m in rows])
    back = kept.cpu().numpy() - new
    assert (back >= 0).all() and (back > 0).any()
    freq = kv.kv_rotary_inv_freq(d, 500000.0)[0]
    rot = kv.KvRotaryShape.of(0, 1, d, d, kv.KV_ROTARY_HALF, "bf16")
    was = kf.double().cpu().numpy()
    k3 = kf.view(cap, 1, d)
    kv.kv_rotary(rot, None, k3, torch.tensor(back, dtype=torch.int32, device="cuda"), freq.cuda(),
                 None, k3, back=True)
    t = back[:, None] * freq.numpy()
    a, b = was[:, :d // 2], was[:, d // 2:]
    turned = np.concatenate([a * np.cos(t) + b * np.sin(t), b * np.cos(t) - a * np.sin(t)], 1)
    assert (np.abs(kf.double().cpu().numpy() - turned) <=
            2.0 ** -8 * np.abs(turned) + 2.0 ** -20 * (np.abs(was).max() + 1)).all()

    # into the pages: a sequence of head tables for each layer
    cols, num = ceil_div(max(rows), page), sum(ceil_div(m, page) for m in rows) + 5
    ps = kv.KvPagedShape.of(layers, hq, hkv, d, hkv, page, cols, "bf16", num)
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    i64 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int64, device="cuda")
    ws = workspace(kv.KV_OP_QUANT_DECODE, ps)
    plens, ring = i32([0] * 4), i32(np.random.default_rng(1).permutation(num))
    state, table = i64([0, num]), i32(np.zeros((4, cols)))
    cu_add, slots = i64([0] * 5), i64([-1] * cap)
    kv.kv_page_map(ps, plens, lens.flatten(), ring, state, table, plens, state, cu_add, slots, ws)
    kp, vp = (torch.zeros(num, 1, page, d, dtype=torch.int8, device="cuda") for _ in range(2))
    if fmt == "e4m3":
        kp, vp = kp.view(torch.float8_e4m3fn), vp.view(torch.float8_e4m3fn)
    ks, vs = (torch.zeros(num, 1, page // 16, device="cuda") for _ in range(2))
    f = FORMATS[fmt]
    kv.kv_quant_write(ps, f, k3, vf.view(cap, 1, d), slots, cu_add[4:], kp, vp, ks, vs, ws)
    kr, vr = (torch.zeros(cap, 1, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kv.kv_quant_read(ps, f, kp, vp, ks, vs, slots, None, kr, vr, ws)
    q = torch.randn(layers, hq, d, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    out = torch.zeros_like(q)
    kv.quant_decode_attn(ps, f, q, None, None, None, None, kp, vp, ks, vs, table, plens, d ** -0.5,
                         out, ws)
    assert kv.kv_check_device_status(ws) == 0
    at = np.concatenate([[0], np.cumsum(rows)])
    for u in range(4):
        seg = slice(at[u], at[u + 1])
        k, v = (x[seg, 0].double().cpu().numpy() for x in (kr, vr))
        for x, y in ((k, kf), (v, vf)):     # a rounding of the block's code for every value
            orig = y[seg].double().cpu().numpy()
            for r0 in range(0, len(x), BLOCK):
                o = orig[r0:r0 + BLOCK]
                lim = (np.maximum(2.0 ** -4 * np.abs(o), 2.0 ** -10 * 2 * np.abs(o).max() / 448)
                       if fmt == "e4m3" else np.abs(o).max() / 127)
                assert (np.abs(x[r0:r0 + BLOCK] - o) <= lim).all()
        for g in range(hq // hkv):
            h = (u % hkv) * (hq // hkv) + g
            z = k @ q[u // hkv, h].double().cpu().numpy() * d ** -0.5
            p = np.exp(z - z.max())
            p /= p.sum()
            want, mag = p @ v, p @ np.abs(v)
            tol = (2.0 ** -8 * np.abs(want) + mag * 2.0 ** -23 * (
                4 * (d + 10) * (1 + np.abs(z).max() * 8) + 3 * len(z)))
            assert (np.abs(out[u // hkv, h].double().cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_steps_back_to_back(fmt):
    """Steps whose kernels start before the ones ahead of them have ended give what steps with waits
    between them give: rows and scales of the step before are read, from sectors that other CTAs
    wrote, and scales change at every step."""
    seqs, hq, hkv, d, page, cols, steps = 24, 16, 8, 64, 32, 9, 60
    num = seqs * cols
    shape = kv.KvPagedShape.of(seqs, hq, hkv, d, 1, page, cols, "bf16", num)
    g = torch.Generator().manual_seed(3)
    size = torch.exp2(torch.arange(steps) % 13 + torch.arange(steps) // 13).view(-1, 1, 1, 1)
    q, k, v = ((torch.randn(steps, seqs, h, d, generator=g) * f).bfloat16().cuda()
               for h, f in ((hq, 1.0), (hkv, size ** 0.25), (hkv, size)))
    start = torch.randint(0, 200, (seqs,), generator=g, dtype=torch.int32)
    got = []
    for wait in (True, False):
        i32 = lambda x: torch.as_tensor(x, dtype=torch.int32).cuda()
        lens, add, state = i32(torch.zeros(seqs)), start.cuda(), torch.tensor([0, num]).cuda()
        ring, table = i32(torch.arange(num)), i32(torch.zeros(seqs, cols))
        cu = torch.zeros(seqs + 1, dtype=torch.int64, device="cuda")
        codes = torch.zeros(2, num, hkv, page, d, dtype=torch.uint8, device="cuda")
        codes = codes.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.int8)
        sc = torch.full((2, num, hkv, page // 16), 2.0 ** -5, device="cuda")
        out = torch.zeros(steps, seqs, hq, d, dtype=torch.bfloat16, device="cuda")
        ws = workspace(kv.KV_OP_QUANT_DECODE, shape)
        slots = torch.full((int(start.sum()),), -1, dtype=torch.int64, device="cuda")
        kv.kv_page_map(shape, lens, add, ring, state, table, lens, state, cu, slots, ws)
        rows = torch.randn(2, len(slots), hkv, d, generator=torch.Generator().manual_seed(5))
        rows = rows.bfloat16().cuda()
        kv.kv_quant_write(shape, FORMATS[fmt], rows[0], rows[1], slots, None, codes[0], codes[1],
                          sc[0], sc[1], ws)
        add.fill_(1)
        torch.cuda.synchronize()
        for i in range(steps):
            for call in (lambda: kv.kv_page_map(shape, lens, add, ring, state, table, lens, state,
                                                cu, slots[:seqs], ws),
                         lambda: kv.quant_decode_attn(shape, FORMATS[fmt], q[i], k[i], v[i], cu,
                                                      slots[:seqs], codes[0], codes[1], sc[0],
                                                      sc[1], table, lens, 0.1, out[i], ws),
                         lambda: kv.quant_decode_attn(shape, FORMATS[fmt], q[i], None, None, None,
                                                      None, codes[0], codes[1], sc[0], sc[1],
                                                      table, lens, 0.1, out[i], ws)):
                call()
                if wait:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert kv.kv_check_device_status(ws) == 0
        got.append([out, codes.view(torch.uint8), sc, table, lens])
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert bool(torch.isfinite(got[0][0]).all())


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_new_row_beside_a_scale_that_is_no_number(fmt, dtype, bad):
    """A new row behind rows of a block whose scale was never set is stored with a scale of its own,
    as kv_quant_write stores it; this step and the next attend over the same numbers."""
    lens = [38, 17, 5, 64]
    a, b = (QuantCache(4, 2, 2, 64, 1, 32, lens, dtype, fmt, 6) for _ in range(2))
    for c in (a, b):
        for name in ("k", "v"):                     # rows 32..36 of the first table
            c.scale_dev[name][c.table_host[0, 1], :, 0] = bad
    x, ws = a.run()
    rows = lambda t: t.reshape(-1, 2, 64).contiguous().cuda()
    kv.kv_quant_write(b.shape, FORMATS[fmt], rows(b.k_new), rows(b.v_new), b.slots, None, *b.args(),
                      ws)
    for name in ("k", "v"):
        assert torch.equal(a.pool[name][0].view(torch.uint8), b.pool[name][0].view(torch.uint8))
        assert torch.equal(a.scale_dev[name].view(torch.int32), b.scale_dev[name].view(torch.int32))
        assert bool(torch.isfinite(a.scale_dev[name][a.table_host[0, 1], :, 0]).all())
    again = a.run(with_new=False, ws=ws)[0]
    assert torch.equal(torch.isnan(x), torch.isnan(again))
    assert torch.equal(x.nan_to_num(nan=7.0), again.nan_to_num(nan=7.0))
    assert bool(torch.isfinite(x[1:]).all())
    # A number held is NaN now where the scale was one, or, that being infinite, where its code was
    # zero (other codes are the largest then, a finite number); in int8 nowhere.  A NaN in K reaches
    # every output of its head, one in V those of its column.
    page = a.table_host[0, 1]
    nan = {n: np.full((2, 5, 64), fmt == "e4m3") & (np.isnan(bad) | (b.num[n][page, :, :5] == 0))
           for n in ("k", "v")}
    want = nan["k"].any((1, 2))[:, None] | nan["v"].any(1)
    assert np.array_equal(torch.isnan(x[0]).cpu().numpy().reshape(2, 2, 64),
                          want[:, None].repeat(2, 1))
    assert kv.kv_check_device_status(ws) == 0


@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan_in_the_only_row_held(where, dtype):
    """A table of one row that is no new one, with a NaN in it: the outputs that it reaches, and nowhere
    else."""
    c = QuantCache(3, 2, 2, 64, 1, 16, [33, 1, 70], dtype, "e4m3", 11, new=[1, 0, 1])
    c.pool[where][1].view(torch.uint8)[c.table_host[1, 0], 0, 0, 7] = 127
    out, ws = c.run()
    torch.cuda.synchronize()
    assert kv.kv_check_device_status(ws) == 0
    nan = torch.isnan(out.cpu().float())
    want = torch.zeros_like(nan)
    if where == "v":
        want[1, :2, 7] = True
    else:
        want[1, :2] = True
    assert torch.equal(nan, want)
