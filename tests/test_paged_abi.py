"""The paged cache's calls without a GPU: workspace sizes, and refusals on the host before
anything is enqueued; and the page map's reference against its invariants."""
import ctypes

import numpy as np
import pytest

import kv_cache_eviction_gb300 as kv
from kv_cache_eviction_gb300 import _build
from tests.paged import ERR_PAGES, ERR_SLOTS, ERR_TABLE, ceil_div, page_map_ref


@pytest.fixture(scope="module")
def L():
    _build.build()
    return kv.lib()


def shape(**kw):
    base = dict(seqs=4, hq=32, hkv=8, d=128, tables=1, page=16, max_pages=64, dtype="bf16",
                num_pages=1000)
    base.update(kw)
    return kv.KvPagedShape.of(**base)


OPS = (kv.KV_OP_PAGE_MAP, kv.KV_OP_PAGED_WRITE, kv.KV_OP_PAGED_DECODE)
P = ctypes.c_void_p(0x1000)
BIG = 1 << 40


def call_map(L, s, lens=P, add=ctypes.c_void_p(0x2000), ring=P, state=P, cap=100, table=P,
             lens_out=P, state_out=P, cu=P, slots=P, ws=P, n=BIG):
    return L.kv_page_map(ctypes.byref(s) if s else None, lens, add, ring, state, cap, table,
                         lens_out, state_out, cu, slots, ws, n, None)


def call_write(L, s, k=P, v=P, stride=0, slots=P, rows=10, n_rows=None, kp=P, vp=P, ws=P, n=BIG):
    return L.kv_paged_write(ctypes.byref(s) if s else None, k, v, stride, slots, rows, n_rows, kp,
                            vp, ws, n, None)


def call_decode(L, s, q=P, kn=P, vn=P, cu=P, slots=P, cap=10, kp=P, vp=P, table=P, lens=P,
                scale=0.1, out=P, ws=P, n=BIG):
    return L.paged_decode_attn(ctypes.byref(s) if s else None, q, kn, vn, cu, slots, cap, kp, vp,
                               table, lens, scale, out, ws, n, None)


@pytest.mark.parametrize("bad", [
    dict(seqs=-1), dict(hq=30), dict(hq=0), dict(d=100), dict(d=0), dict(tables=2), dict(page=0),
    dict(max_pages=0), dict(num_pages=0), dict(dtype=7), dict(page_stride=8 * 16 * 128 - 8),
    dict(page_stride=8 * 16 * 128 + 4), dict(page_stride=-8)])
def test_invalid_shapes(L, bad):
    s = shape(**bad)
    for op in OPS:
        assert kv.kv_paged_workspace_size(op, s) == 0
    assert call_map(L, s) == kv.KV_ERR_INVALID_ARG
    assert call_write(L, s) == kv.KV_ERR_INVALID_ARG
    assert call_decode(L, s) == kv.KV_ERR_INVALID_ARG


@pytest.mark.parametrize("far", [
    dict(hq=128), dict(d=136), dict(hq=512, hkv=512), dict(page=4), dict(page=24),
    dict(page=512), dict(max_pages=1 << 28), dict(num_pages=1 << 31), dict(page_stride=1 << 40),
    dict(seqs=1 << 29)])
def test_unsupported_shapes(L, far):
    s = shape(**far)
    assert call_map(L, s) == kv.KV_ERR_UNSUPPORTED
    assert call_write(L, s) == kv.KV_ERR_UNSUPPORTED
    assert call_decode(L, s) == kv.KV_ERR_UNSUPPORTED


def test_decode_counts_its_tiles_in_31_bits(L):
    s = shape(seqs=1 << 11, max_pages=(1 << 16) - 1, page=16)     # 2^14 heads of 2^20 - 16 rows
    n = kv.kv_paged_workspace_size(kv.KV_OP_PAGED_DECODE, s)
    assert call_decode(L, s, n=n - 1) == kv.KV_ERR_WORKSPACE
    assert call_decode(L, shape(seqs=1 << 11, max_pages=1 << 16)) == kv.KV_ERR_UNSUPPORTED


def test_decode_table_limit(L):
    s = shape(seqs=kv.KV_PAGED_DECODE_MAX_TABLES, max_pages=1, page=8, hkv=1, hq=1)
    n = kv.kv_paged_workspace_size(kv.KV_OP_PAGED_DECODE, s)
    assert call_decode(L, s, n=n - 1) == kv.KV_ERR_WORKSPACE
    s = shape(seqs=kv.KV_PAGED_DECODE_MAX_TABLES + 1, max_pages=1, page=8, hkv=1, hq=1)
    assert call_decode(L, s) == kv.KV_ERR_UNSUPPORTED


def test_workspace_sizes(L):
    for op in OPS:
        n = kv.kv_paged_workspace_size(op, shape())
        assert n >= 256
    assert kv.kv_paged_workspace_size(0, shape()) == 0      # an op of the flat cache
    assert kv.kv_paged_workspace_size(9, shape()) == 0
    for op, call in zip(OPS, (call_map, call_write, call_decode)):
        n = kv.kv_paged_workspace_size(op, shape())
        assert call(L, shape(), n=n - 1) == kv.KV_ERR_WORKSPACE


def test_arguments(L):
    s = shape()
    odd4, odd2 = ctypes.c_void_p(0x1004), ctypes.c_void_p(0x1002)
    inv = kv.KV_ERR_INVALID_ARG
    assert call_map(L, None) == call_write(L, None) == call_decode(L, None) == inv
    for arg in ("lens", "add", "ring", "state", "table", "lens_out", "state_out", "cu", "slots",
                "ws"):
        assert call_map(L, s, **{arg: None}) == inv
        assert call_map(L, s, **{arg: odd2}) == inv
    for arg in ("state", "state_out", "cu", "slots"):
        assert call_map(L, s, **{arg: odd4}) == inv
    assert call_map(L, s, cap=-1) == inv
    assert call_map(L, s, cap=(1 << 31) - 1) == inv
    assert call_map(L, s, add=P) == inv                      # lens_out over add
    # lens_out or free_out over a part of lens or free_state
    assert call_map(L, s, lens_out=ctypes.c_void_p(0x1008)) == inv
    assert call_map(L, s, state_out=ctypes.c_void_p(0x0ff8)) == inv
    assert call_map(L, shape(seqs=kv.KV_PAGE_MAP_MAX_TABLES + 1)) == kv.KV_ERR_UNSUPPORTED
    for arg in ("k", "v", "slots", "kp", "vp", "ws"):
        assert call_write(L, s, **{arg: None}) == inv
        assert call_write(L, s, **{arg: odd4}) == inv
    assert call_write(L, s, n_rows=odd4) == inv
    assert call_write(L, s, rows=-1) == inv
    for stride in (-8, 8 * 128 - 8, 8 * 128 + 4, 1 << 33):
        assert call_write(L, s, stride=stride) == inv
    for arg in ("q", "kp", "vp", "table", "lens", "out", "ws"):
        assert call_decode(L, s, **{arg: None}) == inv
        assert call_decode(L, s, **{arg: odd2}) == inv
    for arg in ("q", "kp", "vp", "kn", "vn", "out", "cu", "slots"):
        assert call_decode(L, s, **{arg: odd4}) == inv
    assert call_decode(L, s, kn=None) == inv
    assert call_decode(L, s, vn=None) == inv
    assert call_decode(L, s, cu=None) == inv
    assert call_decode(L, s, slots=None) == inv
    assert call_decode(L, s, cap=-1) == inv
    assert call_decode(L, s, scale=float("inf")) == inv


def test_empty_calls(L):
    s = shape(seqs=0)
    assert call_map(L, s, None, None, None, None, 0, None, None, None, None, None) == kv.KV_OK
    assert call_decode(L, s, None, None, None, None, None, 0, None, None, None, None, 0.1,
                       None) == kv.KV_OK
    assert call_write(L, shape(), None, None, 0, None, 0, None, None, None) == kv.KV_OK


def test_binding_refuses_host_tensors(L):
    import torch
    s = shape(seqs=1)
    i = torch.zeros(2000, dtype=torch.int32)
    j = torch.zeros(2000, dtype=torch.int64)
    t = torch.zeros(1000, 8, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        kv.kv_page_map(s, i, i, i, j, i, i, j, j, j, i)
    with pytest.raises(ValueError):
        kv.kv_paged_write(s, t[:, 0, 0], t[:, 0, 0], j, None, t, t, i)
    with pytest.raises(ValueError):
        kv.paged_decode_attn(s, t[0, 0], None, None, None, None, t, t, i, i, 0.1, t[0, 0], i)


def test_binding_refuses_rows_that_overlap():
    """Rows a stride of 0 apart (expanded ones) are no dense rows, which 0 means to the library."""
    import torch
    row = torch.zeros(1, 2, 64)
    view = lambda t: kv._rows_view(t, torch.float32, 128, -1, "k")[1:]
    assert view(row) == (1, 128)
    assert view(row.expand(1, 2, 64)) == (1, 128)
    assert view(torch.zeros(5, 6, 64)[:, 2:4]) == (5, 6 * 64)
    assert view(torch.zeros(0, 2, 64)) == (0, 128)
    for t in (row.expand(5, 2, 64), torch.zeros(400).as_strided((3, 2, 64), (64, 64, 1)),
              torch.zeros(5, 1, 64).expand(5, 2, 64)):
        with pytest.raises(ValueError):
            view(t)


def test_reference_map_keeps_every_page():
    """Random steps of the reference: every page is either free or in exactly one table, and
    a table's slots are its rows' places."""
    rng = np.random.default_rng(5)
    page, num, U, cols = 8, 60, 7, 16
    lens = np.zeros(U, int)
    ring, state = np.arange(num), np.array([0, num])
    table = np.full((U, cols), -9)
    seen = set()
    for step in range(200):
        add = rng.integers(-40, 60, U)
        slots = np.full(500, -7)
        ring, state, table, new, cu, slots, codes = page_map_ref(
            lens, add, ring, state, 150, table, slots, page, num)
        seen |= codes
        free = [ring[i % num] for i in range(state[0], state[1])]
        held = [table[u, c] for u in range(U) for c in range(ceil_div(new[u], page))]
        assert sorted(free + held) == list(range(num))
        for u in range(U):
            for i in range(cu[u], min(cu[u + 1], 150)):
                r = lens[u] + i - cu[u]
                if new[u] > lens[u]:
                    assert slots[i] == table[u, r // page] * page + r % page
                else:
                    assert slots[i] == -1
        assert (slots[min(cu[-1], 150):] == -7).all()
        lens = new
    assert seen == {ERR_PAGES, ERR_TABLE, ERR_SLOTS}


def test_write_of_no_sequences(L):
    """With seqs = 0 the row write does nothing either, whatever the number of rows."""
    assert call_write(L, shape(seqs=0)) == kv.KV_OK
    assert call_write(L, shape(seqs=0), None, None, 0, None, 10, None, None, None) == kv.KV_OK
    assert call_write(L, shape(seqs=0), rows=-1) == kv.KV_ERR_INVALID_ARG
    assert call_write(L, shape(seqs=0), ws=None) == kv.KV_ERR_INVALID_ARG


def test_scales_past_the_range_of_their_product_with_log2_e(L):
    """scale * log2(e) is a float32 number too: 2^127 and more is refused, either sign."""
    s = shape()
    n = kv.kv_paged_workspace_size(kv.KV_OP_PAGED_DECODE, s)
    for scale in (2.0 ** 127, -2.0 ** 127, 3e38, -3.4e38, float("nan"), -float("inf")):
        assert call_decode(L, s, scale=scale) == kv.KV_ERR_INVALID_ARG
    for scale in (1.7e38, -1.7e38, 1e-45, 0.0):
        assert call_decode(L, s, scale=scale, n=n - 1) == kv.KV_ERR_WORKSPACE
