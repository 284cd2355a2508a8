"""paged_decode_attn and kv_page_map on the GPU at the edges of what their arguments may hold."""
import pytest
import torch

import kv_cache_eviction_gb300 as kv
from tests.paged import Cache

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
