"""kv_rotary on the GPU against its formula in 64 bits (angles in the host's long double), as a
linear map with its gradient, and with the calls around it."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import kv_cache_eviction_gb300 as kv

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
LAYOUT = {"half": kv.KV_ROTARY_HALF, "interleaved": kv.KV_ROTARY_INTERLEAVED}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kv_cache_eviction_gb300 import _build
    _build.build()
    kv.lib()


def angles(pos, freq):
    """pos * freq modulo a turn, [rows][pairs] float64: the product of a 31-bit and a 53-bit
    number is exact as two 64-bit floats, and so is the remainder of each by 2 pi to 1e-15."""
    two_pi = np.longdouble(2) * np.longdouble("3.14159265358979323846264338327950288")
    hi = np.float32(freq).astype(np.float64)                   # 24 bits: times 31 exact
    lo = freq - hi
    p = np.asarray(pos, np.float64)[:, None]
    t = np.remainder((p * hi).astype(np.longdouble), two_pi) + (p * lo).astype(np.longdouble)
    return np.remainder(t, two_pi).astype(np.float64)


def expected(x, pos, freq, rot, layout, m, back):
    """(out, bound) [rows][heads][d] in 64 bits.  The bound: a sine or cosine is off by the angle's
    error (2^-32 turns of the product's cut and 2^-27 of the float's rounding: below 2^-24 in radians
    together), by two units of its own (2^-23) and by the rounding of its product with m (2^-24); the
    two products and their sum by 2^-24 each, all below 2^-21 (|a| + |b|) m; then the output's
    rounding."""
    y = x.double().numpy()
    t = angles(np.maximum(pos, 0), freq)[:, None]
    c, s = m * np.cos(t), m * np.sin(t) * (-1 if back else 1)
    half = rot // 2
    a, b = (y[..., :half], y[..., half:rot]) if layout == "half" else (y[..., 0:rot:2],
                                                                       y[..., 1:rot:2])
    u, w = a * c - b * s, a * s + b * c
    mag = (np.abs(a) + np.abs(b)) * abs(m) * 2.0 ** -21
    out, tol = y.copy(), np.zeros_like(y)
    if layout == "half":
        out[..., :half], out[..., half:rot] = u, w
        tol[..., :half] = tol[..., half:rot] = mag
    else:
        out[..., 0:rot:2], out[..., 1:rot:2] = u, w
        tol[..., 0:rot:2] = tol[..., 1:rot:2] = mag
    eps = torch.finfo(x.dtype).eps / 2
    tol[..., :rot] += eps * (np.abs(out[..., :rot]) + tol[..., :rot]) + 1e-38
    return out, tol


def positions(rows, seed):
    rng = np.random.default_rng(seed)
    pos = rng.integers(0, 200000, rows)
    pos[rng.random(rows) < 0.2] = -1
    some = [0, 1, 2**31 - 1, 131071, 2**30 + 1, -2**31, 1 << 24]
    pos[:min(rows, len(some))] = some[:rows]
    return pos


def dev(x, dtype):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,hq,hkv,d,rot,m,where", [
    (1, 32, 8, 128, 128, 1.0, "fused"), (7, 6, 2, 80, 24, 1.2, "apart"),
    (300, 5, 1, 72, 72, 1.0, "in place"), (64, 0, 8, 96, 32, 1.0, "apart"),
    (65, 3, 0, 64, 8, 0.5, "in place"), (33, 1, 1, 8, 8, 1.0, "apart"),
    (500, 2, 2, 256, 256, 1.0, "fused"), (9, 33, 7, 128, 64, -1.0, "in place"),
    (2000, 32, 8, 128, 128, 1.0, "in place"), (40, 4, 4, 40, 40, 1.0, "fused"),
    (3, 7, 3, 248, 152, 1.0, "apart")])
def test_rotary(layout, dtype, rows, hq, hkv, d, rot, m, where):
    g = torch.Generator().manual_seed(rows + d)
    dt = DT[dtype]
    x = [torch.randn(rows, h, d, generator=g).to(dt) for h in (hq, hkv)]
    pos = positions(rows, rows)
    freq = kv.kv_rotary_inv_freq(rot, 10000.0)[0]
    s = kv.KvRotaryShape.of(hq, hkv, d, rot, LAYOUT[layout], dtype, m)
    for back in (False, True):
        if where == "apart":
            ins = [t.cuda() for t in x]
            outs = [torch.full_like(t, 9.0) for t in ins]
            old = [torch.full_like(t, 9.0) for t in x]
        else:
            wide = torch.full((rows, hq + 2 * hkv + 1, d), 5.0, dtype=dt, device="cuda")
            ins = [wide[:, :hq], wide[:, hq:hq + hkv]]
            for a, b in zip(ins, x):
                a.copy_(b)
            if where == "in place":
                outs, old = ins, x
            else:
                outs = [torch.full((rows, h + 2, d), 9.0, dtype=dt, device="cuda")[:, 1:1 + h]
                        for h in (hq, hkv)]
                old = [torch.full_like(t, 9.0) for t in x]
        n = min(rows, max(1, rows - 3))
        arg = [t if t.shape[1] else None for t in (*ins, *outs)]
        kv.kv_rotary(s, arg[0], arg[1], dev(pos, torch.int32), freq.cuda(), arg[2], arg[3],
                     dev([n], torch.int64), back)
        torch.cuda.synchronize()
        there = (pos >= 0) & (np.arange(rows) < n)
        for t, out, was in zip(x, outs, old):
            if t.shape[1] == 0:
                continue
            want, tol = expected(t, pos, freq.numpy(), rot, layout, float(np.float32(m)), back)
            got = out.cpu().double().numpy()
            off = np.abs(got - want)[there] > tol[there]
            assert not off.any(), (int(off.sum()), np.argwhere(off)[:3])
            assert np.array_equal(got[~there], was.double().numpy()[~there])
            assert np.array_equal(got[there][..., rot:], t.double().numpy()[there][..., rot:])
        if where != "apart":
            assert bool((wide[:, hq + hkv:] == 5.0).all())


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradient(layout):
    """`back` is the gradient: against the formula's own by autograd in 64 bits, and against
    differences of the call (it is linear, so a difference is exact but for roundings)."""
    rows, h, d, rot, m = 20, 3, 48, 32, 1.25
    g = torch.Generator().manual_seed(4)
    pos, freq = np.arange(rows) * 977, kv.kv_rotary_inv_freq(rot)[0]
    s = kv.KvRotaryShape.of(h, 0, d, rot, LAYOUT[layout], "f32", m)
    x, gy = (torch.randn(rows, h, d, generator=g) for _ in range(2))

    def call(t, back=False):
        out = torch.zeros_like(t, device="cuda")
        kv.kv_rotary(s, t.cuda(), None, dev(pos, torch.int32), freq.cuda(), out, None, back=back)
        return out.cpu()

    grad = call(gy, back=True)
    y = x.double().requires_grad_()
    t = torch.tensor(pos).double()[:, None, None] * freq
    half = rot // 2
    a, b = (y[..., :half], y[..., half:rot]) if layout == "half" else (y[..., 0:rot:2],
                                                                       y[..., 1:rot:2])
    u, w = m * (a * t.cos() - b * t.sin()), m * (a * t.sin() + b * t.cos())
    out = torch.cat([u, w], 2) if layout == "half" else torch.stack([u, w], 3).flatten(2)
    out = torch.cat([out, y[..., rot:]], 2)
    (out * gy.double()).sum().backward()
    # angles here are off by 977 * 20 * 2^-53; the rest is the bound of the call
    assert float((grad.double() - y.grad).abs().max()) < 2.0 ** -20 * 2 * float(gy.abs().max()) * m
    for i, j, k in ((0, 0, 0), (7, 2, 5), (19, 1, 31), (3, 0, 40)):
        e = torch.zeros_like(x)
        e[i, j, k] = 1.0
        diff = ((call(x + e) - call(x)).double() * gy.double()).sum()
        # two outputs of the pair, each with two calls' errors of 2^-20 of the values there
        lim = 2.0 ** -19 * 2 * m * 2 * float((x[i, j].abs() + 1).max() * gy[i, j].abs().max())
        assert abs(float(diff) - float(grad[i, j, k])) < lim


def test_turned_to_and_back():
    """Keys of a compacted cache moved to new positions: kept_idx - new position, back."""
    n, h, d = 400, 2, 128
    rng = np.random.default_rng(6)
    kept = np.sort(rng.choice(100000, n, replace=False))
    new = np.arange(n)
    x = torch.randn(n, h, d, generator=torch.Generator().manual_seed(8))
    freq = kv.kv_rotary_inv_freq(d, 500000.0)[0].cuda()
    s = kv.KvRotaryShape.of(0, h, d, d, kv.KV_ROTARY_HALF, "f32")
    a, b, c = (torch.zeros_like(x, device="cuda") for _ in range(3))
    kv.kv_rotary(s, None, x.cuda(), dev(kept, torch.int32), freq, None, a)
    kv.kv_rotary(s, None, a, dev(kept - new, torch.int32), freq, None, a, back=True)
    kv.kv_rotary(s, None, x.cuda(), dev(new, torch.int32), freq, None, b)
    kv.kv_rotary(s, None, b, dev(new, torch.int32), freq, None, c, back=True)
    mag = 2 * float(x.abs().max())
    assert float((a - b).abs().max()) < 3 * 2.0 ** -20 * mag
    assert float((c.cpu() - x).abs().max()) < 2 * 2.0 ** -20 * mag


def test_many_rows_and_captured():
    """More rows than the grid has warps, in a captured graph replayed with other positions."""
    rows, h, d = 30000, 2, 64
    x = torch.randn(rows, h, d, generator=torch.Generator().manual_seed(1)).bfloat16()
    freq = kv.kv_rotary_inv_freq(d)[0]
    s = kv.KvRotaryShape.of(h, 0, d, d, kv.KV_ROTARY_HALF, "bf16")
    xd, fd = x.cuda(), freq.cuda()
    out = torch.zeros_like(xd)
    pos = dev(np.zeros(rows), torch.int32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kv.kv_rotary(s, xd, None, pos, fd, out, None, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, xd)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        kv.kv_rotary(s, xd, None, pos, fd, out, None)
    for k in range(3):
        p = (np.arange(rows) * 7919 * (k + 1)) % 1000003
        pos.copy_(dev(p, torch.int32))
        g.replay()
        torch.cuda.synchronize()
        want, tol = expected(x, p, freq.numpy(), d, "half", 1.0, False)
        assert (np.abs(out.cpu().double().numpy() - want) <= tol).all()


def test_rows_past_32_bits():
    """Rows whose elements lie past 2^31 and bytes past 2^32."""
    rows, h, d = 1 << 19, 40, 128
    x = torch.zeros(rows, h, d, dtype=torch.bfloat16, device="cuda")
    assert x.numel() > 1 << 31
    x[-3:] = torch.randn(3, h, d, device="cuda")
    keep = x[-3:].cpu()
    freq = kv.kv_rotary_inv_freq(d)[0]
    s = kv.KvRotaryShape.of(h, 0, d, d, kv.KV_ROTARY_HALF, "bf16")
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    kv.kv_rotary(s, x, None, pos, freq.cuda(), x, None)
    p = np.arange(rows - 3, rows)
    want, tol = expected(keep, p, freq.numpy(), d, "half", 1.0, False)
    assert (np.abs(x[-3:].cpu().double().numpy() - want) <= tol).all()
    assert bool((x[:-3] == 0).all())   # (of either sign)


# 2 pi to 10^-59
TWO_PI = Fraction(2 * 314159265358979323846264338327950288419716939937510582097494, 10 ** 59)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("back", [False, True])
def test_any_frequency_below_the_limit(layout, back):
    """Whole turns drop off whatever the frequency's size, at the farthest positions too: angles in
    fractions of whole numbers, the sines in 64 bits, and the bound of expected()."""
    freq = [1.5, 1000.5, 2.0 ** 20 + 0.5, 2.0 ** 33 + 1, 2.0 ** 45 + 0.125, 2.0 ** 52 - 1,
            -7.25, -2.0 ** 40 - 3, 3.0e-5, 2.0 ** -70, 0.0, 977.0 / 1024] + [2.5] * 4
    rot, d, pos = 2 * len(freq), 40, [0, 1, 131071, 2 ** 24 + 1, 2 ** 30 + 7, 2 ** 31 - 1]
    x = torch.randn(len(pos), 3, d, generator=torch.Generator().manual_seed(3))
    s = kv.KvRotaryShape.of(3, 0, d, rot, LAYOUT[layout], "f32")
    out = torch.zeros_like(x, device="cuda")
    kv.kv_rotary(s, x.cuda(), None, dev(pos, torch.int32), dev(freq, torch.float64), out, None,
                 back=back)
    t = np.array([[float(p * Fraction(f) % TWO_PI) for f in freq] for p in pos])[:, None]
    c, n = np.cos(t), np.sin(t) * (-1 if back else 1)
    y, half = x.double().numpy(), rot // 2
    a, b = (y[..., :half], y[..., half:rot]) if layout == "half" else (y[..., 0:rot:2],
                                                                       y[..., 1:rot:2])
    got = out.cpu().double().numpy()
    u, w = (got[..., :half], got[..., half:rot]) if layout == "half" else (got[..., 0:rot:2],
                                                                           got[..., 1:rot:2])
    # (the output's rounding, 2^-24 of it, beside the 2^-21 of the rest)
    tol = (np.abs(a) + np.abs(b)) * (2.0 ** -21 + 2.0 ** -24)
    assert (np.abs(u - (a * c - b * n)) <= tol).all()
    assert (np.abs(w - (a * n + b * c)) <= tol).all()
