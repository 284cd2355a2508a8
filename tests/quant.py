"""Test helpers of the cache in 8 bits: its codes and block scales by their definition, in 64 bits."""
from __future__ import annotations

import numpy as np
import torch

import kv_cache_eviction_gb300 as kv

BLOCK, LEAST = 16, -96
FORMATS = {"e4m3": kv.KV_E4M3, "int8": kv.KV_INT8}
MOST = {"e4m3": 448.0, "int8": 127.0}


def e4m3_numbers():
    """The 256 numbers of e4m3: sign, four bits of exponent (bias 7), three of the fraction."""
    out = np.zeros(256)
    for b in range(256):
        e, f = b >> 3 & 15, b & 7
        x = f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        if b & 127 == 127:
            x = np.nan
        out[b] = -x if b >> 7 else x
    return out


E4M3 = e4m3_numbers()


def numbers(codes, fmt):
    """The numbers of a tensor of codes, as float64."""
    c = codes.cpu()
    if fmt == "int8":
        return c.view(torch.int8).numpy().astype(np.float64)
    return E4M3[c.view(torch.uint8).numpy()]


def nearest(x, fmt):
    """x to the nearest number of the format, halves to the even code; saturated."""
    x = np.asarray(x, np.float64)
    if fmt == "int8":
        return np.clip(np.rint(np.nan_to_num(x, nan=0.0, posinf=1e9, neginf=-1e9)), -127, 127)
    y = np.clip(x, -448, 448)
    step = 2.0 ** (np.maximum(np.frexp(np.nan_to_num(y))[1] - 1, -6) - 3)
    return np.clip(np.rint(y / step) * step, -448, 448)


def scale_for(x, fmt):
    """The scale of a block of values x, by trying every exponent."""
    x = np.abs(np.asarray(x, np.float64))
    x = x[np.isfinite(x)]
    top = x.max() if x.size else 0.0
    t = LEAST
    while top > MOST[fmt] * 2.0 ** t:
        t += 1
    return 2.0 ** t


def put(num, scale, rows, slots, fmt):
    """Rows [n][heads][d] (float64) at their slots, one run of a block after the other; num
    [pages][heads][page][d] and scale [pages][heads][page / 16] float64 are changed in place."""
    page, total = num.shape[2], num.shape[0] * num.shape[2]
    i = 0
    while i < len(slots):
        s = int(slots[i])
        if not 0 <= s < total:
            i += 1
            continue
        n = 1
        while i + n < len(slots) and int(slots[i + n]) == s + n and (s + n) % BLOCK:
            n += 1
        p, r = divmod(s, page)
        b, first = r // BLOCK, r % BLOCK
        for h in range(num.shape[1]):
            now = scale_for(rows[i:i + n, h], fmt)
            if first:
                old = scale[p, h, b]
                now = max(now, old)
                held = slice(b * BLOCK, b * BLOCK + first)
                num[p, h, held] = nearest(num[p, h, held] * (old / now), fmt)
            scale[p, h, b] = now
            num[p, h, r:r + n] = nearest(rows[i:i + n, h] / now, fmt)
        i += n


def random_codes(shape, fmt, gen):
    """Codes of any finite number."""
    c = torch.randint(0, 256, shape, generator=gen, dtype=torch.uint8)
    if fmt == "int8":
        c[c == 128] = 0
        return c.view(torch.int8)
    c[(c & 127) == 127] = 0
    return c.view(torch.float8_e4m3fn)


class Pool:
    """A pool of pages of codes and scales on the host and on the device, pages `extra` bytes
    further apart than dense."""

    def __init__(self, num, heads, page, d, fmt, seed, extra=0, scales=None):
        g = torch.Generator().manual_seed(seed)
        self.fmt, self.page_stride = fmt, (heads * page * d + extra if extra else 0)
        apart, inner = heads * page * d + extra, heads * page * d
        self.size, self.strides = (num, heads, page, d), (apart, page * d, d, 1)
        self.flat, self.host, self.num, self.scale, self.dev, self.scale_dev = {}, {}, {}, {}, {}, {}
        for name in ("k", "v"):
            flat = random_codes((num * apart + 64,), fmt, g)
            self.host[name] = flat
            self.flat[name] = flat.cuda()
            self.dev[name] = self.flat[name][:num * apart].as_strided(self.size, self.strides)
            t = torch.randint(-12, 6, (num, heads, page // BLOCK), generator=g).double()
            s = torch.exp2(t) if scales is None else torch.full_like(t, scales)
            self.scale[name] = s.numpy().copy()
            self.scale_dev[name] = s.float().cuda()
            self.num[name] = numbers(self._strided(flat), fmt)

    def _strided(self, flat):
        n = self.size[0] * self.strides[0]
        return flat.view(torch.uint8)[:n].as_strided(self.size, self.strides).contiguous().view(
            flat.dtype)

    def args(self):
        return (self.dev["k"], self.dev["v"], self.scale_dev["k"], self.scale_dev["v"])

    def put(self, k, v, slots):
        for name, x in (("k", k), ("v", v)):
            put(self.num[name], self.scale[name], x, slots, self.fmt)

    def values(self, name):
        return self.num[name] * np.repeat(self.scale[name], BLOCK, 2)[..., None]

    def check(self):
        """The device's codes and scales are the host's, and nothing between the pages changed."""
        for name in ("k", "v"):
            got = numbers(self._strided(self.flat[name].cpu()), self.fmt)
            want = self.num[name]
            same = (got == want) | (np.isnan(got) & np.isnan(want))
            assert same.all(), (name, int((~same).sum()), np.argwhere(~same)[:4])
            assert np.array_equal(self.scale_dev[name].cpu().double().numpy(), self.scale[name],
                                  equal_nan=True), name
            keep = torch.ones(self.host[name].numel(), dtype=torch.bool)
            keep[:self.size[0] * self.strides[0]].as_strided(self.size, self.strides).fill_(False)
            a, b = self.flat[name].cpu().view(torch.uint8), self.host[name].view(torch.uint8)
            assert torch.equal(a[keep], b[keep]), name
