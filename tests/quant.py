"""Test helpers of the cache in 8 bits: codes and block scales by their definition, in 64 bits."""
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
        self.flat, self.host, self.num = {}, {}, {}
        self.scale, self.dev, self.scale_dev = {}, {}, {}
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


class QuantCache:
    """A paged cache in 8 bits with the given rows per table, as tests.paged.Cache is one of rows:
    pages dealt out in a random order; codes that are NaN (e4m3) in every row that no table holds,
    and NaN for the scale of every block that holds none.  The last row of the tables in `new`
    comes as k_new / v_new."""

    def __init__(self, seqs, hkv, G, d, tables, page, lens, dtype, fmt, seed, new=None, spare=3,
                 extra=0, first_page=0, temp=4.0, spread=1.0):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.seqs, self.hkv, self.G, self.d = seqs, hkv, G, d
        self.tables, self.page, self.dtype, self.fmt = tables, page, dtype, fmt
        self.dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        U, hp, nb = seqs * tables, hkv // tables, page // BLOCK
        self.hp = hp
        lens = [int(x) for x in lens]
        assert len(lens) == U
        new = [n > 0 for n in lens] if new is None else [bool(x) and n > 0
                                                         for x, n in zip(new, lens)]
        used = [-(-n // page) for n in lens]
        self.max_pages = max(1, max(used))
        num = sum(used) + spare
        order = rng.permutation(num) + first_page
        self.num_pages = num + first_page
        table = rng.integers(0, self.num_pages, (U, self.max_pages))
        at = 0
        for u, n in enumerate(used):
            table[u, :n] = order[at:at + n]
            at += n
        inner = hp * page * d
        self.apart = inner + extra
        self.shape = kv.KvPagedShape.of(seqs, hkv * G, hkv, d, tables, page, self.max_pages, dtype,
                                        self.num_pages, self.apart if extra else 0)
        tau = np.exp(rng.random((seqs, hkv * G, 1)) * np.log(8.0)) * temp / 8
        self.q = (torch.randn(seqs, hkv * G, d, generator=g) * torch.tensor(tau)).to(self.dt)
        fresh = {n: (torch.randn(seqs, hkv, d, generator=g) * torch.exp(
            0.7 * torch.randn(seqs, hkv, 1, generator=g))).to(self.dt) for n in ("k", "v")}
        self.k_new, self.v_new = fresh["k"], fresh["v"]
        self.lens, self.new, self.table_host = lens, new, table
        # the places of the rows held before the call: page, row
        self.num, self.scale, codes = {}, {}, {}
        for name in ("k", "v"):
            x = rng.normal(size=(self.num_pages, hp, nb, BLOCK, d)) * np.exp(
                spread * rng.normal(size=(self.num_pages, hp, nb, 1, 1)))
            top = np.abs(x).max((3, 4))
            s = np.exp2(np.ceil(np.log2(top / MOST[fmt])))
            y = nearest(x / s[..., None, None], fmt).reshape(self.num_pages, hp, page, d)
            held = np.zeros((self.num_pages, page), bool)
            for u, n in enumerate(lens):
                n -= new[u]
                r = np.arange(n)
                held[table[u, r // page], r % page] = True
            if fmt == "e4m3":
                y[~held[:, None].repeat(hp, 1)] = np.nan
            s[~held.reshape(self.num_pages, 1, nb, BLOCK).any(3).repeat(hp, 1)] = np.nan
            self.num[name], self.scale[name] = y, s
        # the device's copy of that
        self.pool, self.scale_dev = {}, {}
        for name in ("k", "v"):
            t = torch.tensor(self.num[name])
            c = t.to(torch.int8) if fmt == "int8" else t.float().to(torch.float8_e4m3fn).view(
                torch.uint8)
            flat = torch.full((self.num_pages * self.apart,), 77, dtype=c.dtype)
            flat.as_strided(c.shape, (self.apart, page * d, d, 1)).copy_(c)
            dev = flat.cuda()
            dev = dev if fmt == "int8" else dev.view(torch.float8_e4m3fn)
            self.pool[name] = (dev, dev.as_strided(c.shape, (self.apart, page * d, d, 1)))
            self.scale_dev[name] = torch.tensor(self.scale[name]).float().cuda()
        self.slots_host = [int(table[u, (n - 1) // page]) * page + (n - 1) % page
                           for u, n in enumerate(lens) if new[u]]
        cu = np.concatenate([[0], np.cumsum([int(x) for x in new])])
        self.table = torch.tensor(table).to(torch.int32).cuda()
        self.lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.cu = torch.tensor(cu, dtype=torch.int64, device="cuda")
        self.slots = torch.tensor(self.slots_host, dtype=torch.int64, device="cuda")
        self.qd, self.knd, self.vnd = self.q.cuda(), self.k_new.cuda(), self.v_new.cuda()
        self.softmax_scale = d ** -0.5

    def args(self):
        return (self.pool["k"][1], self.pool["v"][1], self.scale_dev["k"], self.scale_dev["v"])

    def run(self, with_new=True, ws=None, out=None, stream=None):
        out = torch.full((self.seqs, self.hkv * self.G, self.d), float("nan"), dtype=self.dt,
                         device="cuda") if out is None else out
        if ws is None:
            n = kv.kv_paged_workspace_size(kv.KV_OP_QUANT_DECODE, self.shape)
            ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
        x = (self.knd, self.vnd, self.cu, self.slots) if with_new else (None,) * 4
        kv.quant_decode_attn(self.shape, FORMATS[self.fmt], self.qd, *x, *self.args(), self.table,
                             self.lens_t, self.softmax_scale, out, ws, stream)
        return out, ws

    def put(self, skip=()):
        """The new rows, as the definition stores them (tables in `skip` left out)."""
        at = 0
        for u, x in enumerate(self.new):
            if not x:
                continue
            slot = self.slots_host[at]
            at += 1
            if u in skip:
                continue
            b, h0 = u // self.tables, (u % self.tables) * self.hp
            for name, rows in (("k", self.k_new), ("v", self.v_new)):
                put(self.num[name], self.scale[name],
                    rows[b:b + 1, h0:h0 + self.hp].double().numpy(), [slot], self.fmt)

    def check_pools(self):
        """The device's codes and scales are the host's, and nothing between the pages changed."""
        for name in ("k", "v"):
            flat, pool = self.pool[name]
            got, want = numbers(pool.contiguous(), self.fmt), self.num[name]
            same = (got == want) | (np.isnan(got) & np.isnan(want))
            assert same.all(), (name, int((~same).sum()), np.argwhere(~same)[:4])
            assert np.array_equal(self.scale_dev[name].cpu().double().numpy(), self.scale[name],
                                  equal_nan=True), name
            gap = flat.view(torch.uint8).view(self.num_pages, self.apart)
            assert bool((gap[:, self.hp * self.page * self.d:] == 77).all())

    def rows(self, u, name):
        """Table u's rows as the cache holds them, [heads of a page][rows][d] float64."""
        n = self.lens[u]
        pages = self.table_host[u, :-(-n // self.page)]
        x = self.num[name][pages] * np.repeat(self.scale[name][pages], BLOCK, 2)[..., None]
        return x.transpose(1, 0, 2, 3).reshape(self.hp, -1, self.d)[:, :n]

    def expected(self, skip=()):
        """(out, bound) in 64 bits over what the cache holds now, [seqs][hq][d]; `skip`: (table,
        column) pairs whose rows are left out.

        The bound, as in tests.paged: u = 2^-23 a step of a float32 sum; a score is a sum of d
        products of exact factors (fp32 q held to 2^-22, taken as t = 2^-21), plus 2^-36 of q's largest
        element for what fp16 cuts off below it, and two roundings for its scale; an error of a
        score moves its weight by that share, above and below the fraction line; weights are held
        to 2^-22 (2^-21 taken), sums of m of them n u each; two more roundings for V's scale in
        every tile's sum; the last term is the output's rounding.

        A weight w <= 1 (the largest being 1) is held as 2^14 w = hi + lo in fp16.  fp16's numbers are
        2^-24 apart at least: where 2^14 w - hi is no more than 2^-25 * 2^12, lo holds it to 2^-25 only,
        so w is also off by 2^-25 2^-14 = 2^-39."""
        seqs, hkv, G, d = self.seqs, self.hkv, self.G, self.d
        out = np.zeros((seqs, hkv * G, d))
        tol = np.zeros_like(out)
        u23, t_p = 2.0 ** -23, 2.0 ** -21
        t_z = 0.0 if self.dtype == "bf16" else 2.0 ** -21
        half = torch.finfo(self.dt).eps / 2
        q = self.q.double().numpy()
        for tb, n in enumerate(self.lens):
            keep = np.ones(n, bool)
            for (a, c) in skip:
                if a == tb:
                    keep[c * self.page:(c + 1) * self.page] = False
            if not keep.any():
                continue
            ks, vs = self.rows(tb, "k"), self.rows(tb, "v")
            for h in range(self.hp):
                g0 = (tb % self.tables) * self.hp + h
                k, v = ks[h][keep], vs[h][keep]
                for g in range(G):
                    x = q[tb // self.tables, g0 * G + g]
                    c = abs(self.softmax_scale)
                    z = self.softmax_scale * (k @ x)
                    e_z = (c * ((d + 2) * u23 + t_z) * (np.abs(k) @ np.abs(x)) +
                           c * 2.0 ** -36 * np.abs(x).max() * np.abs(k).sum(1) +
                           4 * u23 * (1 + np.abs(z - z.max())))
                    p = np.exp(z - z.max())
                    p /= p.sum()
                    o = p @ v
                    m = len(p)
                    mag = p @ np.abs(v)
                    tol[tb // self.tables, g0 * G + g] = (
                        2 * (p * e_z) @ np.abs(v) + 2 * (p @ e_z) * mag +
                        (2 * m * u23 + 66 * u23 + t_p) * mag + half * np.abs(o) + 1e-30 +
                        2.0 ** -39 * p.max() * np.abs(v).sum(0))
                    out[tb // self.tables, g0 * G + g] = o
        return out, tol

    def check(self, out, skip=()):
        ref, tol = self.expected(skip)
        got = out.double().cpu().numpy()
        assert np.isfinite(got).all(), "not finite"
        bad = np.abs(got - ref) > tol
        if bad.any():
            i = np.unravel_index(np.argmax(np.where(bad, np.abs(got - ref) / tol, 0)), ref.shape)
            raise AssertionError("%d of %d off; worst at %s: got %r, expected %r +- %r" % (
                int(bad.sum()), bad.size, i, got[i], ref[i], tol[i]))
