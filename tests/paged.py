"""Test helpers of the paged cache: the page map's definition step by step in Python, a pool
with pages in an order of its own, and the decode attention in 64 bits with its error bound."""
from __future__ import annotations

import math

import numpy as np
import torch

import kv_cache_eviction_gb300 as kv

ERR_TABLE, ERR_PAGES, ERR_SLOTS, ERR_ID, ERR_RING = 7, 8, 9, 10, 11


def ceil_div(a, b):
    return -(-a // b)


def page_map_ref(lens, add, ring, state, cap, table, slots, page, num_pages):
    """kv_page_map by its definition, one table and one row after the other.  Returns the new
    (ring, state, table, lens, cu, slots) and the set of error codes."""
    ring, table, slots = ring.copy(), table.copy(), slots.copy()
    most = table.shape[1] * page
    head, tail = int(state[0]), int(state[1])
    codes = set()
    ring_ok = 0 <= head <= tail and tail - head <= num_pages
    avail = tail - head if ring_ok else 0
    ask = []
    for n, a in zip(map(int, lens), map(int, add)):
        bad = n < 0 or n > most or n + a > most
        now = n if bad else max(n + a, 0)
        ask.append((n, a, now, bad))
    back_total = sum(max(0, ceil_div(n, page) - ceil_div(now, page))
                     for n, a, now, bad in ask if not bad)
    back_ok = ring_ok and tail + back_total <= head + num_pages
    if not back_ok:
        codes.add(ERR_RING)
    cu, out = [0], []
    asked = taken = back = 0       # pages asked for so far, taken, returned
    for u, (n, a, now, bad) in enumerate(ask):
        gain = max(a, 0)
        cu.append(cu[-1] + gain)
        if bad:
            codes.add(ERR_TABLE)
        need = 0 if bad else max(0, ceil_div(now, page) - ceil_div(n, page))
        ok = not bad
        if gain > 0 and cu[-1] > cap:
            codes.add(ERR_SLOTS)
            ok = False
        if need > 0 and asked + need > avail:
            codes.add(ERR_PAGES)
            ok = False
        if a < 0 and now != n and not back_ok:
            ok = False
        if ok and need:
            for j in range(need):
                table[u, ceil_div(n, page) + j] = ring[(head + asked + j) % num_pages]
            taken = asked + need
        if ok and now < n:
            for c in range(ceil_div(now, page), ceil_div(n, page)):
                ring[(tail + back) % num_pages] = table[u, c]
                back += 1
                if not 0 <= table[u, c] < num_pages:
                    codes.add(ERR_ID)
        asked += need
        for i in range(gain):
            at = cu[u] + i
            if at >= cap:
                break
            slots[at] = -1
            if ok:
                p = int(table[u, (n + i) // page])
                if 0 <= p < num_pages:
                    slots[at] = p * page + (n + i) % page
                else:
                    codes.add(ERR_ID)
        out.append(now if ok else n)
    return (ring, np.array([head + taken, tail + back]), table, np.array(out), np.array(cu), slots,
            codes)


def workspace(op, shape, device="cuda"):
    return torch.zeros(kv.kv_paged_workspace_size(op, shape), dtype=torch.uint8, device=device)


class Cache:
    """A paged cache with the given rows per table: pages dealt out in a random order, junk (NaN
    too) in every row that no table holds.  The last row of the tables in `new` is left as junk
    in the pool and comes as k_new / v_new."""

    def __init__(self, seqs, hkv, G, d, tables, page, lens, dtype, seed, new=None, spare=3,
                 page_stride=0, first_page=0, temp=4.0):
        g = torch.Generator().manual_seed(seed)
        self.seqs, self.hkv, self.G, self.d = seqs, hkv, G, d
        self.tables, self.page, self.dtype = tables, page, dtype
        self.dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        U, hp = seqs * tables, hkv // tables
        lens = [int(x) for x in lens]
        assert len(lens) == U
        new = [n > 0 for n in lens] if new is None else [bool(x) and n > 0
                                                         for x, n in zip(new, lens)]
        used = [ceil_div(n, page) for n in lens]
        self.max_pages = max(1, max(used))
        num = sum(used) + spare
        order = torch.randperm(num, generator=g) + first_page
        self.num_pages = num + first_page
        table = torch.randint(0, self.num_pages, (U, self.max_pages), generator=g)
        at = 0
        for u, n in enumerate(used):
            table[u, :n] = order[at:at + n]
            at += n
        inner = hp * page * d
        self.shape = kv.KvPagedShape.of(seqs, hkv * G, hkv, d, tables, page, self.max_pages,
                                        dtype, self.num_pages, page_stride)
        stride = page_stride or inner
        tau = torch.exp(torch.rand(seqs, hkv * G, 1, generator=g) * math.log(8.0)) * temp / 8
        self.q = (torch.randn(seqs, hkv * G, d, generator=g) * tau).to(self.dt)
        self.k_new = torch.randn(seqs, hkv, d, generator=g).to(self.dt)
        self.v_new = torch.randn(seqs, hkv, d, generator=g).to(self.dt)
        # rows per (table, head of its page), the new one included
        self.rows = {"k": [], "v": []}
        pools = {}
        for name in ("k", "v"):
            flat = torch.full((self.num_pages * stride,), float("nan"), dtype=self.dt)
            pool = flat.as_strided((self.num_pages, hp, page, d), (stride, page * d, d, 1))
            for u, n in enumerate(lens):
                x = torch.randn(hp, n, d, generator=g).to(self.dt)
                if name == "v":
                    x = (x.float() * torch.exp(0.5 * torch.randn(hp, n, 1, generator=g))).to(self.dt)
                h0 = (u % tables) * hp
                if new[u]:
                    fresh = self.k_new if name == "k" else self.v_new
                    x[:, n - 1] = fresh[u // tables, h0:h0 + hp]
                self.rows[name].append(x)
                for j in range(used[u]):
                    n1 = min(page, n - j * page)
                    if new[u] and j == used[u] - 1:
                        n1 -= 1
                    pool[table[u, j], :, :n1] = x[:, j * page:j * page + n1]
            pools[name] = pool
        self.lens, self.new = lens, new
        cu = np.concatenate([[0], np.cumsum([int(x) for x in new])])
        slots = [int(table[u, (n - 1) // page]) * page + (n - 1) % page
                 for u, n in enumerate(lens) if new[u]]
        self.table_host = table
        dev = "cuda"
        self.table = table.to(torch.int32).to(dev)
        self.lens_t = torch.tensor(lens, dtype=torch.int32, device=dev)
        self.cu = torch.tensor(cu, dtype=torch.int64, device=dev)
        self.slots = torch.tensor(slots, dtype=torch.int64, device=dev)
        self.slots_host = slots
        # (as_strided pools keep their page stride on the device)
        self.pool_host = pools
        self.kp, self.vp = (self._to(pools[n], stride) for n in ("k", "v"))
        self.qd, self.knd, self.vnd = self.q.to(dev), self.k_new.to(dev), self.v_new.to(dev)
        self.scale = 1.0 / math.sqrt(d)

    def _to(self, pool, stride):
        flat = torch.full((self.num_pages * stride,), float("nan"), dtype=self.dt, device="cuda")
        t = flat.as_strided(pool.shape, pool.stride())
        t.copy_(pool)
        return t

    def run(self, with_new=True, ws=None, out=None, stream=None):
        out = torch.full((self.seqs, self.hkv * self.G, self.d), float("nan"), dtype=self.dt,
                         device="cuda") if out is None else out
        ws = workspace(kv.KV_OP_PAGED_DECODE, self.shape) if ws is None else ws
        x = (self.knd, self.vnd, self.cu, self.slots) if with_new else (None,) * 4
        kv.paged_decode_attn(self.shape, self.qd, *x, self.kp, self.vp, self.table, self.lens_t,
                             self.scale, out, ws, stream)
        return out, ws

    def expected(self, skip=()):
        """(out, bound) in 64 bits, [seqs][hq][d].  `skip`: (table, column) pairs whose rows are
        left out.

        The bound: u = 2^-23 a step of a float32 sum (half an ulp, doubled for sums that truncate).
        A score is a sum of d products, its error at most e_z = |scale| (d u + t) sum|q||k|, and
        a score's error moves its weight by that share, numerator and denominator alike; sums
        of n weights and products, n u each; t = 2^-21 covers factors held as two parts of 11
        (fp32) or 8 (bf16 weights: 2^-16) bits; the last term is the output's rounding."""
        seqs, hkv, G, d, page = self.seqs, self.hkv, self.G, self.d, self.page
        hp = hkv // self.tables
        out = np.zeros((seqs, hkv * G, d))
        tol = np.zeros_like(out)
        u23 = 2.0 ** -23
        t_z, t_p = (0.0, 2.0 ** -16) if self.dtype == "bf16" else (2.0 ** -21, 2.0 ** -21)
        half = torch.finfo(self.dt).eps / 2
        q = self.q.double().numpy()
        for tb, n in enumerate(self.lens):
            keep = np.ones(n, bool)
            for (a, c) in skip:
                if a == tb:
                    keep[c * page:(c + 1) * page] = False
            if not keep.any():
                continue
            for h in range(hp):
                g0 = (tb % self.tables) * hp + h
                k = self.rows["k"][tb][h].double().numpy()[keep]
                v = self.rows["v"][tb][h].double().numpy()[keep]
                for g in range(G):
                    x = q[tb // self.tables, g0 * G + g]
                    z = self.scale * (k @ x)
                    e_z = abs(self.scale) * (d * u23 + t_z) * (np.abs(k) @ np.abs(x)) + 4 * u23 * (
                        1 + np.abs(z - z.max()))
                    p = np.exp(z - z.max())
                    p /= p.sum()
                    o = p @ v
                    m = len(p)
                    mag = p @ np.abs(v)
                    tol[tb // self.tables, g0 * G + g] = (
                        2 * (p * e_z) @ np.abs(v) + 2 * (p @ e_z) * mag +
                        (2 * m * u23 + 64 * u23 + t_p) * mag + half * np.abs(o) + 1e-30)
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

    def check_pools(self, stored=True):
        """The pools hold what they held, and (stored) the new rows at their slots; nothing else
        changed."""
        hp = self.hkv // self.tables
        for name, pool in (("k", self.kp), ("v", self.vp)):
            want = self.pool_host[name].clone()
            if stored:
                fresh = self.k_new if name == "k" else self.v_new
                at = 0
                for u, x in enumerate(self.new):
                    if x:
                        s = self.slots_host[at]
                        at += 1
                        if 0 <= s < self.num_pages * self.page:
                            h0 = (u % self.tables) * hp
                            want[s // self.page, :, s % self.page] = \
                                fresh[u // self.tables, h0:h0 + hp]
            got = pool.cpu()
            same = (got == want) | (torch.isnan(got) & torch.isnan(want))
            assert bool(same.all()), name
