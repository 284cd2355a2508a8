"""Cases and plain forms of the paged-cache operators.

Three operators that a serving step runs one after the other:

* ``map``: block tables, slot map and free ring brought up to date from the lengths held and the
  rows each table gains or loses;
* ``write``: rows of K and V stored at their slots of the page pool;
* ``decode``: attention of one new token per sequence over the paged cache; the new token's row
  comes as ``k_new`` / ``v_new`` and is stored at its slot in the same pass.

With ``own`` false, ``run`` computes them with elementary torch operations in 32 bits; with
``own`` true it makes the calls of this repository's package.

The lengths are part of a case (drawn from its ``lens_seed``), so its work is known; values,
page numbers and everything else come from the seed given to ``prepare``.
"""
import math
import random

import torch

own = False

_I32, _I64 = torch.int32, torch.int64


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # The block tables of a small batch between two decode steps: pure latency.
        _map("map 8 sequences, one token", seqs=8, tables=1, page=16, mean=900, sigma=0.6,
             grow="one", hkv=8, lens_seed=11),
        # Every head of 4 sequences x 32 layers with a table of its own (an evicted cache).
        _map("map 1024 head tables, one token", seqs=128, tables=8, page=16, mean=1024,
             sigma=0.5, grow="one", hkv=8, lens_seed=12),
        # Prompts of many sequences admitted at once while others finish or are evicted.
        _map("map 96 prompts, some released", seqs=96, tables=1, page=16, mean=8192, sigma=0.7,
             grow="prompt", hkv=8, lens_seed=13),
        # One new row per sequence of a decode batch, from the projections' output.
        _write("write 64 rows", rows=64, heads=8, d=128, dtype="bf16", page=16, fused=True),
        # A whole 128K prompt of one layer.
        _write("write 131072 rows", rows=131072, heads=8, d=128, dtype="bf16", page=16,
               fused=True),
        # Compacted rows of head tables (one head per page), fp32, an odd number of rows.
        _write("write 100003 head rows, fp32", rows=100003, heads=1, d=64, dtype="f32", page=32,
               fused=False),
        # The first tokens after a short prompt, one sequence: latency.
        _decode("decode 1 x 500", seqs=1, hq=32, hkv=8, d=128, tables=1, page=16, mean=500,
                sigma=0.0, dtype="bf16", lens_seed=21),
        # One sequence with a 128K context: the whole card works on one request.
        _decode("decode 1 x 131000", seqs=1, hq=32, hkv=8, d=128, tables=1, page=64, mean=131000,
                sigma=0.0, dtype="bf16", lens_seed=22),
        # A batch of ragged chats.
        _decode("decode 64 ragged, mean 2000", seqs=64, hq=32, hkv=8, d=128, tables=1, page=16,
                mean=2000, sigma=0.8, dtype="bf16", lens_seed=23),
        # 32 layers of one evicted sequence, every head with its own length and table.
        _decode("decode 256 head tables, mean 128", seqs=32, hq=32, hkv=8, d=128, tables=8,
                page=16, mean=128, sigma=0.4, dtype="bf16", lens_seed=24),
        # A full cache of a large batch: the streaming rate.
        _decode("decode 128 ragged, mean 8000", seqs=128, hq=32, hkv=8, d=128, tables=1, page=32,
                mean=8000, sigma=0.3, dtype="bf16", lens_seed=25),
        # fp32, three query heads to a KV head, a head dim that fills no 128-byte line, small pages.
        _decode("decode 5 ragged, fp32, d 72", seqs=5, hq=6, hkv=2, d=72, tables=1, page=8,
                mean=3001, sigma=0.7, dtype="f32", lens_seed=26),
    ]


def draw(rng):
    kind = rng.choice(["map", "write", "decode", "decode"])
    if kind == "map":
        tables = rng.choice([1, 1, 8])
        grow = rng.choice(["one", "prompt"])
        seqs = _spread(rng, 1, 128)
        mean = _spread(rng, 20, 8000)
        if tables > 1 and grow == "prompt":
            mean = min(mean, 1000)
        return _map(None, seqs=seqs, tables=tables, page=rng.choice([8, 16, 32, 64, 128]),
                    mean=mean, sigma=rng.uniform(0.0, 0.9), grow=grow, hkv=8,
                    lens_seed=rng.randrange(1 << 30))
    if kind == "write":
        heads = rng.choice([1, 2, 4, 8])
        return _write(None, rows=_spread(rng, 1, 100000), heads=heads,
                      d=rng.choice([64, 72, 80, 96, 128]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                      page=rng.choice([8, 16, 32, 64, 128, 256]), fused=rng.random() < 0.5)
    hkv = rng.choice([1, 2, 4, 8])
    seqs = _spread(rng, 1, 128)
    most = 500_000 // (seqs * hkv) * 8
    return _decode(None, seqs=seqs, hq=hkv * rng.choice([1, 2, 3, 4, 5, 7, 8]), hkv=hkv,
                   d=rng.choice([64, 80, 96, 128, 128]), tables=rng.choice([1, 1, hkv]),
                   page=rng.choice([8, 16, 16, 32, 64, 128]),
                   mean=_spread(rng, 1, max(2, min(131000, most))), sigma=rng.uniform(0.0, 1.0),
                   dtype=rng.choice(["bf16", "bf16", "f32"]), lens_seed=rng.randrange(1 << 30))


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _case(name, kw):
    return {**({"name": name} if name else {}), **kw}


def _map(name, **kw):
    return _case(name, {"op": "map", **kw})


def _write(name, **kw):
    return _case(name, {"op": "write", **kw})


def _decode(name, **kw):
    return _case(name, {"op": "decode", **kw})


def _lengths(case, count):
    """`count` log-normal lengths of the case's mean, the same for every seed."""
    r = random.Random(case["lens_seed"])
    f = [math.exp(r.gauss(0.0, 1.0) * case["sigma"]) for _ in range(count)]
    top = sum(f) / count
    return [max(1, min(4 * case["mean"], round(x / top * case["mean"]))) for x in f]


def _ceil(a, b):
    return -(-a // b)


def _map_rows(case):
    """Per table: rows held, rows gained (or, negative, lost)."""
    count = case["seqs"] * case["tables"]
    want, r = _lengths(case, count), random.Random(case["lens_seed"] + 1)
    held, add = [], []
    for n in want:
        x = r.random()
        if case["grow"] == "one":          # a decode step: one sequence in sixteen is idle
            held.append(n)
            add.append(0 if x < 1 / 16 else 1)
        elif x < 0.5:                      # a prompt admitted whole
            held.append(0)
            add.append(n)
        elif x < 0.75:                     # the next piece of a prompt
            held.append(n // 2)
            add.append(n - n // 2)
        elif x < 0.9:                      # evicted to a share of its rows
            held.append(n)
            add.append(-(2 * n // 3))
        else:                              # finished
            held.append(n)
            add.append(-n)
    return held, add


def _decode_rows(case):
    """Per table: rows (the new one included), and whether it got a new row."""
    count = case["seqs"] * case["tables"]
    lens = _lengths(case, count)
    r = random.Random(case["lens_seed"] + 1)
    new = [int(r.random() >= 1 / 32) for _ in lens]   # one in thirty-two did not advance
    if count >= 16:
        lens[count // 2], new[count // 2] = 0, 0       # an empty slot of the batch
    return lens, new


def _size(case):
    return 2 if case["dtype"] == "bf16" else 4


def work(case):
    if case["op"] == "map":
        held, add = _map_rows(case)
        page = case["page"]
        pages = rows = 0
        for n, a in zip(held, add):
            m = max(n + a, 0)
            pages += abs(_ceil(m, page) - _ceil(n, page))
            rows += max(a, 0)
        # lens, add in; lens, cu out; per page one entry read and one written; slots out
        return {"bytes": len(held) * (4 + 4 + 4 + 8) + 8 * pages + 8 * rows + 32, "flops": 0}
    if case["op"] == "write":
        row = case["heads"] * case["d"] * _size(case)
        return {"bytes": case["rows"] * (2 * 2 * row + 8), "flops": 0}
    lens, new = _decode_rows(case)
    heads = case["hkv"] // case["tables"]
    rows = sum(lens) * heads                       # K/V rows over all heads
    fresh = sum(new) * heads                       # of them, rows that come as k_new / v_new
    e, d, g = _size(case), case["d"], case["hq"] // case["hkv"]
    q = case["seqs"] * case["hq"] * d
    table = 4 * sum(_ceil(n, case["page"]) for n in lens)
    return {"bytes": e * (2 * d * (rows + fresh) + 2 * q) + table + 4 * len(lens),
            "flops": 4.0 * d * g * rows}


# --------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 2654435761 % (1 << 62) + 17)
    return g


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _tables(case, g, used, slack, columns):
    """A pool's page numbers in an order of their own, dealt out table by table: the block table
    (unused entries hold page numbers of earlier use) and the numbers left over."""
    total = sum(used)
    num = total + slack
    order = torch.randperm(num, generator=g, device="cuda")
    first = torch.tensor([0] + used, device="cuda").cumsum(0)[:-1]
    n = torch.tensor(used, device="cuda")
    col = torch.arange(columns, device="cuda")
    pick = (first[:, None] + col[None, :]).clamp(max=num - 1)
    stale = torch.randint(0, num, pick.shape, generator=g, device="cuda")
    table = torch.where(col[None, :] < n[:, None], order[pick], stale).to(_I32)
    return table.contiguous(), order[total:].to(_I32), num


def prepare(case, seed):
    g = _gen(seed)
    return {"map": _prepare_map, "write": _prepare_write, "decode": _prepare_decode}[case["op"]](
        case, g)


def _prepare_map(case, g):
    held, add = _map_rows(case)
    page = case["page"]
    used = [_ceil(n, page) for n in held]
    need = sum(max(0, _ceil(max(n + a, 0), page) - _ceil(n, page)) for n, a in zip(held, add))
    columns = max(_ceil(max(n, n + a), page) for n, a in zip(held, add)) + 1
    table, free, num = _tables(case, g, used, need + 5 + need // 8, columns)
    # the free ring as some time of use leaves it: it starts anywhere and wraps around
    start = int(torch.randint(0, num, (1,), generator=g, device="cuda"))
    ring = torch.full((num,), -1, dtype=_I32, device="cuda")
    ring[(start + torch.arange(free.numel(), device="cuda")) % num] = free
    rows = sum(max(a, 0) for a in add)
    return {"case": case, "table": table, "num_pages": num,
            "lens": torch.tensor(held, dtype=_I32, device="cuda"),
            "add": torch.tensor(add, dtype=_I32, device="cuda"),
            "ring": ring, "free": torch.tensor([start, start + free.numel()], device="cuda"),
            "lens_out": torch.zeros(len(held), dtype=_I32, device="cuda"),
            "free_out": torch.zeros(2, dtype=_I64, device="cuda"),
            "cu": torch.zeros(len(held) + 1, dtype=_I64, device="cuda"),
            "slots": torch.full((rows + 3,), -1, dtype=_I64, device="cuda")}


def _prepare_write(case, g):
    rows, heads, d, page = case["rows"], case["heads"], case["d"], case["page"]
    dt = _dtype(case)
    num = _ceil(rows, page) + 4
    # rows of sequences one after the other: runs of slots within pages in an order of their own
    order = torch.randperm(num, generator=g, device="cuda")
    at = torch.arange(rows, device="cuda") + page // 2
    slots = order[at // page] * page + at % page
    width = 3 * heads * d if case["fused"] else heads * d     # a fused q, k, v projection's rows
    src = torch.randn(2, rows, width, generator=g, device="cuda").to(dt)
    if case["fused"]:
        k, v = src[0, :, heads * d:2 * heads * d], src[0, :, 2 * heads * d:]
    else:
        k, v = src[0], src[1]
    return {"case": case, "k": k, "v": v, "slots": slots, "num_pages": num,
            "k_pages": torch.zeros(num, heads, page, d, dtype=dt, device="cuda"),
            "v_pages": torch.zeros(num, heads, page, d, dtype=dt, device="cuda")}


def _prepare_decode(case, g):
    lens, new = _decode_rows(case)
    seqs, hq, hkv, d, page = (case[k] for k in ("seqs", "hq", "hkv", "d", "page"))
    dt = _dtype(case)
    used = [_ceil(n, page) for n in lens]
    table, _, num = _tables(case, g, used, 7, max(used) + 1)
    n = torch.tensor(lens, device="cuda")
    fresh = torch.tensor(new, device="cuda")
    cu = torch.cat([fresh.new_zeros(1), fresh.cumsum(0)])
    last = (n - 1).clamp(min=0)
    slot = table.gather(1, (last // page)[:, None])[:, 0].to(_I64) * page + last % page
    heads = hkv // case["tables"]
    # query heads as in this repository's workloads: temperatures from flat to peaked softmaxes
    tau = torch.exp(torch.rand(seqs, hq, 1, generator=g, device="cuda") * math.log(32.0)) * 0.5

    def values(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    def pool():
        p = torch.empty(num, heads, page, d, dtype=dt, device="cuda")
        for i in range(0, num, 16384):
            p[i:i + 16384] = values(*p[i:i + 16384].shape).to(dt)
        return p

    return {"case": case, "num_pages": num, "table": table,
            "lens": torch.tensor(lens, dtype=_I32, device="cuda"),
            "q": (values(seqs, hq, d) * tau).to(dt), "k_new": values(seqs, hkv, d).to(dt),
            "v_new": values(seqs, hkv, d).to(dt), "cu": cu, "slots": slot[fresh > 0].contiguous(),
            "k_pages": pool(), "v_pages": pool(), "scale": 1.0 / math.sqrt(d),
            "out": torch.zeros(seqs, hq, d, dtype=dt, device="cuda")}


# --------------------------------------------------------------------------- passes

def run(state):
    op = state["case"]["op"]
    if own:
        return {"map": _own_map, "write": _own_write, "decode": _own_decode}[op](state)
    return {"map": _plain_map, "write": _plain_write, "decode": _plain_decode}[op](state)


def _map_outputs(s):
    return {"table": s["table"], "lens": s["lens_out"], "cu": s["cu"], "slots": s["slots"],
            "ring": s["ring"], "free": s["free_out"]}


def _plain_map(s):
    page, num = s["case"]["page"], s["num_pages"]
    held, add = s["lens"].to(_I64), s["add"].to(_I64)
    want = (held + add).clamp(min=0)
    gain = add.clamp(min=0)
    before, after = (held + page - 1) // page, (want + page - 1) // page
    need, loss = (after - before).clamp(min=0), (before - after).clamp(min=0)
    s["cu"][1:] = gain.cumsum(0)
    s["lens_out"].copy_(want)
    first, put = need.cumsum(0) - need, loss.cumsum(0) - loss
    head, tail = s["free"][0], s["free"][1]
    s["free_out"].copy_(torch.stack([head + need.sum(), tail + loss.sum()]))
    # pages given: entries [before, after) of a table, from the head of the ring
    col = torch.arange(s["table"].shape[1], device=held.device)[None, :]
    at = (head + first[:, None] + col - before[:, None]) % num
    given = (col >= before[:, None]) & (col < after[:, None])
    # pages returned: entries [after, before), to its tail
    back = (col >= after[:, None]) & (col < before[:, None])
    to = (tail + put[:, None] + col - after[:, None]) % num
    entries = s["table"][back]
    s["table"].copy_(torch.where(given, s["ring"][at], s["table"]))
    s["ring"][to[back]] = entries
    # slots of the rows gained, table after table
    i = torch.arange(s["slots"].numel(), device=held.device)
    u = (torch.searchsorted(s["cu"], i, right=True) - 1).clamp(max=held.numel() - 1)
    row = held[u] + i - s["cu"][u]
    c = (row // page).clamp(max=s["table"].shape[1] - 1)
    slot = s["table"][u, c].to(_I64) * page + row % page
    s["slots"].copy_(torch.where(i < s["cu"][-1], slot, s["slots"]))
    return _map_outputs(s)


def _plain_write(s):
    c = s["case"]
    page, heads, d = c["page"], c["heads"], c["d"]
    p, r = s["slots"] // page, s["slots"] % page
    s["k_pages"][p, :, r] = s["k"].reshape(-1, heads, d)
    s["v_pages"][p, :, r] = s["v"].reshape(-1, heads, d)
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_decode(s):
    c = s["case"]
    seqs, hq, hkv, d, page, tables = (c[k] for k in ("seqs", "hq", "hkv", "d", "page", "tables"))
    heads = hkv // tables
    # the new rows, at their slots
    u = (s["cu"][1:] > s["cu"][:-1]).nonzero()[:, 0]
    slot = s["slots"][s["cu"][u + 1] - 1]
    for pages, rows in ((s["k_pages"], s["k_new"]), (s["v_pages"], s["v_new"])):
        pages[slot // page, :, slot % page] = rows.reshape(seqs * tables, heads, d)[u]

    def rows_of(pages):
        x = pages[s["table"].to(_I64)]                      # [tables][columns][heads][page][d]
        x = x.permute(0, 2, 1, 3, 4).float()
        return x.reshape(seqs, hkv, -1, d)

    k = rows_of(s["k_pages"])
    n = s["lens"].to(_I64).reshape(seqs, tables).repeat_interleave(heads, 1)
    used = torch.arange(k.shape[2], device=k.device)[None, None] < n[:, :, None]
    q = s["q"].float().reshape(seqs, hkv, hq // hkv, d)
    z = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    del k
    z = z.masked_fill(~used[:, :, None], float("-inf"))
    top = z.amax(3, keepdim=True)
    p = torch.exp(z - top.masked_fill(top == float("-inf"), 0.0))
    v = rows_of(s["v_pages"]).masked_fill(~used[..., None], 0.0)
    o = torch.matmul(p, v) / p.sum(3, keepdim=True).clamp(min=1e-30)
    s["out"].copy_(o.reshape(seqs, hq, d))
    return {"out": s["out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _handle(s, op, **kw):
    """The shape and the zeroed workspace that a program keeps beside its cache."""
    if "handle" not in s:
        import kv_cache_eviction_gb300 as kv
        shape = kv.KvPagedShape.of(num_pages=s["num_pages"], **kw)
        n = kv.kv_paged_workspace_size(getattr(kv, op), shape)
        s["handle"] = kv, shape, torch.zeros(n, dtype=torch.uint8, device="cuda")
    return s["handle"]


def _own_map(s):
    c = s["case"]
    kv, shape, ws = _handle(s, "KV_OP_PAGE_MAP", seqs=c["seqs"], hq=c["hkv"], hkv=c["hkv"], d=128,
                            tables=c["tables"], page=c["page"], max_pages=s["table"].shape[1],
                            dtype="bf16")
    kv.kv_page_map(shape, s["lens"], s["add"], s["ring"], s["free"], s["table"], s["lens_out"],
                   s["free_out"], s["cu"], s["slots"], ws)
    return _map_outputs(s)


def _own_write(s):
    c = s["case"]
    kv, shape, ws = _handle(s, "KV_OP_PAGED_WRITE", seqs=1, hq=c["heads"], hkv=c["heads"],
                            d=c["d"], tables=1, page=c["page"], max_pages=s["num_pages"],
                            dtype=c["dtype"])
    kv.kv_paged_write(shape, s["k"], s["v"], s["slots"], None, s["k_pages"], s["v_pages"], ws)
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _own_decode(s):
    c = s["case"]
    kv, shape, ws = _handle(s, "KV_OP_PAGED_DECODE", seqs=c["seqs"], hq=c["hq"], hkv=c["hkv"],
                            d=c["d"], tables=c["tables"], page=c["page"],
                            max_pages=s["table"].shape[1], dtype=c["dtype"])
    kv.paged_decode_attn(shape, s["q"], s["k_new"], s["v_new"], s["cu"], s["slots"],
                         s["k_pages"], s["v_pages"], s["table"], s["lens"], s["scale"], s["out"],
                         ws)
    return {"out": s["out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


# --------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    if case["op"] == "map":
        return None                       # whole numbers
    s = prepare(case, seed)
    page = case["page"]
    if case["op"] == "write":
        heads, d = case["heads"], case["d"]
        got = {}
        for name in ("k", "v"):
            pool = s[name + "_pages"].double().permute(0, 2, 1, 3).reshape(-1, heads * d)
            pool.index_copy_(0, s["slots"], s[name].double())
            got[name + "_pages"] = pool.reshape(-1, page, heads, d).permute(0, 2, 1, 3).contiguous()
        return got
    seqs, hkv, d, tables = case["seqs"], case["hkv"], case["d"], case["tables"]
    lens, new = _decode_rows(case)
    group, heads = case["hq"] // hkv, hkv // tables
    pools = {name: s[name + "_pages"].double() for name in ("k", "v")}
    out = torch.zeros(seqs, hkv, group, d, dtype=torch.float64, device="cuda")
    for u, n in enumerate(lens):
        b, h0 = u // tables, (u % tables) * heads
        if n == 0:
            continue
        pages = s["table"][u, :_ceil(n, page)].long()
        rows = {}
        for name in ("k", "v"):
            if new[u]:
                pools[name][int(pages[-1]), :, (n - 1) % page] = (
                    s[name + "_new"][b, h0:h0 + heads].double())
            rows[name] = pools[name][pages].transpose(0, 1).flatten(1, 2)[:, :n]
        for h in range(heads):
            z = (rows["k"][h] @ s["q"].double()[b].reshape(hkv, group, d)[h0 + h].T) * s["scale"]
            e = (z - z.max(0).values).exp()
            out[b, h0 + h] = (e / e.sum(0)).T @ rows["v"][h]
    return {"out": out.reshape(seqs, -1, d), "k_pages": pools["k"], "v_pages": pools["v"]}
