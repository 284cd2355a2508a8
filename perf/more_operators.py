"""Cases and plain forms of the rotary positions and of the paged cache in 8 bits.

Four operators of one serving step:

* ``rotary``: queries and keys turned by their positions, as a projection leaves them;
* ``write``: rows of K and V stored in 8 bits at their slots of the page pool, with a scale for
  each block of 16 rows and head;
* ``read``: rows of such a pool as the values they stand for;
* ``decode``: attention of one new token per sequence over such a pool; the new token's row comes
  as ``k_new`` / ``v_new`` and is stored at its slot in the same pass.

A block's scale is a power of two: the smallest, from 2^-96 on, that brings the largest of the rows
written into the code's range, and not below the one that the rows held before have (those are
rounded to the new scale).  Products with it are exact, so codes and scales are the same numbers
in 32 and in 64 bits.  A pool is returned as its codes' numbers (float8, or int8) beside its scales.

With ``own`` false, ``run`` computes the operators with elementary torch operations in 32 bits
(angles in 64); with ``own`` true it makes the calls of this repository's package.

Lengths are part of a case (drawn from its ``lens_seed``), so its work is known; values, page
numbers and everything else come from the seed given to ``prepare``.
"""
import math
import random

import torch

own = False

_I32, _I64 = torch.int32, torch.int64
BLOCK = 16          # rows of a block
LEAST = -96         # exponent of the smallest scale


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # One new token of each sequence of a decode batch: latency.
        _rotary("rotary 64 rows", rows=64, hq=32, hkv=8, d=128, rot=128, layout="half",
                dtype="bf16", scaling="none", fused=True, prompt=False),
        # A whole 128K prompt of one layer, from the fused projection's rows.
        _rotary("rotary 131072 rows", rows=131072, hq=32, hkv=8, d=128, rot=128, layout="half",
                dtype="bf16", scaling="linear", fused=True, prompt=True),
        # Interleaved pairs, part of the head, fp32, an odd number of rows.
        _rotary("rotary 20011 rows fp32 part", rows=20011, hq=6, hkv=2, d=80, rot=24,
                layout="interleaved", dtype="f32", scaling="yarn", fused=False, prompt=True),
        # One new row for each sequence of a decode batch, into blocks that hold rows already.
        _write("write 64 rows one each", rows=64, seqs=64, heads=8, d=128, page=16,
               format="e4m3", dtype="bf16", fused=True, lens_seed=31),
        # A whole 128K prompt of one layer, from the fused projection's rows.
        _write("write 131072 rows", rows=131072, seqs=1, heads=8, d=128, page=16, format="e4m3",
               dtype="bf16", fused=True, lens_seed=32),
        # Compacted rows of head tables (one head per page), fp32, in int8.
        _write("write 100003 rows int8 fp32", rows=100003, seqs=256, heads=1, d=64,
               page=32, format="int8", dtype="f32", fused=False, lens_seed=33),
        # The rows of a short shared prefix, for the attention of a prompt's next piece.
        _read("read 513 rows", rows=513, seqs=3, heads=8, d=128, page=16, format="e4m3",
              dtype="bf16", lens_seed=34),
        # The held part of a 128K prompt.
        _read("read 131072 rows int8", rows=131072, seqs=1, heads=8, d=128, page=64,
              format="int8", dtype="bf16", lens_seed=35),
        # The first tokens after a short prompt, one sequence: latency.
        _decode("decode 1 x 500", seqs=1, hq=32, hkv=8, d=128, tables=1, page=16, mean=500,
                sigma=0.0, format="e4m3", dtype="bf16", lens_seed=41),
        # 32 layers of one evicted sequence, every head with its own length and table.
        _decode("decode 256 head tables int8", seqs=32, hq=32, hkv=8, d=128, tables=8,
                page=16, mean=128, sigma=0.4, format="int8", dtype="bf16", lens_seed=42),
        # One sequence with a 128K context, fp32 queries and outputs.
        _decode("decode 1 x 131000 int8 fp32", seqs=1, hq=32, hkv=8, d=128, tables=1, page=64,
                mean=131000, sigma=0.0, format="int8", dtype="f32", lens_seed=43),
        # A full cache of a large batch: the streaming rate.
        _decode("decode 128 ragged 8000", seqs=128, hq=32, hkv=8, d=128, tables=1, page=32,
                mean=8000, sigma=0.3, format="e4m3", dtype="bf16", lens_seed=44),
    ]


def draw(rng):
    kind = rng.choice(["rotary", "write", "read", "decode", "decode"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind == "rotary":
        d = rng.choice([64, 72, 80, 96, 128, 128])
        rot = rng.choice([d, d, d // 2 // 8 * 8, 24, 32])
        hkv = rng.choice([1, 2, 4, 8])
        return _rotary(None, rows=_spread(rng, 1, 60000), hq=hkv * rng.choice([1, 2, 3, 4, 5, 7]),
                       hkv=hkv, d=d, rot=rot, layout=rng.choice(["half", "interleaved"]),
                       dtype=dtype, scaling=rng.choice(["none", "linear", "yarn"]),
                       fused=rng.random() < 0.5, prompt=rng.random() < 0.5)
    page, fmt = rng.choice([16, 16, 32, 64, 128, 256]), rng.choice(["e4m3", "e4m3", "int8"])
    seed = rng.randrange(1 << 30)
    if kind in ("write", "read"):
        rows, heads = _spread(rng, 1, 60000), rng.choice([1, 2, 4, 8])
        seqs = rng.choice([1, min(rows, 5), min(rows, 100), min(rows, 3 + rows // 40)])
        d = rng.choice([32, 64, 80, 96, 112, 128, 128])
        if kind == "read":
            return _read(None, rows=rows, seqs=seqs, heads=heads, d=d, page=page, format=fmt,
                         dtype=dtype, lens_seed=seed)
        return _write(None, rows=rows, seqs=seqs, heads=heads, d=d, page=page, format=fmt,
                      dtype=dtype, fused=rng.random() < 0.5, lens_seed=seed)
    hkv = rng.choice([1, 2, 4, 8])
    seqs = _spread(rng, 1, 128)
    most = 500_000 // (seqs * hkv) * 8
    return _decode(None, seqs=seqs, hq=hkv * rng.choice([1, 2, 3, 4, 5, 7, 8]), hkv=hkv,
                   d=rng.choice([32, 64, 80, 96, 112, 128, 128]), tables=rng.choice([1, 1, hkv]),
                   page=page, mean=_spread(rng, 1, max(2, min(131000, most))),
                   sigma=rng.uniform(0.0, 1.0), format=fmt, dtype=dtype, lens_seed=seed)


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _case(name, kw):
    return {**({"name": name} if name else {}), **kw}


def _rotary(name, **kw):
    return _case(name, {"op": "rotary", **kw})


def _write(name, **kw):
    return _case(name, {"op": "write", **kw})


def _read(name, **kw):
    return _case(name, {"op": "read", **kw})


def _decode(name, **kw):
    return _case(name, {"op": "decode", **kw})


def _ceil(a, b):
    return -(-a // b)


def _counts(case):
    """Rows of each sequence that a write or a read takes: ragged, at least one each."""
    r = random.Random(case["lens_seed"])
    seqs = case["seqs"]
    f = [math.exp(r.gauss(0.0, 1.0) * 0.5) for _ in range(seqs)]
    left, share = case["rows"] - seqs, sum(f)
    got = [1 + int(left * x / share) for x in f]
    for i in range(case["rows"] - sum(got)):
        got[i % seqs] += 1
    return got


def _decode_rows(case):
    """Per table: rows (the new one included), and whether it got a new row."""
    count = case["seqs"] * case["tables"]
    r = random.Random(case["lens_seed"])
    f = [math.exp(r.gauss(0.0, 1.0) * case["sigma"]) for _ in range(count)]
    top = sum(f) / count
    lens = [max(1, min(4 * case["mean"], round(x / top * case["mean"]))) for x in f]
    new = [int(r.random() >= 1 / 32) for _ in lens]   # one in thirty-two did not advance
    if count >= 16:
        lens[count // 2], new[count // 2] = 0, 0       # an empty slot of the batch
    return lens, new


def _size(case):
    return 2 if case["dtype"] == "bf16" else 4


def work(case):
    e = _size(case)
    if case["op"] == "rotary":
        rows, d, heads = case["rows"], case["d"], case["hq"] + case["hkv"]
        return {"bytes": rows * (2 * heads * d * e + 4) + 4 * case["rot"],
                "flops": 3.0 * rows * heads * case["rot"]}
    if case["op"] in ("write", "read"):
        elements = 2 * case["rows"] * case["heads"] * case["d"]
        blocks = sum(_ceil(n, BLOCK) for n in _counts(case)) * case["heads"]
        return {"bytes": elements * (e + 1) + 8 * case["rows"] + 8 * blocks, "flops": 0}
    lens, new = _decode_rows(case)
    heads = case["hkv"] // case["tables"]
    rows, fresh = sum(lens) * heads, sum(new) * heads
    blocks = sum(_ceil(n, BLOCK) for n in lens) * heads
    d, g = case["d"], case["hq"] // case["hkv"]
    table = 4 * sum(_ceil(n, case["page"]) for n in lens)
    return {"bytes": 2 * d * rows + 8 * blocks + 2 * d * fresh * e
                     + 2 * case["seqs"] * case["hq"] * d * e + table + 4 * len(lens),
            "flops": 4.0 * d * g * rows}


# --------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 2654435761 % (1 << 62) + 29)
    return g


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _codes(case):
    return torch.float8_e4m3fn if case["format"] == "e4m3" else torch.int8


def _inv_freq(case):
    """Angles per position of the pairs, in 64 bits: base 500000, stretched eight times by a
    divisor ("linear"), or for the slow pairs only with a ramp between ("yarn")."""
    rot, base, factor, trained = case["rot"], 500000.0, 8.0, 8192.0
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    f = base ** (-i / rot)
    if case["scaling"] == "none":
        return f, 1.0
    if case["scaling"] == "linear":
        return f / factor, 1.0

    def pair(turns):          # the pair that makes so many turns over the trained length
        return rot * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))

    lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), rot // 2 - 1)
    ramp = ((i / 2 - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0


def prepare(case, seed):
    return {"rotary": _prepare_rotary, "write": _prepare_write, "read": _prepare_read,
            "decode": _prepare_decode}[case["op"]](case, _gen(seed))


def _prepare_rotary(case, g):
    rows, hq, hkv, d, dt = (*(case[k] for k in ("rows", "hq", "hkv", "d")), _dtype(case))
    if case["fused"]:         # a fused q, k, v projection's rows
        src = torch.empty(rows, (hq + 2 * hkv) * d, dtype=dt, device="cuda")
        for i in range(0, rows, 16384):
            src[i:i + 16384] = torch.randn(src[i:i + 16384].shape, generator=g, device="cuda")
        q, k = src[:, :hq * d].unflatten(1, (hq, d)), src[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    else:
        q, k = (torch.randn(rows, h, d, generator=g, device="cuda").to(dt) for h in (hq, hkv))
    if case["prompt"]:        # one sequence, from some place on
        start = int(torch.randint(0, 1000, (1,), generator=g, device="cuda"))
        pos = start + torch.arange(rows, device="cuda")
    else:                     # sequences of a batch; an idle one has no position
        pos = torch.randint(0, 131072, (rows,), generator=g, device="cuda")
        pos[torch.rand(rows, generator=g, device="cuda") < 1 / 32] = -1
    f, magnitude = _inv_freq(case)
    return {"case": case, "q": q, "k": k, "pos": pos.to(_I32), "inv_freq": f.cuda(),
            "magnitude": magnitude, "q_out": torch.zeros(rows, hq, d, dtype=dt, device="cuda"),
            "k_out": torch.zeros(rows, hkv, d, dtype=dt, device="cuda")}


def _values(case, g, which, rows, heads):
    """Rows of keys (some columns larger than others) or values (some rows larger)."""
    d = case["d"]
    x = torch.randn(rows, heads, d, generator=g, device="cuda")
    if which == "k":
        return x.mul_(torch.randn(1, heads, d, generator=g, device="cuda").mul(0.7).exp())
    return x.mul_(torch.randn(rows, heads, 1, generator=g, device="cuda").mul(0.5).exp())


def _pool(case, g, which, num, heads):
    """A pool that some time of use has filled: codes and scales of random rows."""
    page, d = case["page"], case["d"]
    codes = torch.empty(num, heads, page, d, dtype=_codes(case), device="cuda")
    scale = torch.empty(num, heads, page // BLOCK, device="cuda")
    step = max(1, (1 << 26) // (heads * page * d))
    for i in range(0, num, step):
        n = min(step, num - i)
        x = _values(case, g, which, n * page // BLOCK * BLOCK, heads)
        x = x.view(n, page // BLOCK, BLOCK, heads, d).permute(0, 3, 1, 2, 4)
        s = _scale_for(x.abs().amax((3, 4)), case["format"])
        scale[i:i + n] = s
        codes[i:i + n] = _encode(x / s[..., None, None], case["format"]).view(codes.dtype).reshape(
            n, heads, page, d)
    return codes, scale


def _slots(case, g):
    """Slots of each sequence's rows, one after the other, from some row of a page on; pages in
    an order of their own."""
    page, counts = case["page"], _counts(case)
    used = [_ceil(n + page - 1, page) for n in counts]
    num = sum(used) + 4
    order = torch.randperm(num, generator=g, device="cuda")
    n = torch.tensor(counts, device="cuda")
    seq = torch.repeat_interleave(torch.arange(len(counts), device="cuda"), n)
    first = torch.tensor([0] + used, device="cuda").cumsum(0)[:-1]
    at = torch.randint(0, page, (len(counts),), generator=g, device="cuda")
    row = torch.arange(seq.numel(), device="cuda") - (n.cumsum(0) - n)[seq] + at[seq]
    return order[first[seq] + row // page] * page + row % page, num


def _prepare_write(case, g):
    rows, heads, d, dt = case["rows"], case["heads"], case["d"], _dtype(case)
    slots, num = _slots(case, g)
    s = {"case": case, "slots": slots, "num_pages": num}
    for name in ("k", "v"):
        s[name + "_pages"], s[name + "_scale"] = _pool(case, g, name, num, heads)
        x = _values(case, g, name, rows, heads).to(dt)
        if case["fused"]:     # beside the rest of a fused projection's rows
            wide = torch.zeros(rows, 3 * heads, d, dtype=dt, device="cuda")
            x = wide[:, heads:2 * heads].copy_(x)
        s[name] = x
    return s


def _prepare_read(case, g):
    rows, heads, d, dt = case["rows"], case["heads"], case["d"], _dtype(case)
    slots, num = _slots(case, g)
    s = {"case": case, "slots": slots, "num_pages": num}
    for name in ("k", "v"):
        s[name + "_pages"], s[name + "_scale"] = _pool(case, g, name, num, heads)
        s[name] = torch.zeros(rows, heads, d, dtype=dt, device="cuda")
    return s


def _prepare_decode(case, g):
    lens, new = _decode_rows(case)
    seqs, hq, hkv, d, page = (case[k] for k in ("seqs", "hq", "hkv", "d", "page"))
    dt, heads = _dtype(case), hkv // case["tables"]
    used = [_ceil(n, page) for n in lens]
    num, columns = sum(used) + 7, max(used) + 1
    order = torch.randperm(num, generator=g, device="cuda")
    held = torch.tensor(used, device="cuda")
    col = torch.arange(columns, device="cuda")
    pick = ((held.cumsum(0) - held)[:, None] + col).clamp(max=num - 1)
    stale = torch.randint(0, num, pick.shape, generator=g, device="cuda")
    table = torch.where(col < held[:, None], order[pick], stale).to(_I32).contiguous()
    n, fresh = torch.tensor(lens, device="cuda"), torch.tensor(new, device="cuda")
    last = (n - 1).clamp(min=0)
    slot = table.gather(1, (last // page)[:, None])[:, 0].to(_I64) * page + last % page
    # query heads as in this repository's workloads: temperatures from flat to peaked softmaxes
    tau = torch.exp(torch.rand(seqs, hq, 1, generator=g, device="cuda") * math.log(32.0)) * 0.5
    s = {"case": case, "num_pages": num, "table": table, "lens": n.to(_I32),
         "q": (torch.randn(seqs, hq, d, generator=g, device="cuda") * tau).to(dt),
         "cu": torch.cat([fresh.new_zeros(1), fresh.cumsum(0)]),
         "slots": slot[fresh > 0].contiguous(), "scale": 1.0 / math.sqrt(d),
         "out": torch.zeros(seqs, hq, d, dtype=dt, device="cuda")}
    for name in ("k", "v"):
        s[name + "_pages"], s[name + "_scale"] = _pool(case, g, name, num, heads)
        s[name + "_new"] = _values(case, g, name, seqs, hkv).to(dt)
    return s


# --------------------------------------------------------------------------- passes

def run(state):
    op = state["case"]["op"]
    if own:
        return {"rotary": _own_rotary, "write": _own_write, "read": _own_read,
                "decode": _own_decode}[op](state)
    return {"rotary": _plain_rotary, "write": _plain_write, "read": _plain_read,
            "decode": _plain_decode}[op](state)


def _scale_for(top, fmt):
    """The smallest power of two, from 2^LEAST on, that holds `top`: top <= 448 (127) of it."""
    m, e = torch.frexp(top)
    t = e - 9 + (m > 0.875) if fmt == "e4m3" else e - 7 + (m > 127 / 128)
    t = torch.where(top > 0, t, LEAST).clamp(min=LEAST).to(_I32)
    return ((t + 127) << 23).view(torch.float32)


def _encode(x, fmt):
    if fmt == "e4m3":
        return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return x.round().clamp(-127.0, 127.0).to(torch.int8)


def _decoded(raw, fmt):
    return (raw.view(torch.float8_e4m3fn) if fmt == "e4m3" else raw).float()


def _raw(codes):
    """Codes as bytes, which can be indexed (int8 stays)."""
    return codes if codes.dtype is torch.int8 else codes.view(torch.uint8)


def _put(codes, scale, x, slots, fmt):
    """Rows x [n][heads][d] at their slots; the rows of one block stand side by side."""
    raw = _raw(codes)
    num, heads, page, d = raw.shape
    per = page // BLOCK
    block = slots // BLOCK
    start = torch.cat([block.new_ones(1, dtype=torch.bool), block[1:] != block[:-1]])
    group = start.cumsum(0) - 1
    at = start.nonzero()[:, 0]
    first, p, b = slots[at] % BLOCK, block[at] // per, block[at] % per
    top = torch.zeros(at.numel(), heads, device=x.device)
    top.scatter_reduce_(0, group[:, None].expand(-1, heads), x.float().abs().amax(2), "amax")
    old = scale[p, :, b]
    s = _scale_for(top, fmt)
    s = torch.where(first[:, None] > 0, torch.maximum(s, old), s)
    # the rows held before, at the new scale
    blocks = raw.view(num, heads, per, BLOCK, d)
    rows = blocks[p, :, b]
    below = torch.arange(BLOCK, device=x.device) < first[:, None]
    again = _encode(_decoded(rows, fmt) * (old / s)[:, :, None, None], fmt)
    blocks[p, :, b] = torch.where(below[:, None, :, None], again, rows)
    scale[p, :, b] = s
    raw[slots // page, :, slots % page] = _encode(x.float() / s[group][:, :, None], fmt)


def _plain_rotary(s):
    c = s["case"]
    rot, half = c["rot"], c["rot"] // 2
    t = s["pos"].double()[:, None] * s["inv_freq"]
    cos = (t.cos() * s["magnitude"]).float()[:, None]
    sin = (t.sin() * s["magnitude"]).float()[:, None]
    there = (s["pos"] >= 0)[:, None, None]
    for x, out in ((s["q"], s["q_out"]), (s["k"], s["k_out"])):
        y = x.float()
        if c["layout"] == "half":
            a, b = y[..., :half], y[..., half:rot]
            turned = torch.cat([a * cos - b * sin, a * sin + b * cos], 2)
        else:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            turned = torch.stack([a * cos - b * sin, a * sin + b * cos], 3).flatten(2)
        y = torch.cat([turned, y[..., rot:]], 2)
        out.copy_(torch.where(there, y, out.float()))
    return {"q": s["q_out"], "k": s["k_out"]}


def _pools(s):
    return {n: s[n] for n in ("k_pages", "v_pages", "k_scale", "v_scale")}


def _plain_write(s):
    for n in ("k", "v"):
        _put(s[n + "_pages"], s[n + "_scale"], s[n], s["slots"], s["case"]["format"])
    return _pools(s)


def _plain_read(s):
    page, fmt = s["case"]["page"], s["case"]["format"]
    p, r = s["slots"] // page, s["slots"] % page
    for n in ("k", "v"):
        x = _decoded(_raw(s[n + "_pages"])[p, :, r], fmt)
        s[n].copy_(x * s[n + "_scale"][p, :, r // BLOCK][:, :, None])
    return {"k": s["k"], "v": s["v"]}


def _plain_decode(s):
    c = s["case"]
    seqs, hq, hkv, d, page, tables = (c[k] for k in ("seqs", "hq", "hkv", "d", "page", "tables"))
    heads, fmt = hkv // tables, c["format"]
    # the new rows, at their slots
    u = (s["cu"][1:] > s["cu"][:-1]).nonzero()[:, 0]
    if u.numel():
        slot = s["slots"][s["cu"][u + 1] - 1]
        for n in ("k", "v"):
            _put(s[n + "_pages"], s[n + "_scale"],
                 s[n + "_new"].reshape(seqs * tables, heads, d)[u], slot, fmt)

    def rows_of(n):
        at = s["table"].to(_I64)
        x = _decoded(_raw(s[n + "_pages"])[at], fmt)            # [tables][columns][heads][page][d]
        x = x.unflatten(3, (page // BLOCK, BLOCK)) * s[n + "_scale"][at][..., None, None]
        return x.permute(0, 2, 1, 3, 4, 5).reshape(seqs, hkv, -1, d)

    k = rows_of("k")
    n = s["lens"].to(_I64).reshape(seqs, tables).repeat_interleave(heads, 1)
    used = torch.arange(k.shape[2], device=k.device)[None, None] < n[:, :, None]
    q = s["q"].float().reshape(seqs, hkv, hq // hkv, d)
    z = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    del k
    z = z.masked_fill(~used[:, :, None], float("-inf"))
    top = z.amax(3, keepdim=True)
    p = torch.exp(z - top.masked_fill(top == float("-inf"), 0.0))
    v = rows_of("v").masked_fill(~used[..., None], 0.0)
    o = torch.matmul(p, v) / p.sum(3, keepdim=True).clamp(min=1e-30)
    s["out"].copy_(o.reshape(seqs, hq, d))
    return {"out": s["out"], **_pools(s)}


def _handle(s, op, **kw):
    """The shape and the zeroed workspace that a program keeps beside its cache."""
    if "handle" not in s:
        import kv_cache_eviction_gb300 as kv
        shape = kv.KvPagedShape.of(num_pages=s["num_pages"], dtype=s["case"]["dtype"], **kw)
        n = kv.kv_paged_workspace_size(getattr(kv, op), shape)
        fmt = kv.KV_E4M3 if s["case"]["format"] == "e4m3" else kv.KV_INT8
        s["handle"] = kv, shape, fmt, torch.zeros(n, dtype=torch.uint8, device="cuda")
    return s["handle"]


def _own_rotary(s):
    c = s["case"]
    if "handle" not in s:
        import kv_cache_eviction_gb300 as kv
        layout = kv.KV_ROTARY_HALF if c["layout"] == "half" else kv.KV_ROTARY_INTERLEAVED
        s["handle"] = kv, kv.KvRotaryShape.of(hq=c["hq"], hkv=c["hkv"], d=c["d"], rot=c["rot"],
                                              layout=layout, dtype=c["dtype"],
                                              magnitude=s["magnitude"])
    kv, shape = s["handle"]
    kv.kv_rotary(shape, s["q"], s["k"], s["pos"], s["inv_freq"], s["q_out"], s["k_out"])
    return {"q": s["q_out"], "k": s["k_out"]}


def _own_write(s):
    c = s["case"]
    kv, shape, fmt, ws = _handle(s, "KV_OP_QUANT_WRITE", seqs=1, hq=c["heads"], hkv=c["heads"],
                                 d=c["d"], tables=1, page=c["page"], max_pages=s["num_pages"])
    kv.kv_quant_write(shape, fmt, s["k"], s["v"], s["slots"], None, s["k_pages"], s["v_pages"],
                      s["k_scale"], s["v_scale"], ws)
    return _pools(s)


def _own_read(s):
    c = s["case"]
    kv, shape, fmt, ws = _handle(s, "KV_OP_QUANT_READ", seqs=1, hq=c["heads"], hkv=c["heads"],
                                 d=c["d"], tables=1, page=c["page"], max_pages=s["num_pages"])
    kv.kv_quant_read(shape, fmt, s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"],
                     s["slots"], None, s["k"], s["v"], ws)
    return {"k": s["k"], "v": s["v"]}


def _own_decode(s):
    c = s["case"]
    kv, shape, fmt, ws = _handle(s, "KV_OP_QUANT_DECODE", seqs=c["seqs"], hq=c["hq"],
                                 hkv=c["hkv"], d=c["d"], tables=c["tables"], page=c["page"],
                                 max_pages=s["table"].shape[1])
    kv.quant_decode_attn(shape, fmt, s["q"], s["k_new"], s["v_new"], s["cu"], s["slots"],
                         s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["table"],
                         s["lens"], s["scale"], s["out"], ws)
    return {"out": s["out"], **_pools(s)}


# --------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "write": _exact_write, "read": _exact_read,
            "decode": _exact_decode}[case["op"]](case, s)


def _exact_rotary(case, s):
    """Each pair as a complex number, times m exp(i t)."""
    rot, there = case["rot"], s["pos"] >= 0
    t = s["pos"].double()[:, None, None] * s["inv_freq"]
    turn = torch.polar(torch.full_like(t, s["magnitude"]), t)
    got = {}
    for name in ("q", "k"):
        x = s[name].double()
        pairs = x[..., :rot].unflatten(2, (2, rot // 2)).transpose(2, 3) if case["layout"] == "half" \
            else x[..., :rot].unflatten(2, (rot // 2, 2))
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z = z.transpose(2, 3) if case["layout"] == "half" else z
        y = torch.cat([z.flatten(2), x[..., rot:]], 2)
        y[~there] = s[name + "_out"].double()[~there]
        got[name] = y
    return got


def _numbers(codes, fmt):
    """The codes' numbers in 64 bits."""
    return codes.float().double() if fmt == "e4m3" else codes.double()


def _round64(x, fmt):
    """To the nearest number of the code, halves to the even one, in 64 bits."""
    if fmt == "int8":
        return x.round().clamp(-127, 127)
    step = torch.exp2(torch.frexp(x)[1].clamp(min=-5).double() - 4)   # of 2^-6 .. : 3 bits behind the first
    return ((x / step).round() * step).clamp(-448, 448)


def _scale64(top, fmt):
    most = 448.0 if fmt == "e4m3" else 127.0
    t = torch.log2(top / most).ceil().clamp(min=LEAST)
    t = torch.where(top > most * torch.exp2(t), t + 1, t)
    return torch.exp2(torch.where((top <= most * torch.exp2(t - 1)) & (t > LEAST), t - 1, t))


def _exact_put(numbers, scale, x, slots, fmt):
    """numbers [pages][heads][page][d], scale [pages][heads][page / 16], both 64 bits; in place."""
    num, heads, page, d = numbers.shape
    # rows of the pool as [slot], blocks as [block]
    flat = numbers.permute(0, 2, 1, 3).clone().reshape(-1, BLOCK, heads, d)
    s = scale.transpose(1, 2).reshape(-1, heads).clone()
    blocks, place = torch.unique(slots // BLOCK, return_inverse=True)
    row = slots % BLOCK
    fresh = torch.full((blocks.numel(), BLOCK, heads, d), float("nan"), dtype=torch.float64,
                       device=x.device)
    fresh[place, row] = x.double()
    given = torch.zeros(blocks.numel(), BLOCK, dtype=torch.bool, device=x.device)
    given[place, row] = True
    held = given.long().cumsum(1) == 0                      # rows before the first one written
    top = fresh.abs().nan_to_num(0.0).amax((1, 3))
    now = _scale64(top, fmt)
    old = s[blocks]
    now = torch.where(held[:, :1], torch.maximum(now, old), now)
    was = flat[blocks]
    kept = _round64(was * (old / now)[:, None, :, None], fmt)
    put = _round64(fresh / now[:, None, :, None], fmt)
    flat[blocks] = torch.where(given[..., None, None], put,
                               torch.where(held[..., None, None], kept, was))
    s[blocks] = now
    numbers.copy_(flat.reshape(num, page, heads, d).permute(0, 2, 1, 3))
    scale.copy_(s.reshape(num, page // BLOCK, heads).transpose(1, 2))


def _exact_pools(s, fmt, k, v, slots):
    got = {}
    for name, x in (("k", k), ("v", v)):
        n, sc = _numbers(s[name + "_pages"], fmt), s[name + "_scale"].double()
        if slots.numel():
            _exact_put(n, sc, x, slots, fmt)
        got[name + "_pages"], got[name + "_scale"] = n, sc
    return got


def _exact_write(case, s):
    got = _exact_pools(s, case["format"], s["k"], s["v"], s["slots"])
    if case["format"] == "int8":
        got = {n: x.to(torch.int8) if "pages" in n else x for n, x in got.items()}
    return got


def _exact_read(case, s):
    page, got = case["page"], {}
    p, r = s["slots"] // page, s["slots"] % page
    for name in ("k", "v"):
        n = _numbers(s[name + "_pages"], case["format"]).permute(0, 2, 1, 3)
        sc = s[name + "_scale"].double().repeat_interleave(BLOCK, 2).permute(0, 2, 1)
        got[name] = n[p, r] * sc[p, r][..., None]
    return got


def _exact_decode(case, s):
    seqs, hkv, d, tables, page = (case[k] for k in ("seqs", "hkv", "d", "tables", "page"))
    lens, new = _decode_rows(case)
    group, heads, fmt = case["hq"] // hkv, hkv // tables, case["format"]
    which = [u for u, x in enumerate(new) if x]
    rows = {n: s[n + "_new"].reshape(seqs * tables, heads, d)[which] for n in ("k", "v")}
    got = _exact_pools(s, fmt, rows["k"], rows["v"], s["slots"])
    q = s["q"].double().reshape(seqs, hkv, group, d)
    out = torch.zeros(seqs, hkv, group, d, dtype=torch.float64, device="cuda")
    for u, n in enumerate(lens):
        if n == 0:
            continue
        b, h0 = u // tables, (u % tables) * heads
        pages = s["table"][u, :_ceil(n, page)].long()
        x = {}
        for name in ("k", "v"):
            sc = got[name + "_scale"][pages].repeat_interleave(BLOCK, 2)[..., None]
            x[name] = (got[name + "_pages"][pages] * sc).transpose(0, 1).flatten(1, 2)[:, :n]
        z = q[b, h0:h0 + heads] @ x["k"].transpose(1, 2) * s["scale"]
        e = (z - z.amax(2, keepdim=True)).exp()
        out[b, h0:h0 + heads] = (e / e.sum(2, keepdim=True)) @ x["v"]
    if fmt == "int8":
        got = {n: t.to(torch.int8) if "pages" in n else t for n, t in got.items()}
    return {"out": out.reshape(seqs, -1, d), **got}
