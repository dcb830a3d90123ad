"""Cases of the operators that surround the packed KV cache in a serving step.

* ``qk_norm_rope``: the norm of every query and key head and the rotation by
  position, read from the strided output of a fused projection and written as
  the fp16 rows that the codec encodes and the attention reads.
* ``attend_window``: attention of one or more query tokens per sequence over
  packed caches, causal, limited to a sliding window plus the first tokens.
* ``fork`` / ``trim`` / ``compact``: the pages of a paged packed cache: a child
  sequence sharing its parent's pages, pages freed that no later query sees,
  and the used pages moved to the front of the pools.

``listed()`` and ``draw()`` give cases, ``prepare()`` their inputs, ``run()`` one
pass (plain torch operations, or this package's calls where ``own`` is true),
``work()`` the bytes and operations of a pass and ``exact()`` its result in 64
bits.
"""

import functools
import math

import numpy as np
import torch

own = False

BLOCK = 16  # positions of a page
SEED = 42  # sign flips of the codec


# ------------------------------------------------------------------ the format


@functools.lru_cache(maxsize=None)
def _levels(bits):
    """The Lloyd-Max levels of N(0,1) on the 2^-14 grid (a tuple, ascending)."""
    m = 1 << (bits - 1)
    x = [3.0 * (k + 0.5) / m for k in range(m)]
    for _ in range(20000):
        b = [0.0] + [0.5 * (x[k - 1] + x[k]) for k in range(1, m)] + [40.0]
        tail = [0.5 * math.erfc(v / math.sqrt(2.0)) for v in b]
        dens = [math.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi) for v in b]
        y = [(dens[k] - dens[k + 1]) / (tail[k] - tail[k + 1]) for k in range(m)]
        moved = max(abs(u - v) for u, v in zip(x, y))
        x = y
        if moved < 1e-15:
            break
    half = [round(v * 16384.0) / 16384.0 for v in x]
    return tuple([-v for v in reversed(half)] + half)


@functools.lru_cache(maxsize=None)
def _signs(d):
    """+-1 of every coordinate: bit 63 of the splitmix64 stream."""
    mask, state, out = (1 << 64) - 1, SEED, []
    for _ in range(d):
        state = (state + 0x9E3779B97F4A7C15) & mask
        z = state
        z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & mask
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & mask
        z ^= z >> 31
        out.append(-1.0 if z >> 63 else 1.0)
    return tuple(out)


@functools.lru_cache(maxsize=None)
def _rotation(d):
    """[d, d] float32: a row c of levels times this is D H c (entries +-1)."""
    h = np.ones((1, 1))
    while h.shape[0] < d:
        h = np.block([[h, h], [h, -h]])
    return torch.from_numpy(h * np.array(_signs(d))[None, :]).float()


def _unpack(packed, bits):
    """uint8 [..., P] -> int64 codes [..., 8 P / bits] of the little-endian bitstream."""
    n = packed.shape[-1] * 8 // bits
    off = torch.arange(n, device=packed.device) * bits
    wide = packed.to(torch.int32)
    nxt = torch.cat([wide[..., 1:], torch.zeros_like(wide[..., :1])], dim=-1)
    words = wide | (nxt << 8)
    return ((words[..., off >> 3] >> (off & 7).to(torch.int32)) & ((1 << bits) - 1)).long()


def _pack(codes, bits):
    """int codes [..., n] -> uint8 [..., n * bits / 8]."""
    per = 8 if bits == 3 else 8 // bits
    size = per * bits // 8
    c = codes.reshape(*codes.shape[:-1], -1, per).to(torch.int32)
    word = torch.zeros_like(c[..., 0])
    for k in range(per):
        word |= c[..., k] << (bits * k)
    parts = [((word >> (8 * k)) & 255).to(torch.uint8) for k in range(size)]
    return torch.stack(parts, dim=-1).reshape(*codes.shape[:-1], -1)


def _packed_rows(shape, d, bits, gen):
    """Packed codes of N(0,1) coordinates and norms near sqrt(d), as an encoder leaves them."""
    levels = torch.tensor(_levels(bits), device="cuda")
    bounds = (levels[1:] + levels[:-1]) / 2
    packed = torch.empty(*shape, d * bits // 8, dtype=torch.uint8, device="cuda")
    flat = packed.view(-1, packed.shape[-1])
    step = 1 << 19
    for i in range(0, flat.shape[0], step):
        n = min(step, flat.shape[0] - i)
        z = torch.randn(n, d, generator=gen, device="cuda")
        flat[i:i + n] = _pack(torch.bucketize(z, bounds, out_int32=True), bits)
    norms = math.sqrt(d) * torch.exp(0.2 * torch.randn(*shape, generator=gen, device="cuda"))
    return packed, norms


def _values(packed, norms, bits, d):
    """Decoded rows [..., d]: norm / d times D H of the levels."""
    levels = torch.tensor(_levels(bits), dtype=torch.float32, device=packed.device)
    rows = levels[_unpack(packed, bits)] @ _rotation(d).to(packed.device)
    return rows * (norms / d).unsqueeze(-1)


# ------------------------------------------------------------------ the cases


def listed():
    return [
        # the tokens of one decode step of a batch, straight from the projection
        {"name": "norm_rope decode 16", "op": "norm_rope", "t": 16, "hq": 32, "hkv": 8, "d": 128, "rot": 128,
         "interleaved": False, "norm": True, "bf16": False, "scale": 1.0, "far": 131072},
        # a prompt's projection from a bf16 model: part of the head rotated, pairs side by side, positions scaled
        {"name": "norm_rope prompt 8191", "op": "norm_rope", "t": 8191, "hq": 32, "hkv": 8, "d": 128, "rot": 64,
         "interleaved": True, "norm": True, "bf16": True, "scale": 1.1386, "far": 1048576},
        # one interactive sequence: the smallest step, where latency counts
        {"name": "window decode 1", "op": "window", "b": 1, "n": 1, "ctx": 1500, "window": 512, "sinks": 4, "hq": 32,
         "hkv": 8, "d": 128, "kb": 4, "vb": 2, "paged": True},
        # a served batch at long contexts
        {"name": "window decode 16 x 8192", "op": "window", "b": 16, "n": 1, "ctx": 32768, "window": 8192, "sinks": 16,
         "hq": 32, "hkv": 8, "d": 128, "kb": 4, "vb": 2, "paged": True},
        # drafted tokens verified together, whole context, contiguous caches at 4 bits
        {"name": "window verify 8 x 5", "op": "window", "b": 8, "n": 5, "ctx": 8000, "window": 0, "sinks": 0, "hq": 32,
         "hkv": 4, "d": 128, "kb": 4, "vb": 4, "paged": False},
        # a long prompt continued in chunks over what the cache holds already
        {"name": "window chunk 2 x 2048", "op": "window", "b": 2, "n": 2048, "ctx": 12000, "window": 4096, "sinks": 64,
         "hq": 32, "hkv": 8, "d": 128, "kb": 4, "vb": 2, "paged": True},
        # a few requests answered in two ways
        {"name": "fork 8", "op": "fork", "rows": 64, "mb": 256, "nb": 4096, "n": 8, "layers": 4, "hkv": 8, "d": 128,
         "kb": 4, "vb": 2},
        # beams of a batch split at one step, all layers
        {"name": "fork 256 beams", "op": "fork", "rows": 512, "mb": 128, "nb": 4096, "n": 256, "layers": 32, "hkv": 8,
         "d": 128, "kb": 4, "vb": 2},
        # pages behind the window given back after a step
        {"name": "trim 8", "op": "trim", "rows": 8, "mb": 64, "window": 256, "sinks": 4},
        {"name": "trim 512 x 2048", "op": "trim", "rows": 512, "mb": 2048, "window": 8192, "sinks": 64},
        # the pools of a small and of a large server brought together
        {"name": "compact 1024", "op": "compact", "rows": 64, "mb": 32, "nb": 1024, "used": 0.5, "layers": 2, "hkv": 4,
         "d": 64, "kb": 3, "vb": 3},
        {"name": "compact 8192", "op": "compact", "rows": 256, "mb": 128, "nb": 8192, "used": 0.6, "layers": 16,
         "hkv": 8, "d": 128, "kb": 4, "vb": 2},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope", "window", "window", "window", "fork", "trim", "compact"])
    d, kb, vb = rng.choice([64, 128, 128, 256]), rng.choice([2, 3, 4, 4]), rng.choice([2, 2, 3, 4])
    if op == "norm_rope":
        hkv = rng.randint(1, 8)
        hq = hkv * rng.randint(1, 8)
        t = min(_log(rng, 1, 8191), 8191 * 40 * 128 // ((hq + hkv) * d))
        return {"op": op, "t": t, "hq": hq, "hkv": hkv, "d": d,
                "rot": rng.choice([d, d, d // 2, d // 4, 2 * rng.randint(1, d // 2)]),
                "interleaved": rng.random() < 0.5, "norm": rng.random() < 0.7, "bf16": rng.random() < 0.5,
                "scale": rng.choice([1.0, 1.1386]), "far": _log(rng, 64, 1048576)}
    if op == "window":
        hkv, group = rng.choice([1, 2, 3, 4, 5, 8, 8]), rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 12])
        n = rng.choice([1, 1, rng.randint(2, 8), _log(rng, 8, 2048)])
        ctx = n + _log(rng, 1, 32768 if n == 1 else 12000)
        c = {"op": op, "b": _log(rng, 1, 32), "n": n, "ctx": ctx, "window": rng.choice([0, _log(rng, 16, 8192)]),
             "sinks": rng.choice([0, 1, 4, 16, rng.randint(2, 100)]), "hq": hkv * group, "hkv": hkv, "d": d, "kb": kb,
             "vb": vb, "paged": rng.random() < 0.6}
        most = work({**listed()[5]})["flops"]
        while c["b"] > 1 and (work(c)["flops"] > most / 2 or c["b"] * _span(c) * hkv * d > 1.3e8):
            c["b"] = c["b"] // 2
        while work(c)["flops"] > most or c["n"] * _span(c) * c["hq"] > 5e8:
            c["n"], c["ctx"] = max(1, c["n"] // 2), max(c["ctx"] - c["n"] // 2, c["ctx"] // 2, 2)
        return c
    if op == "fork":
        n, layers = _log(rng, 1, 256), _log(rng, 1, 32)
        mb = _log(rng, 4, 512)
        nb = 2 * n + _log(rng, 512, 4096 if d < 256 else 2048)
        return {"op": op, "rows": 2 * n + rng.randint(0, 40), "mb": mb, "nb": nb, "n": n, "layers": layers,
                "hkv": rng.choice([1, 2, 4, 8]), "d": d, "kb": kb, "vb": vb}
    if op == "trim":
        mb = _log(rng, 4, 2048)
        return {"op": op, "rows": _log(rng, 1, 512), "mb": mb, "window": _log(rng, 16, 16 * mb),
                "sinks": rng.randint(0, 70)}
    return {"op": op, "rows": _log(rng, 1, 256), "mb": _log(rng, 8, 128), "nb": _log(rng, 64, 8192),
            "used": round(rng.uniform(0.05, 0.95), 3), "layers": _log(rng, 1, 16 if d < 256 else 8),
            "hkv": rng.choice([1, 2, 4, 8]), "d": d, "kb": kb, "vb": vb}


def _lengths(c):
    """Query tokens and context length (they included) of every sequence: ragged, the first one the longest."""
    b = np.arange(c["b"])
    n = c["n"] - (b * 37) % (c["n"] // 3 + 1)
    ctx = np.maximum(c["ctx"] - (b * 531) % (c["ctx"] // 3 + 1), n)
    return n.astype(np.int64), ctx.astype(np.int64)


def _span(c):
    """Cache positions that the longest sequence's queries see together, at most."""
    return c["ctx"] if not c["window"] else min(c["ctx"], c["sinks"] + c["window"] + c["n"] - 1)


def work(case):
    c = case
    if c["op"] == "norm_rope":
        rows = c["t"] * (c["hq"] + c["hkv"])
        return {"bytes": rows * c["d"] * 4 + 4 * c["t"] + 8 * c["rot"], "flops": rows * c["d"] * 8}
    if c["op"] == "window":
        n, ctx = _lengths(c)
        far = c["window"] or 1 << 40
        seen = held = 0
        for m, length in zip(n.tolist(), ctx.tolist()):
            p = np.arange(length - m, length)
            lo = np.maximum(0, p - far + 1)
            seen += int((p + 1 - lo + np.minimum(c["sinks"], lo)).sum())
            held += int(length - lo[0] + min(c["sinks"], lo[0]))
        rows = held * c["hkv"]
        return {"bytes": rows * (c["d"] * (c["kb"] + c["vb"]) // 8 + 8) + int(n.sum()) * c["hq"] * c["d"] * 4,
                "flops": 4 * seen * c["hq"] * c["d"]}
    page = BLOCK * c["hkv"] * (c["d"] * (c["kb"] + c["vb"]) // 8 + 8) * c["layers"] if c["op"] != "trim" else 0
    if c["op"] == "fork":  # the last page of a parent is partly filled 15 times of 16
        return {"bytes": 2 * page * c["n"] * 15 // 16 + 8 * (c["rows"] * c["mb"] + c["nb"]), "flops": 0}
    if c["op"] == "trim":
        return {"bytes": 16 * c["rows"] * c["mb"] + 16 * c["rows"], "flops": 0}
    moved = int(c["nb"] * c["used"] * (1 - c["used"]))
    return {"bytes": 2 * page * moved + 8 * c["rows"] * c["mb"] + 12 * c["nb"], "flops": 0}


# ------------------------------------------------------------------ the inputs


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    if c["op"] == "norm_rope":
        return _prepare_norm_rope(c, gen)
    if c["op"] == "window":
        return _prepare_window(c, gen)
    return _prepare_pages(c, gen)


def _prepare_norm_rope(c, gen):
    t, hq, hkv, d = c["t"], c["hq"], c["hkv"], c["d"]
    kind = torch.bfloat16 if c["bf16"] else torch.float16
    # the projection's row holds queries, keys and values side by side; keys have a few large channels
    qkv = torch.randn(t, (hq + 2 * hkv) * d, generator=gen, device="cuda")
    qkv *= torch.exp(0.5 * torch.randn(1, qkv.shape[1], generator=gen, device="cuda"))
    qkv = qkv.to(kind)
    s = {"case": c, "qkv": qkv, "q": qkv[:, :hq * d].unflatten(1, (hq, d)),
         "k": qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)),
         "positions": torch.randint(0, c["far"], (t,), generator=gen, device="cuda", dtype=torch.int32),
         "inv_freq": 10000.0 ** (-torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64) / c["rot"]),
         "qw": None, "kw": None}
    if c["norm"]:
        s["qw"] = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(kind)
        s["kw"] = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(kind)
    return s


def _prepare_window(c, gen):
    n, ctx = _lengths(c)
    b, hkv, d = c["b"], c["hkv"], c["d"]
    starts = np.concatenate([[0], np.cumsum(n)])
    lo = np.maximum(0, ctx - n + 1 - c["window"]) if c["window"] else np.zeros_like(ctx)
    s = {"case": c, "q": (2 * torch.randn(int(starts[-1]), c["hq"], d, generator=gen, device="cuda")).half(),
         "offsets": torch.tensor(starts, dtype=torch.int32, device="cuda"),
         "ctx": torch.tensor(ctx, dtype=torch.int32, device="cuda"), "max_q": int(n.max()),
         "lo": torch.tensor(lo, device="cuda")}
    if c["paged"]:
        # pages scattered over the pool, those that no query sees given back already
        mb = -(-c["ctx"] // BLOCK)
        j = np.arange(mb)[None, :]
        kept = (j * BLOCK < ctx[:, None]) & ((j * BLOCK + BLOCK > lo[:, None]) | (j * BLOCK < c["sinks"]))
        count = int(kept.sum())
        nb = count + 3
        table = torch.full((b, mb), -1, dtype=torch.int32, device="cuda")
        table[torch.from_numpy(kept).cuda()] = torch.randperm(nb, generator=gen, device="cuda")[:count].int()
        s["table"] = table
        shape = (nb, BLOCK, hkv)
    else:
        shape = (b, c["ctx"], hkv)
    s["k"], s["kn"] = _packed_rows(shape, d, c["kb"], gen)
    s["v"], s["vn"] = _packed_rows(shape, d, c["vb"], gen)
    return s


def _prepare_pages(c, gen):
    rows, mb = c["rows"], c["mb"]
    s = {"case": c}
    if c["op"] == "trim":
        # full rows of distinct pages, a tenth of them shared by the next row; every sixteenth sequence has ended
        table = torch.randperm(rows * mb, generator=gen, device="cuda").view(rows, mb).int()
        shared = (torch.rand(rows, mb, generator=gen, device="cuda") < 0.1) & (torch.arange(rows, device="cuda")[:, None] > 0)
        s["table"] = torch.where(shared, table.roll(1, 0), table)
        s["lens"] = torch.randint(1, mb * BLOCK + 1, (rows,), generator=gen, device="cuda", dtype=torch.int32)
        s["release"] = torch.rand(rows, generator=gen, device="cuda") < 1 / 16
        s["refs"] = torch.zeros(rows * mb, dtype=torch.int32, device="cuda")
        s["refs"].index_add_(0, s["table"].flatten(), torch.ones_like(s["table"]).flatten())
        return s
    nb, lead = c["nb"], (c["layers"], c["nb"], BLOCK, c["hkv"])
    byte = lambda n: torch.randint(0, 256, (*lead, n), generator=gen, device="cuda", dtype=torch.uint8)  # noqa: E731
    s["pools"] = [byte(c["d"] * c["kb"] // 8), torch.randn(*lead, generator=gen, device="cuda"),
                  byte(c["d"] * c["vb"] // 8), torch.randn(*lead, generator=gen, device="cuda")]
    table = torch.full((rows, mb), -1, dtype=torch.int32, device="cuda")
    order = torch.randperm(nb, generator=gen, device="cuda").int()
    s["refs"] = torch.zeros(nb, dtype=torch.int32, device="cuda")
    if c["op"] == "fork":
        # the first n rows are parents of 1 to mb pages each, taken from a pool with room for the children
        n = c["n"]
        held = max(1, min(mb, (nb - n) // n))
        s["lens"] = torch.zeros(rows, dtype=torch.int32, device="cuda")
        s["lens"][:n] = torch.randint(1, held * BLOCK + 1, (n,), generator=gen, device="cuda", dtype=torch.int32)
        pages = (s["lens"][:n, None] + BLOCK - 1) // BLOCK
        mine = order[:n * held].view(n, held)
        mine = torch.where(torch.arange(held, device="cuda")[None] < pages, mine, torch.full_like(mine, -1))
        table[:n, :held] = mine
        s["parents"] = torch.randperm(n, generator=gen, device="cuda").int()
        s["children"] = n + torch.randperm(rows - n, generator=gen, device="cuda")[:n].int()
        s["refs"].index_add_(0, mine.clamp(min=0).flatten(), (mine >= 0).int().flatten())
    else:
        # used pages anywhere in the pool, listed by the rows in turn
        used = int(c["used"] * nb)
        some = order[:used]
        s["refs"][some.long()] = torch.randint(1, 4, (used,), generator=gen, device="cuda", dtype=torch.int32)
        k = min(used, rows * mb)
        table.view(-1)[torch.randperm(rows * mb, generator=gen, device="cuda")[:k]] = some[:k]
    s["table"] = table
    return s


# ------------------------------------------------------------------ one pass


def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


@functools.lru_cache(maxsize=None)
def _codec(d, bits):
    import kv_cache_vector_turboquant_b200 as tq

    return tq.TurboQuant(d, bits, SEED)


def _handle(s):
    """The pools' handle, which a program keeps beside its pools."""
    import kv_cache_vector_turboquant_b200 as tq

    if "handle" not in s:
        s["handle"] = tq.TQPagePools([layer for t in s["pools"] for layer in t.unbind(0)])
    return s["handle"]


def _own_norm_rope(s):
    import kv_cache_vector_turboquant_b200 as tq

    c = s["case"]
    return tq.qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], interleaved=c["interleaved"],
                           rope_scale=c["scale"], q_weight=s["qw"], k_weight=s["kw"], eps=1e-6)


def _own_window(s):
    import kv_cache_vector_turboquant_b200 as tq

    c = s["case"]
    kc, vc = _codec(c["d"], c["kb"]), _codec(c["d"], c["vb"])
    more = {"window": c["window"] or None, "sinks": c["sinks"]}
    if c["n"] > 1:
        more |= {"q_offsets": s["offsets"], "max_q": s["max_q"]}
    if c["paged"]:
        return tq.attend_window_paged(s["q"], kc, vc, s["k"], s["kn"], s["v"], s["vn"], s["table"], s["ctx"], **more)
    return tq.attend_window(s["q"], kc, vc, s["k"], s["kn"], s["v"], s["vn"], s["ctx"], **more)


def _own_fork(s):
    table, lens, refs = _handle(s).fork(s["table"], s["lens"], s["refs"], s["parents"], s["children"])
    return {"table": table, "lens": lens, "refs": refs, "pools": s["pools"]}


def _own_trim(s):
    import kv_cache_vector_turboquant_b200 as tq

    c = s["case"]
    table, lens, refs = tq.pages_trim(s["table"], s["lens"], s["refs"], window=c["window"], sinks=c["sinks"],
                                      release=s["release"])
    return {"table": table, "lens": lens, "refs": refs}


def _own_compact(s):
    table, refs, remap, used = _handle(s).compact(s["table"], s["refs"])
    return {"table": table, "refs": refs, "remap": remap, "used": used, "pools": s["pools"]}


def _plain_norm_rope(s):
    c = s["case"]
    angle = s["positions"].double()[:, None, None] * s["inv_freq"]
    cos, sin = (angle.cos() * c["scale"]).float(), (angle.sin() * c["scale"]).float()
    return tuple(_plain_head(x, w, cos, sin, c) for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])))


def _plain_head(x, weight, cos, sin, c):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + 1e-6) * weight.float()
    rot = c["rot"]
    turned, rest = x[..., :rot], x[..., rot:]
    if c["interleaved"]:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = turned[..., :rot // 2], turned[..., rot // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, rest], dim=-1).half()


def _plain_window(s):
    """Gathers the positions that each sequence's queries may see, decodes them and attends under a mask."""
    c = s["case"]
    d, hkv, b, n = c["d"], c["hkv"], c["b"], s["max_q"]
    dev = s["q"].device
    ctx, lo = s["ctx"].long()[:, None], s["lo"][:, None]
    u = torch.arange(_span(c), device=dev)[None]
    first = torch.clamp(lo, min=c["sinks"])  # the window's part begins behind the sinks
    t = torch.where(u < c["sinks"], u, first + u - c["sinks"])  # [b, span]
    held = t < ctx
    t = torch.where(held, t, torch.zeros_like(t))
    if c["paged"]:
        row = torch.gather(s["table"].long(), 1, t // BLOCK).clamp(min=0) * BLOCK + t % BLOCK
    else:
        row = torch.arange(b, device=dev)[:, None] * c["ctx"] + t
    k = _values(s["k"].flatten(0, 1)[row], s["kn"].flatten(0, 1)[row], c["kb"], d)
    v = _values(s["v"].flatten(0, 1)[row], s["vn"].flatten(0, 1)[row], c["vb"], d)
    # queries padded to the longest sequence
    count = (s["offsets"][1:] - s["offsets"][:-1]).long()[:, None]
    i = torch.arange(n, device=dev)[None]
    at = torch.clamp(s["offsets"][:-1].long()[:, None] + i, max=s["q"].shape[0] - 1)
    q = s["q"][at].float().view(b, n, hkv, c["hq"] // hkv, d)
    place = (ctx - count + i)[:, :, None]  # [b, n, 1]
    seen = held[:, None] & (t[:, None] <= place)
    if c["window"]:
        seen &= (t[:, None] > place - c["window"]) | (t[:, None] < c["sinks"])
    score = q.permute(0, 2, 3, 1, 4).flatten(2, 3) @ k.permute(0, 2, 3, 1) / math.sqrt(d)  # [b, hkv, g n, span]
    score = score.unflatten(2, (-1, n)).masked_fill(~seen[:, None, None], -math.inf)
    top = score.amax(dim=-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(score - top)
    total = p.sum(dim=-1, keepdim=True)
    o = p.flatten(2, 3) @ v.permute(0, 2, 1, 3)
    o = o.unflatten(2, (-1, n)) / torch.where(total > 0, total, torch.ones_like(total))
    o = o.permute(0, 3, 1, 2, 4).reshape(b, n, c["hq"], d)
    token = torch.arange(s["q"].shape[0], device=dev)
    seq = torch.searchsorted(s["offsets"][1:].contiguous(), token, right=True)
    return o[seq, token - s["offsets"][seq].long()].half()


def _plain_fork(s):
    table, lens, refs = s["table"].clone(), s["lens"].clone(), s["refs"].clone()
    parents, children = s["parents"].long(), s["children"].long()
    length = s["lens"][parents].long()
    whole, ragged = length // BLOCK, length % BLOCK > 0
    mine = s["table"][parents].long()
    j = torch.arange(mine.shape[1], device=mine.device)[None]
    # the lowest free pages, one for each child whose last page is partly filled
    free = torch.cumsum((s["refs"] == 0).int(), 0)
    fresh = torch.searchsorted(free, torch.cumsum(ragged.int(), 0).to(free.dtype))
    shared = (j < whole[:, None]) & (mine >= 0)
    last = torch.gather(mine, 1, whole.clamp(max=mine.shape[1] - 1)[:, None])[:, 0]
    refs.index_add_(0, torch.where(shared, mine, 0).flatten(), shared.int().flatten())
    # a child without a partly filled page copies its own first page onto itself and counts nothing
    source = torch.where(ragged, last, mine[:, 0])
    target = torch.where(ragged, fresh, mine[:, 0])
    refs.index_add_(0, target, ragged.int())
    entry = torch.where(shared, mine, torch.where((j == whole[:, None]) & ragged[:, None], fresh[:, None], -1))
    table[children] = entry.int()
    lens[children] = length.int()
    for pool in s["pools"]:
        pool[:, target] = pool[:, source]
    return {"table": table, "lens": lens, "refs": refs, "pools": s["pools"]}


def _plain_trim(s):
    c = s["case"]
    length = s["lens"].long()[:, None]
    first = torch.arange(c["mb"], device=length.device)[None] * BLOCK
    gone = (first >= c["sinks"]) & (first + BLOCK <= length - c["window"]) | s["release"][:, None]
    gone &= s["table"] >= 0
    refs = s["refs"].clone()
    refs.index_add_(0, torch.where(gone, s["table"], 0).flatten(), -gone.int().flatten())
    return {"table": torch.where(gone, -1, s["table"]), "lens": torch.where(s["release"], 0, s["lens"]), "refs": refs}


def _plain_compact(s):
    refs = s["refs"]
    used = refs > 0
    page = torch.arange(refs.numel(), device=refs.device)
    count = used.sum()
    source = torch.nonzero(used & (page >= count))[:, 0]
    target = torch.nonzero(~used & (page < count))[:, 0]
    remap = torch.where(used, page, -1).int()
    remap[source] = target.int()
    packed = torch.where(page < count, refs, 0)
    packed[target] = refs[source]
    table = torch.where(s["table"] >= 0, remap[s["table"].clamp(min=0).long()], -1)
    for pool in s["pools"]:
        pool[:, target] = pool[:, source]
    return {"table": table, "refs": packed, "remap": remap, "used": count.int().view(1), "pools": s["pools"]}


_OWN = {"norm_rope": _own_norm_rope, "window": _own_window, "fork": _own_fork, "trim": _own_trim,
        "compact": _own_compact}
_PLAIN = {"norm_rope": _plain_norm_rope, "window": _plain_window, "fork": _plain_fork, "trim": _plain_trim,
          "compact": _plain_compact}


# ------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    """The operators' results in 64 bits; the pages' are whole numbers and copies, which have no other value."""
    if case["op"] == "norm_rope":
        return _exact_norm_rope(prepare(case, seed))
    if case["op"] == "window":
        return _exact_window(prepare(case, seed))
    return None


def _exact_norm_rope(s):
    c = s["case"]
    half = c["rot"] // 2
    turn = torch.polar(torch.full((c["t"], half), c["scale"], dtype=torch.float64, device="cuda"),
                       s["positions"].double()[:, None] * s["inv_freq"][None])
    i = torch.arange(half, device="cuda")
    a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
    out = []
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        y = x.double().clone()
        if w is not None:
            y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / c["d"] + 1e-6) * w.double()
        z = torch.complex(y[..., a], y[..., b]) * turn[:, None]
        y[..., a], y[..., b] = z.real, z.imag
        out.append(y)
    return tuple(out)


def _exact_rows(packed, norms, bits, d):
    """Decoded rows from the bitstream's single bits, by butterflies."""
    stream = (packed.unsqueeze(-1) >> torch.arange(8, device="cuda", dtype=torch.uint8)) & 1
    code = (stream.reshape(*packed.shape[:-1], d, bits).long() << torch.arange(bits, device="cuda")).sum(-1)
    x = torch.tensor(_levels(bits), dtype=torch.float64, device="cuda")[code]
    h = 1
    while h < d:
        pair = x.unflatten(-1, (d // (2 * h), 2, h))
        a, b = pair[..., 0, :], pair[..., 1, :]
        x = torch.stack([a + b, a - b], dim=-2).flatten(-3)
        h *= 2
    sign = torch.tensor(_signs(d), dtype=torch.float64, device="cuda")
    return norms.double().unsqueeze(-1) / math.sqrt(d) * (sign * x / math.sqrt(d))


def _exact_window(s):
    """One sequence and kv head after another, over every cached position, masked by the definition."""
    c = s["case"]
    d, hkv, g = c["d"], c["hkv"], c["hq"] // c["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    offsets, ctx = s["offsets"].tolist(), s["ctx"].tolist()
    for b in range(c["b"]):
        n, length = offsets[b + 1] - offsets[b], ctx[b]
        t = torch.arange(length, device="cuda")
        p = torch.arange(length - n, length, device="cuda")[:, None]
        seen = t[None] <= p
        if c["window"]:
            seen &= (p - t[None] < c["window"]) | (t[None] < c["sinks"])
        near = seen.any(0).nonzero()[:, 0]
        t, seen = t[near], seen[:, near]
        if c["paged"]:
            page = s["table"][b].long()[t // BLOCK]
            pick = lambda x: x[page, t % BLOCK]  # noqa: E731
        else:
            pick = lambda x: x[b, t]  # noqa: E731
        k = _exact_rows(pick(s["k"]), pick(s["kn"]), c["kb"], d)
        v = _exact_rows(pick(s["v"]), pick(s["vn"]), c["vb"], d)
        for h in range(hkv):
            q = s["q"][offsets[b]:offsets[b + 1], h * g:(h + 1) * g].double()
            score = torch.einsum("igd,td->git", q, k[:, h]) / math.sqrt(d)
            p_ = torch.softmax(score.masked_fill(~seen[None], -math.inf), dim=-1)
            out[offsets[b]:offsets[b + 1], h * g:(h + 1) * g] = torch.einsum("git,td->igd", p_, v[:, h])
    return out
