"""Operators around the compressed KV cache, as cases to be timed and compared.

Four operators that a speculative decoding step over the cache is made of:

* ``rope``   rotary positions applied to a step's queries and keys, the keys
             and values quantised into the cache as they are rotated.  What the
             cache then holds is read back, as the values it stands for.
* ``tree``   attention of a tree of drafted tokens over the cache: every draft
             sees the sequence before the tree and its own ancestors.
* ``commit`` the accepted path of the tree moved to the front of the drafted
             slots, in every layer, and the sequence lengths advanced.
* ``read``   ranges of the cache of several sequences read back in 16 or 32 bits.

The cache is the library's: per vector an fp16 norm and 2-, 3- or 4-bit codes of
the rotated direction (LSB-first), optionally with a 1-bit sketch of the keys'
residual, or (written as 8 bits below) an fp16 scale and int8 values.
Contiguous caches are ``[batch][kv head][slot]``; paged ones are a pool of
blocks with a table.  With ``own`` false everything is elementary torch
operations in 32 bits; with ``own`` true ``run`` calls the library.
"""

import functools
import math

import numpy as np
import torch

own = False

SIGN_SEED = 11  # selects the layer's rotation signs
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DRAFTS_MOST = 64


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the new token of one sequence deep in a long context: the smallest call, launch latency
        {"name": "rope one token", "op": "rope", "batch": 1, "tokens": 1, "hq": 32, "hkv": 8, "d": 128, "kb": 4,
         "vb": 2, "qjl": 0, "page": 0, "rotary": 128, "layout": "half", "scaling": "none", "first": 121007,
         "dtype": "bf16"},
        # drafted tokens of a serving batch into pages; half of each head is rotated
        {"name": "rope drafts paged", "op": "rope", "batch": 16, "tokens": 29, "hq": 32, "hkv": 8, "d": 128, "kb": 4,
         "vb": 4, "qjl": 0, "page": 64, "rotary": 64, "layout": "interleaved", "scaling": "wavelength",
         "first": 40000, "dtype": "fp16"},
        # a long prompt written in one call
        {"name": "rope prompt", "op": "rope", "batch": 1, "tokens": 8192, "hq": 32, "hkv": 8, "d": 128, "kb": 4,
         "vb": 3, "qjl": 0, "page": 0, "rotary": 128, "layout": "half", "scaling": "ramp", "first": 0,
         "dtype": "bf16"},
        # a chat turn with a short history and a small tree
        {"name": "tree short", "op": "tree", "batch": 1, "drafts": 8, "hq": 32, "hkv": 8, "d": 128, "kb": 4, "vb": 2,
         "qjl": 0, "page": 0, "lo": 1001, "hi": 1001, "dtype": "bf16"},
        # a ragged serving batch read through pages
        {"name": "tree batch paged", "op": "tree", "batch": 16, "drafts": 13, "hq": 32, "hkv": 8, "d": 128, "kb": 3,
         "vb": 2, "qjl": 0, "page": 64, "lo": 2048, "hi": 8192, "dtype": "bf16"},
        # the largest tree after a long context
        {"name": "tree wide 32k", "op": "tree", "batch": 1, "drafts": 64, "hq": 32, "hkv": 8, "d": 128, "kb": 4,
         "vb": 2, "qjl": 0, "page": 0, "lo": 32768, "hi": 32768, "dtype": "bf16"},
        # the longest contexts, eight query heads to a kv head
        {"name": "tree 128k", "op": "tree", "batch": 2, "drafts": 25, "hq": 64, "hkv": 8, "d": 128, "kb": 4, "vb": 4,
         "qjl": 0, "page": 0, "lo": 131003, "hi": 131072, "dtype": "fp16"},
        # a layer kept in 8 bits, narrow heads
        {"name": "tree int8 d64", "op": "tree", "batch": 4, "drafts": 17, "hq": 16, "hkv": 4, "d": 64, "kb": 8,
         "vb": 8, "qjl": 0, "page": 0, "lo": 777, "hi": 4001, "dtype": "bf16"},
        # three accepted tokens of one sequence in every layer
        {"name": "commit one", "op": "commit", "layers": 32, "batch": 1, "drafts": 8, "hkv": 8, "d": 128, "kb": 4,
         "vb": 2, "qjl": 0, "page": 0, "capacity": 512},
        # a large serving batch
        {"name": "commit batch", "op": "commit", "layers": 32, "batch": 48, "drafts": 64, "hkv": 8, "d": 128,
         "kb": 4, "vb": 3, "qjl": 0, "page": 0, "capacity": 200},
        # the tail of a conversation handed to another worker
        {"name": "read tail", "op": "read", "batch": 3, "lo": 1, "hi": 187, "hkv": 8, "d": 128, "kb": 4, "vb": 2,
         "qjl": 0, "page": 16, "dtype": "bf16"},
        # a whole context expanded once
        {"name": "read context", "op": "read", "batch": 2, "lo": 32001, "hi": 32768, "hkv": 8, "d": 128, "kb": 4,
         "vb": 2, "qjl": 0, "page": 0, "dtype": "bf16"},
    ]


def _between(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "tree", "tree", "tree", "commit", "read"])
    d = rng.choice([64, 128, 128, 128, 256])
    hkv = rng.choice([1, 2, 4, 8, 8])
    kb, vb = rng.choice([(4, 2), (4, 4), (3, 2), (3, 3), (4, 3), (2, 2), (2, 4), (8, 2), (8, 8), (4, 8)])
    qjl = rng.choice([0, 0, 0, 32, 64]) if kb < 8 else 0
    page = rng.choice([0, 0, 16, 48, 64, 256])
    c = {"op": op, "hkv": hkv, "d": d, "kb": kb, "vb": vb, "qjl": qjl, "page": page}
    if op == "commit":
        c["layers"] = _between(rng, 1, 32)
        c["batch"] = _between(rng, 1, 48)
        c["drafts"] = _between(rng, 1, DRAFTS_MOST)
        c["capacity"] = c["drafts"] + _between(rng, 1, 100)
        c["hkv"], c["d"] = min(hkv, 8), min(d, 128)
        return c
    c["hq"] = hkv * rng.choice([1, 2, 4, 4, 8, 16 if hkv <= 4 else 5])
    c["dtype"] = rng.choice(["bf16", "bf16", "fp16"])
    if op == "rope":
        c["batch"] = _between(rng, 1, 24)
        c["tokens"] = _between(rng, 1, max(1, 8192 * 48 * 128 // (c["batch"] * (c["hq"] + 2 * hkv) * d * 2)))
        c["tokens"] = min(c["tokens"], 8192)
        c["rotary"] = rng.choice([d, d, d // 2, d // 4, 2 * rng.randint(1, d // 2)])
        c["layout"] = rng.choice(["half", "interleaved"])
        c["scaling"] = rng.choice(["none", "linear", "base", "wavelength", "ramp"])
        c["first"] = _between(rng, 1, 500000) - 1
        c["dtype"] = rng.choice(["bf16", "fp16", "fp32"])
    elif op == "tree":
        if qjl or d != 128 or (vb == 8 and kb < 8):  # layers outside the usual serving shape: shorter contexts
            most = 6000
        else:
            most = 60000
        c["batch"] = _between(rng, 1, 12)
        c["drafts"] = _between(rng, 1, DRAFTS_MOST)
        c["hi"] = _between(rng, 1, max(1, most // c["batch"]))
        c["lo"] = rng.choice([c["hi"], max(0, c["hi"] // 3), 0])
    else:
        c["batch"] = _between(rng, 1, 12)
        c["hi"] = _between(rng, 1, max(1, 30000 // c["batch"]))
        c["lo"] = rng.choice([c["hi"], c["hi"] // 2, 0])
        c["dtype"] = rng.choice(["bf16", "fp16", "fp32"])
    return c


def _spread(lo, hi, n):
    """n lengths from lo to hi, the same for every seed."""
    return [hi - (hi - lo) * i // max(1, n - 1) if n > 1 else hi for i in range(n)]


def _path_lens(case):
    """Accepted drafts per sequence: none of them, a few, or all."""
    n = case["drafts"]
    return [min(n, (3 + 5 * b) % (n + 1)) for b in range(case["batch"])]


def _row_bytes(d, bits):
    return d if bits == 8 else d * bits // 8


def _vector_bytes(case):
    """Bytes of one cached token of one kv head: codes, norms, sketch and residual norm."""
    return _row_bytes(case["d"], case["kb"]) + _row_bytes(case["d"], case["vb"]) + 4 + (
        case["qjl"] // 8 + 2 if case["qjl"] else 0)


def work(case):
    d, hkv = case["d"], case["hkv"]
    vec = _vector_bytes(case)
    if case["op"] == "rope":
        tokens, size = case["batch"] * case["tokens"], 4 if case["dtype"] == "fp32" else 2
        moved = tokens * d * size * (2 * case["hq"] + 2 * hkv)  # q in and out, k and v in
        moved += tokens * hkv * (vec + 2 * 2 * d)                # the cache written; K and V read back in bf16
        log = int(math.log2(d))
        sketch = 4 * case["qjl"] * d
        flops = tokens * (3 * case["rotary"] * (case["hq"] + hkv) + hkv * (4 * d * log + 8 * d + sketch))
        return {"bytes": moved, "flops": flops}
    if case["op"] == "tree":
        lens, n = _spread(case["lo"], case["hi"], case["batch"]), case["drafts"]
        keys = sum(x + n for x in lens)
        moved = keys * hkv * vec + 2 * 2 * case["batch"] * n * case["hq"] * d + 8 * case["batch"] * n
        pairs = sum(n * x + n * (n + 1) // 4 for x in lens) * case["hq"]
        return {"bytes": moved, "flops": 4 * d * pairs}
    if case["op"] == "commit":
        rows = sum(_path_lens(case)) * case["layers"] * hkv
        return {"bytes": 2 * rows * vec + 4 * case["batch"] * (case["drafts"] + 3), "flops": 0}
    lens, size = _spread(case["lo"], case["hi"], case["batch"]), 4 if case["dtype"] == "fp32" else 2
    rows = sum(lens) * hkv
    log = int(math.log2(d))
    return {"bytes": rows * (vec + 2 * d * size), "flops": rows * (2 * d * (log + 3) + 2 * case["qjl"] * d)}


# ------------------------------------------------------- tables of the method
@functools.lru_cache(maxsize=None)
def _codebook(d, bits):
    """(centroids, boundaries) of the optimal scalar quantiser of one coordinate of a random unit vector, density
    proportional to (1 - x^2)^((d - 3) / 2): each centroid the mean of its cell, each boundary a midpoint."""
    n = 1 << bits
    node, weight = np.polynomial.legendre.leggauss(160)
    c = (np.arange(n // 2) + 0.5) * min(1.0, 3.0 / math.sqrt(d)) / (n // 2)  # the half above zero
    end = min(1.0, 14.0 / math.sqrt(d))  # (the density beyond it is below 1e-40 of its peak)
    for _ in range(20000):
        edge = np.concatenate([[0.0], 0.5 * (c[1:] + c[:-1]), [end]])
        half = 0.5 * (edge[1:] - edge[:-1])[:, None]
        x = 0.5 * (edge[1:] + edge[:-1])[:, None] + half * node
        f = np.exp(0.5 * (d - 3) * np.log1p(-np.minimum(x * x, 1.0 - 1e-16))) * weight
        new = (f * x).sum(1) / f.sum(1)
        moved, c = np.abs(new - c).max(), new
        if moved < 1e-16:
            break
    c = np.concatenate([-c[::-1], c])
    return c, 0.5 * (c[1:] + c[:-1])


@functools.lru_cache(maxsize=None)
def _signs(d):
    """The rotation's signs: -1 where the top bit of the i-th output of the SplitMix64 generator is set."""
    out, state, mask = [], SIGN_SEED, (1 << 64) - 1
    for _ in range(d):
        state = (state + 0x9E3779B97F4A7C15) & mask
        z = state
        z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & mask
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & mask
        out.append(-1.0 if (z ^ (z >> 31)) >> 63 else 1.0)
    return np.array(out)


@functools.lru_cache(maxsize=None)
def _hadamard(d):
    h = np.ones((1, 1))
    while h.shape[0] < d:
        h = np.block([[h, h], [h, -h]])
    return h


ROPE_BASE = 500000.0
ROPE_FACTOR, ROPE_LOW, ROPE_HIGH, ROPE_TRAINED = 8.0, 1.0, 4.0, 8192.0
RAMP_SLOW, RAMP_FAST = 1.0, 32.0


@functools.lru_cache(maxsize=None)
def _frequencies(rotary, scaling):
    """(radians a position turns each pair, factor on the rotated coordinates)."""
    i = np.arange(rotary // 2, dtype=np.float64)
    base = ROPE_BASE
    if scaling == "base" and rotary > 2:
        base *= ROPE_FACTOR ** (rotary / (rotary - 2.0))
    f = base ** (-2.0 * i / rotary)
    if scaling == "linear":
        f = f / ROPE_FACTOR
    if scaling == "wavelength":
        turns = ROPE_TRAINED * f / (2 * math.pi)  # whole turns within the trained length
        s = np.clip((turns - ROPE_LOW) / (ROPE_HIGH - ROPE_LOW), 0.0, 1.0)
        f = (1 - s) * f / ROPE_FACTOR + s * f
    if scaling == "ramp":
        at = [rotary * math.log(ROPE_TRAINED / (2 * math.pi * b)) / (2 * math.log(ROPE_BASE))
              for b in (RAMP_FAST, RAMP_SLOW)]
        lo, hi = max(0, math.floor(at[0])), min(rotary - 1, math.ceil(at[1]))
        s = np.clip((i - lo) / max(hi - lo, 0.001), 0.0, 1.0)
        return f / ROPE_FACTOR * s + f * (1 - s), 0.1 * math.log(ROPE_FACTOR) + 1.0
    return f, 1.0


# ----------------------------------------------------------------- the inputs
def _vectors(g, shape, spread=1.0):
    """N(0, 1) times a log-normal scale of each (head, channel)."""
    w = spread * torch.randn(shape[-2:], generator=g, device="cuda")
    return torch.randn(shape, generator=g, device="cuda") * torch.exp(w)


def _tables(case):
    def dev(a):
        return torch.tensor(np.array(a, dtype=np.float32), device="cuda")

    t = {"signs": dev(_signs(case["d"])), "had": dev(_hadamard(case["d"]) / math.sqrt(case["d"]))}
    for side, bits in (("k", case["kb"]), ("v", case["vb"])):
        if bits < 8:
            c, b = _codebook(case["d"], bits)
            t[side + "c"], t[side + "b"] = dev(c), dev(b)
    return t


def _cache(case, units, capacity, lead=()):
    """Arrays of a cache of `units` sequences (or blocks) of `capacity` slots."""
    def z(*tail, dtype=torch.uint8):
        return torch.zeros(lead + (units, case["hkv"], capacity) + tail, dtype=dtype, device="cuda")

    c = {"kc": z(_row_bytes(case["d"], case["kb"])), "kn": z(dtype=torch.float16),
         "vc": z(_row_bytes(case["d"], case["vb"])), "vn": z(dtype=torch.float16)}
    if case["qjl"]:
        c["kq"], c["kg"] = z(case["qjl"] // 8), z(dtype=torch.float16)
    return c


def _paged(case, slots, g):
    """(units, capacity, table or None): room for `slots` tokens of every sequence; pages in random order."""
    if not case["page"]:
        return case["batch"], slots, None
    blocks = -(-slots // case["page"])
    order = torch.randperm(case["batch"] * blocks + 3, generator=g, device="cuda")[: case["batch"] * blocks]
    return case["batch"] * blocks + 3, case["page"], order.view(case["batch"], blocks).to(torch.int32)


@functools.lru_cache(maxsize=None)
def _book(d, bits):
    """A codebook of the library: a program makes it once, for all its layers and inputs."""
    from bit_kv_cache_tq_b200 import tq

    return tq.tq_codebook_init(d, bits)


def _handles(case, cache, table):
    """What a user's program keeps of the library's: parameters, codebooks, the cache and the error word."""
    from bit_kv_cache_tq_b200 import tq

    modes = [tq.TQ_MODE_INT8 if b == 8 else tq.TQ_MODE_TURBO for b in (case["kb"], case["vb"])]
    bits = [4 if b == 8 else b for b in (case["kb"], case["vb"])]
    p = tq.make_params(case["d"], case.get("hq", case["hkv"]), case["hkv"], bits[0], bits[1], modes[0], modes[1],
                       case["qjl"], SIGN_SEED)
    books = [_book(case["d"], b) if b < 8 else None for b in (case["kb"], case["vb"])]
    return {"tq": tq, "p": p, "kcb": books[0], "vcb": books[1], "table": table,
            "err": torch.zeros(1, dtype=torch.int32, device="cuda")}


def _cache_tensors(tq, cache, sketch, layer=None):
    a = {k: (v if layer is None else v[layer]) for k, v in cache.items()}
    units, _, capacity = a["kn"].shape
    i16 = {k: a[k].view(torch.int16) for k in ("kn", "vn", "kg") if k in a}
    return tq.CacheTensors(units, capacity, a["kc"], i16["kn"], a.get("kq"), i16.get("kg"), a["vc"], i16["vn"],
                           sketch)


def _fill(case, cache, table, tables, sketch, tokens, g):
    """Quantise random keys and values into slots 0 .. tokens - 1 of every sequence, some sequences at a time."""
    most = max(1, (1 << 18) // max(1, case["batch"] * case["hkv"]))
    for at in range(0, tokens, most):
        n = min(most, tokens - at)
        where = _slots(cache, table, torch.full((case["batch"],), at, device="cuda"), n)
        for side in ("k", "v"):
            x = _vectors(g, (case["batch"], n, case["hkv"], case["d"]))
            _store(cache, side, where, _encode(case, tables, side, x, sketch))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    tables = _tables(case)
    s = {"case": case, "tables": tables, "sketch": None}
    op, batch, d = case["op"], case["batch"], case["d"]
    if case["qjl"]:
        s["sketch"] = torch.randn(case["qjl"], d, generator=g, device="cuda")
    if op == "commit":
        units, capacity, table = _paged(case, case["capacity"], g)
        cache = _cache(case, units, capacity, (case["layers"],))
        for name, a in cache.items():
            a.view(torch.uint8).random_(0, 256, generator=g)
        n = case["drafts"]
        room = case["capacity"] - n
        s["base"] = torch.randint(0, room + 1, (batch,), generator=g, device="cuda").to(torch.int32)
        s["path_lens"] = torch.tensor(_path_lens(case), dtype=torch.int32, device="cuda")
        # an accepted path: distinct drafts in ascending order
        pick = torch.rand(batch, n, generator=g, device="cuda").argsort(1)
        pick = torch.where(torch.arange(n, device="cuda")[None] < s["path_lens"][:, None], pick, n)
        s["path"] = torch.where(pick.sort(1).values < n, pick.sort(1).values, 0).to(torch.int32)
        s["new_lens"] = torch.zeros(batch, dtype=torch.int32, device="cuda")
        s |= {"cache": cache, "table": table}
        if own:
            h = _handles(case, cache, table)
            h["layers"] = h["tq"].draft_layers(
                [(h["p"], _cache_tensors(h["tq"], cache, s["sketch"], i)) for i in range(case["layers"])])
            s["h"] = h
        return s
    if op == "rope":
        n = case["tokens"]
        slots = n + 37
        units, capacity, table = _paged(case, slots, g)
        cache = _cache(case, units, capacity)
        s["q"] = torch.randn(batch, n, case["hq"], d, generator=g, device="cuda").to(DTYPES[case["dtype"]])
        # (half the spread of a cache's history: where one channel of a narrow head outweighs the rest, all its rotated
        # coordinates lie at one distance from a code's border, and any rounding moves them all)
        s["k"] = _vectors(g, (batch, n, case["hkv"], d), 0.5).to(DTYPES[case["dtype"]])
        s["v"] = _vectors(g, (batch, n, case["hkv"], d), 0.5).to(DTYPES[case["dtype"]])
        # slots in a window of the cache; positions as of a context that began far earlier, one depth of a tree
        # holding several of them
        s["at"] = torch.randint(0, slots - n + 1, (batch,), generator=g, device="cuda").to(torch.int32)
        step = torch.arange(n, device="cuda")[None] if n > 64 else torch.randint(
            0, n, (batch, n), generator=g, device="cuda").sort(1).values
        start = torch.randint(0, 1000, (batch, 1), generator=g, device="cuda") + case["first"]
        s["positions"] = (start + step).to(torch.int32).contiguous()
        f, factor = _frequencies(case["rotary"], case["scaling"])
        s["freq"], s["factor"] = torch.tensor(f, device="cuda"), factor
        s["q_out"] = torch.empty_like(s["q"])
        s["counts"] = torch.full((batch,), n, dtype=torch.int32, device="cuda")
        s["out"] = [torch.empty(batch, n, case["hkv"], d, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    elif op == "tree":
        n = case["drafts"]
        lens = _spread(case["lo"], case["hi"], batch)
        units, capacity, table = _paged(case, case["hi"] + n + 5, g)
        cache = _cache(case, units, capacity)
        s["base"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["q"] = torch.randn(batch, n, case["hq"], d, generator=g, device="cuda").to(DTYPES[case["dtype"]])
        s["mask"] = _trees(batch, n, g)
        s["out_buf"] = torch.empty_like(s["q"])
    else:
        lens = _spread(case["lo"], case["hi"], batch)
        units, capacity, table = _paged(case, case["hi"] + 40, g)
        cache = _cache(case, units, capacity)
        s["at"] = torch.randint(0, 41, (batch,), generator=g, device="cuda").to(torch.int32)
        s["counts"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["out"] = [torch.zeros(batch, case["hi"], case["hkv"], d, dtype=DTYPES[case["dtype"]], device="cuda")
                    for _ in "kv"]
    if op != "rope":
        _fill(case, cache, table, tables, s["sketch"], case["hi"] + (case["drafts"] if op == "tree" else 40), g)
    s |= {"cache": cache, "table": table}
    if own:
        h = _handles(case, cache, table)
        tq = h["tq"]
        h["cache"] = _cache_tensors(tq, cache, s["sketch"])
        if op == "rope":
            kind = {"none": tq.TQ_ROPE_SCALE_NONE, "linear": tq.TQ_ROPE_SCALE_LINEAR, "base": tq.TQ_ROPE_SCALE_BASE,
                    "wavelength": tq.TQ_ROPE_SCALE_WAVELENGTH, "ramp": tq.TQ_ROPE_SCALE_RAMP}[case["scaling"]]
            low, high = (RAMP_SLOW, RAMP_FAST) if case["scaling"] == "ramp" else (ROPE_LOW, ROPE_HIGH)
            h["rope"] = tq.tq_rope_init(
                case["rotary"], tq.TQ_ROPE_HALF if case["layout"] == "half" else tq.TQ_ROPE_INTERLEAVED, ROPE_BASE,
                scaling=kind, factor=ROPE_FACTOR, low=low, high=high, trained_len=ROPE_TRAINED)
        if op == "tree":
            h["ws"] = torch.zeros(max(16, tq.tq_tree_workspace_bytes(h["p"], batch, case["drafts"])),
                                  dtype=torch.uint8, device="cuda")
        s["h"] = h
    return s


def _trees(batch, n, g):
    """A random tree per sequence, a 64-bit mask per draft: its ancestors and itself."""
    chance = torch.rand(batch, n, generator=g, device="cuda")
    parent = (chance * (torch.arange(n, device="cuda")[None] + 1)).long() - 1  # -1: a child of the last token
    parent = torch.minimum(parent, torch.arange(n, device="cuda")[None] - 1)
    seen = torch.zeros(batch, n + 1, dtype=torch.int64, device="cuda")  # the last column: no draft
    rows = torch.arange(batch, device="cuda")
    for t in range(n):
        bit = 1 << t if t < 63 else -(1 << 63)
        seen[:, t] = seen[rows, torch.where(parent[:, t] < 0, n, parent[:, t])] | bit
    return seen[:, :n].contiguous()


# ------------------------------------------------------------- the plain form
def _slots(cache, table, first, n):
    """Indexes (unit, slot), each [batch, n], of tokens first[b] .. first[b] + n - 1 of every sequence; those past the
    end of the cache's room are clamped to it."""
    capacity = cache["kn"].shape[-1]
    at = first.long()[:, None] + torch.arange(n, device="cuda")[None]
    return _units(table, capacity, at)


def _units(table, capacity, at):
    rows = torch.arange(at.shape[0], device="cuda")[:, None]
    if table is None:
        return rows.expand_as(at), at.clamp(0, capacity - 1)
    at = at.clamp(0, capacity * table.shape[1] - 1)
    return table.long()[rows, at // capacity], at % capacity


def _pack(codes, bits):
    """[..., d] codes to [..., d bits / 8] bytes, least significant bit first."""
    eight = codes.view(*codes.shape[:-1], -1, 8)
    word = (eight << (bits * torch.arange(8, device="cuda"))).sum(-1)
    byte = (word[..., None] >> (8 * torch.arange(bits, device="cuda"))) & 255
    return byte.flatten(-2).to(torch.uint8)


def _unpack(rows, bits):
    """[..., d bits / 8] bytes to [..., d] codes."""
    if bits == 3:
        b = rows.view(*rows.shape[:-1], -1, 3).int()
        word = b[..., 0] | (b[..., 1] << 8) | (b[..., 2] << 16)
        codes = (word[..., None] >> (3 * torch.arange(8, device="cuda", dtype=torch.int32))) & 7
    else:
        shift = torch.arange(0, 8, bits, device="cuda", dtype=torch.uint8)
        codes = (rows[..., None] >> shift) & ((1 << bits) - 1)
    return codes.flatten(-2).long()


def _encode(case, tables, side, x, sketch):
    """What the cache stores of vectors x [batch, n, hkv, d], fp32."""
    bits = case[side + "b"]
    if bits == 8:
        scale = (x.abs().amax(-1) / 127.0).half()
        wide = scale.float()
        inverse = torch.where((wide > 0) & torch.isfinite(wide), 1.0 / wide, 0.0)
        q = (x * inverse[..., None]).round().clamp(-127, 127).to(torch.int8)
        return {"c": q.view(torch.uint8), "n": scale}
    norm = x.square().sum(-1).sqrt()
    y = (x * tables["signs"]) @ tables["had"]
    y = torch.where(norm[..., None] > 0, y / norm[..., None], 0.0)
    codes = (y[..., None] > tables[side + "b"]).sum(-1)
    out = {"c": _pack(codes, bits), "n": norm.half()}
    if side == "k" and case["qjl"]:
        r = y - tables["kc"][codes]
        bit = (r @ sketch.t() >= 0).long()
        out |= {"q": _pack(bit, 1), "g": r.square().sum(-1).sqrt().half()}
    return out


def _store(cache, side, where, enc):
    for name, a in enc.items():
        cache[side + name][where[0], :, where[1]] = a


def _decode(case, s, side, where):
    """fp32 values [batch, n, hkv, d] of the cache's slots `where`."""
    cache, tables, bits = s["cache"], s["tables"], case[side + "b"]
    norm = cache[side + "n"][where[0], :, where[1]].float()[..., None]
    rows = cache[side + "c"][where[0], :, where[1]]
    if bits == 8:
        return rows.view(torch.int8).float() * norm
    y = tables[side + "c"][_unpack(rows, bits)]
    if side == "k" and case["qjl"]:
        z = 2.0 * _unpack(cache["kq"][where[0], :, where[1]], 1).float() - 1.0
        gamma = cache["kg"][where[0], :, where[1]].float()[..., None]
        y = y + gamma * (math.sqrt(0.5 * math.pi) / case["qjl"]) * (z @ s["sketch"])
    return (y @ tables["had"]) * tables["signs"] * norm


def _turned(case, s, x):
    """x [batch, n, heads, d] with rotary positions applied, fp32."""
    angle = s["positions"].double()[..., None] * s["freq"]  # (32 bits lose the angle of a far position)
    cos, sin = (angle.cos() * s["factor"]).float()[:, :, None], (angle.sin() * s["factor"]).float()[:, :, None]
    x, r = x.float(), case["rotary"]
    if case["layout"] == "half":
        a, b = x[..., : r // 2], x[..., r // 2: r]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., r:]], -1)


def _read_plain(case, s, n, dtype):
    where = _slots(s["cache"], s["table"], s["at"], n)
    live = (torch.arange(n, device="cuda")[None] < s["counts"][:, None])[..., None, None]
    return [torch.where(live, _decode(case, s, side, where), 0.0).to(dtype) for side in "kv"]


def _rope_plain(case, s):
    where = _slots(s["cache"], s["table"], s["at"], case["tokens"])
    _store(s["cache"], "k", where, _encode(case, s["tables"], "k", _turned(case, s, s["k"]), s["sketch"]))
    _store(s["cache"], "v", where, _encode(case, s["tables"], "v", s["v"].float(), None))
    k, v = _read_plain(case, s, case["tokens"], torch.bfloat16)
    return {"q": _turned(case, s, s["q"]).to(s["q"].dtype), "k": k, "v": v}


def _tree_plain(case, s):
    batch, n, hkv, d = case["batch"], case["drafts"], case["hkv"], case["d"]
    total = case["hi"] + n
    where = _slots(s["cache"], s["table"], torch.zeros(batch, device="cuda"), total)
    k, v = _decode(case, s, "k", where), _decode(case, s, "v", where)
    q = s["q"].float().view(batch, n, hkv, -1, d)
    scores = torch.einsum("bthgd,bkhd->bhgtk", q, k) * (1.0 / math.sqrt(d))
    # slot k is before the tree, or draft k - base, which the row's mask names
    at = torch.arange(total, device="cuda")[None] - s["base"].long()[:, None]
    bit = (s["mask"][:, :, None] >> at.clamp(0, 63)[:, None]) & 1
    seen = (at < 0)[:, None] | ((at >= 0) & (at < n))[:, None] & (bit == 1)
    scores = torch.where(seen[:, None, None], scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(torch.isfinite(top), top, 0.0))
    total_p = p.sum(-1, keepdim=True)
    p = p / torch.where(total_p > 0, total_p, 1.0)
    out = torch.einsum("bhgtk,bkhd->bthgd", p, v)
    return out.reshape(batch, n, case["hq"], d).to(s["q"].dtype)


def _commit_plain(case, s):
    n, capacity = case["drafts"], s["cache"]["kn"].shape[-1]
    step = torch.arange(n, device="cuda")[None]
    live = step < s["path_lens"][:, None]
    # (slots past the accepted path are copied to themselves)
    to = _units(s["table"], capacity, s["base"].long()[:, None] + step)
    of = _units(s["table"], capacity, s["base"].long()[:, None] + torch.where(live, s["path"].long(), step))
    for a in s["cache"].values():
        a[:, to[0], :, to[1]] = a[:, of[0], :, of[1]]
    s["new_lens"].copy_(s["base"] + s["path_lens"])


def _state(s):
    """The whole cache after a move, byte for byte (the rows are carried over as they are, so what they stand for is
    as before), and the new lengths."""
    return {"cache": {k: v.view(torch.int16) if v.dtype == torch.float16 else v for k, v in s["cache"].items()},
            "lens": s["new_lens"]}


def run(state):
    case, s = state["case"], state
    if not own:
        if case["op"] == "rope":
            return _rope_plain(case, s)
        if case["op"] == "tree":
            return _tree_plain(case, s)
        if case["op"] == "read":
            return _read_plain(case, s, case["hi"], DTYPES[case["dtype"]])
        _commit_plain(case, s)
        return _state(s)
    h = s["h"]
    tq, p, kcb, vcb, err, table = h["tq"], h["p"], h["kcb"], h["vcb"], h["err"], h["table"]
    if case["op"] == "commit":
        if table is None:
            tq.tq_commit_drafts(h["layers"], s["path"], s["path_lens"], s["base"], s["new_lens"], err)
        else:
            tq.tq_commit_drafts_paged(h["layers"], table, s["path"], s["path_lens"], s["base"], s["new_lens"], err)
        return _state(s)
    cache = h["cache"]
    if case["op"] == "tree":
        if table is None:
            tq.tq_tree_attention(p, kcb, vcb, s["q"], s["mask"], s["base"], cache, s["out_buf"], h["ws"], error=err)
        else:
            tq.tq_tree_attention_paged(p, kcb, vcb, s["q"], s["mask"], s["base"], cache, table, s["out_buf"],
                                       h["ws"], error=err)
        return s["out_buf"]
    if case["op"] == "rope":
        if table is None:
            tq.tq_rope_append(p, kcb, vcb, h["rope"], s["q"], s["k"], s["v"], s["at"], cache, s["q_out"],
                              rope_positions=s["positions"], error=err)
        else:
            tq.tq_rope_append_paged(p, kcb, vcb, h["rope"], s["q"], s["k"], s["v"], s["at"], cache, table,
                                    s["q_out"], rope_positions=s["positions"], error=err)
    k, v = s["out"]
    if table is None:
        tq.tq_read_back(p, kcb, vcb, cache, s["at"], s["counts"], k, v, error=err)
    else:
        tq.tq_read_back_paged(p, kcb, vcb, cache, table, s["at"], s["counts"], k, v, error=err)
    return {"q": s["q_out"], "k": k, "v": v} if case["op"] == "rope" else [k, v]


# ------------------------------------------------ the definition, in 64 bits
def _fwht64(x):
    """Walsh-Hadamard transform of the last axis by butterflies, over sqrt(d)."""
    d, h = x.shape[-1], 1
    while h < d:
        y = x.reshape(*x.shape[:-1], d // (2 * h), 2, h)
        x = torch.stack([y[..., 0, :] + y[..., 1, :], y[..., 0, :] - y[..., 1, :]], -2).reshape(x.shape)
        h *= 2
    return x / math.sqrt(d)


def _bits64(rows, bits):
    """Codes of packed rows [n, bytes], bit by bit."""
    plane = (rows.long()[..., None] >> torch.arange(8, device="cuda")) & 1
    plane = plane.reshape(*rows.shape[:-1], -1, bits)
    return (plane << torch.arange(bits, device="cuda")).sum(-1)


def _values64(case, side, codes, norm, sketch=None, qbits=None, gamma=None):
    d = case["d"]
    if case[side + "b"] == 8:
        return codes.double() * norm.double()[..., None]
    y = torch.tensor(_codebook(d, case[side + "b"])[0], device="cuda")[codes]
    if qbits is not None:
        y = y + (gamma.double() * math.sqrt(math.pi / 2) / case["qjl"])[..., None] * torch.matmul(
            torch.where(qbits > 0, 1.0, -1.0).double(), sketch.double())
    return _fwht64(y) * torch.tensor(_signs(d), device="cuda") * norm.double()[..., None]


def _sequence64(case, s, b, side, first, count):
    """[count, hkv, d] in 64 bits of sequence b's slots from `first`, walked page by page."""
    cache, got = s["cache"], []
    unit = cache["kn"].shape[-1]
    at = first
    while at < first + count:
        block = b if s["table"] is None else int(s["table"][b, at // unit])
        lo = at if s["table"] is None else at % unit
        n = min(first + count - at, unit - lo)
        sl = slice(lo, lo + n)
        raw, norm = cache[side + "c"][block, :, sl], cache[side + "n"][block, :, sl]
        bits = case[side + "b"]
        codes = raw.view(torch.int8) if bits == 8 else _bits64(raw, bits)
        q = {}
        if side == "k" and case["qjl"]:
            q = {"sketch": s["sketch"], "qbits": _bits64(cache["kq"][block, :, sl], 1),
                 "gamma": cache["kg"][block, :, sl]}
        got.append(_values64(case, side, codes, norm, **q))
        at += n
    if not got:
        return torch.zeros(0, case["hkv"], case["d"], dtype=torch.float64, device="cuda")
    return torch.cat(got, 1).transpose(0, 1)


def _rotate64(case, x, positions):
    f, factor = _frequencies(case["rotary"], case["scaling"])
    out = x.clone()
    turn = torch.polar(torch.full((positions.numel(), 1, len(f)), factor, dtype=torch.float64, device="cuda"),
                       positions.double()[:, None, None] * torch.tensor(f, device="cuda"))
    half = case["rotary"] // 2
    first = torch.arange(half, device="cuda") * (1 if case["layout"] == "half" else 2)
    second = first + (half if case["layout"] == "half" else 1)
    z = torch.complex(x[..., first], x[..., second]) * turn
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _stored64(case, side, x, sketch):
    """What the cache's encoding of x [n, hkv, d] (64 bits) stands for."""
    d, bits = case["d"], case[side + "b"]
    if bits == 8:
        scale = (x.abs().amax(-1).float() / 127.0).half()
        # (whole-number codes follow the definition's 32-bit steps)
        inverse = torch.where(scale > 0, 1.0 / scale.float(), torch.zeros_like(scale, dtype=torch.float32))
        return _values64(case, side, (x.float() * inverse[..., None]).round().clamp(-127, 127), scale)
    norm = torch.linalg.vector_norm(x, dim=-1)
    unit = torch.where(norm[..., None] > 0, x / norm[..., None], torch.zeros_like(x))
    y = _fwht64(unit * torch.tensor(_signs(d), device="cuda"))
    c, edges = (torch.tensor(t, device="cuda") for t in _codebook(d, bits))
    codes = torch.searchsorted(edges, y.contiguous(), right=False)
    q = {}
    if side == "k" and case["qjl"]:
        r = y - c[codes]
        q = {"sketch": sketch, "qbits": (torch.matmul(r, sketch.double().t()) >= 0).long(),
             "gamma": torch.linalg.vector_norm(r, dim=-1).half()}
    return _values64(case, side, codes, norm.half(), **q)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "commit":
        return None  # whole numbers only
    batch = case["batch"]
    if case["op"] == "rope":
        q, k, v = [], [], []
        for b in range(batch):
            q.append(_rotate64(case, s["q"][b].double(), s["positions"][b]))
            k.append(_stored64(case, "k", _rotate64(case, s["k"][b].double(), s["positions"][b]),
                               s["sketch"]))
            v.append(_stored64(case, "v", s["v"][b].double(), None))
        return {"q": torch.stack(q), "k": torch.stack(k), "v": torch.stack(v)}
    if case["op"] == "read":
        out = [torch.zeros(batch, case["hi"], case["hkv"], case["d"], dtype=torch.float64, device="cuda")
               for _ in "kv"]
        for b, n in enumerate(s["counts"].tolist()):
            for o, side in zip(out, "kv"):
                o[b, :n] = _sequence64(case, s, b, side, int(s["at"][b]), n)
        return out
    n, group = case["drafts"], case["hq"] // case["hkv"]
    out = torch.zeros(batch, n, case["hq"], case["d"], dtype=torch.float64, device="cuda")
    for b, base in enumerate(s["base"].tolist()):
        k, v = (_sequence64(case, s, b, side, 0, base + n) for side in "kv")
        hidden = torch.zeros(n, base + n, dtype=torch.bool, device="cuda")
        for t, word in enumerate(s["mask"][b].tolist()):
            for j in range(n):
                hidden[t, base + j] = not (word >> j) & 1
        for h in range(case["hq"]):
            score = s["q"][b, :, h].double() @ k[:, h // group].t() / math.sqrt(case["d"])
            out[b, :, h] = torch.softmax(score.masked_fill(hidden, -math.inf), -1) @ v[:, h // group]
    return out
