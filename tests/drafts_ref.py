"""Plain fp64 references for the drafted-token operators: rotary positions from
their definition, a paged or contiguous cache filled through the library's own
append, attention under a tree mask from the oracle's reconstruction of the
stored bytes."""

import math

import numpy as np
import torch

import harness as H
from bit_kv_cache_tq_b200 import inputs, tq

EPS = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def frequencies(r, base, scaling, factor, low, high, trained):
    i = np.arange(r // 2, dtype=np.float64)
    b = base * factor ** (r / (r - 2.0)) if scaling == tq.TQ_ROPE_SCALE_BASE and r > 2 else base
    f = b ** (-2.0 * i / r)
    if scaling == tq.TQ_ROPE_SCALE_LINEAR:
        return f / factor, 1.0
    if scaling == tq.TQ_ROPE_SCALE_WAVELENGTH:
        s = np.clip((trained * f / (2 * math.pi) - low) / (high - low), 0, 1)
        return (1 - s) * f / factor + s * f, 1.0
    if scaling == tq.TQ_ROPE_SCALE_RAMP:
        def at(n):
            return r * math.log(trained / (2 * math.pi * n)) / (2 * math.log(base))
        i0, i1 = max(0.0, math.floor(at(high))), min(r - 1.0, math.ceil(at(low)))
        s = np.clip((i - i0) / max(i1 - i0, 0.001), 0, 1)
        return s * f / factor + (1 - s) * f, max(1.0, 0.1 * math.log(factor) + 1.0)
    return f, 1.0


def rotate(x, positions, r, layout, freqs, magnitude):
    """x [batch, n, heads, d] fp64, positions [batch, n] -> rotated, and the sum of magnitudes of the products."""
    angle = positions.astype(np.float64)[..., None, None] * freqs
    c, s = magnitude * np.cos(angle), magnitude * np.sin(angle)
    out, big = x.copy(), np.zeros_like(x)
    first = slice(0, r // 2) if layout == tq.TQ_ROPE_HALF else slice(0, r, 2)
    second = slice(r // 2, r) if layout == tq.TQ_ROPE_HALF else slice(1, r, 2)
    a, b = x[..., first], x[..., second]
    out[..., first], out[..., second] = a * c - b * s, b * c + a * s
    big[..., first] = big[..., second] = (np.abs(a) + np.abs(b)) * magnitude
    return out, big


def make_cache(layer, batch, slots, page=0, seed=0, extra_blocks=2):
    """(cache, table or None); pages in random order, the pool's spare blocks among them."""
    if not page:
        return tq.alloc_cache(layer.params, batch, slots), None
    per = -(-slots // page)
    g = torch.Generator().manual_seed(seed)
    order = torch.randperm(batch * per + extra_blocks, generator=g)[: batch * per]
    pool = tq.alloc_cache(layer.params, batch * per + extra_blocks, page)
    return pool, order.view(batch, per).to(torch.int32).cuda()


def append(layer, cache, table, k, v, at):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pos = torch.tensor(at, dtype=torch.int32, device="cuda")
    if table is None:
        tq.tq_quantize_append(layer.params, layer.kcb, layer.vcb, k, v, pos, cache, err)
    else:
        tq.tq_quantize_append_paged(layer.params, layer.kcb, layer.vcb, k, v, pos, cache, table, err)
    assert tq.tq_read_device_error(err) == (tq.TQ_OK, 0)


def fill(layer, cache, table, batch, tokens, seed):
    """Random keys and values in slots 0 .. tokens - 1 of every sequence."""
    k = inputs.lognormal_kv(batch, tokens, layer.hkv, layer.d, seed=seed, layer=1, which=inputs.K, device="cuda")
    v = inputs.lognormal_kv(batch, tokens, layer.hkv, layer.d, seed=seed, layer=1, which=inputs.V, device="cuda")
    append(layer, cache, table, k, v, [0] * batch)


def contiguous(layer, cache, table, batch, tokens):
    """The first `tokens` slots of every sequence of a paged cache, as a contiguous cache on the device."""
    if table is None:
        return cache
    out = tq.alloc_cache(layer.params, batch, tokens)
    at = torch.arange(tokens, device="cuda")
    blk = table.long()[:, at // cache.capacity]
    for name in ("k_codes", "k_norms", "k_qjl", "k_gamma", "v_codes", "v_norms"):
        src = getattr(cache, name)
        if src is not None:
            getattr(out, name).copy_(src[blk, :, at % cache.capacity].transpose(1, 2))
    return out


def tree_attention(layer, cache, q, masks, bases, drafts):
    """q [batch, n, hq, d] fp64 -> [batch, n, hq, d] fp64 over a contiguous cache; rows past a sequence's drafts are
    NaN, rows that see nothing zero."""
    batch, n, hq, d = q.shape
    g = hq // layer.hkv
    sm = layer.params.sm_scale or 1.0 / math.sqrt(d)
    out = np.full(q.shape, np.nan)
    for b in range(batch):
        total = bases[b] + drafts[b]
        khat = [H.stored_hat(layer, cache, b, h, total, 0) for h in range(layer.hkv)]
        vhat = [H.stored_hat(layer, cache, b, h, total, 1) for h in range(layer.hkv)]
        for t in range(drafts[b]):
            see = np.concatenate([np.ones(bases[b], bool),
                                  np.array([(int(masks[b, t]) >> j) & 1 for j in range(drafts[b])], bool)])
            for h in range(hq):
                if not see.any():
                    out[b, t, h] = 0.0
                    continue
                s = sm * (khat[h // g][see] @ q[b, t, h])
                p = np.exp(s - s.max())
                out[b, t, h] = (p / p.sum()) @ vhat[h // g][see]
    return out


def random_tree(batch, n, seed):
    """int64 [batch, n]: bits of each draft's ancestors and itself (parents among the earlier drafts, or none)."""
    rng = np.random.default_rng(seed)
    masks = np.zeros((batch, n), dtype=np.uint64)
    for b in range(batch):
        for t in range(n):
            parent = int(rng.integers(-1, t)) if t else -1
            masks[b, t] = np.uint64(1 << t) | (masks[b, parent] if parent >= 0 else np.uint64(0))
    return masks.view(np.int64)
