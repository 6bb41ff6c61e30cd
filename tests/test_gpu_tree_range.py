"""Tree attention over the whole range of what a cache and its queries may
hold, against the plain fp64 reference of drafts_ref.py: value scales and
norms from the smallest to the largest that fp16 stores, queries far from one,
softmax references that have to be raised again and again, long contexts,
slots at the end of the int32 range.  Tolerances as in test_gpu_drafts.py:
2e-3 relative L2 per row and the rounding of the output.

The 2e-3 covers what the operands round.  A score is a sum of d products of
about |q| |k| / d each, so an error e of each (independent) moves it by
e |q| |k| sm / sqrt(d): here |q| |k| sm is at most 120 (keys of norm 30 with
lognormal channels, times 4 where norms grow), so the key table's 6e-5 (rms
of the 4-bit table in fp16) move a weight by 6.4e-4 of itself, and a query in
11 bits (2^-12.3 rms, bf16 outputs only, whose tolerance has 2^-8 more) by
5e-4, or 2.1e-3 where norms grow; weights and values in fp16 add 2^-12.8 each."""

import numpy as np
import pytest
import torch

import drafts_ref as R
from bit_kv_cache_tq_b200 import tq
from test_gpu_drafts import BF16, FP16, FP32, _check_rows, _layer, _tree_call

pytestmark = pytest.mark.gpu


def _half(t):
    """The fp16 values of a tensor of stored norms (a view)."""
    return t.view(torch.float16)


def _run(layer, cache, q, mask, bases, drafts, dtype):
    out = torch.full(q.shape, 7.0, dtype=dtype, device="cuda")
    err = _tree_call(layer, q.cuda(), torch.from_numpy(mask).cuda(), bases, cache, None, out)
    assert tq.tq_read_device_error(err) == (tq.TQ_OK, 0)
    want = R.tree_attention(layer, cache, q.double().numpy(), mask, bases, [drafts] * len(bases))
    assert np.isfinite(want).all()
    return out, want


# ------------------------------------------------------------------- values
@pytest.mark.parametrize("scale", [600.0, 60000.0, 2.0 ** -22])
@pytest.mark.parametrize("d,kb", [(128, 4), (128, 8), (64, 4), (256, 8)])
def test_int8_values_of_any_scale(d, kb, scale):
    """Every scale that fp16 holds (its product with a code of 127 does not fit fp16): all slots', or that of one draft
    which only some rows see."""
    layer = _layer(d, 8, 2, kb, 8, seed=6)
    base, n = 150, 20
    mask = R.random_tree(1, n, seed=5)
    q = torch.randn(1, n, 8, d, generator=torch.Generator().manual_seed(3))
    for where in (slice(None), base + 3):
        cache, _ = R.make_cache(layer, 1, 190)
        R.fill(layer, cache, None, 1, 190, seed=2)
        _half(cache.v_norms)[0, :, where] = scale
        for dtype in (FP32, BF16):
            _check_rows(*_run(layer, cache, q.to(dtype), mask, [base], n, dtype), dtype)


@pytest.mark.parametrize("power", [-20, -14, 8])
@pytest.mark.parametrize("d,vb,qjl", [(128, 2, 0), (128, 4, 0), (64, 3, 0), (128, 2, 32), (256, 4, 0)])
def test_turbo_values_of_any_norm(d, vb, qjl, power):
    """Norms of all slots near 10 2^power, and every other tile's at that while the rest stay as they were.  The layers
    of d = 128 without a sketch round a value row's rotated coordinates at one scale for all norms, by at most 2^-25 of
    it, a scale of 2 or more (a quarter of the codebook's, which lies in [8, 16)): 2^-26 each, weights that add up to
    one keep it there, the inverse rotation keeps the L2 norm, so a row may be off by another 2^-26 sqrt(128)."""
    floor = 2.0 ** -26 * 128 ** 0.5 if d == 128 and not qjl else 0.0
    layer = _layer(d, 8, 2, 3, vb, qjl, seed=6)
    base, n = 200, 12
    mask = R.random_tree(1, n, seed=5)
    q = torch.randn(1, n, 8, d, generator=torch.Generator().manual_seed(3))
    for every in (64, 128):
        cache, _ = R.make_cache(layer, 1, 230)
        R.fill(layer, cache, None, 1, 230, seed=2)
        norms = _half(cache.v_norms)
        for at in range(0, 230, every):
            norms[:, :, at:at + 64] *= 2.0 ** power
        for dtype in (FP32, BF16):
            out, want = _run(layer, cache, q.to(dtype), mask, [base], n, dtype)
            off = np.linalg.norm(out.cpu().double().numpy() - want, axis=-1)
            assert np.all(off <= (R.H.ATTN_TOL + R.EPS[dtype]) * np.linalg.norm(want, axis=-1) + floor)


# ------------------------------------------------------------------ queries
@pytest.mark.parametrize("keys", ["large", "small", "ordinary"])
@pytest.mark.parametrize("d,kb,qjl", [(128, 4, 0), (128, 8, 0), (64, 2, 0), (128, 3, 64), (256, 8, 0)])
def test_queries_of_any_magnitude(d, kb, qjl, keys):
    """Small queries against keys whose norms reach 60000, large ones against keys whose norms end at 2^-14 (the scores
    stay as they were, but for a factor below two), and rows of ordinary and of small queries next to each other: no
    query is cut, none loses its bits."""
    layer = _layer(d, 8, 2, kb, 4, qjl, seed=6)
    base, n = 200, 20
    mask = R.random_tree(1, n, seed=5)
    q = torch.randn(1, n, 8, d, generator=torch.Generator().manual_seed(3))
    cache, _ = R.make_cache(layer, 1, 230)
    R.fill(layer, cache, None, 1, 230, seed=2)
    norms = _half(cache.k_norms)[:, :, :base + n]
    if keys == "ordinary":
        q[:, ::3] *= 2.0 ** -10
    else:
        factor = (60000.0 if keys == "large" else 2.0 ** -14) / norms.float().amax().item()
        norms.copy_(norms.float() * factor)
        q *= 2.0 ** -np.ceil(np.log2(factor))
    for dtype in (FP32, BF16):
        _check_rows(*_run(layer, cache, q.to(dtype), mask, [base], n, dtype), dtype)


@pytest.mark.parametrize("power", [-120, 100])
@pytest.mark.parametrize("d,kb", [(128, 4), (128, 8), (64, 4)])
def test_queries_at_the_ends_of_fp32(d, kb, power):
    """A draft that sees itself alone gets its own value, whatever its score."""
    layer = _layer(d, 4, 2, kb, 4, seed=6)
    cache, _ = R.make_cache(layer, 1, 16)
    R.fill(layer, cache, None, 1, 16, seed=2)
    mask = np.array([[1 << t for t in range(9)]], dtype=np.int64)
    q = torch.randn(1, 9, 4, d, generator=torch.Generator().manual_seed(3)) * 2.0 ** power
    for dtype in (FP32, BF16):
        _check_rows(*_run(layer, cache, q.to(dtype), mask, [0], 9, dtype), dtype)


# --------------------------------------------------------------- references
RAISE = [  # d, hq, hkv, kb, vb, qjl, base, drafts, dtype: one and two terms, paired and not, whole units and pieces
    (128, 8, 1, 4, 2, 0, 3000, 30, BF16),
    (128, 8, 2, 4, 2, 0, 3000, 30, BF16),
    (128, 8, 2, 4, 4, 0, 3000, 30, FP16),
    (128, 4, 1, 3, 3, 0, 3000, 30, FP32),
    (128, 8, 1, 8, 8, 0, 3000, 30, BF16),
    (64, 8, 2, 4, 2, 0, 1500, 30, BF16),
    (128, 8, 2, 3, 2, 32, 1500, 30, FP32),
    (256, 8, 2, 4, 2, 0, 1500, 30, FP16),
]


@pytest.mark.parametrize("few_blocks", [False, True])
@pytest.mark.parametrize("d,hq,hkv,kb,vb,qjl,base,drafts,dtype", RAISE)
def test_references_raised_tile_after_tile(d, hq, hkv, kb, vb, qjl, base, drafts, dtype, few_blocks):
    """Keys whose norms grow along the context, so that every row's largest score rises over its tiles; many sequences
    (few_blocks) leave each block whole units, so that one stream sees the whole rise."""
    layer = _layer(d, hq, hkv, kb, vb, qjl, seed=6)
    batch = 160 if few_blocks else 1
    if few_blocks:
        base = 500
    total = base + drafts
    cache, _ = R.make_cache(layer, batch, total + 2)
    one, _ = R.make_cache(layer, 1, total + 2)
    R.fill(layer, one, None, 1, total, seed=2)
    grow = torch.linspace(0.1, 4.0, total + 2, device="cuda")
    _half(one.k_norms).mul_(grow.half())
    for name in ("k_codes", "k_norms", "k_qjl", "k_gamma", "v_codes", "v_norms"):
        if getattr(one, name) is not None:
            getattr(cache, name).copy_(getattr(one, name).expand_as(getattr(cache, name)))
    mask = R.random_tree(1, drafts, seed=5)
    q = torch.randn(1, drafts, hq, d, generator=torch.Generator().manual_seed(3)).to(dtype)
    qs, masks = q.expand(batch, -1, -1, -1).contiguous(), np.repeat(mask, batch, 0)
    out = torch.full(qs.shape, 7.0, dtype=dtype, device="cuda")
    err = _tree_call(layer, qs.cuda(), torch.from_numpy(masks).cuda(), [base] * batch, cache, None, out)
    assert tq.tq_read_device_error(err) == (tq.TQ_OK, 0)
    want = R.tree_attention(layer, one, q.double().numpy(), mask, [base], [drafts])
    # bf16 outputs take their queries in 11 bits: an entry is off by 2^-12.3 of itself (rms: uniform within half a step,
    # the mantissa spread evenly), a score by 2^-12.3 sm |q| |k| / sqrt(d), independent from key to key; of the scores
    # of a row that share its weight, none is off by more than 4.5 such (15 million draws), so no weight by more than
    # twice that against its row's others
    tol = R.H.ATTN_TOL + R.EPS[dtype]
    if dtype == BF16:
        k = max(np.linalg.norm(R.H.stored_hat(layer, one, 0, h, total, 0), axis=-1).max() for h in range(hkv))
        tol += 9 * 2.0 ** -12.3 * q.double().norm(dim=-1).max().item() * k / d
    for b in {0, batch // 2, batch - 1}:
        assert R.H.rel_l2_per_vector(out[b:b + 1].cpu().double().numpy(), want).max() <= tol


@pytest.mark.parametrize("d,hq,kb,vb,qjl,dtype", [(128, 16, 4, 2, 0, BF16), (128, 4, 3, 4, 0, FP32),
                                                  (128, 4, 3, 2, 64, BF16), (64, 4, 4, 8, 0, BF16)])
def test_a_long_context(d, hq, kb, vb, qjl, dtype):
    """40000 slots of one kv head."""
    layer = _layer(d, hq, 1, kb, vb, qjl, seed=6)
    base, n = 40000, 20
    cache, _ = R.make_cache(layer, 1, base + n)
    R.fill(layer, cache, None, 1, base + n, seed=2)
    mask = R.random_tree(1, n, seed=5)
    q = torch.randn(1, n, hq, d, generator=torch.Generator().manual_seed(3)).to(dtype)
    _check_rows(*_run(layer, cache, q, mask, [base], n, dtype), dtype)


# ---------------------------------------------------------------- positions
def test_drafts_in_the_last_tile_of_the_int32_range():
    """A paged sequence of 2^31 - 16 slots (one block of zeros named again and again, then one with the drafts): each
    draft sees the slots before the tree and itself, and its query is closest to the next draft's key, which it does
    not see.  Its own score is 60 above the zeros' (2^31 of them weigh less than e^-38), so its output is its value."""
    layer = _layer(128, 1, 1, 2, 2, seed=6)
    block, per, n = 16 * 262657, 511, 20
    base = block * per - n
    assert block * per == 2 ** 31 - 16
    pool = tq.alloc_cache(layer.params, 2, block)
    table = torch.zeros(1, per, dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(1, n, 1, 128, generator=g) for _ in "kv")
    R.append(layer, pool, torch.ones(1, 1, dtype=torch.int32, device="cuda"), k.cuda(), v.cuda(), [block - n])
    q = 12.0 * (k + 1.5 * k.roll(-1, 1))

    class Last:
        batch, capacity = 1, n
    last = Last()
    for name in ("k_codes", "k_norms", "v_codes", "v_norms"):
        setattr(last, name, getattr(pool, name)[1:, :, block - n:])
    mask = torch.tensor([[1 << t for t in range(n)]], dtype=torch.int64)
    want = R.tree_attention(layer, last, q.double().numpy(), mask.numpy(), [0], [n])
    scores = np.einsum("td,td->t", q[0, :, 0].double().numpy(),
                       R.H.stored_hat(layer, last, 0, 0, n, 0)) / np.sqrt(128.0)
    assert scores.min() > 60.0
    for dtype in (FP32, BF16):
        out = torch.full(q.shape, 7.0, dtype=dtype, device="cuda")
        err = _tree_call(layer, q.to(dtype).cuda(), mask.cuda(), [base], pool, table, out)
        assert tq.tq_read_device_error(err) == (tq.TQ_OK, 0)
        _check_rows(out, want, dtype)


@pytest.mark.parametrize("power", [-6, 5])
def test_a_codebook_scale_of_the_callers(power):
    """The scale of the fp16 tables is the caller's to choose; a power of two of the usual one rounds the keys the same."""
    layer = _layer(128, 8, 2, 4, 8, seed=6)
    cache, _ = R.make_cache(layer, 1, 230)
    R.fill(layer, cache, None, 1, 230, seed=2)
    mask = R.random_tree(1, 20, seed=5)
    q = torch.randn(1, 20, 8, 128, generator=torch.Generator().manual_seed(3))
    out, _ = _run(layer, cache, q, mask, [200], 20, FP32)
    layer.kcb.fp16_scale *= 2.0 ** power
    again, want = _run(layer, cache, q, mask, [200], 20, FP32)
    _check_rows(again, want, FP32)
    assert torch.equal(out, again)
