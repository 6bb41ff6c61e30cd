"""The operators of a speculative decoding step over the compressed cache, on
the GPU, against plain fp64 references: rotary positions fused with the append,
attention of a tree of drafts, the commit of an accepted path, ranges read
back.  Tolerances (each half a step of the type, where a value is rounded):

* turned queries: the angle is off by at most 2 pi 2^-26 (a fraction of a turn
  below 1/2 rounded to fp32), sine and cosine by 2 ulp (2^-23), their product
  with the magnitude by 2^-24, the two products and the sum by 2^-24 each:
  together below 2^-21 (|a| + |b|) g, then the rounding to the type;
* the cache's codes and norms: the rules of harness.py;
* reconstructions: the inverse rotation keeps the L2 norm, so a vector is off
  by the fp32 steps (below 2^-20 of it in L2: log2 d + 4 roundings) and, in 16
  bits, by the fp16 rounding of its centroids (2^-11) and of the output;
* attention: 2e-3 relative L2 per row, as for the other attention calls, plus
  the rounding of the output."""

import math

import numpy as np
import pytest
import torch

import drafts_ref as R
import harness as H
from bit_kv_cache_tq_b200 import inputs, tq

pytestmark = pytest.mark.gpu
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
I8 = tq.TQ_MODE_INT8


def _err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _names(cache):
    return [n for n in ("k_codes", "k_norms", "k_qjl", "k_gamma", "v_codes", "v_norms") if getattr(cache, n) is not None]


# ------------------------------------------------------------ rotary append
ROPE = [  # d, hq, hkv, kb, vb, qjl, batch, n, page, rotary, layout, scaling, dtype
    (128, 32, 8, 4, 2, 0, 1, 1, 0, 128, "half", "NONE", BF16),
    (128, 32, 8, 4, 4, 0, 3, 29, 64, 64, "interleaved", "WAVELENGTH", FP16),
    (128, 8, 2, 3, 2, 64, 2, 70, 0, 128, "half", "RAMP", FP32),
    (128, 6, 2, 2, 3, 0, 2, 33, 16, 64, "half", "LINEAR", BF16),
    (128, 4, 4, 4, 3, 0, 1, 41, 0, 32, "half", "BASE", BF16),
    (128, 4, 1, 4, 2, 0, 2, 17, 48, 90, "half", "NONE", FP32),
    (128, 4, 1, 3, 3, 0, 2, 17, 0, 90, "interleaved", "RAMP", FP16),
    (64, 16, 4, 8, 8, 0, 2, 19, 0, 64, "half", "NONE", BF16),
    (64, 5, 5, 4, 2, 32, 1, 7, 0, 2, "interleaved", "NONE", FP32),
    (64, 4, 2, 2, 2, 0, 5, 130, 256, 16, "half", "WAVELENGTH", FP16),
    (256, 8, 2, 4, 4, 0, 1, 23, 0, 256, "interleaved", "LINEAR", BF16),
    (256, 2, 1, 8, 2, 0, 2, 600, 0, 128, "half", "RAMP", BF16),
    (256, 4, 2, 3, 4, 128, 1, 5, 32, 256, "half", "NONE", FP16),
]


def _layer(d, hq, hkv, kb, vb, qjl=0, seed=5, sm_scale=0.0):
    modes = [I8 if b == 8 else tq.TQ_MODE_TURBO for b in (kb, vb)]
    return H.Layer(d, hq, hkv, k_bits=4 if kb == 8 else kb, v_bits=4 if vb == 8 else vb, k_mode=modes[0],
                   v_mode=modes[1], qjl_dims=qjl, seed=seed, sm_scale=sm_scale)


def _check_stored(layer, cache, b, start, x, which):
    """The codes, norms and sketch of x [n, hkv, d] fp64 in slots start .. of sequence b."""
    codes, norms = (cache.k_codes, cache.k_norms) if which == 0 else (cache.v_codes, cache.v_norms)
    mode, bits = layer.side(which)
    n = x.shape[0]
    for h in range(layer.hkv):
        sl = slice(start, start + n)
        enc = layer.oracle_encode(x[:, h], which)
        got = codes[b, h, sl].cpu().numpy()
        nb = norms[b, h, sl].cpu().numpy().view(np.uint16)
        if mode == I8:
            # the turned key differs from the fp64 one in its last bits: a step of q, an ulp of the scale
            H.check_norms(nb, enc["norm16"])
            diff = np.abs(got.view(np.int8).astype(int) - enc["q"])
            assert diff.max() <= 1 and np.mean(diff > 0) < 1e-3 + 2 * np.mean(nb != H.fp16_bits(enc["norm16"]))
            continue
        _, t = H.oracle_codebook(layer.d, bits)
        _, _, off = H.check_codes(got, enc, bits, layer.d, t)
        H.check_norms(nb, enc["norm16"])
        if which == 0 and layer.params.qjl_dims:
            H.check_qjl(cache.k_qjl[b, h, sl].cpu().numpy(), cache.k_gamma[b, h, sl].cpu().numpy(), enc, off,
                        layer.params.qjl_dims)


@pytest.mark.parametrize("d,hq,hkv,kb,vb,qjl,batch,n,page,rotary,layout,scaling,dtype", ROPE)
def test_rope_append(d, hq, hkv, kb, vb, qjl, batch, n, page, rotary, layout, scaling, dtype):
    layer = _layer(d, hq, hkv, kb, vb, qjl)
    slots = n + 21
    cache, table = R.make_cache(layer, batch, slots, page)
    for name in _names(cache):
        getattr(cache, name).view(torch.uint8).fill_(0x5A)
    g = torch.Generator().manual_seed(d + n)
    k, v = (inputs.lognormal_kv(batch, n, hkv, d, seed=9, layer=0, which=w).to(dtype) for w in (0, 1))
    q = torch.randn(batch, n, hq, d, generator=g).to(dtype)
    at = [(7 * b + 3) % (slots - n + 1) for b in range(batch)]
    pos = torch.randint(0, 200000, (batch, n), generator=g, dtype=torch.int32)
    kind, lay = getattr(tq, "TQ_ROPE_SCALE_" + scaling), getattr(tq, "TQ_ROPE_" + layout.upper())
    low, high = (1.0, 32.0) if scaling == "RAMP" else (1.0, 4.0)
    rope = tq.tq_rope_init(rotary, lay, 500000.0, kind, 8.0, low, high, 8192.0)
    q_out, err = torch.zeros_like(q, device="cuda"), _err()
    args = [layer.params, layer.kcb, layer.vcb, rope, q.cuda(), k.cuda(), v.cuda(), _ints(at), cache]
    (tq.tq_rope_append if table is None else tq.tq_rope_append_paged)(
        *args, *([] if table is None else [table]), q_out, rope_positions=pos.cuda(), error=err)
    assert tq.tq_read_device_error(err) == (tq.TQ_OK, 0)
    freqs, mag = R.frequencies(rotary, 500000.0, kind, 8.0, low, high, 8192.0)
    want, big = R.rotate(q.double().numpy(), pos.numpy(), rotary, lay, freqs, mag)
    off = np.abs(q_out.cpu().double().numpy() - want)
    assert np.all(off <= 2.0 ** -21 * big + R.EPS[dtype] * np.abs(want) * (1 + 2.0 ** -8) + 1e-30), off.max()
    kr, _ = R.rotate(k.double().numpy(), pos.numpy(), rotary, lay, freqs, mag)
    flat = R.contiguous(layer, cache, table, batch, slots)
    for b in range(batch):
        _check_stored(layer, flat, b, at[b], kr[b], 0)
        _check_stored(layer, flat, b, at[b], v[b].double().numpy(), 1)
        other = [i for i in range(slots) if not at[b] <= i < at[b] + n]
        for name in _names(flat):
            assert torch.all(getattr(flat, name)[b, :, other].contiguous().view(torch.uint8) == 0x5A), name


def test_rope_append_slices_in_place_and_slot_positions():
    """q, k, v as slices of one projection's output (the result of separate contiguous tensors, bit for bit); q turned
    in place; no positions given: the slots; positions at both ends of int32; no queries."""
    layer = _layer(128, 8, 2, 4, 2)
    batch, n, d = 2, 11, 128
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn(batch, n, 12 * d, generator=g).to(BF16).cuda()
    q, k, v = (qkv[..., a * d: z * d].unflatten(-1, (-1, d)) for a, z in ((0, 8), (8, 10), (10, 12)))
    rope = tq.tq_rope_init(128, base=10000.0)
    for positions in (None, torch.tensor([[2 ** 31 - 1] * n, [-2 ** 31] * n], dtype=torch.int32, device="cuda")):
        got = []
        for strided in (True, False):
            cache = tq.alloc_cache(layer.params, batch, 64)
            a = [t if strided else t.contiguous() for t in (q, k, v)]
            out, err = torch.empty(batch, n, 8, d, dtype=BF16, device="cuda"), _err()
            tq.tq_rope_append(layer.params, layer.kcb, layer.vcb, rope, *a, _ints([5, 40]), cache, out,
                              rope_positions=positions, error=err)
            assert tq.tq_read_device_error(err) == (tq.TQ_OK, 0)
            got.append([out] + [getattr(cache, x) for x in _names(cache)])
        assert all(torch.equal(x, y) for x, y in zip(*got))
        pos = np.array([[5], [40]]) + np.arange(n) if positions is None else positions.cpu().numpy()
        want, big = R.rotate(q.cpu().double().numpy(), pos, 128, 0, *R.frequencies(128, 10000.0, 0, 1, 1, 4, 1))
        # (fp64 loses 2^-53 of an angle of 2^31 radians in the reference: 2.4e-7)
        off = np.abs(got[0][0].cpu().double().numpy() - want)
        assert np.all(off <= (2.0 ** -21 + 2.4e-7) * big + 2.0 ** -8 * np.abs(want) * 1.01)
        inplace = q.contiguous()
        tq.tq_rope_append(layer.params, layer.kcb, layer.vcb, rope, inplace, k, v, _ints([5, 40]), cache, inplace,
                          rope_positions=positions)
        assert torch.equal(inplace, got[0][0])
        alone = tq.alloc_cache(layer.params, batch, 64)
        tq.tq_rope_append(layer.params, layer.kcb, layer.vcb, rope, None, k, v, _ints([5, 40]), alone, None,
                          rope_positions=positions)
        assert all(torch.equal(getattr(alone, x), y) for x, y in zip(_names(alone), got[0][1:]))


@pytest.mark.parametrize("rotary", [90, 32])
def test_rope_in_place_with_partners_in_other_lanes(rotary):
    layer = _layer(128, 8, 2, 4, 2)
    g = torch.Generator().manual_seed(2)
    q, k = torch.randn(3, 50, 8, 128, generator=g).to(FP16).cuda(), torch.randn(3, 50, 2, 128, generator=g).to(FP16).cuda()
    rope = tq.tq_rope_init(rotary)
    cache, out = tq.alloc_cache(layer.params, 3, 60), torch.empty_like(q)
    tq.tq_rope_append(layer.params, layer.kcb, layer.vcb, rope, q, k, k, _ints([0, 1, 10]), cache, out)
    tq.tq_rope_append(layer.params, layer.kcb, layer.vcb, rope, q, k, k, _ints([0, 1, 10]), cache, q)
    assert torch.equal(q, out)


def test_rope_append_refuses_a_position_on_the_device():
    """A sequence past the capacity, or behind a bad block-table entry, is left alone; the others and all queries are
    not."""
    layer = _layer(128, 4, 2, 4, 2)
    rope = tq.tq_rope_init(128)
    k = torch.ones(2, 3, 2, 128, dtype=BF16, device="cuda")
    q = torch.ones(2, 3, 4, 128, dtype=BF16, device="cuda")
    for at in ([4, 30], [4, -1]):
        cache, err, out = tq.alloc_cache(layer.params, 2, 32), _err(), torch.zeros_like(q)
        tq.tq_rope_append(layer.params, layer.kcb, layer.vcb, rope, q, k, k, _ints(at), cache, out,
                          rope_positions=torch.zeros(2, 3, dtype=torch.int32, device="cuda"), error=err)
        assert tq.tq_read_device_error(err) == (tq.TQ_ERR_DEVICE, tq.TQ_DEVERR_POSITION)
        assert not cache.k_norms[1].any() and not cache.v_codes[1].any() and cache.k_norms[0, :, 4:7].all()
        assert torch.equal(out, q)
    pool, err = tq.alloc_cache(layer.params, 3, 16), _err()
    table = torch.tensor([[0, 1], [7, -1]], dtype=torch.int32, device="cuda")
    tq.tq_rope_append_paged(layer.params, layer.kcb, layer.vcb, rope, q, k, k, _ints([14, 14]), pool, table, out,
                            error=err)
    assert tq.tq_read_device_error(err) == (tq.TQ_ERR_DEVICE, tq.TQ_DEVERR_PAGE)
    assert not pool.k_norms[2].any() and pool.k_norms[0, :, 14:].all() and pool.k_norms[1, :, :1].all()


# ------------------------------------------------------------- tree attention
TREE = [  # d, hq, hkv, kb, vb, qjl, bases, drafts, page, q dtype, out dtype
    (128, 32, 8, 4, 2, 0, [1001], 8, 0, BF16, BF16),
    (128, 32, 8, 3, 2, 0, [2048, 333, 64], 13, 64, BF16, BF16),
    (128, 8, 2, 4, 4, 0, [700, 0], 64, 0, FP16, FP16),
    (128, 8, 1, 2, 3, 0, [63, 65, 1], 33, 16, FP32, FP32),
    (128, 16, 1, 3, 4, 0, [515], 50, 48, BF16, FP32),
    (128, 10, 2, 4, 3, 0, [130, 200], 27, 0, BF16, BF16),
    (128, 4, 4, 2, 2, 0, [5000], 1, 256, FP16, BF16),
    (128, 8, 2, 8, 2, 0, [300, 5], 17, 0, BF16, BF16),
    (128, 8, 2, 8, 8, 0, [300, 77], 9, 32, FP32, FP32),
    (128, 8, 2, 4, 8, 0, [150], 21, 0, BF16, FP16),
    (128, 8, 2, 3, 2, 64, [200, 90], 12, 0, BF16, FP32),
    (128, 8, 2, 4, 2, 0, [700, 0, 63], 64, 0, BF16, BF16),
    (128, 16, 1, 3, 4, 0, [515, 300], 50, 48, FP16, BF16),
    (128, 10, 2, 8, 3, 0, [1300], 27, 0, FP32, BF16),
    (64, 16, 4, 8, 8, 0, [777, 1500], 17, 0, BF16, BF16),
    (64, 6, 2, 4, 2, 32, [100], 5, 16, FP32, FP32),
    (256, 8, 2, 4, 4, 0, [119, 333], 30, 64, FP16, FP16),
    (256, 16, 1, 2, 3, 256, [90], 7, 0, BF16, FP32),
]


def _tree_call(layer, q, mask, bases, cache, table, out, ws=None, draft_lens=None, stream=None):
    err = _err()
    if ws is None:
        ws = torch.empty(max(16, tq.tq_tree_workspace_bytes(layer.params, q.shape[0], q.shape[1])), dtype=torch.uint8,
                         device="cuda").fill_(0xFF)
    args = [layer.params, layer.kcb, layer.vcb, q, mask, _ints(bases), cache]
    kw = dict(draft_lens=None if draft_lens is None else _ints(draft_lens), error=err, stream=stream)
    if table is None:
        tq.tq_tree_attention(*args, out, ws, **kw)
    else:
        tq.tq_tree_attention_paged(*args, table, out, ws, **kw)
    return err


def _check_rows(got, want, dtype):
    rel = H.rel_l2_per_vector(got.cpu().double().numpy(), want)
    assert rel.max() <= H.ATTN_TOL + R.EPS[dtype], rel.max()


@pytest.mark.parametrize("d,hq,hkv,kb,vb,qjl,bases,drafts,page,qt,ot", TREE)
def test_tree_attention(d, hq, hkv, kb, vb, qjl, bases, drafts, page, qt, ot):
    layer = _layer(d, hq, hkv, kb, vb, qjl, seed=31)
    batch, total = len(bases), max(bases) + drafts
    cache, table = R.make_cache(layer, batch, total + 3, page, seed=3)
    R.fill(layer, cache, table, batch, total, seed=17)
    mask = R.random_tree(batch, drafts, seed=4)
    q = torch.randn(batch, drafts, hq, d, generator=torch.Generator().manual_seed(8)).to(qt)
    out = torch.full(q.shape, 7.0, dtype=ot, device="cuda")
    err = _tree_call(layer, q.cuda(), torch.from_numpy(mask).cuda(), bases, cache, table, out)
    assert tq.tq_read_device_error(err) == (tq.TQ_OK, 0)
    want = R.tree_attention(layer, R.contiguous(layer, cache, table, batch, total), q.double().numpy(), mask, bases,
                            [drafts] * batch)
    _check_rows(out, want, ot)


@pytest.mark.parametrize("d,kb,vb,page", [(128, 4, 2, 0), (128, 3, 4, 16), (128, 8, 8, 0), (64, 4, 4, 0)])
def test_tree_ragged_drafts_and_rows_that_see_nothing(d, kb, vb, page):
    """Draft counts 0 .. n: rows past them keep what they held, bits past them are ignored; an empty sequence whose
    draft sees nothing yields zeros; slots that no row sees may hold NaN and infinities."""
    layer = _layer(d, 8, 2, kb, vb, seed=6)
    bases, lens, n = [0, 40, 0, 129], [5, 0, 64, 9], 64
    cache, table = R.make_cache(layer, 4, 200, page, seed=1)
    R.fill(layer, cache, table, 4, 200, seed=2)
    mask = R.random_tree(4, n, seed=5)
    mask[0, 2] = 0                       # a row that sees nothing
    mask[0, 3] = -1                      # bits past the draft count
    mask[2, 63] = np.int64(-2 ** 63)     # the last bit alone
    mask[3] &= ~np.int64(1 << 4)         # draft 4 is seen by nobody
    q = torch.randn(4, n, 8, d, generator=torch.Generator().manual_seed(3)).to(BF16)
    out = torch.full(q.shape, 7.0, dtype=BF16, device="cuda")
    want = R.tree_attention(layer, R.contiguous(layer, cache, table, 4, 200), q.double().numpy(), mask, bases, lens)
    slot = bases[3] + 4
    unit, at = (3, slot) if table is None else (int(table[3, slot // page]), slot % page)
    for side in (cache.k_norms, cache.v_norms):
        side[unit, 0, at], side[unit, 1, at] = 0x7E00, 0x7C00  # NaN, infinity
    for b, first in ((0, 5), (1, 40), (3, 129 + 9)):
        for s in range(first, first + 2):  # slots behind the drafts
            u, a = (b, s) if table is None else (int(table[b, s // page]), s % page)
            cache.k_norms[u, :, a] = cache.v_norms[u, :, a] = 0x7E00
    err = _tree_call(layer, q.cuda(), torch.from_numpy(mask).cuda(), bases, cache, table, out, draft_lens=lens)
    assert tq.tq_read_device_error(err) == (tq.TQ_OK, 0)
    for b in range(4):
        assert torch.all(out[b, lens[b]:] == 7.0)
        if lens[b]:
            seen = [t for t in range(lens[b]) if not (b == 0 and t == 2)]
            _check_rows(out[b, seen], want[b, seen], BF16)
    assert not out[0, 2].any()


def test_tree_rows_that_see_a_nan_are_nan():
    """A value that is not finite reaches the rows that see it, and only those."""
    for kb, vb in ((4, 2), (8, 8)):
        layer = _layer(128, 8, 2, kb, vb, seed=6)
        cache, _ = R.make_cache(layer, 1, 100)
        R.fill(layer, cache, None, 1, 100, seed=2)
        cache.v_norms[0, 1, 70 + 3] = 0x7E00
        mask = R.random_tree(1, 20, seed=5)
        q = torch.randn(1, 20, 8, 128, generator=torch.Generator().manual_seed(3)).to(BF16).cuda()
        out = torch.empty_like(q)
        _tree_call(layer, q, torch.from_numpy(mask).cuda(), [70], cache, None, out)
        sees = torch.tensor([bool((int(m) >> 3) & 1) for m in mask[0]])
        assert torch.equal(torch.isnan(out[0, :, 4:]).all(-1).all(-1).cpu(), sees)
        assert not torch.isnan(out[0, :, :4]).any() and not torch.isnan(out[0, ~sees]).any()


def test_tree_refuses_lengths_on_the_device():
    layer = _layer(128, 8, 2, 4, 2)
    cache, _ = R.make_cache(layer, 4, 64)
    R.fill(layer, cache, None, 4, 64, seed=2)
    mask = torch.from_numpy(R.random_tree(4, 8, seed=5)).cuda()
    q = torch.randn(4, 8, 8, 128, generator=torch.Generator().manual_seed(3)).to(BF16).cuda()
    good = torch.empty_like(q)
    _tree_call(layer, q, mask, [20, 20, 20, 20], cache, None, good)
    for bases, lens in (([20, 57, -1, 56], None), ([20, 20, 20, 20], [8, 9, -1, 8])):
        out = torch.full_like(q, 7.0)
        err = _tree_call(layer, q, mask, bases, cache, None, out, draft_lens=lens)
        assert tq.tq_read_device_error(err) == (tq.TQ_ERR_DEVICE, tq.TQ_DEVERR_SEQLEN)
        assert torch.equal(out[0], good[0]) and not out[1].any() and not out[2].any() and out[3].any()


def test_tree_flags_a_bad_page():
    layer = _layer(128, 8, 2, 4, 2)
    cache, table = R.make_cache(layer, 2, 64, 16)
    R.fill(layer, cache, table, 2, 64, seed=2)
    mask = torch.from_numpy(R.random_tree(2, 8, seed=5)).cuda()
    q = torch.randn(2, 8, 8, 128, generator=torch.Generator().manual_seed(3)).to(BF16).cuda()
    good, out = torch.empty_like(q), torch.empty_like(q)
    _tree_call(layer, q, mask, [20, 20], cache, table, good)
    for bad in (-1, cache.batch, 2 ** 31 - 1):
        broken = table.clone()
        broken[1, 1] = bad
        broken[1, 3] = bad  # (past the sequence's slots: not read)
        err = _tree_call(layer, q, mask, [20, 20], cache, broken, out)
        assert tq.tq_read_device_error(err) == (tq.TQ_ERR_DEVICE, tq.TQ_DEVERR_PAGE)
        assert torch.equal(out[0], good[0])


def test_tree_of_one_draft_is_a_decode_step():
    layer = _layer(128, 32, 8, 4, 2)
    cache, _ = R.make_cache(layer, 2, 900)
    R.fill(layer, cache, None, 2, 900, seed=2)
    q = torch.randn(2, 1, 32, 128, generator=torch.Generator().manual_seed(3)).cuda()
    out = torch.empty_like(q)
    _tree_call(layer, q, torch.ones(2, 1, dtype=torch.int64, device="cuda"), [850, 31], cache, None, out)
    ref, st, _ = H.gpu_decode(layer, q[:, 0], cache, [851, 32])
    assert st == tq.TQ_OK
    assert H.rel_l2_per_vector(out[:, 0].cpu().numpy(), ref).max() < 2 * H.ATTN_TOL


def test_tree_many_units_and_a_scale():
    """More (sequence, kv head) pairs than a block's schedule holds, and a softmax scale of the layer's own."""
    layer = _layer(128, 32, 32, 4, 2, sm_scale=0.31)
    batch, n = 130, 3
    cache, _ = R.make_cache(layer, batch, 80)
    R.fill(layer, cache, None, batch, 80, seed=2)
    bases = [(11 * b) % 78 for b in range(batch)]
    mask = R.random_tree(batch, n, seed=5)
    q = torch.randn(batch, n, 32, 128, generator=torch.Generator().manual_seed(3)).to(BF16)
    out = torch.empty_like(q, device="cuda")
    _tree_call(layer, q.cuda(), torch.from_numpy(mask).cuda(), bases, cache, None, out)
    for b in (0, 1, 64, 129):
        class One:
            batch, capacity = 1, 80
        one = One()
        for name in ("k_codes", "k_norms", "v_codes", "v_norms"):
            setattr(one, name, getattr(cache, name)[b:b + 1])
        want = R.tree_attention(layer, one, q[b:b + 1].double().numpy(), mask[b:b + 1], bases[b:b + 1], [n])
        _check_rows(out[b:b + 1], want, BF16)


@pytest.mark.parametrize("scale", [2.0 ** -12, 2.0 ** 6, 2.0 ** 9])
def test_tree_with_small_and_large_vectors(scale):
    """Norms far from one (values near 1e-3 and near 1e4): the fp16 operands keep their precision.  Where a norm passes
    the fp16 range it is stored as infinity, and the head's rows are not finite, in the reference or here."""
    layer = _layer(128, 8, 2, 4, 2)
    cache, _ = R.make_cache(layer, 1, 300)
    k = inputs.lognormal_kv(1, 300, 2, 128, seed=1, layer=1, which=0, device="cuda")
    v = (inputs.lognormal_kv(1, 300, 2, 128, seed=1, layer=1, which=1, device="cuda").float() * scale).to(BF16)
    R.append(layer, cache, None, k, v, [0])
    mask = R.random_tree(1, 12, seed=5)
    q = torch.randn(1, 12, 8, 128, generator=torch.Generator().manual_seed(3))
    out = torch.empty_like(q, device="cuda")
    _tree_call(layer, q.cuda(), torch.from_numpy(mask).cuda(), [280], cache, None, out)
    want = R.tree_attention(layer, cache, q.double().numpy(), mask, [280], [12])
    fine = np.isfinite(want).all((0, 1, 3))
    assert fine.all() == (scale < 2.0 ** 9) and fine.any()
    _check_rows(out[:, :, torch.from_numpy(fine)], want[:, :, fine], FP32)
    assert not torch.isfinite(out[:, :, torch.from_numpy(~fine)]).any()


# --------------------------------------------------------------------- commit
def _commit_layers(specs, batch, slots, page, seed):
    layers, tables = [], None
    g = torch.Generator(device="cuda").manual_seed(seed)
    for d, hkv, kb, vb, qjl in specs:
        layer = _layer(d, hkv, hkv, kb, vb, qjl)
        cache, table = R.make_cache(layer, batch, slots, page, seed=seed)
        for name in _names(cache):
            getattr(cache, name).view(torch.uint8).random_(0, 256, generator=g)
        layers.append((layer, cache))
        tables = table
    return layers, tables


@pytest.mark.parametrize("page", [0, 16, 48])
@pytest.mark.parametrize("order", ["ascending", "any"])
def test_commit_drafts(page, order):
    """Layers of different heads, widths and modes; paths of 0 .. 64 drafts, in ascending or any order and with
    repeats; every byte of every cache, and the new lengths."""
    specs = [(128, 8, 4, 2, 0), (128, 2, 3, 3, 64), (64, 3, 8, 8, 0), (256, 1, 8, 4, 0), (256, 2, 2, 2, 256),
             (128, 1, 2, 8, 32), (64, 5, 3, 3, 0), (64, 6, 3, 4, 32), (256, 9, 3, 8, 0)]
    batch, n = 5, 64
    layers, table = _commit_layers(specs, batch, 150, page, seed=3)
    rng = np.random.default_rng(1)
    lens = [0, 1, 7, 64, 33]
    base = [3, 0, 80, 150 - 64, 17]
    path = np.zeros((batch, n), dtype=np.int32)
    for b in range(batch):
        p = rng.permutation(64)[: lens[b]] if order == "ascending" else rng.integers(0, 64, lens[b])
        path[b, : lens[b]] = np.sort(p) if order == "ascending" else p
    before = [{m: getattr(c, m).clone() for m in _names(c)} for _, c in layers]
    new, err = _ints([-5] * batch), _err()
    held = tq.draft_layers([(y.params, c) for y, c in layers])
    args = [held] + ([] if table is None else [table])
    (tq.tq_commit_drafts if table is None else tq.tq_commit_drafts_paged)(
        *args, torch.from_numpy(path).cuda(), _ints(lens), _ints(base), new, err)
    assert tq.tq_read_device_error(err) == (tq.TQ_OK, 0)
    assert new.tolist() == [a + b for a, b in zip(base, lens)]

    def where(b, slot):
        return (b, slot) if table is None else (int(table[b, slot // page]), slot % page)

    for (_, c), old in zip(layers, before):
        for name, a in old.items():
            want = a.clone()
            for b in range(batch):
                for i in range(lens[b]):
                    (u, s), (fu, fs) = where(b, base[b] + i), where(b, base[b] + int(path[b, i]))
                    want[u, :, s] = a[fu, :, fs]
            assert torch.equal(getattr(c, name), want), name


def test_commit_refuses_on_the_device():
    """A draft index, length or slot out of range, or a bad page: that sequence is left alone and keeps its length."""
    layers, _ = _commit_layers([(128, 2, 4, 2, 0)], 6, 40, 0, seed=3)
    layer, cache = layers[0]
    before = {m: getattr(cache, m).clone() for m in _names(cache)}
    path = torch.tensor([[1, 64], [-1, 2], [1, 2], [1, 2], [3, 4], [5, 6]], dtype=torch.int32, device="cuda")
    new, err = _ints([0] * 6), _err()
    tq.tq_commit_drafts(tq.draft_layers([(layer.params, cache)]), path, _ints([2, 2, 3, -1, 2, 2]),
                        _ints([0, 0, 0, 0, 36, -1]), new, err)
    assert tq.tq_read_device_error(err) == (tq.TQ_ERR_DEVICE, tq.TQ_DEVERR_POSITION)
    assert new.tolist() == [0, 0, 0, 0, 36, -1]
    assert all(torch.equal(getattr(cache, m), a) for m, a in before.items())
    layers, table = _commit_layers([(128, 2, 4, 2, 0)], 2, 40, 16, seed=3)
    layer, cache = layers[0]
    before = {m: getattr(cache, m).clone() for m in _names(cache)}
    table[:, 1] = 999
    path = torch.tensor([[14, 2], [1, 2]], dtype=torch.int32, device="cuda")
    tq.tq_commit_drafts_paged(tq.draft_layers([(layer.params, cache)]), table, path, _ints([2, 0]), _ints([6, 6]),
                              new[:2], err)
    assert tq.tq_read_device_error(err) == (tq.TQ_ERR_DEVICE, tq.TQ_DEVERR_POSITION | tq.TQ_DEVERR_PAGE)
    assert all(torch.equal(getattr(cache, m), a) for m, a in before.items()) and new[:2].tolist() == [6, 6]


def test_commit_of_many_layers():
    """More layers than one launch takes."""
    layers, _ = _commit_layers([(64, 1, 2, 2, 0)] * 150, 2, 16, 0, seed=4)
    before = [c.k_codes.clone() for _, c in layers]
    new = _ints([0, 0])
    tq.tq_commit_drafts(tq.draft_layers([(y.params, c) for y, c in layers]), _ints([[3, 5], [1, 0]]), _ints([2, 1]),
                        _ints([8, 2]), new)
    assert new.tolist() == [10, 3]
    for (_, c), a in zip(layers, before):
        want = a.clone()
        want[0, :, 8], want[0, :, 9], want[1, :, 2] = a[0, :, 11], a[0, :, 13], a[1, :, 3]
        assert torch.equal(c.k_codes, want)


# ------------------------------------------------------------------ read back
READ = [(128, 8, 4, 2, 0, 0), (128, 3, 3, 3, 0, 16), (128, 2, 2, 4, 64, 48), (64, 5, 4, 3, 0, 0), (64, 2, 3, 8, 32, 0),
        (256, 2, 4, 2, 0, 64), (256, 1, 2, 3, 128, 0), (128, 4, 8, 8, 0, 0), (256, 3, 8, 4, 0, 32)]


@pytest.mark.parametrize("d,hkv,kb,vb,qjl,page", READ)
@pytest.mark.parametrize("dtype", [FP32, BF16, FP16])
def test_read_back(d, hkv, kb, vb, qjl, page, dtype):
    layer = _layer(d, hkv, hkv, kb, vb, qjl)
    slots, starts, counts = 211, [0, 60, 17, 210, 211], [211, 1, 97, 1, 0]
    cache, table = R.make_cache(layer, 5, slots, page)
    R.fill(layer, cache, table, 5, slots, seed=12)
    outs = [torch.full((5, 211, hkv, d), 7.0, dtype=dtype, device="cuda") for _ in "kv"]
    err = _err()
    args = [layer.params, layer.kcb, layer.vcb, cache] + ([] if table is None else [table])
    (tq.tq_read_back if table is None else tq.tq_read_back_paged)(*args, _ints(starts), _ints(counts), *outs, error=err)
    assert tq.tq_read_device_error(err) == (tq.TQ_OK, 0)
    flat = R.contiguous(layer, cache, table, 5, slots)
    tol = 2.0 ** -20 if dtype == FP32 else 2.0 ** -11 + R.EPS[dtype]
    for which, out in enumerate(outs):
        for b in range(5):
            assert torch.all(out[b, counts[b]:] == 7.0)
            for h in range(hkv):
                want = H.stored_hat(layer, flat, b, h, slots, which)[starts[b]: starts[b] + counts[b]]
                if counts[b]:
                    rel = H.rel_l2_per_vector(out[b, : counts[b], h].cpu().double().numpy(), want)
                    assert rel.max() <= tol, (which, rel.max())
    # one side alone: the same bits
    alone = torch.full_like(outs[1], 7.0)
    (tq.tq_read_back if table is None else tq.tq_read_back_paged)(*args, _ints(starts), _ints(counts), None, alone)
    assert torch.equal(alone, outs[1])


def test_read_back_refuses_on_the_device():
    layer = _layer(128, 2, 2, 4, 2)
    cache, _ = R.make_cache(layer, 5, 40)
    R.fill(layer, cache, None, 5, 40, seed=1)
    out = torch.full((5, 10, 2, 128), 7.0, device="cuda")
    err = _err()
    tq.tq_read_back(layer.params, layer.kcb, layer.vcb, cache, _ints([-1, 31, 0, 0, 30]), _ints([2, 10, 11, -1, 10]),
                    out, None, error=err)
    assert tq.tq_read_device_error(err) == (tq.TQ_ERR_DEVICE, tq.TQ_DEVERR_POSITION)
    assert torch.all(out[:4] == 7.0) and not torch.any(out[4] == 7.0)
    pool, table = R.make_cache(layer, 2, 40, 16)
    R.fill(layer, pool, table, 2, 40, seed=1)
    table[0, 1] = pool.batch
    out, err = torch.full((2, 40, 2, 128), 7.0, device="cuda"), _err()
    tq.tq_read_back_paged(layer.params, layer.kcb, layer.vcb, pool, table, _ints([0, 0]), _ints([40, 40]), out,
                          error=err)
    assert tq.tq_read_device_error(err) == (tq.TQ_ERR_DEVICE, tq.TQ_DEVERR_PAGE)
    assert torch.all(out[0, 16:32] == 7.0) and not torch.any(out[0, :16] == 7.0) and not torch.any(out[1] == 7.0)


# ------------------------------------------------------------------- together
def _step(s, stream=None):
    """One speculative step of a layer: drafts turned and appended at their depths, their attention, the commit of the
    accepted path, and the next token's decode over what is left."""
    y = s["layer"]
    args = [y.params, y.kcb, y.vcb]
    kw = dict(error=s["err"], stream=stream)
    if s["table"] is None:
        tq.tq_rope_append(*args, s["rope"], s["q"], s["k"], s["v"], s["base"], s["cache"], s["q_out"],
                          rope_positions=s["pos"], **kw)
        tq.tq_tree_attention(*args, s["q_out"], s["mask"], s["base"], s["cache"], s["out"], s["ws"], **kw)
        tq.tq_commit_drafts(s["layers"], s["path"], s["lens"], s["base"], s["new"], **kw)
        tq.tq_decode_attention(*args, s["q1"], s["cache"], s["new"], 400, s["out1"], s["ws1"], **kw)
    else:
        tq.tq_rope_append_paged(*args, s["rope"], s["q"], s["k"], s["v"], s["base"], s["cache"], s["table"],
                                s["q_out"], rope_positions=s["pos"], **kw)
        tq.tq_tree_attention_paged(*args, s["q_out"], s["mask"], s["base"], s["cache"], s["table"], s["out"], s["ws"],
                                   **kw)
        tq.tq_commit_drafts_paged(s["layers"], s["table"], s["path"], s["lens"], s["base"], s["new"], **kw)
        tq.tq_decode_attention_paged(*args, s["q1"], s["cache"], s["table"], s["new"], 400, s["out1"], s["ws1"], **kw)


def _step_state(page):
    layer = _layer(128, 16, 4, 4, 2, seed=44)
    batch, n, base = 3, 16, [300, 7, 129]
    cache, table = R.make_cache(layer, batch, 400, page)
    R.fill(layer, cache, table, batch, 400, seed=3)
    g = torch.Generator().manual_seed(12)
    mask = R.random_tree(batch, n, seed=6)
    depth = np.array([[bin(int(m) & (2 ** 64 - 1)).count("1") - 1 for m in row] for row in mask])
    paths = [[j for j in range(n) if (int(mask[b, [5, 15, 0][b]]) >> j) & 1] for b in range(batch)]
    s = {"layer": layer, "cache": cache, "table": table, "rope": tq.tq_rope_init(128, base=10000.0),
         "q": torch.randn(batch, n, 16, 128, generator=g).to(BF16).cuda(),
         "k": inputs.lognormal_kv(batch, n, 4, 128, seed=1, layer=2, which=0, device="cuda"),
         "v": inputs.lognormal_kv(batch, n, 4, 128, seed=1, layer=2, which=1, device="cuda"),
         "base": _ints(base), "pos": torch.tensor(np.array(base)[:, None] + depth, dtype=torch.int32, device="cuda"),
         "mask": torch.from_numpy(mask).cuda(), "err": _err(), "new": _ints([0] * batch),
         "path": _ints([p + [0] * (n - len(p)) for p in paths]), "lens": _ints([len(p) for p in paths]),
         "q1": torch.randn(batch, 16, 128, generator=g).to(BF16).cuda(),
         "out1": torch.empty(batch, 16, 128, device="cuda"), "layers": tq.draft_layers([(layer.params, cache)])}
    s["q_out"], s["out"] = torch.empty_like(s["q"]), torch.empty_like(s["q"])
    s["ws"] = torch.empty(tq.tq_tree_workspace_bytes(layer.params, batch, n), dtype=torch.uint8, device="cuda")
    s["ws1"] = torch.zeros(tq.tq_decode_workspace_bytes(layer.params, batch, 400), dtype=torch.uint8, device="cuda")
    return s, base, paths


@pytest.mark.parametrize("page", [0, 64])
def test_a_speculative_step(page):
    """The four calls as a decoding loop makes them: each draft's output is the decode of its own path, and the decode
    after the commit is that of the accepted sequence."""
    s, base, paths = _step_state(page)
    layer = s["layer"]
    before = R.contiguous(layer, s["cache"], s["table"], 3, 400)
    history = {m: getattr(before, m).clone() for m in _names(before)}
    _step(s)
    assert tq.tq_read_device_error(s["err"]) == (tq.TQ_OK, 0)
    assert s["new"].tolist() == [b + len(p) for b, p in zip(base, paths)]
    # a second cache that only ever saw the accepted tokens, appended one after the other at their positions
    other = tq.alloc_cache(layer.params, 3, 400)
    for m, a in history.items():
        getattr(other, m).copy_(a)
    flat = R.contiguous(layer, s["cache"], s["table"], 3, 400)
    for b, p in enumerate(paths):
        for i, t in enumerate(p):
            one, err = tq.alloc_cache(layer.params, 1, 400), _err()
            out = torch.empty(1, 1, 16, 128, dtype=BF16, device="cuda")
            tq.tq_rope_append(layer.params, layer.kcb, layer.vcb, s["rope"], s["q"][b:b + 1, t:t + 1],
                              s["k"][b:b + 1, t:t + 1], s["v"][b:b + 1, t:t + 1], _ints([base[b] + i]), one, out,
                              error=err)
            assert torch.equal(out[0, 0], s["q_out"][b, t])
            for m in _names(one):
                getattr(other, m)[b, :, base[b] + i] = getattr(one, m)[0, :, base[b] + i]
        last, end = p[-1], base[b] + len(p)
        for m in _names(other):
            assert torch.equal(getattr(flat, m)[b, :, :end], getattr(other, m)[b, :, :end]), m
        ref, st, _ = H.gpu_decode(layer, s["q_out"][b, last][None].expand(3, -1, -1).contiguous(), other, [end] * 3)
        rel = H.rel_l2_per_vector(s["out"][b, last].cpu().double().numpy(), ref[b])
        assert rel.max() < 2 * H.ATTN_TOL + R.EPS[BF16]
    ref, st, _ = H.gpu_decode(layer, s["q1"], other, s["new"].tolist())
    assert H.rel_l2_per_vector(s["out1"].cpu().numpy(), ref).max() < 2 * H.ATTN_TOL


@pytest.mark.parametrize("page", [0, 64])
def test_a_captured_step_and_another_stream(page):
    """The step captured once and replayed gives the eager step's bits; so does a step on a stream of its own."""
    s, _, _ = _step_state(page)
    names = _names(s["cache"])
    start = {m: getattr(s["cache"], m).clone() for m in names}

    def results():
        torch.cuda.synchronize()
        return [s[x].clone() for x in ("q_out", "out", "new", "out1")] + [getattr(s["cache"], m).clone() for m in names]

    def reset():
        for m in names:
            getattr(s["cache"], m).copy_(start[m])
        for x in ("q_out", "out", "out1"):
            s[x].fill_(3.0)
        torch.cuda.synchronize()

    _step(s)
    want = results()
    reset()
    side = torch.cuda.Stream()
    _step(s, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, results()))
    reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _step(s)
    for _ in range(3):
        reset()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, results()))
    assert tq.tq_read_device_error(s["err"]) == (tq.TQ_OK, 0)


def test_two_trees_at_once():
    """Two calls in flight on two streams, a workspace each."""
    layer = _layer(128, 16, 4, 4, 2)
    cache, _ = R.make_cache(layer, 2, 3000)
    R.fill(layer, cache, None, 2, 3000, seed=1)
    mask = torch.from_numpy(R.random_tree(2, 16, seed=2)).cuda()
    qs = [torch.randn(2, 16, 16, 128, generator=torch.Generator().manual_seed(i)).to(BF16).cuda() for i in range(2)]
    want = []
    for q in qs:
        out = torch.empty_like(q)
        _tree_call(layer, q, mask, [2900, 1000], cache, None, out)
        want.append(out)
    n = tq.tq_tree_workspace_bytes(layer.params, 2, 16)
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in qs]
    outs, streams = [torch.empty_like(q) for q in qs], [torch.cuda.Stream() for _ in qs]
    base, err = _ints([2900, 1000]), _err()
    torch.cuda.synchronize()
    for _ in range(5):
        for q, w, o, st in zip(qs, ws, outs, streams):
            tq.tq_tree_attention(layer.params, layer.kcb, layer.vcb, q, mask, base, cache, o, w, error=err, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_tree_many_short_units_in_one_block():
    """Blocks that walk a dozen units of one tile each, of which one of the two streams has none."""
    layer = _layer(128, 32, 32, 4, 2)
    batch, n = 60, 5
    cache, _ = R.make_cache(layer, batch, 64)
    R.fill(layer, cache, None, batch, 64, seed=4)
    bases = [b % 60 for b in range(batch)]
    mask = R.random_tree(batch, n, seed=6)
    q = torch.randn(batch, n, 32, 128, generator=torch.Generator().manual_seed(7))
    for dtype in (BF16, FP32):
        qd = q.to(dtype)
        outs = []
        for _ in range(5):
            out = torch.empty_like(qd, device="cuda")
            _tree_call(layer, qd.cuda(), torch.from_numpy(mask).cuda(), bases, cache, None, out)
            outs.append(out)
        assert all(torch.equal(o, outs[0]) for o in outs)
        for b in (0, 7, 31, 59):
            class One:
                batch, capacity = 1, 64
            one = One()
            for name in ("k_codes", "k_norms", "v_codes", "v_norms"):
                setattr(one, name, getattr(cache, name)[b:b + 1])
            want = R.tree_attention(layer, one, qd[b:b + 1].double().numpy(), mask[b:b + 1], bases[b:b + 1], [n])
            _check_rows(outs[0][b:b + 1], want, dtype)


@pytest.mark.parametrize("kb,qjl", [(4, 0), (8, 0), (3, 32)])
def test_read_back_of_many_sequences(kb, qjl):
    """More sequences than a grid's second dimension holds: the last ones give what a short batch gives."""
    layer = _layer(64, 1, 1, kb, 2, qjl)
    batch, slots, n = 66000, 16, 2
    cache, _ = R.make_cache(layer, batch, slots)
    few, _ = R.make_cache(layer, 3, slots)
    R.fill(layer, few, None, 3, slots, seed=3)
    for name in _names(cache):
        getattr(cache, name)[-3:] = getattr(few, name)
    starts, counts = _ints([0] * (batch - 3) + [1, 0, 14]), _ints([0] * (batch - 3) + [2, 1, 2])
    out = [torch.full((batch, n, 1, 64), 7.0, dtype=BF16, device="cuda") for _ in "kv"]
    want = [torch.full((3, n, 1, 64), 7.0, dtype=BF16, device="cuda") for _ in "kv"]
    err = _err()
    tq.tq_read_back(layer.params, layer.kcb, layer.vcb, cache, starts, counts, *out, error=err)
    tq.tq_read_back(layer.params, layer.kcb, layer.vcb, few, starts[-3:].clone(), counts[-3:].clone(), *want, error=err)
    assert tq.tq_read_device_error(err) == (tq.TQ_OK, 0)
    for o, w in zip(out, want):
        assert torch.equal(o[-3:], w) and torch.all(o[:-3] == 7.0)


def test_calls_from_two_threads():
    """Two host threads with layers of different widths, a stream each: no call depends on the other's launch state."""
    import threading
    work = []
    for d, qjl, kb in ((256, 0, 4), (256, 256, 4), (128, 32, 3), (128, 128, 3)):
        layer = _layer(d, 4, 2, kb, 2, qjl)
        cache, _ = R.make_cache(layer, 1, 300)
        R.fill(layer, cache, None, 1, 300, seed=d + qjl)
        q = torch.randn(1, 4, 4, d, generator=torch.Generator().manual_seed(qjl)).to(BF16).cuda()
        mask, base = torch.from_numpy(R.random_tree(1, 4, seed=2)).cuda(), _ints([280])
        ws = torch.empty(tq.tq_tree_workspace_bytes(layer.params, 1, 4), dtype=torch.uint8, device="cuda")
        out, back = torch.empty_like(q), torch.empty(1, 300, 2, d, device="cuda")
        work.append((layer, cache, q, mask, base, ws, out, back, _ints([0]), _ints([300])))

    def call(w, stream=None):
        layer, cache, q, mask, base, ws, out, back, start, count = w
        tq.tq_tree_attention(layer.params, layer.kcb, layer.vcb, q, mask, base, cache, out, ws, stream=stream)
        tq.tq_read_back(layer.params, layer.kcb, layer.vcb, cache, start, count, None, back, stream=stream)

    for w in work:
        call(w)
    torch.cuda.synchronize()
    want = [(w[6].clone(), w[7].clone()) for w in work]
    failed = []

    def run(w):
        try:
            stream = torch.cuda.Stream()
            for _ in range(100):
                call(w, stream)
            stream.synchronize()
        except Exception as e:  # noqa: BLE001 - reported below
            failed.append(e)

    threads = [threading.Thread(target=run, args=(w,)) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    assert all(torch.equal(w[6], a) and torch.equal(w[7], b) for w, (a, b) in zip(work, want))


def test_binding_refuses_places_and_types():
    """Host tensors beside device ones, types without a code, a workspace with gaps: refused before the library."""
    layer = _layer(128, 4, 2, 4, 2)
    cache, _ = R.make_cache(layer, 1, 64)
    rope, pos = tq.tq_rope_init(128), _ints([0])
    q, k = torch.zeros(1, 1, 4, 128, device="cuda"), torch.zeros(1, 1, 2, 128, device="cuda")
    mask = torch.ones(1, 1, dtype=torch.int64, device="cuda")
    ws = torch.empty(tq.tq_tree_workspace_bytes(layer.params, 1, 1), dtype=torch.uint8, device="cuda")
    a = (layer.params, layer.kcb, layer.vcb)
    for stream in (None, torch.cuda.Stream()):
        for args in ((q.cpu(), k, k, pos, cache, q), (q, k.cpu(), k, pos, cache, q), (q, k, k, pos, cache, q.cpu()),
                     (q.double(), k.double(), k.double(), pos, cache, q.double())):
            with pytest.raises(ValueError):
                tq.tq_rope_append(*a, rope, *args, stream=stream)
        for args in ((q.cpu(), mask, pos, cache, q, ws), (q, mask, pos, cache, q.cpu(), ws),
                     (q, mask, pos, cache, q, ws.cpu()), (q, mask, pos, cache, q, ws[::2]),
                     (q, mask, pos, cache, q.double(), ws)):
            with pytest.raises(ValueError):
                tq.tq_tree_attention(*a, *args, stream=stream)
        for out in (k.cpu(), k.double()):
            with pytest.raises(ValueError):
                tq.tq_read_back(*a, cache, pos, pos, out, stream=stream)


@pytest.mark.parametrize("d,kb,vb,qjl", [(128, 4, 2, 0), (64, 3, 2, 32), (64, 3, 8, 0), (128, 8, 3, 0)])
def test_commit_of_layers_in_one_allocation(d, kb, vb, qjl):
    """Layers that lie in one allocation at their own sizes, so that all but the first are aligned to their rows only."""
    layers, batch, hkv, capacity, n = 3, 3, 1, 37, 9
    layer = _layer(d, hkv, hkv, kb, vb, qjl)
    g = torch.Generator().manual_seed(d + kb)
    rows = batch * hkv * capacity

    def stack(per_row, dtype=torch.uint8):
        a = torch.randint(0, 256, (layers * rows * per_row,), generator=g, dtype=torch.uint8).cuda()
        shape = (layers, batch, hkv, capacity) + (() if dtype is torch.int16 else (per_row,))
        return a.view(dtype).view(shape)

    one = tq.alloc_cache(layer.params, 1, 16)
    a = {"k_codes": stack(one.k_codes.shape[-1]), "v_codes": stack(one.v_codes.shape[-1]),
         "k_norms": stack(2, torch.int16), "v_norms": stack(2, torch.int16)}
    if qjl:
        a["k_qjl"], a["k_gamma"] = stack(qjl // 8), stack(2, torch.int16)
    before = {m: t.clone() for m, t in a.items()}
    caches = [tq.CacheTensors(batch, capacity, a["k_codes"][i], a["k_norms"][i], a["k_qjl"][i] if qjl else None,
                              a["k_gamma"][i] if qjl else None, a["v_codes"][i], a["v_norms"][i], one.qjl_matrix)
              for i in range(layers)]
    assert caches[1].k_norms.data_ptr() % 16
    base, paths = [0, 11, 28], [[1, 4, 8], [], [0, 2, 3, 5, 6, 7]]
    path = torch.zeros(batch, n, dtype=torch.int32)
    for b, p in enumerate(paths):
        path[b, : len(p)] = torch.tensor(p, dtype=torch.int32)
    new, err = _ints([0] * batch), _err()
    tq.tq_commit_drafts(tq.draft_layers([(layer.params, c) for c in caches]), path.cuda(),
                        _ints([len(p) for p in paths]), _ints(base), new, err)
    assert tq.tq_read_device_error(err) == (tq.TQ_OK, 0)
    for m, t in a.items():
        want = before[m].clone()
        for b, p in enumerate(paths):
            for i, x in enumerate(p):
                want[:, b, :, base[b] + i] = before[m][:, b, :, base[b] + x]
        assert torch.equal(t, want), m
    assert new.tolist() == [base[b] + len(p) for b, p in enumerate(paths)]


@pytest.mark.parametrize("d,kb,qjl,dtype", [(64, 8, 0, BF16), (128, 3, 32, FP32), (256, 4, 0, BF16)])
def test_tree_of_one_long_and_several_short_sequences(d, kb, qjl, dtype):
    """Pieces of equal length over a batch whose lengths are far apart, one sequence without drafts among them."""
    layer = _layer(d, 8, 2, kb, 2, qjl)
    bases, lens, n = [2900, 0, 1, 64, 1200, 5], [7, 7, 0, 3, 1, 7], 7
    cache, _ = R.make_cache(layer, 6, 2912)
    R.fill(layer, cache, None, 6, 2912, seed=d)
    mask = R.random_tree(6, n, seed=8)
    q = torch.randn(6, n, 8, d, generator=torch.Generator().manual_seed(d)).to(dtype)
    out = torch.full_like(q, 7.0, device="cuda")
    err = _tree_call(layer, q.cuda(), torch.from_numpy(mask).cuda(), bases, cache, None, out, draft_lens=lens)
    assert tq.tq_read_device_error(err) == (tq.TQ_OK, 0)
    want = R.tree_attention(layer, cache, q.double().numpy(), mask, bases, lens)
    for b, m in enumerate(lens):
        assert torch.all(out[b, m:] == 7.0)
        if m:
            _check_rows(out[b: b + 1, :m], want[b: b + 1, :m], dtype)
