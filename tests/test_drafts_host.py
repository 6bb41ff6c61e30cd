"""Argument checks and the rotary tables of the drafted-token calls, on the
host: an invalid call is refused before anything is launched (no GPU here)."""

import ctypes
import math

import numpy as np
import pytest
import torch

import drafts_ref as R
from bit_kv_cache_tq_b200 import tq

LIB = tq.library()
BUF = np.zeros(4096 + 16, dtype=np.uint8)
AT = (BUF.ctypes.data + 15) // 16 * 16  # an aligned address that no refused call reads


def _setup(**kw):
    p = tq.make_params(128, 8, 2, 4, 2, **kw)
    c = tq.tq_cache(3, 64, AT, AT, None, None, AT, AT, None)
    return p, tq.tq_codebook_init(128, 4), tq.tq_codebook_init(128, 2), c


def _ref(x):
    return None if x is None else ctypes.byref(x)


# ---------------------------------------------------------------- rotary tables
@pytest.mark.parametrize("scaling", [tq.TQ_ROPE_SCALE_NONE, tq.TQ_ROPE_SCALE_LINEAR, tq.TQ_ROPE_SCALE_BASE,
                                     tq.TQ_ROPE_SCALE_WAVELENGTH, tq.TQ_ROPE_SCALE_RAMP])
@pytest.mark.parametrize("rotary", [2, 32, 90, 128, 256])
def test_rope_tables_hold_the_frequencies(scaling, rotary):
    """turns[i] is f_i / 2 pi to within one part in 2^52 plus half of 2^-64."""
    low, high = (1.0, 32.0) if scaling == tq.TQ_ROPE_SCALE_RAMP else (1.0, 4.0)
    rope = tq.tq_rope_init(rotary, tq.TQ_ROPE_INTERLEAVED, 500000.0, scaling, 8.0, low, high, 8192.0)
    f, magnitude = R.frequencies(rotary, 500000.0, scaling, 8.0, low, high, 8192.0)
    got = np.array([t / 2.0 ** 64 for t in rope.turns[: rotary // 2]])
    assert np.all(np.abs(got - f / (2 * math.pi)) <= f * 2.0 ** -50 + 2.0 ** -64)
    assert rope.magnitude == pytest.approx(magnitude, rel=1e-15)
    assert (rope.rotary_dims, rope.layout) == (rotary, tq.TQ_ROPE_INTERLEAVED)
    assert not any(rope.turns[rotary // 2:])


def test_rope_table_magnitude_and_fast_frequencies():
    assert tq.tq_rope_init(64, magnitude=0.75).magnitude == 0.75
    assert tq.tq_rope_init(64, scaling=tq.TQ_ROPE_SCALE_RAMP, factor=0.5).magnitude == 1.0
    # more than one turn a position: kept modulo one
    rope = tq.tq_rope_init(2, scaling=tq.TQ_ROPE_SCALE_LINEAR, factor=0.01)
    assert rope.turns[0] / 2.0 ** 64 == pytest.approx(math.fmod(100 / (2 * math.pi), 1.0), abs=1e-13)


@pytest.mark.parametrize("kw", [
    dict(rotary_dims=0), dict(rotary_dims=3), dict(rotary_dims=258), dict(rotary_dims=-2), dict(layout=2),
    dict(base=1.0), dict(base=float("nan")), dict(base=float("inf")), dict(scaling=5), dict(scaling=-1),
    dict(scaling=1, factor=0.0), dict(scaling=2, factor=-1.0), dict(scaling=3, factor=float("inf")),
    dict(scaling=3, low=4.0, high=4.0), dict(scaling=4, low=0.0), dict(scaling=4, trained_len=0.0),
    dict(scaling=3, trained_len=float("nan")), dict(magnitude=-1.0), dict(magnitude=float("inf"))])
def test_rope_init_refuses(kw):
    with pytest.raises(tq.TqError) as e:
        tq.tq_rope_init(**{"rotary_dims": 64, **kw})
    assert e.value.status == tq.TQ_ERR_INVALID_ARG


# ---------------------------------------------------------------- rotary append
def _rope_status(paged=False, params=None, **kw):
    p, kcb, vcb, c = _setup(**(params or {}))
    rope = tq.tq_rope_init(128)
    for name in ("rotary_dims", "layout", "magnitude"):
        if name in kw:
            setattr(rope, name, kw.pop(name))
    a = dict(params=p, kcb=kcb, vcb=vcb, rope=rope, q=AT, q_stride=0, k=AT, k_stride=0, v=AT, v_stride=0,
             dtype=tq.TQ_BF16, n_new=3, positions=AT, rope_positions=AT, cache=c, q_out=AT, err=None,
             table=tq.tq_block_table(AT, 2, 4))
    a.update(kw)
    args = [_ref(a[x]) for x in ("params", "kcb", "vcb", "rope")]
    args += [a[x] for x in ("q", "q_stride", "k", "k_stride", "v", "v_stride", "dtype", "n_new", "positions",
                            "rope_positions")] + [_ref(a["cache"])]
    if paged:
        return LIB.tq_rope_append_paged(*args, _ref(a["table"]), a["q_out"], a["err"], None)
    return LIB.tq_rope_append(*args, a["q_out"], a["err"], None)


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("status,kw", [
    (tq.TQ_ERR_INVALID_ARG, dict(rope=None)), (tq.TQ_ERR_INVALID_ARG, dict(k=None)),
    (tq.TQ_ERR_INVALID_ARG, dict(v=None)), (tq.TQ_ERR_INVALID_ARG, dict(positions=None)),
    (tq.TQ_ERR_INVALID_ARG, dict(q=None)), (tq.TQ_ERR_INVALID_ARG, dict(q_out=None)),
    (tq.TQ_ERR_INVALID_ARG, dict(n_new=0)), (tq.TQ_ERR_INVALID_ARG, dict(dtype=3)),
    (tq.TQ_ERR_INVALID_ARG, dict(rotary_dims=130)), (tq.TQ_ERR_INVALID_ARG, dict(rotary_dims=7)),
    (tq.TQ_ERR_INVALID_ARG, dict(layout=2)), (tq.TQ_ERR_INVALID_ARG, dict(magnitude=0.0)),
    (tq.TQ_ERR_INVALID_ARG, dict(magnitude=float("nan"))), (tq.TQ_ERR_INVALID_ARG, dict(k_stride=248)),
    (tq.TQ_ERR_INVALID_ARG, dict(q_stride=1016)), (tq.TQ_ERR_INVALID_ARG, dict(v_stride=-256)),
    (tq.TQ_ERR_INVALID_ARG, dict(q_stride=1032)), (tq.TQ_ERR_ALIGNMENT, dict(k_stride=257)),
    (tq.TQ_ERR_ALIGNMENT, dict(v_stride=260)), (tq.TQ_ERR_ALIGNMENT, dict(k=AT + 8)),
    (tq.TQ_ERR_ALIGNMENT, dict(q=AT + 2)), (tq.TQ_ERR_ALIGNMENT, dict(q_out=AT + 4)),
    (tq.TQ_ERR_CAPACITY, dict(n_new=257)), (tq.TQ_ERR_INVALID_ARG, dict(kcb=None)),
    (tq.TQ_ERR_INVALID_ARG, dict(vcb=tq.tq_codebook_init(64, 2))), (tq.TQ_ERR_INVALID_ARG, dict(cache=None)),
    (tq.TQ_ERR_INVALID_ARG, dict(params=dict(qjl_dims=64)))])
def test_rope_append_refuses(paged, status, kw):
    assert _rope_status(paged, **kw) == status


def test_rope_append_refuses_a_bad_table_or_block_size():
    assert _rope_status(True, table=None) == tq.TQ_ERR_INVALID_ARG
    assert _rope_status(True, table=tq.tq_block_table(None, 2, 4)) == tq.TQ_ERR_INVALID_ARG
    assert _rope_status(True, cache=tq.tq_cache(3, 24, AT, AT, None, None, AT, AT, None)) == tq.TQ_ERR_INVALID_ARG


# --------------------------------------------------------------- tree attention
def _tree_status(paged=False, params=None, **kw):
    p, kcb, vcb, c = _setup(**(params or {}))
    a = dict(params=p, kcb=kcb, vcb=vcb, q=AT, q_dtype=tq.TQ_BF16, n_draft=4, mask=AT, base=AT, lens=None, cache=c,
             out=AT, out_dtype=tq.TQ_BF16, ws=AT, ws_bytes=1 << 40, table=tq.tq_block_table(AT, 2, 4))
    a.update(kw)
    args = [_ref(a["params"]), _ref(a["kcb"]), _ref(a["vcb"])]
    args += [a[x] for x in ("q", "q_dtype", "n_draft", "mask", "base", "lens")] + [_ref(a["cache"])]
    args += ([_ref(a["table"])] if paged else [])
    args += [a[x] for x in ("out", "out_dtype", "ws", "ws_bytes")] + [None, None]
    return (LIB.tq_tree_attention_paged if paged else LIB.tq_tree_attention)(*args)


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("status,kw", [
    (tq.TQ_ERR_INVALID_ARG, dict(q=None)), (tq.TQ_ERR_INVALID_ARG, dict(out=None)),
    (tq.TQ_ERR_INVALID_ARG, dict(mask=None)), (tq.TQ_ERR_INVALID_ARG, dict(base=None)),
    (tq.TQ_ERR_INVALID_ARG, dict(n_draft=0)), (tq.TQ_ERR_UNSUPPORTED, dict(n_draft=65)),
    (tq.TQ_ERR_INVALID_ARG, dict(q_dtype=3)), (tq.TQ_ERR_INVALID_ARG, dict(out_dtype=-1)),
    (tq.TQ_ERR_ALIGNMENT, dict(q=AT + 8)), (tq.TQ_ERR_ALIGNMENT, dict(out=AT + 2)),
    (tq.TQ_ERR_INVALID_ARG, dict(kcb=tq.tq_codebook_init(128, 3))), (tq.TQ_ERR_INVALID_ARG, dict(vcb=None)),
    (tq.TQ_ERR_INVALID_ARG, dict(cache=None)), (tq.TQ_ERR_INVALID_ARG, dict(params=dict(qjl_dims=64)))])
def test_tree_attention_refuses(paged, status, kw):
    assert _tree_status(paged, **kw) == status


def test_tree_workspace_refuses():
    p = tq.make_params(128, 8, 2)
    n = ctypes.c_size_t()
    for batch, drafts, status in ((0, 4, tq.TQ_ERR_INVALID_ARG), (1, 0, tq.TQ_ERR_INVALID_ARG),
                                  (1, 65, tq.TQ_ERR_UNSUPPORTED)):
        assert LIB.tq_tree_workspace_bytes(ctypes.byref(p), batch, drafts, ctypes.byref(n)) == status
    assert LIB.tq_tree_workspace_bytes(ctypes.byref(p), 1, 4, None) == tq.TQ_ERR_INVALID_ARG


# ----------------------------------------------------------------------- commit
def _commit_status(paged=False, n_layers=2, change=None, **kw):
    p, _, _, c = _setup()
    params, caches = (tq.tq_params * 2)(p, p), (tq.tq_cache * 2)(c, c)
    if change:
        change(params, caches)
    a = dict(path=AT, max_path=8, lens=AT + 16, base=AT + 32, new=AT + 48, table=tq.tq_block_table(AT, 2, 4))
    a.update(kw)
    args = [n_layers, params, caches] + ([_ref(a["table"])] if paged else [])
    args += [a[x] for x in ("path", "max_path", "lens", "base", "new")] + [None, None]
    return (LIB.tq_commit_drafts_paged if paged else LIB.tq_commit_drafts)(*args)


def _set(which, i, name, value):
    def change(params, caches):
        setattr((params, caches)[which][i], name, value)
    return change


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("status,kw", [
    (tq.TQ_ERR_INVALID_ARG, dict(n_layers=0)), (tq.TQ_ERR_INVALID_ARG, dict(path=None)),
    (tq.TQ_ERR_INVALID_ARG, dict(lens=None)), (tq.TQ_ERR_INVALID_ARG, dict(base=None)),
    (tq.TQ_ERR_INVALID_ARG, dict(max_path=0)), (tq.TQ_ERR_INVALID_ARG, dict(max_path=65)),
    (tq.TQ_ERR_INVALID_ARG, dict(new=AT + 32)), (tq.TQ_ERR_INVALID_ARG, dict(new=AT + 16)),
    (tq.TQ_ERR_INVALID_ARG, dict(change=_set(1, 1, "capacity", 128))),
    (tq.TQ_ERR_INVALID_ARG, dict(change=_set(1, 1, "batch", 4))),
    (tq.TQ_ERR_INVALID_ARG, dict(change=_set(1, 1, "v_norms", None))),
    (tq.TQ_ERR_ALIGNMENT, dict(change=_set(1, 0, "k_codes", AT + 8))),
    (tq.TQ_ERR_INVALID_ARG, dict(change=_set(0, 1, "qjl_dims", 64))),
    (tq.TQ_ERR_UNSUPPORTED, dict(change=_set(0, 1, "head_dim", 512)))])
def test_commit_refuses(paged, status, kw):
    assert _commit_status(paged, **kw) == status


def test_commit_paged_refuses_a_missing_table():
    assert _commit_status(True, table=None) == tq.TQ_ERR_INVALID_ARG
    assert _commit_status(True, table=tq.tq_block_table(None, 2, 4)) == tq.TQ_ERR_INVALID_ARG


# -------------------------------------------------------------------- read back
def _read_status(paged=False, **kw):
    p, kcb, vcb, c = _setup()
    a = dict(kcb=kcb, vcb=vcb, cache=c, starts=AT, counts=AT, most=4, dtype=tq.TQ_BF16, k=AT, v=AT,
             table=tq.tq_block_table(AT, 2, 4))
    a.update(kw)
    args = [_ref(p), _ref(a["kcb"]), _ref(a["vcb"]), _ref(a["cache"])] + ([_ref(a["table"])] if paged else [])
    args += [a[x] for x in ("starts", "counts", "most", "dtype", "k", "v")] + [None, None]
    return (LIB.tq_read_back_paged if paged else LIB.tq_read_back)(*args)


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("status,kw", [
    (tq.TQ_ERR_INVALID_ARG, dict(starts=None)), (tq.TQ_ERR_INVALID_ARG, dict(counts=None)),
    (tq.TQ_ERR_INVALID_ARG, dict(most=0)), (tq.TQ_ERR_INVALID_ARG, dict(k=None, v=None)),
    (tq.TQ_ERR_INVALID_ARG, dict(dtype=7)), (tq.TQ_ERR_ALIGNMENT, dict(k=AT + 8)),
    (tq.TQ_ERR_ALIGNMENT, dict(v=AT + 2)), (tq.TQ_ERR_INVALID_ARG, dict(kcb=None)),
    (tq.TQ_ERR_INVALID_ARG, dict(vcb=None)), (tq.TQ_ERR_INVALID_ARG, dict(cache=None))])
def test_read_back_refuses(paged, status, kw):
    assert _read_status(paged, **kw) == status


# ------------------------------------------------------------------ the binding
def test_binding_finds_token_strides():
    qkv = torch.zeros(2, 5, 12 * 128)
    q = qkv[..., : 8 * 128].unflatten(-1, (-1, 128))
    assert tq._token_stride(q, "q") == 12 * 128
    assert tq._token_stride(torch.zeros(2, 5, 8, 128), "q") == 0
    assert tq._token_stride(qkv[:, :1, : 8 * 128].unflatten(-1, (-1, 128)), "q") == 5 * 12 * 128
    for bad in (torch.zeros(2, 8, 5, 128).transpose(1, 2), torch.zeros(2, 5, 8, 256)[..., ::2],
                torch.zeros(2, 7, 8, 128)[:, :5], torch.zeros(1, 1, 8, 128).expand(3, 1, 8, 128)):
        with pytest.raises(ValueError):
            tq._token_stride(bad, "q")


def _cpu_call():
    p, kcb, vcb, _ = _setup()
    u8 = torch.zeros(64, dtype=torch.uint8)
    return p, kcb, vcb, tq.CacheTensors(2, 16, u8, u8, None, None, u8, u8, None), torch.zeros(2, dtype=torch.int32)


def test_binding_refuses_host_tensors_and_wrong_shapes():
    """Shapes, types and places are checked before the library is called."""
    p, kcb, vcb, cache, i32 = _cpu_call()
    k, q = torch.zeros(2, 3, 2, 128), torch.zeros(2, 3, 8, 128)
    rope = tq.tq_rope_init(128)
    for args in ((q, k, k, i32, cache, q), (q, k[:, :2], k, i32, cache, q), (q, k, k.half(), i32, cache, q),
                 (q, k[:1], k[:1], i32, cache, q), (None, k, k, i32, cache, q)):
        with pytest.raises(ValueError):
            tq.tq_rope_append(p, kcb, vcb, rope, *args)
    mask = torch.zeros(2, 3, dtype=torch.int64)
    ws = torch.zeros(16, dtype=torch.uint8)
    for args in ((q, mask, i32), (q[:, :2], mask, i32), (q.transpose(1, 2), mask, i32), (q, mask.int(), i32)):
        with pytest.raises(ValueError):
            tq.tq_tree_attention(p, kcb, vcb, *args, cache, q, ws)
    path = torch.zeros(2, 4, dtype=torch.int32)
    for bad in (path, path[0], path.long()):
        with pytest.raises(ValueError):
            tq.tq_commit_drafts(tq.draft_layers([(p, cache)]), bad, i32, i32)
    for outs in ((k, k), (k, k.half()), (q, None), (None, k[:1])):
        with pytest.raises(ValueError):
            tq.tq_read_back(p, kcb, vcb, cache, i32, i32, *outs)


def test_more_refusals_of_values_and_places():
    """Values that leave the kernels' range, addresses they could not load, and calls without anything to do."""
    for kw in (dict(scaling=tq.TQ_ROPE_SCALE_LINEAR, factor=5e-324),
               dict(scaling=tq.TQ_ROPE_SCALE_WAVELENGTH, factor=5e-324, trained_len=2.0)):
        with pytest.raises(tq.TqError) as e:  # a frequency past the doubles
            tq.tq_rope_init(64, **kw)
        assert e.value.status == tq.TQ_ERR_INVALID_ARG
    for paged in (False, True):
        for magnitude in (1e300, 1e-300):  # infinity and zero in fp32
            assert _rope_status(paged, magnitude=magnitude) == tq.TQ_ERR_INVALID_ARG
        assert _tree_status(paged, mask=AT + 4) == tq.TQ_ERR_ALIGNMENT
    p, kcb, vcb, cache, i32 = _cpu_call()
    with pytest.raises(ValueError):
        tq.draft_layers([])
    with pytest.raises(ValueError):
        tq.tq_read_back(p, kcb, vcb, cache, i32, i32)


def test_commit_takes_rows_at_their_own_alignment():
    """Norms need 2 bytes, codes of whole 16-byte rows 16, of 24-byte rows 8 (the calls that load them otherwise: 16).
    An index that no layer can hold ends the accepted calls before anything is launched."""
    for name, at, status in (("k_norms", AT + 2, tq.TQ_OK), ("v_norms", AT + 6, tq.TQ_OK),
                             ("k_norms", AT + 1, tq.TQ_ERR_ALIGNMENT), ("v_codes", AT + 8, tq.TQ_ERR_ALIGNMENT)):
        def change(params, caches, name=name, at=at):
            setattr(caches[0], name, at)
            caches[1].batch = 0 if status == tq.TQ_OK else 3  # (the second layer is refused for its batch)
        assert _commit_status(change=change) == (tq.TQ_ERR_INVALID_ARG if status == tq.TQ_OK else status)

    def narrow(off):
        def change(params, caches):
            params[0] = params[1] = tq.make_params(64, 8, 2, 3, 3)
            caches[0].k_codes = AT + off
            caches[1].batch = 0
        return change
    assert _commit_status(change=narrow(8)) == tq.TQ_ERR_INVALID_ARG
    assert _commit_status(change=narrow(4)) == tq.TQ_ERR_ALIGNMENT
