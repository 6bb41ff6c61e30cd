"""What the binding's drafted-token calls refuse before the library sees an
address: cache arrays on several devices, error words that are none."""

import pytest
import torch

from bit_kv_cache_tq_b200 import tq

ARRAYS = ("k_codes", "k_norms", "k_qjl", "k_gamma", "v_codes", "v_norms", "qjl_matrix")


def _cache(**elsewhere):
    arrays = {name: torch.zeros(64, dtype=torch.uint8, device=elsewhere.get(name, "cpu")) for name in ARRAYS}
    return tq.CacheTensors(2, 16, **arrays)


@pytest.mark.parametrize("name", ARRAYS)
def test_a_cache_lies_on_one_device(name):
    _cache()
    with pytest.raises(ValueError, match="more than one device"):
        _cache(**{name: "meta"})


def test_the_layers_of_a_commit_lie_on_one_device():
    p = tq.make_params(128, 8, 2)
    there = _cache(**{name: "meta" for name in ARRAYS})
    tq.draft_layers([(p, there), (p, there)])
    with pytest.raises(ValueError, match="more than one device"):
        tq.draft_layers([(p, _cache()), (p, there)])


@pytest.mark.parametrize("error", [torch.zeros(4, dtype=torch.uint8), torch.zeros(1, dtype=torch.int64),
                                   torch.zeros(0, dtype=torch.int32)])
def test_error_words_have_32_bits(error):
    """An atomic OR of 32 bits goes to the word's address: a byte's may not be aligned, an empty tensor has none."""
    p, kcb, vcb = tq.make_params(128, 8, 2, 4, 2), tq.tq_codebook_init(128, 4), tq.tq_codebook_init(128, 2)
    cache, i32 = _cache(), torch.zeros(2, dtype=torch.int32)
    q, k = torch.zeros(2, 3, 8, 128), torch.zeros(2, 3, 2, 128)
    mask, ws = torch.zeros(2, 3, dtype=torch.int64), torch.zeros(16, dtype=torch.uint8)
    path = torch.zeros(2, 4, dtype=torch.int32)
    for call in (lambda: tq.tq_rope_append(p, kcb, vcb, tq.tq_rope_init(128), q, k, k, i32, cache, q, error=error),
                 lambda: tq.tq_tree_attention(p, kcb, vcb, q, mask, i32, cache, q, ws, error=error),
                 lambda: tq.tq_commit_drafts(tq.draft_layers([(p, cache)]), path, i32, i32, error=error),
                 lambda: tq.tq_read_back(p, kcb, vcb, cache, i32, i32, k, k, error=error)):
        with pytest.raises(ValueError, match="32-bit"):
            call()
