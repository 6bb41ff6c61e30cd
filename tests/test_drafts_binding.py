"""What the binding's drafted-token calls refuse before the library sees an
address: cache arrays on several devices."""

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
