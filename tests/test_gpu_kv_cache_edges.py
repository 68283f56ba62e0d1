"""The 8-bit key / value cache at the ends of its arguments' ranges."""

import pytest
import torch

from audio_generation_b200 import h3
from tests.test_gpu_kv_cache import BF, Cache, _new, _store_formula

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts", [[1], [40], [1, 0, 33, 2], [1] * 48])
@pytest.mark.parametrize("most", [2 ** 31 - 1, 2 ** 31 - 40, 2 ** 24])
def test_store_with_a_loose_bound_on_new_tokens(counts, most):
    """max_new is a bound: any larger number stores what the exact one does."""
    cache = Cache([31] * len(counts), 2, 64, 32, spare=64)
    k, v = _new(counts, 2, 64, BF)
    kc, ks = _store_formula(cache, cache.kc, cache.ks, counts, k, False)
    vc, vs = _store_formula(cache, cache.vc, cache.vs, counts, v, True)
    cache.store(counts, k, v, max_new=most)
    assert h3.h3_text_error() == h3.H3_OK
    assert torch.equal(cache.ks, ks) and torch.equal(cache.vs, vs)
    assert torch.equal(cache.kc, kc) and torch.equal(cache.vc, vc)
