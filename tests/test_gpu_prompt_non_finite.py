"""Infinities and NaN in prompts beyond the short form's length: a row holds what
the formula over its own keys gives, whatever its tiles hold beside them."""

import pytest
import torch

from tests.test_gpu_prompt_attention import BF, HF, _allowed, _offsets, _reference, _run
from tests.text_testlib import DEV, assert_within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("QH,KH,D", [(2, 2, 64), (7, 1, 128), (10, 2, 128)])
def test_bad_values_in_tiles_shared_with_others(QH, KH, D, dtype, bad):
    """A v in the middle of one prompt and one in the first token of the next: later
    keys of a row's diagonal tile, and keys of a neighbour in its last."""
    lengths = [300, 411, 290]
    offsets = _offsets(lengths)
    hits = [(offsets[1] + 130, 9), (offsets[2], 33)]

    def poison(q, k, v):
        for row, channel in hits:
            v[row, 0, channel] = bad

    q, k, v, o, offsets, scale = _run(lengths, QH, KH, D, dtype, prepare=poison)
    touched = torch.zeros(offsets[-1], QH, D, dtype=torch.bool, device=DEV)
    for row, channel in hits:
        v[row, 0, channel] = 0
        end = next(e for e in offsets if e > row)
        touched[row:end, :QH // KH, channel] = True
    assert torch.equal(torch.isfinite(o), ~touched)
    ref, a = _reference(q, k, v, offsets, scale)
    keep = ~touched
    assert_within(o[keep], ref[keep], _allowed(ref, a, dtype)[keep])
