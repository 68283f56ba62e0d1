"""Infinities and NaN in prompts beyond the short form's length: a row holds what
the formula over its own keys gives, whatever its tiles hold beside them."""

import pytest
import torch

from audio_generation_b200 import h3
from tests.test_gpu_prompt_attention import BF, HF, _allowed, _offsets, _reference, _run
from tests.text_testlib import DEV, STEP, assert_within

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


@pytest.mark.parametrize("at,most_ms", [(4, 3.0), (3000, 12.0), (5950, 20.0)])
@pytest.mark.parametrize("which", ["k", "v", "kv"])
def test_a_bad_token_in_a_long_prompt(which, at, most_ms):
    """A NaN k reaches every later row of its heads, an infinite v one channel of
    them. The time is bounded: rows of one tile and the 128 keys around the bad v are
    computed again, 32 to a warp, at about 50 to 100 cycles a key, at most 10 ms for
    6000 keys; every later row, key by key at 600 cycles, would be 60 ms."""
    QH, KH, D, T = 8, 2, 128, 6000

    def poison(q, k, v):
        if "k" in which:
            k[at, 0, 7] = float("nan")
        if "v" in which:
            v[at, 1, 5] = float("inf")

    q, k, v, o, offsets, scale = _run([T], QH, KH, D, BF, prepare=poison)
    touched = torch.zeros(T, QH, D, dtype=torch.bool, device=DEV)
    if "k" in which:
        touched[at:, :4] = True
        assert bool(torch.isnan(o[at:, :4]).all())
    if "v" in which:
        touched[at:, 4:, 5] = True
    assert torch.equal(torch.isfinite(o), ~touched)
    again = torch.empty_like(o)
    p = h3.h3_prompts_prepare(offsets, QH, KH, D)
    times = []
    for _ in range(3):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        h3.h3_prompt_attention(p, BF, q, QH * D, k, KH * D, v, KH * D, scale, again, QH * D)
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b))
    assert torch.equal(again.view(torch.int16), o.view(torch.int16))  # NaN too
    assert min(times) < most_ms, times
    if "k" in which:
        k[at, 0, 7] = 0
    if "v" in which:
        v[at, 1, 5] = 0
    ref, w = _reference(q, k, v, offsets, scale)
    assert_within(o[~touched], ref[~touched], _allowed(ref, w, BF)[~touched])


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("at", [8, 9, 10, 11, 12, 140, 150])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_key_before_scores_that_grow(bad, at, dtype):
    """The running maximum moves by far more than 2^100 after it: its rows stay NaN,
    by either form of the exponential."""
    def grow(q, k, v):
        q.fill_(1.0)
        k.copy_((torch.arange(k.shape[0], device=DEV) / 8)[:, None, None].expand_as(k))
        k[at, 0, 5] = bad
    q, k, v, o, offsets, scale = _run([700], 4, 2, 64, dtype, prepare=grow)
    nan = torch.zeros(700, 4, dtype=torch.bool, device=DEV)
    nan[at:, :2] = True
    assert torch.equal(torch.isnan(o).all(-1), nan) and torch.equal(torch.isfinite(o).all(-1), ~nan)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_keys_of_minus_infinity_weigh_nothing(dtype):
    """Scores of -inf, for a whole first tile of keys and for some later ones: weight
    0, and NaN only for rows that have no other score."""
    def minus(q, k, v):
        q[:, :, 0] = 1.0
        k[:, :, 0] = 0.0
        k[:200, 0, 0] = -float("inf")
        k[250:300, 1, 0] = -float("inf")
    q, k, v, o, offsets, scale = _run([700], 4, 2, 64, dtype, prepare=minus)
    assert bool(torch.isnan(o[:200, :2]).all())
    assert bool(torch.isfinite(o[200:, :2]).all()) and bool(torch.isfinite(o[:, 2:]).all())
    ref, a = _reference(q, k, v, offsets, scale)
    for rows, heads in ((slice(200, None), slice(0, 2)), (slice(None), slice(2, 4))):
        assert_within(o[rows, heads], ref[rows, heads], _allowed(ref, a, dtype)[rows, heads])


@pytest.mark.parametrize("lengths", [[40, 7], [600]])
def test_the_largest_values_of_the_type_average_to_themselves(lengths):
    """Sums of bfloat16's largest number leave float32, their average does not."""
    def largest(q, k, v):
        v.fill_(torch.finfo(BF).max)
        v[:, :, 1::2] *= -1
        v[:, :, 2] = 1.0
    q, k, v, o, offsets, scale = _run(lengths, 4, 2, 64, BF, prepare=largest)
    assert bool((o[:, :, 0] >= torch.finfo(BF).max * (1 - 4 * STEP[BF])).all())
    assert bool(torch.isfinite(o).all())
    ref, a = _reference(q, k, v, offsets, scale)
    assert_within(o, ref, _allowed(ref, a, BF))
