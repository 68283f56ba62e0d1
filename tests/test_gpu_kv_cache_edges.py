"""The 8-bit key / value cache at the ends of its arguments' ranges."""

import math

import pytest
import torch

from audio_generation_b200 import h3
from tests.test_gpu_kv_cache import BF, HF, Cache, _attention_formula, _new, _store_formula
from tests.text_testlib import DEV, STEP, TINY, assert_within, gen

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


def test_store_into_wide_tables_of_many_sequences():
    """4000 sequences whose tables have 9000 blocks for 64 heads: more (sequence,
    block, head) triples than a grid may have, of which 40 rows can touch few."""
    n, width, KH, D, BT = 4000, 9000, 64, 64, 32
    cache = Cache([0, 0], KH, D, BT, spare=32)
    first = cache.table[:, 0].clone()
    counts = [0] * n
    counts[17], counts[3990] = 30, 10
    cache.table = torch.full((n, width), -1, dtype=torch.int32, device=DEV)
    cache.table[17, 0], cache.table[3990, 0] = first[0], first[1]
    cache.width, cache.lengths = width, torch.zeros(n, dtype=torch.int32, device=DEV)
    k, v = _new([30, 10], KH, D, HF)
    pair = Cache([0, 0], KH, D, BT, spare=32)
    want = [_store_formula(pair, pair.kc, pair.ks, [30, 10], k, False),
            _store_formula(pair, pair.vc, pair.vs, [30, 10], v, True)]
    cache.store(counts, k, v, max_new=width * BT)
    assert h3.h3_text_error() == h3.H3_OK
    assert torch.equal(cache.kc, want[0][0]) and torch.equal(cache.ks, want[0][1])
    assert torch.equal(cache.vc, want[1][0]) and torch.equal(cache.vs, want[1][1])


@pytest.mark.parametrize("lengths", [[9001], [40, 64, 300], [70] * 500])
@pytest.mark.parametrize("scale", [1e34, 1e-36])
def test_attention_over_values_at_the_ends_of_the_range(lengths, scale):
    """Values up to 4e36, which bfloat16 holds but not their sum over the tokens, and
    down to 1e-36: averages of them like any others (the bound of values between)."""
    QH, KH, D = 8, 2, 128
    cache = Cache(lengths, KH, D, 64)
    cache.vs.mul_(scale / 0.01)
    q = torch.randn(len(lengths), QH, D, generator=gen(4), device=DEV).to(BF)
    o = cache.attend(q, 1 / math.sqrt(D))
    assert h3.h3_text_error() == h3.H3_OK
    ref, a = _attention_formula(cache, q, lengths, 1 / math.sqrt(D))
    assert_within(o, ref, a * (2.0 ** -11 + 2.4e-4) + ref.abs() * STEP[BF] * 1.01
                  + 127 * float(cache.vs.max()) * 2.0 ** -24 + 64 * TINY[BF])


@pytest.mark.parametrize("D,BT", [(64, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("factor", [16.0, 256.0])
def test_attention_of_queries_with_outlier_channels(D, BT, factor):
    """A few channels far above the rest. An element of q is off by up to half of its
    row's largest one's 32512th, so a score by that times sum |k| scale; weights are
    off by twice the largest such error, which is added to the usual bound."""
    QH, KH, lengths = 8, 2, [700, 33]
    cache = Cache(lengths, KH, D, BT)
    q = torch.randn(2, QH, D, generator=gen(11), device=DEV)
    q[:, :, 3] *= factor
    q[:, ::2, 40] *= factor / 4
    q = q.to(BF)
    scale = 1 / math.sqrt(D) / factor  # weights spread over the tokens
    o = cache.attend(q, scale)
    assert h3.h3_text_error() == h3.H3_OK
    ref, a = _attention_formula(cache, q, lengths, scale)
    off = torch.zeros(2, QH, 1, dtype=torch.float64, device=DEV)
    for s, n in enumerate(lengths):
        k, _ = cache.values(s, n)
        most = k.abs().sum(-1).amax(-1).repeat_interleave(QH // KH)
        off[s, :, 0] = q[s].double().abs().amax(-1) / 32512 / 2 * most * scale
    assert_within(o, ref, a * (2.0 ** -11 + 2.4e-4 + torch.expm1(2 * off))
                  + ref.abs() * STEP[BF] * 1.01 + 64 * TINY[BF])


@pytest.mark.parametrize("e", [-124, -118, -100, -60, 60, 100, 120])
def test_attention_of_queries_and_scales_at_the_ends_of_the_range(e):
    """q times a power of two and the scale divided by it: the same bits, also where
    one of them is near the end of float32."""
    cache = Cache([333, 9], 1, 128, 64)
    q = torch.rand(2, 4, 128, generator=gen(2), device=DEV) + 1  # in [1, 2): no bits are lost
    q *= torch.randint(0, 2, q.shape, generator=gen(3), device=DEV) * 2 - 1
    want = cache.attend(q.to(BF), 0.125)
    got = cache.attend((q.to(BF).double() * 2.0 ** e).to(BF), 0.125 * 2.0 ** -e)
    assert torch.equal(got, want)
    assert h3.h3_text_error() == h3.H3_OK
