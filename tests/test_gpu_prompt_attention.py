"""Causal attention over packed prompts against its formula in 64 bits."""

import ctypes
import math

import pytest
import torch

from audio_generation_b200 import h3
from tests.text_testlib import DEV, STEP, TINY, assert_within, gen

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


def _offsets(lengths, first=0):
    out = [first]
    for n in lengths:
        out.append(out[-1] + n)
    return out


def _reference(q, k, v, offsets, scale):
    """o and sum_j w_j |v_j| (what a relative error of the weights is relative to)."""
    T, QH, D = q.shape
    G = QH // k.shape[1]
    o = torch.zeros(T, QH, D, dtype=torch.float64, device=DEV)
    a = torch.zeros_like(o)
    for lo, hi in zip(offsets[:-1], offsets[1:]):
        for h in range(QH):
            for r in range(lo, hi, 2048):
                e = min(hi, r + 2048)
                s = q[r:e, h].double() @ k[lo:hi, h // G].double().T * scale
                s.masked_fill_(torch.arange(lo, hi, device=DEV)
                               > torch.arange(r, e, device=DEV)[:, None], -math.inf)
                w = torch.softmax(s, 1)
                vv = v[lo:hi, h // G].double()
                o[r:e, h] = w @ vv
                a[r:e, h] = w @ vv.abs()
    return o, a


def _allowed(o, a, dtype):
    """The weights are rounded to `dtype` (half a step of each), their exponents
    come from float32 scores of D terms (below 1e-4 for the inputs here: 128 x
    2^-24 x sum |q k| scale, |q k| about 7) and an exponential within 1.02e-4: 2^-12
    together; the result is rounded once."""
    return a * (STEP[dtype] + 2.0 ** -12) + o.abs() * STEP[dtype] * 1.01 + 64 * TINY[dtype]


def _run(lengths, QH, KH, D, dtype, seed=0, first=0, tail=0, scale=None, prepare=None, boost=1.0):
    g = gen(seed + sum(lengths) + QH)
    offsets = _offsets(lengths, first)
    T = offsets[-1] + tail
    scale = scale or 1 / math.sqrt(D)
    q = (torch.randn(T, QH, D, generator=g, device=DEV) * boost).to(dtype)
    k = torch.randn(T, KH, D, generator=g, device=DEV).to(dtype)
    v = torch.randn(T, KH, D, generator=g, device=DEV).to(dtype)
    if prepare:
        prepare(q, k, v)
    o = torch.full((T, QH, D), 9.0, dtype=dtype, device=DEV)
    p = h3.h3_prompts_prepare(offsets, QH, KH, D)
    h3.h3_prompt_attention(p, dtype, q, QH * D, k, KH * D, v, KH * D, scale, o, QH * D)
    assert h3.h3_text_error() == h3.H3_OK
    assert bool((o[:first] == 9).all()) and bool((o[offsets[-1]:] == 9).all())
    p.close()
    return q, k, v, o, offsets, scale


def _check(lengths, QH, KH, D, dtype, **kw):
    q, k, v, o, offsets, scale = _run(lengths, QH, KH, D, dtype, **kw)
    ref, a = _reference(q, k, v, offsets, scale)
    lo, hi = offsets[0], offsets[-1]
    assert_within(o[lo:hi], ref[lo:hi], _allowed(ref, a, dtype)[lo:hi], str(lengths))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("QH,KH", [(1, 1), (2, 1), (6, 2), (5, 1), (7, 1), (8, 1), (24, 1), (3, 3),
                                   (100, 1), (128, 1), (10, 2)])
def test_group_sizes(QH, KH, D, dtype):
    """Groups that fill a tile, that leave rows idle, and one that is a tile."""
    _check([1, 130, 2, 300, 17], QH, KH, D, dtype)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("lengths", [
    [1], [2], [127], [128], [129], [255, 256, 257], [0, 5, 0, 0, 9, 0], [1] * 70, [513, 1, 385],
    [63, 64, 65, 31, 33]])
def test_lengths(lengths, dtype):
    _check(lengths, 4, 2, 128, dtype)
    _check(lengths, 3, 3, 64, dtype)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("QH,KH,lengths", [
    (1, 1, [1, 17, 2, 60, 77, 5, 128, 33, 0, 64]), (14, 2, [1, 17, 2, 60, 77, 5, 128, 33, 0, 64]),
    (5, 5, [127, 128, 126]), (24, 1, [3, 31, 32, 33]), (128, 1, [9, 30, 2]), (100, 1, [1]),
    (40, 8, [8] * 31), (3, 1, [21, 22, 43]), (8, 8, [140]), (4, 2, [256, 3, 255])])
def test_short_prompts(QH, KH, lengths, D, dtype):
    """Batches without a prompt of more than 256 tokens, as few as take their own form."""
    _check(lengths, QH, KH, D, dtype, first=3, tail=70)


def test_many_short_prompts():
    """So many that the other form is taken again."""
    _check([100, 37, 128, 5] * 24, 24, 2, 128, BF)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_non_finite_values_in_short_prompts(bad, dtype):
    lengths, QH, KH, hit = [40, 90, 30], 6, 2, 40 + 17

    def poison(q, k, v):
        v[hit, 1, 70] = bad
        v[hit + 1:40 + 90, 0] = torch.finfo(dtype).max
        q[3, 2, 9] = float("nan")
        k[40 + 90 + 11, 0, 4] = float("nan")

    clean, o = (_run(lengths, QH, KH, 128, dtype, prepare=f)[3] for f in (None, poison))
    touched = torch.zeros(sum(lengths), QH, dtype=torch.bool, device=DEV)
    touched[hit:130, 3:] = True      # rows that attend the bad v
    touched[hit + 1:130, :3] = True  # and the largest
    touched[3, 2] = True
    touched[141:, :3] = True
    diff = (o.double() - clean.double()).abs()[~touched]
    assert bool((diff <= 3 * STEP[dtype] * (clean.double().abs()[~touched] + 1)).all())
    assert not bool(torch.isfinite(o[hit:130, 3:, 70]).any())
    assert bool(torch.isfinite(o[hit:130, 3:, :70]).all())
    assert bool(torch.isnan(o[3, 2]).all()) and bool(torch.isnan(o[141:, :3]).all())


def test_long_prompt():
    _check([5000, 70], 5, 1, 128, BF)


def test_rows_before_and_behind_the_prompts_stay():
    _check([40, 200], 4, 1, 128, BF, first=13, tail=29)


@pytest.mark.parametrize("scale", [1e-3, 0.7])
def test_scales(scale):
    """Nearly uniform and nearly one-hot weights. At scale 0.7 a score's error is
    0.7 / 0.088 = 8 times that of the default scale, below 2^-12 x 8."""
    q, k, v, o, offsets, s = _run([300, 77], 4, 2, 128, BF, scale=scale)
    ref, a = _reference(q, k, v, offsets, s)
    assert_within(o, ref, _allowed(ref, a, BF) + a * 2.0 ** -9)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_the_maximum_moves_late_and_far(dtype):
    """Scores that grow along the keys: every tile raises the running maximum."""
    def grow(q, k, v):
        q.fill_(1.0)
        k.copy_((torch.arange(k.shape[0], device=DEV) / 16)[:, None, None].expand_as(k))
    q, k, v, o, offsets, s = _run([700], 4, 2, 64, dtype, prepare=grow)
    ref, a = _reference(q, k, v, offsets, s)
    # scores up to 700 / 16 x 8 = 350: 64 terms of float32 sums of one sign, 64 x
    # 2^-24 x 350 = 1.3e-3 in the exponent
    assert_within(o, ref, _allowed(ref, a, dtype) + a * 2e-3)


def test_fp16_long_tails_of_small_weights():
    """4000 keys with weights 2^-20 of the largest: together 0.4 % of the sum."""
    def spike(q, k, v):
        q.zero_(); k.zero_()
        q[:, :, 0] = 8.0
        k[0, :, 0] = 8.0 * math.log(2) * 20 / 8  # score 20 ln 2 x 8 / sqrt(64) above the rest
        v[1:] = 100.0
        v[0] = 0.0
    q, k, v, o, offsets, s = _run([4000], 2, 1, 64, HF, prepare=spike)
    ref, a = _reference(q, k, v, offsets, s)
    assert_within(o, ref, _allowed(ref, a, HF))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("QH,KH", [(2, 2), (7, 1)])
def test_non_finite_values_stay_with_the_rows_that_attend_them(bad, QH, KH):
    """A bad k or v at token t of a prompt reaches rows >= t of that prompt only,
    whatever tile it shares with others; so does a bad q, its own row."""
    lengths = [70, 200, 90]
    offsets = _offsets(lengths)
    hit = offsets[1] + 37

    def poison_v(q, k, v):
        v[hit, 0, 5] = bad

    def poison_k(q, k, v):
        k[hit, 0, 5] = float("nan")

    def poison_q(q, k, v):
        q[hit, 0, 5] = float("nan")

    clean, *_ = [_run(lengths, QH, KH, 128, BF)[3]]
    rows = torch.arange(offsets[-1], device=DEV)
    below = (rows >= hit) & (rows < offsets[2])
    heads = torch.arange(QH, device=DEV) < QH // KH
    for poison in (poison_v, poison_k, poison_q):
        o = _run(lengths, QH, KH, 128, BF, prepare=poison)[3]
        if poison is poison_q:
            touched = torch.zeros(offsets[-1], QH, dtype=torch.bool, device=DEV)
            touched[hit, 0] = True
        else:
            touched = below[:, None] & heads
        finite = torch.isfinite(o).all(-1)
        assert bool((finite == ~touched).all())
        keep = ~touched
        if poison is poison_v:
            # rows of the bad tile come from plain float32 arithmetic: not the
            # tiles' bits, the same value within both roundings
            diff = (o.double() - clean.double()).abs()[keep]
            assert bool((diff <= 3 * STEP[BF] * (clean.double().abs()[keep] + 1)).all())
            other = touched[:, :, None] & (torch.arange(128, device=DEV) != 5)
            assert bool(torch.isfinite(o[other.expand_as(o)]).all())
        else:
            assert torch.equal(o[keep], clean[keep])


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D", [64, 128])
def test_a_nan_key_reaches_every_row_behind_it(D, dtype):
    """At any place among the keys of a tile: the rows from it on are NaN, no other."""
    lengths = [140] * 66

    def poison(q, k, v):
        for i in range(66):
            k[140 * i + 2 * i + 1, 0, 3] = float("nan")

    o = _run(lengths, 2, 1, D, dtype, prepare=poison)[3].view(66, 140, 2, D)
    rows = torch.arange(140, device=DEV)
    reached = rows >= 2 * torch.arange(66, device=DEV)[:, None] + 1
    assert torch.equal(torch.isnan(o).all(-1).all(-1), reached)
    assert torch.equal(torch.isfinite(o).all(-1).all(-1), ~reached)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_the_largest_values_behind_a_row_do_not_reach_it(dtype):
    """The type's largest number in v at every later token, at both signs: not a bit
    of the rows before changes."""
    lengths, hit = [150, 300, 40], 150 + 101
    clean = _run(lengths, 5, 1, 128, dtype)[3]

    def largest(q, k, v):
        v[hit:] = torch.finfo(dtype).max
        v[hit::2] *= -1

    assert torch.equal(_run(lengths, 5, 1, 128, dtype, prepare=largest)[3][:hit], clean[:hit])


def test_garbage_behind_the_last_prompt_is_not_read_into_it():
    def garbage(q, k, v):
        for x in (q, k, v):
            x[150:] = float("nan")
    _check([100, 50], 4, 2, 128, BF, tail=90, prepare=garbage)


def test_slices_of_one_projection():
    QH, KH, D, T = 10, 2, 64, 333
    qkv = torch.randn(T, (QH + 2 * KH) * D + 64, generator=gen(5), device=DEV).to(BF)
    q, k, v = (x.view(T, -1, D) for x in qkv[:, :-64].split([QH * D, KH * D, KH * D], 1))
    out = torch.full((T, QH * D + 32), 4.0, dtype=BF, device=DEV)
    offsets = [0, 100, 333]
    p = h3.h3_prompts_prepare(offsets, QH, KH, D)
    h3.h3_prompt_attention(p, BF, q, q.stride(0), k, k.stride(0), v, v.stride(0), 0.125, out,
                           out.stride(0))
    ref, a = _reference(q, k, v, offsets, 0.125)
    assert_within(out[:, :QH * D].view(T, QH, D), ref, _allowed(ref, a, BF))
    assert bool((out[:, QH * D:] == 4).all())


def test_two_batches_two_streams_and_a_graph():
    """Two prompts objects used at once on two streams give what they give alone,
    and a captured call follows its inputs."""
    QH, KH, D = 8, 2, 128
    work = []
    for seed, lengths in ((1, [400, 31]), (2, [7, 90, 333])):
        g = gen(seed)
        T = sum(lengths)
        x = [torch.randn(T, h, D, generator=g, device=DEV).to(BF) for h in (QH, KH, KH)]
        work.append((h3.h3_prompts_prepare(_offsets(lengths), QH, KH, D), x,
                     torch.empty(T, QH, D, dtype=BF, device=DEV)))

    def call(p, x, o):
        h3.h3_prompt_attention(p, BF, x[0], QH * D, x[1], KH * D, x[2], KH * D, 0.1, o, QH * D)

    alone = []
    for w in work:
        call(*w)
        alone.append(w[2].clone())
        w[2].zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    for _ in range(5):
        for s, w in zip(streams, work):
            with torch.cuda.stream(s):
                call(*w)
    torch.cuda.synchronize()
    for w, want in zip(work, alone):
        assert torch.equal(w[2], want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(*work[0])
    p, x, o = work[0]
    x[2].mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, alone[0] * 2)  # a doubled v doubles every product and sum exactly


def test_no_prompts_and_empty_prompts():
    for offsets in ([0], [5], [3, 3, 3]):
        p = h3.h3_prompts_prepare(offsets, 4, 2, 64)
        o = torch.ones(8, 4, 64, dtype=BF, device=DEV)
        h3.h3_prompt_attention(p, BF, o, 256, o, 128, o, 128, 0.1, o, 256)
        assert bool((o == 1).all())


def test_refusals_of_the_call():
    L = h3.lib()
    p = h3.h3_prompts_prepare([0, 4], 4, 2, 64)
    x = torch.zeros(4, 4, 64, dtype=BF, device=DEV)
    ok, odd = ctypes.c_void_p(x.data_ptr()), ctypes.c_void_p(x.data_ptr() + 8)

    def call(type=0, q=ok, qs=256, k=ok, ks=128, v=ok, vs=128, scale=0.1, o=ok, os=256):
        return L.h3_prompt_attention(p.handle, type, q, qs, k, ks, v, vs, scale, o, os, None)

    for kw in (dict(type=2), dict(type=-1), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=math.inf), dict(scale=math.nan), dict(q=None), dict(k=None),
               dict(v=None), dict(o=None)):
        assert call(**kw) == h3.H3_ERR_ARG, kw
    for kw in (dict(qs=248), dict(qs=257), dict(ks=120), dict(vs=132), dict(os=255),
               dict(qs=1 << 39)):
        assert call(**kw) == h3.H3_ERR_SHAPE, kw
    for kw in (dict(q=odd), dict(k=odd), dict(v=odd), dict(o=odd)):
        assert call(**kw) == h3.H3_ERR_ALIGN, kw
    assert L.h3_prompt_attention(None, 0, ok, 256, ok, 128, ok, 128, 0.1, ok, 256,
                                 None) == h3.H3_ERR_ARG


@pytest.mark.parametrize("lengths", [[40], [40, 300]])
def test_rows_past_two_to_the_31_elements(lengths):
    """q and o rows so far apart that their offsets do not fit 32 bits: the short
    form and the other give what they give for dense rows."""
    QH, KH, D, T = 2, 1, 64, sum(lengths)
    stride = (2 ** 31 // (T - 8)) // 8 * 8
    g = gen(T)
    q = torch.randn(T, QH, D, generator=g, device=DEV).to(BF)
    k, v = (torch.randn(T, KH, D, generator=g, device=DEV).to(BF) for _ in range(2))
    far = torch.empty(T * stride, dtype=BF, device=DEV).view(T, stride)
    far[:, :QH * D] = q.view(T, -1)
    p = h3.h3_prompts_prepare(_offsets(lengths), QH, KH, D)
    dense = torch.empty_like(q)
    apart = torch.empty(T * stride, dtype=BF, device=DEV).view(T, stride)
    h3.h3_prompt_attention(p, BF, q, QH * D, k, KH * D, v, KH * D, 0.1, dense, QH * D)
    h3.h3_prompt_attention(p, BF, far, stride, k, KH * D, v, KH * D, 0.1, apart, stride)
    assert torch.equal(apart[:, :QH * D], dense.view(T, -1))
    assert h3.h3_text_error() == h3.H3_OK
