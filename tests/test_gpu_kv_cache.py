"""The text model's 8-bit key / value cache: stored codes and scales bit for bit
against the definition in 64 bits, and attention over the cache against its
formula in 64 bits on the values the cache stands for."""

import math

import pytest
import torch

from audio_generation_b200 import h3
from tests.text_testlib import DEV, STEP, TINY, assert_within, gen, rand_codes

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Cache:
    """A pool and its tables; blocks are dealt out in a scrambled order."""

    def __init__(self, lengths, KH, D, BT, spare=0, seed=0, pool_extra=2):
        g = gen(seed + 17 * BT + D)
        self.BT, self.KH, self.D = BT, KH, D
        need = [max(1, -(-(n + spare) // BT)) for n in lengths]
        self.width = max(need)
        pool = sum(need) + pool_extra
        ids = torch.randperm(pool, generator=g, device=DEV).tolist()
        rows = []
        for n in need:
            rows.append([ids.pop() for _ in range(n)] + [-1] * (self.width - n))
        self.table = _i32(rows)
        self.kc = rand_codes(g, pool, KH, BT, D)
        self.vc = rand_codes(g, pool, KH, D, BT)
        self.ks = torch.rand(pool, KH, generator=g, device=DEV) * 0.02 + 0.01
        self.vs = torch.rand(pool, KH, generator=g, device=DEV) * 0.02 + 0.01
        self.lengths = _i32(lengths)
        self.c = h3.make_kv_cache(self.kc, self.vc, self.ks, self.vs)

    def values(self, seq, n):
        """k, v [KH, n, D] that the first n tokens of a sequence stand for, in 64 bits."""
        ids = self.table[seq, :-(-n // self.BT)].long() if n else self.table[seq, :0].long()
        k = self.kc[ids].double() * self.ks[ids].double()[:, :, None, None]
        v = self.vc[ids].double() * self.vs[ids].double()[:, :, None, None]
        return (k.transpose(0, 1).reshape(self.KH, -1, self.D)[:, :n],
                v.permute(1, 0, 3, 2).reshape(self.KH, -1, self.D)[:, :n])

    def store(self, counts, k, v, max_new=None, lengths=None, offsets=None, rows=None):
        if offsets is None:
            offsets = [0]
            for n in counts:
                offsets.append(offsets[-1] + n)
        h3.h3_kv_cache_store(self.c, len(counts), max(counts) if max_new is None else max_new,
                             self.table, self.width,
                             self.lengths if lengths is None else lengths, _i32(offsets), k.dtype,
                             k, k.stride(0), v, v.stride(0), rows)

    def attend(self, q, scale, ws=None):
        n, QH, _ = q.shape
        need = h3.h3_cache_attention_workspace_size(self.c, n, QH, self.width)
        if ws is None:
            ws = torch.full((need + 16,), 255, dtype=torch.uint8, device=DEV)
        o = torch.full_like(q, 5.0)
        h3.h3_cache_attention(self.c, n, QH, self.table, self.width, self.lengths, q.dtype, q,
                              q.stride(0), scale, o, o.stride(0), ws, need)
        return o


def _rounded(x, scale):
    return torch.round(x / scale).clamp(-127, 127).to(torch.int8)


def _store_formula(cache, codes, scales, counts, x, turned):
    """One of K and V by the definition, block by block in 64 bits."""
    codes, scales = codes.clone(), scales.clone()
    if turned:
        codes = codes.transpose(2, 3).contiguous()
    lengths, table = cache.lengths.tolist(), cache.table.tolist()
    row = 0
    for s, n in enumerate(counts):
        new, p = x[row:row + n].double(), lengths[s]
        row += n
        while len(new):
            b, at = table[s][p // cache.BT], p % cache.BT
            part, new = new[:cache.BT - at], new[cache.BT - at:]
            for h in range(cache.KH):
                top = float((part[:, h].abs().max() / 127).float())
                old = float(scales[b, h]) if at else 0.0
                scale = max(top, old)
                if scale == 0:
                    codes[b, h, at:at + len(part)] = 0
                else:
                    if scale > old and at:
                        codes[b, h, :at] = _rounded(codes[b, h, :at].double() * old, scale)
                    codes[b, h, at:at + len(part)] = _rounded(part[:, h], scale)
                scales[b, h] = scale
            p += len(part)
    return (codes.transpose(2, 3).contiguous() if turned else codes), scales


def _check_store(cache, counts, k, v):
    kc, ks = _store_formula(cache, cache.kc, cache.ks, counts, k, False)
    vc, vs = _store_formula(cache, cache.vc, cache.vs, counts, v, True)
    cache.store(counts, k, v)
    assert h3.h3_text_error() == h3.H3_OK
    assert torch.equal(cache.ks, ks) and torch.equal(cache.vs, vs)
    assert torch.equal(cache.kc, kc) and torch.equal(cache.vc, vc)


def _new(counts, KH, D, dtype, seed=3):
    g = gen(seed + sum(counts))
    return [torch.randn(sum(counts), KH, D, generator=g, device=DEV).to(dtype) for _ in range(2)]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D,BT", [(64, 32), (64, 64), (64, 128), (128, 32), (128, 64), (128, 128)])
def test_store(D, BT, dtype):
    """Every place in a block for a first and a last token, whole blocks, and the
    rest of the pool untouched."""
    lengths = [0, 1, BT - 1, BT, BT + 1, 3, 5, 2 * BT + 7, 0]
    counts = [1, 1, 1, 1, 2 * BT + 5, BT - 3, 0, BT, 3 * BT]
    cache = Cache(lengths, 3, D, BT, spare=3 * BT + 8)
    _check_store(cache, counts, *_new(counts, 3, D, dtype))


@pytest.mark.parametrize("n_seq", [3, 40, 257, 700])
def test_store_of_very_different_counts(n_seq):
    """Far fewer blocks than sequences times the largest number of tokens: nothing,
    one or a few tokens next to prompts of several blocks, at any place of a block;
    the rows of k and v go on behind the last sequence."""
    BT, D = 32, 64
    counts = [(0, 1, 2, 33)[i % 4] if i % 97 else 300 + i for i in range(n_seq)]
    lengths = [(0, 31, 32, 45)[(i // 4) % 4] for i in range(n_seq)]
    cache = Cache(lengths, 1, D, BT, spare=max(counts))
    k, v = _new(counts + [9], 1, D, BF)
    _check_store(cache, counts, k, v)


def test_store_reports_a_bad_sequence_among_very_different_counts():
    BT, D = 32, 64
    counts, lengths = [300, 1, 0, 40, 2], [5, 31, 7, 64, 0]
    cache = Cache(lengths, 2, D, BT, spare=300)
    k, v = _new(counts, 2, D, BF)
    want, scales = cache.kc, cache.ks
    for s in (0, 1, 2, 4):  # sequence 3 is left out
        part = [c if i == s else 0 for i, c in enumerate(counts)]
        row = sum(counts[:s])
        want, scales = _store_formula(cache, want, scales, part, k[row:row + counts[s]], False)
    cache.store(counts, k, v, lengths=_i32(lengths[:3] + [-1] + lengths[4:]))
    assert h3.h3_text_error() == h3.H3_ERR_LAYOUT
    assert torch.equal(cache.kc, want) and torch.equal(cache.ks, scales)


def test_store_token_by_token_grows_the_scale():
    """Forty single tokens, some far larger than all before: the earlier codes are
    rounded again, exactly once per growth."""
    cache = Cache([0, 30], 2, 64, 32, spare=48)
    for i in range(40):
        k, v = _new([1, 1], 2, 64, BF, seed=i)
        if i % 7 == 3:
            k, v = k * (i + 2), v * (i + 3)
        _check_store(cache, [1, 1], k, v)
        cache.lengths += 1


def test_storing_again_changes_nothing():
    cache = Cache([5, 70], 2, 128, 64, spare=100)
    k, v = _new([80, 90], 2, 128, HF)
    cache.store([80, 90], k, v)
    before = [x.clone() for x in (cache.kc, cache.vc, cache.ks, cache.vs)]
    cache.store([80, 90], k, v)
    assert all(torch.equal(a, b) for a, b in
               zip(before, (cache.kc, cache.vc, cache.ks, cache.vs)))


def test_store_zeros_then_values():
    """A block of zeros has scale 0 and takes the scale of what comes later."""
    cache = Cache([0], 1, 64, 32, spare=32)
    k, v = _new([3], 1, 64, BF)
    _check_store(cache, [3], k * 0, v * 0)
    b = int(cache.table[0, 0])
    assert float(cache.ks[b, 0]) == 0 == float(cache.vs[b, 0])
    cache.lengths += 3
    _check_store(cache, [3], k * 1e-3, v * 1e-3)
    assert 0 < float(cache.ks[b, 0]) < 1e-3


def test_store_non_finite_values_mark_their_block_and_head():
    cache = Cache([10], 2, 64, 32, spare=80)
    k, v = _new([60], 2, 64, BF)
    k[30, 1, 7] = float("inf")     # token 40: the second block
    v[2, 0, 0] = float("nan")      # token 12: the first
    cache.store([60], k, v)
    t = cache.table[0].tolist()
    bad_k = torch.isnan(cache.ks[t[:3]])
    bad_v = torch.isnan(cache.vs[t[:3]])
    assert bad_k.tolist() == [[False, False], [False, True], [False, False]]
    assert bad_v.tolist() == [[True, False], [False, False], [False, False]]
    assert int(cache.kc[t[1], 1].abs().max()) == 0
    assert int(cache.vc[t[0], 0, :, :32].abs().max()) == 0
    # more tokens in a marked block: it stays marked
    cache.lengths += 60
    k, v = _new([2], 2, 64, BF)
    cache.store([2], k, v)
    assert torch.isnan(cache.ks[t[1], 1])


def test_store_from_slices_of_one_projection():
    KH, D = 2, 128
    qkv = torch.randn(70, 10 * D, generator=gen(4), device=DEV).to(BF)
    k, v = qkv[:, 6 * D:8 * D].view(70, KH, D), qkv[:, 8 * D:].view(70, KH, D)
    cache = Cache([9, 0], KH, D, 64, spare=70)
    _check_store(cache, [50, 20], k, v)


def test_bad_tables_lengths_and_offsets_are_reported_and_touch_nothing_else():
    """Every kind of device-side nonsense that the calls check: the good sequence
    next to it is served as ever, the error is reported, nothing else is written."""
    KH, D, BT = 1, 64, 32
    for bad in ("table", "table_high", "negative", "too_long", "count", "offset", "rows"):
        cache = Cache([40, 40], KH, D, BT, spare=8)
        k, v = _new([4, 4], KH, D, BF)
        offsets, rows = [0, 4, 8], None
        if bad == "table":
            cache.table[0, 1] = -5
        elif bad == "table_high":
            cache.table[0, 1] = cache.kc.shape[0]
        elif bad == "negative":
            cache.lengths[0] = -3
        elif bad == "too_long":
            cache.lengths[0] = cache.width * BT - 2
        elif bad == "count":
            offsets = [-4, 4, 8]
        elif bad == "offset":
            offsets = [4, 0, 4]
        elif bad == "rows":
            offsets, rows = [8, 12, 16], 8
        good = None
        if bad not in ("rows",):
            lo = offsets[1]
            part = [x[lo:lo + 4] for x in (k, v)]
            good = Cache([40, 40], KH, D, BT, spare=8)
            good_k = _store_formula(good, good.kc, good.ks, [0, 4], part[0], False)
        before = [x.clone() for x in (cache.kc, cache.ks)]
        cache.store([4, 4], k, v, max_new=4, offsets=offsets, rows=rows)
        assert h3.h3_text_error() == h3.H3_ERR_LAYOUT, bad
        assert h3.h3_text_error() == h3.H3_OK
        want = good_k if good is not None else before
        assert torch.equal(cache.kc, want[0]) and torch.equal(cache.ks, want[1]), bad


def _attention_formula(cache, q, lengths, scale, skip=()):
    n, QH, D = q.shape
    o = torch.zeros(n, QH, D, dtype=torch.float64, device=DEV)
    a = torch.zeros_like(o)
    for s, L in enumerate(lengths):
        if L == 0:
            continue
        k, v = cache.values(s, L)
        keep = torch.ones(L, dtype=torch.bool, device=DEV)
        for (seq, page) in skip:
            if seq == s:
                keep[page * cache.BT:(page + 1) * cache.BT] = False
        k, v = k[:, keep], v[:, keep]
        qq = q[s].double().view(cache.KH, -1, D)
        w = torch.softmax(qq @ k.transpose(1, 2) * scale, -1)
        o[s] = (w @ v).view(QH, D)
        a[s] = (w @ v.abs()).view(QH, D)
    return o, a


def _check_attention(lengths, QH, KH, D, BT, dtype, seed=0, scale=None, boost=1.0):
    cache = Cache(lengths, KH, D, BT, seed=seed)
    q = (torch.randn(len(lengths), QH, D, generator=gen(seed + QH), device=DEV) * boost).to(dtype)
    scale = scale or 1 / math.sqrt(D)
    o = cache.attend(q, scale)
    assert h3.h3_text_error() == h3.H3_OK
    ref, a = _attention_formula(cache, q, lengths, scale)
    # weights in fp16 (half a step, 2^-11), float32 scores of D terms (values
    # within 3, sum |q k| scale below 30: 128 x 2^-24 x 30 = 2.3e-4), one rounding
    assert_within(o, ref, a * (2.0 ** -11 + 2.4e-4) * boost
                  + ref.abs() * STEP[dtype] * 1.01 + 64 * TINY[dtype])
    return cache, q, o


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D,BT", [(64, 32), (64, 64), (64, 128), (128, 32), (128, 64), (128, 128)])
def test_attention_lengths(D, BT, dtype):
    lengths = [1, 2, 0, BT // 2, BT // 2 + 1, BT - 1, BT, BT + 1, 5 * BT + 3, 17 * BT, 1000, 2777]
    _check_attention(lengths, 10, 2, D, BT, dtype)


@pytest.mark.parametrize("QH,KH", [(1, 1), (8, 8), (7, 1), (16, 1), (17, 1), (40, 1), (128, 2),
                                   (24, 3)])
def test_attention_groups(QH, KH):
    """Groups that fill the rows of a product, that leave some idle, that take several."""
    _check_attention([300, 1, 65], QH, KH, 128, 64, BF)
    _check_attention([90, 700], QH, KH, 64, 32, HF)


@pytest.mark.parametrize("n_seq,length", [(1, 9001), (1, 64), (300, 70), (3, 20000)])
def test_attention_splits(n_seq, length):
    """Many ranges joined, one range, more sequences than the chip has room for."""
    rng = gen(length)
    lengths = torch.randint(1, length + 1, (n_seq,), generator=rng, device=DEV).tolist()
    lengths[-1] = length
    _check_attention(lengths, 4, 2, 128, 64, BF, seed=length)


@pytest.mark.parametrize("D,BT,QH", [(64, 32, 8), (128, 32, 20), (64, 64, 32), (128, 64, 8),
                                     (64, 128, 40), (128, 128, 12)])
def test_attention_many_blocks_per_range(D, BT, QH):
    """Every range runs through its ring and its list several times and through
    several sequences; repeated, since what could go wrong is a matter of timing."""
    KH = 4
    lengths = [(3 + 7 * i % 11) * 40 * BT + 13 * i for i in range(12)]
    cache, q, o = _check_attention(lengths, QH, KH, D, BT, BF, seed=D + BT)
    ws = torch.empty(h3.h3_cache_attention_workspace_size(cache.c, 12, QH, cache.width),
                     dtype=torch.uint8, device=DEV)
    for _ in range(30):
        again = cache.attend(q, 1 / math.sqrt(D), ws=ws)
        assert torch.equal(again, o)
    assert h3.h3_text_error() == h3.H3_OK


def test_attention_of_large_queries():
    """Scores up to about 60: their float32 error grows with them."""
    _check_attention([500, 40], 4, 2, 64, 64, BF, boost=8.0)


@pytest.mark.parametrize("order", [1, -1])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_attention_over_v_scales_far_apart(dtype, order):
    """Blocks whose V scales differ by up to all of float32's range, the smallest
    subnormal or zero, first or last: a token's weight counts whatever its value's
    size. Values are summed relative to the largest V scale: 2^-24 of that."""
    BT = 32
    lengths, QH, KH, D = [9 * BT - 5, 300 * BT], 5, 1, 64
    cache = Cache(lengths, KH, D, BT)
    factors = [1.0, 2.0 ** -7, 2.0 ** -9, 2.0 ** -14, 2.0 ** -20, 2.0 ** -31, 2.0 ** -80, 1e-39,
               0.0]
    for s, n in enumerate(lengths):
        blocks = cache.table[s, :-(-n // BT)].long()
        f = torch.tensor([factors[::order][i * len(factors) // len(blocks)]
                          for i in range(len(blocks))], device=DEV)
        cache.vs[blocks] *= f[:, None]
    q = torch.randn(2, QH, D, generator=gen(3), device=DEV).to(dtype)
    o = cache.attend(q, 0.125)
    ref, a = _attention_formula(cache, q, lengths, 0.125)
    largest = 127 * float(cache.vs.max())
    assert_within(o, ref, a * (2.0 ** -11 + 2.4e-4) + ref.abs() * STEP[dtype] * 1.01
                  + largest * 2.0 ** -24 + 64 * TINY[dtype])


def test_attention_is_the_same_every_time():
    cache, q, o = _check_attention([5000, 17, 2222], 8, 2, 128, 64, BF)
    for _ in range(5):
        assert torch.equal(cache.attend(q, 1 / math.sqrt(128)), o)


def test_attention_tiny_and_huge_queries():
    """Powers of two on q come out as they went in: the rows are scaled exactly."""
    cache = Cache([333], 1, 64, 64)
    q = torch.randn(1, 2, 64, generator=gen(2), device=DEV).to(BF)
    want = cache.attend(q, 0.125)
    for e in (-60, 40):
        got = cache.attend((q.float() * 2.0 ** e).to(BF), 0.125 * 2.0 ** -e)
        assert torch.equal(got, want)


def test_non_finite_queries_and_blocks():
    cache = Cache([200, 150], 2, 128, 64)
    q = torch.randn(2, 8, 128, generator=gen(1), device=DEV).to(BF)
    clean = cache.attend(q, 0.1)
    q2 = q.clone()
    q2[0, 3, 9] = float("inf")
    o = cache.attend(q2, 0.1)
    assert bool(torch.isnan(o[0, 3]).all())
    o[0, 3] = clean[0, 3]
    assert torch.equal(o, clean)
    # a marked block: NaN for the heads of its kv head, in its sequence only
    cache.vs[int(cache.table[1, 1]), 1] = float("nan")
    o = cache.attend(q, 0.1)
    assert bool(torch.isnan(o[1, 4:]).all())
    assert torch.equal(o[0], clean[0]) and torch.equal(o[1, :4], clean[1, :4])
    # behind the end of a sequence nothing is read: slots, scales, table entries
    cache = Cache([100], 1, 64, 32, spare=64)
    q = torch.randn(1, 4, 64, generator=gen(1), device=DEV).to(HF)
    clean = cache.attend(q, 0.1)
    cache.ks[cache.table[0, 4:].long()] = float("nan")
    cache.vs[cache.table[0, 4:].long()] = float("nan")
    last = int(cache.table[0, 3])
    cache.kc[last, :, 4:] = 99
    cache.vc[last, :, :, 4:] = 99
    assert torch.equal(cache.attend(q, 0.1), clean)
    cache.table[0, 4:] = -7
    assert torch.equal(cache.attend(q, 0.1), clean)
    assert h3.h3_text_error() == h3.H3_OK


def test_attention_with_bad_tables_and_lengths():
    """A block that does not exist counts as tokens that are not there; lengths are
    limited; both are reported."""
    lengths = [200, 100]
    cache = Cache(lengths, 1, 64, 32)
    q = torch.randn(2, 4, 64, generator=gen(6), device=DEV).to(BF)
    good = cache.table.clone()
    cache.table[0, 2] = cache.kc.shape[0]
    cache.table[0, 5] = -1
    o = cache.attend(q, 0.1)
    assert h3.h3_text_error() == h3.H3_ERR_LAYOUT
    cache.table.copy_(good)
    ref, a = _attention_formula(cache, q, lengths, 0.1, skip=[(0, 2), (0, 5)])
    assert_within(o, ref, a * (2.0 ** -11 + 2.4e-4) + ref.abs() * STEP[BF] * 1.01)
    cache.table[1, :] = -1
    o = cache.attend(q, 0.1)
    assert bool((o[1] == 0).all()) and h3.h3_text_error() == h3.H3_ERR_LAYOUT
    cache.table.copy_(good)
    full = cache.width * 32
    cache.lengths.copy_(_i32([full + 5, -9]))
    o = cache.attend(q, 0.1)
    assert h3.h3_text_error() == h3.H3_ERR_LAYOUT
    cache.lengths.copy_(_i32([full, 0]))
    assert torch.equal(o, cache.attend(q, 0.1)) and bool((o[1] == 0).all())
    assert h3.h3_text_error() == h3.H3_OK


def test_shared_blocks():
    """Sequences that share their first blocks (a common instruction)."""
    cache = Cache([160, 150, 140], 2, 64, 32)
    cache.table[1, :3] = cache.table[0, :3]
    cache.table[2, :4] = cache.table[0, :4]
    q = torch.randn(3, 6, 64, generator=gen(8), device=DEV).to(BF)
    o = cache.attend(q, 0.125)
    ref, a = _attention_formula(cache, q, [160, 150, 140], 0.125)
    assert_within(o, ref, a * (2.0 ** -11 + 2.4e-4) + ref.abs() * STEP[BF] * 1.01)


def test_cache_past_four_gigabytes():
    """Blocks whose codes start past 2^32 bytes."""
    KH, D, BT = 8, 128, 128
    pool = (2 ** 32 + 2 ** 27) // (KH * D * BT)
    kc = torch.empty(pool, KH, BT, D, dtype=torch.int8, device=DEV)
    vc = torch.empty(pool, KH, D, BT, dtype=torch.int8, device=DEV)
    ks, vs = (torch.zeros(pool, KH, device=DEV) for _ in range(2))
    cache = Cache([0], KH, D, BT, spare=300)
    cache.kc, cache.vc, cache.ks, cache.vs = kc, vc, ks, vs
    cache.c = h3.make_kv_cache(kc, vc, ks, vs)
    cache.table = _i32([[pool - 1, pool - 700, 5]])
    k, v = _new([300], KH, D, BF)
    cache.store([300], k, v)
    cache.lengths.copy_(_i32([300]))
    q = torch.randn(1, 16, D, generator=gen(8), device=DEV).to(BF)
    o = cache.attend(q, 0.1)
    got_k, got_v = cache.values(0, 300)
    for got, x in ((got_k, k), (got_v, v)):
        x = x.double().transpose(0, 1)
        # half a step of the largest value's 127th
        assert float((got - x).abs().max()) <= float(x.abs().max()) / 127 / 2 * 1.0001
    ref, a = _attention_formula(cache, q, [300], 0.1)
    assert_within(o, ref, a * (2.0 ** -11 + 2.4e-4) + ref.abs() * STEP[BF] * 1.01)


def test_streams_and_a_captured_step():
    """Store, raise the lengths and attend as one captured step, replayed; two
    caches at once on two streams."""
    KH, D, BT, QH = 2, 64, 32, 8
    cache = Cache([50, 0, 31], KH, D, BT, spare=12)
    twin = Cache([50, 0, 31], KH, D, BT, spare=12)
    k, v = _new([1, 1, 1], KH, D, BF)
    q = torch.randn(3, QH, D, generator=gen(1), device=DEV).to(BF)
    offsets = _i32([0, 1, 2, 3])
    o = torch.empty_like(q)
    need = h3.h3_cache_attention_workspace_size(cache.c, 3, QH, cache.width)
    ws = torch.empty(need + 16, dtype=torch.uint8, device=DEV)

    def step():
        h3.h3_kv_cache_store(cache.c, 3, 1, cache.table, cache.width, cache.lengths, offsets, BF,
                             k, k.stride(0), v, v.stride(0))
        cache.lengths.add_(1)
        h3.h3_cache_attention(cache.c, 3, QH, cache.table, cache.width, cache.lengths, BF, q,
                              QH * D, 0.125, o, QH * D, ws, need)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(8):
        nk, nv = _new([1, 1, 1], KH, D, BF, seed=50 + i)
        k.copy_(nk)
        v.copy_(nv)
        graph.replay()
        twin.store([1, 1, 1], nk, nv)
        twin.lengths += 1
        assert torch.equal(o, twin.attend(q, 0.125))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    want = twin.attend(q, 0.125)
    got = []
    torch.cuda.synchronize()
    for s, c in zip(streams, (cache, twin)):
        with torch.cuda.stream(s):
            got += [c.attend(q, 0.125) for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got)


def test_no_work():
    cache = Cache([3], 1, 64, 32)
    k, v = _new([0], 1, 64, BF)
    before = cache.kc.clone()
    cache.store([0], k, v)
    q = torch.empty(0, 2, 64, dtype=BF, device=DEV)
    h3.h3_cache_attention(cache.c, 0, 2, cache.table, 1, cache.lengths, BF, q, 128, 0.1, q, 128,
                          None, 0)
    assert torch.equal(before, cache.kc)
