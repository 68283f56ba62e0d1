"""The int8 linear layer: row lengths on both sides of every choice of a block size,
and products with scales at the ends of float32's range."""

import pytest
import torch

from audio_generation_b200 import h3
from tests.text_testlib import DEV, STEP, assert_within, gen, rand_codes

pytestmark = pytest.mark.gpu
F32 = torch.float32
# few rows, with and without a shared K axis; turned; by pairs of CTAs
SHAPES = [(3, 300, 272), (40, 2000, 5120), (700, 10, 528), (2500, 640, 272)]


def _product(a, sa, w, sw):
    out = torch.empty(len(a), len(w), device=DEV)
    h3.h3_matmul_int8(len(a), len(w), a.shape[1], a, sa, w, sw, F32, out, len(w))
    return out, a.double() @ w.double().T


def _spread(g, n, low, high):
    """Powers of ten in [low, high] with both signs."""
    e = torch.rand(n, generator=g, device=DEV, dtype=torch.float64) * (high - low) + low
    sign = torch.randint(0, 2, (n,), generator=g, device=DEV) * 2 - 1
    return (10.0 ** e * sign).float()


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("ends", [((-44, -37), (-6, 34)), ((-6, 34), (-44, -37)),
                                  ((-30, 20), (-30, 20)), ((8, 36), (-30, -8)), ((-38, 38), (0, 0))])
def test_scales_far_from_one(M, N, K, ends):
    """Scales that are subnormal, huge, or whose product leaves float32 either way: a
    value is off by three half steps wherever it is a normal number, a subnormal
    one by a step of those too, and one past the range is infinite."""
    g = gen(M + N)
    a, w = rand_codes(g, M, K), rand_codes(g, N, K)
    sa, sw = _spread(g, M, *ends[0]), _spread(g, N, *ends[1])
    out, sums = _product(a, sa, w, sw)
    ref = sums * sa.double()[:, None] * sw.double()
    inside = ref.abs() < torch.finfo(F32).max * (1 - 4 * STEP[F32])
    assert int(inside.sum()) > 0.2 * inside.numel()
    assert_within(out[inside], ref[inside], ref[inside].abs() * 3.01 * STEP[F32] + 2.0 ** -149)
    beyond = ref.abs() > torch.finfo(F32).max * (1 + 4 * STEP[F32])
    assert torch.equal(out[beyond].double(), ref[beyond].sign() * float("inf"))


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_a_sum_of_zero_is_zero_whatever_its_scales(M, N, K):
    a = torch.zeros(M, K, dtype=torch.int8, device=DEV)
    w = rand_codes(gen(1), N, K)
    sa, sw = torch.full((M,), 1e30, device=DEV), torch.full((N,), 1e25, device=DEV)
    out, _ = _product(a, sa, w, sw)
    assert bool((out == 0).all())


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_nan_scales_reach_their_row_and_column(M, N, K):
    g = gen(2)
    a, w = rand_codes(g, M, K), rand_codes(g, N, K)
    sa, sw = torch.ones(M, device=DEV), torch.ones(N, device=DEV)
    sa[1] = sw[N - 1] = float("nan")
    out, sums = _product(a, sa, w, sw)
    nan = torch.zeros(M, N, dtype=torch.bool, device=DEV)
    nan[1] = nan[:, N - 1] = True
    assert torch.equal(torch.isnan(out), nan)
    assert torch.equal(out[~nan], sums[~nan].float())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, F32])
@pytest.mark.parametrize("vectors", [257, 512, 513, 767, 768, 769, 1023, 1024, 1025, 1536, 1537,
                                     1792, 2047, 2048, 2049])
def test_row_lengths_around_the_block_sizes(vectors, dtype):
    """Bit for bit, at and beside the numbers of 16-byte vectors where a form ends."""
    per = 16 // dtype.itemsize
    rows, K = 600, (vectors * per + 15) // 16 * 16
    x = torch.randn(rows, K, generator=gen(vectors), device=DEV).to(dtype)
    codes = torch.full((rows, K), 77, dtype=torch.int8, device=DEV)
    scales = torch.full((rows,), -7.0, device=DEV)
    h3.h3_quantize_int8_rows(dtype, rows, K, x, K, codes, scales)
    want = (x.double().abs().amax(1) / 127).float()
    assert torch.equal(scales, want)
    assert torch.equal(codes, (x.double() / want.double()[:, None]).round().to(torch.int8))
