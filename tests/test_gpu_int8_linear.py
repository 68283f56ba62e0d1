"""The text model's 8-bit integer linear layer against its formula in 64 bits:
codes and scales of quantized rows bit for bit, products of codes (whose integer
sums are exact) within the rounding of the scaling and of the output type."""

import pytest
import torch

from audio_generation_b200 import h3
from tests.text_testlib import DEV, STEP, TINY, assert_within, gen, rand_codes

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def _quantize(x, K, stride=None):
    rows = x.shape[0]
    codes = torch.full((rows, K), 77, dtype=torch.int8, device=DEV)
    scales = torch.full((rows,), -7.0, device=DEV)
    h3.h3_quantize_int8_rows(x.dtype, rows, K, x, stride or x.stride(0), codes, scales)
    return codes, scales


def _formula(x):
    x = x.double()
    scale = (x.abs().amax(1) / 127).float()  # 53 bits rounded to 24: the float32 quotient
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    return (x / scale.double()[:, None]).round().clamp(-127, 127).to(torch.int8), scale


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,K", [(1, 16), (3, 512), (9, 528), (5, 2048), (1, 5120), (7, 14336),
                                    (2, 32784), (2, 65552), (1, 131056), (0, 64), (700, 1024),
                                    (700, 4096), (650, 5120), (601, 14336), (599, 20480),
                                    (595, 65536)])
def test_codes_and_scales_bit_for_bit(dtype, rows, K):
    """Every group size and register count of the kernel, and its two-pass form."""
    x = (torch.randn(rows, K, generator=gen(K + rows), device=DEV) * 3).to(dtype)
    codes, scales = _quantize(x, K)
    want, ws = _formula(x)
    assert torch.equal(scales, ws) and torch.equal(codes, want)


@pytest.mark.parametrize("dtype", TYPES)
def test_ties_go_to_the_even_code(dtype):
    """Rows whose scale is a power of two times 127 / 127: every half is a tie."""
    half = torch.arange(-254, 255, device=DEV).float() / 2      # -127 .. 127 in halves
    x = torch.cat([half, torch.zeros(528 - half.numel(), device=DEV)])
    x = torch.stack([x, x * 0.25, x * 64]).to(dtype)
    codes, scales = _quantize(x, 528)
    assert torch.equal(scales, torch.tensor([1.0, 0.25, 64.0], device=DEV))
    want = half.double().round()                                # torch rounds ties to even
    for r in range(3):
        assert torch.equal(codes[r, :half.numel()].double(), want)


def test_small_and_empty_rows():
    x = torch.zeros(4, 64, device=DEV)
    x[1, 3], x[2, 5], x[3, 7] = 1e-45, 3e-38, 1e-37
    x[3, 8] = -5e-38
    codes, scales = _quantize(x, 64)
    want, ws = _formula(x)
    assert torch.equal(codes, want) and torch.equal(scales, ws)
    assert scales[0] == 1 and int(codes[0].abs().max()) == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_non_finite_row_is_marked_and_alone(dtype, bad):
    x = torch.randn(5, 1040, generator=gen(1), device=DEV).to(dtype)
    x[2, 1039] = bad
    codes, scales = _quantize(x, 1040)
    assert bool(torch.isnan(scales[2])) and int(codes[2].abs().max()) == 0
    keep = torch.tensor([0, 1, 3, 4], device=DEV)
    want, ws = _formula(x[keep])
    assert torch.equal(codes[keep], want) and torch.equal(scales[keep], ws)


@pytest.mark.parametrize("dtype", TYPES)
def test_strided_rows(dtype):
    wide = torch.randn(6, 400, generator=gen(2), device=DEV).to(dtype)
    x = wide[:, 16:16 + 272]
    codes, scales = _quantize(x, 272)
    want, ws = _formula(x.contiguous())
    assert torch.equal(codes, want) and torch.equal(scales, ws)


def _product(M, N, K, dtype, seed=0, stride=None, a=None, w=None):
    g = gen(seed + M + 7 * N + 13 * K)
    a = rand_codes(g, M, K) if a is None else a
    w = rand_codes(g, N, K) if w is None else w
    sa = torch.rand(M, generator=g, device=DEV) + 0.5
    sw = (torch.rand(N, generator=g, device=DEV) + 0.5) * 2.0 ** -14
    stride = stride or N
    out = torch.full((M, stride), -3.0, dtype=dtype, device=DEV)
    h3.h3_matmul_int8(M, N, K, a, sa, w, sw, dtype, out, stride)
    ref = (a.double() @ w.double().T) * sa.double()[:, None] * sw.double()
    # the sum's rounding to 24 bits, the scales' product, their product: 3 half
    # steps of float32, then the output type's
    allowed = ref.abs() * (3.01 * STEP[torch.float32]
                           + (0 if dtype == torch.float32 else STEP[dtype] * 1.001)) + TINY[dtype]
    assert_within(out[:, :N], ref, allowed, f"{M}x{N}x{K}")
    assert bool((out[:, N:] == -3).all())
    assert h3.h3_text_error() == h3.H3_OK


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 16), (1, 128, 128), (2, 129, 144), (15, 1000, 1040), (16, 14336, 5120), (17, 255, 2064),
    (32, 640, 14336), (33, 32003, 256), (64, 5376, 1024), (65, 100, 4096), (128, 384, 2560),
    (129, 256, 128), (256, 257, 528), (333, 1003, 5376), (700, 1, 64), (1025, 2048, 1040),
    (130, 1500, 5120), (513, 300, 5120), (1030, 129, 2064), (2048, 640, 1296), (2049, 3000, 272),
    (300, 19000, 512), (256, 5120, 2064), (144, 2559, 4112), (400, 2564, 5120), (1500, 1024, 4096)])
def test_product(M, N, K, dtype):
    _product(M, N, K, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", [
    (300, 1, 64), (2290, 10, 9040), (1000, 3, 14320), (4097, 17, 272), (129, 128, 528),
    (5000, 100, 144), (20001, 33, 48), (127, 9, 4096), (4517, 275, 224), (2392, 382, 16),
    (2051, 3001, 160), (4097, 64, 272), (3001, 128, 1040), (9000, 96, 2064)])
def test_product_of_many_rows_and_few_or_odd_columns(M, N, K, dtype):
    _product(M, N, K, dtype)


@pytest.mark.parametrize("stride", [10, 11, 16, 32])
def test_narrow_rows_of_out_apart(stride):
    _product(777, 10, 1040, torch.bfloat16, stride=stride)


@pytest.mark.parametrize("M", [5, 300])
@pytest.mark.parametrize("stride", [1001, 1008, 1537])
def test_rows_of_out_apart(M, stride):
    """Aligned and odd strides; what lies between the rows is left as it was."""
    _product(M, 1001, 272, torch.bfloat16, stride=stride)


@pytest.mark.parametrize("M", [3, 200])
def test_the_longest_sum_of_extremes(M):
    """K = 131056 products of -128 with -128: 2147221504 fits 32 bits, barely."""
    K, N = 131056, 130
    a = torch.full((M, K), -128, dtype=torch.int8, device=DEV)
    w = torch.full((N, K), -128, dtype=torch.int8, device=DEV)
    w[1::2] = 127
    _product(M, N, K, torch.float32, a=a, w=w)


def test_empty_products_touch_nothing():
    out = torch.ones(4, 4, device=DEV)
    one = torch.ones(16, device=DEV)
    codes = torch.ones(4, 16, dtype=torch.int8, device=DEV)
    h3.h3_matmul_int8(0, 4, 16, codes, one, codes, one, torch.float32, out, 4)
    h3.h3_matmul_int8(4, 0, 16, codes, one, codes, one, torch.float32, out, 4)
    assert bool((out == 1).all())


@pytest.mark.parametrize("M", [4, 260])
def test_a_marked_row_stays_alone(M):
    """A NaN scale makes its own row NaN and no other."""
    g = gen(3)
    a, w = rand_codes(g, M, 256), rand_codes(g, 300, 256)
    sa, sw = torch.ones(M, device=DEV), torch.ones(300, device=DEV)
    sa[2] = float("nan")
    out = torch.empty(M, 300, device=DEV)
    h3.h3_matmul_int8(M, 300, 256, a, sa, w, sw, torch.float32, out, 300)
    nan = torch.isnan(out)
    assert bool(nan[2].all()) and int(nan.sum()) == 300


@pytest.mark.parametrize("M", [1, 40, 777])
def test_linear_layer_on_a_stream_and_in_a_graph(M):
    """Quantize and product as a layer runs them: on a side stream, then captured
    and replayed on new inputs; both against the layer in 64 bits."""
    g = gen(9)
    K, N = 2048, 1536
    w = torch.randn(N, K, generator=g, device=DEV) * 0.05
    wc, ws = _quantize(w, K)
    x = torch.randn(M, K, generator=g, device=DEV).bfloat16()
    codes = torch.empty(M, K, dtype=torch.int8, device=DEV)
    scales = torch.empty(M, device=DEV)
    out = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)

    def layer():
        h3.h3_quantize_int8_rows(x.dtype, M, K, x, K, codes, scales)
        h3.h3_matmul_int8(M, N, K, codes, scales, wc, ws, out.dtype, out, N)

    def check():
        c, s = _formula(x)
        ref = (c.double() @ wc.double().T) * s.double()[:, None] * ws.double()
        assert_within(out, ref, ref.abs() * (STEP[torch.bfloat16] * 1.01) + 1e-30)
        # int8 steps: the layer itself is within a few percent of the real product
        full = x.double() @ w.double().T
        assert float((out.double() - full).norm() / full.norm()) < 0.03

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.synchronize()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    for seed in (1, 2):
        x.copy_(torch.randn(M, K, generator=gen(seed), device=DEV))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        check()


@pytest.mark.parametrize("M,N,stride", [
    (5, 40, 2 ** 29 + 8), (300, 40, 2 ** 23), (300, 600, 2 ** 23)])
def test_out_past_two_to_the_31_elements(M, N, stride):
    """Few rows, turned and by pairs: row offsets that do not fit 32 bits."""
    g = gen(M + N)
    a, w = rand_codes(g, M, 272), rand_codes(g, N, 272)
    sa, sw = torch.ones(M, device=DEV), torch.ones(N, device=DEV)
    whole = torch.empty(M * stride, dtype=torch.bfloat16, device=DEV)
    out = whole.view(M, stride)
    out[:, :N + 8] = -3
    h3.h3_matmul_int8(M, N, 272, a, sa, w, sw, torch.bfloat16, out, stride)
    ref = (a.double() @ w.double().T)
    assert torch.equal(out[:, :N], ref.float().to(torch.bfloat16))
    assert bool((out[:, N:N + 8] == -3).all())
