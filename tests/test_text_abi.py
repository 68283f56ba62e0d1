"""Refusals of the text model's operators: every bad argument is answered on the
host, before any device work (the pointers here are never dereferenced)."""

import ctypes
import os
import re

import pytest

from audio_generation_b200 import h3

P = ctypes.c_void_p(256)
ODD = ctypes.c_void_p(264)


def _quantize(type=h3.H3_BF16, rows=4, K=64, x=P, stride=64, codes=P, scales=P):
    return h3.lib().h3_quantize_int8_rows(type, rows, K, x, stride, codes, scales, None)


@pytest.mark.parametrize("kw,status", [
    (dict(type=3), h3.H3_ERR_ARG), (dict(type=-1), h3.H3_ERR_ARG), (dict(rows=-1), h3.H3_ERR_ARG),
    (dict(K=0), h3.H3_ERR_ARG), (dict(x=None), h3.H3_ERR_ARG), (dict(codes=None), h3.H3_ERR_ARG),
    (dict(scales=None), h3.H3_ERR_ARG), (dict(K=72, stride=72), h3.H3_ERR_SHAPE),
    (dict(stride=56), h3.H3_ERR_SHAPE), (dict(stride=68), h3.H3_ERR_SHAPE),
    (dict(x=ODD), h3.H3_ERR_ALIGN), (dict(codes=ODD), h3.H3_ERR_ALIGN),
    (dict(scales=ODD), h3.H3_ERR_ALIGN), (dict(rows=0, x=None), h3.H3_OK)])
def test_quantize_refusals(kw, status):
    assert _quantize(**kw) == status


def _matmul(M=4, N=8, K=64, a=P, sa=P, w=P, sw=P, type=h3.H3_F16, out=P, stride=8):
    return h3.lib().h3_matmul_int8(M, N, K, a, sa, w, sw, type, out, stride, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), h3.H3_ERR_ARG), (dict(N=-1), h3.H3_ERR_ARG), (dict(K=0), h3.H3_ERR_ARG),
    (dict(type=7), h3.H3_ERR_ARG), (dict(a=None), h3.H3_ERR_ARG), (dict(sa=None), h3.H3_ERR_ARG),
    (dict(w=None), h3.H3_ERR_ARG), (dict(sw=None), h3.H3_ERR_ARG), (dict(out=None), h3.H3_ERR_ARG),
    (dict(K=24), h3.H3_ERR_SHAPE), (dict(K=131072), h3.H3_ERR_SHAPE),
    (dict(M=2 ** 30 + 1), h3.H3_ERR_SHAPE),
    (dict(N=2 ** 30 + 1, stride=2 ** 31), h3.H3_ERR_SHAPE),
    (dict(stride=7), h3.H3_ERR_SHAPE), (dict(a=ODD), h3.H3_ERR_ALIGN),
    (dict(sa=ODD), h3.H3_ERR_ALIGN), (dict(w=ODD), h3.H3_ERR_ALIGN),
    (dict(sw=ODD), h3.H3_ERR_ALIGN), (dict(out=ODD), h3.H3_ERR_ALIGN),
    (dict(M=0, a=None), h3.H3_OK), (dict(N=0, w=None), h3.H3_OK)])
def test_matmul_refusals(kw, status):
    assert _matmul(**kw) == status


def test_binding_names_types_by_torch_dtype():
    import torch
    assert [h3._type(t) for t in (torch.bfloat16, torch.float16, torch.float32)] == [0, 1, 2]
    assert h3._type(torch.float64) == -1
    with pytest.raises(h3.H3Error):
        h3.h3_quantize_int8_rows(torch.float64, 1, 16, 256, 16, 256, 256, stream=0)


def _prepare(offsets=(0, 5), n=None, q=8, kv=2, D=128, out=True):
    arr = (ctypes.c_int32 * len(offsets))(*offsets)
    p = ctypes.c_void_p()
    return h3.lib().h3_prompts_prepare(arr, len(offsets) - 1 if n is None else n, q, kv, D,
                                       ctypes.byref(p) if out else None)


@pytest.mark.parametrize("kw,status", [
    (dict(out=False), h3.H3_ERR_ARG), (dict(n=-1), h3.H3_ERR_ARG), (dict(q=0), h3.H3_ERR_ARG),
    (dict(kv=0), h3.H3_ERR_ARG), (dict(kv=3), h3.H3_ERR_SHAPE),
    (dict(q=258, kv=2), h3.H3_ERR_SHAPE), (dict(D=96), h3.H3_ERR_SHAPE),
    (dict(D=0), h3.H3_ERR_SHAPE), (dict(offsets=(-1, 5)), h3.H3_ERR_LAYOUT),
    (dict(offsets=(0, 5, 4)), h3.H3_ERR_LAYOUT),
    (dict(offsets=(0, 2147483647, -2147483648)), h3.H3_ERR_LAYOUT)])
def test_prompts_refusals(kw, status):
    assert _prepare(**kw) == status


def test_prompts_null_arguments():
    L = h3.lib()
    p = ctypes.c_void_p()
    assert L.h3_prompts_prepare(None, 0, 8, 2, 128, ctypes.byref(p)) == h3.H3_ERR_ARG
    L.h3_prompts_destroy(None)
    assert L.h3_prompt_attention(None, 0, P, 8, P, 8, P, 8, 1.0, P, 8, None) == h3.H3_ERR_ARG
    with pytest.raises(h3.H3Error):
        h3.h3_prompts_prepare([], 8, 2, 128)


def _cache(n_blocks=4, block=64, kv=2, D=128, k=256, v=256, ks=256, vs=256):
    return h3.h3_kv_cache(n_blocks, block, kv, D, k, v, ks, vs)


_BAD_CACHES = [
    (dict(n_blocks=-1), h3.H3_ERR_ARG), (dict(kv=0), h3.H3_ERR_ARG),
    (dict(block=16), h3.H3_ERR_SHAPE), (dict(block=0), h3.H3_ERR_SHAPE),
    (dict(block=96), h3.H3_ERR_SHAPE), (dict(D=32), h3.H3_ERR_SHAPE),
    (dict(k=None), h3.H3_ERR_ARG), (dict(v=None), h3.H3_ERR_ARG), (dict(ks=None), h3.H3_ERR_ARG),
    (dict(vs=None), h3.H3_ERR_ARG), (dict(k=264), h3.H3_ERR_ALIGN), (dict(v=264), h3.H3_ERR_ALIGN),
    (dict(ks=264), h3.H3_ERR_ALIGN), (dict(vs=264), h3.H3_ERR_ALIGN)]


def _store(cache=None, n=2, most=3, table=P, width=4, lengths=P, offsets=P, type=h3.H3_BF16, rows=6,
           k=P, ks=256, v=P, vs=256):
    return h3.lib().h3_kv_cache_store(ctypes.byref(cache or _cache()), n, most, table, width,
                                      lengths, offsets, type, rows, k, ks, v, vs, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), h3.H3_ERR_ARG), (dict(most=-1), h3.H3_ERR_ARG), (dict(rows=-1), h3.H3_ERR_ARG),
    (dict(type=h3.H3_F32), h3.H3_ERR_ARG), (dict(type=9), h3.H3_ERR_ARG),
    (dict(width=-1), h3.H3_ERR_ARG), (dict(width=0), h3.H3_ERR_SHAPE),
    (dict(width=1 << 26), h3.H3_ERR_SHAPE), (dict(ks=248), h3.H3_ERR_SHAPE),
    (dict(vs=260), h3.H3_ERR_SHAPE), (dict(table=None), h3.H3_ERR_ARG),
    (dict(lengths=None), h3.H3_ERR_ARG), (dict(offsets=None), h3.H3_ERR_ARG),
    (dict(k=None), h3.H3_ERR_ARG), (dict(v=None), h3.H3_ERR_ARG), (dict(k=ODD), h3.H3_ERR_ALIGN),
    (dict(v=ODD), h3.H3_ERR_ALIGN), (dict(table=ODD), h3.H3_ERR_ALIGN),
    (dict(lengths=ODD), h3.H3_ERR_ALIGN), (dict(offsets=ODD), h3.H3_ERR_ALIGN),
    (dict(n=0, table=None), h3.H3_OK), (dict(most=0, k=None), h3.H3_OK),
    (dict(rows=0, k=None), h3.H3_OK)])
def test_store_refusals(kw, status):
    assert _store(**kw) == status


@pytest.mark.parametrize("kw,status", _BAD_CACHES)
def test_bad_caches(kw, status):
    assert _store(cache=_cache(**kw)) == status
    assert _attend(cache=_cache(**kw), ws_bytes=1 << 40) == status


def _attend(cache=None, n=2, q_heads=8, table=P, width=4, lengths=P, type=h3.H3_F16, q=P, qs=1024,
            scale=0.1, o=P, os=1024, ws=P, ws_bytes=1 << 30):
    return h3.lib().h3_cache_attention(ctypes.byref(cache or _cache()), n, q_heads, table, width,
                                       lengths, type, q, qs, scale, o, os, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), h3.H3_ERR_ARG), (dict(q_heads=0), h3.H3_ERR_ARG),
    (dict(type=h3.H3_F32), h3.H3_ERR_ARG), (dict(scale=0.0), h3.H3_ERR_ARG),
    (dict(scale=-0.1), h3.H3_ERR_ARG), (dict(scale=float("nan")), h3.H3_ERR_ARG),
    (dict(scale=float("inf")), h3.H3_ERR_ARG), (dict(width=-1), h3.H3_ERR_ARG),
    (dict(width=0), h3.H3_ERR_SHAPE), (dict(width=1 << 27), h3.H3_ERR_SHAPE),
    (dict(q_heads=7, qs=896, os=896), h3.H3_ERR_SHAPE), (dict(qs=1016), h3.H3_ERR_SHAPE),
    (dict(os=1028), h3.H3_ERR_SHAPE), (dict(table=None), h3.H3_ERR_ARG),
    (dict(lengths=None), h3.H3_ERR_ARG), (dict(q=None), h3.H3_ERR_ARG),
    (dict(o=None), h3.H3_ERR_ARG), (dict(ws=None), h3.H3_ERR_ARG),
    (dict(ws_bytes=16), h3.H3_ERR_WORKSPACE), (dict(q=ODD), h3.H3_ERR_ALIGN),
    (dict(o=ODD), h3.H3_ERR_ALIGN), (dict(ws=ODD), h3.H3_ERR_ALIGN),
    (dict(table=ODD), h3.H3_ERR_ALIGN), (dict(lengths=ODD), h3.H3_ERR_ALIGN),
    (dict(n=0, q=None), h3.H3_OK)])
def test_cache_attention_refusals(kw, status):
    assert _attend(**kw) == status


def test_cache_attention_workspace_size():
    c = _cache()
    size = h3.h3_cache_attention_workspace_size
    assert size(c, 0, 8, 9) == 0 == size(c, 1, 7, 9) == size(c, 1, 8, 0)
    # two parts of 8 rows of 128 sums and two statistics per range, at most three
    # ranges per SM whatever the number of sequences
    assert 0 < size(c, 1, 8, 1) < size(c, 2, 8, 40) < size(c, 40, 8, 375)
    assert size(c, 40, 8, 375) == size(c, 4000, 8, 375) <= 3 * 148 * (2 * 8 * (128 * 4 + 8) + 16)
    with pytest.raises(h3.H3Error) as e:
        import torch
        h3.make_kv_cache(torch.zeros(1, 1, 32, 64), torch.zeros(1, 1, 32, 64), None, None)
    assert e.value.status == h3.H3_ERR_SHAPE


def test_binding_refuses_values_of_the_wrong_device():
    """Where CUDA is in use a host tensor is refused by the binding; where it is not
    (device -1 on both sides) the address goes to the library's own checks."""
    import torch
    x = torch.zeros(64)
    with pytest.raises(h3.H3Error) as e:
        h3._dev_ptr(x, 0, "somewhere")
    assert e.value.status == h3.H3_ERR_ARG and "somewhere" in str(e.value)
    assert h3._dev_ptr(x, -1, "x") == x.data_ptr()
    assert h3._dev_ptr(None, 0, "x") is None and h3._dev_ptr(4096, 0, "x") == 4096


def test_exp2_cubic_of_prompt_attention():
    """The part of its exponentials on the FMA pipe, in the kernel's float32 steps
    with the coefficients its source has: within the bound stated there, exactly 0
    for masked keys, and a NaN as the largest number."""
    np = pytest.importorskip("numpy")
    src = open(os.path.join(os.path.dirname(h3.__file__), "csrc", "prompt_attention.cu")).read()
    c3, c2, c1, c0, magic, low = (
        np.float32(re.search(r"\b%s = (-?[\d.]+)f" % c, src).group(1))
        for c in ("kExpC3", "kExpC2", "kExpC1", "kExpC0", "kRoundMagic", "kExpLowest"))
    bound = float(re.search(r"relative error\n// \(([\de.-]+)\)", src).group(1))

    def fma(a, b, c):  # the float64 product of float32 operands is exact
        return (a.astype(np.float64) * b + np.float64(c)).astype(np.float32)

    def exp2(x):
        x = np.maximum(x, low)  # a NaN stays
        x = np.where(np.isnan(x), np.uint32(0x7fffffff).view(np.float32), x)  # as on the GPU
        t = x + magic
        f = x - (t - magic)
        p = fma(fma(fma(np.full_like(f, c3), f, c2), f, c1), f, c0)
        bits = p.view(np.int32).astype(np.int64) + (t.view(np.int32).astype(np.int64) << 23)
        return (bits & 0xFFFFFFFF).astype(np.uint32).view(np.float32)

    x = np.concatenate([np.linspace(-125, 15, 1400001),
                        np.linspace(-0.5, 0.5, 200001)]).astype(np.float32)
    rel = np.abs(exp2(x).astype(np.float64) / np.exp2(x.astype(np.float64)) - 1).max()
    assert 0.9 * bound < rel <= bound
    assert (exp2(np.array([-127, -128, -1e30, -np.inf], np.float32)) == 0).all()
    below = exp2(np.linspace(-127, -125, 100001).astype(np.float32))
    assert (below >= 0).all() and below.max() <= 2.0 ** -125 * 1.001
    assert exp2(np.array([np.nan], np.float32))[0] == np.finfo(np.float32).max
