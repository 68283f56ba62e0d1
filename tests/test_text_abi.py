"""Refusals of the text model's operators: every bad argument is answered on the
host, before any device work (the pointers here are never dereferenced)."""

import ctypes

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
