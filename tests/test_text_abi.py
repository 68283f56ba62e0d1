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
