"""The binding's own checks of the text model's operators, without a GPU."""

import pytest
import torch

from audio_generation_b200 import h3

BF = torch.bfloat16


def _calls():
    bf, codes, scales = torch.zeros(4, 4, 64, dtype=BF), torch.zeros(4, 256).char(), torch.ones(4)
    kc, vc = torch.zeros(2, 2, 32, 64).char(), torch.zeros(2, 2, 64, 32).char()
    ks, i32 = torch.zeros(2, 2), torch.zeros(4, dtype=torch.int32)
    cache = h3.h3_kv_cache(2, 32, 2, 64, 256, 256, 256, 256)
    return [
        (h3.h3_quantize_int8_rows, [BF, 4, 256, bf, 256, codes, scales]),
        (h3.h3_matmul_int8, [4, 4, 256, codes, scales, codes, scales, BF, bf, 4]),
        (h3.h3_prompt_attention, [h3.Prompts(None, 4), BF, bf, 256, bf, 128, bf, 128, 0.1, bf, 256]),
        (h3.make_kv_cache, [kc, vc, ks, ks]),
        (h3.h3_kv_cache_store, [cache, 1, 4, i32, 1, i32, i32, BF, bf, 128, bf, 128]),
        (h3.h3_cache_attention, [cache, 1, 4, i32, 1, i32, BF, bf, 256, 0.1, bf, 256, codes, 1024])]


@pytest.mark.skipif(torch.cuda.is_initialized(), reason="CUDA is in use in this process")
@pytest.mark.parametrize("call", range(6))
def test_host_tensors_are_refused_before_cuda_is_in_use(call, monkeypatch):
    """In every place, and before the library is called: it would take the address for
    device memory. (Other arguments are addresses, which nothing looks up.)"""
    class NoLibrary:
        h3_status_string = h3.lib().h3_status_string

        def __getattr__(self, name):
            def called(*args):
                raise AssertionError(name + " was called")
            return called
    monkeypatch.setattr(h3, "lib", NoLibrary)
    fn, args = _calls()[call]
    for i, a in enumerate(args):
        if not isinstance(a, torch.Tensor):
            continue
        if fn is h3.make_kv_cache:  # its shapes come from the tensors
            given = list(args)
        else:
            given = [256 if isinstance(b, torch.Tensor) and j != i else b
                     for j, b in enumerate(args)]
        if fn is h3.h3_kv_cache_store:
            given.append(4)  # rows
        with pytest.raises(h3.H3Error) as e:
            fn(*given)
        assert e.value.status == h3.H3_ERR_ARG and "cpu" in str(e.value)


def _pool(n=3, KH=2, BT=32, D=64):
    return [torch.zeros(n, KH, BT, D).char(), torch.zeros(n, KH, D, BT).char(),
            torch.zeros(n, KH), torch.zeros(n, KH)]


@pytest.mark.parametrize("which,other", [
    (0, lambda t: torch.zeros(3, 4, 32, 64).char()[:, ::2]),  # every other head of a larger pool
    (1, lambda t: torch.zeros(3, 2, 64, 64).char()[..., :32]),
    (1, lambda t: torch.zeros(3, 2, 32, 64).char().transpose(2, 3)),
    (0, lambda t: t.half()), (1, lambda t: t.float()),
    (2, lambda t: torch.ones(1, 2).expand(3, 2)), (3, lambda t: torch.ones(2, 3).t()),
    (2, lambda t: t.double()), (3, lambda t: t[:2]), (2, lambda t: torch.ones(3))])
def test_a_pool_that_is_not_what_its_sizes_say_is_refused(which, other, monkeypatch):
    """Strides that the library cannot know, and tensors that end before it does."""
    monkeypatch.setattr(h3, "_current_device", lambda: -1)  # let host tensors pass
    pool = _pool()
    assert h3.make_kv_cache(*pool).n_blocks == 3
    pool[which] = other(pool[which])
    with pytest.raises(h3.H3Error) as e:
        h3.make_kv_cache(*pool)
    assert e.value.status == h3.H3_ERR_SHAPE


@pytest.mark.parametrize("offsets", [[0, 2 ** 32 + 4], [2 ** 32, 2 ** 32 + 4], [0, 5, 2 ** 33 + 9]])
def test_offsets_past_int32_are_refused(offsets, monkeypatch):
    class NoLibrary:
        h3_status_string = h3.lib().h3_status_string

        @staticmethod
        def h3_prompts_prepare(*args):
            raise AssertionError("called with other offsets")
    monkeypatch.setattr(h3, "lib", NoLibrary)
    with pytest.raises(h3.H3Error) as e:
        h3.h3_prompts_prepare(offsets, 4, 2, 64)
    assert e.value.status == h3.H3_ERR_LAYOUT
