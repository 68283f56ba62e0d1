"""Child process of tests/test_gpu_text_timeout.py (not collected by pytest).

Loads the test-only fault-injection build of the library given on the command
line and runs the named case with it; prints status codes and outputs as JSON.
"""

import ctypes
import json
import sys

import torch

BF = torch.bfloat16


def cache_case(h3):
    """So many short sequences that every range of the attention's work has several
    segments."""
    n, QH, KH, D, BT, width = 1500, 8, 2, 128, 64, 5
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    kc, vc = (torch.randint(-127, 128, s, generator=g, device="cuda", dtype=torch.int8)
              for s in ((40, KH, BT, D), (40, KH, D, BT)))
    ks, vs = (torch.rand(40, KH, generator=g, device="cuda") * 0.02 + 0.01 for _ in range(2))
    table = torch.randint(0, 40, (n, width), generator=g, device="cuda", dtype=torch.int32)
    lengths = torch.randint(1, width * BT + 1, (n,), generator=g, device="cuda", dtype=torch.int32)
    q = torch.randn(n, QH, D, generator=g, device="cuda").to(BF)
    cache = h3.make_kv_cache(kc, vc, ks, vs)
    need = h3.h3_cache_attention_workspace_size(cache, n, QH, width)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")

    def attend():
        o = torch.zeros_like(q)
        h3.h3_cache_attention(cache, n, QH, table, width, lengths, BF, q, QH * D, 0.1, o, QH * D,
                              ws, need)
        return h3.h3_text_error(), o.float().cpu().view(-1).view(torch.int32).tolist()[::97]

    return attend


def cache(h3, lib):
    lib.h3_test_cache_skip_unit.restype = ctypes.c_int
    lib.h3_test_cache_skip_unit.argtypes = [ctypes.c_int]
    attend, out = cache_case(h3), {}
    for unit in (0, 1, 2, 7):
        assert lib.h3_test_cache_skip_unit(unit) == 0
        out["skipped_%d" % unit] = attend()[0]
    assert lib.h3_test_cache_skip_unit(-1) == 0
    out["normal"], out["values"] = attend()
    return out


def prompt(h3, lib):
    """One prompt with an infinite v near its end: the rows computed again by plain
    arithmetic take far longer than a wait may."""
    T, D, at = 200000, 64, 199900
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    q, k, v = (torch.randn(T, 1, D, generator=g, device="cuda").to(BF) for _ in range(3))
    v[at, 0, 5] = float("inf")
    o = torch.zeros_like(q)
    p = h3.h3_prompts_prepare([0, T], 1, 1, D)
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    h3.h3_prompt_attention(p, BF, q, D, k, D, v, D, 0.125, o, D)
    b.record()
    status = h3.h3_text_error()
    bad = ~torch.isfinite(o[:, 0])
    want = torch.zeros_like(bad)
    want[at:, 5] = True
    v[at, 0, 5] = 0
    clean = torch.zeros_like(q)
    h3.h3_prompt_attention(p, BF, q, D, k, D, v, D, 0.125, clean, D)
    # the values are means of many: about 0.01, their weights rounded to 2^-8 or not
    diff = (o - clean).float().abs()[:, 0].masked_fill(want, 0)[8:]
    return {"status": status, "as_expected": bool(torch.equal(bad, want)),
            "again": h3.h3_text_error(), "diff": float(diff.max()), "ms": a.elapsed_time(b)}


def bits(x):
    return x.contiguous().view(-1).view(torch.int16).tolist()[::97]


def prompts_case(h3):
    QH, KH, D, lengths = 10, 2, 128, [900, 5, 700, 300]
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    T = sum(lengths)
    q, k, v = (torch.randn(T, n, D, generator=g, device="cuda").to(BF) for n in (QH, KH, KH))
    offsets = [sum(lengths[:i]) for i in range(5)]
    p = h3.h3_prompts_prepare(offsets, QH, KH, D)

    def attend():
        o = torch.zeros_like(q)
        h3.h3_prompt_attention(p, BF, q, QH * D, k, KH * D, v, KH * D, 0.1, o, QH * D)
        return h3.h3_text_error(), bits(o)
    return attend


def products_case(h3, M, N, K):
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    a, w = (torch.randint(-127, 128, (n, K), generator=g, device="cuda", dtype=torch.int8)
            for n in (M, N))
    sa, sw = (torch.rand(n, generator=g, device="cuda") * 0.01 for n in (M, N))

    def product():
        out = torch.zeros(M, N, dtype=BF, device="cuda")
        h3.h3_matmul_int8(M, N, K, a, sa, w, sw, BF, out, N)
        return h3.h3_text_error(), bits(out)
    return product


# by pairs of CTAs; few rows, with and without a shared K axis; turned
SHAPES = [(4000, 2048, 2048), (40, 40000, 2048), (16, 1024, 8192), (3000, 100, 8192)]


def skipping(call, setter):
    setter.restype, setter.argtypes = ctypes.c_int, [ctypes.c_int]
    out = {}
    for n in (0, 1, 5):
        assert setter(n) == 0
        out["skipped_%d" % n] = call()[0]
    assert setter(-1) == 0
    out["normal"], out["values"] = call()
    return out


def prompts(h3, lib):
    return skipping(prompts_case(h3), lib.h3_test_prompt_skip_keys)


def products(h3, lib):
    return [skipping(products_case(h3, *s), lib.h3_test_int8_skip_step) for s in SHAPES]


def main(lib_path: str, case: str) -> None:
    from audio_generation_b200 import h3
    h3.LIB_PATH = lib_path
    h3._lib = None
    cases = {"cache": cache, "prompt": prompt, "prompts": prompts, "products": products}
    print("RESULT " + json.dumps(cases[case](h3, h3.lib())))


if __name__ == "__main__":
    main(*sys.argv[1:])
