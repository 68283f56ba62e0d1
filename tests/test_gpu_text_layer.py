"""The text model's operators run together, as a layer uses them: projections on
int8 codes, causal attention over packed prompts straight from the projection's
rows, keys and values into the 8-bit cache, then single tokens against the cache."""

import math

import pytest
import torch

from audio_generation_b200 import h3
from tests.text_testlib import DEV, gen

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
H, QH, KH, D, BT = 768, 10, 2, 64, 64
QKV = (QH + 2 * KH) * D
SCALE = 1 / math.sqrt(D)


class Linear:
    """A weight [N, K] as codes and channel scales, its input's buffers for M rows."""

    def __init__(self, w):
        self.w = w
        self.N, self.K = w.shape
        self.codes = torch.empty(self.N, self.K, dtype=torch.int8, device=DEV)
        self.scales = torch.empty(self.N, device=DEV)
        h3.h3_quantize_int8_rows(w.dtype, self.N, self.K, w, self.K, self.codes, self.scales)

    def __call__(self, x, out):
        M = x.shape[0]
        codes = torch.empty(M, self.K, dtype=torch.int8, device=DEV)
        scales = torch.empty(max(M, 4), device=DEV)
        h3.h3_quantize_int8_rows(x.dtype, M, self.K, x, x.stride(0), codes, scales)
        h3.h3_matmul_int8(M, self.N, self.K, codes, scales, self.codes, self.scales, out.dtype,
                          out, out.stride(0))
        return out


class Layer:
    def __init__(self, seed=0):
        g = gen(seed)
        self.qkv = Linear((torch.randn(QKV, H, generator=g, device=DEV) * H ** -0.5).to(BF))
        self.o = Linear((torch.randn(H, QH * D, generator=g, device=DEV) * (QH * D) ** -0.5).to(BF))

    @staticmethod
    def heads(rows):
        return (x.view(len(rows), -1, D) for x in rows.split([QH * D, KH * D, KH * D], 1))

    def prompts(self, x, offsets):
        rows = self.qkv(x, torch.empty(len(x), QKV, dtype=BF, device=DEV))
        q, k, v = self.heads(rows)
        att = torch.empty(len(x), QH, D, dtype=BF, device=DEV)
        p = h3.h3_prompts_prepare(offsets, QH, KH, D)
        h3.h3_prompt_attention(p, BF, q, QKV, k, QKV, v, QKV, SCALE, att, QH * D)
        y = self.o(att.view(len(x), -1), torch.empty(len(x), H, device=DEV))
        return rows, att, y

    def reference(self, x, offsets):
        """The layer in 64 bits on unrounded weights and activations."""
        rows = x.double() @ self.qkv.w.double().T
        q, k, v = self.heads(rows)
        att = torch.zeros(len(x), QH, D, dtype=torch.float64, device=DEV)
        for lo, hi in zip(offsets[:-1], offsets[1:]):
            kk, vv = (t[lo:hi].repeat_interleave(QH // KH, 1).transpose(0, 1) for t in (k, v))
            s = q[lo:hi].transpose(0, 1) @ kk.transpose(1, 2) * SCALE
            s.masked_fill_(torch.ones(hi - lo, hi - lo, dtype=torch.bool, device=DEV).triu(1),
                           -math.inf)
            att[lo:hi] = (torch.softmax(s, -1) @ vv).transpose(0, 1)
        return att.view(len(x), -1) @ self.o.w.double().T


def _rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def test_prompts_through_a_layer():
    """Normal rows of 768: an int8 step is the row's largest, about 3.2 of its
    deviations, over 127, so a rounding is off by 0.025 / sqrt(12) = 0.7 % of a
    deviation; two factors in each of the projections of q, k, v and o, and the
    weights moved by about 1.5 % through q and k: 0.7 % x sqrt(2 + 2 + 4) = 2 %."""
    offsets = [0, 37, 37, 167, 172, 500]
    x = torch.randn(offsets[-1], H, generator=gen(5), device=DEV).to(BF)
    layer = Layer()
    _, _, y = layer.prompts(x, offsets)
    assert _rel(y, layer.reference(x, offsets)) < 0.04
    assert h3.h3_text_error() == h3.H3_OK


def test_generation_continues_the_prompts():
    """After the prompts' keys and values have entered the cache, each generated
    token's attention is what the packed prompt attention gives for the prompt one
    token longer, but for the cache's 8 bits: a block's step is its largest value,
    about 4.3 deviations, over 127, so each rounding is off by 1 % of a deviation,
    in v and, through the weights, in k: 1.4 %, bounded by 4 %."""
    lengths = [37, 130, 5, 64]
    offsets = [0]
    for n in lengths:
        offsets.append(offsets[-1] + n)
    n, layer = len(lengths), Layer(1)
    x = torch.randn(offsets[-1], H, generator=gen(6), device=DEV).to(BF)
    rows, _, _ = layer.prompts(x, offsets)
    width, pool = 4, 4 * n + 1
    table = torch.randperm(pool, generator=gen(7), device=DEV)[:4 * n].to(torch.int32).view(n, 4)
    kc = torch.empty(pool, KH, BT, D, dtype=torch.int8, device=DEV)
    vc = torch.empty(pool, KH, D, BT, dtype=torch.int8, device=DEV)
    ks, vs = torch.empty(pool, KH, device=DEV), torch.empty(pool, KH, device=DEV)
    cache = h3.make_kv_cache(kc, vc, ks, vs)
    held = torch.zeros(n, dtype=torch.int32, device=DEV)
    _, k, v = layer.heads(rows)
    h3.h3_kv_cache_store(cache, n, max(lengths), table, width, held,
                         torch.tensor(offsets, dtype=torch.int32, device=DEV), BF, k, QKV, v, QKV)
    held += torch.tensor(lengths, dtype=torch.int32, device=DEV)

    token = torch.empty(n, H, dtype=BF, device=DEV)
    new = torch.empty(n, QKV, dtype=BF, device=DEV)
    att = torch.empty(n, QH, D, dtype=BF, device=DEV)
    y = torch.empty(n, H, device=DEV)
    need = h3.h3_cache_attention_workspace_size(cache, n, QH, width)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    one = torch.arange(n + 1, dtype=torch.int32, device=DEV)
    q1, k1, v1 = layer.heads(new)

    def step():
        layer.qkv(token, new)
        h3.h3_kv_cache_store(cache, n, 1, table, width, held, one, BF, k1, QKV, v1, QKV)
        held.add_(1)
        h3.h3_cache_attention(cache, n, QH, table, width, held, BF, q1, QKV, SCALE, att, QH * D,
                              ws, need)
        layer.o(att.view(n, -1), y)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    seqs = [[rows[a:b]] for a, b in zip(offsets[:-1], offsets[1:])]
    for i in range(70):  # through a block's end and into the next
        token.copy_(torch.randn(n, H, generator=gen(100 + i), device=DEV))
        graph.replay()
        for s in range(n):
            seqs[s].append(new[s:s + 1].clone())
        if i not in (0, 1, 26, 27, 69):
            continue
        packed = torch.cat([torch.cat(s) for s in seqs])
        ends = [0]
        for s in range(n):
            ends.append(ends[-1] + lengths[s] + i + 1)
        q, k, v = layer.heads(packed)
        full = torch.empty(len(packed), QH, D, dtype=BF, device=DEV)
        p = h3.h3_prompts_prepare(ends, QH, KH, D)
        h3.h3_prompt_attention(p, BF, q, QKV, k, QKV, v, QKV, SCALE, full, QH * D)
        last = torch.tensor(ends[1:], device=DEV) - 1
        for s in range(n):
            assert _rel(att[s], full[last[s]]) < 0.04, (i, s)
    assert held.tolist() == [m + 70 for m in lengths]
    assert h3.h3_text_error() == h3.H3_OK


def test_first_calls_may_be_captured(tmp_path):
    """A process whose first calls of every operator happen inside a capture."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
import torch
from audio_generation_b200 import h3
M, N, K, D = 5, 256, 256, 64
x = torch.randn(M, K, device="cuda").bfloat16()
c, s = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(8, device="cuda")
w, ws = torch.ones(N, K, dtype=torch.int8, device="cuda"), torch.ones(N, device="cuda")
out = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
p = h3.h3_prompts_prepare([0, 2, 5], 2, 1, D)
o = torch.zeros(M, 2, D, dtype=torch.bfloat16, device="cuda")
q = out.view(M, 4, D)
kc = torch.zeros(3, 1, 32, D, dtype=torch.int8, device="cuda")
vc = torch.zeros(3, 1, D, 32, dtype=torch.int8, device="cuda")
ks, vs = torch.zeros(4, 1, device="cuda")[:3], torch.zeros(4, 1, device="cuda")[:3]
table = torch.tensor([[0, 1], [2, -1]], dtype=torch.int32, device="cuda")
lens = torch.tensor([0, 0], dtype=torch.int32, device="cuda")
offs = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda")
cache = h3.make_kv_cache(kc, vc, ks, vs)
need = h3.h3_cache_attention_workspace_size(cache, 2, 2, 2)
wsp = torch.empty(need, dtype=torch.uint8, device="cuda")
got = torch.zeros(2, 2, D, dtype=torch.bfloat16, device="cuda")
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    h3.h3_quantize_int8_rows(x.dtype, M, K, x, K, c, s)
    h3.h3_matmul_int8(M, N, K, c, s, w, ws, out.dtype, out, N)
    h3.h3_prompt_attention(p, out.dtype, q, N, out[:, 128:], N, out[:, 192:], N, 0.1, o, 128)
    h3.h3_kv_cache_store(cache, 2, 3, table, 2, lens, offs, out.dtype, out[:, 128:], N,
                         out[:, 192:], N)
    lens.add_(offs.diff().int())
    h3.h3_cache_attention(cache, 2, 2, table, 2, lens, out.dtype, q[1::3], 3 * N, 0.1, got, 128,
                          wsp, need)
g.replay()
torch.cuda.synchronize()
assert h3.h3_text_error() == h3.H3_OK
ref = (x.double().sum(1))[:, None].expand(M, N)
# 256 roundings to a step of about 3.3 / 127: 0.0075 x 16 = 0.12 together
assert float((out.double() - ref).abs().max()) < 0.5
# q[1] and q[4] are the last tokens of the two sequences
want = torch.stack([o[1], o[4]]).double()
assert float((got.double() - want).abs().max()) < 0.02 * float(want.abs().max()) + 1e-3
print("captured")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                       timeout=120)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_host_tensors_are_refused():
    """Addresses that a kernel would fault on do not reach one: in every place of
    every call of the binding."""
    g = dict(device=DEV)
    bf = torch.zeros(4, 4, 64, dtype=BF, **g)
    codes, scales = torch.zeros(4, 256, dtype=torch.int8, **g), torch.ones(4, **g)
    kc, vc = torch.zeros(2, 2, 32, 64, dtype=torch.int8, **g), torch.zeros(2, 2, 64, 32,
                                                                          dtype=torch.int8, **g)
    ks = torch.zeros(2, 2, **g)
    i32 = torch.zeros(4, dtype=torch.int32, **g)
    p = h3.h3_prompts_prepare([0, 4], 4, 2, 64)
    cache = h3.make_kv_cache(kc, vc, ks, ks)
    ws = torch.empty(1 << 20, dtype=torch.uint8, **g)
    calls = [
        (h3.h3_quantize_int8_rows, [BF, 4, 256, bf, 256, codes, scales]),
        (h3.h3_matmul_int8, [4, 4, 256, codes, scales, codes, scales, BF, bf, 4]),
        (h3.h3_prompt_attention, [p, BF, bf, 256, bf, 128, bf, 128, 0.1, bf.clone(), 256]),
        (h3.make_kv_cache, [kc, vc, ks, ks]),
        (h3.h3_kv_cache_store, [cache, 1, 4, i32, 1, i32, i32, BF, bf, 128, bf, 128]),
        (h3.h3_cache_attention, [cache, 1, 4, i32, 1, i32, BF, bf, 256, 0.1, bf.clone(), 256, ws,
                                 1 << 20])]
    for fn, args in calls:
        for i, a in enumerate(args):
            if not isinstance(a, torch.Tensor):
                continue
            with pytest.raises(h3.H3Error) as e:
                fn(*args[:i], a.cpu(), *args[i + 1:])
            assert e.value.status == h3.H3_ERR_ARG
    torch.cuda.synchronize()
