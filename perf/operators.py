"""Cases and plain forms of the text model's operators: the 8-bit integer linear
layer (h3_quantize_int8_rows, h3_matmul_int8), causal attention over packed
prompts (h3_prompt_attention), and the 8-bit key / value cache with the single-
token attention that reads it (h3_kv_cache_store, h3_cache_attention).

A case is a dict of plain values; its kind says which operator it runs. Lengths
of ragged cases are a function of the case alone (log-uniform between its
shortest and longest, from its "mix"), so that the work is known before any
input exists. Where `own` is false, run() computes the operators' formulas with
elementary torch operations; where it is true it makes a user's calls.
"""

import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # One generated token's activations entering the projections of a text
        # model of the transformer's text width (5120): latency is all that counts.
        {"name": "quantize-token", "kind": "quantize", "rows": 1, "K": 5120, "type": "bf16"},
        # The SwiGLU output of a batch of prompts (ffn 14336) before the down
        # projection: pure bandwidth.
        {"name": "quantize-prompts", "kind": "quantize", "rows": 8192, "K": 14336, "type": "bf16"},
        # One token through an up projection, text width 5120 to ffn 14336: the
        # 73 MB of codes are read for one row.
        {"name": "product-token", "kind": "product", "M": 1, "N": 14336, "K": 5120, "out": "bf16"},
        # f32 logits of 48 sequences over a vocabulary of odd size: few rows,
        # many columns, rows of the output not 16-byte aligned.
        {"name": "product-logits", "kind": "product", "M": 48, "N": 32003, "K": 5120, "out": "f32"},
        # A batch of prompts (odd row count) through hidden 5376 -> ffn 14336.
        {"name": "product-prompts", "kind": "product", "M": 8191, "N": 14336, "K": 5376,
         "out": "bf16"},
        # Captions of 3 to 77 tokens from many requests at once, a small text
        # model's heads (14 over 2, 64 wide).
        {"name": "prompts-captions", "kind": "prompts", "prompts": 64, "shortest": 3,
         "longest": 77, "mix": 1, "q_heads": 14, "kv_heads": 2, "D": 64, "type": "f16"},
        # Long instructions of different lengths, grouped heads in fives.
        {"name": "prompts-mixed", "kind": "prompts", "prompts": 12, "shortest": 120,
         "longest": 2500, "mix": 2, "q_heads": 40, "kv_heads": 8, "D": 128, "type": "bf16"},
        # One long context at the transformer's head count (56 x 128, grouped by 7).
        {"name": "prompts-long", "kind": "prompts", "prompts": 1, "shortest": 8192,
         "longest": 8192, "mix": 3, "q_heads": 56, "kv_heads": 8, "D": 128, "type": "bf16"},
        # A generation step: one new token of each sequence enters the cache.
        {"name": "store-step", "kind": "store", "seqs": 48, "shortest": 0, "longest": 3000,
         "new_least": 1, "new_most": 1, "mix": 4, "kv_heads": 8, "D": 128, "block": 64,
         "type": "bf16"},
        # Prompts entering the cache behind what is there already (shared
        # instructions), block borders anywhere.
        {"name": "store-prompts", "kind": "store", "seqs": 16, "shortest": 0, "longest": 700,
         "new_least": 200, "new_most": 4000, "mix": 5, "kv_heads": 8, "D": 128, "block": 64,
         "type": "bf16"},
        # One sequence alone: its 4001 cached tokens have to be spread over the chip.
        {"name": "cached-one", "kind": "cached", "seqs": 1, "shortest": 4001, "longest": 4001,
         "mix": 6, "q_heads": 40, "kv_heads": 8, "D": 128, "block": 64, "type": "bf16"},
        # A serving batch of very different lengths.
        {"name": "cached-many", "kind": "cached", "seqs": 40, "shortest": 500,
         "longest": 24000, "mix": 7, "q_heads": 40, "kv_heads": 8, "D": 128, "block": 64,
         "type": "bf16"},
    ]


def _log_int(rng, lo, hi):
    """A whole number in [lo, hi], spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    kind = rng.choice(["quantize", "product", "product", "prompts", "prompts", "store", "cached",
                       "cached"])
    heads = rng.choice([(8, 8), (14, 2), (16, 4), (32, 8), (40, 8), (56, 8), (24, 1)])
    width = rng.choice([64, 128])
    two = rng.choice(["bf16", "f16"])
    mix = rng.randrange(1 << 30)
    if kind == "quantize":
        K = 16 * _log_int(rng, 4, 896)
        t = rng.choice(["bf16", "f16", "f32"])
        return {"kind": kind, "K": K, "type": t,
                "rows": _log_int(rng, 1, min(16384, 352000000 // (K * (SIZE[t] + 1))))}
    if kind == "product":
        N, K = _log_int(rng, 1, 32003), 16 * _log_int(rng, 1, 896)
        most = max(1, min(8192, (8191 * 14336 * 5376) // (N * K)))
        return {"kind": kind, "M": _log_int(rng, 1, most), "N": N, "K": K,
                "out": rng.choice(["bf16", "f16", "f32"])}
    if kind == "prompts":
        longest = _log_int(rng, 1, 4500)
        shortest = _log_int(rng, 1, longest)
        most = max(1, min(96, (56 * 8192 * 8192) // (heads[0] * longest * longest),
                          16384 // longest))
        return {"kind": kind, "prompts": _log_int(rng, 1, most), "shortest": shortest,
                "longest": longest, "mix": mix, "q_heads": heads[0], "kv_heads": heads[1],
                "D": width, "type": two}
    block = rng.choice([32, 64, 128])
    if kind == "store":
        new = _log_int(rng, 1, 4000)
        longest = _log_int(rng, 1, 2500)
        most = max(1, min(64, 32768 // max(new, longest)))
        return {"kind": kind, "seqs": _log_int(rng, 1, most), "shortest": rng.choice([0, longest]),
                "longest": longest, "new_least": _log_int(rng, 1, new), "new_most": new,
                "mix": mix, "kv_heads": min(8, heads[1]), "D": width, "block": block, "type": two}
    longest = _log_int(rng, 1, 24000)
    most = max(1, min(128, 160000 // longest))
    return {"kind": kind, "seqs": _log_int(rng, 1, most), "shortest": _log_int(rng, 1, longest),
            "longest": longest, "mix": mix, "q_heads": heads[0], "kv_heads": heads[1], "D": width,
            "block": block, "type": two}


def _lengths(case, n, least, most, salt):
    """n lengths in [least, most], log-uniform, a function of the case; the
    first is `most`. A `least` of zero keeps its zero for about one in six."""
    rng = random.Random("%s/%s" % (case["mix"], salt))
    out = [most]
    for _ in range(n - 1):
        if least == 0 and rng.random() < 1 / 6:
            out.append(0)
        else:
            out.append(_log_int(rng, max(1, least), max(1, most)))
    rng.shuffle(out)
    return out


def _cache_shape(case):
    """Lengths before, new tokens, blocks of each sequence and of the pool."""
    n = case["seqs"]
    before = _lengths(case, n, case["shortest"], case["longest"], "before")
    new = ([0] * n if case["kind"] == "cached" else
           _lengths(case, n, case["new_least"], case["new_most"], "new"))
    blocks = [max(1, -(-(b + a) // case["block"])) for b, a in zip(before, new)]
    return before, new, blocks, sum(blocks) + 3


def _offsets(lengths):
    out = [0]
    for x in lengths:
        out.append(out[-1] + x)
    return out


def _activations(g, rows, K, dtype):
    """Normal values with a few channels an order of magnitude larger, as the
    inputs of a language model's projections have them."""
    x = torch.randn(rows, K, generator=g, device=DEV)
    gain = torch.ones(K, device=DEV)
    hot = torch.randint(0, K, (max(1, K // 256),), generator=g, device=DEV)
    gain[hot] = 12.0
    return (x * gain).to(dtype)


def _codes(g, *shape):
    return (torch.randn(*shape, generator=g, device=DEV) * 32).round_().clamp_(-127, 127).to(
        torch.int8)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    kind = case["kind"]
    s = {"case": case}
    if kind == "quantize":
        rows, K = case["rows"], case["K"]
        s["x"] = _activations(g, rows, K, TYPES[case["type"]])
        s["codes"] = torch.empty(rows, K, dtype=torch.int8, device=DEV)
        s["scales"] = torch.empty(rows, dtype=torch.float32, device=DEV)
        return s
    if kind == "product":
        M, N, K = case["M"], case["N"], case["K"]
        s["a"], s["w"] = _codes(g, M, K), _codes(g, N, K)
        s["a_scales"] = torch.rand(M, generator=g, device=DEV) * 0.05 + 0.01
        s["w_scales"] = torch.rand(N, generator=g, device=DEV) * 4e-4 + 1e-4
        s["out"] = torch.empty(M, N, dtype=TYPES[case["out"]], device=DEV)
        return s
    D, dtype, KH = case["D"], TYPES[case["type"]], case["kv_heads"]
    if kind == "prompts":
        lengths = _lengths(case, case["prompts"], case["shortest"], case["longest"], "prompts")
        T, QH = sum(lengths), case["q_heads"]
        # one projection's output: q, k and v are slices of its rows
        qkv = torch.randn(T, (QH + 2 * KH) * D, generator=g, device=DEV).to(dtype)
        s["q"], s["k"], s["v"] = (x.view(T, -1, D) for x in
                                  qkv.split([QH * D, KH * D, KH * D], dim=1))
        s["o"] = torch.empty(T, QH, D, dtype=dtype, device=DEV)
        s["offsets"] = torch.tensor(_offsets(lengths), dtype=torch.int32, device=DEV)
        s["n"], s["longest"] = len(lengths), max(lengths)
        if own:  # the handle a serving program makes once for a batch of prompts
            from audio_generation_b200 import h3
            s["handle"] = h3.h3_prompts_prepare(_offsets(lengths), QH, KH, D)
        return s
    before, new, blocks, pool = _cache_shape(case)
    n, BT = case["seqs"], case["block"]
    width = max(blocks)
    ids = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    slot = torch.arange(width, device=DEV)
    first = torch.tensor(_offsets(blocks)[:-1], device=DEV)
    used = slot < torch.tensor(blocks, device=DEV)[:, None]
    table = torch.where(used, ids[(first[:, None] + slot).clamp(max=pool - 1)], -1).to(torch.int32)
    s["table"] = table.contiguous()
    s["lengths"] = torch.tensor(before, dtype=torch.int32, device=DEV)
    s["k_codes"] = _codes(g, pool, KH, BT, D)
    s["v_codes"] = _codes(g, pool, KH, D, BT)
    s["k_scales"] = torch.rand(pool, KH, generator=g, device=DEV) * 0.02 + 0.02
    s["v_scales"] = torch.rand(pool, KH, generator=g, device=DEV) * 0.02 + 0.02
    s["n"], s["width"] = n, width
    if kind == "store":
        T = sum(new)
        s["k"] = torch.randn(T, KH, D, generator=g, device=DEV).to(dtype)
        s["v"] = torch.randn(T, KH, D, generator=g, device=DEV).to(dtype)
        s["offsets"] = torch.tensor(_offsets(new), dtype=torch.int32, device=DEV)
        s["most"] = max(new)
        return s
    QH = case["q_heads"]
    s["longest"] = max(before)
    s["q"] = torch.randn(n, QH, D, generator=g, device=DEV).to(dtype)
    s["o"] = torch.empty(n, QH, D, dtype=dtype, device=DEV)
    if own:  # the workspace a serving program keeps
        from audio_generation_b200 import h3
        cache = h3.make_kv_cache(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"])
        s["ws_bytes"] = h3.h3_cache_attention_workspace_size(cache, n, QH, width)
        s["ws"] = torch.empty(max(16, s["ws_bytes"]), dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------- plain forms

def _round_to_codes(x, scale):
    """rint(x / scale) in [-127, 127]. The quotient of two 32-bit values is
    taken in 64 bits, where it cannot round onto a tie it is not on."""
    return (x.double() / scale.double()).round_().clamp_(-127, 127).to(torch.int8)


def _a_127th(peak):
    """peak / 127 rounded to 32 bits. (Divided by a plain number, a 32-bit tensor
    is multiplied by the number's rounded reciprocal.)"""
    return (peak.double() / 127).float()


def _plain_quantize(s):
    x = s["x"].float()
    scale = _a_127th(x.abs().amax(1))
    scale = torch.where(scale > 0, scale, 1.0)
    return _round_to_codes(x, scale[:, None]), scale


def _plain_product(s):
    # sums of integer products past 2^24: in 64 bits they are exact
    acc = s["a"].double() @ s["w"].double().T
    return (acc * s["a_scales"].double()[:, None] * s["w_scales"].double()).to(s["out"].dtype)


def _plain_prompts(s, wide=torch.float32):
    """Every prompt padded to the longest, one masked softmax over all of them."""
    T, QH, D = s["q"].shape
    KH, n, L = s["k"].shape[1], s["n"], s["longest"]
    start, end = s["offsets"][:-1, None].long(), s["offsets"][1:, None].long()
    at = start + torch.arange(L, device=DEV)                     # [n, L] packed rows
    real = at < end
    at = at.clamp(max=T - 1)
    q = s["q"][at].to(wide).view(n, L, KH, QH // KH, D).permute(0, 2, 3, 1, 4)
    k = s["k"][at].to(wide).permute(0, 2, 3, 1)[:, :, None]      # [n, KH, 1, D, L]
    v = s["v"][at].to(wide).permute(0, 2, 1, 3)[:, :, None]      # [n, KH, 1, L, D]
    p = (q @ k).mul_(1 / math.sqrt(D))
    later = torch.ones(L, L, dtype=torch.bool, device=DEV).triu_(1)
    p.masked_fill_(later, -math.inf)
    p.sub_(p.amax(-1, keepdim=True)).exp_()
    norm = p.sum(-1, keepdim=True)
    o = (p @ v) / norm                                           # [n, KH, G, L, D]
    return o.permute(0, 3, 1, 2, 4).reshape(n, L, QH, D)[real].to(s["q"].dtype)


def _plain_store_one(s, x, codes, scales, by_token):
    """One of K and V. codes [pool, KH, block, D] where by_token, else transposed."""
    x = x.float()                                                # [T, KH, D]
    offsets, before = s["offsets"].long(), s["lengths"].long()
    T, n, BT = x.shape[0], s["n"], s["case"]["block"]
    seq = torch.repeat_interleave(torch.arange(n, device=DEV), offsets.diff(), output_size=T)
    pos = before[seq] + torch.arange(T, device=DEV) - offsets[seq]
    block, slot = s["table"][seq, pos // BT].long(), pos % BT
    peak = torch.zeros_like(scales)
    peak.index_reduce_(0, block, x.abs().amax(-1), "amax")
    touched = torch.zeros(len(scales), dtype=torch.bool, device=DEV)
    touched[block] = True
    # the block a sequence was in the middle of keeps its earlier tokens
    held = torch.zeros(len(scales), dtype=torch.int64, device=DEV)
    held.index_reduce_(0, s["table"].gather(1, (before // BT).clamp(max=s["width"] - 1)[:, None])
                       .view(-1).clamp(min=0).long(), before % BT, "amax")
    held = torch.where(touched, held, 0)
    new = torch.maximum(_a_127th(peak), torch.where(held[:, None] > 0, scales, 0.0))
    new = torch.where(new > 0, new, 1.0)
    new = torch.where(touched[:, None], new, scales)
    out = codes.clone() if by_token else codes.transpose(2, 3).contiguous()
    b = held.nonzero().view(-1)
    earlier = (torch.arange(BT, device=DEV) < held[b, None])[:, None, :, None]
    again = _round_to_codes(out[b].double() * scales[b, :, None, None].double(),
                            new[b, :, None, None])
    out[b] = torch.where(earlier, again, out[b])
    out[block, :, slot] = _round_to_codes(x, new[block][:, :, None])
    return out if by_token else out.transpose(2, 3).contiguous(), new


def _plain_store(s):
    kc, ks = _plain_store_one(s, s["k"], s["k_codes"], s["k_scales"], True)
    vc, vs = _plain_store_one(s, s["v"], s["v_codes"], s["v_scales"], False)
    return kc, vc, ks, vs


def _plain_cached(s, wide=torch.float32):
    n, QH, D = s["q"].shape
    KH, BT, L = s["k_codes"].shape[1], s["k_codes"].shape[2], s["width"] * s["k_codes"].shape[2]
    t = s["table"].clamp(min=0).long()                           # [n, width]
    k = s["k_codes"][t].to(wide).mul_(s["k_scales"][t].to(wide)[..., None, None])
    v = s["v_codes"][t].to(wide).mul_(s["v_scales"][t].to(wide)[..., None, None])
    k = k.permute(0, 2, 1, 3, 4).reshape(n, KH, L, D)
    v = v.permute(0, 2, 1, 4, 3).reshape(n, KH, L, D)
    q = s["q"].to(wide).view(n, KH, QH // KH, D)
    p = (q @ k.transpose(2, 3)).mul_(1 / math.sqrt(D))
    behind = torch.arange(L, device=DEV) >= s["lengths"][:, None]
    p.masked_fill_(behind[:, None, None], -math.inf)
    p.sub_(p.amax(-1, keepdim=True)).exp_()
    o = (p @ v) / p.sum(-1, keepdim=True)
    return o.view(n, QH, D).to(s["q"].dtype)


def run(s):
    kind = s["case"]["kind"]
    if not own:
        return {"quantize": _plain_quantize, "product": _plain_product, "prompts": _plain_prompts,
                "store": _plain_store, "cached": _plain_cached}[kind](s)
    from audio_generation_b200 import h3
    case = s["case"]
    if kind == "quantize":
        h3.h3_quantize_int8_rows(s["x"].dtype, case["rows"], case["K"], s["x"], case["K"],
                                 s["codes"], s["scales"])
        return s["codes"], s["scales"]
    if kind == "product":
        h3.h3_matmul_int8(case["M"], case["N"], case["K"], s["a"], s["a_scales"], s["w"],
                          s["w_scales"], s["out"].dtype, s["out"], case["N"])
        return s["out"]
    scale = 1 / math.sqrt(case["D"])
    if kind == "prompts":
        h3.h3_prompt_attention(s["handle"], s["q"].dtype, s["q"], s["q"].stride(0), s["k"],
                               s["k"].stride(0), s["v"], s["v"].stride(0), scale, s["o"],
                               s["o"].stride(0))
        return s["o"]
    cache = h3.make_kv_cache(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"])
    if kind == "store":
        h3.h3_kv_cache_store(cache, s["n"], s["most"], s["table"], s["width"], s["lengths"],
                             s["offsets"], s["k"].dtype, s["k"], s["k"].stride(0), s["v"],
                             s["v"].stride(0))
        return s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"]
    h3.h3_cache_attention(cache, s["n"], case["q_heads"], s["table"], s["width"], s["lengths"],
                          s["q"].dtype, s["q"], s["q"].stride(0), scale, s["o"],
                          s["o"].stride(0), s["ws"], s["ws_bytes"])
    return s["o"]


# ---------------------------------------------------------------- work, 64 bits

def work(case):
    kind = case["kind"]
    if kind == "quantize":
        n = case["rows"] * case["K"]
        return {"bytes": n * (SIZE[case["type"]] + 1) + 4 * case["rows"], "flops": 4 * n}
    if kind == "product":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K + N * K + 4 * (M + N) + M * N * SIZE[case["out"]],
                "flops": 2 * M * N * K}
    D, size, KH = case["D"], SIZE[case["type"]], case["kv_heads"]
    if kind == "prompts":
        lengths = _lengths(case, case["prompts"], case["shortest"], case["longest"], "prompts")
        return {"bytes": sum(lengths) * D * size * 2 * (case["q_heads"] + KH),
                "flops": sum(4 * D * case["q_heads"] * (x * (x + 1) // 2) for x in lengths)}
    before, new, blocks, pool = _cache_shape(case)
    if kind == "store":
        # new values read, their codes written, the touched blocks' scales; a
        # block begun earlier may have to be read and written again
        values = 2 * sum(new) * KH * D
        again = 2 * KH * D * sum(b % case["block"] for b, a in zip(before, new) if a)
        touched = sum(-(-(b + a) // case["block"]) - b // case["block"]
                      for b, a in zip(before, new) if a)
        return {"bytes": values * (size + 1) + 2 * again + 8 * KH * touched,
                "flops": 4 * (values + again)}
    tokens = sum(before)
    return {"bytes": 2 * tokens * KH * D + 2 * case["seqs"] * case["q_heads"] * D * size
            + 8 * KH * sum(blocks), "flops": 4 * tokens * case["q_heads"] * D}


def exact(case, seed):
    """The definitions in 64 bits, sequence by sequence and head by head."""
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "quantize":
        codes, scales = [], []
        for rows in s["x"].split(1024):
            top = (rows.abs().max(dim=1).values.double() / 127.0).float()  # held in 32 bits
            scale = torch.where(top > 0, top, torch.ones_like(top))
            ratio = rows.double() / scale.double().unsqueeze(1)
            codes.append(torch.round(ratio).clamp(-127, 127).to(torch.int8))
            scales.append(scale.double())
        return torch.cat(codes), torch.cat(scales)
    if kind == "product":
        w = s["w"].double() * s["w_scales"].double().unsqueeze(1)
        return torch.cat([(rows.double() * sc.double().unsqueeze(1)) @ w.T for rows, sc in
                          zip(s["a"].split(2048), s["a_scales"].split(2048))])
    scale = 1.0 / math.sqrt(case["D"])
    if kind == "prompts":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        group = case["q_heads"] // case["kv_heads"]
        edges = s["offsets"].tolist()
        for lo, hi in zip(edges[:-1], edges[1:]):
            for h in range(case["q_heads"]):
                k, v = (s[x][lo:hi, h // group].double() for x in ("k", "v"))
                for r in range(lo, hi, 4096):
                    q = s["q"][r:min(hi, r + 4096), h].double()
                    row = torch.arange(r, r + len(q), device=DEV)
                    sc = (q @ k.T * scale).where(
                        torch.arange(lo, hi, device=DEV) <= row[:, None], -math.inf)
                    out[r:r + len(q), h] = torch.softmax(sc, dim=1) @ v
        return out
    table, lengths = s["table"].tolist(), s["lengths"].tolist()
    BT, KH = case["block"], case["kv_heads"]
    if kind == "store":
        got = []
        edges = s["offsets"].tolist()
        for name, swap in (("k", False), ("v", True)):
            codes, scales = s[name + "_codes"].clone(), s[name + "_scales"].clone()
            if swap:
                codes = codes.transpose(2, 3).contiguous()
            for i in range(case["seqs"]):
                x, p = s[name][edges[i]:edges[i + 1]].double(), lengths[i]
                while len(x):
                    b, at = table[i][p // BT], p % BT
                    part, x = x[:BT - at], x[BT - at:]
                    top = (part.abs().amax(dim=(0, 2)) / 127.0).float()  # [KH], held in 32 bits
                    if at:
                        top = torch.maximum(top, scales[b])
                    top = torch.where(top > 0, top, torch.ones_like(top))
                    wide = top.double()[:, None, None]
                    if at:
                        old = codes[b, :, :at].double() * scales[b].double()[:, None, None]
                        codes[b, :, :at] = torch.round(old / wide).clamp(-127, 127).to(torch.int8)
                    ratio = part.permute(1, 0, 2) / wide
                    codes[b, :, at:at + len(part)] = torch.round(ratio).clamp(-127, 127).to(
                        torch.int8)
                    scales[b] = top
                    p += len(part)
            got += [codes.transpose(2, 3).contiguous() if swap else codes, scales.double()]
        return got[0], got[2], got[1], got[3]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    for i, L in enumerate(lengths):
        ids = torch.tensor(table[i][:-(-L // BT)], device=DEV)
        k = (s["k_codes"][ids].double() * s["k_scales"][ids].double()[..., None, None])
        v = (s["v_codes"][ids].double() * s["v_scales"][ids].double()[..., None, None])
        k = k.transpose(0, 1).reshape(KH, -1, case["D"])[:, :L]
        v = v.permute(1, 0, 3, 2).reshape(KH, -1, case["D"])[:, :L]
        q = s["q"][i].double().view(KH, -1, case["D"])
        out[i] = (torch.softmax(q @ k.transpose(1, 2) * scale, dim=-1) @ v).view(-1, case["D"])
    return out
