"""Helpers shared by the tests of the text model's operators."""

from __future__ import annotations

import torch

DEV = "cuda"
STEP = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16, torch.float32)}
TINY = {t: torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2 for t in STEP}


def gen(seed: int) -> torch.Generator:
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def rand_codes(g, *shape):
    return torch.randint(-127, 128, shape, generator=g, device=DEV, dtype=torch.int8)


def assert_within(got, ref, allowed, what=""):
    """|got - ref| <= allowed elementwise; got finite, NaN never hides."""
    got = got.double()
    assert bool(torch.isfinite(got).all()), f"{what}: non-finite values"
    over = ((got - ref).abs() - allowed).amax().item() if got.numel() else 0.0
    assert over <= 0, f"{what}: {over:.3e} over the allowance"
