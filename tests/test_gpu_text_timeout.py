"""Bounded waits of the text model's operators that run out: the call returns, the
error is reported, and the next call is served as ever. With the test-only build
of the library (50 ms wait limit; an entry point that leaves copies out, so that
nothing completes the barrier a wait is on), in a child process."""

import json
import os
import subprocess
import sys

import pytest

from audio_generation_b200 import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def child(tmp_path_factory):
    lib = B.build_fault_injection(str(tmp_path_factory.mktemp("lib") / "libh3_fault_injection.so"))

    def run(case):
        r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "text_fault_child.py"), lib,
                            case], cwd=ROOT, capture_output=True, text=True, timeout=300,
                           env=dict(os.environ, PYTHONPATH=ROOT))
        line = [l for l in r.stdout.splitlines() if l.startswith("RESULT ")]
        assert r.returncode == 0 and line, r.stderr[-3000:]
        return json.loads(line[0][len("RESULT "):])
    return run


def test_a_cache_block_that_does_not_come(child):
    """Copies left out for the first, the second or a later unit of every range, so
    that the wait of one team of warps runs out in a segment which others follow."""
    from audio_generation_b200 import h3
    from tests.text_fault_child import cache_case
    res = child("cache")
    for unit in (0, 1, 2, 7):
        assert res["skipped_%d" % unit] == h3.H3_ERR_TIMEOUT
    assert res["normal"] == h3.H3_OK
    status, values = cache_case(h3)()  # the product library on the same inputs: the same bits
    assert status == h3.H3_OK and values == res["values"]


def test_rows_computed_again_do_not_let_a_wait_run_out(child):
    """A bad v near the end of 200000 tokens, so that the rows of its tile before it
    have to be computed again, under a limit of 50 ms for a wait: at about 50 cycles a
    key the rows of a warp take longer than that. Rows of eight tokens and more: a
    product's weights are rounded to 2^-8 of each, |v| is below 6, and both results
    to 2^-8 of at most 3."""
    from audio_generation_b200 import h3
    res = child("prompt")
    assert res["status"] == h3.H3_OK and res["again"] == h3.H3_OK
    assert res["as_expected"] and res["diff"] < 6 * 2.0 ** -8 + 2 * 3 * 2.0 ** -8
    assert res["ms"] > 50


def _check_skipped(res, again):
    from audio_generation_b200 import h3
    for n in (0, 1, 5):
        assert res["skipped_%d" % n] == h3.H3_ERR_TIMEOUT, n
    assert res["normal"] == h3.H3_OK
    status, values = again()  # the product library on the same inputs: the same bits
    assert status == h3.H3_OK and values == res["values"]


def test_a_key_tile_that_does_not_come(child):
    """Prompt attention: other fetches are in flight when the wait runs out."""
    from audio_generation_b200 import h3
    from tests.text_fault_child import prompts_case
    _check_skipped(child("prompts"), prompts_case(h3))


def test_a_step_of_a_product_that_does_not_come(child):
    """Every form of the product of int8 codes, clusters that join their sums included."""
    from audio_generation_b200 import h3
    from tests.text_fault_child import SHAPES, products_case
    for shape, res in zip(SHAPES, child("products")):
        _check_skipped(res, products_case(h3, *shape))
