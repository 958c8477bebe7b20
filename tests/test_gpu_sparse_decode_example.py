"""The serving operators and the indexer together, as the example runs them."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "sparse_decode", os.path.join(ROOT, "examples", "sparse_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("requests,prompt,steps", [(3, 200, 70), (16, 4000, 5)])
def test_example(example, requests, prompt, steps):
    r = example.run(requests, prompt, steps)
    assert r["errors"] == [0, 0]
    # two eager steps, then the replays (a captured call does not run)
    assert r["cached"].tolist() == (r["prompt_lens"] + 2 + steps).tolist()
    # values are of order one: one bf16 rounding each side, and sums in another
    # order of the same positions
    assert r["covered"] > 0 and r["diff_covered"] <= 2 * 2.0 ** -8 * 4
    if prompt < example.TOPK:
        assert r["covered"] == requests
