"""The tree decoding example: a tree step agrees with decoding its branch token
by token, through projections, plan, append and attention."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("cache", ["bf16", "s8"])
def test_tree_example(qmm, cuda, cache):
    spec = importlib.util.spec_from_file_location("tree_decode", os.path.join(ROOT, "examples", "tree_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.main(cache)
