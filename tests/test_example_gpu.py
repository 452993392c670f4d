"""examples/sparse_decode.py: the serving operators together, captured in a
graph, each step checked against the definition."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "sparse_decode.py")


def test_sparse_decode():
    spec = importlib.util.spec_from_file_location("sparse_decode", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    module.main(requests=5, prompt=200, steps=5, k=64, heads=8, hidden=256, say=lambda *a: None)
