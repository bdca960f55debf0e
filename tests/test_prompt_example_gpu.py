"""The prompt example's calls together: in both layers the last piece's rows and the last token attend as the float64
oracle does over the cache, and the first layer's cache is the same whatever the prompt is cut into, but for codes next to
a border: the projection of another number of rows may round an FP16 value the other way (2^-11 of it), which moves less
than one code in a hundred."""
import importlib.util
import os

import numpy as np
import pytest

from gpu_util import host
from oracle import rope
from test_kv4_chunk_gpu import _compare

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "prompt.py")
    spec = importlib.util.spec_from_file_location("prompt_example", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    return example


def _attends(ex, layer, q, heads, n, sinks):
    rows = q.shape[0]
    ref = rope.chunks(q.cpu().numpy(), layer["cache"].cpu().numpy(), layer["table"].cpu().numpy(), [n], [0, rows], ex.K_SCALE,
                      ex.V_SCALE, ex.DIM ** -0.5, layer["window"], sinks)
    _compare(host(heads), ref["lse"], ref, ex.DIM, np.ones(rows, bool))


@pytest.mark.parametrize("prompt,piece", [(100, 100), (100, 33), (100, 1), (1, 1), (70, 64)])
def test_a_prompt_in_pieces(prompt, piece):
    ex = _example()
    got = ex.serve(prompt, piece, tokens=3, window=24, sinks=4)
    assert len(got["picked"]) == 3
    last = (prompt - 1) // piece * piece
    for layer in got["layers"]:
        q, heads = layer["last"]
        assert q.shape[0] == prompt - last
        _attends(ex, layer, q, heads, prompt, 4)
        q, heads = layer["token"]
        _attends(ex, layer, q, heads, prompt + 3, 4)
    whole = ex.serve(prompt, prompt, tokens=0, window=24, sinks=4)["layers"][0]
    again = ex.serve(prompt, piece, tokens=0, window=24, sinks=4)["layers"][0]
    assert float((whole["cache"] != again["cache"]).float().mean()) < 0.01
