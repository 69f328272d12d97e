"""The verify loop of examples/tree_verify.py keeps its workspaces: their number does not grow with the calls."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
def test_one_workspace_for_all_chunks_and_trees(monkeypatch, dtype):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_moe_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("tree_verify_workspaces", os.path.join(ROOT, "examples", "tree_verify.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    target, made, alloc = ex.Target(), [], ex.dfv.alloc_workspace
    monkeypatch.setattr(ex.dfv, "alloc_workspace", lambda n, *a, **k: made.append(n) or alloc(n, *a, **k))
    counts = []
    for chunk, steps in ((40, 1), (3, 5)):  # one chunk and one step, or 14 and five
        made.clear()
        server = ex.Server(target, [list(range(40)), list(range(25))], 32, 4, chunk=chunk, dtype=dtype)
        for _ in range(steps):
            tree, toks, pos = server.batch([[1, 2, 3], [4, 5]], [[1, 3, 7], [1, 3]])
            server.reserve(3)
            server.run(tree, toks, pos)
        counts.append(len(made))
    assert counts[0] == counts[1]
