"""The build's two parts: the C library, which needs nvcc alone, and the Python binding, which needs torch's headers and
is tied to the torch it was built against (CPU, with stand-ins for the compilers)."""
from __future__ import annotations

import os
import stat

import pytest

from speculative_decoding_moe_gb300 import build as b


@pytest.fixture
def scratch(tmp_path, monkeypatch):
    """Builds in tmp_path with compilers that only create their output."""
    tool = tmp_path / "tool"
    tool.write_text('#!/bin/sh\nwhile [ $# -gt 0 ]; do if [ "$1" = -o ]; then : > "$2"; fi; shift; done\n')
    tool.chmod(tool.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setattr(b, "NVCC", str(tool))
    monkeypatch.setenv("CXX", str(tool))
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libdfv.so"))
    monkeypatch.setattr(b, "BIND", str(tmp_path / "_dfvbind.so"))
    return tmp_path


def test_the_library_is_linked_where_the_binding_cannot_be_built(scratch, monkeypatch):
    monkeypatch.setenv("CXX", "false")
    assert not b.up_to_date()
    with pytest.raises(RuntimeError, match="binding"):
        b.build()
    assert os.path.exists(b.LIB) and not os.path.exists(b.BIND)
    assert not b.up_to_date()


def test_another_torch_makes_the_binding_stale(scratch, monkeypatch):
    import torch
    assert not b.up_to_date()
    b.build()
    assert b.up_to_date()
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    assert not b.up_to_date()
    b.build()
    assert b.up_to_date()
    os.remove(b.BIND)
    assert not b.up_to_date()
