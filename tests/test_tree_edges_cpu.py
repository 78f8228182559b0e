"""Trees of drafted tokens without a GPU: calls whose arguments end a process or are not what they
seem."""

from __future__ import annotations

import ctypes
import os
import subprocess
import sys

import numpy as np  # noqa: F401
import pytest

import mixed_chunked_prefill_gb300 as mcp  # noqa: F401
from mixed_chunked_prefill_gb300 import _capi
from test_tree_cpu import INVALID, OK, P16, keep, lib  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def alone(code):
    """Run `code` in a process that sees no GPU (nothing in it may reach one)."""
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="", PYTHONPATH=os.pathsep.join([ROOT, ROOT + "/tests"]))
    return subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=300)


@pytest.mark.parametrize("caches", ["None", "()"])
@pytest.mark.parametrize("stride", [0, 64])
def test_kept_paths_of_no_layers_read_no_caches(lib, caches, stride):  # noqa: F811
    """Lengths alone: with no layers the arrays of caches may be empty or not there, listed or at one
    distance.  Without a GPU the call comes as far as its launch."""
    got = alone("import mixed_chunked_prefill_gb300 as m; from test_tree_cpu import keep; "
                f"print('status', keep(m.load(), ks={caches}, vs={caches}, num_layers=0, layer_stride={stride}))")
    assert got.returncode == 0 and f"status {_capi.MCP_ERR_CUDA}" in got.stdout, (got.returncode, got.stderr)
