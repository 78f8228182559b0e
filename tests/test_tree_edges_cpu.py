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


def overlapping(ks, vs, size, layers, stride):
    """Whether any two of a call's caches share a byte, one pair after another."""
    if stride:
        ks, vs = ([x[0] + 2 * stride * l for l in range(layers)] for x in (ks, vs))
    all_of = list(ks) + list(vs)
    return any(abs(a - b) < size for i, a in enumerate(all_of) for b in all_of[:i])


SIZE = 8 * 16 * 2 * 64 * 2  # bytes of a cache of `keep`


@pytest.mark.parametrize("ks,vs,more", [
    ((0, 0), (2, 3), {}), ((0, 1), (2, 0), {}), ((0, 1), (2, 2), {}), ((0,), (0,), dict(num_layers=1)),
    ((0, 1), (1.5, 3), {}), ((3, 0), (1, 2.99), {}), ((5, 1), (3, 5 - 1 / 1024), {}),
    ((0,), (0,), dict(layer_stride=SIZE)), ((0,), (0.5,), dict(layer_stride=SIZE)),
    ((0,), (1,), dict(layer_stride=SIZE // 2)),        # K's second layer is V's first
    ((2,), (0,), dict(layer_stride=SIZE // 2, num_layers=3)),
    ((0,), (8,), dict(layer_stride=SIZE // 2 - 8)),    # layers that run into each other
    ((0,), (1 - 1 / 1024,), dict(layer_stride=64, num_layers=1)),
    ((0,), (40.5,), dict(layer_stride=SIZE, num_layers=30)),
])
def test_kept_paths_refuse_caches_that_share_memory(lib, ks, vs, more):  # noqa: F811
    """The same cache listed twice, for two layers or for K and V, would have its rows moved twice."""
    ks, vs = ([P16 + int(x * SIZE) // 16 * 16 for x in xs] for xs in (ks, vs))
    assert overlapping(ks, vs, SIZE, more.get("num_layers", 2), more.get("layer_stride", 0))
    assert keep(lib, ks=ks, vs=vs, **more) == INVALID and b"caches overlap" in lib.mcp_last_error()


def test_kept_paths_take_caches_that_only_touch(lib):  # noqa: F811
    """Pools that hold K and V of a layer, or of all layers, side by side, in any order: they come as
    far as their launch."""
    rng = np.random.default_rng(1)
    calls = []
    for _ in range(300):
        layers, listed = int(rng.integers(1, 6)), rng.random() < 0.5
        if listed:
            at = P16 + SIZE * rng.choice(40, 2 * layers, replace=rng.random() < 0.3) + 16 * rng.integers(0, 3)
            calls.append((at[:layers].tolist(), at[layers:].tolist(), layers, 0))
        else:
            k, v = (P16 + SIZE * rng.integers(0, 12, 2) // 2).tolist()
            calls.append(([k], [v], layers, int(SIZE // 4 * rng.integers(1, 9))))
    got = alone("import mixed_chunked_prefill_gb300 as m; from test_tree_cpu import keep; lib = m.load()\n"
                f"for k, v, n, s in {calls}:\n"
                "    print(keep(lib, ks=k, vs=v, num_layers=n, layer_stride=s))")
    want = [INVALID if overlapping(k, v, SIZE, n, s) else _capi.MCP_ERR_CUDA for k, v, n, s in calls]
    assert got.returncode == 0 and [int(x) for x in got.stdout.split()] == want, got.stderr
    assert 50 < want.count(INVALID) < 250


@pytest.mark.filterwarnings("error")
def test_options_that_are_none_warn():
    """A misspelt option would leave the plan at its defaults without a word."""
    for make in (lambda: mcp.PlanOptions(prefil_split_tokens=128),
                 lambda: setattr(mcp.PlanOptions(), "trees", 1)):
        with pytest.raises(UserWarning, match="has no option '(prefil_split_tokens|trees)'"):
            make()
    options = mcp.PlanOptions(152, prefill_split_tokens=128, tree=1)
    options.decode_split_tokens = 64
    assert [getattr(options, n) for n in ("num_sms", "decode_split_tokens", "prefill_split_tokens", "tree")] == [
        152, 64, 128, 1]
    assert mcp.PlanOptions.from_buffer_copy(options).prefill_split_tokens == 128
