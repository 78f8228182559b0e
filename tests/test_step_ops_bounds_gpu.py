"""Recurrent layers over segments whose bounds are far outside the stream."""

from __future__ import annotations

import numpy as np
import pytest

from mixed_chunked_prefill_gb300 import _capi
from test_step_ops_edges_gpu import DT, err_word, i32, mcp, scan_inputs, values  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

LOW, HIGH = -(1 << 31), (1 << 31) - 1
# decreases by more than 2^31, whose difference in 32 bits is a length of 1 and more
WILD = [[0, HIGH, LOW, 20], [0, 2, LOW, 20], [0, HIGH - 1, LOW + 1, 20], [0, HIGH - 3, LOW + 40, 20], [0, 20, LOW, HIGH],
        [0, 4, HIGH, LOW + 500]]


@pytest.mark.parametrize("cu", WILD)
@pytest.mark.parametrize("T", [20, 400])
def test_conv_of_bounds_far_outside(mcp, cu, T):  # noqa: F811
    """Reported; the inputs are rows whose neighbours are NaN, and outputs and states stay finite."""
    rng, d, K, R = np.random.default_rng(T), 72, 4, 5
    x = torch.full((T + 8, d), float("nan"), dtype=DT["bf16"], device="cuda")
    x[4:T + 4] = values(rng, (T, d), "bf16")[1]
    w, b = values(rng, (d, K), "bf16")[1], values(rng, (d,), "bf16")[1]
    state = values(rng, (R, K - 1, d), "bf16")[1]
    out, err = torch.full((T + 8, d), 7.0, dtype=DT["bf16"], device="cuda"), err_word()
    mcp.mixed_conv(x[4:T + 4], w, b, state, i32([0, 1, 2]), i32(cu), i32([T] * 3), "silu", out[4:T + 4], err)
    assert int(err) & _capi.DEVERR_SEGMENT
    assert (out[:4] == 7).all() and (out[T + 4:] == 7).all() and torch.isfinite(out).all()
    assert torch.isfinite(state).all()


@pytest.mark.parametrize("cu", WILD)
@pytest.mark.parametrize("T", [20, 400])
def test_scan_of_bounds_far_outside(mcp, cu, T):  # noqa: F811
    rng, d, N, R = np.random.default_rng(T), 72, 16, 5
    v = {k: t[1] for k, t in scan_inputs(rng, T + 8, d, N, 1, "bf16", R, True, 1.0).items()}
    for k in ("x", "dt", "z", "B", "C"):
        v[k][:4], v[k][T + 4:] = float("nan"), float("nan")
    out, err, at = torch.full((T + 8, d), 7.0, dtype=torch.bfloat16, device="cuda"), err_word(), slice(4, T + 4)
    mcp.mixed_scan(v["x"][at], v["dt"][at], v["A"], v["B"][at], v["C"][at], v["state"], i32([0, 1, 2]), i32(cu),
                   i32([T] * 3), D=v["D"], z=v["z"][at], dt_bias=v["bias"], out=out[at], error_word=err)
    assert int(err) & _capi.DEVERR_SEGMENT
    assert (out[:4] == 7).all() and (out[T + 4:] == 7).all() and torch.isfinite(out).all()
    assert torch.isfinite(v["state"]).all()
