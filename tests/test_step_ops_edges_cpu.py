"""Operators around a step's attention, without a GPU: refusals at the ends of what the
calls take."""

from __future__ import annotations

import ctypes

import numpy as np
import pytest

from mixed_chunked_prefill_gb300 import _capi
from test_step_ops_cpu import INVALID, OK, P16, UNSUPPORTED, conv, counts, lib, logits, pool, scan

assert lib is not None  # the fixture that builds and loads the library


@pytest.mark.parametrize("cap,over,ids,S,status", [
    (-1, {}, P16, 4, INVALID), ((1 << 30) + 1, {}, P16, 4, UNSUPPORTED), (64, dict(num_pages=0), P16, 4, INVALID),
    (64, {}, None, 4, INVALID), (64, {}, P16, 8193, UNSUPPORTED), (0, {}, None, 0, OK), (-1, {}, None, 0, INVALID),
])
def test_commit_built_step_refusals(lib, cap, over, ids, S, status):
    p = pool(**over)
    assert lib.mcp_commit_built_step(ctypes.byref(p), ids, P16, None, S, cap, None, None) == status
    assert lib.mcp_commit_built_step(None, P16, P16, None, 4, 64, None, None) == INVALID
    assert _capi.MAX_TOKENS == 1 << 30


@pytest.mark.parametrize("over,status", [
    (dict(rows=(1 << 30) + 1, n=4, cu=P16), UNSUPPORTED), (dict(rows=0x7fffffff, n=0, cu=P16, flags=2), UNSUPPORTED),
    (dict(rows=1 << 30, n=5), INVALID),  # at the bound the other checks go on
])
def test_update_token_counts_of_many_rows(lib, over, status):
    """The rows' 32-bit indices are rounded up to whole CTAs."""
    assert counts(lib, **over) == status


def test_misaligned_arrays_are_refused(lib):
    """Addresses inside an int32 or fp32, for each array of each call (refused before a launch)."""
    bad, p = P16 + 2, ctypes.byref(pool())
    for k in range(9):  # ids, q_lens | cu, sk, bt, slots, positions, logits_indices, error word
        a = [P16] * 9
        a[k] = bad
        assert lib.mcp_build_step_tables(p, *a[:2], 4, 64, *a[2:], None) == INVALID, k
    for k in range(4):
        a = [P16] * 4
        a[k] = bad
        assert lib.mcp_commit_step(p, *a[:3], 4, a[3], None) == INVALID, k
        assert lib.mcp_commit_built_step(p, *a[:3], 4, 64, a[3], None) == INVALID, k
    for k in range(3):
        meta = [P16] * 3
        meta[k] = bad
        assert conv(lib, meta=meta, out=2 * P16) == INVALID
        assert scan(lib, meta=meta, tensors=dict(out=2 * P16)) == INVALID
    for name in ("ids", "tokens", "seen", "cnt", "cu"):
        assert counts(lib, **{name: bad}) == INVALID, name
    for name in ("request_ids", "seen", "temperature", "repetition_penalty", "frequency_penalty",
                 "presence_penalty", "bias_offsets", "bias_tokens", "bias_values", "mask", "mask_rows"):
        given = dict(bias_offsets=P16, bias_tokens=P16, bias_values=P16, mask=P16)
        assert logits(lib, tensors={**given, name: bad}) == INVALID, name


@pytest.mark.parametrize("call", [conv, scan])
def test_recurrent_sizes_past_32_bits(lib, call):
    """Channels whose index would wrap when rounded up to a launch, and more tasks of the long
    segments than 32 bits number (2^20 segments of 5 tokens, 2^18 channels)."""
    wide = dict(x_stride=(1 << 30) + 8, out_stride=(1 << 30) + 8)
    many = dict(num_seqs=1 << 20, total_tokens=5 << 20, channels=1 << 18, x_stride=1 << 18, out_stride=1 << 18)
    out = dict(out=2 * P16)
    if call is scan:
        wide.update(dt_stride=(1 << 30) + 8, z_stride=(1 << 30) + 8)
        many.update(dt_stride=1 << 18, z_stride=1 << 18)
        out = dict(tensors=out)
    assert call(lib, channels=(1 << 30) + 8, **wide, **out) == UNSUPPORTED
    if call is scan:
        assert call(lib, **many, **out) == UNSUPPORTED


@pytest.mark.parametrize("ids,q", [([0], [2 ** 31 - 1]), ([0, 1], [2 ** 31 - 1] * 2), ([1], np.array([2 ** 32 + 1])),
                                   (np.array([2 ** 32]), [1]), ([1], [2 ** 31])])
def test_step_lengths_past_32_bits(ids, q):
    """Lengths and rows are checked before they become 32 bits: nothing wraps into range."""
    from types import SimpleNamespace

    from mixed_chunked_prefill_gb300.step import RequestTables, StepTables

    pool_ = SimpleNamespace(max_requests=4, max_pages_per_seq=1 << 20, page_size=64)
    tables = SimpleNamespace(pool=pool_, commits=0, device="cpu", lens_h=np.array([5, 0, 0, 0]), free_h=1 << 26)
    with pytest.raises(ValueError):
        StepTables(tables, ids, q, None, None)
    step = SimpleNamespace(pool=pool_, after=0, ids_h=np.array([0]), sk_h=np.array([7], dtype=np.int32))
    with pytest.raises(ValueError):
        RequestTables.commit(tables, step, np.array([2 ** 32 + 1]))


def test_raw_streams_are_of_the_tables_device(monkeypatch):
    """A stream given as an address is one of the tables' device, whatever the current one is."""
    import contextlib

    torch = pytest.importorskip("torch")
    from types import SimpleNamespace

    from mixed_chunked_prefill_gb300 import step

    made = []
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda ptr, device=None: made.append((ptr, device)))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(step, "build_step_tables", lambda *a: None)
    pool_ = SimpleNamespace(max_requests=4, max_pages_per_seq=4, page_size=16)
    dev = torch.device("cpu")
    tables = SimpleNamespace(pool=pool_, commits=0, device=dev, lens_h=np.zeros(4, np.int64), free_h=9, error_word=None)
    built = step.StepTables(tables, [0, -1, 2], [5, 0, 20], 64, 77)
    assert made == [(77, dev)] and built.cu_h.tolist() == [0, 5, 5, 25] and tables.last is built
