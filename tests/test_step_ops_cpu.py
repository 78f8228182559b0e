"""Operators around a step's attention, without a GPU: the refusals of the C
entries (returned before anything is launched) and the definitions the GPU tests
compare with, pinned to hand-written values and to each other."""

from __future__ import annotations

import ctypes

import numpy as np
import pytest

import mixed_chunked_prefill_gb300 as mcp
from mixed_chunked_prefill_gb300 import _capi
from oracle import step_ops_ref as ref

OK, INVALID, UNSUPPORTED = _capi.MCP_OK, _capi.MCP_ERR_INVALID_ARG, _capi.MCP_ERR_UNSUPPORTED
P16 = 0x10000  # an address that is never read: every call here is refused before a launch


@pytest.fixture(scope="module", autouse=True)
def lib():
    from mixed_chunked_prefill_gb300 import build

    build.build()
    return mcp.load()


def pool(**over):
    f = dict(max_requests=8, max_pages_per_seq=16, page_size=16, num_pages=64, request_pages=P16,
             request_lens=P16, free_pages=P16, free_count=P16)
    f.update(over)
    return _capi.RequestPool(*(f[n] for n, _ in _capi.RequestPool._fields_))


def build_tables(lib, p, ids=P16, q=P16, S=4, cap=64, cu=P16, sk=P16, bt=P16, slots=P16):
    return lib.mcp_build_step_tables(ctypes.byref(p) if p is not None else None, ids, q, S, cap, cu,
                                     sk, bt, slots, None, None, None, None)


@pytest.mark.parametrize("over,status", [
    (dict(max_requests=0), INVALID), (dict(max_pages_per_seq=0), INVALID),
    (dict(num_pages=0), INVALID), (dict(max_requests=(1 << 24) + 1), UNSUPPORTED),
    (dict(page_size=4), UNSUPPORTED), (dict(page_size=0), UNSUPPORTED),
    (dict(max_pages_per_seq=(1 << 28) + 1, page_size=1), UNSUPPORTED),
    (dict(max_pages_per_seq=1 << 27), UNSUPPORTED), (dict(request_pages=None), INVALID),
    (dict(request_lens=None), INVALID), (dict(free_pages=None), INVALID),
    (dict(free_count=None), INVALID), (dict(request_pages=P16 + 8), INVALID),
])
def test_pool_refusals(lib, over, status):
    assert build_tables(lib, pool(**over)) == status
    assert lib.mcp_commit_step(ctypes.byref(pool(**over)), P16, P16, None, 4, None, None) == status
    assert lib.mcp_last_error()


@pytest.mark.parametrize("over,status", [
    (dict(S=-1), INVALID), (dict(S=8193), UNSUPPORTED), (dict(cap=-1), INVALID),
    (dict(ids=None), INVALID), (dict(q=None), INVALID), (dict(cu=None), INVALID),
    (dict(sk=None), INVALID), (dict(bt=None), INVALID), (dict(slots=None), INVALID),
    (dict(bt=P16 + 4), INVALID), (dict(slots=P16 + 4), INVALID), (dict(cap=(1 << 30) + 1), UNSUPPORTED),
])
def test_build_step_tables_refusals(lib, over, status):
    assert build_tables(lib, pool(), **over) == status


def test_tables_without_a_pool(lib):
    assert build_tables(lib, None) == INVALID
    assert lib.mcp_commit_step(None, P16, P16, None, 4, None, None) == INVALID
    assert lib.mcp_commit_step(ctypes.byref(pool()), None, P16, None, 4, None, None) == INVALID
    assert lib.mcp_commit_step(ctypes.byref(pool()), None, None, None, 0, None, None) == OK


def conv(lib, meta=(P16, P16, P16), x=P16, w=P16, b=None, state=P16, out=P16, **over):
    f = dict(num_seqs=3, total_tokens=10, num_requests=4, channels=64, width=4, dtype=0,
             activation=1, reserved=0, x_stride=64, out_stride=64)
    f.update(over)
    d = _capi.ConvDesc(*(f[n] for n, _ in _capi.ConvDesc._fields_))
    return lib.mcp_mixed_conv(ctypes.byref(d), x, w, b, state, *meta, out, None, None)


@pytest.mark.parametrize("over,status", [
    (dict(num_seqs=-1), INVALID), (dict(total_tokens=-1), INVALID), (dict(num_requests=0), INVALID),
    (dict(channels=0), INVALID), (dict(channels=60), INVALID), (dict(width=1), UNSUPPORTED),
    (dict(width=5), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(activation=2), INVALID),
    (dict(reserved=1), INVALID), (dict(x_stride=56), INVALID), (dict(x_stride=68), INVALID),
    (dict(out_stride=60), INVALID), (dict(meta=(None, P16, P16)), INVALID),
    (dict(meta=(P16, None, P16)), INVALID), (dict(meta=(P16, P16, None)), INVALID),
    (dict(x=None), INVALID), (dict(x=P16 + 8), INVALID), (dict(w=None), INVALID),
    (dict(b=P16 + 2), INVALID), (dict(state=None), INVALID), (dict(state=P16 + 8), INVALID),
    (dict(out=None), INVALID), (dict(num_seqs=0), OK), (dict(total_tokens=0, x=None), OK),
    (dict(), INVALID),  # out == x
    (dict(num_seqs=(1 << 20) + 1), UNSUPPORTED), (dict(total_tokens=(1 << 30) + 1), UNSUPPORTED),
    (dict(num_requests=(1 << 24) + 1), UNSUPPORTED),
    (dict(num_seqs=1 << 20, channels=1 << 20, x_stride=1 << 20, out_stride=1 << 20, out=2 * P16),
     UNSUPPORTED),  # 2^31 CTAs
])
def test_mixed_conv_refusals(lib, over, status):
    assert conv(lib, **over) == status


def scan(lib, meta=(P16, P16, P16), tensors=(), workspace=(None, 0), **over):
    f = dict(num_seqs=3, total_tokens=10, num_requests=4, channels=64, state_size=16, num_groups=1,
             dtype=0, softplus=1, x_stride=64, dt_stride=64, z_stride=64, b_stride=16, c_stride=16,
             out_stride=64)
    f.update(over)
    d = _capi.ScanDesc(*(f[n] for n, _ in _capi.ScanDesc._fields_))
    a = {n: P16 for n, _ in _capi.ScanTensors._fields_}
    a.update(tensors)
    t = _capi.ScanTensors(*(a[n] for n, _ in _capi.ScanTensors._fields_))
    return lib.mcp_mixed_scan(ctypes.byref(d), ctypes.byref(t), *meta, *workspace, None, None)


@pytest.mark.parametrize("over,status", [
    (dict(num_seqs=-1), INVALID), (dict(channels=4), INVALID), (dict(num_requests=0), INVALID),
    (dict(state_size=4), UNSUPPORTED), (dict(state_size=128), UNSUPPORTED),
    (dict(state_size=12), UNSUPPORTED), (dict(num_groups=0), INVALID), (dict(num_groups=3), INVALID),
    (dict(num_groups=4, b_stride=64, c_stride=64), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED),
    (dict(softplus=2), INVALID), (dict(b_stride=8), INVALID), (dict(c_stride=20), INVALID),
    (dict(z_stride=0), INVALID), (dict(dt_stride=65), INVALID), (dict(meta=(P16, None, P16)), INVALID),
    *[(dict(tensors={n: None}), INVALID) for n in ("x", "dt", "A", "B", "C", "state", "out")],
    *[(dict(tensors={n: P16 + 8}), INVALID) for n in
      ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "state", "out")],
    (dict(workspace=(P16 + 128, 1 << 40)), INVALID),
    (dict(total_tokens=100000, channels=8192, x_stride=8192, dt_stride=8192, z_stride=8192,
          out_stride=8192, workspace=(P16, 256)), _capi.MCP_ERR_WORKSPACE_TOO_SMALL),
    (dict(num_seqs=0), OK), (dict(total_tokens=0), OK),
    *[(dict(tensors={n: 2 * P16 for n in ("x", "dt", "B", "C", "z") if n != same}), INVALID)
      for same in ("x", "dt", "B", "C", "z")],  # out is that one
    (dict(num_seqs=(1 << 20) + 1), UNSUPPORTED), (dict(total_tokens=(1 << 30) + 1), UNSUPPORTED),
    (dict(num_requests=(1 << 24) + 1), UNSUPPORTED),
])
def test_mixed_scan_refusals(lib, over, status):
    assert scan(lib, **over) == status


def counts(lib, ids=P16, rows=4, tokens=P16, n=4, cu=None, seen=P16, cnt=P16, R=4, V=100, flags=0):
    return lib.mcp_update_token_counts(ids, rows, tokens, n, cu, seen, cnt, R, V, flags, None, None)


@pytest.mark.parametrize("over,status", [
    (dict(rows=-1), INVALID), (dict(n=-1), INVALID), (dict(R=0), INVALID), (dict(V=0), INVALID),
    (dict(flags=4), INVALID), (dict(n=5), INVALID), (dict(ids=None), INVALID),
    (dict(tokens=None), INVALID), (dict(seen=None), INVALID), (dict(cnt=None), INVALID),
    (dict(rows=0, n=0), OK), (dict(rows=0, n=7, cu=P16), OK),
    (dict(n=(1 << 30) + 1, cu=P16), UNSUPPORTED), (dict(V=(1 << 28) + 1), UNSUPPORTED),
])
def test_update_token_counts_refusals(lib, over, status):
    assert counts(lib, **over) == status


def logits(lib, tensors=(), **over):
    f = dict(num_rows=2, vocab_size=100, num_requests=4, dtype=0, out_dtype=0, num_biases=3,
             num_masks=2, reserved=0, logits_stride=100, out_stride=100)
    f.update(over)
    d = _capi.LogitsDesc(*(f[n] for n, _ in _capi.LogitsDesc._fields_))
    a = dict(logits=P16, out=2 * P16, request_ids=P16, seen=P16, counts=P16)
    a.update(tensors)
    t = _capi.LogitsTensors(*(a.get(n) for n, _ in _capi.LogitsTensors._fields_))
    return lib.mcp_process_logits(ctypes.byref(d), ctypes.byref(t), None, None)


@pytest.mark.parametrize("over,status", [
    (dict(num_rows=-1), INVALID), (dict(vocab_size=0), INVALID), (dict(dtype=3), UNSUPPORTED),
    (dict(dtype=0, out_dtype=1), UNSUPPORTED), (dict(dtype=2, out_dtype=0), UNSUPPORTED),
    (dict(reserved=1), INVALID), (dict(logits_stride=99), INVALID), (dict(out_stride=0), INVALID),
    (dict(num_rows=0x7fffffff, vocab_size=4096, logits_stride=4096, out_stride=4096), UNSUPPORTED),
    (dict(num_biases=-1), INVALID), (dict(num_masks=-1), INVALID), (dict(num_requests=0), INVALID),
    (dict(tensors=dict(logits=None)), INVALID), (dict(tensors=dict(out=None)), INVALID),
    (dict(tensors=dict(logits=P16 + 1)), INVALID), (dict(out_dtype=2, tensors=dict(out=P16 + 2)), INVALID),
    (dict(out_dtype=2, tensors=dict(out=P16)), INVALID),
    (dict(out_stride=128, tensors=dict(out=P16)), INVALID),
    (dict(tensors=dict(seen=None)), INVALID), (dict(tensors=dict(counts=None)), INVALID),
    (dict(tensors=dict(counts=P16 + 4)), INVALID),
    (dict(tensors=dict(request_ids=None, repetition_penalty=P16)), INVALID),
    (dict(tensors=dict(request_ids=None, presence_penalty=P16)), INVALID),
    (dict(tensors=dict(bias_offsets=P16, bias_tokens=P16)), INVALID),
    (dict(num_masks=1, tensors=dict(mask=P16)), INVALID),
    (dict(tensors=dict(mask_rows=P16)), INVALID), (dict(num_rows=0), OK),
])
def test_process_logits_refusals(lib, over, status):
    assert logits(lib, **over) == status


def test_python_calls_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        mcp.build_step_tables(_capi.RequestPool(), i, i, i, i, i, i)
    with pytest.raises(ValueError):
        mcp.make_request_pool(i.view(1, 2), i, i, i, 16)
    with pytest.raises(ValueError):
        mcp.process_logits(torch.zeros(2, 8))
    with pytest.raises(ValueError):
        mcp.update_token_counts(i, i, i, i, 8)
    with pytest.raises(ValueError):
        mcp.mixed_conv(torch.zeros(2, 8), i, i, i, i, i, i)
    with pytest.raises(ValueError):
        mcp.mixed_scan(torch.zeros(2, 8), i, i, i, i, i, i, i, i)


# ------------------------------------------------------------------ the definitions
def test_pool_definition_by_hand():
    p = ref.Pool(num_pages=6, page_size=8, max_requests=3, max_pages_per_seq=4)
    cu, sk, bt, slots, pos, rows, taken = p.build([2, -1, 0], [9, 5, 3], 14)
    assert cu.tolist() == [0, 9, 9, 12] and sk.tolist() == [9, 0, 3]
    # three new pages, the top of the list in segment order: 3, 4 for row 2, 5 for row 0
    assert bt.tolist() == [[3, 4, -1, -1], [-1] * 4, [5, -1, -1, -1]]
    assert slots.tolist() == [24, 25, 26, 27, 28, 29, 30, 31, 32, 40, 41, 42, -1, -1]
    assert pos.tolist() == [0, 1, 2, 3, 4, 5, 6, 7, 8, 0, 1, 2, 0, 0] and rows.tolist() == [8, 11, -1]
    p.commit([2, -1, 0], [9, 5, 3], [8, 0, 3], taken)  # one token of row 2 was rejected
    assert p.free == [0, 1, 2, 4] and p.lens == [3, 0, 8] and p.pages == [[5], [], [3]]
    cu, sk, bt, *_, taken = p.build([2], [1], 1)
    assert bt.tolist() == [[3, 4, -1, -1]] and sk.tolist() == [9]
    with pytest.raises(ref.StepError):
        p.build([2, 2], [1, 1], 8)
    with pytest.raises(ref.StepError):
        p.build([2], [25], 32)


def test_pool_agrees_with_the_host_slot_mapping(lib):
    rng = np.random.default_rng(3)
    p = ref.Pool(200, 16, 6, 20)
    for _ in range(6):
        ids = rng.permutation(6)[:4].tolist()
        q = rng.integers(0, 40, 4).tolist()
        cu, sk, bt, slots, pos, rows, taken = p.build(ids, q, sum(q))
        assert np.array_equal(mcp.build_slot_mapping(bt, cu, sk, 16, 200), slots)
        idx = mcp.build_logits_indices(cu)
        assert np.array_equal(idx, rows[:len(idx)]) and (rows[len(idx):] == -1).all()
        p.commit(ids, q, sk.tolist(), taken)


def test_conv_and_scan_in_chunks_equal_one_shot():
    rng = np.random.default_rng(5)
    T, d, K, N = 23, 8, 4, 8
    x, w, b = rng.normal(size=(T, d)), rng.normal(size=(d, K)), rng.normal(size=d)
    st = rng.normal(size=(2, K - 1, d))
    whole, _, end = ref.conv(x, w, b, st, [1], [0, T], [T], True, "fp32")
    h = rng.normal(size=(2, d, N))
    args = dict(A=-rng.random((d, N)), D=rng.normal(size=d), dt_bias=rng.normal(size=d))
    B, C, dt, z = (rng.normal(size=s) for s in ((T, 1, N), (T, 1, N), (T, d), (T, d)))
    ywhole, _, hend, _ = ref.scan(x, dt, args["A"], B, C, args["D"], z, args["dt_bias"], True, h, [0],
                                  [0, T], [T], "fp32")
    a, outs, ys, s, hh = 0, [], [], st, h
    for n in (1, 2, 7, 13):
        o, _, s = ref.conv(x[a:a + n], w, b, s, [1], [0, n], [a + n], True, "fp32")
        y, _, hh, _ = ref.scan(x[a:a + n], dt[a:a + n], args["A"], B[a:a + n], C[a:a + n], args["D"],
                               z[a:a + n], args["dt_bias"], True, hh, [0], [0, n], [a + n], "fp32")
        outs.append(o)
        ys.append(y)
        a += n
    assert np.allclose(np.concatenate(outs), whole, rtol=1e-12, atol=1e-12) and np.array_equal(s, end)
    assert np.allclose(np.concatenate(ys), ywhole, rtol=1e-12, atol=1e-12)
    assert np.allclose(hh, hend, rtol=1e-12)


def test_scan_definition_by_hand():
    # one channel pair, one state doubled: h = e^{-ln2} h + x, y = h + 2 x
    ln2 = np.log(2.0)
    x = np.array([[1.0, 0.0], [0.0, 2.0]])
    A = np.full((2, 1), -1.0)
    y, _, h, _ = ref.scan(x, np.full((2, 2), ln2), A, np.full((2, 1, 1), 1 / ln2), np.ones((2, 1, 1)),
                          np.full(2, 2.0), None, np.zeros(2), False, np.array([[[4.0], [8.0]]]), [0],
                          [0, 2], [5], "fp32")
    assert np.allclose(y, [[2 + 1 + 2, 4], [1.5, 2 + 2 + 4]]) and np.allclose(h, [[[1.5], [4.0]]])


def test_logits_definition_by_hand():
    x = np.array([[2.0, -2.0, 1.0, 4.0]])
    seen = np.zeros((1, 2, 4), bool)
    seen[0, 0, 0] = seen[0, 1, 1] = True
    cnt = np.array([[0, 3, 0, 0]])
    y, _ = ref.logits(x, [0], seen, cnt, [0.5], [2.0], [0.25], [1.0], {0: {2: 0.5}},
                      [np.array([1, 1, 1, 0], bool)], "fp32")
    assert y.tolist() == [[2.0, 2 * (-4 - 0.75 - 1), 3.0, -np.inf]]
    assert ref.pack_bits(np.array([1, 0, 0, 0, 1] + [0] * 27 + [1], bool)).tolist() == [17, 1]
