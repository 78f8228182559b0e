"""Operators around a step's attention on the GPU: calls that their documentation allows
at the edges of what they take -- refused steps that are committed all the same, steps
built in another order than they are committed, malformed streams, factors near the ends
of fp32, streams of many segments."""

from __future__ import annotations

import ctypes

import numpy as np
import pytest

from mixed_chunked_prefill_gb300 import _capi
from oracle import step_ops_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_step_ops_gpu import (  # noqa: E402
    DT, Device, device_state, err_word, f64, i32, mcp, run_scan, scan_inputs, stream, values)

assert mcp is not None  # the fixture that builds and loads the library


# --------------------------------------------------------------------------- tables
@pytest.mark.parametrize("ids,q,cap", [([0, 1], [5, 4], 8), ([1], [20], 8), ([2], [1], 0),
                                       ([0, -1, 1], [13, 9, 33], 45)])
@pytest.mark.parametrize("how", ["keep", "end", "cut"])
def test_step_past_max_tokens_is_not_committed(mcp, ids, q, cap, how):
    """A step that the build refused for max_tokens alone: the commit refuses it too, also
    where the step needs no new page."""
    p, d = ref.Pool(10, 16, 3, 4), Device(mcp, 10, 16, 3, 4)
    want = p.build([2, 0], [17, 3], 20)
    d.build([2, 0], [17, 3], 20)
    d.commit([2, 0], [17, 3])
    p.commit([2, 0], [17, 3], [17, 3], want[6])
    new = {"keep": None, "end": [0] * len(ids), "cut": [max(0, p.lens[r]) if r >= 0 else 0 for r in ids]}[how]
    before = [t.clone() for t in (d.pages, d.lens, d.free, d.count)]
    cu, *_ = d.build(ids, q, cap)
    assert int(d.err) == _capi.DEVERR_REQUEST and not cu.any()
    d.err.zero_()
    d.commit(ids, q, new)
    assert int(d.err) == _capi.DEVERR_REQUEST
    assert all(torch.equal(a, b) for a, b in zip(before, (d.pages, d.lens, d.free, d.count)))
    d.err.zero_()
    want = p.build(ids, q, 60)  # with room it is sound
    for got, w in zip(d.build(ids, q, 60), want[:6]):
        assert np.array_equal(got, w)
    new = want[1].tolist() if new is None else new
    d.commit(ids, q, None if how == "keep" else new)
    p.commit(ids, q, new, want[6])
    d.equal(p)


def test_commit_is_told_max_tokens(mcp):
    """A handle that has built nothing takes every step unless it is told the build's
    max_tokens; so does the C entry without the argument."""
    d = Device(mcp, 10, 16, 3, 4)
    one, many = i32([1]), i32([20])
    for cap, lens in ((19, 0), (20, 20)):
        mcp.commit_step(d.pool, one, many, None, d.err, max_tokens=cap)
        assert int(d.lens[1]) == lens and int(d.err) == (0 if lens else _capi.DEVERR_REQUEST)
        d.err.zero_()
    mcp.commit_step(d.pool, one, many, None, d.err)
    assert int(d.lens[1]) == 40 and int(d.err) == 0
    lib = mcp.load()
    s = torch.cuda.current_stream().cuda_stream
    assert lib.mcp_commit_step(ctypes.byref(d.pool), one.data_ptr(), many.data_ptr(), None, 1,
                               d.err.data_ptr(), s) == 0
    assert int(d.lens[1]) == 60 and int(d.err) == 0


def test_captured_step_past_max_tokens(mcp):
    """Build and commit in one graph of fixed max_tokens: a replay with too many tokens
    leaves the pool as it was, the next goes on from there."""
    p, d = ref.Pool(10, 16, 3, 4), Device(mcp, 10, 16, 3, 4)
    ids, q = i32([-1, -1]), i32([0, 0])
    cu, sk, bt = i32([0] * 3), i32([0] * 2), torch.zeros((2, 4), dtype=torch.int32, device="cuda")
    slots = torch.zeros(24, dtype=torch.int64, device="cuda")

    def calls():
        mcp.build_step_tables(d.pool, ids, q, cu, sk, bt, slots, error_word=d.err)
        mcp.commit_step(d.pool, ids, q, None, d.err)

    calls()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
        calls()
    torch.cuda.synchronize()
    for step in (([0, 2], [20, 4]), ([0, 1], [13, 12]), ([1, 0], [15, 9]), ([2, 1], [25, 0])):
        ids.copy_(i32(step[0]))
        q.copy_(i32(step[1]))
        g.replay()
        torch.cuda.synchronize()
        if sum(step[1]) <= 24:
            want = p.build(*step, 24)
            p.commit(*step, want[1].tolist(), want[6])
            assert np.array_equal(bt.cpu().numpy(), want[2])
        else:
            assert int(d.err) == _capi.DEVERR_REQUEST
            d.err.zero_()
        d.equal(p)


@pytest.mark.parametrize("later", [[([0], [20])], [([0], [20]), ([0], [40])], [([1, 0], [40, 20]), ([3], [1])],
                                   [([0, 1], [0, 0])], [([0, 1], [20, 20])]])
def test_step_committed_after_another_was_built(mcp, later):
    """A step is valid until the next commit: other steps built since, over the same page
    rows, change nothing for it; they are stale behind it."""
    from mixed_chunked_prefill_gb300.step import RequestTables

    tables, p = RequestTables(20, 16, 4, 6), ref.Pool(20, 16, 4, 6)
    first = ([2, 1], [7, 3])
    want = p.build(*first, 10)
    tables.commit(tables.step(*first))
    p.commit(*first, want[1].tolist(), want[6])
    a = tables.step([0, 1], [20, 20])
    want = p.build([0, 1], [20, 20], 40)
    others = [tables.step(*s) for s in later]
    tables.commit(a)
    p.commit([0, 1], [20, 20], want[1].tolist(), want[6])
    for got, w in zip((a.cu_seqlens_q, a.seqlens_k, a.block_tables, a.slot_mapping, a.positions,
                       a.logits_indices), want):
        assert np.array_equal(got.cpu().numpy(), w)
    for s in others:
        with pytest.raises(ValueError):
            tables.commit(s)
    tables.check()
    n = len(p.free)
    assert int(tables.free_count) == tables.free_h == n and tables.free_pages[:n].tolist() == p.free
    assert tables.request_lens.tolist() == p.lens == tables.lens_h.tolist()
    for r, pages in enumerate(p.pages):
        assert tables.request_pages[r, :len(pages)].tolist() == pages
    tables.release([0, 1, 2])
    assert sorted(tables.free_pages.tolist()) == list(range(20))


def test_sizes_past_32_bits_are_refused(mcp):
    """A size that the C structures cannot hold is refused by the binding: 2^32 + 8 tokens
    would be taken for 8."""
    V, n = 40, (1 << 32) + 8
    sd, cd = device_state(np.zeros((2, 2, V), bool), np.zeros((2, V), np.int64))
    tokens = torch.empty(n, dtype=torch.int32, device="cuda")
    tokens[:8] = 3
    with pytest.raises(ValueError):
        mcp.update_token_counts(i32([0, 1]), tokens, sd, cd, V, i32([0, 4, 8]))
    assert not sd.any() and not cd.any()
    d = Device(mcp, 10, 16, 3, 4)
    one = i32([1])
    with pytest.raises(ValueError):
        mcp.commit_step(d.pool, one, one, None, d.err, max_tokens=n)
    with pytest.raises(ValueError):
        mcp.build_step_tables(d.pool, one, one, i32([0, 0]), one, i32([[0] * 4]), tokens.view(torch.int64)[:1].expand(n))
    with pytest.raises(ValueError):
        mcp.make_request_pool(d.pages, d.lens, tokens, d.count, 16)


# ------------------------------------------------------------------ malformed streams
def bad_streams():
    """Prefix sums that decrease, overlap or leave the stream, most with tokens enough for
    runs: (ids, cu, sk, T)."""
    rng = np.random.default_rng(77)
    out = [([0, 1, 2], [0, 2, 1, 9], [9, 9, 9], 9), ([0, 1, 2], [0, 5, 3, 12], [9, 9, 9], 12),
           ([0, 1, 2, 3], [0, 20, 17, 18, 40], [40] * 4, 40), ([1, 0], [0, 16, 15], [16, 16], 30),
           ([2, 1, 0], [0, 100, 2, 100], [100] * 3, 100), ([0, 1, 2, 3], [0, 200, 0, 200, 1], [200] * 4, 200)]
    for _ in range(60):
        T, S = int(rng.integers(5, 60)), int(rng.integers(1, 7))
        cu = rng.integers(-2, T + 3, S + 1)
        cu[0] = 0
        if (np.diff(cu) >= 0).all() and cu.min() >= 0 and cu.max() <= T:
            cu[-1] = T + 1
        out.append((rng.permutation(S).tolist(), cu.tolist(), [T] * S, T))
    return out


@pytest.mark.parametrize("K,dtype,d", [(4, "bf16", 72), (3, "fp16", 8), (2, "bf16", 520)])
def test_conv_of_malformed_streams(mcp, K, dtype, d):
    """Reported, and nothing outside the stream's rows and the named requests is touched: the
    inputs are a slice of rows whose neighbours are NaN, which no finite output can have met."""
    rng = np.random.default_rng(K)
    for ids, cu, sk, T in bad_streams():
        R = len(ids) + 2
        x = torch.full((T + 8, d), float("nan"), dtype=DT[dtype], device="cuda")
        x[4:T + 4] = values(rng, (T, d), dtype)[1]
        w, b = values(rng, (d, K), dtype)[1], values(rng, (d,), dtype)[1]
        state = values(rng, (R, K - 1, d), dtype)[1]
        kept = state.clone()
        out = torch.full((T + 8, d), 7.0, dtype=DT[dtype], device="cuda")
        err = err_word()
        mcp.mixed_conv(x[4:T + 4], w, b, state, i32(ids), i32(cu), i32(sk), "silu", out[4:T + 4], err)
        assert int(err) & _capi.DEVERR_SEGMENT, (cu, T)
        assert (out[:4] == 7).all() and (out[T + 4:] == 7).all() and torch.isfinite(out).all(), (cu, T)
        assert torch.isfinite(state).all() and torch.equal(state[len(ids):], kept[len(ids):])


@pytest.mark.parametrize("N,d", [(16, 72), (64, 40)])
def test_scan_of_malformed_streams(mcp, N, d):
    rng = np.random.default_rng(N)
    for ids, cu, sk, T in bad_streams():
        R = len(ids) + 2
        v = {k: t[1] for k, t in scan_inputs(rng, T + 8, d, N, 1, "bf16", R, True, 1.0).items()}
        for k in ("x", "dt", "z", "B", "C"):
            v[k][:4], v[k][T + 4:] = float("nan"), float("nan")
        kept = v["state"].clone()
        out = torch.full((T + 8, d), 7.0, dtype=torch.bfloat16, device="cuda")
        err = err_word()
        at = slice(4, T + 4)
        mcp.mixed_scan(v["x"][at], v["dt"][at], v["A"], v["B"][at], v["C"][at], v["state"], i32(ids), i32(cu),
                       i32(sk), D=v["D"], z=v["z"][at], dt_bias=v["bias"], out=out[at], error_word=err)
        assert int(err) & _capi.DEVERR_SEGMENT, (cu, T)
        assert (out[:4] == 7).all() and (out[T + 4:] == 7).all() and torch.isfinite(out).all(), (cu, T)
        assert torch.isfinite(v["state"]).all() and torch.equal(v["state"][len(ids):], kept[len(ids):])


# ---------------------------------------------------------------------- ends of fp32
def scan_both(mcp, v, ids, cu, sk, R, T, d, N, softplus):
    """(out, state) without and with a workspace: a segment in one piece and in several."""
    lib = mcp.load()
    dev = {k: t[1] for k, t in v.items()}
    desc = _capi.ScanDesc(len(ids), T, R, d, N, 1, 0, softplus, d, d, d, N, N, d)
    need = ctypes.c_size_t()
    assert lib.mcp_mixed_scan_workspace(ctypes.byref(desc), ctypes.byref(need)) == 0 and need.value > 256
    ws = torch.full((need.value,), 255, dtype=torch.uint8, device="cuda")
    got = []
    for n in (0, need.value):
        out = torch.full((T, d), 7.0, dtype=torch.bfloat16, device="cuda")
        st = dev["state"].clone()
        tensors = _capi.ScanTensors(*(t.data_ptr() for t in (
            dev["x"], dev["dt"], dev["A"], dev["B"], dev["C"], dev["D"], dev["z"])), None, st.data_ptr(),
            out.data_ptr())
        meta = [i32(a) for a in (ids, cu, sk)]
        assert lib.mcp_mixed_scan(ctypes.byref(desc), ctypes.byref(tensors), *(t.data_ptr() for t in meta),
                                  ws.data_ptr() if n else None, n, None,
                                  torch.cuda.current_stream().cuda_stream) == 0
        got.append((f64(out), f64(st)))
    return got


@pytest.mark.parametrize("name", ["zero", "grows", "shrinks", "kept"])
def test_carried_states_at_the_ends_of_fp32(mcp, name):
    """Factors over a whole piece that leave fp32 where the state times them does not: a state
    of 0 stays 0, a small one that grows and falls again comes back, a large one falls to
    what is left of it, and A = 0 keeps it whatever the steps sum to."""
    rng = np.random.default_rng(3)
    T, d, N = 320, 64, 16
    ids, cu, sk = [1], [0, T], [T + 9]
    v = scan_inputs(rng, T, d, N, 1, "bf16", 2, False, 1.0)

    def put(k, a):
        t = torch.from_numpy(np.broadcast_to(a, v[k][0].shape).copy()).to(v[k][1].dtype)
        v[k] = (t.double().numpy(), t.cuda())

    A, dt = np.ones((d, N)), np.zeros((T, 1))
    if name == "zero":  # nothing comes in before the last tokens
        dt += 3.0
        x = np.zeros((T, 1))
        x[T - 3:] = 1.0
        put("x", x)
        put("state", 0.0)
    elif name == "grows":  # e^96 up and down again within four pieces, from 1e-30
        dt[64:96], dt[96:128] = 3.0, -3.0
        put("x", 0.0)
        put("state", 1e-30 * rng.uniform(1, 2, (2, d, N)))
    elif name == "shrinks":  # e^-96 of 1e30
        dt[64:96] = 3.0
        A = -A
        put("x", 0.0)
        put("state", 1e30 * rng.uniform(1, 2, (2, d, N)))
    else:
        dt = np.full((T, d), float(torch.finfo(torch.bfloat16).min))
        A = 0 * A
        put("x", 0.0)
    put("A", A)
    put("dt", dt)
    h = {k: t[0] for k, t in v.items()}
    want, bound, end, ebound = ref.scan(h["x"], h["dt"], h["A"], h["B"], h["C"], h["D"], h["z"], 0 * h["bias"],
                                        False, h["state"], ids, cu, sk, "bf16")
    for out, st in scan_both(mcp, v, ids, cu, sk, 2, T, d, N, 0):
        assert np.isfinite(st).all()
        assert (np.abs(st - end) <= ebound).all()
        assert (np.abs(out - want) <= bound).all()


# --------------------------------------------------------------------------- logits
def test_biases_of_another_shape_are_refused(mcp):
    """Biases are one list with offsets; a [rows, k] pair would lose most of them."""
    x = torch.zeros((3, 64), device="cuda")
    off, tok, val = i32([0, 2, 4, 6]), i32([1, 5, 2, 9, 3, 7]), torch.ones(6, device="cuda")
    for bias in ((off, tok.view(3, 2), val.view(3, 2)), (off, tok, val.view(3, 2)), (off, tok.view(3, 2), val),
                 (off, tok, val[:5]), (off, tok, None), (off, None, val), (None, tok, val),
                 (off.view(2, 2), tok, val)):
        with pytest.raises((ValueError, TypeError, mcp.MCPError)):
            mcp.process_logits(x, bias=bias)
    assert not x.any()
    mcp.process_logits(x, bias=(off, tok, val))
    assert int(x.sum()) == 6
    mcp.process_logits(x, bias=(i32([0] * 4), tok[:0], val[:0]))
    assert int(x.sum()) == 6


SILU_AT = np.concatenate([np.linspace(-97.25, -80, 70), np.linspace(-12, 12, 97), [-3e38, -1e4, -128.0, 100.0, 3e38, 0.0]])


@pytest.mark.parametrize("T", [1, 3, 80])
def test_silu_far_below_zero(mcp, T):
    """v / (1 + exp(-v)) down to where bf16 has no value for it, in the convolution (one tap of
    1: its sum is exact) and as the scan's gate (B = 0, D x = 1).  Off by at most what the
    definition allows its roundings, and an fp32 step where the quotient is subnormal."""
    d = 256
    v = torch.from_numpy(np.resize(SILU_AT, (T, d))).to(torch.bfloat16)
    v64 = v.double().numpy()
    with np.errstate(over="ignore"):
        want = ref._silu(v64)
        err = np.where(want == 0, 0, ref._silu_err(np.where(want == 0, 0, v64), 0))
    # the quotient's own step, times v
    bound = ref._rounded(want, err + np.minimum(np.abs(v64), 128) * 2.0 ** -149, "bf16")
    w = torch.zeros((d, 2), dtype=torch.bfloat16, device="cuda")
    w[:, 1] = 1
    meta = i32([0]), i32([0, T]), i32([T])
    got = f64(mcp.mixed_conv(v.cuda(), w, None, torch.zeros((1, 1, d), dtype=torch.bfloat16, device="cuda"), *meta))
    assert (np.abs(got - want) <= bound).all()
    one = torch.ones((T, d), dtype=torch.bfloat16, device="cuda")
    bc = torch.zeros((T, 1, 16), dtype=torch.bfloat16, device="cuda")
    got = f64(mcp.mixed_scan(one, one, -torch.ones((d, 16), device="cuda"), bc, bc,
                             torch.zeros((1, d, 16), device="cuda"), *meta, D=torch.ones(d, device="cuda"), z=v.cuda()))
    assert (np.abs(got - want) <= bound).all()


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("what", ["temperature", "repetition"])
def test_logits_over_the_largest_divisors(mcp, what, inplace):
    """Divisors whose reciprocal is subnormal in fp32: quotients that are normal numbers are
    within 3 x 2^-24 (a reciprocal, a product, and half of it again)."""
    rng = np.random.default_rng(5)
    B, V = 64, 130
    by = np.concatenate([[2.0 ** 125, 2.0 ** 126, 2.0 ** 127], rng.uniform(8e37, 3.4e38, B - 3)]).astype(np.float32)
    rows = (10.0 ** rng.uniform(1.5, 38, (B, V))).astype(np.float32)
    if what == "temperature":
        rows *= rng.choice([-1, 1], (B, V))
    src = torch.from_numpy(rows).cuda()
    kw = dict(temperature=torch.from_numpy(by).cuda())
    if what == "repetition":
        seen = np.ones((B, 2, V), bool)
        seen[:, 1] = False
        sd, cd = device_state(seen, np.zeros((B, V), np.int64))
        kw = dict(request_ids=i32(range(B)), seen=sd, counts=cd, repetition_penalty=torch.from_numpy(by).cuda())
    got = f64(mcp.process_logits(src, None if inplace else torch.empty_like(src), **kw))
    want = rows.astype(np.float64) / by.astype(np.float64)[:, None]
    normal = np.abs(want) >= 2.0 ** -126
    assert normal.mean() > 0.9
    assert (np.abs(got - want) <= np.where(normal, 3 * 2.0 ** -24 * np.abs(want), 2.0 ** -148)).all()


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("what", ["temperature", "repetition"])
def test_logits_are_divided(mcp, what, inplace):
    """Quotients in fp32 are off by half a step (2^-24 of them, and 2^-44 of the way there);
    infinities and NaN stay what a division makes of them, by powers of two as well."""
    rng = np.random.default_rng(9)
    B, V = 60, 4099
    by = np.concatenate([[0.25, 0.5, 1.0, 2.0, 64.0, 0.7], 2.0 ** rng.uniform(-40, 40, 20), rng.uniform(0.2, 2, B - 26)])
    by = by.astype(np.float32)
    rows = (rng.normal(size=(B, V)) * 4).astype(np.float32)
    if what == "repetition":
        rows = np.abs(rows)
    rows[:, :3] = np.inf, 0.0, np.nan
    if what == "temperature":
        rows[:, 3] = -np.inf
    src = torch.from_numpy(rows).cuda()
    kw = dict(temperature=torch.from_numpy(by).cuda())
    if what == "repetition":
        seen = np.zeros((B, 2, V), bool)
        seen[:, 0] = True
        sd, cd = device_state(seen, np.zeros((B, V), np.int64))
        kw = dict(request_ids=i32(range(B)), seen=sd, counts=cd, repetition_penalty=torch.from_numpy(by).cuda())
    got = f64(mcp.process_logits(src, None if inplace else torch.empty_like(src), **kw))
    want = rows.astype(np.float64) / by.astype(np.float64)[:, None]
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine], want[~fine], equal_nan=True)
    assert (np.abs(got[fine] - want[fine]) <= 2.0 ** -24 * (1 + 2.0 ** -20) * np.abs(want[fine])).all()


@pytest.mark.parametrize("cu", [[0, 0, 0, 0], [0, 0, 3, 3]])
@pytest.mark.parametrize("prompt", [True, False])
def test_rows_that_cannot_be_cleared_are_reported(mcp, cu, prompt):
    """A row outside the state is reported also where it has no token to add."""
    V, R = 70, 2
    seen, counts = np.ones((R, 2, V), bool), np.full((R, V), 3, np.int64)
    sd, cd = device_state(seen, counts)
    err = err_word()
    ids = [R, 1, -1]
    tokens = [5, 5, 69][:cu[-1]]
    mcp.update_token_counts(i32(ids), i32(tokens), sd, cd, V, i32(cu), prompt, True, err)
    assert int(err) == _capi.DEVERR_REQUEST
    want = device_state(*ref.update_counts(seen, counts, ids, tokens, cu, V, prompt, True))
    assert torch.equal(sd, want[0]) and torch.equal(cd, want[1])


@pytest.mark.parametrize("padded", [False, True])
def test_attention_on_padded_tables(mcp, padded):
    """A step whose slot map is longer than its tokens: keys and values of its tokens alone,
    or padded like the slot map."""
    import math

    from mixed_chunked_prefill_gb300.step import MixedStep, RequestTables

    rng = np.random.default_rng(17)
    Hq, Hkv, D, P, cap = 4, 2, 64, 16, 64
    outs = []
    for room in (None, cap):
        tables = RequestTables(12, P, 3, 4)
        tb = tables.step([1, 0], [21, 9], room)
        T = int(tb.cu_h[-1])
        step = MixedStep.from_tables(tb, Hq, Hkv, D, 1 / math.sqrt(D))
        kc = torch.zeros((12, P, Hkv, D), dtype=torch.bfloat16, device="cuda")
        vc = torch.zeros_like(kc)
        n = cap if padded and room else T
        if not outs:
            q, k, v = (values(rng, (cap, h, D), "bf16")[1] for h in (Hq, Hkv, Hkv))
        out = torch.zeros((n, Hq, D), dtype=torch.bfloat16, device="cuda")
        step.run(q[:n].contiguous(), k[:n].contiguous(), v[:n].contiguous(), kc, vc, out)
        step.check()
        outs.append((out[:T], kc, vc))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    with pytest.raises(ValueError):
        step.append(k[:T - 1].contiguous(), v[:T - 1].contiguous(), kc, vc)
    with pytest.raises(ValueError):
        step.append(torch.cat([k, k]), torch.cat([v, v]), kc, vc)


def test_tables_on_another_stream(mcp):
    """Tables, commit and attention's append on a stream of the caller's, behind what it holds."""
    p, d = ref.Pool(8, 16, 2, 4), Device(mcp, 8, 16, 2, 4)
    s, busy = torch.cuda.Stream(), torch.randn((2048, 2048), device="cuda")
    o = dict(cu=i32([77] * 2), sk=i32([77]), bt=i32([[77] * 4]), slots=torch.full((20,), 77, device="cuda"),
             pos=i32([77] * 20), rows=i32([77]))
    ids, late, q = i32([1]), i32([-1]), i32([20])
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(20):
            torch.mm(busy, busy)
        late.copy_(ids)
    mcp.build_step_tables(d.pool, late, q, o["cu"], o["sk"], o["bt"], o["slots"], o["pos"], o["rows"], d.err,
                          s.cuda_stream)
    mcp.commit_step(d.pool, late, q, None, d.err, s)
    s.synchronize()
    want = p.build([1], [20], 20)
    for got, w in zip(o.values(), want):
        assert np.array_equal(got.cpu().numpy(), w)
    p.commit([1], [20], [20], want[6])
    d.equal(p)


# ------------------------------------------------------------------- many segments
def test_conv_of_many_segments(mcp):
    """Three hundred segments, decodes with speculated tokens among chunks."""
    rng = np.random.default_rng(51)
    lens = rng.choice([1, 1, 1, 1, 2, 3, 4, 5, 17, 33, 0, 64], 300)
    ids, cu, sk, R, T = stream(rng, lens, rng.choice([0, 9], 300), 4, 3)
    for K, d, dtype in ((4, 136, "bf16"), (2, 520, "fp16")):
        x, xd = values(rng, (T, d), dtype)
        w, wd = values(rng, (d, K), dtype)
        b, bd = values(rng, (d,), dtype)
        st, sd = values(rng, (R, K - 1, d), dtype)
        out = torch.full((T, d), 7.0, dtype=DT[dtype], device="cuda")
        err = err_word()
        mcp.mixed_conv(xd, wd, bd, sd, i32(ids), i32(cu), i32(sk), "silu", out, err)
        want, bound, end = ref.conv(x, w, b, st, ids, cu, sk, True, dtype)
        n = cu[-1]
        assert int(err) == 0 and (f64(out)[n:] == 7).all()
        assert (np.abs(f64(out)[:n] - want[:n]) <= bound[:n]).all()
        assert np.array_equal(f64(sd), end)


@pytest.mark.parametrize("N,G,d,dtype", [(16, 1, 72, "bf16"), (64, 2, 64, "fp16"), (8, 1, 264, "bf16"),
                                         (32, 3, 96, "bf16")])
def test_scan_of_many_segments(mcp, N, G, d, dtype):
    """Decodes, padding inside the stream and long segments (many cut) in several blocks of 32."""
    rng = np.random.default_rng(N)
    lens = np.concatenate([rng.choice([1, 1, 2, 3, 4, 0], 90), rng.integers(5, 70, 40), [210, 131, 300, 65, 97]])
    rng.shuffle(lens)
    ids, cu, sk, R, T = stream(rng, lens, rng.choice([0, 9], len(lens)), 3, 2)
    for s in (20, 77):
        ids[s] = -1  # a padding segment that has tokens: left out
    v = scan_inputs(rng, T, d, N, G, dtype, R, True, 1.0)
    out = torch.full((T, d), 7.0, dtype=DT[dtype], device="cuda")
    err = err_word()
    _, (want, bound, end, ebound) = run_scan(mcp, v, ids, cu, sk, "Dzb", True, dtype, out, err)
    ran = np.zeros(T, bool)
    for s, r in enumerate(ids):
        ran[cu[s]:cu[s + 1]] = r >= 0
    assert int(err) == 0 and (f64(out)[~ran] == 7).all()
    assert (np.abs(f64(out)[ran] - want[ran]) <= bound[ran]).all()
    assert (np.abs(f64(v["state"][1]) - end) <= ebound).all()


def test_scan_of_more_segments_than_one_load(mcp):
    """A decode batch in which a warp's share is more than the 32 segments whose metadata it
    loads at once: bit for bit what calls of a few segments each give, and some of them
    against the definition."""
    rng = np.random.default_rng(61)
    S, d, N, R = 700, 8192, 16, 701
    g = torch.Generator(device="cuda")
    g.manual_seed(3)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)

    x, dt, z, B, C = normal(S, d), normal(S, d), normal(S, d), normal(S, 1, N), normal(S, 1, N)
    A, D, bias = -normal(d, N, dtype=torch.float32).exp(), normal(d, dtype=torch.float32), normal(d, dtype=torch.float32)
    state = normal(R, d, N, dtype=torch.float32)
    ids = torch.from_numpy(rng.permutation(R)[:S]).int().cuda()
    ids[rng.permutation(S)[:40]] = -1
    sk = torch.from_numpy(rng.choice([1, 9], S)).int().cuda()
    cu = torch.arange(S + 1, dtype=torch.int32, device="cuda")
    states, outs = [], []
    for step in (S, 60):
        st, out, err = state.clone(), torch.full((S, d), 7.0, dtype=torch.bfloat16, device="cuda"), err_word()
        for a in range(0, S, step):
            s = slice(a, min(S, a + step))
            mcp.mixed_scan(x[s], dt[s], A, B[s], C[s], st, ids[s], cu[:s.stop - a + 1].contiguous(), sk[s], D=D, z=z[s],
                           dt_bias=bias, out=out[s], error_word=err)
        assert int(err) == 0
        states.append(st)
        outs.append(out)
    assert torch.equal(*states) and torch.equal(*outs)
    for s in [0, 1, 31, 32, 33, 600, 607, 608, 609, 640, S - 1] + rng.integers(0, S, 8).tolist():
        r = int(ids[s])
        if r < 0:
            assert (outs[0][s] == 7).all()
            continue
        want, bound, end, ebound = ref.scan(*(f64(t[s:s + 1]) for t in (x, dt)), f64(A), *(f64(t[s:s + 1]) for t in (B, C)),
                                            f64(D), f64(z[s:s + 1]), f64(bias), True, f64(state[r:r + 1]), [0], [0, 1],
                                            [int(sk[s])], "bf16")
        assert (np.abs(f64(outs[0][s]) - want[0]) <= bound[0]).all()
        assert (np.abs(f64(states[0][r]) - end[0]) <= ebound[0]).all()


@pytest.mark.parametrize("lens,pad", [([50], 60), ([1] * 9 + [200, 7] + [1] * 9, 300), ([5, 4, 30], 39)])
@pytest.mark.parametrize("N,d", [(16, 72), (64, 40)])
def test_long_segments_among_more_slots_than_tokens(mcp, lens, pad, N, d):
    """A padded step with at most as many tokens as segment slots may still hold a chunk."""
    rng = np.random.default_rng(len(lens) + N)
    ids, cu, sk, R, T = stream(rng, lens, [5] * len(lens), pad, 0)
    assert T <= len(ids)
    v = scan_inputs(rng, T, d, N, 1, "bf16", R, True, 1.0)
    out, err = torch.full((T, d), 7.0, dtype=torch.bfloat16, device="cuda"), err_word()
    _, (want, bound, end, ebound) = run_scan(mcp, v, ids, cu, sk, "Dzb", True, "bf16", out, err)
    assert int(err) == 0 and (np.abs(f64(out) - want) <= bound).all()
    assert (np.abs(f64(v["state"][1]) - end) <= ebound).all()
