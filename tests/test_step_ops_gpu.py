"""Operators around a step's attention on the GPU, against their definitions in 64
bits.  Whole numbers must be equal; floating values stay inside the bounds that the
definitions carry along (roundings of every intermediate, half a step of the type)."""

from __future__ import annotations

import ctypes

import numpy as np
import pytest

from mixed_chunked_prefill_gb300 import _capi
from oracle import step_ops_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def mcp():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from mixed_chunked_prefill_gb300 import build

    build.build()
    import mixed_chunked_prefill_gb300 as m

    m.load()
    return m


def i32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


def f64(t):
    return t.double().cpu().numpy()


def err_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# --------------------------------------------------------------------------- tables
class Device:
    """A pool on the device and the calls of one step, beside ref.Pool."""

    def __init__(self, m, num_pages, P, R, width):
        self.m, self.width = m, width
        self.pages = torch.full((R, width), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(R, dtype=torch.int32, device="cuda")
        self.free = torch.arange(num_pages, dtype=torch.int32, device="cuda")
        self.count = i32([num_pages])
        self.err = err_word()
        self.pool = m.make_request_pool(self.pages, self.lens, self.free, self.count, P)

    def build(self, ids, q, cap, stream=None):
        S = len(ids)
        o = dict(cu=torch.full((S + 1,), 77, dtype=torch.int32, device="cuda"),
                 sk=torch.full((S,), 77, dtype=torch.int32, device="cuda"),
                 bt=torch.full((S, self.width), 77, dtype=torch.int32, device="cuda"),
                 slots=torch.full((cap,), 77, dtype=torch.int64, device="cuda"),
                 pos=torch.full((cap,), 77, dtype=torch.int32, device="cuda"),
                 rows=torch.full((S,), 77, dtype=torch.int32, device="cuda"))
        self.m.build_step_tables(self.pool, i32(ids), i32(q), o["cu"], o["sk"], o["bt"], o["slots"],
                                 o["pos"], o["rows"], self.err, stream)
        return [o[k].cpu().numpy() for k in ("cu", "sk", "bt", "slots", "pos", "rows")]

    def commit(self, ids, q, new=None):
        self.m.commit_step(self.pool, i32(ids), i32(q), None if new is None else i32(new), self.err)

    def equal(self, p: ref.Pool):
        assert int(self.count) == len(p.free)
        assert self.free[:len(p.free)].tolist() == p.free
        assert self.lens.tolist() == p.lens
        pages = self.pages.cpu().numpy()
        for r, have in enumerate(p.pages):
            assert pages[r, :len(have)].tolist() == have, r
        assert int(self.err) == 0


@pytest.mark.parametrize("P,width,R,seed", [(1, 97, 9, 0), (8, 33, 7, 1), (16, 64, 40, 2),
                                            (32, 2051, 5, 3), (64, 3, 300, 4), (16, 4100, 3, 5)])
def test_steps_of_a_server(mcp, P, width, R, seed):
    """Twelve steps: prompts, chunks, decodes and padding, with commits that keep everything,
    reject the last tokens, or end requests."""
    rng = np.random.default_rng(seed)
    most = min(width * P, 3000)
    num_pages = R * (-(-most // P))
    p, d = ref.Pool(num_pages, P, R, width), Device(mcp, num_pages, P, R, width)
    for step in range(12):
        ids = rng.permutation(R)[:rng.integers(1, R + 1)]
        ids = np.where(rng.random(len(ids)) < 0.15, -1, ids).tolist()
        q = [0 if r < 0 else int(min(most - p.lens[r], rng.choice([0, 1, 1, 2, P, P + 1, 37, most])))
             for r in ids]
        q = [7 if r < 0 else n for r, n in zip(ids, q)]  # a padding segment's length means nothing
        T = sum(n for r, n in zip(ids, q) if r >= 0)
        cap = T + int(rng.integers(0, 3)) * 11
        want = p.build(ids, q, cap)
        for _ in range(2):  # building changes nothing: the same step again is the same
            for got, w in zip(d.build(ids, q, cap), want[:6]):
                assert np.array_equal(got, w)
        if step % 3 == 0:
            new = want[1].tolist()
            d.commit(ids, q)
        else:
            new = [0 if r < 0 else 0 if rng.random() < 0.3 else int(rng.integers(0, s + 1)) if
                   rng.random() < 0.3 else int(s) for r, s in zip(ids, want[1])]
            d.commit(ids, q, new)
        p.commit(ids, q, new, want[6])
        d.equal(p)


def test_many_segments(mcp):
    """The largest step: 8192 segments, and a commit over several CTAs."""
    rng = np.random.default_rng(11)
    S, P = 8192, 16
    p, d = ref.Pool(3 * S, P, S + 5, 4), Device(mcp, 3 * S, P, S + 5, 4)
    ids = rng.permutation(S + 5)[:S].tolist()
    q = rng.integers(0, 40, S).tolist()
    want = p.build(ids, q, sum(q))
    for got, w in zip(d.build(ids, q, sum(q)), want[:6]):
        assert np.array_equal(got, w)
    new = [int(rng.integers(0, s + 1)) for s in want[1]]
    d.commit(ids, q, new)
    p.commit(ids, q, new, want[6])
    d.equal(p)


def test_no_segments(mcp):
    d = Device(mcp, 4, 16, 2, 2)
    cu, sk, bt, slots, pos, rows = d.build([], [], 5)
    assert cu.tolist() == [0] and slots.tolist() == [-1] * 5 and pos.tolist() == [0] * 5
    d.commit([], [])
    d.equal(ref.Pool(4, 16, 2, 2))


@pytest.mark.parametrize("ids,q,cap,bit", [
    ([0, 1, 0], [1, 1, 1], 8, 0x80), ([0, 3], [1, 1], 8, 0x80), ([1], [-1], 8, 0x80),
    ([1], [65], 99, 0x80), ([0, 1], [5, 4], 8, 0x80), ([0, 1, 2], [60, 60, 60], 200, 0x80),
    ([0, 1, 2], [60, 60, 40], 200, 0x40),
])
def test_refused_steps_change_nothing(mcp, ids, q, cap, bit):
    p, d = ref.Pool(10, 16, 3, 4), Device(mcp, 10, 16, 3, 4)
    want = p.build([2, 0], [17, 3], 20)
    d.build([2, 0], [17, 3], 20)
    d.commit([2, 0], [17, 3])
    p.commit([2, 0], [17, 3], [17, 3], want[6])
    before = d.pages.clone()
    for _ in range(2):
        cu, sk, bt, slots, pos, rows = d.build(ids, q, cap)
        assert int(d.err) == bit
        assert not cu.any() and not sk.any() and not pos.any()
        assert (bt == -1).all() and (slots == -1).all() and (rows == -1).all()
        d.err.zero_()
        for new in (None, [0] * len(ids)):
            if (cap < sum(q)) and bit == 0x80 and max(q) < 10:
                continue  # only the tables were too short: the commit of such a step is sound
            d.commit(ids, q, new)
            assert int(d.err) & bit
            d.err.zero_()
        assert torch.equal(before, d.pages)
        d.equal(p)


@pytest.mark.parametrize("new", [[-1], [21]])
def test_refused_commit_changes_nothing(mcp, new):
    p, d = ref.Pool(10, 16, 3, 4), Device(mcp, 10, 16, 3, 4)
    d.build([1], [20], 20)
    d.commit([1], [20], new)
    assert int(d.err) == 0x80
    d.err.zero_()
    d.equal(p)


def test_damaged_free_count_is_refused(mcp):
    for bad in (-1, 11):
        d = Device(mcp, 10, 16, 3, 4)
        d.count.fill_(bad)
        cu, *_ = d.build([1], [20], 20)
        assert int(d.err) == 0x40 and not cu.any()
        d.commit([1], [20])
        assert int(d.count) == bad and not d.lens.any()


# ------------------------------------------------------------------- packed streams
def stream(rng, lens, hist, pad, behind):
    """Metadata of a packed stream with padding segments behind it: (ids, cu, sk, requests, T)."""
    n = len(lens)
    ids = rng.permutation(n + 2)[:n].tolist() + [-1] * pad
    lens = list(lens) + [0] * pad
    hist = list(hist) + [0] * pad
    cu = np.concatenate([[0], np.cumsum(lens)])
    return ids, cu.tolist(), [a + b for a, b in zip(lens, hist)], n + 2, int(cu[-1]) + behind


def values(rng, shape, dtype, scale=1.0):
    """Random values of a type, as float64 and on the device."""
    t = torch.from_numpy(rng.normal(size=shape) * scale).to(DT[dtype])
    return t.double().numpy(), t.cuda()


STREAMS = {
    "decodes": ([1] * 9, [5] * 9, 2, 3),
    "one token": ([1], [0], 0, 0),
    "mixed": ([1, 3, 0, 2, 40, 1, 0, 17], [4, 0, 9, 8, 12, 0, 0, 3], 1, 5),
    "runs": ([15, 16, 17, 1, 2, 31, 33], [0, 3, 0, 3, 1, 0, 2], 0, 0),
    "starts at run ends": ([14, 2, 15, 2, 13, 4, 64], [1] * 7, 0, 1),
    "a chunk": ([300], [1000], 3, 0),
}


@pytest.mark.parametrize("name", STREAMS)
@pytest.mark.parametrize("K,dtype,d,silu,bias", [(4, "bf16", 72, True, True), (2, "fp16", 8, False, True),
                                                 (3, "bf16", 1032, True, False),
                                                 (4, "fp16", 2048, True, True)])
def test_conv(mcp, name, K, dtype, d, silu, bias):
    rng = np.random.default_rng(len(name) + K)
    ids, cu, sk, R, T = stream(rng, *STREAMS[name])
    x, _ = values(rng, (T, d), dtype)
    x[cu[-1]:] = np.nan  # behind the stream: not read
    wide = torch.full((T, 2 * d), float("nan"), dtype=DT[dtype], device="cuda")
    wide[:, d:] = torch.from_numpy(x).to(DT[dtype])
    w, wd = values(rng, (d, K), dtype)
    b, bd = values(rng, (d,), dtype)
    st, sd = values(rng, (R, K - 1, d), dtype)
    out = torch.full((T, d), 7.0, dtype=DT[dtype], device="cuda")
    err = err_word()
    got = mcp.mixed_conv(wide[:, d:], wd, bd if bias else None, sd, i32(ids), i32(cu), i32(sk),
                         "silu" if silu else "none", out, err)
    want, bound, end = ref.conv(x, w, b if bias else 0 * b, st, ids, cu, sk, silu, dtype)
    assert got is out and int(err) == 0
    n = cu[-1]
    assert (np.abs(f64(out)[:n] - want[:n]) <= bound[:n]).all()
    assert (f64(out)[n:] == 7).all()
    assert np.array_equal(f64(sd), end)


def scan_inputs(rng, T, d, N, G, dtype, R, softplus, spread):
    v = dict(x=values(rng, (T, d), dtype), z=values(rng, (T, d), dtype),
             B=values(rng, (T, G, N), dtype), C=values(rng, (T, G, N), dtype))
    dt = rng.normal(size=(T, d)) * spread - (3 if softplus else 0)
    dt = torch.from_numpy(dt if softplus else np.abs(dt) * 0.1).to(DT[dtype])
    v["dt"] = (dt.double().numpy(), dt.cuda())
    for k, a in dict(A=-np.exp(rng.normal(size=(d, N))), D=rng.normal(size=d),
                     bias=rng.normal(size=d), state=rng.normal(size=(R, d, N))).items():
        t = torch.from_numpy(a).float()
        v[k] = (t.double().numpy(), t.cuda())
    return v


def run_scan(mcp, v, ids, cu, sk, parts, softplus, dtype, out, err, stream=None):
    dev = {k: t[1] for k, t in v.items()}
    got = mcp.mixed_scan(dev["x"], dev["dt"], dev["A"], dev["B"], dev["C"], dev["state"], i32(ids),
                         i32(cu), i32(sk), D=dev["D"] if "D" in parts else None,
                         z=dev["z"] if "z" in parts else None,
                         dt_bias=dev["bias"] if "b" in parts else None, softplus=softplus, out=out,
                         error_word=err, stream=stream)
    h = {k: t[0] for k, t in v.items()}
    want = ref.scan(h["x"], h["dt"], h["A"], h["B"], h["C"], h["D"] if "D" in parts else 0 * h["D"],
                    h["z"] if "z" in parts else None, h["bias"] if "b" in parts else 0 * h["bias"],
                    softplus, h["state"], ids, cu, sk, dtype)
    return got, want


@pytest.mark.parametrize("name", STREAMS)
@pytest.mark.parametrize("N,G,d,dtype,parts,softplus", [
    (16, 1, 40, "bf16", "Dzb", True), (8, 1, 8, "fp16", "", False), (16, 2, 64, "fp16", "zb", True),
    (32, 1, 72, "bf16", "Db", True), (64, 3, 96, "fp16", "Dz", False), (8, 1, 264, "bf16", "Dzb", True),
])
def test_scan(mcp, name, N, G, d, dtype, parts, softplus):
    rng = np.random.default_rng(len(name) + N)
    ids, cu, sk, R, T = stream(rng, *STREAMS[name])
    v = scan_inputs(rng, T, d, N, G, dtype, R, softplus, 2.0)
    n = cu[-1]
    for k in ("x", "dt", "z", "B", "C"):  # behind the stream: not read
        v[k][0][n:], v[k][1][n:] = np.nan, float("nan")
    out = torch.full((T, d), 7.0, dtype=DT[dtype], device="cuda")
    err = err_word()
    _, (want, bound, end, ebound) = run_scan(mcp, v, ids, cu, sk, parts, softplus, dtype, out, err)
    assert int(err) == 0
    assert (np.abs(f64(out)[:n] - want[:n]) <= bound[:n]).all()
    assert (f64(out)[n:] == 7).all()
    assert (np.abs(f64(v["state"][1]) - end) <= ebound).all()
    untouched = sorted(set(range(R)) - {r for i, r in enumerate(ids) if r >= 0 and cu[i + 1] > cu[i]})
    assert np.array_equal(f64(v["state"][1])[untouched], v["state"][0][untouched])


def test_scan_of_large_and_vanishing_steps(mcp):
    """Steps for which exp(d A) is 0 or 1, softplus far on both sides, rows of zeros."""
    rng = np.random.default_rng(2)
    T, d, N = 70, 32, 16
    ids, cu, sk = [1], [0, T], [T + 9]
    v = scan_inputs(rng, T, d, N, 1, "bf16", 2, True, 30.0)
    for k in (0, 1):
        v["A"][k][3], v["A"][k][4] = -1e30, 0.0
        v["x"][k][10:20] = 0
    out, err = torch.empty((T, d), dtype=torch.bfloat16, device="cuda"), err_word()
    _, (want, bound, end, ebound) = run_scan(mcp, v, ids, cu, sk, "Dzb", True, "bf16", out, err)
    assert (np.abs(f64(out) - want) <= bound).all()
    assert (np.abs(f64(v["state"][1]) - end) <= ebound).all()


@pytest.mark.parametrize("T", [1, 3, 70, 400])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_scan_of_infinite_steps(mcp, T, dtype):
    """A step of minus infinity (or the type's lowest value) is softplus 0: the state stays
    and the output is C h + D x, as for a step of -9984.  The highest value with x = 0 ends
    in a state of 0, and NaN stays NaN in its own channel."""
    rng = np.random.default_rng(T)
    d, N = 64, 16
    ids, cu, sk = [1], [0, T], [T + 9]
    v = scan_inputs(rng, T, d, N, 1, dtype, 2, True, 1.0)
    at = T // 2
    v["A"][1][41] = 0.0
    states, outs = [], []
    for low in (-9984.0, float("-inf"), torch.finfo(DT[dtype]).min):
        dt, st = v["dt"][1].clone(), v["state"][1].clone()
        dt[at, :32] = low
        dt[0, 32:40] = torch.finfo(DT[dtype]).max
        dt[at, 40] = float("nan")
        x = v["x"][1].clone()
        x[:, 32:40] = 0
        dt[:, 41], x[:, 41] = torch.finfo(DT[dtype]).max, 0
        outs.append(mcp.mixed_scan(x, dt, v["A"][1], v["B"][1], v["C"][1], st, i32(ids), i32(cu), i32(sk),
                                   D=v["D"][1], z=v["z"][1], dt_bias=v["bias"][1]))
        states.append(st)
    for o, s in zip(outs, states):
        keep = torch.arange(d, device="cuda") != 40
        assert torch.equal(o[:, keep], outs[0][:, keep]) and torch.equal(s[:, keep], states[0][:, keep])
        assert torch.isfinite(s[:, keep]).all() and not s[1, 32:40].any()
        assert torch.equal(s[1, 41], v["state"][1][1, 41])  # A = 0: kept, whatever the step
        assert s[1, 40].isnan().all() and o[at:, 40].isnan().all() and torch.isfinite(o[:at]).all()


def test_scan_in_one_piece_and_in_several(mcp):
    """The C entry without a workspace runs a segment in one piece, with one in several
    (of which those in between are run twice); both stay in the bounds, and a workspace
    that is too small is refused."""
    rng = np.random.default_rng(12)
    T, d, N = 500, 96, 16
    lens, hist = [70, 1, 300, 129], [0, 4, 9, 9]
    ids, cu, sk, R, T = stream(rng, lens, hist, 1, 2)
    v = scan_inputs(rng, T, d, N, 1, "bf16", R, True, 1.0)
    h = {k: t[0] for k, t in v.items()}
    want, bound, end, ebound = ref.scan(h["x"], h["dt"], h["A"], h["B"], h["C"], h["D"], h["z"], h["bias"],
                                        True, h["state"], ids, cu, sk, "bf16")
    dev = {k: t[1] for k, t in v.items()}
    lib = mcp.load()
    meta = [i32(a) for a in (ids, cu, sk)]
    S = len(ids)
    desc = _capi.ScanDesc(S, T, R, d, N, 1, 0, 1, d, d, d, N, N, d)
    need = ctypes.c_size_t()
    assert lib.mcp_mixed_scan_workspace(ctypes.byref(desc), ctypes.byref(need)) == 0 and need.value > 256
    stream_ = torch.cuda.current_stream().cuda_stream
    results = []
    for n in (0, need.value - 1, need.value):
        ws = torch.full((max(n, 1),), 255, dtype=torch.uint8, device="cuda")
        out = torch.full((T, d), 7.0, dtype=torch.bfloat16, device="cuda")
        st = dev["state"].clone()
        tensors = _capi.ScanTensors(*(t.data_ptr() for t in (
            dev["x"], dev["dt"], dev["A"], dev["B"], dev["C"], dev["D"], dev["z"], dev["bias"], st, out)))
        r = lib.mcp_mixed_scan(ctypes.byref(desc), ctypes.byref(tensors), *(t.data_ptr() for t in meta),
                               ws.data_ptr() if n else None, n, None, stream_)
        if n == need.value - 1:
            assert r == _capi.MCP_ERR_WORKSPACE_TOO_SMALL and torch.equal(st, dev["state"])
            continue
        assert r == 0
        assert (np.abs(f64(out)[:cu[-1]] - want[:cu[-1]]) <= bound[:cu[-1]]).all()
        assert (np.abs(f64(st) - end) <= ebound).all()
        results.append(st)
    assert not torch.equal(*results)  # the second was cut


def test_parts_of_wider_rows(mcp):
    """x and z from one projection, B and C from another, the output inside a wider buffer."""
    rng = np.random.default_rng(8)
    T, d, N = 37, 64, 16
    v = scan_inputs(rng, T, d, N, 1, "bf16", 3, True, 1.0)
    xz = torch.cat([v["x"][1], v["z"][1]], 1)
    bc = torch.cat([torch.zeros(T, 24, dtype=torch.bfloat16, device="cuda"), v["B"][1].flatten(1),
                    v["C"][1].flatten(1)], 1)
    v["x"], v["z"] = (v["x"][0], xz[:, :d]), (v["z"][0], xz[:, d:])
    v["B"], v["C"] = (v["B"][0], bc[:, 24:40].unflatten(1, (1, N))), (v["C"][0], bc[:, 40:].unflatten(1, (1, N)))
    wide = torch.full((T, 3 * d), 5.0, dtype=torch.bfloat16, device="cuda")
    _, (want, bound, *_) = run_scan(mcp, v, [2], [0, T], [T], "Dzb", True, "bf16", wide[:, d:2 * d], None)
    assert (np.abs(f64(wide[:, d:2 * d]) - want) <= bound).all()
    assert (wide[:, :d] == 5).all() and (wide[:, 2 * d:] == 5).all()


@pytest.mark.parametrize("ids,cu,sk,bit,good", [
    ([0, 5], [0, 2, 4], [2, 2], 0x80, [0]),      # a request row outside the state
    ([0, 1], [0, 2, 9], [2, 9], 0x200, [0]),     # a segment past the stream
    ([0, 1], [0, 4, 2], [4, 0], 0x200, []),      # a decreasing prefix sum
    ([0, 1], [0, 2, 4], [2, 1], 0x200, [0, 1]),  # a length that leaves out the segment's tokens
    ([3, 3, 0], [0, 1, 2, 4], [1, 1, 2], 0x80, [2]),  # a request twice
])
def test_bad_streams_are_reported(mcp, ids, cu, sk, bit, good):
    rng = np.random.default_rng(1)
    T, d, K, N = 4, 16, 4, 8
    x, xd = values(rng, (T, d), "bf16")
    w, wd = values(rng, (d, K), "bf16")
    b, bd = values(rng, (d,), "bf16")
    st, sd = values(rng, (4, K - 1, d), "bf16")
    out, err = torch.full((T, d), 7.0, dtype=torch.bfloat16, device="cuda"), err_word()
    mcp.mixed_conv(xd, wd, bd, sd, i32(ids), i32(cu), i32(sk), "silu", out, err)
    assert int(err) == bit
    for s in good:
        want, bound, _ = ref.conv(x, w, b, st, [ids[s]], [cu[s], cu[s + 1]], [sk[s]], True, "bf16")
        rows = slice(cu[s], cu[s + 1])
        assert (np.abs(f64(out)[rows] - want[rows]) <= bound[rows]).all()
    v = scan_inputs(rng, T, d, N, 1, "bf16", 4, True, 1.0)
    err.zero_()
    mcp.mixed_scan(v["x"][1], v["dt"][1], v["A"][1], v["B"][1], v["C"][1], v["state"][1], i32(ids),
                   i32(cu), i32(sk), out=out, error_word=err)
    assert int(err) == bit
    assert np.array_equal(f64(v["state"][1])[2], v["state"][0][2])  # no segment's request


# --------------------------------------------------------------------------- logits
def token_state(rng, R, V, many):
    seen, counts = np.zeros((R, 2, V), bool), np.zeros((R, V), np.int64)
    for r in range(R):
        seen[r, 0, rng.integers(0, V, many)] = True
        np.add.at(counts[r], rng.integers(0, max(1, V // 3), many), 1)
    seen[:, 1] = counts > 0
    return seen, counts


def device_state(seen, counts):
    R, _, V = seen.shape
    wide = np.zeros((R, -(-V // 32) * 32), np.int64)
    wide[:, :V] = counts
    return torch.from_numpy(ref.pack_bits(seen)).cuda(), i32(wide)


@pytest.mark.parametrize("V", [1, 31, 32, 1000, 70001])
@pytest.mark.parametrize("prompt,reset", [(True, True), (False, False), (False, True), (True, False)])
def test_update_counts(mcp, V, prompt, reset):
    rng = np.random.default_rng(V)
    R = 6
    seen, counts = token_state(rng, R, V, 50)
    sd, cd = device_state(seen, counts)
    ids = [4, -1, 0, 4, 2, 3]  # padding, and a request twice
    lens = [0, 5, 700, 33, 1, 257]
    cu = np.concatenate([[0], np.cumsum(lens)])
    tokens = np.minimum(V - 1, (V ** rng.random(cu[-1])).astype(int))
    tokens[::17] = -1
    tokens = np.concatenate([tokens, [1 << 30] * 9])  # behind the last row: not read
    err = err_word()
    mcp.update_token_counts(i32(ids), i32(tokens), sd, cd, V, i32(cu), prompt, reset, err)
    seen, counts = ref.update_counts(seen, counts, ids, tokens, cu, V, prompt, reset)
    want = device_state(seen, counts)
    assert torch.equal(sd, want[0]) and torch.equal(cd, want[1]) and int(err) == 0
    one = [int(t) for t in rng.integers(0, V, R)]
    mcp.update_token_counts(i32(ids), i32(one), sd, cd, V, error_word=err)
    want = device_state(*ref.update_counts(seen, counts, ids, one, None, V, False, False))
    assert torch.equal(sd, want[0]) and torch.equal(cd, want[1]) and int(err) == 0


@pytest.mark.parametrize("lens,prompt,V,first", [
    ([9000, 0, 0, 3, 5000, 1, 8000], True, 1000, 0), ([30000], True, 50000, 0),
    ([5, 7, 0, 40000], True, 300001, 3), ([12000, 0, 9000], False, 70, 1),
    ([3000, 6000, 1023, 1024, 1025], True, 262200, 0), ([20001, 1], False, 5001, 2),
    ([0] * 20 + [45000], True, 128000, 0),
])
@pytest.mark.parametrize("reset", [False, True])
def test_counts_of_long_texts(mcp, lens, prompt, V, first, reset):
    """Texts long enough for bitmaps, between short and empty ones, on addresses of any
    alignment, with padding tokens, rows of the same request and ranges left out."""
    rng = np.random.default_rng(len(lens) + V + first)
    R, rows, W = 6, len(lens), -(-V // 32)
    ids = rng.integers(0, R, rows)
    cu = np.concatenate([[0], np.cumsum(lens)]) + first
    n = int(cu[-1]) + 100  # tokens behind the last row are not read
    tokens = np.minimum(((V + 1.0) ** rng.random(n) - 1).astype(np.int64), V - 1)
    tokens[rng.random(n) < 0.05] = -1
    tokens[rng.integers(first, int(cu[-1]))] = V
    seen, counts = token_state(rng, R, V, 40)
    sd, cd = device_state(seen, counts)
    err = i32([0])
    td = i32(np.concatenate([[0] * (first % 4), tokens]))[first % 4:]
    mcp.update_token_counts(i32(ids), td, sd, cd, V, i32(cu), prompt, reset, err)
    legal = np.where(tokens >= V, -1, tokens)
    seen, counts = ref.update_counts(seen, counts, ids, legal, cu, V, prompt, reset)
    want = device_state(seen, counts)
    assert torch.equal(sd, want[0]) and torch.equal(cd, want[1])
    assert int(err) == _capi.DEVERR_TOKEN_RANGE and W == sd.shape[2]


def test_counts_out_of_range_are_left_out(mcp):
    seen, counts = np.zeros((2, 2, 40), bool), np.zeros((2, 40), np.int64)
    for ids, tok, bit in (([0, 1], [40, 3], 0x100), ([2, 1], [1, 3], 0x80)):
        sd, cd = device_state(seen, counts)
        err = err_word()
        mcp.update_token_counts(i32(ids), i32(tok), sd, cd, 40, reset=True, error_word=err)
        assert int(err) == bit
        want = device_state(*ref.update_counts(seen, counts, ids, tok, None, 40, False, True))
        assert torch.equal(sd, want[0]) and torch.equal(cd, want[1])


def logit_case(rng, B, V, dtype):
    R = B + 2
    x, xd = values(rng, (B, V), dtype, 4.0)
    seen, counts = token_state(rng, R, V, 60)
    ids = rng.permutation(R)[:B]
    if B > 2:
        ids[1] = -1
    p = {k: torch.from_numpy(rng.uniform(*r, B)).float() for k, r in
         dict(temperature=(0.3, 2), repetition_penalty=(0.5, 2), frequency_penalty=(-1, 1),
              presence_penalty=(-1, 1)).items()}
    p["temperature"][0] = 0 if B > 1 else 1
    if B > 3:
        p["temperature"][3] = 1
    bias = {i: {int(v): float(np.float32(rng.normal() * 5)) for v in
                sorted(rng.choice(V, min(V, 7 + i), replace=False))} for i in range(0, B, 2)}
    bias.setdefault(0, {})[V - 1] = float("-inf")
    mrows = np.where(rng.random(B) < 0.5, -1, rng.integers(0, 3, B))
    allow = rng.random((3, V)) < 0.3
    allow[2] = False  # a mask that leaves nothing
    if B > 4:
        mrows[4] = 2
    return x, xd, seen, counts, ids, p, bias, mrows, allow


def bias_tensors(bias, B):
    off, tok, val = [0], [], []
    for i in range(B):
        for v in sorted(bias.get(i, {})):
            tok.append(v)
            val.append(bias[i][v])
        off.append(len(tok))
    return i32(off), i32(tok), torch.tensor(val, dtype=torch.float32, device="cuda")


@pytest.mark.parametrize("B,V", [(1, 1), (5, 33), (7, 2048), (3, 2049), (6, 50001), (5, 32000)])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"),
                                       ("fp32", "fp32"), ("bf16", None), ("fp32", None)])
@pytest.mark.parametrize("on", ["all", "penalties", "mask", "nothing"])
def test_logits(mcp, B, V, dtype, out, on):
    rng = np.random.default_rng(B + V)
    x, xd, seen, counts, ids, p, bias, mrows, allow = logit_case(rng, B, V, dtype)
    sd, cd = device_state(seen, counts)
    kw, h = {}, dict(temperature=None, rho=np.ones(B), freq=np.zeros(B), pres=np.zeros(B), bias={},
                     allow=None, ids=None)
    if on in ("all", "penalties"):
        kw.update(request_ids=i32(ids), seen=sd, counts=cd)
        kw.update({k: t.cuda() for k, t in p.items() if k != "temperature"})
        h.update(ids=ids.tolist(), rho=p["repetition_penalty"].double().numpy(),
                 freq=p["frequency_penalty"].double().numpy(), pres=p["presence_penalty"].double().numpy())
    if on == "all":
        kw.update(temperature=p["temperature"].cuda(), bias=bias_tensors(bias, B))
        h.update(temperature=p["temperature"].double().numpy(), bias=bias)
    if on in ("all", "mask"):
        kw.update(mask=torch.from_numpy(ref.pack_bits(allow)).cuda(), mask_rows=i32(mrows))
        h["allow"] = [allow[m] if m >= 0 else None for m in mrows]
        if B > 2:
            x[:, 3], xd[:, 3] = np.nan, float("nan")  # where a mask takes it, it is gone
    err = err_word()
    dst = None if out is None else torch.full((B, V), 3.0, dtype=DT[out], device="cuda")
    got = mcp.process_logits(xd, dst, error_word=err, **kw)
    assert int(err) == 0 and got is (xd if out is None else dst)
    want, bound = ref.logits(x, h["ids"], seen, counts, h["temperature"], h["rho"], h["freq"], h["pres"],
                             h["bias"], h["allow"], out or dtype)
    g = f64(got)
    for i in range(B):
        if h["ids"] is not None and h["ids"][i] < 0:  # padding: not written
            assert (g[i] == 3).all() if out is not None else np.array_equal(g[i], x[i], equal_nan=True)
            continue
        fine = np.isfinite(want[i])
        assert (np.abs(g[i][fine] - want[i][fine]) <= bound[i][fine]).all()
        assert np.array_equal(g[i][~fine], want[i][~fine], equal_nan=True)


@pytest.mark.parametrize("V,dtype,out,off,temp", [
    (60001, "bf16", None, 0, True), (60001, "fp16", None, 0, False), (60002, "fp32", None, 0, True),
    (60000, "bf16", "fp32", 0, True), (60001, "bf16", "fp32", 1, True), (60003, "fp32", "fp32", 3, False),
    (65536, "bf16", "bf16", 0, True),
])
def test_logits_of_rows_in_several_parts(mcp, V, dtype, out, off, temp):
    """Rows that several CTAs take, each of them more than one tile, with most tokens seen:
    every token is processed once, also where one part ends and the next begins."""
    rng = np.random.default_rng(V + off)
    B, R = 90, 4
    x, _ = values(rng, (B, V), dtype, 4.0)
    wide = torch.zeros((B, V + off), dtype=DT[dtype], device="cuda")
    wide[:, off:] = torch.from_numpy(x).to(DT[dtype])
    seen = rng.random((R, 2, V)) < 0.7
    counts = np.where(seen[:, 1], rng.integers(1, 9, (R, V)), 0)
    sd, cd = device_state(seen, counts)
    ids = rng.integers(0, R, B)
    f = {k: torch.from_numpy(rng.uniform(*r, B)).float() for k, r in
         dict(repetition_penalty=(0.5, 2), frequency_penalty=(-1, 1), presence_penalty=(-1, 1),
              temperature=(0.3, 2)).items()}
    allow = rng.random((2, V)) < 0.6
    mrows = rng.integers(-1, 2, B)
    dst = None if out is None else torch.empty((B, V), dtype=DT[out], device="cuda")
    got = mcp.process_logits(
        wide[:, off:], dst, i32(ids), sd, cd, f["temperature"].cuda() if temp else None,
        f["repetition_penalty"].cuda(), f["frequency_penalty"].cuda(), f["presence_penalty"].cuda(),
        mask=torch.from_numpy(ref.pack_bits(allow)).cuda(), mask_rows=i32(mrows))
    n = {k: t.double().numpy() for k, t in f.items()}
    want, bound = ref.logits(x, ids, seen, counts, n["temperature"] if temp else None,
                             n["repetition_penalty"], n["frequency_penalty"], n["presence_penalty"], {},
                             [allow[m] if m >= 0 else None for m in mrows], out or dtype)
    g = f64(got)
    fine = np.isfinite(want)
    assert (np.abs(g[fine] - want[fine]) <= bound[fine]).all()
    assert np.array_equal(g[~fine], want[~fine])
    assert not wide[:, :off].any()


@pytest.mark.parametrize("inplace", [False, True])
def test_logits_with_the_smallest_temperatures(mcp, inplace):
    """Temperatures whose reciprocal is no fp32 number: quotients are right where they are
    finite and infinite where they are not.  Each is two products with three roundings
    (reciprocal, product, and the half step of a subnormal temperature's own scaling: none,
    2^64 being a power of two), so within 3 x 2^-24."""
    temps = np.array([1e-45, 1e-40, 2.8e-39, 3e-39, 9e-38, 1.1e-37, 1.0, 3e38], np.float32)
    x = np.array([0.0, 1e-38, -2e-38, 3e-7, -1.0, 2.5, 1e30, -np.inf], np.float32)
    V = 70
    rows = np.tile(np.resize(x, V), (len(temps), 1))
    src = torch.from_numpy(rows).cuda()
    got = mcp.process_logits(src, None if inplace else torch.empty_like(src),
                             temperature=torch.from_numpy(temps).cuda())
    with np.errstate(over="ignore"):
        want = rows.astype(np.float64) / temps.astype(np.float64)[:, None]
        as32 = want.astype(np.float32)
    g = got.cpu().numpy()
    normal = np.isfinite(as32) & (np.abs(want) > 2e-38)
    assert np.array_equal(g[~np.isfinite(as32)], as32[~np.isfinite(as32)])
    assert (np.abs(g[normal] - want[normal]) <= 3 * 2.0 ** -24 * np.abs(want[normal])).all()
    small = np.isfinite(as32) & ~normal  # subnormal quotients: steps of 2^-149
    assert (np.abs(g[small] - want[small]) <= 2.0 ** -148 + 3 * 2.0 ** -24 * np.abs(want[small])).all()


def test_logits_of_a_padded_head(mcp):
    """Rows of a head whose vocabulary is padded, in place: the padding stays as it was."""
    rng = np.random.default_rng(4)
    B, V = 4, 1003
    x, xd, seen, counts, ids, p, *_ = logit_case(rng, B, V, "bf16")
    ids = np.array([3, 1, 0, 5])
    for pad, off in ((21, 0), (24, 0), (5, 1)):
        wide = torch.full((B, V + pad), 9.0, dtype=torch.bfloat16, device="cuda")
        wide[:, off:off + V] = xd
        sd, cd = device_state(seen, counts)
        mcp.process_logits(wide[:, off:off + V], request_ids=i32(ids), seen=sd, counts=cd,
                           presence_penalty=p["presence_penalty"].cuda(), temperature=p["temperature"].cuda())
        want, bound = ref.logits(x, ids, seen, counts, p["temperature"].double().numpy(), np.ones(B),
                                 np.zeros(B), p["presence_penalty"].double().numpy(), {}, None, "bf16")
        assert (np.abs(f64(wide[:, off:off + V]) - want) <= bound).all()
        assert (wide[:, :off] == 9).all() and (wide[:, off + V:] == 9).all()


def test_bad_logit_rows_are_reported(mcp):
    rng = np.random.default_rng(6)
    V = 100
    seen, counts = token_state(rng, 3, V, 10)
    sd, cd = device_state(seen, counts)
    mask = torch.zeros((1, 4), dtype=torch.int32, device="cuda")
    x, xd = values(rng, (2, V), "fp32")
    out, err = torch.full((2, V), 3.0, device="cuda"), err_word()
    mcp.process_logits(xd, out, i32([3, 0]), sd, cd, mask=mask, mask_rows=i32([-1, 1]), error_word=err)
    assert int(err) == 0x80 and (out == 3).all()
    val = torch.ones(4, device="cuda")
    for tok, off, bit in (([1, 1, 2, 3], [0, 4, 4], 0x100), ([1, 5, 4, 9], [0, 2, 4], 0),
                          ([1, 5, 4, 9], [0, 3, 4], 0x100), ([0, 1, 2, 100], [0, 2, 4], 0x100),
                          ([-1, 0, 1, 2], [0, 3, 4], 0x100), ([0, 1, 2, 3], [0, 2, 5], 0x100),
                          ([0, 1, 2, 3], [0, 3, 2], 0x100)):
        err.zero_()
        mcp.process_logits(xd, out, bias=(i32(off), i32(tok), val), error_word=err)
        assert int(err) == bit, (tok, off)


# --------------------------------------------------------------------------- together
def test_decode_loop_of_a_hybrid_model(mcp):
    """A few steps as a server runs them: tables from lengths, append and attention on them,
    convolution and scan on the same stream, logits processed with the counts of the tokens
    picked so far -- against the definitions, each fed by what ran before it."""
    import math

    import oracle
    from harness import rel_rms
    from mixed_chunked_prefill_gb300.step import LogitsState, MixedStep, RequestTables

    rng = np.random.default_rng(21)
    Hq, Hkv, D, P, V, d, K, N, R = 8, 2, 64, 16, 503, 64, 4, 16, 6
    tables = RequestTables(60, P, R, 12)
    state = LogitsState(R, V)
    shape = (60, P, Hkv, D)
    kc = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = torch.full_like(kc, float("nan"))
    hist = {r: ([], []) for r in range(R)}  # K and V rows of each request, float64
    w, wd = values(rng, (d, K), "bf16", 0.5)
    b, bd = values(rng, (d,), "bf16", 0.1)
    conv_h, conv_d = values(rng, (R, K - 1, d), "bf16")
    v0 = scan_inputs(rng, 1, d, N, 1, "bf16", R, True, 1.0)
    scan_h = v0["state"][0]
    serr = np.zeros_like(scan_h)
    prompts = {4: 37, 1: 20}
    seen, counts = np.zeros((R, 2, V), bool), np.zeros((R, V), np.int64)
    texts = {r: rng.integers(0, V, n) for r, n in prompts.items()}
    state.admit(i32(list(prompts)), i32(np.concatenate(list(texts.values()))),
                i32(np.concatenate([[0], np.cumsum(list(prompts.values()))])))
    for r, t in texts.items():
        seen, counts = ref.update_counts(seen, counts, [r], t, [0, len(t)], V, True, True)
    plan = [([4, 1], [30, 20]), ([4, -1, 1], [7, 0, 1]), ([1, 4], [1, 1]), ([4], [1])]
    for ids, q in plan:
        tb = tables.step(ids, q)
        T = int(tb.cu_h[-1])
        step = MixedStep.from_tables(tb, Hq, Hkv, D, 1 / math.sqrt(D))
        (qh, qd), (kh, kd), (vh, vd) = (values(rng, (T, h, D), "bf16") for h in (Hq, Hkv, Hkv))
        out = torch.full((T, Hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        step.run(qd, kd, vd, kc, vc, out)
        step.check()
        x, xd = values(rng, (T, d), "bf16")
        y = mcp.mixed_conv(xd, wd, bd, conv_d, tb.request_ids, tb.cu_seqlens_q, tb.seqlens_k)
        v = scan_inputs(rng, T, d, N, 1, "bf16", R, True, 1.0)
        v["x"] = (f64(y), y)
        v["A"], v["state"] = v0["A"], (scan_h, v0["state"][1])
        cu, sk = tb.cu_h.tolist(), tb.sk_h.tolist()
        so = torch.empty_like(y)
        got, (want, bound, scan_h, e1) = run_scan(mcp, v, ids, cu, sk, "Dzb", True, "bf16", so, None)
        # the state error of earlier steps goes on in the rows that ran, at most undamped
        serr = np.where(e1 > 0, serr + e1, serr)
        carried = np.concatenate([np.full((q_, d), (np.abs(v["C"][0][a:a + q_]).max() * serr[r]).sum(-1).max()
                                          * 2 * np.abs(v["z"][0][a:a + q_]).max() + 0.0)
                                  for r, q_, a in zip(ids, q, cu) if r >= 0] or [np.zeros((0, d))])
        assert (np.abs(f64(so) - want) <= bound + carried).all()
        cw, cb_, conv_h = ref.conv(x, w, b, conv_h, ids, cu, sk, True, "bf16")
        assert (np.abs(f64(y) - cw) <= cb_).all()
        assert np.array_equal(f64(conv_d), conv_h)
        rows = tb.logits_indices[: sum(n > 0 for n in q)]
        picked = torch.empty((len(rows), d), dtype=torch.bfloat16, device="cuda")
        mcp.gather_rows(so, rows, picked)
        assert torch.equal(picked, so[rows.long()])
        live = [r for r, n in zip(ids, q) if n > 0]
        lh, ld = values(rng, (len(live), V), "bf16", 3.0)
        pen = torch.full((len(live),), 0.7, device="cuda")
        res = state.process(ld, i32(live), torch.empty((len(live), V), device="cuda"),
                            presence_penalty=pen, frequency_penalty=pen, repetition_penalty=pen + 1)
        p64 = pen.double().cpu().numpy()
        want, bound = ref.logits(lh, live, seen, counts, None, (pen + 1).double().cpu().numpy(), p64, p64, {},
                                 None, "fp32")
        assert (np.abs(f64(res) - want) <= bound).all()
        tok = res.argmax(-1).int()
        state.add(i32(live), tok)
        seen, counts = ref.update_counts(seen, counts, live, tok.tolist(), None, V, False, False)
        dv = device_state(seen, counts)
        assert torch.equal(state.seen, dv[0]) and torch.equal(state.counts, dv[1])
        # attention against the oracle on the requests' own rows
        for s, r in enumerate(ids):
            if r < 0:
                continue
            a, e = cu[s], cu[s + 1]
            hist[r][0].extend(kh[a:e])
            hist[r][1].extend(vh[a:e])
            ks, vs = np.array(hist[r][0]), np.array(hist[r][1])
            for t in range(a, e):
                m = sk[s] - (e - 1 - t)
                for h in range(Hq):
                    sc = ks[:m, h // (Hq // Hkv)] @ qh[t, h] / math.sqrt(D)
                    pr = np.exp(sc - sc.max())
                    o = (pr / pr.sum()) @ vs[:m, h // (Hq // Hkv)]
                    assert np.abs(f64(out[t, h]) - o).max() <= 2e-2
        tables.commit(tb)
    tables.check()
    state.check()
    tables.release([4, 1])
    tables.check()
    assert int(tables.free_count) == 60 == tables.free_h
    assert sorted(tables.free_pages.tolist()) == list(range(60))


def test_captured_step_follows_its_inputs(mcp):
    """One captured graph of all calls, replayed with other lengths, tokens and padding."""
    rng = np.random.default_rng(31)
    S, P, cap, V, R, d, N, K = 4, 16, 64, 333, 5, 32, 16, 4
    p, dv = ref.Pool(40, P, R, 6), Device(mcp, 40, P, R, 6)
    ids_d, q_d, new_d = i32([0] * S), i32([0] * S), i32([0] * S)
    cu, sk = torch.zeros(S + 1, dtype=torch.int32, device="cuda"), i32([0] * S)
    bt, slots = torch.zeros((S, 6), dtype=torch.int32, device="cuda"), torch.zeros(cap, dtype=torch.int64, device="cuda")
    rows = i32([0] * S)
    v = scan_inputs(rng, cap, d, N, 1, "bf16", R, True, 1.0)
    w, wd = values(rng, (d, K), "bf16")
    ch, cd = values(rng, (R, K - 1, d), "bf16")
    zero = torch.zeros(d, dtype=torch.bfloat16, device="cuda")
    conv_out = torch.zeros((cap, d), dtype=torch.bfloat16, device="cuda")
    scan_out = torch.zeros_like(conv_out)
    seen, counts = np.zeros((R, 2, V), bool), np.zeros((R, V), np.int64)
    sd, cnt = device_state(seen, counts)
    tok_d = i32([0] * S)
    lh, ld = values(rng, (S, V), "fp32")
    lo = torch.zeros((S, V), device="cuda")
    pen = torch.full((S,), 0.5, device="cuda")
    dev = {k: t[1] for k, t in v.items()}

    def calls():
        mcp.build_step_tables(dv.pool, ids_d, q_d, cu, sk, bt, slots, None, rows, dv.err)
        mcp.mixed_conv(dev["x"], wd, zero, cd, ids_d, cu, sk, out=conv_out, error_word=dv.err)
        mcp.mixed_scan(dev["x"], dev["dt"], dev["A"], dev["B"], dev["C"], dev["state"], ids_d, cu, sk,
                       D=dev["D"], z=dev["z"], dt_bias=dev["bias"], out=scan_out, error_word=dv.err)
        mcp.update_token_counts(ids_d, tok_d, sd, cnt, V, error_word=dv.err)
        mcp.process_logits(ld, lo, ids_d, sd, cnt, frequency_penalty=pen, error_word=dv.err)
        mcp.commit_step(dv.pool, ids_d, q_d, new_d, dv.err)

    ids_d.fill_(-1)  # an empty step before the capture: module loading
    calls()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            calls()
    torch.cuda.synchronize()
    state = v["state"][0]
    serr = 0.0
    for _ in range(5):
        ids = rng.permutation(R)[:S]
        ids[rng.integers(0, S)] = -1
        ids = ids.tolist()
        q = [0 if r < 0 else int(min(96 - p.lens[r], rng.integers(0, 17))) for r in ids]
        tok = rng.integers(0, V, S)
        want = p.build(ids, q, cap)
        new = [0 if r < 0 or rng.random() < 0.2 else int(s) for r, s in zip(ids, want[1])]
        for t, a in ((ids_d, ids), (q_d, q), (new_d, new), (tok_d, tok)):
            t.copy_(i32(a))
        conv_out.fill_(7)
        scan_out.fill_(7)
        lo.fill_(3)
        g.replay()
        torch.cuda.synchronize()
        p.commit(ids, q, new, want[6])
        dv.equal(p)
        for got, a in zip((cu, sk, bt, slots), want):
            assert np.array_equal(got.cpu().numpy(), a)
        n = int(want[0][-1])
        cw, cb, ch = ref.conv(v["x"][0], w, np.zeros(d), ch, ids, want[0], want[1], True, "bf16")
        assert (np.abs(f64(conv_out)[:n] - cw[:n]) <= cb[:n]).all() and (f64(conv_out)[n:] == 7).all()
        assert np.array_equal(f64(cd), ch)
        yw, yb, state, e = ref.scan(v["x"][0], v["dt"][0], v["A"][0], v["B"][0], v["C"][0], v["D"][0],
                                    v["z"][0], v["bias"][0], True, state, ids, want[0], want[1], "bf16")
        # earlier replays' state error, undamped, through C and the gate
        carried = serr * N * np.abs(v["C"][0]).max() * 2 * np.abs(v["z"][0]).max()
        assert (np.abs(f64(scan_out)[:n] - yw[:n]) <= yb[:n] + carried).all()
        assert (f64(scan_out)[n:] == 7).all()
        assert (np.abs(f64(dev["state"]) - state) <= e + serr).all()
        serr += e.max()
        seen, counts = ref.update_counts(seen, counts, ids, tok, None, V, False, False)
        lw, lb = ref.logits(lh, ids, seen, counts, None, np.ones(S), np.full(S, 0.5), np.zeros(S), {}, None, "fp32")
        for i, r in enumerate(ids):
            assert (f64(lo)[i] == 3).all() if r < 0 else (np.abs(f64(lo)[i] - lw[i]) <= lb[i]).all()


def test_captured_calls_of_several_launches(mcp):
    """Calls that launch kernels beside each other, captured: a scan in pieces (two graphs
    share its workspace) and texts counted on cleared rows, replayed in turn, give what the
    same calls give one by one."""
    rng = np.random.default_rng(33)
    d, N, V, R = 96, 16, 3000, 4
    sets = []
    for k in range(2):
        ids, cu, sk, rows, T = stream(rng, [700, 2, 333, 90, 1], [0, 3, 8, 0, 7], 1, 0)
        v = scan_inputs(rng, T, d, N, 1, "bf16", rows, True, 1.0)
        lens = rng.integers(1500, 4000, 6)
        text = i32(rng.integers(0, V, lens.sum()))
        sets.append(dict(v={n: t[1] for n, t in v.items()}, meta=[i32(a) for a in (ids, cu, sk)], T=T, text=text,
                         rows=i32(rng.integers(0, R, 6)), cu=i32(np.concatenate([[0], np.cumsum(lens)])),
                         state0=v["state"][1].clone(), out=torch.zeros((T, d), dtype=torch.bfloat16, device="cuda"),
                         tok=device_state(np.zeros((R, 2, V), bool), np.zeros((R, V), np.int64))))
    desc = _capi.ScanDesc(6, sets[0]["T"], 7, d, N, 1, 0, 1, d, d, d, N, N, d)
    n = ctypes.c_size_t()
    assert mcp.load().mcp_mixed_scan_workspace(ctypes.byref(desc), ctypes.byref(n)) == 0 and n.value > 256
    shared = torch.empty(n.value, dtype=torch.uint8, device="cuda")

    def calls(s):
        v = s["v"]
        v["state"].copy_(s["state0"])
        mcp.mixed_scan(v["x"], v["dt"], v["A"], v["B"], v["C"], v["state"], *s["meta"], D=v["D"], z=v["z"],
                       dt_bias=v["bias"], out=s["out"], workspace=shared)
        for prompt in (True, False):
            mcp.update_token_counts(s["rows"], s["text"], *s["tok"], V, s["cu"], prompt, prompt)

    want = []
    for s in sets:
        calls(s)
        want.append([t.clone() for t in (s["out"], s["v"]["state"], *s["tok"])])
    torch.cuda.synchronize()
    graphs = []
    for s in sets:
        side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
            calls(s)
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(5):
        shared.fill_(255)
        for s, g in zip(sets, graphs):
            s["out"].zero_()
            g.replay()
        for s, w in zip(sets, want):
            assert all(torch.equal(a, b) for a, b in zip((s["out"], s["v"]["state"], *s["tok"]), w))


def test_calls_on_another_stream(mcp):
    """The calls run on the stream they are given, behind what that stream already holds."""
    rng = np.random.default_rng(41)
    s = torch.cuda.Stream()
    x, xd = values(rng, (64, 4096), "fp32")
    seen, counts = token_state(rng, 64, 4096, 40)
    sd, cd = device_state(seen, counts)
    ids, pen = i32(range(64)), torch.full((64,), 0.5, device="cuda")
    late, out = torch.zeros_like(xd), torch.empty_like(xd)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(20):
            torch.mm(xd.view(512, 512), xd.view(512, 512))
        late.copy_(xd)
    mcp.process_logits(late, out, ids, sd, cd, presence_penalty=pen, stream=s)
    d = Device(mcp, 8, 16, 2, 4)
    torch.cuda.synchronize()
    want, bound = ref.logits(x, list(range(64)), seen, counts, None, np.ones(64), np.zeros(64),
                             np.full(64, 0.5), {}, None, "fp32")
    assert (np.abs(f64(out) - want) <= bound).all()
    p = ref.Pool(8, 16, 2, 4)
    s.synchronize()
    for got, w in zip(d.build([1], [20], 20, s.cuda_stream), p.build([1], [20], 20)):
        s.synchronize()
    assert int(d.err) == 0


def test_results_taken_for_another_stream(mcp):
    """A result (and a workspace) that the call takes for itself is memory of the stream it
    runs on, not memory that the current stream has freed but still writes."""
    rng = np.random.default_rng(42)
    d, N = 64, 16
    ids, cu, sk, R, T = stream(rng, [300, 1, 190], [0, 3, 7], 1, 0)
    v = scan_inputs(rng, T, d, N, 1, "bf16", R, True, 1.0)
    w = values(rng, (d, 4), "bf16", 0.5)[1]
    meta = [i32(a) for a in (ids, cu, sk)]
    state = torch.zeros((R, 3, d), dtype=torch.bfloat16, device="cuda")
    x, dt, B, C = (v[k][1] for k in ("x", "dt", "B", "C"))

    def calls(st, **kw):
        y = mcp.mixed_conv(x, w, None, state.clone() if st is None else st[0], *meta, **kw)
        s = mcp.mixed_scan(x, dt, v["A"][1], B, C, v["state"][1].clone() if st is None else st[1], *meta, **kw)
        return y, s

    want = calls(None)
    torch.cuda.synchronize()
    other, busy = torch.cuda.Stream(), torch.randn((4096, 4096), device="cuda")
    n = ctypes.c_size_t()
    desc = _capi.ScanDesc(len(ids), T, R, d, N, 1, 0, 1, d, d, d, N, N, d)
    assert mcp.load().mcp_mixed_scan_workspace(ctypes.byref(desc), ctypes.byref(n)) == 0
    for s in (other, other.cuda_stream):
        kept = state.clone(), v["state"][1].clone()
        blocks = [torch.empty_like(want[0]), torch.empty_like(want[1]),
                  torch.empty(n.value, dtype=torch.uint8, device="cuda")]
        torch.cuda.synchronize()
        for _ in range(20):
            torch.mm(busy, busy)
        for b in blocks:
            b.view(torch.uint8).fill_(255)
        del b, blocks
        got = calls(kept, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_stale_steps_are_refused(mcp):
    """A step may be committed once, and not behind another commit."""
    from mixed_chunked_prefill_gb300.step import RequestTables

    tables, others = RequestTables(20, 16, 4, 6), RequestTables(20, 16, 4, 6)
    a, b = tables.step([0], [20]), tables.step([1], [40])
    with pytest.raises(ValueError):
        others.commit(a)
    tables.commit(b)
    for step in (a, b):
        with pytest.raises(ValueError):
            tables.commit(step)
    tables.commit(tables.step([0, 1], [20, 1]))
    tables.check()
    assert int(tables.free_count) == tables.free_h == 20 - 2 - 3
    tables.release([1, 0])
    assert sorted(tables.free_pages.tolist()) == list(range(20))


def test_python_refusals(mcp):
    x = torch.zeros((4, 16), dtype=torch.bfloat16, device="cuda")
    ids, cu, sk = i32([0]), i32([0, 4]), i32([4])
    w, st = torch.zeros((16, 4), dtype=torch.bfloat16, device="cuda"), torch.zeros((1, 3, 16), dtype=torch.bfloat16, device="cuda")
    mcp.mixed_conv(x, w, None, st, ids, cu, sk)
    for kw, e in ((dict(x=x.T), ValueError), (dict(weight=w.float()), TypeError),
                  (dict(weight=w[:, :3]), ValueError), (dict(state=st[:, :2]), ValueError),
                  (dict(cu_seqlens_q=ids), ValueError), (dict(seqlens_k=sk.long()), TypeError),
                  (dict(activation="gelu"), ValueError), (dict(out=x[:2]), ValueError),
                  (dict(x=x.float(), weight=w.float(), state=st.float()), mcp.MCPError),
                  (dict(x=x[:, 4:12], weight=w[:8].contiguous(), state=st[..., :8].contiguous()), mcp.MCPError)):
        a = dict(x=x, weight=w, bias=None, state=st, request_ids=ids, cu_seqlens_q=cu, seqlens_k=sk)
        a.update(kw)
        with pytest.raises(e):
            mcp.mixed_conv(**a)
    d = Device(mcp, 8, 16, 2, 4)
    d.pool.device = 1  # as if it had been made there
    for call in (lambda: d.build([1], [20], 20, None), lambda: mcp.commit_step(d.pool, ids, ids)):
        with pytest.raises(ValueError, match="cuda:1"):
            call()
    f = torch.zeros((2, 64), device="cuda")
    with pytest.raises(ValueError):
        mcp.process_logits(f.T)
    with pytest.raises(mcp.MCPError):
        mcp.process_logits(f[:1].expand(2, 64))
    with pytest.raises(ValueError):
        mcp.process_logits(f, request_ids=i32([0, 1]))
    with pytest.raises(mcp.MCPError):
        mcp.process_logits(f, temperature=None, presence_penalty=f[0, :2])
    with pytest.raises(ValueError):
        mcp.process_logits(f, mask=i32([[0]]), mask_rows=i32([0, 0]))
    with pytest.raises(TypeError):
        mcp.process_logits(f.int())
