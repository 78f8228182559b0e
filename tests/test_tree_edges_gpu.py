"""Trees of drafted tokens on the GPU: calls that only some contents, lengths or orders of work bring
about."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import draft_ref as ref  # noqa: F401
from test_tree_gpu import SEGMENTS, Drafts, Step, bits_of, cumulated, err_word, i32, mcp  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------ attention
@pytest.mark.parametrize("segments,hq,hkv,D,split", [
    ([(6, 700, "tree")], 8, 2, 128, 128),                  # parts of a row at once
    ([(6, 1500, "tree"), (1, 90, None)], 8, 2, 128, 128),  # in batches
    ([(30, 1200, "tree")] * 4, 64, 2, 128, 640),           # more rows than the GPU merges at once
    ([(5, 5200, "tree")], 4, 2, 128, 128),                 # more parts than lanes
    ([(6, 900, "tree")], 4, 2, 64, 128), ([(6, 900, "forest")], 4, 2, 96, 128),
    ([(6, 900, "chain")], 4, 2, 256, 128)])
def test_replays_merge_the_parts_of_their_own_contents(mcp, segments, hq, hkv, D, split):  # noqa: F811
    """A graph replayed without a pause: the merge, launched beside the forward, never takes parts
    or LSEs that the replay before it left in the workspace."""
    steps = [Step(segments, hq, hkv, D, 16, seed=s) for s in (41, 42, 43)]
    steps[1].qs *= 4  # other LSEs, too
    want = []
    for st in steps:
        out, lse = st.run(mcp, prefill_split_tokens=split)
        st.check(mcp, out, lse)
        want.append((out, lse))
    st = steps[0]
    plan, ws = st.plan(mcp, prefill_split_tokens=split)
    assert plan.num_combine > 0
    sets = [(s.qs, s.k, s.v, i32(s.bt), s.masks()[0]) for s in steps]
    buf = [x.clone() for x in sets[0]]
    mask_rows, cu, sk = st.masks()[1], i32(st.cu), i32(st.lens)
    out, lse = torch.empty_like(st.qs), torch.empty((st.T, hq), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mcp.mixed_attn_fwd_tree(plan, buf[0], buf[1], buf[2], buf[3], cu, sk, buf[4], mask_rows, out, lse, ws)
    got = []
    for turn in range(9):
        for b, x in zip(buf, sets[turn % 3]):
            b.copy_(x)
        graph.replay()
        got.append((out.clone(), lse.clone()))
    torch.cuda.synchronize()
    for turn, pair in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(pair, want[turn % 3])), turn


@pytest.mark.parametrize("D,P,split", [(64, 8, 0), (96, 16, 0), (128, 16, 0), (256, 32, 0), (128, 1, 0),
                                       (128, 16, 128), (256, 16, 128)])
def test_rows_that_see_different_numbers_of_infinities(mcp, D, P, split):  # noqa: F811
    """Infinities and NaN all over a tree's V: each row takes those of the tokens that it sees, one
    row a handful and its neighbour a hundred, and what it does not see stays out."""
    st = Step([(120, 130, "tree"), (33, 300, "chain"), (40, 0, "forest")], 6, 2, D, P, seed=D + P + split)
    odd = [float("inf"), -float("inf"), float("nan")]
    for s in range(3):
        for i in np.flatnonzero(st.rng.random(st.q[s]) < 0.4):
            page, off = st.slots(s, np.array([st.hist[s] + i]))
            for c in st.rng.integers(0, D, 3):
                st.v[page, off, int(st.rng.integers(0, 2)), int(c)] = odd[int(st.rng.integers(0, 3))]
    out, lse = st.run(mcp, **(dict(prefill_split_tokens=split) if split else {}))
    mcp.check_device_errors(st.error)
    out = out.double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        for s in range(3):
            page, off = st.slots(s, np.arange(st.lens[s]))
            k, v = (c[page, off].double().cpu().numpy() for c in (st.k, st.v))
            a, b = st.cu[s], st.cu[s + 1]
            want, wl, mass = ref.tree_attention(st.qs[a:b].double().cpu().numpy(), k, v, st.hist[s], st.bits[s],
                                                st.scale)
            good = np.isfinite(want)
            assert good.any() and not good.all()
            # infinities keep their sign, both signs and NaN give NaN
            assert np.array_equal(np.where(good, 0, out[a:b]), np.where(good, 0, want), equal_nan=True), s
            bound = 2.0 ** -8 * (np.abs(want) + mass) * 1.01 + 1e-3 * mass + 1e-6  # as in Step.compare
            assert (np.abs(out[a:b] - want)[good] <= bound[good]).all(), s
            assert (np.abs(lse[a:b].double().cpu().numpy() - wl) <= 1e-3).all(), s


# ------------------------------------------------------------------ segments that are none
LOW, HIGH = -(1 << 31), (1 << 31) - 1
# bounds whose difference leaves 32 bits, and others that are far outside
WILD = [(2, LOW), (HIGH, LOW), (HIGH - 1, LOW + 5), (0, LOW), (LOW, HIGH), (LOW, 0), (HIGH, 3), (-1, 3)]


@pytest.mark.parametrize("a,b", WILD)
@pytest.mark.parametrize("row", [0, -1])
def test_masks_of_bounds_far_outside(mcp, a, b, row):  # noqa: F811
    """The segment is reported and left out, whatever its bounds; the one beside it is not touched."""
    err = err_word()
    mask = torch.full((8, 1), 7, dtype=torch.int32, device="cuda")
    pos = i32([-5] * 4)
    mcp.build_tree_masks(i32([-1, 0, 0, 1]), i32([a, b]), i32([100]), i32([row]), mask, pos, err)
    assert bits_of(err) & mcp.DEVERR_SEGMENT
    assert (mask == 7).all() and (pos == -5).all()


@pytest.mark.parametrize("a,b", WILD)
@pytest.mark.parametrize("draft", [True, False])
def test_verification_of_bounds_far_outside(mcp, a, b, draft):  # noqa: F811
    d = Drafts([4], 5000, "fp32", "tree", draft, seed=3)
    err, path, new = err_word(), i32([9] * 4), i32([9] * 4)
    accepted, _, _ = d.run(mcp, err, cu_rows=i32([a, b]), path=path, new_tokens=new)
    assert bits_of(err) == mcp.DEVERR_SEGMENT and accepted.tolist() == [0]
    assert (path == 9).all() and (new == 9).all()


@pytest.mark.parametrize("a,b", WILD)
@pytest.mark.parametrize("rows", [None, [0, 1], [0, 4]])
def test_kept_paths_of_bounds_far_outside(mcp, a, b, rows):  # noqa: F811
    """Lengths that are none: of a segment's tokens, of its rows, or of both."""
    st = Step([(4, 30, "tree")], 2, 2, 64, 16, seed=6)
    k, v = st.k.clone(), st.v.clone()
    for cu, cu_rows in ([(a, b), rows], [rows or (0, 4), (a, b)]):
        # (-1, 3) is four tokens whose place in the stream is not looked at: a path of four rows, or
        # no drafts beside one row
        sound = (cu == (-1, 3) and cu_rows is not None)
        err = err_word()
        new = mcp.kv_keep_path(st.k, st.v, i32(st.bt), i32(cu), i32([34]), i32([1]), i32([0, 1, 2, 3]),
                               cu_rows=None if cu_rows is None else i32(cu_rows), error_word=err)
        assert bits_of(err) == (0 if sound else mcp.DEVERR_SEGMENT), (cu, cu_rows)
        assert new.tolist() == [31 if sound and cu_rows == [0, 4] else 34], (cu, cu_rows)
    assert torch.equal(st.k.view(torch.int16), k.view(torch.int16))
    assert torch.equal(st.v.view(torch.int16), v.view(torch.int16))


def test_kept_paths_of_no_layers(mcp):  # noqa: F811
    """The lengths alone, whatever distance is given for layers that are not there."""
    import ctypes

    from mixed_chunked_prefill_gb300 import _capi

    st = Step([(5, 30, "chain"), (1, 3, None)], 2, 2, 64, 16)
    bt, cu, sk, acc, path = i32(st.bt), i32(st.cu), i32(st.lens), i32([2, 1]), i32([0, 2, -1, -1, -1, 0])
    for stride in (0, 64):
        new, err = i32([-7, -7]), err_word()
        d = _capi.KeepDesc(2, 6, 0, 2, 64, 16, st.bt.shape[1], st.pages, stride)
        assert mcp.load().mcp_kv_keep_path(
            ctypes.byref(d), None, None, bt.data_ptr(), cu.data_ptr(), sk.data_ptr(), None, acc.data_ptr(),
            path.data_ptr(), new.data_ptr(), err.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
        assert new.tolist() == [32, 4] and bits_of(err) == 0


def test_kept_paths_of_a_cache_given_twice_are_refused(mcp):  # noqa: F811
    """Its rows would be moved twice: 2 -> 1 and 4 -> 2, and then 2, which holds 4 now, -> 1."""
    st = Step([(5, 30, "chain")], 2, 2, 64, 16)
    args = (i32(st.bt), i32(st.cu), i32(st.lens), i32([3]), i32([0, 2, 4, -1, -1]))
    before = st.k.clone()
    layers = torch.stack([st.k, st.v])
    # an expanded tensor is its one layer listed twice
    for k, v in (([st.k, st.k], [st.v, layers[1]]), (st.k, st.k), (layers, layers),
                 (st.k.expand(2, *st.k.shape), st.v.expand(2, *st.k.shape))):
        with pytest.raises(mcp.MCPError, match="caches overlap"):
            mcp.kv_keep_path(k, v, *args)
    assert torch.equal(st.k.view(torch.int16), before.view(torch.int16))
    mcp.kv_keep_path([st.k, layers[0]], [st.v, layers[1]], *args)
    moved = st.slots(0, np.array([31, 32])), st.slots(0, np.array([32, 34]))
    assert torch.equal(st.k[moved[0]].view(torch.int16), before[moved[1]].view(torch.int16))


# ------------------------------------------------------------------------ steps' options
@pytest.mark.parametrize("some_rows", [False, True])
def test_a_step_with_trees_keeps_its_callers_options(mcp, some_rows):  # noqa: F811
    """MixedStep sets the trees in a copy of the options that it is given: the splits asked for are the
    plan's, and their parts are merged to the same results."""
    from mixed_chunked_prefill_gb300.step import MixedStep

    st = Step(SEGMENTS, 8, 2, 128, 16, seed=33)
    rows = np.flatnonzero(st.rng.random(st.T) < 0.4) if some_rows else None
    options, items = mcp.PlanOptions(prefill_split_tokens=128), []
    for given in (options, None):
        step = MixedStep(st.hq, st.hkv, st.D, st.P, st.pages, st.scale, st.cu, st.lens, st.bt, options=given,
                         rows=rows, trees=st.tree, parents=st.parents)
        assert step.plan.tree == 1
        items.append((step.plan.num_items, step.plan.num_combine))
        out = torch.full_like(st.qs, float("nan"))
        lse = torch.full((st.T, st.hq), float("nan"), device="cuda")
        step.attention(st.qs, st.k, st.v, out, lse)
        step.check()
        st.compare(out, lse, rows)
    assert items[0][1] > 0 and items[0] != items[1]
    assert options.tree == 0 and options.prefill_split_tokens == 128


# ----------------------------------------------------------------------- verification
def refused_twice(V, seed, delta, others):
    """Rows p and q of a root with two nodes of token 0, which p does not have, so that both are
    refused and c = 1 + N, N = sum max(p - q, 0).  q of the other tokens are multiples of 2^-24 that
    add up to 1 and p = q (1 + delta) rounded to fp32, which makes N = delta up to the roundings: p - c q
    is what p was rounded by, but for `others` tokens of larger p."""
    rng = np.random.default_rng(seed)
    k = np.floor(rng.dirichlet(np.ones(V - 1)) * (2 ** 24 - V)).astype(np.int64) + 1
    k[0] += 2 ** 24 - k.sum()
    q = np.concatenate([[0.5], k / 2.0 ** 24]).astype(np.float32)
    p = (q.astype(np.float64) * (1 + delta)).astype(np.float32)
    p[0] = 0
    d = Drafts([3], V, "fp32", "star", True, seed=seed)
    for at in others:  # more of one token, and as much less of another: N as before
        p[at] += np.float32(2.0 ** -20)
        p[at + 1] -= np.float32(2.0 ** -20)
    d.target[:], d.draft[:] = torch.tensor(p), torch.tensor(q)
    d.tokens[:] = 0
    d.u[:] = 0.5
    return d, p.astype(np.float64), q.astype(np.float64)


@pytest.mark.parametrize("V", [300, 5000, 40000])
@pytest.mark.parametrize("others", [[], [20, 80, 200]])
def test_what_remains_is_what_the_rows_were_rounded_by(mcp, V, others):  # noqa: F811
    """After two refusals p - c q lies below the rounding of c q nearly everywhere.  What remains is
    those differences, not nothing (the token would be drawn from p then), and the token is drawn
    from them."""
    for seed in range(6):
        d, p, q = refused_twice(V, seed, 0.37 + 0.01 * seed, others)
        c = 1 + np.maximum(p - q, 0).sum()
        w = np.maximum(p - c * q, 0)
        assert 0 < w.sum() < 2.0 ** -15 and (others or (np.abs(p - c * q)[1:] <= 2.0 ** -22 * p[1:]).all())
        # c is a sum of V differences as a pair of fp32, off by 2^-44 (2^-49 of the sum for each value
        # of a lane, 160 at most); so is each c q, by 2^-47 of it: prefix sums of w are off by less
        # than 2^-43 of sum p + c sum q < 4
        off = 2.0 ** -41
        s = np.concatenate([[0], np.cumsum(w)])
        for last in (0.01, 0.3, 0.5, 0.77, 0.99):
            d.u_last[:] = last
            accepted, path, new = d.run(mcp, err_word())
            v, aim = int(new[0]), float(d.u_last[0]) * s[-1]
            assert accepted.tolist() == [1] and path.tolist() == [0, -1, -1]
            assert s[v] <= aim + off and aim - off <= s[v + 1], (seed, last, v)
            assert w[v] > 0 or abs(p[v] - c * q[v]) < off


@pytest.mark.parametrize("copies", [1, 64])
@pytest.mark.parametrize("children", [0, 1, 2, 4, 6])
def test_borders_of_what_remains_when_the_draft_is_close(mcp, copies, children):  # noqa: F811
    """Rows of 128000 values whose draft is off by half a percent, every child refused: what remains is
    a thousandth of p.  Random numbers right above and below borders between two tokens find the
    token that 64-bit sums give."""
    V, rng = 128000, np.random.default_rng(children)
    z = rng.standard_normal(V) * 2.5
    p, q = (np.exp(x) / np.exp(x).sum() for x in (z, z + rng.standard_normal(V) * 0.005))
    p[0] = 0  # the children's token
    p, q = p.astype(np.float32), q.astype(np.float32)
    c, P, Q = 0.0, p.astype(np.float64), q.astype(np.float64)
    mass = 1.0
    for _ in range(children):
        c += mass
        mass = np.maximum(P - c * Q, 0).sum()
    w = np.maximum(P - c * Q, 0)
    s = np.concatenate([[0], np.cumsum(w)])
    assert children == 0 or 2.0 ** -13 < s[-1] < 2.0 ** -7
    # A lane adds up n values, n = 500 where a CTA has the row, and sums of w are off by at most
    # n^2 2^-48 of themselves (its low word is at most n 2^-24 of the high one, and rounded n times by
    # 2^-24 of that); a weight by 2^-47 of p + c q.  All of p: sums off by 2^-30; a part of 2^-7 with
    # the weights' part: 2^-37 + 2^-45, and c is a sum of up to six such.  Rounds of 16 and of 8 CTAs
    # have n = 32 and 63 and so 2^-36 of all, 2^-43 + 2^-45 of a part: with c, 2^-36 and 2^-39.
    off = 2.0 ** -36 if children == 0 else 2.0 ** -39
    rows = children + 1
    d = Drafts([rows] * copies, 4, "fp32", "star", True)
    d.V = V
    d.target, d.draft = (torch.tensor(x).cuda().expand(rows * copies, V).contiguous() for x in (p, q))
    d.tokens[:], d.u[:] = 0, 0.5
    told = 0
    for _ in range(-(-256 // copies)):
        at = rng.choice(np.flatnonzero(w > 0), copies, p=w[w > 0] / s[-1])  # a border is the one before it
        u = (s[at] / s[-1]).astype(np.float32)
        up = rng.random(copies) < 0.5
        d.u_last = np.where(up, np.nextafter(u, np.float32(1)), np.nextafter(u, np.float32(0))).astype(np.float32)
        accepted, path, new = d.run(mcp, err_word())
        assert (accepted == 1).all()
        aim = d.u_last.astype(np.float64) * s[-1]
        v = new.cpu().numpy()[::rows]
        assert (w[v] > 0).all() and (s[v] <= aim + off).all() and (aim - off <= s[v + 1]).all()
        told += ((s[v] <= aim - off) & (aim + off <= s[v + 1])).sum()
    assert told > 100  # most numbers lie further from the borders than the sums may be off


@pytest.mark.parametrize("V", [3000, 30000])
def test_nothing_remains_within_a_rounding(mcp, V):  # noqa: F811
    """After two refusals p is below c q everywhere, by less than one and a half units of its last
    place, and above c q's rounded value in some places: nothing remains, and the token is p's."""
    some = 0
    for seed in range(4):
        rng = np.random.default_rng(seed)
        first = float(np.float32(1.25 + 0.1 * seed))
        c = first + 0.45 * 2.0 ** -23  # the second fp32 of c as large as it gets

        def below(x):  # the largest fp32 that is not above x
            y = x.astype(np.float32)
            return np.where(y > x, np.nextafter(y, np.float32(0)), y).astype(np.float32)

        # q of the tokens but 0 add up to 1 + h, so that N = sum (p - q) = c h + c - 1 - h - (what p was
        # rounded by, r), and 1 + N = c + (c - 1) h - r, above c by a tenth of r where h = 1.1 r / (c - 1)
        k = np.floor(rng.dirichlet(np.ones(V - 1) * 4) * (2 ** 24 - V)).astype(np.int64) + 1
        k[0] += 2 ** 24 - k.sum()
        q = k / 2.0 ** 24
        r = (c * q - below(c * q)).sum()
        q *= 1 + 1.1 * r / (c - 1)
        q = np.concatenate([[0.5], q]).astype(np.float32)
        p = below(c * q.astype(np.float64))
        p[0] = 0
        P, Q = p.astype(np.float64), q.astype(np.float64)
        now = 1 + np.maximum(P - Q, 0).sum()
        if ((P - now * Q) / Q).max() > -2.0 ** -32:
            continue  # q's own rounding moved its sum too far
        some += int((p > np.float32(now) * q).sum())
        d = Drafts([3], V, "fp32", "star", True, seed=seed)
        d.target[:], d.draft[:] = torch.tensor(p), torch.tensor(q)
        d.tokens[:], d.u[:] = 0, 0.5
        s = np.concatenate([[0], np.cumsum(P)])
        for last in (0.03, 0.4, 0.8, 0.999):
            d.u_last[:] = last
            err = err_word()
            accepted, _, new = d.run(mcp, err)
            v, aim = int(new[0]), float(d.u_last[0]) * s[-1]
            assert bits_of(err) == 0 and accepted.tolist() == [1]
            assert p[v] > 0 and s[v] <= aim + 2.0 ** -36 and aim - 2.0 ** -36 <= s[v + 1], (seed, last, v)
    assert some > 100
