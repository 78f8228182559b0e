"""Trees of drafted tokens without a GPU: refusals of the C entries (nothing is launched), the
plans of steps with trees, and the definitions against each other."""

from __future__ import annotations

import ctypes

import numpy as np
import pytest

import mixed_chunked_prefill_gb300 as mcp
from mixed_chunked_prefill_gb300 import _capi
from oracle import draft_ref as ref
from plan_tools import ITEM, plan_host

INVALID, UNSUPPORTED, OK = _capi.MCP_ERR_INVALID_ARG, _capi.MCP_ERR_UNSUPPORTED, _capi.MCP_OK
P16 = 1 << 20  # an aligned address that no refused call looks at


@pytest.fixture(scope="module")
def lib():
    from mixed_chunked_prefill_gb300 import build

    build.build()
    return mcp.load()


@pytest.mark.parametrize("over,status", [
    (dict(S=-1), INVALID), (dict(T=-1), INVALID), (dict(rows=-1), INVALID), (dict(words=0), INVALID),
    (dict(words=33), UNSUPPORTED), (dict(S=(1 << 20) + 1), UNSUPPORTED),
    (dict(T=(1 << 30) + 1), UNSUPPORTED), (dict(rows=(1 << 30) + 1), UNSUPPORTED),
    *[(dict([(n, None)]), INVALID) for n in ("parents", "cu", "sk", "mask_rows", "mask")],
    *[(dict([(n, P16 + 2)]), INVALID) for n in
      ("parents", "cu", "sk", "mask_rows", "mask", "positions", "err")],
    (dict(S=0, cu=None), OK), (dict(T=0, parents=None), OK),
])
def test_build_tree_masks_refusals(lib, over, status):
    a = dict(parents=P16, cu=P16, sk=P16, mask_rows=P16, S=2, T=10, rows=10, words=1, mask=P16,
             positions=P16, err=None)
    a.update(over)
    assert lib.mcp_build_tree_masks(a["parents"], a["cu"], a["sk"], a["mask_rows"], a["S"], a["T"],
                                    a["rows"], a["words"], a["mask"], a["positions"], a["err"],
                                    None) == status


def verify(lib, tensors=(), **over):
    f = dict(num_seqs=2, total_rows=8, vocab_size=100, dtype=2, target_stride=100, draft_stride=100)
    f.update(over)
    d = _capi.VerifyDesc(*(f[n] for n, _ in _capi.VerifyDesc._fields_))
    a = {n: P16 for n, _ in _capi.VerifyTensors._fields_}
    a.update(tensors)
    t = _capi.VerifyTensors(*(a[n] for n, _ in _capi.VerifyTensors._fields_))
    return lib.mcp_verify_drafts(ctypes.byref(d), ctypes.byref(t), None, None)


@pytest.mark.parametrize("over,status", [
    (dict(num_seqs=-1), INVALID), (dict(total_rows=-1), INVALID), (dict(vocab_size=0), INVALID),
    (dict(dtype=3), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED), (dict(target_stride=99), INVALID),
    (dict(draft_stride=0), INVALID), (dict(num_seqs=(1 << 20) + 1), UNSUPPORTED),
    (dict(total_rows=(1 << 30) + 1), UNSUPPORTED),
    (dict(vocab_size=(1 << 28) + 1, target_stride=1 << 29, draft_stride=1 << 29), UNSUPPORTED),
    *[(dict(tensors={n: None}), INVALID) for n in
      ("target", "tokens", "cu_rows", "uniform", "final_uniform", "accepted", "path", "new_tokens")],
    *[(dict(tensors={n: P16 + 2}), INVALID) for n, _ in _capi.VerifyTensors._fields_],
    (dict(tensors=dict(target=P16 + 1), dtype=0), INVALID),
    (dict(num_seqs=0, tensors=dict(cu_rows=None)), OK),
])
def test_verify_drafts_refusals(lib, over, status):
    assert verify(lib, **over) == status


def test_verify_drafts_without_structures(lib):
    assert lib.mcp_verify_drafts(None, None, None, None) == INVALID
    assert lib.mcp_kv_keep_path(None, None, None, None, None, None, None, None, None, None, None,
                                None) == INVALID


def keep(lib, ks=(P16, P16), vs=(P16, P16), **over):
    a = dict(bt=P16, cu=P16, sk=P16, cu_rows=None, accepted=P16, path=P16, new_lens=None, err=None)
    f = dict(num_seqs=2, total_rows=8, num_layers=2, num_kv_heads=2, head_dim=64, page_size=16,
             max_pages_per_seq=4, num_pages=8, layer_stride=0)
    for name, value in over.items():
        (a if name in a else f)[name] = value
    d = _capi.KeepDesc(*(f[n] for n, _ in _capi.KeepDesc._fields_))
    arrays = [None if x is None else (ctypes.c_void_p * len(x))(*x) for x in (ks, vs)]
    return lib.mcp_kv_keep_path(ctypes.byref(d), *arrays, a["bt"], a["cu"], a["sk"], a["cu_rows"],
                                a["accepted"], a["path"], a["new_lens"], a["err"], None)


@pytest.mark.parametrize("over,status", [
    (dict(num_seqs=-1), INVALID), (dict(total_rows=-1), INVALID), (dict(num_layers=-1), INVALID),
    (dict(num_kv_heads=0), INVALID), (dict(head_dim=0), INVALID), (dict(max_pages_per_seq=0), INVALID),
    (dict(num_pages=0), INVALID), (dict(page_size=4), UNSUPPORTED), (dict(page_size=0), UNSUPPORTED),
    (dict(num_kv_heads=1, head_dim=12), INVALID), (dict(num_layers=1025), UNSUPPORTED),
    (dict(num_seqs=(1 << 20) + 1), UNSUPPORTED), (dict(total_rows=(1 << 30) + 1), UNSUPPORTED),
    (dict(max_pages_per_seq=(1 << 28) + 1), UNSUPPORTED),
    (dict(num_kv_heads=1 << 14, head_dim=128), UNSUPPORTED),
    *[(dict([(n, None)]), INVALID) for n in ("bt", "cu", "sk", "accepted", "path", "ks", "vs")],
    *[(dict([(n, P16 + 2)]), INVALID) for n in
      ("bt", "cu", "sk", "cu_rows", "accepted", "path", "new_lens", "err")],
    (dict(layer_stride=-8), INVALID), (dict(layer_stride=12), INVALID),
    (dict(layer_stride=64, ks=(None,)), INVALID), (dict(ks=(P16, None)), INVALID), (dict(vs=(P16 + 8, P16)), INVALID), (dict(num_seqs=0), OK),
])
def test_kv_keep_path_refusals(lib, over, status):
    assert keep(lib, **over) == status


def test_results_may_not_overlap(lib):
    """A result at an input's address, over its last word, or at another result's."""
    def at(i):
        return P16 + (i << 16)

    def refused(status):
        return status == INVALID and b"overlap" in lib.mcp_last_error()

    names = ("parents", "cu", "sk", "mask_rows", "mask", "positions", "err")
    good = {n: at(i) for i, n in enumerate(names)}
    ends = dict(parents=36, cu=8, sk=4, mask_rows=4, err=0, mask=76, positions=36)  # the last word
    for result in ("mask", "positions"):
        for other in names:
            for off in (0, ends[other]):
                a = {**good, result: good[other] + off}
                if other != result:
                    assert refused(lib.mcp_build_tree_masks(
                        a["parents"], a["cu"], a["sk"], a["mask_rows"], 2, 10, 10, 2, a["mask"],
                        a["positions"], a["err"], None)), (result, other, off)

    names = [n for n, _ in _capi.VerifyTensors._fields_]
    good = {n: at(i) for i, n in enumerate(names)}
    ends = dict(target=4 * 1399 - 400, draft=4 * 1399 - 400, cu_rows=8, final_uniform=4, accepted=4)
    for result in ("accepted", "path", "new_tokens"):
        for other in names:
            if other != result:
                for off in (0, ends.get(other, 28)):
                    a = {**good, result: good[other] + off}
                    assert refused(verify(lib, a, target_stride=180, draft_stride=180)), (result, other, off)
    for big in (1 << 40, (1 << 63) - 1):  # rows past all addresses
        assert refused(verify(lib, {**good, "path": good["draft"] + 4}, draft_stride=big))

    names = ("bt", "cu", "sk", "cu_rows", "accepted", "path", "err")
    good = {n: at(i) for i, n in enumerate(names)}
    ends = dict(bt=28, cu=8, sk=4, cu_rows=8, accepted=4, path=28, err=0)
    for other in names:
        for off in (0, ends[other]):
            assert refused(keep(lib, **good, new_lens=good[other] + off)), (other, off)


def test_tree_forward_refusals(lib):
    d = mcp.make_desc(2, 9, 8, 2, 64, 16, 4, 8, 0.125)
    cu, sk = [0, 1, 9], [20, 30]

    def fwd(plan, mask=P16, rows=8, words=1, mask_rows=P16, q=P16, ws=P16, nbytes=1 << 30):
        return lib.mcp_mixed_attn_fwd_tree(ctypes.byref(plan), q, P16, P16, P16, P16, P16, mask, rows,
                                           words, mask_rows, P16, None, ws, nbytes, None)

    opts = mcp.PlanOptions(num_sms=152)
    plain = plan_host(d, cu, sk, opts=opts)[1]
    assert fwd(plain) == INVALID and b"tree" in lib.mcp_last_error()
    opts.tree = 1
    plan = plan_host(d, cu, sk, opts=opts)[1]
    assert plan.tree == 1
    for bad in (dict(mask=None), dict(mask=P16 + 2), dict(rows=-1), dict(words=0), dict(words=-1),
                dict(mask_rows=None), dict(mask_rows=P16 + 1), dict(q=None), dict(q=P16 + 8),
                dict(ws=None), dict(ws=P16 + 128)):
        assert fwd(plan, **bad) == INVALID, bad
    assert fwd(plan, nbytes=64) == _capi.MCP_ERR_WORKSPACE_TOO_SMALL
    assert fwd(mcp.Plan()) == INVALID
    empty = plan_host(mcp.make_desc(1, 0, 8, 2, 64, 16, 4, 8, 0.125), [0, 0], [5], opts=opts)[1]
    assert fwd(empty, mask_rows=None) == OK


@pytest.mark.parametrize("tree", [2, -1])
def test_plan_refuses_other_tree_values(lib, tree):
    opts = mcp.PlanOptions(num_sms=152, tree=tree)
    assert plan_host(mcp.make_desc(1, 1, 8, 2, 64, 16, 4, 8, 0.125), [0, 1], [5], opts=opts)[0] == INVALID


def plan_rows(lib, d, cu, k, rows, opts):
    """(status, plan, items) of mcp_mixed_attn_plan_rows_host with options."""
    arrays = [np.ascontiguousarray(x, dtype=np.int32) for x in (cu, k, rows)]
    plan, at = mcp.Plan(), [a.ctypes.data_as(ctypes.c_void_p) for a in arrays]
    args = (ctypes.byref(d), *at, len(rows), ctypes.byref(opts), ctypes.byref(plan))
    assert lib.mcp_mixed_attn_plan_rows_host(*args, None, 0) == OK
    buf = np.zeros(max(1, int(plan.off_part_o)), dtype=np.uint8)
    st = lib.mcp_mixed_attn_plan_rows_host(*args, buf.ctypes.data_as(ctypes.c_void_p), buf.size)
    return st, plan, buf[:plan.num_items * 32].view(ITEM).copy()


@pytest.mark.parametrize("hq,hkv,dim,page", [(8, 2, 64, 16), (4, 4, 128, 8), (32, 8, 128, 32),
                                            (3, 1, 96, 64), (8, 8, 256, 16), (2, 2, 64, 1)])
def test_plans_of_trees_cover_every_row_once(lib, hq, hkv, dim, page):
    """Segments of several tokens take tensor-core tiles, the others what they took; the items
    cover every (segment, head, token, key) once, the keys as far as the unit's last token sees."""
    q, k = [1, 4, 2, 0, 70, 1, 300], [9, 4, 700, 5, 9000, 2048, 512]
    cu = np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
    d = mcp.make_desc(len(q), int(cu[-1]), hq, hkv, dim, page, -(-9000 // page), 20000, 0.125)
    for rows in (None, [0, 2, 3, 6, 7, 20, 77, 300]):
        opts = mcp.PlanOptions(num_sms=152, tree=1)
        st, plan, items = plan_rows(lib, d, cu, k, rows, opts) if rows else plan_host(
            d, cu, k, opts=opts)[:3]
        assert st == OK
        covered = {}
        for it in items:
            several = q[it["seg"]] > 1
            assert not (several and it["kind"] == 0)
            for h in range(it["kv_head"], it["kv_head"] + it["num_heads"]):
                for t in range(it["q_begin"], it["q_begin"] + it["q_count"]):
                    covered.setdefault((it["seg"], h, t), []).append((it["kv_begin"], it["kv_end"]))
        want = {(s, t) for s, n in enumerate(q) for t in range(n)}
        if rows:
            want = {(int(np.searchsorted(cu, r, side="right")) - 1, r) for r in rows}
            want = {(s, r - int(cu[s])) for s, r in want}
        assert set(covered) == {(s, h, t) for s, t in want for h in range(hkv)}
        for (s, h, t), spans in covered.items():
            spans.sort()
            assert spans[0][0] == 0 and spans[-1][1] >= k[s] - q[s] + t + 1
            assert all(a[1] == b[0] for a, b in zip(spans, spans[1:]))


def test_tree_rows_of_chains_and_stars():
    bits, depth = ref.tree_rows([-1, 0, 1, 2])
    assert (bits == np.tril(np.ones((4, 4), bool))).all() and depth.tolist() == [0, 1, 2, 3]
    bits, depth = ref.tree_rows([-1, 0, 0, 0])
    assert bits.sum() == 7 and depth.tolist() == [0, 1, 1, 1]
    bits, depth = ref.tree_rows([-1, -1, 1, 5])  # two roots, and a parent behind its token
    assert depth.tolist() == [0, 0, 1, 0] and not bits[1, 0]
    assert ref.pack(np.eye(33, dtype=bool), 2)[31, 0] == np.int32(-(1 << 31))


@pytest.mark.parametrize("given", [False, True])
def test_verified_tokens_are_distributed_like_the_target(given):
    """All ways that a small tree can go, weighed by their probability, give the target's first
    token: the definition's formulas for repeated refusals lose nothing."""
    rng = np.random.default_rng(5)
    V = 5
    p, q = rng.dirichlet(np.ones(V)), rng.dirichlet(np.ones(V))
    target, draft = np.tile(p, (4, 1)), np.tile(q, (4, 1))
    parents = [-1, 0, 0, 0]
    got = np.zeros(V)
    grid = (np.arange(24) + 0.5) / 24
    cases = [(1, 3, 3)] if given else list(np.ndindex(V, V, V))
    for kids in cases:
        weight = 1.0 if given else np.prod([q[x] for x in kids])
        # the three decisions' shares of [0, 1), one after the other
        c, mass, left, gone = 0.0, 1.0, weight, set()
        for x in kids:
            if given:
                ok = 0.0 if x in gone or mass == 0 else min(1.0, p[x] / mass)
            else:
                ok = 0.0 if mass == 0 else min(1.0, max(0.0, p[x] - c * q[x]) / (mass * q[x]))
            got[x] += left * ok
            left *= 1 - ok
            if given:
                mass -= 0.0 if x in gone else p[x]
                gone.add(x)
            else:
                c += mass
                mass = np.maximum(p - c * q, 0).sum()
        w = np.array([0 if v in gone else p[v] for v in range(V)]) if given else np.maximum(p - c * q, 0)
        if w.sum() > 0:
            got += left * w / w.sum()
        # the walk itself decides as those shares say
        for u in grid:
            path, new = ref.verify(target, [0, *kids], [0, u, u, u], 0.3, parents,
                                   None if given else draft)
            first = p[kids[0]] / (1 if given else q[kids[0]])
            assert (len(path) > 1 and path[1] == 1) == (u < first)
            assert len(path) == len(new)
    np.testing.assert_allclose(got, p, atol=1e-12)
