"""Trees of drafted tokens on the GPU, against their definitions in 64 bits: masks and positions,
attention, verification, the move of the accepted path, and all of them as a server runs them."""

from __future__ import annotations

import numpy as np
import pytest

from mixed_chunked_prefill_gb300 import _capi
from oracle import draft_ref as ref

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


def err_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def bits_of(word):
    """Error bits, and the word cleared."""
    v = int(word.item())
    word.zero_()
    return v


def make_tree(rng, n, shape):
    if shape == "chain":
        return np.arange(n) - 1
    if shape == "star":
        return np.where(np.arange(n) > 0, 0, -1)
    if shape == "forest":
        return np.array([int(rng.integers(-1, i)) if i else -1 for i in range(n)])
    return np.array([int(rng.integers(0, i)) if i else -1 for i in range(n)])


def cumulated(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)


# ---------------------------------------------------------------------------- masks
@pytest.mark.parametrize("sizes,words,shape", [
    ([1], 1, "chain"), ([1, 2, 3, 31, 32], 1, "tree"), ([33, 64, 5], 2, "tree"), ([64, 0, 7], 3, "chain"),
    ([128, 97], 4, "star"), ([200, 1, 255], 8, "forest"), ([1024], 32, "chain"), ([1024, 1000], 32, "tree"),
    ([7] * 300, 1, "tree"),
])
def test_masks(mcp, sizes, words, shape):
    rng = np.random.default_rng(sum(sizes) + words)
    # causal segments (-1) between the trees, some without tokens; rows kept free before and between
    q, tree = [], []
    for n in sizes:
        q += [n, int(rng.integers(0, 600))]
        tree += [True, False]
    hist = rng.integers(0, 100000, len(q))
    cu, T = cumulated(q), sum(q)
    at, mask_rows = 2, []
    for n, t in zip(q, tree):
        mask_rows.append(at if t else -1)
        at += n + 1 if t else 0
    parents = np.full(T + 3, 77)
    want = np.full((at, words), 123456, dtype=np.int32)
    pos = np.full(T + 3, -5)
    for s, n in enumerate(q):
        pos[cu[s]:cu[s + 1]] = hist[s] + np.arange(n)
        if tree[s] and n:
            p = make_tree(rng, n, shape)
            parents[cu[s]:cu[s + 1]] = p
            b, depth = ref.tree_rows(p)
            want[mask_rows[s]:mask_rows[s] + n] = ref.pack(b, words)
            pos[cu[s]:cu[s + 1]] = hist[s] + depth
    mask = torch.full((at, words), 123456, dtype=torch.int32, device="cuda")
    positions, err = i32(np.full(T + 3, -5)), err_word()
    args = (i32(parents), i32(cu), i32(hist + q), i32(mask_rows), mask)
    mcp.build_tree_masks(*args, positions, error_word=err)
    assert bits_of(err) == 0
    assert (mask.cpu().numpy() == want).all() and (positions.cpu().numpy() == pos).all()
    mcp.build_tree_masks(*args)  # without positions, and again over its own result
    assert (mask.cpu().numpy() == want).all()


def test_masks_of_malformed_trees(mcp):
    err, pos = err_word(), i32(np.full(12, -5))
    mask = torch.full((9, 1), 7, dtype=torch.int32, device="cuda")
    # a parent that is its token, and one behind it: taken for none
    mcp.build_tree_masks(i32([-1, 1, 3, 2] + [0] * 8), i32([0, 4]), i32([14]), i32([0]), mask, pos, err)
    assert bits_of(err) == mcp.DEVERR_TREE
    assert mask[:4, 0].tolist() == [1, 2, 4, 12] and pos[:4].tolist() == [10, 10, 10, 11]
    # more rows than there are, more tokens than a row has bits: left out
    mask.fill_(7)
    mcp.build_tree_masks(i32([-1, 0] * 6), i32([0, 2, 12]), i32([2, 10]), i32([8, -1]), mask, pos, err)
    assert bits_of(err) == mcp.DEVERR_TREE and (mask == 7).all()
    parents = i32(np.arange(33) - 1)
    mcp.build_tree_masks(parents, i32([0, 33]), i32([33]), i32([0]),
                         torch.zeros((40, 1), dtype=torch.int32, device="cuda"), None, err)
    assert bits_of(err) == mcp.DEVERR_TREE
    # a segment past the tokens, a history below zero, lengths that decrease
    mcp.build_tree_masks(i32([-1] * 4), i32([0, 5]), i32([5]), i32([0]), mask, None, err)
    assert bits_of(err) == mcp.DEVERR_SEGMENT and (mask == 7).all()
    mcp.build_tree_masks(i32([-1] * 4), i32([0, 2]), i32([1]), i32([-1]), mask, None, err)
    assert bits_of(err) == mcp.DEVERR_SEGMENT
    mcp.build_tree_masks(i32([-1] * 4), i32([0, 2, 1]), i32([2, 2]), i32([-1, -1]), mask, None, err)
    assert bits_of(err) == mcp.DEVERR_SEGMENT


def test_masks_of_lengths_at_the_end_of_32_bits(mcp):
    for low in (-(1 << 31), -1, 3):
        for rows in ([0], [-1]):
            err, mask = err_word(), torch.zeros((4, 1), dtype=torch.int32, device="cuda")
            mcp.build_tree_masks(i32([-1, 0, 0, 1]), i32([0, 4]), i32([low]), i32(rows), mask, None, err)
            assert bits_of(err) == mcp.DEVERR_SEGMENT
            assert mask[:, 0].tolist() == ([1, 3, 5, 11] if rows == [0] else [0] * 4)


# ------------------------------------------------------------------------ attention
class Step:
    """A step of segments (tokens, history, shape or None for causal) with random contents."""

    def __init__(self, segments, hq, hkv, D, P, seed=0, spare=3):
        rng = np.random.default_rng(seed)
        self.rng, self.hq, self.hkv, self.D, self.P = rng, hq, hkv, D, P
        self.q, self.hist = [s[0] for s in segments], [s[1] for s in segments]
        self.tree = [s[2] is not None for s in segments]
        self.lens = [a + b for a, b in zip(self.q, self.hist)]
        held = [-(-n // P) for n in self.lens]
        self.pages = sum(held) + spare
        perm = rng.permutation(self.pages)
        self.bt = np.full((len(segments), max(1, max(held))), -1)
        at = 0
        for s, n in enumerate(held):
            self.bt[s, :n] = perm[at:at + n]
            at += n
        self.cu, self.T = cumulated(self.q), sum(self.q)
        self.parents = np.concatenate([make_tree(rng, n, sh) if sh else np.arange(n) - 1
                                       for n, _, sh in segments]).astype(np.int64)
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape):
            return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

        self.qs = normal(self.T, hq, D)
        # what no token of a request lies in holds NaN
        self.k, self.v = (torch.full((self.pages, P, hkv, D), float("nan"), device="cuda",
                                     dtype=torch.bfloat16) for _ in range(2))
        for s, n in enumerate(self.lens):
            page, off = self.slots(s, np.arange(n))
            self.k[page, off], self.v[page, off] = normal(n, hkv, D), normal(n, hkv, D)
        self.scale = D ** -0.5
        self.bits = [ref.tree_rows(self.parents[self.cu[s]:self.cu[s + 1]])[0] for s in range(len(self.q))]

    def slots(self, s, pos):
        return (torch.as_tensor(self.bt[s, pos // self.P]).cuda(), torch.as_tensor(pos % self.P).cuda())

    def masks(self, words=None):
        sizes = [n if t else 0 for n, t in zip(self.q, self.tree)]
        words = words or max(1, -(-max(sizes) // 32))
        rows = cumulated(sizes)
        mask = np.concatenate([np.zeros((0, words), np.int32)] + [
            ref.pack(b, words) for b, t in zip(self.bits, self.tree) if t])
        return i32(mask).reshape(len(mask), words), i32(np.where(self.tree, rows[:-1], -1))

    def plan(self, m, rows=None, **options):
        desc = m.make_desc(len(self.q), self.T, self.hq, self.hkv, self.D, self.P, self.bt.shape[1],
                           self.pages, self.scale)
        opts = m.PlanOptions(tree=1, **options)

        def make(ws=None):
            if rows is None:
                return m.mixed_attn_plan(desc, self.cu, self.lens, opts, ws)
            return m.mixed_attn_plan_rows(desc, self.cu, self.lens, rows, opts, ws)

        ws = torch.empty(max(256, make().workspace_bytes), dtype=torch.uint8, device="cuda")
        return make(ws), ws

    def run(self, m, mask=None, mask_rows=None, rows=None, **options):
        plan, ws = self.plan(m, rows, **options)
        if mask is None:
            mask, mask_rows = self.masks()
        out = torch.full_like(self.qs, float("nan"))
        lse = torch.full((self.T, self.hq), float("nan"), device="cuda")
        m.mixed_attn_fwd_tree(plan, self.qs, self.k, self.v, i32(self.bt), i32(self.cu), i32(self.lens),
                              mask, mask_rows, out, lse, ws)
        self.error = m.workspace_error_word(plan, ws)
        return out, lse

    def check(self, m, out, lse, rows=None):
        m.check_device_errors(self.error)
        self.compare(out, lse, rows)

    def compare(self, out, lse, rows=None):
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for s, n in enumerate(self.q):
            if not n:
                continue
            page, off = self.slots(s, np.arange(self.lens[s]))
            k, v = (c[page, off].double().cpu().numpy() for c in (self.k, self.v))
            a, b = self.cu[s], self.cu[s + 1]
            want, wl, mass = ref.tree_attention(self.qs[a:b].double().cpu().numpy(), k, v, self.hist[s],
                                                self.bits[s], self.scale)
            mine = np.arange(a, b) if rows is None else np.intersect1d(np.arange(a, b), rows)
            # the output's rounding (2^-8 of it) and that of each weight to bf16 (2^-8 of the sum of
            # weight |v|).  Scores: sums of D products in fp32, |q k| scale < 40 a score at most, off by
            # D 2^-23 times that, 2.5e-4 at D = 256 by D = 64 products' 64 2^-23 40 = 3e-4: less than
            # 1e-3 of the weights and of the LSE with the exponentials' own 2^-22.
            bound = 2.0 ** -8 * (np.abs(want) + mass) * 1.01 + 1e-3 * mass + 1e-6
            err = np.abs(out[mine] - want[mine - a])
            assert (err <= bound[mine - a]).all(), (s, float((err / bound[mine - a]).max()))
            assert (np.abs(lse[mine] - wl[mine - a]) <= 1e-3).all(), s


SEGMENTS = [(17, 100, "tree"), (1, 300, None), (5, 0, "tree"), (64, 129, "tree"), (40, 65, None), (1, 0, "tree"),
            (0, 9, None), (2, 127, "star"), (33, 191, "forest"), (3, 253, "chain"), (130, 31, "tree")]


@pytest.mark.parametrize("hq,hkv,D,P", [
    (8, 2, 128, 16), (4, 4, 64, 16), (8, 1, 128, 8), (3, 1, 96, 32), (7, 1, 128, 64), (8, 8, 256, 16),
    (4, 2, 128, 1), (8, 4, 64, 8), (6, 2, 96, 8), (4, 1, 256, 32), (4, 2, 64, 1), (16, 1, 128, 16)])
def test_attention_of_trees(mcp, hq, hkv, D, P):
    st = Step(SEGMENTS, hq, hkv, D, P, seed=hq * D + P)
    st.check(mcp, *st.run(mcp))


@pytest.mark.parametrize("n", [2, 3, 31, 32, 33, 63, 96, 127, 128, 129, 200])
@pytest.mark.parametrize("hist", [0, 1, 127, 128, 500])
def test_attention_where_tiles_end(mcp, n, hist):
    st = Step([(n, hist, "tree")], 4, 2, 64, 16, seed=n + hist)
    st.check(mcp, *st.run(mcp))


@pytest.mark.parametrize("split", [128, 256, 1024])
@pytest.mark.parametrize("D,P", [(128, 16), (256, 32), (64, 1)])
def test_attention_with_split_keys(mcp, split, D, P):
    """Parts that hold no visible key of some rows, and parts that end inside the tree."""
    st = Step([(150, 700, "tree"), (30, 2040, "forest"), (1, 1500, None), (70, 200, None)], 8, 2, D, P, seed=split)
    st.check(mcp, *st.run(mcp, prefill_split_tokens=split))


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("hist", [1200, 5200])
def test_attention_with_many_parts(mcp, D, hist):
    """10 and 41 parts of a row; few rows and more than the GPU merges at once."""
    st = Step([(5, hist, "tree")], 8, 2, D, 16, seed=D + hist)
    st.check(mcp, *st.run(mcp, prefill_split_tokens=128))
    if hist == 1200:
        st = Step([(30, hist, "tree")] * 4, 64, 2, D, 16, seed=D)
        st.check(mcp, *st.run(mcp, prefill_split_tokens=640))


def test_attention_of_any_mask_of_tokens_before(mcp):
    """Masks that no tree has: bits of tokens behind a token, and of words that are not there, do
    not count; rows with more words than their tree needs."""
    st = Step([(50, 77, "tree"), (20, 3, "tree")], 8, 2, 128, 16, seed=3)
    st.bits = [st.rng.random((n, n)) < 0.5 for n in st.q]
    mask, mask_rows = st.masks()
    st.check(mcp, *st.run(mcp, mask, mask_rows))
    mask[:, 1] |= -(1 << 18)  # tokens 50 .. 63 are none of theirs
    st.check(mcp, *st.run(mcp, mask, mask_rows))
    wide, mask_rows = st.masks(5)
    st.check(mcp, *st.run(mcp, wide, mask_rows))
    st.bits[0][:, 32:] = False  # a row of one word hides what it has no bits for
    st.check(mcp, *st.run(mcp, mask[:, :1].contiguous(), mask_rows))


def test_attention_of_a_mask_without_rows(mcp):
    """A mask row that is not there: reported, and its token sees its history and itself."""
    st = Step([(9, 40, "tree"), (6, 10, "tree")], 8, 2, 128, 16, seed=4)
    mask, mask_rows = st.masks()
    out, lse = st.run(mcp, mask[:12].contiguous(), mask_rows)
    st.bits[1][3:] = False
    with pytest.raises(mcp.MCPError):
        mcp.check_device_errors(st.error)
    mcp.check_device_errors(st.error)  # cleared
    st.compare(out, lse)
    none = torch.zeros((0, 1), dtype=torch.int32, device="cuda")
    st.bits = [np.eye(n, dtype=bool) for n in st.q]
    out, lse = st.run(mcp, none, mask_rows)
    with pytest.raises(mcp.MCPError):
        mcp.check_device_errors(st.error)
    st.compare(out, lse)
    st.tree = [False, False]  # no trees at all: causal, with a mask of no rows
    st.bits = [np.tril(np.ones((n, n), dtype=bool)) for n in st.q]
    st.check(mcp, *st.run(mcp, none, i32([-1, -1])))


@pytest.mark.parametrize("D,P", [(128, 16), (64, 8), (96, 32), (256, 64), (128, 1)])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_hidden_tokens_may_hold_anything(mcp, D, P, what):
    """Infinities and NaN in K and V of tokens that a row does not see change nothing in it; the
    rows that see them get what the sum gives."""
    n, hist = 40, 150
    st = Step([(n, hist, "tree"), (6, 20, "star")], 4, 2, D, P, seed=D + P)
    clean_out, clean_lse = st.run(mcp)
    x = n - 9  # a token, and in V one element
    page, off = st.slots(0, np.array([hist + x]))
    keep_v = st.v[page, off].clone()
    st.v[page, off, 1, D // 2] = what
    out, lse = st.run(mcp)
    mcp.check_device_errors(st.error)
    sees = torch.as_tensor(np.concatenate([st.bits[0][:, x] & (np.arange(n) >= x), np.zeros(6, bool)])).cuda()
    assert torch.equal(out[~sees], clean_out[~sees]) and torch.equal(lse, clean_lse)
    hit = out[sees][:, 2:, D // 2].float()
    assert hit.numel() and (torch.isnan(hit).all() if what != what else (hit == what).all())
    rest = out[sees].clone()
    rest[:, 2:, D // 2] = clean_out[sees][:, 2:, D // 2]
    # the element was 0 to the others, which it never was a part of
    assert torch.equal(rest, clean_out[sees])
    st.v[page, off] = keep_v
    st.k[page, off, 1, 3] = what
    out, lse = st.run(mcp)
    mcp.check_device_errors(st.error)
    assert torch.equal(out[~sees], clean_out[~sees]) and torch.equal(lse[~sees], clean_lse[~sees])


def test_attention_of_listed_rows(mcp):
    st = Step(SEGMENTS, 8, 2, 128, 16, seed=9)
    rows = np.sort(st.rng.choice(st.T, 60, replace=False))
    out, lse = st.run(mcp, rows=rows)
    st.check(mcp, out, lse, rows)
    others = np.setdiff1d(np.arange(st.T), rows)
    assert torch.isnan(out[torch.as_tensor(others).cuda()]).all()


def test_chains_are_causal(mcp):
    """A chain's tree and a causal segment are the same attention."""
    segments = [(20, 500, "chain"), (64, 64, "chain"), (3, 1000, "chain")]
    st = Step(segments, 8, 2, 128, 16, seed=11)
    out, lse = st.run(mcp)
    none = torch.zeros((0, 1), dtype=torch.int32, device="cuda")
    causal, cl = st.run(mcp, none, i32([-1] * 3))
    assert torch.equal(out, causal) and torch.equal(lse, cl)


def test_attention_of_padded_rows(mcp):
    """Queries behind the step's tokens are padding: their rows are not written."""
    st = Step([(9, 40, "tree"), (1, 10, None)], 8, 2, 128, 16, seed=14)
    plan, ws = st.plan(mcp)
    mask, mask_rows = st.masks()
    q = torch.cat([st.qs, torch.full((6, 8, 128), float("nan"), dtype=torch.bfloat16, device="cuda")])
    out, lse = torch.full_like(q, 7.0), torch.full((st.T + 6, 8), 7.0, device="cuda")
    mcp.mixed_attn_fwd_tree(plan, q, st.k, st.v, i32(st.bt), i32(st.cu), i32(st.lens), mask, mask_rows, out, lse, ws)
    mcp.check_device_errors(mcp.workspace_error_word(plan, ws))
    st.compare(out[:st.T], lse[:st.T])
    assert (out[st.T:] == 7).all() and (lse[st.T:] == 7).all()


@pytest.mark.parametrize("hq,hkv", [(128, 1), (100, 1), (64, 1), (66, 2)])
def test_attention_of_large_groups(mcp, hq, hkv):
    """One to three tokens a tile."""
    st = Step([(7, 150, "tree"), (3, 300, "star"), (1, 40, None)], hq, hkv, 64, 16, seed=hq)
    st.check(mcp, *st.run(mcp))


def test_attention_of_a_mask_of_many_words(mcp):
    """More tokens than build_tree_masks takes: any mask of 1100 tokens."""
    st = Step([(1100, 200, "chain")], 2, 1, 64, 16, seed=15)
    st.bits = [st.rng.random((1100, 1100)) < 0.3]
    st.check(mcp, *st.run(mcp))


def test_attention_refusals(mcp):
    st = Step([(4, 10, "tree")], 4, 2, 64, 16)
    plan, ws = st.plan(mcp)
    mask, mask_rows = st.masks()
    good = dict(plan=plan, q=st.qs, k_cache=st.k, v_cache=st.v, block_tables=i32(st.bt), cu_seqlens_q=i32(st.cu),
                seqlens_k=i32(st.lens), tree_mask=mask, mask_rows=mask_rows, out=torch.empty_like(st.qs),
                lse=None, workspace=ws)
    mcp.mixed_attn_fwd_tree(**good)
    for name, bad, error in [
            ("q", st.qs[:3], ValueError), ("q", st.qs.float(), TypeError), ("out", st.qs[:3], ValueError),
            ("k_cache", st.k[:1], ValueError), ("v_cache", st.v.cpu(), ValueError),
            ("block_tables", i32(st.bt)[:, :0], ValueError), ("cu_seqlens_q", i32([0, 4, 4]), ValueError),
            ("seqlens_k", i32(st.lens).long(), TypeError), ("tree_mask", mask[0], ValueError),
            ("tree_mask", mask.T.expand(4, 4).T[:, ::2], ValueError), ("mask_rows", i32([0, 0]), ValueError),
            ("mask_rows", None, _capi.MCPError), ("lse", torch.zeros(4, 3, device="cuda"), ValueError),
            ("workspace", None, _capi.MCPError), ("workspace", ws[:128], _capi.MCPError)]:
        with pytest.raises(error):
            mcp.mixed_attn_fwd_tree(**{**good, name: bad})
    plain = mcp.mixed_attn_plan(plan.desc, st.cu, st.lens, None, ws)
    with pytest.raises(_capi.MCPError, match="tree"):
        mcp.mixed_attn_fwd_tree(**{**good, "plan": plain})


def test_waits_that_run_out_end_a_step_with_trees(mcp):
    """The abort path (no Q tile arrives, waits give up after 1 ms): no row is written, the error
    is reported, and the next plan in the same workspace runs."""
    st = Step([(40, 200, "tree"), (1, 30, None), (20, 0, "star")], 8, 2, 128, 16, seed=12)
    plan, ws = st.plan(mcp, test_stall=1)
    mask, mask_rows = st.masks()
    out = torch.full_like(st.qs, float("nan"))
    lse = torch.full((st.T, 8), float("nan"), device="cuda")
    args = (st.qs, st.k, st.v, i32(st.bt), i32(st.cu), i32(st.lens), mask, mask_rows, out, lse)
    mcp.mixed_attn_fwd_tree(plan, *args, ws)
    with pytest.raises(_capi.MCPError) as e:
        mcp.check_device_errors(mcp.workspace_error_word(plan, ws))
    assert e.value.status == _capi.MCP_ERR_TIMEOUT
    trees = torch.as_tensor([True] * 40 + [False] + [True] * 20).cuda()
    assert torch.isnan(out[trees]).all() and not torch.isnan(out[~trees]).any()
    desc, options = plan.desc, mcp.PlanOptions(tree=1)
    big = torch.empty(max(ws.numel(), mcp.mixed_attn_plan(desc, st.cu, st.lens, options).workspace_bytes),
                      dtype=torch.uint8, device="cuda")
    plan = mcp.mixed_attn_plan(desc, st.cu, st.lens, options, big)
    mcp.mixed_attn_fwd_tree(plan, *args, big)
    mcp.check_device_errors(mcp.workspace_error_word(plan, big))
    st.compare(out, lse)


def test_attention_past_32_bits(mcp):
    """Pages whose elements lie past 2^31 of the caches."""
    P, H, D, pages = 16, 8, 128, (1 << 31) // (16 * 8 * 128) + 64
    st = Step([(20, 300, "tree"), (1, 100, None), (34, 90, "star")], 8, H, D, P, seed=13)
    big_k = torch.empty((pages, P, H, D), dtype=torch.bfloat16, device="cuda")
    big_v = torch.empty_like(big_k)
    used = torch.as_tensor(np.unique(st.bt[st.bt >= 0])).cuda()
    top = pages - 1 - torch.arange(st.pages, device="cuda")
    big_k[top[used]], big_v[top[used]] = st.k[used], st.v[used]
    big_v[top[used[0]]] = st.v[used[0]]
    st.bt = np.where(st.bt >= 0, pages - 1 - st.bt, -1)
    st.k, st.v, st.pages = big_k, big_v, pages
    st.check(mcp, *st.run(mcp))
    page, off = st.slots(0, np.array([300 + 5]))
    st.v[page, off, 0, 0] = float("inf")  # read again by the rows that see it
    out, _ = st.run(mcp)
    sees = torch.as_tensor(st.bits[0][:, 5]).cuda()
    assert torch.isinf(out[:20][sees][:, 0, 0].float()).all()
    assert torch.isfinite(out[:20][~sees].float()).all()


# ----------------------------------------------------------------------- verification
class Drafts:
    """Trees of drafted tokens with the probabilities that they are tried against."""

    def __init__(self, sizes, V, dtype="fp32", shape="tree", draft=True, seed=0, spread=2.0, gap=0, wide=0):
        rng = np.random.default_rng(seed)
        self.sizes, self.V, self.cu, R = sizes, V, cumulated(sizes), sum(sizes)
        z = rng.standard_normal((R, V)) * spread

        def rows(logits):
            e = np.exp(logits - logits.max(1, keepdims=True)) if R else logits
            full = torch.zeros((R + gap, V + wide), dtype=DT[dtype], device="cuda")
            part = full[:R, wide // 2:wide // 2 + V]
            part.copy_(torch.as_tensor(e / e.sum(1, keepdims=True) if R else e))
            return part

        self.target = rows(z)
        self.draft = rows(z + rng.standard_normal((R, V)) * 0.8) if draft else None
        self.parents = np.concatenate([make_tree(rng, n, shape) for n in sizes] + [[]]).astype(np.int64)
        self.chain = shape == "chain"
        self.tokens = np.zeros(R, dtype=np.int64)
        for s, n in enumerate(sizes):
            a = self.cu[s]
            for i in range(1, n):
                up = a + max(0, self.parents[a + i])
                if draft:
                    w = ref._clean(self.draft[up].double().cpu().numpy())
                    self.tokens[a + i] = rng.choice(V, p=w / w.sum()) if w.sum() > 0 else 0
                else:
                    top = np.argsort(-self.target[up].double().cpu().numpy(), kind="stable")
                    self.tokens[a + i] = top[min(V - 1, int(rng.integers(0, 4)))]
        self.u = rng.random(R).astype(np.float32)
        self.u_last = rng.random(len(sizes)).astype(np.float32)

    def run(self, m, err=None, **kw):
        f32 = dict(dtype=torch.float32, device="cuda")
        args = dict(target_probs=self.target, tokens=i32(self.tokens), cu_rows=i32(self.cu),
                    uniform=torch.tensor(self.u, **f32), final_uniform=torch.tensor(self.u_last, **f32),
                    parents=None if self.chain else i32(self.parents), draft_probs=self.draft, error_word=err)
        return m.verify_drafts(**{**args, **kw})

    def want(self):
        accepted, path, new = [], np.full(sum(self.sizes), -1), np.full(sum(self.sizes), -1)
        target = self.target.double().cpu().numpy()
        draft = None if self.draft is None else self.draft.double().cpu().numpy()
        for s, n in enumerate(self.sizes):
            a, b = self.cu[s], self.cu[s + 1]
            if not n:
                accepted.append(0)
                continue
            p, t = ref.verify(target[a:b], self.tokens[a:b], self.u[a:b], self.u_last[s],
                              self.parents[a:b], None if draft is None else draft[a:b])
            path[a:a + len(p)], new[a:a + len(t)] = p, t
            accepted.append(len(p))
        return np.array(accepted), path, new

    def check(self, m, bits=0, **kw):
        err = err_word()
        got = self.run(m, err, **kw)
        assert bits_of(err) == bits
        for name, g, w in zip(("accepted", "path", "new"), got, self.want()):
            assert g.cpu().numpy().tolist() == w.tolist(), name
        return got


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("shape,draft", [("chain", True), ("tree", True), ("star", True), ("forest", True),
                                         ("chain", False), ("tree", False), ("star", False)])
@pytest.mark.parametrize("V", [1, 2, 7, 1000, 4099])
def test_verify(mcp, dtype, shape, draft, V):
    d = Drafts([1, 5, 0, 12, 2, 33, 1, 8], V, dtype, shape, draft, seed=V, spread=1.5 if V < 10 else 3.0)
    d.check(mcp)


@pytest.mark.parametrize("V,dtype,wide", [(128000, "fp32", 0), (50257, "bf16", 0), (50257, "fp32", 3),
                                          (33333, "fp16", 6), (8192, "bf16", 8)])
@pytest.mark.parametrize("draft", [True, False])
def test_verify_large_vocabularies(mcp, V, dtype, wide, draft):
    """Rows shared by clusters of CTAs, of every alignment, and part of wider rows."""
    Drafts([1, 6, 4], V, dtype, "tree", draft, seed=V, spread=2.5, wide=wide).check(mcp)
    Drafts([3] * 40, V // 8, dtype, "chain", draft, seed=V, spread=2.5, wide=wide).check(mcp)


def test_verify_rows_of_different_alignment(mcp):
    d = Drafts([4, 6], 5001, "bf16", "tree", True, seed=1)
    wide = torch.zeros((10, 5010), dtype=torch.bfloat16, device="cuda")
    wide[:, 1:5002] = d.draft
    d.draft = wide[:, 1:5002]
    d.check(mcp)


def test_verify_many_segments(mcp):
    """More clusters than the GPU holds at once."""
    Drafts([2, 3, 1, 4] * 200, 20000, "fp32", "tree", True, seed=2).check(mcp)


def test_verify_long_trees(mcp):
    Drafts([1024, 1000], 64, "fp32", "chain", True, seed=3).check(mcp)
    Drafts([1024], 64, "fp32", "star", True, seed=4).check(mcp)
    Drafts([700], 64, "fp32", "star", False, seed=5).check(mcp)


@pytest.mark.parametrize("draft", [True, False])
def test_verify_numbers_at_their_ends(mcp, draft):
    """Random numbers of 0 and 1: the first and the last token with any weight."""
    for u, last in [(0.0, 0.0), (1.0, 1.0), (0.0, 1.0), (1.0, 0.0)]:
        d = Drafts([5, 7, 1], 900, "fp32", "tree", draft, seed=6)
        d.target[:, :3] = 0
        d.target[:, -2:] = 0
        d.u[:], d.u_last[:] = u, last
        d.check(mcp)


def test_verify_equal_and_disjoint_rows(mcp):
    d = Drafts([6, 6, 6], 500, "fp32", "star", True, seed=7)
    d.draft.copy_(d.target)  # everything is accepted
    accepted = d.check(mcp)[0]
    assert accepted.tolist() == [2, 2, 2]
    d.u[:] = 1.0  # or refused, and nothing remains: the target itself
    d.check(mcp)
    d = Drafts([4, 5], 500, "fp32", "chain", True, seed=8)
    d.target[:, ::2] = 0
    d.draft[:, 1::2] = 0
    d.tokens = d.tokens // 2 * 2
    assert d.check(mcp)[0].tolist() == [1, 1]


def test_verify_greedy_rows(mcp):
    """One-hot targets: the drafts that are the likeliest tokens, then the next of them."""
    d = Drafts([6, 9], 300, "bf16", "tree", False, seed=9)
    best = d.target.float().argmax(1)
    d.target.zero_()
    d.target[torch.arange(15).cuda(), best] = 1
    for draft in (None, torch.full_like(d.target, 1 / 256)):
        d.draft = draft
        d.check(mcp)


def test_verify_the_same_token_twice(mcp):
    for draft in (True, False):
        d = Drafts([8, 8], 40, "fp32", "star", draft, seed=10)
        d.tokens[:] = d.tokens[1]
        d.u[:] = 0.99
        d.check(mcp)


def test_verify_entries_that_are_no_probabilities(mcp):
    for draft in (True, False):
        d = Drafts([9, 4, 4], 2000, "fp32", "tree", draft, seed=11)
        for m in (d.target, d.draft):
            if m is not None:
                m[:, 5::50], m[:, 6::50], m[:, 7::50], m[:, 8::50] = (
                    float("nan"), -0.5, float("inf"), -float("inf"))
        d.check(mcp)
    d.target[d.cu[1]:d.cu[2]] = 0  # a row without any
    d.tokens[:] = -1               # padding: no drafts at all
    d.check(mcp, bits=mcp.DEVERR_PROBS)


def test_verify_nothing(mcp):
    """No segments, no rows, segments without rows."""
    f = torch.zeros(0, device="cuda")
    none = torch.zeros((0, 50), device="cuda")
    got = mcp.verify_drafts(none, i32([]), i32([0]), f, f)
    assert [x.shape[0] for x in got] == [0, 0, 0]
    err = err_word()
    got = mcp.verify_drafts(none, i32([]), i32([0, 0, 0]), f, torch.zeros(2, device="cuda"), error_word=err)
    assert got[0].tolist() == [0, 0] and bits_of(err) == 0


def test_verify_malformed_drafts(mcp):
    d = Drafts([5, 5], 100, "fp32", "tree", True, seed=12)
    d.u[:] = 0.0
    d.tokens[1], d.tokens[2] = 100, -7
    d.check(mcp, bits=mcp.DEVERR_TOKEN_RANGE)
    d.tokens[1:3] = 5
    d.parents[7] = 2  # itself: under none
    d.check(mcp, bits=mcp.DEVERR_TREE)
    d.parents[7] = 0
    # segments that are not there: nothing of theirs is written
    out = [i32([9] * 2), i32([9] * 10), i32([9] * 10)]
    for cu in ([0, 5, 11], [0, 5, 3], [-1, 5, 10]):
        err = err_word()
        accepted, path, new = d.run(mcp, err, cu_rows=i32(cu), accepted=out[0].clone(), path=out[1].clone(),
                                    new_tokens=out[2].clone())
        assert bits_of(err) == mcp.DEVERR_SEGMENT
        bad = 0 if cu[0] < 0 else 1
        assert accepted.tolist()[bad] == 0
        assert (path[5 * bad:5 * bad + 5] == 9).all() and (new[5 * bad:5 * bad + 5] == 9).all()
    big = Drafts([1025], 8, "fp32", "star", False, seed=1)
    err = err_word()
    assert big.run(mcp, err)[0].tolist() == [0] and bits_of(err) == mcp.DEVERR_SEGMENT


def test_verify_leaves_rows_behind_the_last_segment(mcp):
    d = Drafts([4, 3, 5], 100, "fp32", "tree", True, seed=13)
    out = i32([9] * 2), i32([9] * 12), i32([9] * 12)
    accepted, path, new = d.run(mcp, cu_rows=i32([0, 4, 7]), final_uniform=torch.rand(2, device="cuda"),
                                accepted=out[0], path=out[1], new_tokens=out[2])
    assert (path[7:] == 9).all() and (new[7:] == 9).all() and (path[:7] != 9).all()


@pytest.mark.parametrize("draft", [True, False])
def test_verified_tokens_are_distributed_like_the_target(mcp, draft):
    """100000 small trees over the same rows: the first token out is distributed as p, whatever q."""
    S, V, n = 100000, 6, 4
    rng = np.random.default_rng(14)
    p, q = rng.dirichlet(np.ones(V)), rng.dirichlet(np.ones(V))
    target = torch.tensor(p, dtype=torch.float32, device="cuda").expand(S * n, V).contiguous()
    dq = torch.tensor(q, dtype=torch.float32, device="cuda").expand(S * n, V).contiguous() if draft else None
    tokens = rng.choice(V, size=S * n, p=q) if draft else np.tile([0, 2, 4, 5], S)
    g = torch.Generator(device="cuda").manual_seed(15)
    _, _, new = mcp.verify_drafts(target, i32(tokens), i32(np.arange(S + 1) * n),
                                  torch.rand(S * n, generator=g, device="cuda"),
                                  torch.rand(S, generator=g, device="cuda"),
                                  parents=i32(np.tile([-1, 0, 0, 0], S)), draft_probs=dq)
    first = np.bincount(new[::n].cpu().numpy(), minlength=V) / S
    assert (np.abs(first - p) < 5 * np.sqrt(p * (1 - p) / S)).all()  # five standard deviations


def test_verify_rows_past_32_bits(mcp):
    """The last rows of matrices of more than 2^31 elements."""
    V, n = 100000, 6
    R = (1 << 31) // V + 20
    d = Drafts([n], V, "bf16", "tree", True, seed=16)
    target, draft = (torch.empty((R, V), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    target[R - n:], draft[R - n:] = d.target, d.draft
    tokens, parents = (torch.full((R,), -1, dtype=torch.int32, device="cuda") for _ in range(2))
    tokens[R - n:], parents[R - n:] = i32(d.tokens), i32(d.parents)
    u = torch.zeros(R, device="cuda")
    u[R - n:] = torch.tensor(d.u)
    accepted, path, new = mcp.verify_drafts(target, tokens, i32([R - n, R]), u, torch.tensor(d.u_last).cuda(),
                                            parents=parents, draft_probs=draft)
    want = d.want()
    assert accepted.tolist() == want[0].tolist()
    assert path[R - n:].tolist() == want[1].tolist() and new[R - n:].tolist() == want[2].tolist()


def test_verify_at_once_on_two_streams(mcp):
    a, b = (Drafts([7] * 50, 40000, "fp32", "tree", True, seed=s) for s in (17, 18))
    want = [a.run(mcp), b.run(mcp)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = [d.run(mcp, stream=st) for d, st in zip((a, b), streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(g, w))


def test_verify_refusals(mcp):
    d = Drafts([3, 4], 50)
    d.run(mcp)
    f = torch.zeros(7, device="cuda")
    for name, bad, error in [
            ("target_probs", d.target.double(), TypeError), ("target_probs", d.target.int(), TypeError),
            ("target_probs", d.target.cpu(), ValueError), ("target_probs", d.target[0], ValueError),
            ("target_probs", d.target.T.contiguous().T, ValueError), ("draft_probs", d.target[:6], ValueError),
            ("draft_probs", d.target.half(), TypeError), ("tokens", i32([0] * 6), ValueError),
            ("tokens", f, TypeError), ("parents", i32([0] * 6), ValueError), ("cu_rows", i32([[0, 7]]), ValueError),
            ("cu_rows", torch.zeros(0, dtype=torch.int32, device="cuda"), ValueError), ("uniform", f[:6], ValueError),
            ("uniform", f.double(), TypeError), ("final_uniform", f[:1], ValueError),
            ("accepted", i32([0]), ValueError), ("path", i32([0] * 6), ValueError),
            ("new_tokens", f, TypeError), ("error_word", f, TypeError)]:
        with pytest.raises(error):
            d.run(mcp, **{name: bad})


# ------------------------------------------------------------------------------- keep
def paths(rng, sizes):
    accepted, path = [], []
    for n in sizes:
        m = int(rng.integers(1, n + 1)) if n else 0
        rest = np.sort(rng.choice(np.arange(1, n), m - 1, replace=False)) if m > 1 else []
        accepted.append(m)
        path += [0, *rest][:m] + [-1] * (n - m)
    return np.array(accepted), np.array(path, dtype=np.int64)


@pytest.mark.parametrize("P", [1, 8, 16, 32, 64])
@pytest.mark.parametrize("layers,H,D", [(1, 2, 64), (3, 1, 8), (70, 1, 96), (2, 8, 128)])
def test_keep(mcp, P, layers, H, D):
    rng = np.random.default_rng(P + layers)
    sizes = [1, 20, 0, 64, 7, 300, 2]
    st = Step([(n, int(rng.integers(0, 200)), None) for n in sizes], H, H, 64, P, seed=P)
    accepted, path = paths(rng, sizes)
    g = torch.Generator(device="cuda").manual_seed(P)
    k, v = (torch.randn((layers, st.pages, P, H, D), generator=g, device="cuda").to(torch.bfloat16)
            for _ in range(2))
    want = [x.view(torch.int16).cpu().numpy() for x in (k, v)]
    for w in want:
        for s, n in enumerate(sizes):
            for layer in w:
                ref.keep(layer, st.bt[s], st.hist[s], path[st.cu[s]:st.cu[s] + accepted[s]], P)
    lists = [x.clone().unbind(0) for x in (k, v)]
    err = err_word()
    args = (i32(st.bt), i32(st.cu), i32(st.lens), i32(accepted), i32(path))
    new = mcp.kv_keep_path(k, v, *args, error_word=err)
    assert bits_of(err) == 0 and new.tolist() == [h + a for h, a in zip(st.hist, accepted)]
    for got, w in zip((k, v), want):
        assert (got.view(torch.int16).cpu().numpy() == w).all()
    mcp.kv_keep_path(list(lists[0]), lists[1], *args)
    for got, w in zip(lists, want):
        assert all((a.view(torch.int16).cpu().numpy() == b).all() for a, b in zip(got, w))


def test_keep_in_a_pool_of_both(mcp):
    """K and V of each layer side by side in one tensor."""
    st = Step([(9, 20, None), (4, 7, None)], 2, 2, 64, 16, seed=8)
    pool = torch.randn((3, 2, st.pages, 16, 2, 64), device="cuda").to(torch.bfloat16)
    want = pool.view(torch.int16).cpu().numpy()
    accepted, path = [3, 2], [0, 4, 7] + [-1] * 6 + [0, 3, -1, -1]
    for layer in range(3):
        for half in range(2):
            for s in range(2):
                ref.keep(want[layer, half], st.bt[s], st.hist[s],
                         path[st.cu[s]:st.cu[s] + accepted[s]], 16)
    mcp.kv_keep_path(pool[:, 0], pool[:, 1], i32(st.bt), i32(st.cu), i32(st.lens), i32(accepted), i32(path))
    assert (pool.view(torch.int16).cpu().numpy() == want).all()
    with pytest.raises(ValueError):  # a layer's cache that is not dense
        mcp.kv_keep_path(pool[:, 0, :, ::2], pool[:, 1, :, ::2], i32(st.bt), i32(st.cu), i32(st.lens),
                         i32(accepted), i32(path))


def test_keep_of_steps_with_chunks(mcp):
    """Segments that have fewer rows than tokens had no drafts: they keep what they have."""
    sizes = [300, 6, 1, 40, 0]
    st = Step([(n, 30 + n, None) for n in sizes], 2, 2, 64, 16, seed=5)
    rows = [1, 6, 1, 0, 0]
    accepted, path = [1, 3, 1, 0, 0], [0, 0, 2, 5, -1, -1, -1, 0]
    k, v = st.k.clone(), st.v.clone()
    for w in (st.k, st.v):
        w = w.view(torch.int16)
        a, b = st.slots(1, np.array([36 + 2, 36 + 5]))
        rows2 = w[a, b].clone()
        a, b = st.slots(1, np.array([36 + 1, 36 + 2]))
        w[a, b] = rows2
    err = err_word()
    new = mcp.kv_keep_path(k, v, i32(st.bt), i32(st.cu), i32(st.lens), i32(accepted), i32(path),
                           cu_rows=i32(cumulated(rows)), error_word=err)
    assert bits_of(err) == 0 and new.tolist() == [630, 39, 32, 110, 30]
    for got, w in ((k, st.k), (v, st.v)):
        assert torch.equal(got.view(torch.int16), w.view(torch.int16))


@pytest.mark.parametrize("accepted,path,change,bits", [
    ([4], [0, 2, 2, 3, 0], {}, "TREE"), ([3], [0, 3, 1, 0, 0], {}, "TREE"), ([2], [0, 5, 0, 0, 0], {}, "TREE"),
    ([2], [-1, 2, 0, 0, 0], {}, "TREE"), ([6], [0, 1, 2, 3, 4], {}, "TREE"), ([-1], [0] * 5, {}, "TREE"),
    ([2], [0, 3, 0, 0, 0], dict(sk=[4]), "SEGMENT"), ([2], [0, 3, 0, 0, 0], dict(cu=[0, -1]), "SEGMENT"),
    ([2], [0, 3, 0, 0, 0], dict(cu_rows=[1, 6]), "SEGMENT"), ([2], [0, 3, 0, 0, 0], dict(sk=[10000]), "SEGMENT"),
    ([2], [0, 3, 0, 0, 0], dict(cu_rows=[0, -1]), "SEGMENT")])
def test_keep_of_malformed_paths(mcp, accepted, path, change, bits):
    st = Step([(5, 30, None)], 2, 2, 64, 16, seed=6)
    sk = change.get("sk", st.lens)
    before, err = st.k.clone(), err_word()
    new = mcp.kv_keep_path(st.k, st.v, i32(st.bt), i32(change.get("cu", st.cu)), i32(sk), i32(accepted),
                           i32(path), cu_rows=i32(change["cu_rows"]) if "cu_rows" in change else None,
                           error_word=err)
    assert bits_of(err) == getattr(mcp, "DEVERR_" + bits)
    assert new.tolist() == list(sk) and torch.equal(st.k.view(torch.int16), before.view(torch.int16))


def test_keep_of_lengths_at_the_end_of_32_bits(mcp):
    st = Step([(5, 30, "chain"), (1, 3, None)], 2, 2, 64, 16)
    k, v = st.k.clone(), st.v.clone()
    for low in (-(1 << 31), -(1 << 31) + 4, -1, 4):
        err = err_word()
        new = mcp.kv_keep_path(st.k, st.v, i32(st.bt), i32(st.cu), i32([low, 4]), i32([2, 1]),
                               i32([0, 2, -1, -1, -1, 0]), error_word=err)
        assert bits_of(err) == mcp.DEVERR_SEGMENT and new.tolist() == [low, 4]
    assert (k.view(torch.int16) == st.k.view(torch.int16)).all()
    assert (v.view(torch.int16) == st.v.view(torch.int16)).all()


def test_keep_leaves_out_pages_outside_the_pool(mcp):
    st = Step([(40, 10, None)], 2, 2, 64, 16, seed=7)
    bt, err = st.bt.copy(), err_word()
    bt[0, 1], bt[0, 2] = st.pages, -3
    before = st.k.clone()
    mcp.kv_keep_path(st.k, st.v, i32(bt), i32(st.cu), i32(st.lens), i32([3]),
                     i32([0, 10, 38] + [-1] * 37), error_word=err)
    assert bits_of(err) == mcp.DEVERR_PAGE_RANGE
    a, b = st.slots(0, np.array([12]))
    c, d = st.slots(0, np.array([10 + 38]))
    before[a, b] = before[c, d]  # the one move whose pages are there
    assert torch.equal(st.k.view(torch.int16), before.view(torch.int16))


def test_keep_past_32_bits(mcp):
    P, H, D, pages = 16, 8, 128, (1 << 31) // (16 * 8 * 128) + 8
    k = torch.zeros((pages, P, H, D), dtype=torch.bfloat16, device="cuda")
    k[pages - 1, 3], k[2, 1] = 5, 7
    v = k.clone()
    bt = i32([[1, pages - 2], [2, pages - 1]])
    new = mcp.kv_keep_path(k, v, bt, i32([0, 20, 40]), i32([20, 20]), i32([1, 3]),
                           i32([0] + [-1] * 19 + [0, 17, 19] + [-1] * 17))
    assert new.tolist() == [1, 3]
    for c in (k, v):
        assert (c[2, 2] == 5).all() and (c[2, 1] == 0).all() and (c[pages - 1, 3] == 5).all()
        assert float(c.float().sum()) == 2 * 5 * H * D


def test_keep_refusals(mcp):
    st = Step([(5, 30, None)], 2, 2, 64, 16)
    good = dict(k_caches=st.k, v_caches=st.v, block_tables=i32(st.bt), cu_seqlens_q=i32(st.cu),
                seqlens_k=i32(st.lens), accepted=i32([1]), path=i32([0] * 5))
    mcp.kv_keep_path(**good)
    for name, bad, error in [
            ("k_caches", [], ValueError), ("k_caches", [st.k, st.k], ValueError), ("k_caches", st.k[0], ValueError),
            ("k_caches", st.k.float(), TypeError), ("k_caches", st.k.cpu(), ValueError),
            ("v_caches", st.v[:1], ValueError), ("v_caches", st.v[..., :32], ValueError),
            ("k_caches", [st.k[0]], ValueError), ("k_caches", 3, TypeError),
            ("block_tables", i32(st.bt)[0], ValueError), ("accepted", i32([1, 1]), ValueError),
            ("path", i32([[0] * 5]), ValueError), ("cu_rows", i32([0]), ValueError),
            ("new_lens", i32([0, 0]), ValueError), ("seqlens_k", i32([[3]]), ValueError)]:
        with pytest.raises(error):
            mcp.kv_keep_path(**{**good, name: bad})


# ---------------------------------------------------------- a step of host metadata
@pytest.mark.parametrize("some_rows", [False, True])
def test_a_step_of_host_metadata(mcp, some_rows):
    """MixedStep built from lists on the host: its masks and positions, the append of the step's
    K/V, and the attention of all rows or of some."""
    from mixed_chunked_prefill_gb300.step import MixedStep

    st = Step(SEGMENTS, 8, 2, 128, 16, seed=31)
    own = [st.slots(s, np.arange(h, n)) for s, (h, n) in enumerate(zip(st.hist, st.lens))]
    at = tuple(torch.cat(x) for x in zip(*own))
    k_new, v_new = st.k[at].clone(), st.v[at].clone()
    st.k[at] = st.v[at] = float("nan")
    rows = np.flatnonzero(st.rng.random(st.T) < 0.3) if some_rows else None
    options = mcp.PlanOptions(split_kv=256)
    step = MixedStep(st.hq, st.hkv, st.D, st.P, st.pages, st.scale, st.cu, st.lens, st.bt, options=options,
                     rows=rows, trees=st.tree, parents=st.parents)
    assert options.tree == 0  # the caller's stay as they were
    bits, depths = zip(*(ref.tree_rows(st.parents[a:b]) for a, b in zip(st.cu, st.cu[1:])))
    assert step.trees.positions.tolist() == [h + int(x) for h, d in zip(st.hist, depths) for x in d]
    mask, mask_rows = st.masks()
    assert torch.equal(step.trees.tree_mask, mask) and torch.equal(step.trees.mask_rows, mask_rows)
    out = torch.full_like(st.qs, float("nan"))
    lse = torch.full((st.T, st.hq), float("nan"), device="cuda")
    step.run(st.qs, k_new, v_new, st.k, st.v, out, lse)
    step.check()
    st.compare(out, lse, rows)
    if some_rows:
        others = np.setdiff1d(np.arange(st.T), rows)
        assert torch.isnan(out[others]).all() and torch.isnan(lse[others]).all()


def test_a_step_of_host_metadata_refusals(mcp):
    from mixed_chunked_prefill_gb300.step import MixedStep

    def step(q, hist, **more):
        lens = [a + b for a, b in zip(q, hist)]
        width = -(-max(lens) // 16)
        bt = np.arange(len(q) * width).reshape(len(q), width)
        return MixedStep(4, 2, 64, 16, bt.size, 0.125, cumulated(q), lens, bt, **more)

    step([3, 1], [5, 9], trees=[True, False], parents=[-1, 0, 0, -1])
    step([1024], [0], trees=[True], parents=np.arange(1024) - 1).check()
    for bad in (dict(trees=[True, False]), dict(parents=[-1, 0, 0, -1]),
                dict(trees=[True], parents=[-1, 0, 0, -1]), dict(trees=[True, False], parents=[-1, 0, 0]),
                dict(trees=[True, False], parents=[[-1, 0, 0, -1]])):
        with pytest.raises(ValueError):
            step([3, 1], [5, 9], **bad)
    with pytest.raises(ValueError):  # a tree of more tokens than a mask has bits
        step([1025], [0], trees=[True], parents=np.arange(1025) - 1)
    step([1025], [0], trees=[False], parents=np.arange(1025) - 1).check()  # a chunk has no limit


# ------------------------------------------------------------------ all of them together
def test_serving_with_drafted_trees(mcp):
    """Requests served with trees beside chunks and decodes: tables, masks, append, attention,
    verification, the kept paths, token counts and the commit, step after step.  The caches then
    hold each request's accepted tokens in order, and attention over them is the definition's."""
    from mixed_chunked_prefill_gb300.step import LogitsState, MixedStep, RequestTables

    R, P, H, G, D, V, layers = 5, 16, 2, 2, 64, 400, 3
    rng = np.random.default_rng(20)
    tables = RequestTables(80, P, R, 12)
    state = LogitsState(R, V)
    kc, vc = (torch.full((layers, 80, P, H, D), float("nan"), dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(21)
    held = [[torch.zeros((layers, 2, 0, H, D), dtype=torch.bfloat16, device="cuda")][0] for _ in range(R)]
    said = [[] for _ in range(R)]
    prompt = [30, 17, 90, 5, 44]
    state.admit(i32(range(R)), torch.zeros(0, dtype=torch.int32, device="cuda"), i32([0] * (R + 1)))
    for step_no in range(6):
        ids = list(rng.permutation(R))
        q, tree = [], []
        for r in ids:
            if tables.lens_h[r] == 0:
                q.append(prompt[r]), tree.append(False)       # its prompt
            elif rng.random() < 0.25:
                q.append(1), tree.append(False)               # a decode
            else:
                q.append(int(rng.integers(2, 20))), tree.append(True)
        st = tables.step(ids, q)
        T = sum(q)
        parents = np.concatenate([make_tree(rng, n, "tree" if t else "chain") for n, t in zip(q, tree)])
        step = MixedStep.from_tables(st, H * G, H, D, D ** -0.5, trees=tree, parents=parents)
        bits, depth = zip(*(ref.tree_rows(parents[a:b]) for a, b in zip(st.cu_h, st.cu_h[1:])))
        hist = [int(tables.lens_h[r]) for r in ids]
        assert step.trees.positions.tolist() == [h + int(x) for h, d in zip(hist, depth) for x in d]
        new_kv = torch.randn((layers, 2, T, H, D), generator=g, device="cuda").to(torch.bfloat16)
        for layer in range(layers):
            qs = torch.randn((T, H * G, D), generator=g, device="cuda").to(torch.bfloat16)
            out = torch.empty_like(qs)
            step.run(qs, new_kv[layer, 0], new_kv[layer, 1], kc[layer], vc[layer], out)
            for s, r in enumerate(ids):
                a, b = st.cu_h[s], st.cu_h[s + 1]
                k, v = (torch.cat([held[r][layer, i], new_kv[layer, i, a:b]]).double().cpu().numpy()
                        for i in range(2))
                want, _, mass = ref.tree_attention(qs[a:b].double().cpu().numpy(), k, v, hist[s], bits[s],
                                                   D ** -0.5)
                bound = 2.0 ** -8 * (np.abs(want) + mass) * 1.01 + 1e-3 * mass + 1e-6  # as above
                assert (np.abs(out[a:b].double().cpu().numpy() - want) <= bound).all()
        # rows of probabilities: every token of trees and decodes, the last one of prompts
        counts = [n if t else 1 for n, t in zip(q, tree)]
        cu_rows = cumulated(counts)
        d = Drafts(counts, V, "fp32", "tree", True, seed=22 + step_no)
        d.parents = np.concatenate([p for p in (
            parents[st.cu_h[s]:st.cu_h[s + 1]] if tree[s] else np.array([-1]) for s in range(R))])
        err = err_word()
        accepted, path, new = d.check(mcp)
        state.add(st.request_ids, new, i32(cu_rows))
        new_lens = step.keep(kc, vc, accepted, path, i32(cu_rows))
        step.check()
        tables.commit(st, new_lens.cpu().numpy())
        tables.check()
        acc, pth, tok = accepted.tolist(), path.tolist(), new.tolist()
        for s, r in enumerate(ids):
            a = st.cu_h[s]
            places = pth[cu_rows[s]:cu_rows[s] + acc[s]] if tree[s] or q[s] == 1 else range(q[s])
            held[r] = torch.cat([held[r], new_kv[:, :, [a + i for i in places]]], 2)
            said[r] += tok[cu_rows[s]:cu_rows[s] + acc[s]]
            assert held[r].shape[2] == tables.lens_h[r] == new_lens[s]
    pages = tables.request_pages.cpu().numpy()
    for r in range(R):
        n = int(tables.lens_h[r])
        at = torch.as_tensor(pages[r, np.arange(n) // P]).cuda(), torch.as_tensor(np.arange(n) % P).cuda()
        for layer in range(layers):
            assert torch.equal(kc[layer][at], held[r][layer, 0]) and torch.equal(vc[layer][at], held[r][layer, 1])
        assert state.counts[r, :V].tolist() == np.bincount(said[r], minlength=V).tolist()


def test_captured_and_replayed(mcp):
    """Masks, attention, verification and keep in one graph, replayed with other trees, drafts and
    contents; a second graph over the same workspace in turn."""
    def fresh(seed):
        st = Step([(20, 100, "tree"), (1, 40, None), (33, 2100, "tree")], 8, 2, 128, 16, seed=seed)
        return st, Drafts(st.q, 9000, "fp32", "tree", True, seed=seed)

    st, d = fresh(1)
    d.parents = st.parents
    plan, ws = st.plan(mcp)
    assert plan.num_combine > 0
    mask = torch.zeros((53, 2), dtype=torch.int32, device="cuda")
    mask_rows = i32([0, -1, 20])
    buf = dict(parents=i32(st.parents), bt=i32(st.bt), tokens=i32(d.tokens), u=torch.tensor(d.u).cuda(),
               last=torch.tensor(d.u_last).cuda(), target=d.target.clone(), draft=d.draft.clone(),
               q=st.qs.clone(), k=st.k.clone(), v=st.v.clone())
    cu, sk = i32(st.cu), i32(st.lens)
    out, lse = torch.empty_like(st.qs), torch.empty((st.T, 8), device="cuda")
    pos = torch.zeros(st.T, dtype=torch.int32, device="cuda")
    acc, path, new, lens = i32([0] * 3), i32([0] * st.T), i32([0] * st.T), i32([0] * 3)

    def calls():
        mcp.build_tree_masks(buf["parents"], cu, sk, mask_rows, mask, pos)
        mcp.mixed_attn_fwd_tree(plan, buf["q"], buf["k"], buf["v"], buf["bt"], cu, sk, mask, mask_rows, out, lse, ws)
        mcp.verify_drafts(buf["target"], buf["tokens"], cu, buf["u"], buf["last"], parents=buf["parents"],
                          draft_probs=buf["draft"], accepted=acc, path=path, new_tokens=new)
        mcp.kv_keep_path(buf["k"], buf["v"], buf["bt"], cu, sk, acc, path, new_lens=lens)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for gr in graphs:
        with torch.cuda.graph(gr):
            calls()
    for turn, seed in enumerate((2, 3, 4, 5)):
        st, d = fresh(seed)
        d.parents = st.parents
        for name, x in dict(parents=i32(st.parents), bt=i32(st.bt), tokens=i32(d.tokens), u=torch.tensor(d.u),
                            last=torch.tensor(d.u_last), target=d.target, draft=d.draft, q=st.qs, k=st.k,
                            v=st.v).items():
            buf[name].copy_(x)
        graphs[turn % 2].replay()
        torch.cuda.synchronize()
        st.compare(out, lse)
        for g, w in zip((acc, path, new), d.want()):
            assert g.tolist() == w.tolist()
        want = st.k.view(torch.int16).cpu().numpy()
        for s in range(3):
            ref.keep(want, st.bt[s], st.hist[s], path.tolist()[st.cu[s]:st.cu[s] + int(acc[s])], 16)
        assert (buf["k"].view(torch.int16).cpu().numpy() == want).all()
        assert lens.tolist() == [h + a for h, a in zip(st.hist, acc.tolist())]


def test_on_another_stream(mcp):
    """Results, and what a call takes for them, belong to the stream it is given."""
    d = Drafts([6] * 40, 30000, "fp32", "tree", True, seed=30)
    want = d.run(mcp)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = d.run(mcp, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    got = d.run(mcp, stream=side.cuda_stream)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_the_same_results_every_time(mcp):
    st = Step([(40, 3000, "tree")] * 3, 8, 2, 128, 16, seed=31)
    first = [x.clone() for x in st.run(mcp)]
    d = Drafts([9] * 20, 100000, "fp32", "star", True, seed=32)
    answers = [x.clone() for x in d.run(mcp)]
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(st.run(mcp), first))
        assert all(torch.equal(a, b) for a, b in zip(d.run(mcp), answers))
