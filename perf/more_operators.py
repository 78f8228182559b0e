"""The operators of a step that runs trees of drafted tokens, as cases to time and compare.

A request's segment holds its last token and a tree of tokens drafted behind it.

``masks``    which tokens of its tree each token sees, and its position, from the
             tokens' parents
``attn``     attention of a mixed step over the paged cache in which tree segments
             see their history and their own branch
``verify``   the path of a tree that the target's probabilities accept, and the token
             behind it, from given random numbers
``keep``     the accepted path's K/V moved behind the history, in every layer

``own`` False computes the plain form with elementary torch operations, True calls
the package's entry points.  Both take what ``prepare`` returns.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # four requests with small trees: latency
        dict(name="masks-4", op="masks", seqs=4, lo=12, hi=16, ctx_lo=100, ctx_hi=4096, chunks=0,
             chunk=0),
        # a large server's step: a thousand trees around four chunks of prompts
        dict(name="masks-1024", op="masks", seqs=1024, lo=48, hi=128, ctx_lo=64, ctx_hi=32768,
             chunks=4, chunk=2048),
        # one user's tree over a medium context: few rows, a long axis
        dict(name="attn-one", op="attn", seqs=1, lo=32, hi=32, ctx_lo=8192, ctx_hi=8192, hq=32,
             hkv=8, dim=128, page=16, chunks=0, chunk=0, lse=False),
        # a serving batch: trees and contexts of all lengths
        dict(name="attn-serve", op="attn", seqs=32, lo=16, hi=64, ctx_lo=1024, ctx_hi=16384, hq=32,
             hkv=8, dim=128, page=16, chunks=0, chunk=0, lse=True),
        # small trees beside two chunks of prompts with history
        dict(name="attn-mixed", op="attn", seqs=48, lo=2, hi=9, ctx_lo=1024, ctx_hi=8192, hq=64,
             hkv=8, dim=128, page=32, chunks=2, chunk=512, lse=False),
        # the largest batch: 64 trees of up to 64 tokens over long contexts
        dict(name="attn-long", op="attn", seqs=64, lo=33, hi=64, ctx_lo=4096, ctx_hi=32768, hq=32,
             hkv=8, dim=128, page=16, chunks=0, chunk=0, lse=False),
        # one user's chain of five drafts: latency
        dict(name="verify-one", op="verify", seqs=1, lo=6, hi=6, vocab=128000, dtype="fp32",
             shape="chain", draft=True),
        # a batch of chains from a draft model
        dict(name="verify-chains", op="verify", seqs=64, lo=4, hi=8, vocab=128000, dtype="fp32",
             shape="chain", draft=True),
        # trees whose branches were drawn from a draft model
        dict(name="verify-trees", op="verify", seqs=32, lo=16, hi=32, vocab=128000, dtype="fp32",
             shape="tree", draft=True),
        # trees of a draft model's likeliest tokens, probabilities in 16 bits, an odd vocabulary
        dict(name="verify-given", op="verify", seqs=256, lo=5, hi=12, vocab=50257, dtype="bf16",
             shape="tree", draft=False),
        # one request in 32 layers: launches
        dict(name="keep-one", op="keep", seqs=1, lo=32, hi=32, ctx_lo=300, ctx_hi=300, hkv=8,
             dim=128, page=16, layers=32),
        # a batch in 32 layers
        dict(name="keep-64", op="keep", seqs=64, lo=16, hi=64, ctx_lo=100, ctx_hi=500, hkv=8,
             dim=128, page=16, layers=32),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _span(rng, lo, hi):
    a, b = _log_int(rng, lo, hi), _log_int(rng, lo, hi)
    return min(a, b), max(a, b)


def draw(rng):
    op = rng.choice(["masks", "attn", "attn", "attn", "verify", "verify", "keep"])
    if op == "masks":
        seqs = _log_int(rng, 1, 1024)
        # at most the mask words of the largest listed case
        lo, hi = _span(rng, 1, min(1024, max(32 if seqs * 32 <= 360000 else 1,
                                             int((360000 * 32 / seqs) ** 0.5) - 32)))
        ctx_lo, ctx_hi = _span(rng, 1, 32768)
        return dict(op=op, seqs=seqs, lo=lo, hi=hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi,
                    chunks=rng.randint(0, 4), chunk=_log_int(rng, 2, 2048))
    if op == "attn":
        hkv = rng.choice([1, 2, 4, 8, 8])
        hq = hkv * rng.choice([g for g in (1, 2, 3, 4, 4, 7, 8) if g * hkv <= 64])
        dim = rng.choice([64, 96, 128, 128, 128, 256])
        seqs = _log_int(rng, 1, 64)
        lo, hi = _span(rng, 1, min(200, 4096 // seqs))
        # at most the cache and the products of the largest listed case
        room = min(64 * 18000 * 1024 // (hkv * dim), 64 * 49 * 18000 * 4096 // (hi * hq * dim))
        ctx_lo, ctx_hi = _span(rng, 1, max(2, min(32768, room // seqs)))
        return dict(op=op, seqs=seqs, lo=lo, hi=hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi, hq=hq, hkv=hkv,
                    dim=dim, page=rng.choice([1, 8, 16, 16, 32, 64]), chunks=rng.choice([0, 0, 1, 2]),
                    chunk=_log_int(rng, 2, 512), lse=rng.random() < 0.5)
    if op == "verify":
        vocab = _log_int(rng, 1000, 128000)
        draft = rng.random() < 0.6
        # at most the rows and the walks' ends of the largest listed cases
        seqs = _log_int(rng, 1, min(256, 64 * 128000 // vocab))
        lo, hi = _span(rng, 1, max(1, min(64, 1000 * 128000 // vocab // seqs)))
        return dict(op=op, seqs=seqs, lo=lo, hi=hi, vocab=vocab,
                    dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]),
                    shape=rng.choice(["chain", "tree"]), draft=draft)
    seqs = _log_int(rng, 1, 64)
    lo, hi = _span(rng, 1, 64)
    ctx_lo, ctx_hi = _span(rng, 1, 500)
    return dict(op=op, seqs=seqs, lo=lo, hi=hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi,
                hkv=rng.choice([1, 2, 4, 8]), dim=rng.choice([64, 96, 128]),
                page=rng.choice([1, 8, 16, 32, 64]), layers=_log_int(rng, 1, 32))


def _spread(n, lo, hi, step):
    """``n`` whole numbers spread over lo .. hi, the first the largest."""
    return [hi - int((i * step) % 1.0 * (hi - lo + 1)) for i in range(n)]


def _nodes(case):
    return _spread(case["seqs"], case["lo"], case["hi"], 0.6180339887)


def _history(case):
    """Tokens held by each tree's request, then by each chunk's."""
    ctx = _spread(case["seqs"], case["ctx_lo"], case["ctx_hi"], 0.7548776662)
    return ctx + [max(0, case["ctx_hi"] - case["chunk"])] * case["chunks"]


# ---------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _uniform(g, *shape):
    return torch.rand(shape, generator=g, device="cuda")


def _pack(bits):
    """[..., 32 n] truth values to [..., n] int32 words, bit 0 the first."""
    w = (bits.unflatten(-1, (-1, 32)).long() << torch.arange(32, device=bits.device)).sum(-1)
    return torch.where(w >= 2**31, w - 2**32, w).int()


def _trees(g, nodes, shape="tree"):
    """[len(nodes), most nodes] parents: a chain's, or each node under one before it."""
    n, S = max(nodes), len(nodes)
    i = torch.arange(n, device="cuda")
    if shape == "chain":
        return (i - 1).expand(S, n)
    up = (_uniform(g, S, n).double() * i).long()
    return torch.where(i > 0, torch.minimum(up, (i - 1).clamp(min=0)), -1)


def _visible(parents):
    """[S, n, n] truth values: token i sees token j of its tree."""
    S, n = parents.shape
    seen = torch.zeros((S, n, n), dtype=torch.bool, device="cuda")
    row = torch.arange(S, device="cuda")
    for i in range(n):
        p = parents[:, i]
        seen[:, i] = seen[row, p.clamp(min=0)] & (p >= 0)[:, None]
        seen[:, i, i] = True
    return seen


def _ragged(nodes):
    """(segment, place) of every token of the packed stream."""
    lens = torch.tensor(nodes, device="cuda")
    seg = torch.repeat_interleave(torch.arange(len(nodes), device="cuda"), lens)
    first = lens.cumsum(0) - lens
    return seg, torch.arange(len(seg), device="cuda") - first[seg], lens


def _step(case, g):
    """The segments of a step in a random order: trees and, where a case has them, chunks."""
    trees = _nodes(case)
    lens, hist = trees + [case["chunk"]] * case["chunks"], _history(case)
    order = torch.randperm(len(lens), generator=g, device="cuda").cpu().tolist()
    q, h = [lens[i] for i in order], [hist[i] for i in order]
    tree = [i < len(trees) for i in order]
    at = [0]
    for n, t in zip(q, tree):
        at.append(at[-1] + (n if t else 0))
    q_d = torch.tensor(q, device="cuda")
    cu = torch.nn.functional.pad(q_d.cumsum(0), (1, 0)).int()
    sk = (q_d + torch.tensor(h, device="cuda")).int()
    s = dict(op=case["op"], q=q, hist=h, tree=tree, cu=cu, sk=sk, rows=at[-1],
             words=-(-max(trees) // 32),
             mask_rows=torch.tensor([a if t else -1 for a, t in zip(at, tree)], dtype=torch.int32,
                                    device="cuda"))
    parents = _trees(g, trees)
    seg, place, _ = _ragged(q)
    which = torch.tensor([i if i < len(trees) else 0 for i in order], device="cuda")
    live = torch.tensor(tree, device="cuda")[seg]
    col = place.clamp(max=parents.shape[1] - 1)
    s["parents"] = torch.where(live, parents[which[seg], col], place - 1).int()
    return s, parents, which, seg, place, live


def _prepare_masks(case, g):
    s = _step(case, g)[0]
    s["mask"] = torch.zeros((s["rows"], s["words"]), dtype=torch.int32, device="cuda")
    s["positions"] = torch.zeros(sum(s["q"]), dtype=torch.int32, device="cuda")
    return s


def _tables(g, lens, page):
    """Block tables over a shuffled pool for requests of ``lens`` tokens, -1 behind."""
    held = [-(-n // page) for n in lens]
    pages = sum(held) + 5
    perm = torch.randperm(pages, generator=g, device="cuda").int()
    seg, place, _ = _ragged(held)
    bt = torch.full((len(lens), max(held)), -1, dtype=torch.int32, device="cuda")
    bt[seg, place] = perm[: len(seg)]
    return bt, pages


def _prepare_attn(case, g):
    s, parents, which, seg, place, live = _step(case, g)
    n = parents.shape[1]
    mask = torch.nn.functional.pad(_visible(parents), (0, 32 * s["words"] - n))
    s["mask"] = _pack(mask[which[seg[live]], place[live]])
    lens = [a + b for a, b in zip(s["q"], s["hist"])]
    P, H, D, T = case["page"], case["hkv"], case["dim"], sum(s["q"])
    s["bt"], pages = _tables(g, lens, P)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)

    s.update(q_rows=normal(T, case["hq"], D), k=normal(pages, P, H, D), v=normal(pages, P, H, D),
             scale=D ** -0.5, hq=case["hq"], hkv=H, dim=D, page=P,
             out=torch.zeros((T, case["hq"], D), dtype=torch.bfloat16, device="cuda"),
             lse=torch.zeros((T, case["hq"]), device="cuda") if case["lse"] else None)
    if own:  # the plan of the step, which its layers share
        import mixed_chunked_prefill_gb300 as mcp

        desc = mcp.make_desc(len(lens), T, case["hq"], H, D, P, s["bt"].shape[1], pages, s["scale"])
        cu, sk, options = s["cu"].cpu().numpy(), s["sk"].cpu().numpy(), mcp.PlanOptions(tree=1)
        sizing = mcp.mixed_attn_plan(desc, cu, sk, options)
        s["workspace"] = torch.empty(max(256, sizing.workspace_bytes), dtype=torch.uint8,
                                     device="cuda")
        s["plan"] = mcp.mixed_attn_plan(desc, cu, sk, options, s["workspace"])
    return s


def _prepare_verify(case, g):
    nodes, V, dt = _nodes(case), case["vocab"], DTYPES[case["dtype"]]
    parents = _trees(g, nodes, case["shape"])
    seg, place, lens = _ragged(nodes)
    R = len(seg)
    first = lens.cumsum(0) - lens
    up = parents[seg, place]
    target = torch.empty((R, V), dtype=dt, device="cuda")
    draft = torch.empty((R, V), dtype=dt, device="cuda") if case["draft"] else None
    tokens = torch.zeros(R, dtype=torch.int32, device="cuda")
    step = max(1, (1 << 25) // V)
    # peaked rows as a model has them; the draft model's are the same with noise
    for a in range(0, R, step):
        z = torch.randn((min(step, R - a), V), generator=g, device="cuda") * 3
        target[a:a + step] = torch.softmax(z, 1).to(dt)
        if draft is not None:
            z += torch.randn(z.shape, generator=g, device="cuda") * 0.7
            draft[a:a + step] = torch.softmax(z, 1).to(dt)
    # a node's token: drawn from its parent's draft row, else one of the parent's likeliest
    kids = (first[seg] + up.clamp(min=0)).long()
    rank = torch.zeros(R, dtype=torch.int64, device="cuda")
    same = (kids[:, None] == kids) & (place > 0)
    rank = torch.tril(same, -1).sum(1)
    for a in range(0, R, step):
        k = kids[a:a + step]
        if draft is not None:
            e = -torch.log(1 - _uniform(g, len(k), V))
            tokens[a:a + step] = (draft[k].float() / e.clamp(min=1e-20)).argmax(1).int()
        else:
            top = target[k].topk(min(V, 64), dim=1).indices
            tokens[a:a + step] = top.gather(1, rank[a:a + step, None].clamp(max=top.shape[1] - 1))[:, 0].int()
    return dict(op="verify", target=target, draft=draft, tokens=tokens, nodes=max(nodes),
                parents=up.int().contiguous() if case["shape"] == "tree" else None,
                cu=torch.nn.functional.pad(lens.cumsum(0), (1, 0)).int(),
                u=_uniform(g, R), u_last=_uniform(g, len(nodes)))


def _kept(case):
    """Accepted tokens of each tree."""
    return [min(n, 1 + (3 + 5 * i) % 7) for i, n in enumerate(_nodes(case))]


def _prepare_keep(case, g):
    q, P, H, D = _nodes(case), case["page"], case["hkv"], case["dim"]
    hist = _spread(case["seqs"], case["ctx_lo"], case["ctx_hi"], 0.7548776662)
    bt, pages = _tables(g, [a + b for a, b in zip(q, hist)], P)
    seg, place, lens = _ragged(q)
    kept = torch.tensor(_kept(case), device="cuda")
    # a path: the root and some of the tokens behind it, in order
    n = max(q)
    order = _uniform(g, len(q), n)
    order[:, 0] = -1
    i = torch.arange(n, device="cuda")
    order = order.masked_fill(i >= lens[:, None], 2)
    chosen = order.argsort(1).argsort(1) < kept[:, None]
    path = torch.where(chosen, i, n).sort(1).values
    path = torch.where(i < kept[:, None], path, -1)

    def caches():  # of all layers
        return torch.randn((case["layers"], pages, P, H, D), generator=g, device="cuda",
                           dtype=torch.bfloat16)

    return dict(op="keep", k=caches(), v=caches(), bt=bt, accepted=kept.int(),
                path=path[seg, place].int(), page=P,
                cu=torch.nn.functional.pad(lens.cumsum(0), (1, 0)).int(),
                sk=(lens + torch.tensor(hist, device="cuda")).int(),
                new_lens=torch.zeros(len(q), dtype=torch.int32, device="cuda"))


def prepare(case, seed):
    return {"masks": _prepare_masks, "attn": _prepare_attn, "verify": _prepare_verify,
            "keep": _prepare_keep}[case["op"]](case, _gen(seed))


# ------------------------------------------------------------------------- plain forms
def _plain_masks(s):
    """The parents' rows are taken over by doubling: after k rounds a row reaches 2^k up."""
    cu, T = s["cu"].long(), len(s["parents"])
    t = torch.arange(T, device="cuda")
    seg = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    place = t - cu[seg]
    at = s["mask_rows"].long()[seg]
    tree = at >= 0
    own_row = torch.where(tree, at + place, 0)[tree]
    up = s["parents"].long()[tree]
    up = torch.where(up >= 0, own_row - place[tree] + up, -1)  # rows of the parents
    rows, n = s["rows"], 32 * s["words"]
    up = torch.full((rows,), -1, device="cuda").scatter_(0, own_row, up)
    col = torch.zeros(rows, dtype=torch.int64, device="cuda").scatter_(0, own_row, place[tree])
    bits = torch.zeros((rows, n), dtype=torch.bool, device="cuda")
    bits[torch.arange(rows, device="cuda"), col] = True
    depth = (up >= 0).long()
    for _ in range(max(1, (n - 1).bit_length())):
        on = up >= 0
        above = up.clamp(min=0)
        bits |= bits[above] & on[:, None]
        depth += torch.where(on, depth[above], 0)
        up = torch.where(on, up[above], -1)
    s["mask"].copy_(_pack(bits))
    hist = (s["sk"].long() - cu[1:] + cu[:-1])[seg]
    place[tree] = depth[own_row]
    s["positions"].copy_(hist + place)
    return dict(mask=s["mask"], positions=s["positions"])


def _segment_bits(s, i, n):
    """[n, n] truth values: which of its segment's tokens each token sees."""
    if not s["tree"][i]:
        return torch.tril(torch.ones((n, n), dtype=torch.bool, device="cuda"))
    a = sum(q for q, t in zip(s["q"][:i], s["tree"]) if t)
    w = s["mask"][a:a + n].long()
    return ((w[:, :, None] >> torch.arange(32, device="cuda")) & 1).flatten(1)[:, :n] != 0


def _attend(s, dtype, outs):
    """Segment after segment in ``dtype``."""
    G, at = s["hq"] // s["hkv"], 0
    for i, (n, h) in enumerate(zip(s["q"], s["hist"])):
        held = -(-(n + h) // s["page"])
        pages = s["bt"][i, :held].long()
        k, v = (c[pages].flatten(0, 1)[:n + h].to(dtype).transpose(0, 1) for c in (s["k"], s["v"]))
        q = s["q_rows"][at:at + n].to(dtype).unflatten(1, (s["hkv"], G)).permute(1, 2, 0, 3)
        x = torch.matmul(q.flatten(1, 2), k.transpose(1, 2)).unflatten(1, (G, n)) * s["scale"]
        x[..., h:] = x[..., h:].masked_fill(~_segment_bits(s, i, n), -math.inf)
        m = x.amax(-1, keepdim=True)
        x = torch.exp(x - m)
        l = x.sum(-1, keepdim=True)
        y = torch.matmul(x.flatten(1, 2), v).unflatten(1, (G, n)) / l
        outs[0][at:at + n] = y.permute(2, 0, 1, 3).flatten(1, 2).to(outs[0].dtype)
        if outs[1] is not None:
            outs[1][at:at + n] = (m + torch.log(l))[..., 0].permute(2, 0, 1).flatten(1, 2)
        at += n
    return [o for o in outs if o is not None]


def _plain_verify(s):
    """Node after node over all requests at once; rows in 64 bits, because a token lies
    between two of the row's sums."""
    cu = s["cu"].long()
    first, n = cu[:-1], cu[1:] - cu[:-1]
    S, (R, V) = len(first), s["target"].shape
    seg = torch.arange(S, device="cuda")
    tokens, u = s["tokens"].long(), s["u"].double()
    cur = torch.zeros_like(first)
    c = torch.zeros(S, dtype=torch.float64, device="cuda")
    mass = torch.ones(S, dtype=torch.float64, device="cuda")
    kept = torch.ones_like(first)
    path = torch.full((R + 1,), -1, dtype=torch.int64, device="cuda")
    new = path.clone()
    path[first] = 0
    gone = None if s["draft"] is not None else torch.zeros((S, V), dtype=torch.bool, device="cuda")
    for i in range(1, s["nodes"]):
        r = (first + i).clamp(max=R - 1)
        up = torch.full_like(first, i - 1) if s["parents"] is None else s["parents"].long()[r]
        here = (i < n) & (up == cur)
        x, row = tokens[r], first + cur
        p = s["target"][row, x].double()
        if s["draft"] is not None:
            q = s["draft"][row, x].double()
            ok = here & (u[r] * mass * q < p - c * q)
        else:
            p = torch.where(gone[seg, x], 0, p)
            ok = here & (u[r] * mass < p)
        no = here & ~ok
        path[torch.where(ok, first + kept, R)] = i
        new[torch.where(ok, first + kept - 1, R)] = x
        kept += ok
        if s["draft"] is not None:
            c = torch.where(no, c + mass, c)
            rest = (s["target"][row].double() - c[:, None] * s["draft"][row].double()).clamp(min=0).sum(1)
            mass = torch.where(no, rest, mass)
        else:
            gone[seg, x] |= no
            mass = torch.where(no, (mass - p).clamp(min=0), mass)
            gone &= ~ok[:, None]
        cur = torch.where(ok, i, cur)
        c, mass = torch.where(ok, 0, c), torch.where(ok, 1, mass)
    p = s["target"][first + cur].double()
    if s["draft"] is not None:
        w = (p - c[:, None] * s["draft"][first + cur].double()).clamp(min=0)
    else:
        w = torch.where(gone, 0, p)
    w = torch.where(w.sum(1, keepdim=True) > 0, w, p)
    sums = w.cumsum(1)
    at = torch.searchsorted(sums, (s["u_last"].double() * sums[:, -1])[:, None], right=True)[:, 0]
    last = V - 1 - (w > 0).flip(1).int().argmax(1)
    new[first + kept - 1] = torch.minimum(at, last)
    return dict(accepted=kept.int(), path=path[:R].int(), new=new[:R].int())


def _plain_keep(s):
    cu, sk, P = s["cu"].long(), s["sk"].long(), s["page"]
    t = torch.arange(len(s["path"]), device="cuda")
    seg = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    k, hist = t - cu[seg], sk - cu[1:] + cu[:-1]
    on = (k < s["accepted"].long()[seg]).nonzero()[:, 0]
    seg, k, src = seg[on], k[on], s["path"].long()[on]

    def slot(pos):
        return s["bt"][seg, pos // P].long() * P + pos % P

    a, b = slot(hist[seg] + src), slot(hist[seg] + k)
    for caches in (s["k"], s["v"]):
        for cache in caches:
            flat = cache.flatten(0, 1)
            flat[b] = flat[a]
    s["new_lens"].copy_(hist + s["accepted"])
    return dict(k=s["k"], v=s["v"], new_lens=s["new_lens"])


# ------------------------------------------------------------------------ this package
def _run_own(s):
    import mixed_chunked_prefill_gb300 as mcp

    op = s["op"]
    if op == "masks":
        mcp.build_tree_masks(s["parents"], s["cu"], s["sk"], s["mask_rows"], s["mask"],
                             s["positions"])
        return dict(mask=s["mask"], positions=s["positions"])
    if op == "attn":
        mcp.mixed_attn_fwd_tree(s["plan"], s["q_rows"], s["k"], s["v"], s["bt"], s["cu"], s["sk"],
                                s["mask"], s["mask_rows"], s["out"], s["lse"], s["workspace"])
        return [s["out"]] if s["lse"] is None else [s["out"], s["lse"]]
    if op == "verify":
        accepted, path, new = mcp.verify_drafts(s["target"], s["tokens"], s["cu"], s["u"],
                                                s["u_last"], parents=s["parents"],
                                                draft_probs=s["draft"])
        return dict(accepted=accepted, path=path, new=new)
    mcp.kv_keep_path(s["k"], s["v"], s["bt"], s["cu"], s["sk"], s["accepted"], s["path"],
                     new_lens=s["new_lens"])
    return dict(k=s["k"], v=s["v"], new_lens=s["new_lens"])


def run(state):
    if own:
        return _run_own(state)
    if state["op"] == "attn":
        return _attend(state, torch.float32, [state["out"], state["lse"]])
    return {"masks": _plain_masks, "verify": _plain_verify, "keep": _plain_keep}[state["op"]](state)


# ------------------------------------------------------------------------------- work
def work(case):
    nodes, S = _nodes(case), case["seqs"]
    op = case["op"]
    if op == "masks":
        tree, words = sum(nodes), -(-max(nodes) // 32)
        T, n = tree + case["chunks"] * case["chunk"], S + case["chunks"]
        # the trees' parents and the segments read, masks and positions written
        return {"bytes": 4 * tree + 12 * n + 4 * words * tree + 4 * T, "flops": 0}
    if op == "attn":
        q = nodes + [case["chunk"]] * case["chunks"]
        hist = _history(case)
        T, words = sum(q), -(-max(nodes) // 32)
        keys = sum(a + b for a, b in zip(q, hist))
        row = case["hkv"] * case["dim"]
        # K and V once, queries and outputs, masks and tables
        b = 4 * keys * row + 4 * T * case["hq"] * case["dim"] + 4 * words * sum(nodes)
        b += 4 * keys / case["page"] + 12 * len(q) + (4 * T * case["hq"] if case["lse"] else 0)
        # pairs: the history and the token itself, half of a chunk's own tokens
        pairs = sum(n * (h + 1) for n, h in zip(q, hist)) + case["chunks"] * case["chunk"] ** 2 / 2
        return {"bytes": b, "flops": 4.0 * pairs * case["hq"] * case["dim"]}
    if op == "verify":
        size = 4 if case["dtype"] == "fp32" else 2
        # the row at which each walk ends, the nodes' numbers and the answers
        b = S * case["vocab"] * size * (2 if case["draft"] else 1) + sum(nodes) * (20 + 2 * size) + 12 * S
        return {"bytes": b, "flops": 2.0 * S * case["vocab"]}
    moved = sum(a - 1 for a in _kept(case))
    return {"bytes": 8 * moved * case["layers"] * case["hkv"] * case["dim"] + 8 * sum(nodes) + 16 * S,
            "flops": 0}


# ------------------------------------------------------------------------------ exact
def exact(case, seed):
    """The attention in 64 bits, each token's hidden keys picked out one by one, and the
    caches after their moves; masks and paths are whole numbers."""
    if case["op"] == "keep":
        s = prepare(case, seed)
        cu, path, P = s["cu"].tolist(), s["path"].tolist(), s["page"]
        accepted, bt = s["accepted"].tolist(), s["bt"].tolist()
        lens = []
        for i, kept in enumerate(accepted):
            hist = int(s["sk"][i]) - (cu[i + 1] - cu[i])
            lens.append(hist + kept)
            for k in range(kept):  # a path's places rise: none is overwritten before it is read
                a, b = hist + path[cu[i] + k], hist + k
                for cache in (s["k"], s["v"]):
                    cache[:, bt[i][b // P], b % P] = cache[:, bt[i][a // P], a % P]
        return dict(k=s["k"].double(), v=s["v"].double(), new_lens=torch.tensor(lens))
    if case["op"] != "attn":
        return None
    if work(case)["flops"] > 5e12:
        return None
    s = prepare(case, seed)
    G, T = s["hq"] // s["hkv"], len(s["q_rows"])
    out = torch.empty((T, s["hq"], s["dim"]), dtype=torch.float64, device="cuda")
    lse = torch.empty((T, s["hq"]), dtype=torch.float64, device="cuda")
    t, row = 0, 0
    for i, (n, h) in enumerate(zip(s["q"], s["hist"])):
        pos = torch.arange(n + h, device="cuda")
        page, off = s["bt"][i].long()[pos // s["page"]], pos % s["page"]
        k, v = s["k"][page, off].double(), s["v"][page, off].double()
        words = s["mask"][row:row + n].cpu().tolist() if s["tree"][i] else None
        row += n if s["tree"][i] else 0
        for head in range(s["hkv"]):
            q = s["q_rows"][t:t + n, head * G:(head + 1) * G].double()
            x = torch.einsum("ngd,kd->ngk", q, k[:, head]) * s["scale"]
            for a in range(n):
                hidden = range(a + 1, n) if words is None else [
                    b for b in range(n) if not words[a][b // 32] >> (b % 32) & 1]
                if len(hidden):
                    x[a, :, torch.tensor(list(hidden), device="cuda") + h] = -math.inf
            lse[t:t + n, head * G:(head + 1) * G] = torch.logsumexp(x, -1)
            out[t:t + n, head * G:(head + 1) * G] = torch.einsum("ngk,kd->ngd", torch.softmax(x, -1),
                                                                 v[:, head])
        t += n
    return [out] if s["lse"] is None else [out, lse]
