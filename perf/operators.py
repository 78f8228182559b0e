"""The operators around the attention of a serving step, as cases to time and compare.

State of each request lives on the GPU next to its KV pages, and the operators
that read and update it are measured here:

``tables``   block tables, slot map, positions and sampled rows of a step, built
             from request lengths, with pages taken from a free list
``oneshot``  the same for requests that end with their prompt: build, then commit
             with every page given back
``conv``     the short causal convolution of a recurrent layer over the packed
             stream, with each request's last inputs kept between steps
``scan``     the selective state space scan that follows it, with each request's
             state kept between steps
``counts``   which tokens a request has had (prompt marks, output counts)
``logits``   biases, penalties for repeated tokens, temperature and grammar masks

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
        # a large server's captured step: 1024 segments, eight of them padding
        dict(name="tables-wide", op="tables", seqs=1024, chunks=16, chunk=512, pad=8,
             ctx_lo=64, ctx_hi=32768, page=16),
        # a handful of prompts that are only scored and end at once: latency
        dict(name="oneshot-8", op="oneshot", seqs=8, prompt=512, page=16),
        # a batch job's scored prompts, 8-token pages: many pages given back together
        dict(name="oneshot-512", op="oneshot", seqs=512, prompt=2048, page=8),
        # one token each for 256 decodes of a wide layer
        dict(name="conv-decode", op="conv", decodes=256, lens="", channels=8192, width=4,
             dtype="bf16", silu=True, pad=0),
        # 64 decodes around a 2048-token chunk with history
        dict(name="conv-chunk", op="conv", decodes=64, lens="2048h", channels=8192, width=4,
             dtype="bf16", silu=True, pad=0),
        # the same 256 decodes: every request's state is read and written once
        dict(name="scan-decode", op="scan", decodes=256, lens="", channels=8192, states=16,
             groups=1, dtype="bf16", gate=True, softplus=True, pad=0),
        # two decodes and a 1808-token chunk after a long history
        dict(name="scan-chunk", op="scan", decodes=2, lens="1808h", channels=4096, states=16,
             groups=1, dtype="fp16", gate=True, softplus=True, pad=0),
        # whole prompts of different lengths, packed
        dict(name="scan-prompts", op="scan", decodes=0, lens="2048 1777 1500 1111 900 511 257 88",
             channels=8192, states=16, groups=1, dtype="bf16", gate=True, softplus=True, pad=0),
        # one sampled token each for a decode batch (some rows are padding)
        dict(name="counts-decode", op="counts", requests=256, rows=250, pad=6, vocab=128000,
             prompt=0, output=1, reset=False),
        # requests re-admitted after preemption: rows cleared, prompts and outputs counted again
        dict(name="counts-admit", op="counts", requests=64, rows=64, pad=0, vocab=128000,
             prompt=32768, output=4096, reset=True),
        # greedy decoding of 64 rows in place: no temperature, half the rows under a grammar
        dict(name="logits-greedy", op="logits", rows=64, vocab=128000, dtype="bf16", out="bf16",
             history=2000, bias=16, mask="half", temperature=False, inplace=True),
        # the largest batch: bf16 logits to the sampler's fp32, everything on
        dict(name="logits-512", op="logits", rows=512, vocab=128000, dtype="bf16", out="fp32",
             history=2000, bias=16, mask="half", temperature=True, inplace=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "oneshot", "conv", "scan", "scan", "counts", "logits", "logits"])
    if op == "tables":
        page = rng.choice([1, 8, 16, 16, 32, 64])
        seqs = _log_int(rng, 1, 1024)
        # at most the page table of the largest listed case
        ctx_hi = _log_int(rng, 64, max(64, min(131072, 8_000_000 * page // seqs)))
        chunks = rng.randint(0, min(seqs, 16))
        return dict(op=op, seqs=seqs, chunks=chunks, chunk=_log_int(rng, 2, 2048),
                    pad=rng.randint(0, 9), ctx_lo=_log_int(rng, 1, ctx_hi), ctx_hi=ctx_hi, page=page)
    if op == "oneshot":
        return dict(op=op, seqs=_log_int(rng, 1, 512), prompt=_log_int(rng, 1, 2048),
                    page=rng.choice([8, 16, 32, 64]))
    if op == "counts":
        requests = _log_int(rng, 1, 256)
        rows = rng.randint(1, requests)
        reset = rng.random() < 0.5
        cap = max(1, 2_000_000 // rows)
        return dict(op=op, requests=requests, rows=rows, pad=rng.randint(0, 9),
                    vocab=_log_int(rng, 1000, 128000),
                    prompt=_log_int(rng, 1, min(32768, cap)) if reset else 0,
                    output=_log_int(rng, 1, min(4096, cap)), reset=reset)
    if op in ("conv", "scan"):
        channels = 8 * _log_int(rng, 8, 1024)
        states = rng.choice([8, 16, 16, 32, 64])
        room = 8192 * 8192 // channels // (max(1, states // 16) if op == "scan" else 1)
        decodes = min(256, room // 8, _log_int(rng, 1, 256)) if rng.random() < 0.7 else 0
        lens, left = [], room - decodes
        for _ in range(rng.randint(0 if decodes else 1, 4)):
            n = _log_int(rng, 1, max(1, min(2048, left // 4)))
            lens.append("%d%s" % (n, rng.choice(["", "h"])))
        case = dict(op=op, decodes=decodes, lens=" ".join(lens), channels=channels,
                    dtype=rng.choice(["bf16", "bf16", "fp16"]), pad=rng.randint(0, 9))
        if op == "conv":
            return dict(case, width=rng.choice([2, 3, 4, 4]), silu=rng.random() < 0.8)
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if channels % (32 * g) == 0 or g == 1])
        return dict(case, states=states, groups=groups, gate=rng.random() < 0.8,
                    softplus=rng.random() < 0.8)
    inplace = rng.random() < 0.4
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    return dict(op=op, rows=_log_int(rng, 1, 256), vocab=_log_int(rng, 1000, 128000), dtype=dtype,
                out=dtype if inplace or rng.random() < 0.5 else "fp32",
                history=_log_int(rng, 1, 8192), bias=rng.choice([0, 1, 7, 16, 100]),
                mask=rng.choice(["none", "half", "all"]), temperature=rng.random() < 0.6,
                inplace=inplace)


# ---------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randint(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int64)


def _width(case):
    """Pages of the longest request that a case can have."""
    if case["op"] == "oneshot":
        return -(-case["prompt"] // case["page"])
    more = case["chunk"] if case["chunks"] else 1
    return -(-(case["ctx_hi"] - 1 + more) // case["page"])


def _pages_state(case, g, have, q, cap, pad):
    """Page tables and free list for requests holding ``have`` tokens, at rows given
    by a random permutation; the step's ids with ``pad`` padding entries between."""
    dev, P, n, width = "cuda", case["page"], int(have.numel()), _width(case)
    held = (have + P - 1) // P
    num_pages = n * width + 17
    perm = torch.randperm(num_pages, generator=g, device=dev).int()
    rows = torch.randperm(n, generator=g, device=dev)
    j = torch.arange(width, device=dev)
    first = held.cumsum(0) - held
    held_pages = torch.where(j < held[:, None], perm[(first[:, None] + j).clamp(max=num_pages - 1)], -1)
    request_pages = torch.full((n + 1, width), -1, dtype=torch.int32, device=dev)
    request_pages[rows] = held_pages
    lens = torch.zeros(n + 1, dtype=torch.int32, device=dev)
    lens[rows] = have.int()
    taken = int(held.sum())
    free = torch.full((num_pages,), -1, dtype=torch.int32, device=dev)
    free[: num_pages - taken] = perm[taken:]
    ids = torch.full((n + pad,), -1, dtype=torch.int32, device=dev)
    q_lens = torch.zeros(n + pad, dtype=torch.int32, device=dev)
    at = torch.randperm(n + pad, generator=g, device=dev)[:n].sort().values
    ids[at], q_lens[at] = rows.int(), q.int()
    S = n + pad
    s = dict(op=case["op"], P=P, request_pages=request_pages, request_lens=lens, free_pages=free,
             free_count=torch.tensor([num_pages - taken], dtype=torch.int32, device=dev),
             ids=ids, q=q_lens, cap=cap,
             cu=torch.empty(S + 1, dtype=torch.int32, device=dev),
             sk=torch.empty(S, dtype=torch.int32, device=dev),
             bt=torch.empty((S, width), dtype=torch.int32, device=dev),
             slots=torch.empty(cap, dtype=torch.int64, device=dev),
             pos=torch.empty(cap, dtype=torch.int32, device=dev),
             rows=torch.empty(S, dtype=torch.int32, device=dev))
    if own:  # the handle on the pool, which a program makes once with its tensors
        import mixed_chunked_prefill_gb300 as mcp

        s["pool"] = mcp.make_request_pool(request_pages, lens, free, s["free_count"], P)
    return s


def _tokens(g, n, vocab):
    """Token ids as text has them: a few very often, most of them hardly ever."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    return ((vocab + 1.0) ** u - 1).long().clamp(max=vocab - 1)


def _pack(bits):
    """[..., 32 n] truth values to [..., n] int32 words, token 0 in the lowest bit."""
    w = bits.unflatten(-1, (-1, 32)).long() << torch.arange(32, device=bits.device)
    w = w.sum(-1)
    return torch.where(w >= 2**31, w - 2**32, w).int()


def _token_state(g, requests, vocab, prompt, output):
    """(seen [requests, 2, words], counts [requests, 32 words]) of requests with
    ``prompt`` prompt tokens and ``output`` sampled ones each."""
    words = -(-vocab // 32)
    counts = torch.zeros((requests, 32 * words), dtype=torch.int32, device="cuda")
    marks = torch.zeros((requests, 32 * words), dtype=torch.bool, device="cuda")
    row = torch.arange(requests, device="cuda")[:, None]
    if prompt:
        marks[row, _tokens(g, requests * prompt, vocab).view(requests, prompt)] = True
    if output:
        t = _tokens(g, requests * output, vocab).view(requests, output)
        counts.scatter_add_(1, t, torch.ones_like(t, dtype=torch.int32))
    seen = torch.empty((requests, 2, words), dtype=torch.int32, device="cuda")
    for r in range(0, requests, 64):  # packing goes through 8 bytes a token
        seen[r:r + 64, 0], seen[r:r + 64, 1] = _pack(marks[r:r + 64]), _pack(counts[r:r + 64] > 0)
    return seen, counts


def _stream(case, g):
    """A packed stream: decodes with history among whole prompts and chunks ("h": with
    history).  ``rows`` more tokens than the last segment ends at stand behind it."""
    lens = [(1, True)] * case["decodes"]
    lens += [(int(w.rstrip("h")), w.endswith("h")) for w in case["lens"].split()]
    n, pad = len(lens), case["pad"]
    order = torch.randperm(n, generator=g, device="cuda").cpu().tolist()
    q = torch.tensor([lens[i][0] for i in order] + [0] * pad)
    hist = torch.tensor([1000 + 7 * i if lens[i][1] else 0 for i in order] + [0] * pad)
    rows = torch.randperm(n + 2, generator=g, device="cuda")[:n].int()
    return dict(op=case["op"], lens=q.tolist(), tokens=int(q.sum()) + pad,
                cu=torch.nn.functional.pad(q.cumsum(0), (1, 0)).int().cuda(),
                sk=(q + hist).int().cuda(), requests=n + 2,
                ids=torch.nn.functional.pad(rows, (0, pad), value=-1))


def _prepare_recurrent(case, g):
    s = _stream(case, g)
    T, d, dt, R = s["tokens"], case["channels"], DTYPES[case["dtype"]], s["requests"]

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device="cuda") * scale

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo

    # x is the first half of the input projection's rows, the gate the second
    xz = normal(T, 2 * d).to(dt)
    s.update(x=xz[:, :d], out=torch.zeros((T, d), dtype=dt, device="cuda"))
    if case["op"] == "conv":
        K = case["width"]
        s.update(weight=normal(d, K, scale=K ** -0.5).to(dt), bias=normal(d, scale=0.1).to(dt),
                 silu=case["silu"], state=normal(R, K - 1, d).to(dt))
        return s
    N, G = case["states"], case["groups"]
    # steps of 0.001 to 0.1 through softplus, decay rates 1 .. N: slow and fast states
    step = torch.exp(uniform(math.log(1e-3), math.log(1e-1), d))
    s["A"] = -(torch.arange(1, N + 1, device="cuda", dtype=torch.float32)
               * uniform(0.9, 1.1, d, N)).contiguous()
    s["D"] = uniform(0.5, 1.5, d)
    s["softplus"] = case["softplus"]
    if case["softplus"]:
        s["dt"] = normal(T, d, scale=0.5).to(dt)
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    else:
        s["dt"], s["dt_bias"] = (step * uniform(0.5, 1.5, T, d)).to(dt), None
    bc = normal(T, 2 * G * N).to(dt)  # one projection gives both
    s["B"], s["C"] = bc[:, :G * N].unflatten(1, (G, N)), bc[:, G * N:].unflatten(1, (G, N))
    s["z"] = xz[:, d:] if case["gate"] else None
    s["state"] = normal(R, d, N, scale=0.3)
    return s


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op in ("conv", "scan"):
        return _prepare_recurrent(case, g)
    if op == "tables":
        n = case["seqs"]
        have = _randint(g, case["ctx_lo"], case["ctx_hi"], n) - 1
        q = torch.ones(n, dtype=torch.int64, device="cuda")
        if case["chunks"]:
            at = torch.randperm(n, generator=g, device="cuda")[: case["chunks"]]
            q[at] = case["chunk"]
        tokens = n + case["chunks"] * (case["chunk"] - 1)
        return _pages_state(case, g, have, q, -(-tokens // 64) * 64, case["pad"])
    if op == "oneshot":
        n = case["seqs"]
        s = _pages_state(case, g, torch.zeros(n, dtype=torch.int64, device="cuda"),
                         _randint(g, 1, case["prompt"], n), n * case["prompt"], 0)
        s["new_lens"] = torch.zeros(n, dtype=torch.int32, device="cuda")
        return s
    if op == "counts":
        R, n, vocab = case["requests"], case["rows"], case["vocab"]
        seen, counts = _token_state(g, R, vocab, 300, 200)
        ids = torch.full((n + case["pad"],), -1, dtype=torch.int32, device="cuda")
        at = torch.randperm(n + case["pad"], generator=g, device="cuda")[:n].sort().values
        ids[at] = torch.randperm(R, generator=g, device="cuda")[:n].int()
        s = dict(op=op, vocab=vocab, seen=seen, counts=counts, ids=ids, reset=case["reset"])
        for what in ("prompt", "output"):
            if not case[what]:
                continue
            lens = torch.zeros(n + case["pad"], dtype=torch.int64, device="cuda")
            lens[at] = _randint(g, max(1, case[what] // 2), case[what], n)
            s["cu_" + what] = torch.nn.functional.pad(lens.cumsum(0), (1, 0)).int()
            s[what] = _tokens(g, int(lens.sum()), vocab).int()
        return s
    B, V, dt = case["rows"], case["vocab"], DTYPES[case["dtype"]]
    R = B + 3
    seen, counts = _token_state(g, R, V, case["history"], max(1, case["history"] // 4))
    def uniform(lo, hi):
        return torch.rand(B, generator=g, device="cuda") * (hi - lo) + lo

    s = dict(op=op, V=V, seen=seen, counts=counts, inplace=case["inplace"],
             out=DTYPES[case["out"]],
             logits=(torch.randn((B, V), generator=g, device="cuda") * 4).to(dt),
             ids=torch.randperm(R, generator=g, device="cuda")[:B].int(),
             repetition=uniform(1.0, 1.5), frequency=uniform(0.0, 1.0), presence=uniform(0.0, 1.0),
             temperature=uniform(0.2, 1.8) if case["temperature"] else None,
             bias=None, mask=None, mask_rows=None)
    if case["bias"]:  # each row biases its own tokens, in rising order
        k = min(case["bias"], V // 2)
        step = V // k
        tok = torch.arange(k, device="cuda") * step + torch.randint(
            0, step, (B, k), generator=g, device="cuda")
        s["bias"] = (torch.arange(B + 1, device="cuda", dtype=torch.int32) * k,
                     tok.reshape(-1).int(),
                     torch.randn(B * k, generator=g, device="cuda") * 5)
    if case["mask"] != "none":  # a grammar allows a small part of the tokens
        n = B if case["mask"] == "all" else max(1, B // 2)
        words = -(-V // 32)
        m = torch.empty((n, words), dtype=torch.int32, device="cuda")
        for r in range(0, n, 64):
            part = torch.rand((min(64, n - r), 32 * words), generator=g, device="cuda")
            m[r:r + 64] = _pack(part < 0.02)
        s["mask"] = m
        if n < B:
            rows = torch.full((B,), -1, dtype=torch.int32, device="cuda")
            rows[torch.randperm(B, generator=g, device="cuda")[:n]] = torch.arange(
                n, dtype=torch.int32, device="cuda")
            s["mask_rows"] = rows
    if not case["inplace"]:  # the sampler's buffer
        s["result"] = torch.empty((B, V), dtype=s["out"], device="cuda")
    return s


# ------------------------------------------------------------------------- plain forms
def _lengths(s):
    """Per segment: row of its request, tokens held, tokens and pages before and after."""
    R, P = s["request_lens"].numel(), s["P"]
    ids, q = s["ids"].long(), s["q"].long()
    pad = ids < 0
    row = torch.where(pad, R - 1, ids)  # the last row belongs to no request
    have = torch.where(pad, 0, s["request_lens"][row].long())
    total = have + torch.where(pad, 0, q)
    return row, have, total, (have + P - 1) // P, (total + P - 1) // P


def _plain_build(s):
    P, cap = s["P"], s["cap"]
    row, have, total, held, after = _lengths(s)
    S, (R, width) = row.numel(), s["request_pages"].shape
    need = after - held
    q = total - have
    cu = torch.nn.functional.pad(q.cumsum(0), (1, 0))
    base = s["free_count"].long() - need.sum() + need.cumsum(0) - need
    j = torch.arange(width, device="cuda")
    at = (base[:, None] + j - held[:, None]).clamp(0, s["free_pages"].numel() - 1)
    new = (j >= held[:, None]) & (j < after[:, None])
    pages = torch.where(new, s["free_pages"][at], s["request_pages"][row])
    s["request_pages"][row] = pages
    bt = torch.where(j < after[:, None], pages, -1)
    t = torch.arange(cap, device="cuda")
    seg = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=S - 1)
    pos = have[seg] + t - cu[seg]
    slot = bt[seg, (pos // P).clamp(max=width - 1)].long() * P + pos % P
    live = t < cu[-1]
    some = q > 0
    rows = torch.full((S + 1,), -1, dtype=torch.int32, device="cuda")
    rows[torch.where(some, some.cumsum(0) - 1, S)] = (cu[1:] - 1).int()
    rows[S] = -1
    return dict(cu=cu.int(), sk=total.int(), bt=bt, slots=torch.where(live, slot, -1),
                pos=torch.where(live, pos, 0).int(), rows=rows[:S],
                request_pages=s["request_pages"])


def _plain_commit(s):
    row, have, total, held, after = _lengths(s)
    P, N = s["P"], s["free_pages"].numel()
    new = s["new_lens"].long()
    keep = (new + P - 1) // P
    back = after - keep
    base = s["free_count"].long() - (after - held).sum()
    j = torch.arange(s["request_pages"].shape[1], device="cuda")
    give = (j >= keep[:, None]) & (j < after[:, None])
    to = torch.where(give, base + (back.cumsum(0) - back)[:, None] + j - keep[:, None], N)
    free = torch.nn.functional.pad(s["free_pages"], (0, 1))
    free[to] = s["request_pages"][row]
    s["free_pages"].copy_(free[:N])
    s["free_count"].copy_(base + back.sum())
    s["request_lens"][row] = new.int()
    return dict(request_lens=s["request_lens"], free_pages=s["free_pages"],
                free_count=s["free_count"])


def _segments(s):
    """Per token: its segment, its first token, request row, and whether history exists."""
    cu = s["cu"].long()
    t = torch.arange(sum(s["lens"]), device="cuda")
    seg = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    lens = cu[1:] - cu[:-1]
    old = (s["sk"].long() > lens) & (lens > 0)
    return t, seg, cu[seg], s["ids"].long()[seg], old[seg]


def _plain_conv(s):
    x, w, state = s["x"].float(), s["weight"].float(), s["state"]
    K = w.shape[1]
    t, seg, first, row, old = _segments(s)

    def tap(at):
        """Inputs at tokens ``at``: the stream's, the kept ones before it, else zero."""
        back = (at - first).clamp(min=1 - K, max=-1)
        kept = torch.where(old[:, None], state[row, K - 1 + back].float(), 0)
        return torch.where((at >= first)[:, None], x[at.clamp(min=0)], kept)

    taps = [tap(t - K + 1 + k) for k in range(K)]
    y = s["bias"].float() + sum(v * w[:, k] for k, v in enumerate(taps))
    if s["silu"]:
        y = y / (1 + torch.exp(-y))
    s["out"][: t.numel()] = y.to(s["out"].dtype)
    last = s["cu"].long()[1:] - 1
    live = (s["ids"] >= 0).nonzero()[:, 0]
    state[s["ids"][live].long()] = torch.stack(
        [v[last[live]] for v in taps[1:]], 1).to(state.dtype)
    return dict(out=s["out"], state=state)


def _plain_scan(s):
    """h = exp(dt A) h + dt B x, y = C h + D x, token by token, all segments at once."""
    A, D = s["A"], s["D"]
    n = sum(s["lens"])
    x, B, C = s["x"][:n].float(), s["B"][:n].float(), s["C"][:n].float()
    dt = s["dt"][:n].float()
    if s["softplus"]:
        dt = dt + s["dt_bias"]
        dt = dt.clamp(min=0) + torch.log1p(torch.exp(-dt.abs()))
    wide = A.shape[0] // B.shape[1]
    order = sorted((i for i, k in enumerate(s["lens"]) if k), key=lambda i: -s["lens"][i])
    left = sorted((s["lens"][i] for i in order), reverse=True)
    order = torch.tensor(order, device="cuda")
    rows, first = s["ids"].long()[order], s["cu"].long()[order]
    fresh = s["sk"][order] == s["cu"][order + 1] - s["cu"][order]
    h = s["state"][rows]
    h[fresh] = 0
    y = torch.empty_like(x)
    m = len(left)
    for j in range(left[0]):
        while left[m - 1] <= j:
            m -= 1
        at = first[:m] + j
        b, c = (v[at].repeat_interleave(wide, 1) for v in (B, C))
        d = dt[at][..., None]
        h[:m] = torch.exp(d * A) * h[:m] + d * x[at][..., None] * b
        y[at] = (h[:m] * c).sum(-1)
    y = y + D * x
    if s["z"] is not None:
        z = s["z"][:n].float()
        y = y * (z / (1 + torch.exp(-z)))
    s["state"][rows] = h
    s["out"][:n] = y.to(s["out"].dtype)
    return dict(out=s["out"], state=s["state"])


def _bits(words):
    """[..., n] int32 words to [..., 32 n] truth values."""
    return ((words[..., None] >> torch.arange(32, device=words.device, dtype=torch.int32)) & 1
            ).bool().flatten(-2)


def _plain_mark(marks, ids, tokens, cu):
    """Marks of rows ``ids`` with each row's tokens added: [rows, tokens] truth values."""
    t = torch.arange(tokens.numel(), device="cuda")
    seg = torch.searchsorted(cu[1:].long().contiguous(), t, right=True)
    marks[ids.long()[seg], tokens.long()] = True


def _plain_counts(s):
    seen, counts, ids = s["seen"], s["counts"], s["ids"].long()
    live = ids[ids >= 0]
    if s["reset"]:
        seen[live], counts[live] = 0, 0
    if "prompt" in s:
        marks = _bits(seen[:, 0])
        _plain_mark(marks, ids, s["prompt"], s["cu_prompt"])
        seen[:, 0] = _pack_plain(marks)
    if "output" in s:
        cu, tok = s["cu_output"].long(), s["output"].long()
        t = torch.arange(tok.numel(), device="cuda")
        seg = torch.searchsorted(cu[1:].contiguous(), t, right=True)
        at = ids[seg] * counts.shape[1] + tok
        counts.view(-1).scatter_add_(0, at, torch.ones_like(at, dtype=torch.int32))
        marks = _bits(seen[:, 1])
        _plain_mark(marks, ids, s["output"], s["cu_output"])
        seen[:, 1] = _pack_plain(marks)
    return dict(seen=seen, counts=counts)


def _pack_plain(marks):
    """Words of 32 truth values each: eight to a byte, four bytes to a word."""
    b = marks.unflatten(-1, (-1, 8)).byte()
    b = (b << torch.arange(8, device="cuda", dtype=torch.uint8)).sum(-1, dtype=torch.uint8)
    return b.view(torch.int32)


def _plain_logits(s):
    V, ids = s["V"], s["ids"].long()
    x = s["logits"].float()
    if s["bias"] is not None:
        off, tok, val = s["bias"]
        row = torch.searchsorted(off[1:].contiguous(), torch.arange(
            tok.numel(), device="cuda", dtype=torch.int32), right=True)
        x[row, tok.long()] = x[row, tok.long()] + val
    state = s["seen"][ids]
    c = s["counts"][ids][:, :V].float()
    seen = (_bits(state[:, 0]) | _bits(state[:, 1]))[:, :V]
    rep = s["repetition"][:, None]
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["frequency"][:, None] * c - s["presence"][:, None] * (c > 0)
    if s["temperature"] is not None:
        x = x / s["temperature"][:, None]
    if s["mask"] is not None:
        allow = _bits(s["mask"])[:, :V]
        if s["mask_rows"] is not None:
            m = s["mask_rows"].long()
            allow = allow[m.clamp(min=0)] | (m < 0)[:, None]
        x = torch.where(allow, x, -math.inf)
    if s["inplace"]:
        s["logits"].copy_(x)
        return s["logits"]
    return x.to(s["out"])


# -------------------------------------------------------------------------------- run
def _own_build(mcp, s):
    mcp.build_step_tables(s["pool"], s["ids"], s["q"], s["cu"], s["sk"], s["bt"], s["slots"],
                          s["pos"], s["rows"])
    return dict(cu=s["cu"], sk=s["sk"], bt=s["bt"], slots=s["slots"], pos=s["pos"], rows=s["rows"],
                request_pages=s["request_pages"])


def _run_own(s):
    import mixed_chunked_prefill_gb300 as mcp

    op = s["op"]
    if op == "tables":
        return _own_build(mcp, s)
    if op == "oneshot":
        built = _own_build(mcp, s)
        mcp.commit_step(s["pool"], s["ids"], s["q"], s["new_lens"])
        return {**built, "request_lens": s["request_lens"], "free_pages": s["free_pages"],
                "free_count": s["free_count"]}
    if op == "conv":
        mcp.mixed_conv(s["x"], s["weight"], s["bias"], s["state"], s["ids"], s["cu"], s["sk"],
                       activation="silu" if s["silu"] else "none", out=s["out"])
        return dict(out=s["out"], state=s["state"])
    if op == "scan":
        mcp.mixed_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], s["state"], s["ids"], s["cu"],
                       s["sk"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"], softplus=s["softplus"],
                       out=s["out"])
        return dict(out=s["out"], state=s["state"])
    if op == "counts":
        if "prompt" in s:
            mcp.update_token_counts(s["ids"], s["prompt"], s["seen"], s["counts"], s["vocab"],
                                    cu_tokens=s["cu_prompt"], prompt=True, reset=s["reset"])
        if "output" in s:
            mcp.update_token_counts(s["ids"], s["output"], s["seen"], s["counts"], s["vocab"],
                                    cu_tokens=s["cu_output"],
                                    reset=s["reset"] and "prompt" not in s)
        return dict(seen=s["seen"], counts=s["counts"])
    return mcp.process_logits(
        s["logits"], None if s["inplace"] else s["result"], request_ids=s["ids"], seen=s["seen"],
        counts=s["counts"], temperature=s["temperature"], repetition_penalty=s["repetition"],
        frequency_penalty=s["frequency"], presence_penalty=s["presence"], bias=s["bias"],
        mask=s["mask"], mask_rows=s["mask_rows"])


def run(state):
    if own:
        return _run_own(state)
    op = state["op"]
    if op == "tables":
        return _plain_build(state)
    if op == "oneshot":
        built = _plain_build(state)
        return {**built, **_plain_commit(state)}
    return {"conv": _plain_conv, "scan": _plain_scan, "counts": _plain_counts,
            "logits": _plain_logits}[op](state)


# ------------------------------------------------------------------------------- work
def _distinct(n, vocab):
    """Expected number of different tokens among ``n`` of ``_tokens``."""
    import numpy as np

    v = np.arange(vocab + 1, dtype=np.float64)
    cdf = np.log1p(v) / math.log(vocab + 1.0)
    return float(-np.expm1(n * np.log1p(-np.diff(cdf).clip(max=1 - 1e-12))).sum())


def work(case):
    op = case["op"]
    if op in ("tables", "oneshot"):
        P, S, width = case["page"], case["seqs"], _width(case)
        if op == "tables":
            T, pad = S + case["chunks"] * (case["chunk"] - 1), case["pad"]
            held, cap = S * ((case["ctx_lo"] + case["ctx_hi"]) / 2 - 1) / P, T
        else:
            T, pad, held, cap = S * (case["prompt"] + 1) / 2, 0, 0, S * case["prompt"]
        new = T / P
        pages = held + new
        # ids, lengths and held pages read, new pages read and entered, tables and slots written
        bytes_ = (S + pad) * (4 * 3 + 4 * 3 + 4 * width) + 4 * pages + 4 * new + 12 * cap
        if op == "oneshot":  # every page read and put back, lengths written
            bytes_ += 8 * pages + 4 * S
        return {"bytes": bytes_, "flops": 0}
    if op in ("conv", "scan"):
        lens = [1] * case["decodes"] + [int(w.rstrip("h")) for w in case["lens"].split()]
        old = case["decodes"] + case["lens"].count("h")
        T, n, d = sum(lens), len(lens), case["channels"]
        if op == "conv":
            K = case["width"]  # rows in and out, the kept inputs read and written, the weights
            return {"bytes": 4 * T * d + 2 * (K - 1) * d * (n + old) + 2 * d * (K + 1) + 12 * n,
                    "flops": 2.0 * T * d * K}
        N = case["states"]  # x, dt, z in and y out, B and C, the states read and written, A
        b = 2 * T * d * (4 if case["gate"] else 3) + 4 * T * N * case["groups"]
        b += 4 * d * N * (n + old) + 4 * d * (N + 2) + 12 * n
        return {"bytes": b, "flops": 7.0 * T * d * N}
    if op == "counts":
        n, V = case["rows"], case["vocab"]
        words = -(-V // 32)
        p, o = case["prompt"] * 0.75, case["output"] * 0.75 if case["output"] > 1 else 1
        b = n * (4 * (p + o) + 4 + 4)
        b += n * (8 * _distinct(o, V) + 8 * min(words, _distinct(o, V)))  # counts, marks
        if p:
            b += n * 4 * min(words, _distinct(p, V))
        if case["reset"]:  # both planes written, the marked counts cleared
            b += n * (4 * 3 * words + 4 * _distinct(200, V))
        return {"bytes": b, "flops": n * o}
    B, V, h = case["rows"], case["vocab"], case["history"]
    size, out = (4 if case["dtype"] == "fp32" else 2), (4 if case["out"] == "fp32" else 2)
    outs = _distinct(max(1, h // 4), V)
    share = {"none": 0.0, "half": 0.5, "all": 1.0}[case["mask"]]
    b = B * (8 * (-(-V // 32)) + 4 * outs + 8 * case["bias"] + 24) + share * B * V / 8
    if case["inplace"] and not case["temperature"]:
        # only what changes: seen and biased tokens, and those that the mask takes
        touched = _distinct(h + max(1, h // 4), V) + case["bias"]
        b += B * touched * (size + out) * (1 - 0.98 * share) + share * 0.98 * B * V * out
    else:
        b += B * V * ((1 - 0.98 * share) * size + out)
    return {"bytes": b, "flops": 4.0 * B * V}


# ------------------------------------------------------------------------------ exact
def _exact_conv(s):
    x, w, state = s["x"].double(), s["weight"].double(), s["state"].double()
    out, K = s["out"].double(), w.shape[1]
    a = 0
    for i, n in enumerate(s["lens"]):
        if not n:
            continue
        r = int(s["ids"][i])
        kept = state[r] if int(s["sk"][i]) > n else torch.zeros_like(state[r])
        v = torch.cat([kept, x[a:a + n]])
        y = torch.einsum("tck,ck->tc", v.unfold(0, K, 1), w) + s["bias"].double()
        out[a:a + n] = y * torch.sigmoid(y) if s["silu"] else y
        state[r] = v[n:]
        a += n
    return dict(out=out, state=state)


def _exact_scan(s):
    state, out = s["state"].double(), s["out"].double()
    A, D = s["A"].double(), s["D"].double()
    d, N = A.shape
    G = s["B"].shape[1]
    a = 0
    for i, n in enumerate(s["lens"]):
        if not n:
            continue
        r = int(s["ids"][i])
        h = state[r] if int(s["sk"][i]) > n else torch.zeros_like(state[r])
        x, dt = s["x"][a:a + n].double(), s["dt"][a:a + n].double()
        if s["softplus"]:
            dt = torch.nn.functional.softplus(dt + s["dt_bias"].double())
        B, C = s["B"][a:a + n].double(), s["C"][a:a + n].double()
        y = D * x
        for t in range(n):
            b, c = (v[t, :, None].expand(G, d // G, N).reshape(d, N) for v in (B, C))
            h = torch.exp(dt[t, :, None] * A).mul_(h).addcmul_((dt[t] * x[t])[:, None], b)
            y[t] += torch.einsum("cn,cn->c", h, c)
        if s["z"] is not None:
            y *= torch.nn.functional.silu(s["z"][a:a + n].double())
        out[a:a + n], state[r] = y, h
        a += n
    return dict(out=out, state=state)


def exact(case, seed):
    """The definitions in 64 bits, segment by segment and row by row; tables and counts
    are whole numbers."""
    if case["op"] not in ("conv", "scan", "logits"):
        return None
    s = prepare(case, seed)
    if case["op"] != "logits":
        return _exact_conv(s) if case["op"] == "conv" else _exact_scan(s)
    B, V = s["logits"].shape
    y = s["logits"].double()
    word = torch.arange(V, device="cuda") // 32
    bit = torch.arange(V, device="cuda") % 32
    for i in range(B):
        r = int(s["ids"][i])
        if s["bias"] is not None:
            a, b = int(s["bias"][0][i]), int(s["bias"][0][i + 1])
            y[i].index_add_(0, s["bias"][1][a:b].long(), s["bias"][2][a:b].double())
        had = (((s["seen"][r, 0][word] | s["seen"][r, 1][word]) >> bit) & 1) != 0
        rho = s["repetition"][i].double()
        y[i] = torch.where(had & (y[i] > 0), y[i] / rho, torch.where(had, y[i] * rho, y[i]))
        n = s["counts"][r, :V].double()
        y[i] -= s["frequency"][i].double() * n + s["presence"][i].double() * n.clamp(max=1)
        if s["temperature"] is not None:
            y[i] /= s["temperature"][i].double()
        m = -1 if s["mask"] is None else i if s["mask_rows"] is None else int(s["mask_rows"][i])
        if m >= 0:
            y[i][((s["mask"][m][word] >> bit) & 1) == 0] = -math.inf
    return y
