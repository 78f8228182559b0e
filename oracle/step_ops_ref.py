"""Plain definitions of the operators around a step's attention, in Python integers
and float64: page tables and slots from request lengths, the short causal
convolution and the selective scan over a packed stream, token counts and logits.

Each floating result comes with a bound on how far an fp32 computation rounded once
may be off, built from the same loop: half a step of the output type, and 2^-24 of
every intermediate term times the operations it goes through.
"""

from __future__ import annotations

import numpy as np

U = 2.0 ** -24  # half a step of fp32, relative


class StepError(Exception):
    pass


class Pool:
    """Page lists of requests and a free list, as Python lists."""

    def __init__(self, num_pages, page_size, max_requests, max_pages_per_seq):
        self.P, self.width, self.R = page_size, max_pages_per_seq, max_requests
        self.num_pages = num_pages
        self.free = list(range(num_pages))
        self.pages = [[] for _ in range(max_requests)]
        self.lens = [0] * max_requests

    def build(self, ids, q_lens, max_tokens):
        """(cu, seqlens_k, block_tables, slots, positions, logits_indices, new pages per segment)."""
        P = self.P
        live = [r for r in ids if r >= 0]
        if len(set(live)) != len(live) or any(r >= self.R for r in live):
            raise StepError("request")
        cu, sk, bt, slots, pos, rows, taken = [0], [], [], [], [], [], []
        need = [0 if r < 0 else -(-(self.lens[r] + q) // P) - -(-self.lens[r] // P)
                for r, q in zip(ids, q_lens)]
        K = sum(need)
        if any(r >= 0 and (q < 0 or self.lens[r] + q > self.width * P) for r, q in zip(ids, q_lens)):
            raise StepError("request")
        if sum(q for r, q in zip(ids, q_lens) if r >= 0) > max_tokens:
            raise StepError("request")
        if K > len(self.free):
            raise StepError("pages")
        at = len(self.free) - K
        for r, q, n in zip(ids, q_lens, need):
            if r < 0:
                cu.append(cu[-1])
                sk.append(0)
                bt.append([-1] * self.width)
                taken.append([])
                continue
            fresh = self.free[at:at + n]
            at += n
            pages = self.pages[r] + fresh
            for p in range(self.lens[r], self.lens[r] + q):
                slots.append(pages[p // P] * P + p % P)
                pos.append(p)
            cu.append(cu[-1] + q)
            sk.append(self.lens[r] + q)
            bt.append(pages + [-1] * (self.width - len(pages)))
            if q:
                rows.append(cu[-1] - 1)
            taken.append(fresh)
        T = cu[-1]
        return (np.array(cu), np.array(sk, dtype=np.int64),
                np.array(bt, dtype=np.int64).reshape(len(ids), self.width),
                np.array(slots + [-1] * (max_tokens - T), dtype=np.int64),
                np.array(pos + [0] * (max_tokens - T), dtype=np.int64),
                np.array(rows + [-1] * (len(ids) - len(rows)), dtype=np.int64), taken)

    def commit(self, ids, q_lens, new_lens, taken):
        del self.free[len(self.free) - sum(map(len, taken)):]
        for r, q, to, fresh in zip(ids, q_lens, new_lens, taken):
            if r < 0:
                continue
            pages = self.pages[r] + fresh
            keep = -(-to // self.P)
            self.free += pages[keep:]
            self.pages[r], self.lens[r] = pages[:keep], to


def half_step(dtype):
    """(relative half step, absolute half step of the subnormals) of an output type."""
    return {"bf16": (2.0 ** -8, 2.0 ** -134), "fp16": (2.0 ** -11, 2.0 ** -25),
            "fp32": (2.0 ** -24, 2.0 ** -149)}[dtype]


def _rounded(ref, err, dtype):
    """Bound of a value that is ``err`` off ``ref`` and rounded to ``dtype``."""
    rel, sub = half_step(dtype)
    return err + rel * (np.abs(ref) + err) + sub


def _silu(a):
    with np.errstate(over="ignore"):
        return a / (1 + np.exp(-a))


def _silu_err(a, err):
    """silu of a value ``err`` off: its slope stays below 1.1; exp, the sum, the quotient
    are each within 2 ulp (4 U) and exp's argument within U |a|."""
    return 1.1 * err + np.abs(_silu(a)) * U * (16 + np.abs(a))


def conv(x, weight, bias, state, ids, cu, sk, silu, dtype):
    """(out, bound, state afterwards) of the convolution over the packed stream; rows of out
    that no segment covers are NaN."""
    T, d = x.shape
    K = weight.shape[1]
    out, bound = np.full((T, d), np.nan), np.zeros((T, d))
    state = state.copy()
    for s, r in enumerate(ids):
        a, b = cu[s], cu[s + 1]
        if r < 0 or a == b:
            continue
        kept = state[r] if sk[s] > b - a else np.zeros_like(state[r])
        v = np.concatenate([kept, x[a:b]])
        for t in range(a, b):
            terms = [weight[:, k] * v[t - a + k] for k in range(K)]
            y = bias + sum(terms)
            mag = np.abs(bias) + sum(map(np.abs, terms))
            err = (K + 1) * U * mag
            if silu:
                y, err = _silu(y), _silu_err(y, err)
            out[t], bound[t] = y, _rounded(y, err, dtype)
        state[r] = v[len(v) - (K - 1):]
    return out, bound, state


def scan(x, dt, A, B, C, D, z, dt_bias, softplus, state, ids, cu, sk, dtype):
    """(out, bound, state, state bound).  Error per step: exp(d A) as 2^(d (A log2 e)) has
    three roundings of its exponent and 2 ulp (4 U) of its own; softplus 12 U (its exp, log1p
    within 2 ulp, two sums) and the rounding of dt + dt_bias; the rest is one rounding an
    operation."""
    T, d = x.shape
    G, N = B.shape[1:]
    out, bound = np.full((T, d), np.nan), np.zeros((T, d))
    state, serr = state.copy(), np.zeros_like(state)
    wide = d // G
    for s, r in enumerate(ids):
        a, b = cu[s], cu[s + 1]
        if r < 0 or a == b:
            continue
        h = state[r] if sk[s] > b - a else np.zeros_like(state[r])
        e = np.zeros_like(h)
        for t in range(a, b):
            v = dt[t] + dt_bias
            rel = U * np.ones(d)
            if softplus:
                step = np.logaddexp(0, v)
                # the slope of ln softplus is below 1: an absolute error of U |v| is relative
                rel = 12 * U + U * np.abs(v)
            else:
                step = v
                rel = np.where(v != 0, U * (np.abs(dt[t]) + np.abs(dt_bias)) / np.maximum(np.abs(v), 1e-300), 0)
            bt, ct = np.repeat(B[t], wide, 0), np.repeat(C[t], wide, 0)
            z0 = step[:, None] * A
            f = np.exp(z0)
            in_ = (step * x[t])[:, None] * bt
            frel = 4 * U + np.abs(z0) * (3 * U + rel[:, None])
            e = f * e + np.abs(f * h) * frel + np.abs(in_) * (2 * U + rel[:, None])
            e += np.abs(h) * 2.0 ** -126  # exp below the normal numbers is 0
            h = f * h + in_
            e = e + U * np.abs(h)
            y = (ct * h).sum(1) + D * x[t]
            mag = np.abs(ct * h).sum(1) + np.abs(D * x[t])
            err = (np.abs(ct) * e).sum(1) + (N + 2) * U * mag
            if z is not None:
                g = _silu(z[t])
                err = err * np.abs(g) + np.abs(y) * _silu_err(z[t], 0) + U * np.abs(y * g)
                y = y * g
            out[t], bound[t] = y, _rounded(y, err, dtype)
        state[r], serr[r] = h, e
    return out, bound, state, serr


def update_counts(seen, counts, ids, tokens, cu, vocab, prompt, reset):
    """seen [R, 2, vocab] truth values and counts [R, vocab], updated copies."""
    seen, counts = seen.copy(), counts.copy()
    if reset:
        for r in ids:
            if 0 <= r < len(seen):
                seen[r], counts[r] = False, 0
    for i, r in enumerate(ids):
        for v in (tokens[cu[i]:cu[i + 1]] if cu is not None else tokens[i:i + 1]):
            if 0 <= r < len(seen) and 0 <= v < vocab:
                if prompt:
                    seen[r, 0, v] = True
                else:
                    seen[r, 1, v] = True
                    counts[r, v] += 1
    return seen, counts


def pack_bits(bits):
    """[..., V] truth values to [..., ceil(V / 32)] int32 words, token 0 in the lowest bit."""
    V = bits.shape[-1]
    padded = np.zeros(bits.shape[:-1] + (-(-V // 32) * 32,), dtype=np.uint8)
    padded[..., :V] = bits
    return np.ascontiguousarray(np.packbits(padded, axis=-1, bitorder="little")).view(np.int32)


def logits(x, ids, seen, counts, temperature, rho, freq, pres, bias, allow, dtype):
    """(out, bound): rows of padding (ids < 0) are NaN.  ``bias``: {row: {token: value}};
    ``allow``: per row truth values or None."""
    B, V = x.shape
    out, bound = np.full((B, V), np.nan), np.zeros((B, V))
    for i in range(B):
        r = ids[i] if ids is not None else 0
        if r < 0:
            continue
        y, mag = x[i].copy(), np.abs(x[i])
        for v, b in bias.get(i, {}).items():
            y[v] += b
            mag[v] += abs(b)
        err = U * mag
        if ids is not None:
            had = seen[r, 0] | seen[r, 1]
            # near 0 the sign, and with it the factor, may differ: both are of the size of err
            k = np.where(had, np.where(y > 0, 1 / rho[i], rho[i]), 1.0)
            err = np.where(had, max(rho[i], 1 / rho[i]) * err + U * np.abs(y * k), err)
            y = y * k
            c = counts[r] * freq[i]
            mag = np.abs(y) + np.abs(c) + np.where(counts[r] > 0, abs(pres[i]), 0)
            y = y - c - np.where(counts[r] > 0, pres[i], 0)
            err = np.where(counts[r] > 0, err + 3 * U * mag, err)
        if temperature is not None and temperature[i] > 0:
            y, err = y / temperature[i], err / temperature[i]
            err = err + 2 * U * np.abs(y)
        if allow is not None and allow[i] is not None:
            y = np.where(allow[i], y, -np.inf)
        with np.errstate(invalid="ignore"):
            bound[i] = np.where(np.isfinite(y), _rounded(y, err, dtype), 0)
        out[i] = y
    return out, bound
