"""CPU oracle for the serving-step operators -- test infrastructure.

Plain Python and numpy in 64 bits; it shares no code with the CUDA library.

* ``page_table_update``: a literal stack of free pages, pushed and popped one
  page at a time.
* ``slot_map``: loops over requests and tokens.
* ``rope``: rotation by exact integer phases, cosine and sine in fp64.
* ``token_logprobs``: log-softmax, entropy and order by (logit, id) in fp64.
"""
from __future__ import annotations

import math

import numpy as np


def page_table_update(lens, page_size, table, held, free):
    """table: list of lists; held: list; free: list used as a stack (its end is
    the top).  Returns (table, held, free, flagged rows)."""
    table, held, free = [list(t) for t in table], list(held), list(free)
    need, flagged = [], []
    for r, n in enumerate(lens):
        want = held[r] if n == -1 else -(-n // page_size)
        if n < -1 or want > len(table[r]) or not 0 <= held[r] <= len(table[r]):
            flagged.append(r)
            want = held[r]
        need.append(want)
    for r in reversed(range(len(lens))):
        if need[r] < held[r]:
            for j in reversed(range(need[r], held[r])):
                free.append(table[r][j])
            held[r] = need[r]
    full = False
    for r in range(len(lens)):
        grow = need[r] - held[r]
        if grow <= 0 or r in flagged:
            continue
        if full or grow > len(free):
            full = True
            flagged.append(r)
            continue
        for j in range(held[r], need[r]):
            table[r][j] = free.pop()
        held[r] = need[r]
    return table, held, free, sorted(flagged)


def slot_map(table, page_size, rows, prefix, tree, parents):
    """(kv_indptr, kv_indices, qo_indptr, out_cache_loc, positions); parents:
    one list a request, or None for chains."""
    kv_ptr, kv, q_ptr, loc, pos = [0], [], [0], [], []
    for r in range(len(prefix)):
        pages = table[rows[r]]
        slot = lambda j: int(pages[j // page_size]) * page_size + j % page_size  # noqa: E731
        kv += [slot(j) for j in range(prefix[r])]
        loc += [slot(prefix[r] + t) for t in range(tree[r])]
        for t in range(tree[r]):
            depth, up = 0, t - 1 if parents is None else parents[r][t]
            while up >= 0:
                depth += 1
                up = up - 1 if parents is None else parents[r][up]
            pos.append(prefix[r] + depth)
        kv_ptr.append(len(kv))
        q_ptr.append(len(loc))
    as64 = lambda v: np.array(v, dtype=np.int64)  # noqa: E731
    return np.array(kv_ptr, dtype=np.int32), as64(kv), as64(q_ptr), as64(loc), as64(pos)


def rope(x, positions, turns, amplitude, half, inverse=False):
    """x: fp64 [tokens, ..., d]; returns (rotated, |x1| + |x2| at both members
    of each pair, which bounds the rounding of the rotation)."""
    x = np.asarray(x, dtype=np.float64)
    d = x.shape[-1]
    out, mag = np.empty_like(x), np.empty_like(x)
    for t, p in enumerate(positions):
        for i in range(d // 2):
            phase = (int(p) * int(turns[i])) % (1 << 64)
            a = 2.0 * math.pi * (phase / float(1 << 64))
            if inverse:
                a = -a
            c, s = amplitude * math.cos(a), amplitude * math.sin(a)
            j, k = (i, i + d // 2) if half else (2 * i, 2 * i + 1)
            x1, x2 = x[t, ..., j], x[t, ..., k]
            out[t, ..., j], out[t, ..., k] = x1 * c - x2 * s, x1 * s + x2 * c
            mag[t, ..., j] = mag[t, ..., k] = abs(amplitude) * (np.abs(x1) + np.abs(x2))
    return out, mag


def token_logprobs(logits, inv_temperature, tokens, rows, top_k):
    """logits: fp64 [n, V] (exact values); inv_temperature: fp32 values or None;
    tokens[i] under row rows[i].  Returns a dict; "mean" and "square" are the
    means of |d| and d^2 under the row's distribution (error bounds)."""
    logits = np.asarray(logits, dtype=np.float64)
    n, v = logits.shape
    scale = np.ones(n) if inv_temperature is None else np.asarray(inv_temperature, dtype=np.float64)
    stats = np.empty((3, n))
    top_tokens = np.full((top_k, n), -1, dtype=np.int32)
    top_logprobs = np.full((top_k, n), -np.inf)
    mean, square = np.zeros(n), np.zeros(n)
    bad = np.zeros(n, dtype=bool)
    for r in range(n):
        x, s = logits[r], scale[r]
        with np.errstate(over="ignore", invalid="ignore"):
            m = float(np.float32(x.max() * s)) if len(x) else -np.inf
        bad[r] = bool(np.isnan(x).any() or np.isposinf(x).any() or not (s > 0 and np.isfinite(s)) or
                      (x.max() > -np.inf and not np.isfinite(m)))
        if bad[r]:
            stats[:, r] = np.nan
            top_logprobs[:, r] = np.nan
            continue
        if x.max() == -np.inf:
            stats[:, r] = -np.inf, -np.inf, 0.0
            continue
        d = x * s - m
        e = np.exp(d)
        total = e.sum()
        log_total = math.log(total)
        live = e > 0
        u = float((e[live] * d[live]).sum())
        stats[:, r] = m, log_total, log_total - u / total
        mean[r] = float((e[live] * np.abs(d[live])).sum()) / total
        square[r] = float((e[live] * d[live] ** 2).sum()) / total
        order = np.lexsort((np.arange(v), -x))[:top_k]
        for k, i in enumerate(order):
            if x[i] > -np.inf:
                top_tokens[k, r], top_logprobs[k, r] = i, d[i] - log_total
    given = np.empty(len(tokens))
    for i, (t, r) in enumerate(zip(tokens, rows)):
        if not 0 <= r < n or not -1 <= t < v:
            given[i] = np.nan
        elif t == -1:
            given[i] = 0.0
        elif bad[r]:
            given[i] = np.nan
        elif logits[r, t] == -np.inf:
            given[i] = -np.inf
        else:
            given[i] = (logits[r, t] * scale[r] - stats[0, r]) - stats[1, r]
    return dict(stats=stats, top_tokens=top_tokens, top_logprobs=top_logprobs, logprobs=given, mean=mean,
                square=square, bad=bad)
