"""CPU oracle for the operators of the attention layer -- test infrastructure.

Plain torch in 64 bits on the CPU; it shares no code with the CUDA library.
Every function also returns the sums of magnitudes that its rounding bounds
are counted from.

* ``head_product``: one matrix product a head.
* ``prefill``: a softmax over each query's visible keys, row by row.
* ``norm``: root-mean-square norm (the rotation is ``step_ops.rope``).
"""
from __future__ import annotations

import math

import torch


def head_product(x, w):
    """x [tokens, heads, k], w [heads, k, n]: (out, sum |x w|), fp64."""
    x, w = x.double().cpu(), w.double().cpu()
    return torch.einsum("thk,hkn->thn", x, w), torch.einsum("thk,hkn->thn", x.abs(), w.abs())


def prefill(q, k_nope, k_rope, v, qo_indptr, kv_indptr, scale, causal=True):
    """Dict of fp64 results, NaN in rows of no request: out, lse; and spread =
    sum p |v - out|, mag = sum p |v|, smag = the row's largest scale sum |q k|."""
    q, k_nope, k_rope, v = (t.double().cpu() for t in (q, k_nope, k_rope, v))
    rows, heads = q.shape[:2]
    full = lambda *s: torch.full(s, math.nan, dtype=torch.float64)  # noqa: E731
    res = {"out": full(rows, heads, 128), "lse": full(rows, heads), "spread": full(rows, heads, 128),
           "mag": full(rows, heads, 128), "smag": full(rows, heads)}
    for r in range(len(qo_indptr) - 1):
        q0, n = int(qo_indptr[r]), int(qo_indptr[r + 1] - qo_indptr[r])
        k0, length = int(kv_indptr[r]), int(kv_indptr[r + 1] - kv_indptr[r])
        for i in range(n):
            seen = max(0, length - n + i + 1) if causal else length
            row = q0 + i
            if seen == 0:
                for key in ("out", "spread", "mag", "smag"):
                    res[key][row] = 0.0
                res["lse"][row] = -math.inf
                continue
            keys = slice(k0, k0 + seen)
            s = (torch.einsum("hd,jhd->hj", q[row, :, :128], k_nope[keys]) + q[row, :, 128:] @ k_rope[keys].t()) * scale
            a = (torch.einsum("hd,jhd->hj", q[row, :, :128].abs(), k_nope[keys].abs())
                 + q[row, :, 128:].abs() @ k_rope[keys].abs().t()) * scale
            p = torch.softmax(s, dim=1)
            out = torch.einsum("hj,jhd->hd", p, v[keys])
            res["out"][row] = out
            res["lse"][row] = torch.logsumexp(s, dim=1)
            res["spread"][row] = torch.einsum("hj,jhd->hd", p, (v[keys] - out).abs())
            res["mag"][row] = torch.einsum("hj,jhd->hd", p, v[keys].abs())
            res["smag"][row] = a.amax(dim=1)
    return res


def norm(x, weight, eps):
    """x / sqrt(mean(x^2) + eps) * weight over the last dimension, fp64."""
    x = x.double().cpu()
    return x / torch.sqrt((x * x).mean(dim=-1, keepdim=True) + eps) * weight.double().cpu()
