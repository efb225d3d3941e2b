"""Attention in 64 bits, written from its definition, with bounds on what the
kernels' roundings may change.

A bf16 rounding is off by at most 2^-8 of the value, a binary32 one by 2^-24.
The kernels form scores, sums and statistics in binary32 and round to bf16:
the softmax's numerators before their product with the values, P and dS before
their products in the gradients, and each result.  The bounds below add these
up, element by element, over the sums' absolute values."""
import math

import torch

U = 2.0 ** -8          # of a bf16 rounding
E = 2.0 ** -24         # of a binary32 rounding


def visible(n_q, n_k, window, sinks, device="cpu"):
    """[n_q, n_k]: key j is seen by the query at position p = n_k - n_q + i."""
    p = torch.arange(n_q, device=device)[:, None] + (n_k - n_q)
    j = torch.arange(n_k, device=device)[None, :]
    seen = j <= p
    if window:
        seen = seen & ((j > p - window) | (j < sinks))
    return seen


def attend(q, k, v, scale, window=0, sinks=0, d_out=None, lookup=None):
    """One head in 64 bits: q [n_q, D], k and v [n_k, D].  A dict of value and
    bound (suffix _t) of out and lse, and with d_out of dq, dk and dv.
    Masked values of v (and, with gradients, of everything) count as 0."""
    q, k, v = q.double(), k.double(), v.double()
    n_q, n_k, dim = len(q), len(k), q.shape[1]
    seen = visible(n_q, n_k, window, sinks, q.device)
    none = ~seen.any(1)
    s = torch.where(seen, scale * (q @ k.T), -math.inf) if n_k else torch.zeros(n_q, 0, dtype=torch.float64, device=q.device)
    lse = torch.logsumexp(s, 1) if n_k else torch.full((n_q,), -math.inf, dtype=torch.float64, device=q.device)
    p = torch.where(none[:, None], 0.0, torch.exp(s - torch.where(none, 0.0, lse)[:, None]))
    # a score: dim products and sums in binary32 (and a scale or two); its
    # exponent's argument is formed by one multiplication and a fused one of
    # numbers as large as the score, the power is off by a few last places
    mag = scale * (q.abs() @ k.abs().T)
    ds = torch.where(seen, (dim + 8) * E * mag + 4 * E * s.abs().nan_to_num(0, 0, 0), 0.0)
    rel = ds.amax(1, keepdim=True) if n_k else torch.zeros(n_q, 1, dtype=torch.float64, device=q.device)
    rel = 2 * rel + (n_k + 16) * E                    # of a numerator and of the sum below it
    r = {"out": p @ v, "lse": lse}
    r["out_t"] = (U + rel) * (p @ v.abs()) + U * r["out"].abs() + 1e-30
    r["lse_t"] = rel[:, 0] + 4 * E * (lse.abs().nan_to_num(0, 0, 0) + 1)
    if d_out is None:
        return r
    g = d_out.double()
    dp = g @ v.T
    delta = (g * r["out"]).sum(1, keepdim=True)
    d = p * (dp - delta)
    # delta is formed from the rounded result
    delta_t = (g.abs() * r["out_t"]).sum(1, keepdim=True) + (dim + 2) * E * (g.abs() * r["out"].abs()).sum(1, keepdim=True)
    rel = rel + r["lse_t"][:, None]                   # P = exp(s - lse)
    p_t = (U + rel) * p
    d_t = (U + rel) * d.abs() + p * (1 + U) * (delta_t + (dim + 2) * E * (g.abs() @ v.abs().T))
    many = 1 + (n_q + n_k + 64) * E
    r["dq"], r["dk"], r["dv"] = scale * (d @ k), scale * (d.T @ q), p.T @ g
    r["dq_t"] = many * scale * (d_t @ k.abs()) + (n_k + 4) * E * scale * (d.abs() @ k.abs()) + U * r["dq"].abs() + 1e-30
    # dk and dv are rounded after the heads' sum: the caller adds that part
    r["dk_t"] = many * scale * (d_t.T @ q.abs()) + (n_q + 4) * E * scale * (d.abs().T @ q.abs()) + 1e-30
    r["dv_t"] = many * (p_t.T @ g.abs()) + (n_q + 4) * E * (p.T @ g.abs()) + 1e-30
    return r


def ragged(q, k, v, cu_q, cu_k, scale, window=0, sinks=0, d_out=None):
    """All sequences and heads: q [rows, hq, D], k and v [rows, hkv, D] (of
    any float type); cu_q, cu_k lists.  Dict of 64-bit values and bounds laid
    out as the operator's results; rows of no sequence are 0 with bound -1."""
    hq, hkv = q.shape[1], k.shape[1]
    group = hq // hkv
    f = dict(dtype=torch.float64, device=q.device)
    r = {x: torch.zeros(q.shape, **f) for x in ("out", "dq")}
    r.update({x: torch.zeros(k.shape, **f) for x in ("dk", "dv")}, lse=torch.zeros(q.shape[:2], **f))
    r.update({x + "_t": torch.full_like(y, -1.0) for x, y in list(r.items())})
    for b in range(len(cu_q) - 1):
        a, c = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        for x in ("dk_t", "dv_t"):
            r[x][c] = 0
        for h in range(hq):
            one = attend(q[a, h], k[c, h // group], v[c, h // group], scale, window, sinks, None if d_out is None else d_out[a, h])
            for x, y in one.items():
                if x[:2] in ("dk", "dv"):
                    r[x][c, h // group] += y
                else:
                    r[x][a, h] = y
        for x in ("dk", "dv"):
            r[x + "_t"][c] += U * r[x][c].abs() + group * E * r[x][c].abs()
    return r


def paged(cache, table, length):
    """Keys and values of a sequence out of a cache, as 64-bit values
    [length, heads, D]."""
    page = cache[0].shape[1]
    j = torch.arange(length, device=cache[0].device)
    at = (table.long()[j // page], j % page)
    res = []
    for i in range(2):
        x = cache[i][at].to(torch.float32).double()
        if len(cache) == 4:
            x = x * cache[2 + i][at].double()[..., None]
        res.append(x)
    return res


def close(got, want, tol, what):
    """Every element within its bound; infinities in their places.  A bound
    below 0 marks what is not checked."""
    got = got.double().to(want.device)
    checked = tol >= 0
    same = torch.isinf(want) & (got == want)
    bad = checked & ~same & ~((got - want).abs() <= tol)
    if bad.any():
        i = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} beyond their bounds; first at {i}: "
                             f"{float(got[i])} for {float(want[i])} +- {float(tol[i])}")
