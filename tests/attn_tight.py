"""Bounds that notice a rounding more: of one head's results whose numerators
are held to 2^-16 (single tokens split each into two bf16 numbers), and of
gradients whose delta comes from its definition, not from the rounded out.

Sums and names as in attn_ref, from which the values come."""
import torch

import attn_ref as ref

E, U = ref.E, ref.U


def _rel(q, k, scale, seen, s):
    """Of a numerator and of a sum, as in attn_ref.attend."""
    mag = scale * (q.abs() @ k.abs().T)
    ds = torch.where(seen, (q.shape[1] + 8) * E * mag + 4 * E * s.abs().nan_to_num(0, 0, 0), 0.0)
    return 2 * ds.amax(1, keepdim=True) + (k.shape[0] + 16) * E


def _softmax(q, k, scale, window, sinks):
    seen = ref.visible(len(q), len(k), window, sinks, q.device)
    s = torch.where(seen, scale * (q @ k.T), -torch.inf)
    return seen, s, torch.softmax(s, 1).nan_to_num(0)


def out_bound(q, k, v, scale, window=0, sinks=0):
    """Of the results of single tokens: each numerator is the sum of two bf16
    numbers, the second a rounding of what the first leaves: U of U."""
    q, k, v = q.double(), k.double(), v.double()
    seen, s, p = _softmax(q, k, scale, window, sinks)
    return (U * U + _rel(q, k, scale, seen, s)) * (p @ v.abs()) + U * (p @ v).abs() + 1e-30


def grad_bounds(q, k, v, scale, d_out, window=0, sinks=0):
    """dq and dk of one query head with delta = sum of P dP in binary32: its
    error is that of P and of dP, with no rounding to bf16 before dS'."""
    q, k, v, g = q.double(), k.double(), v.double(), d_out.double()
    n_q, n_k, dim = len(q), len(k), q.shape[1]
    seen, s, p = _softmax(q, k, scale, window, sinks)
    lse = torch.logsumexp(s, 1, keepdim=True).nan_to_num(0, 0, 0)
    rel = _rel(q, k, scale, seen, s)
    rel = 2 * rel + 4 * E * (lse.abs() + 1)          # P = exp(s - lse): lse has the same error
    dp = g @ v.T
    dp_t = (dim + 2) * E * (g.abs() @ v.abs().T)
    delta = (p * dp).sum(1, keepdim=True)
    delta_t = (rel + (n_k + 4) * E) * (p * dp.abs()).sum(1, keepdim=True) + (p * dp_t).sum(1, keepdim=True)
    # dP - delta is formed in the sum of the products: its roundings are of delta, too
    d = p * (dp - delta)
    d_t = (U + rel) * d.abs() + p * (1 + U) * (delta_t + dp_t + (dim + 2) * E * delta.abs())
    many = 1 + (n_q + n_k + 64) * E
    dq, dk = scale * (d @ k), scale * (d.T @ q)
    return {"dq": dq, "dq_t": many * scale * (d_t @ k.abs()) + (n_k + 4) * E * scale * (d.abs() @ k.abs()) + U * dq.abs() + 1e-30,
            "dk": dk, "dk_t": many * scale * (d_t.T @ q.abs()) + (n_q + 4) * E * scale * (d.abs().T @ q.abs()) + U * dk.abs() + 1e-30}
