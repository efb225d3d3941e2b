"""The tight bounds notice what they are for: one bf16 number a numerator, and
a delta from the rounded result (CPU only; the mistakes are planted in the
reference)."""
import pytest
import torch

import attn_ref as ref
import attn_tight as tight

BF16 = torch.bfloat16


def bf(x):
    return x.to(BF16).double()


def cancelling(g, n, dim, q, k, scale):
    """Values of which the softmax leaves hardly anything: the last key's are
    minus the others' mean, as far as bf16 goes."""
    p = torch.softmax(scale * (q.double() @ k.double().T), 1)
    v = 1 + torch.rand(n, dim, generator=g, device=q.device, dtype=torch.float64)
    v[-1] = -(p[0, :-1, None] * bf(v[:-1])).sum(0) / p[0, -1]
    return v.to(BF16)


def test_one_number_a_numerator():
    g = torch.Generator().manual_seed(2)
    n, dim = 24, 64
    q, k = (0.25 * torch.randn(1, dim, generator=g)).to(BF16), torch.randn(n, dim, generator=g).to(BF16)
    v = cancelling(g, n, dim, q, k, 0.125)
    want, tol = ref.attend(q, k, v, 0.125)["out"], tight.out_bound(q, k, v, 0.125)
    w = torch.exp(0.125 * (q.double() @ k.double().T))
    w = w / w.max()
    first = bf(w)
    two = first + bf(w - first)
    ref.close(bf((two @ v.double()) / w.sum()), want, tol, "two numbers")
    with pytest.raises(AssertionError):
        ref.close(bf((first @ v.double()) / w.sum()), want, tol, "one number")


@pytest.mark.parametrize("keys", [9, 100])
def test_delta_of_the_rounded_result(keys):
    g = torch.Generator().manual_seed(keys)
    n, dim = 8, 64
    q, k, go = (torch.randn(x, dim, generator=g).to(BF16) for x in (n, keys, n))
    v = (64 + torch.randn(keys, dim, generator=g)).to(BF16)      # a mean that all values share
    want = tight.grad_bounds(q, k, v, 0.125, go)
    s = 0.125 * (q.double() @ k.double().T)
    p = torch.softmax(torch.where(ref.visible(n, keys, 0, 0), s, -torch.inf), 1)
    dp = go.double() @ v.double().T

    def grads(delta):
        d = bf(p * (dp - delta))
        return bf(0.125 * d @ k.double()), bf(0.125 * d.T @ q.double())
    good = grads((p * dp).sum(1, keepdim=True))
    bad = grads((go.double() * bf(p @ v.double())).sum(1, keepdim=True))
    for x, y, name in zip(good, bad, ("dq", "dk")):
        ref.close(x, want[name], want[name + "_t"], name)
        with pytest.raises(AssertionError):
            ref.close(y, want[name], want[name + "_t"], name)
