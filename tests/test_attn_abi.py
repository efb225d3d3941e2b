"""Argument checks of the rotary append and of attention, and what their bounds
rest on (CPU only: every call here fails validation or has nothing to do)."""
import ctypes
import math

import pytest
import torch

import attn_ref as ref
import tensor_all_reduce_amd as tar
from test_block_types import FakeTensor

G = 2 ** 32
A, B, C, D, E, F, H, I, J, K = (G * k for k in range(1, 11))      # never dereferenced
INV, ALIGN, ALIAS, UNS, OK = tar.AR_ERR_INVALID, tar.AR_ERR_ALIGN, tar.AR_ERR_ALIAS, tar.AR_ERR_UNSUPPORTED, tar.AR_OK


def hm(p=A, ts=1024, hs=128):
    return None if p is None else ctypes.byref(tar._Heads(p, ts, hs))


def kv(k=E, v=F, ks=None, vs=None, pages=8, size=16, heads=2, dim=128, st=(4096, 256, 128), ss=(32, 2, 1), fmt=0):
    return ctypes.byref(tar._KVCache(k, v, ks, vs, pages, size, heads, dim, *st, *ss, fmt))


SMALL = dict(ks=H, vs=I, fmt=tar.AR_FMT_E4M3)


def rope(q=True, k=True, v=True, tokens=4, hq=8, hkv=2, dim=128, cs=J, rows=64, rot=128, pos=K, qo=True, ko=None, cache=None,
         slots=None, flags=0):
    q, k, v, qo = (x if x is not True else y for x, y in ((q, hm(A)), (k, hm(B)), (v, hm(C)), (qo, hm(D))))
    return tar.lib().ar_rope_kv(q, k, v, tokens, hq, hkv, dim, cs, rows, rot, pos, qo, ko, cache, slots, flags, None)


def test_rope_refusals():
    c, s = kv(), 11 * G
    good = dict(cache=c, slots=s)
    assert rope(**good, tokens=0) == OK and rope(q=None, qo=None, hq=0, k=None, v=None, hkv=0) == OK
    assert rope() == INV                                             # keys that go nowhere
    assert rope(**good, flags=4) == INV and rope(**good, rot=24) == INV and rope(**good, rot=144) == INV
    assert rope(**good, dim=120) == INV and rope(**good, dim=0) == INV
    assert rope(cache=kv(dim=256), slots=s, dim=256) == UNS and rope(**good, tokens=2 ** 31) == UNS
    assert rope(**good, q=None) == INV and rope(**good, qo=None) == INV and rope(**good, hq=0) == INV
    assert rope(**good, k=None) == INV and rope(**good, hkv=0) == INV and rope(**good, v=None) == INV
    assert rope(cache=c) == INV and rope(**good, cs=None) == INV and rope(**good, pos=None) == INV and rope(**good, rows=0) == INV
    assert rope(cache=kv(heads=3), slots=s) == INV and rope(cache=kv(dim=64), slots=s) == INV
    assert rope(**good, tokens=2 ** 28) == UNS                       # more work than a grid counts
    for bad in (dict(q=hm(A + 8)), dict(k=hm(B + 2)), dict(v=hm(C + 8)), dict(qo=hm(D + 4)), dict(ko=hm(H + 8)),
                dict(q=hm(A, 1028)), dict(k=hm(B, 1024, 132)), dict(cs=J + 4), dict(pos=K + 2), dict(slots=s + 4)):
        assert rope(**{**good, **bad}) == ALIGN, bad
    assert rope(**good, qo=hm(A, 1024, 136)) == ALIAS                # over its input, but not exactly
    assert rope(**good, qo=hm(A + 16)) == ALIAS and rope(**good, qo=hm(B)) == ALIAS
    assert rope(**good, qo=hm(D, 512)) == ALIAS                      # two tokens in one place
    assert rope(**good, ko=hm(D)) == ALIAS and rope(**good, ko=hm(E)) == ALIAS and rope(**good, qo=hm(J)) == ALIAS
    assert rope(cache=kv(k=A), slots=s) == ALIAS and rope(cache=kv(v=K), slots=s) == ALIAS and rope(cache=kv(k=s), slots=s) == ALIAS


def test_cache_refusals():
    def at(**k):
        return rope(cache=kv(**k), slots=11 * G, tokens=1)
    assert at(fmt=1) == INV and at(k=None) == INV and at(v=None) == INV and at(fmt=2) == INV
    assert at(pages=0) == INV and at(size=0) == INV and at(pages=2 ** 60, size=16) == INV
    assert at(pages=2 ** 27, size=16) == UNS
    assert at(k=E + 8) == ALIGN and at(v=F + 2) == ALIGN and at(st=(4100, 256, 128)) == ALIGN and at(st=(4096, 252, 128)) == ALIGN
    assert at(**SMALL, st=(4104, 256, 128)) == ALIGN and at(ks=H + 2, vs=I, fmt=2) == ALIGN
    assert at(v=E) == ALIAS and at(v=E + 2048) == ALIAS              # values among the keys
    assert at(st=(4096, 128, 128)) == ALIAS and at(st=(2048, 256, 128)) == ALIAS and at(st=(0, 256, 128)) == ALIAS
    assert at(**SMALL, ss=(32, 1, 1)) == ALIAS and at(ks=H, vs=H, fmt=2) == ALIAS and at(ks=E, vs=I, fmt=2) == ALIAS
    assert at(st=(2 ** 62, 256, 128)) == INV


def decode(q=True, cache=None, table=J, ts=8, tp=8, lens=K, seqs=3, hq=8, scale=0.1, window=0, sinks=0, out=True, lse=None, lt=8,
           lh=1, ws=None, wb=0):
    q, out = hm(A) if q is True else q, hm(B) if out is True else out
    return tar.lib().ar_attn_decode(q, cache or kv(), table, ts, tp, lens, seqs, hq, scale, window, sinks, out, lse, lt, lh, ws, wb,
                                    None)


MASK = [(dict(hq=7), INV), (dict(hq=0), INV), (dict(scale=0.0), INV), (dict(scale=-1.0), INV), (dict(scale=math.nan), INV),
        (dict(scale=math.inf), INV), (dict(scale=2.0 ** -65), UNS), (dict(scale=2.0 ** 65), UNS), (dict(hq=2 ** 17), UNS)]


def test_decode_refusals():
    for bad, rc in MASK:
        assert decode(**bad) == rc, bad
    assert decode(seqs=0) == OK and decode(seqs=0, q=None) == OK
    assert decode(q=None) == INV and decode(out=None) == INV and decode(table=None) == INV and decode(lens=None) == INV
    assert decode(tp=0) == INV and decode(ts=7) == INV and decode(seqs=2 ** 31) == UNS
    assert decode(cache=kv(dim=144)) == UNS and decode(cache=kv(dim=8)) == INV
    assert decode(q=hm(A + 8)) == ALIGN and decode(out=hm(B, 1020)) == ALIGN and decode(table=J + 2) == ALIGN
    assert decode(lens=K + 1) == ALIGN and decode(lse=C + 2) == ALIGN and decode(ws=D + 8, wb=100) == ALIGN
    assert decode(out=hm(A + 16)) == ALIAS and decode(out=hm(E)) == ALIAS and decode(out=hm(J)) == ALIAS
    assert decode(lse=B) == ALIAS and decode(lse=C, lt=0) == ALIAS and decode(lse=K) == ALIAS
    need = tar.attn_decode_workspace(3, 8, 2, 128)
    assert decode(ws=B, wb=need) == ALIAS and decode(ws=F - 64, wb=need) == ALIAS
    # a row of tiles that 32 bits do not count
    assert decode(seqs=2 ** 20, tp=2 ** 26, ts=2 ** 26) == UNS
    assert tar.attn_decode_workspace(0, 8, 2, 128) == 0 and tar.attn_decode_workspace(3, 7, 2, 128) == 0
    assert tar.attn_decode_workspace(3, 8, 2, 136) == 0 and tar.attn_decode_workspace(3, 8, 2, 64) == need


def attn(q=True, k=True, v=True, cq=J, ck=K, seqs=2, rq=10, rk=12, hq=8, hkv=2, dim=128, scale=0.1, window=0, sinks=0, out=True,
         lse=None, lt=8, lh=1):
    q, k, v, out = (x if x is not True else hm(y) for x, y in ((q, A), (k, B), (v, C), (out, D)))
    return tar.lib().ar_attn(q, k, v, cq, ck, seqs, rq, rk, hq, hkv, dim, scale, window, sinks, out, lse, lt, lh, None)


def test_attn_refusals():
    for bad, rc in MASK:
        assert attn(**bad) == rc, bad
    assert attn(seqs=0) == OK and attn(rq=0, q=None) == OK
    assert attn(hkv=3) == INV and attn(dim=72) == INV and attn(dim=256) == UNS and attn(rq=2 ** 31) == UNS and attn(rk=2 ** 31) == UNS
    for x in ("q", "k", "v", "out"):
        assert attn(**{x: None}) == INV and attn(**{x: hm(E + 8)}) == ALIGN and attn(**{x: hm(E, 1025)}) == ALIGN, x
    assert attn(cq=None) == INV and attn(ck=None) == INV and attn(cq=J + 2) == ALIGN and attn(ck=K + 2) == ALIGN
    assert attn(out=hm(B)) == ALIAS and attn(out=hm(A, 1024, 136)) == ALIAS and attn(out=hm(J)) == ALIAS
    assert attn(out=hm(D, 1016)) == ALIAS and attn(lse=D) == ALIAS and attn(lse=E, lt=1) == ALIAS and attn(lse=E + 2) == ALIGN
    assert attn(rq=2 ** 30, hq=2 ** 15, hkv=1, q=hm(A, 2 ** 22), out=hm(2 ** 60, 2 ** 22)) == UNS   # a grid too large


def paged(q=True, cache=None, table=J, ts=8, tp=8, lens=K, cq=12 * G, seqs=2, rq=10, hq=8, scale=0.1, out=True, lse=None):
    q, out = hm(A) if q is True else q, hm(B) if out is True else out
    return tar.lib().ar_attn_paged(q, cache or kv(), table, ts, tp, lens, cq, seqs, rq, hq, scale, 0, 0, out, lse, 8, 1, None)


def test_paged_refusals():
    for bad, rc in MASK:
        assert paged(**bad) == rc, bad
    assert paged(seqs=0) == OK and paged(rq=0) == OK
    assert paged(q=None) == INV and paged(cq=None) == INV and paged(lens=None) == INV and paged(table=None) == INV and paged(ts=4) == INV
    assert paged(out=hm(F)) == ALIAS and paged(cache=kv(v=B)) == ALIAS and paged(lse=J) == ALIAS
    assert paged(cache=kv(**{**SMALL, "ks": B})) == ALIAS


def bwd(q=True, k=True, v=True, o=True, lse=E, go=True, cq=J, ck=K, seqs=2, rq=10, rk=12, hq=8, hkv=2, dim=128, scale=0.1, window=0,
        sinks=0, dq=True, dk=True, dv=True, ws=14 * G, wb=None):
    names = ((q, A), (k, B), (v, C), (o, D), (go, F), (dq, H), (dk, I), (dv, 13 * G))
    q, k, v, o, go, dq, dk, dv = (x if x is not True else hm(y) for x, y in names)
    wb = tar.attn_bwd_workspace(rq, rk, seqs, hq, hkv, dim, window, sinks) if wb is None else wb
    return tar.lib().ar_attn_bwd(q, k, v, o, lse, 8, 1, go, cq, ck, seqs, rq, rk, hq, hkv, dim, scale, window, sinks, dq, dk, dv, ws,
                                 wb, None)


def test_bwd_refusals():
    for bad, rc in MASK:
        assert bwd(**bad, wb=2 ** 20) == rc, bad
    assert bwd(seqs=0) == OK and bwd(rq=0, rk=0) == OK
    assert bwd(dk=None) == INV and bwd(dv=None) == INV and bwd(dq=None, dk=None, dv=None) == INV
    for x in ("q", "k", "v", "o", "go"):
        assert bwd(**{x: None}) == INV and bwd(**{x: hm(15 * G + 8)}) == ALIGN, x
    for x in ("dq", "dk", "dv"):
        assert bwd(**{x: hm(15 * G, 1020)}) == ALIGN and bwd(**{x: hm(A)}) == ALIAS and bwd(**{x: hm(E)}) == ALIAS, x
        assert bwd(**{x: hm(14 * G)}) == ALIAS and bwd(**{x: hm(15 * G, 128)}) == ALIAS, x
    assert bwd(dk=hm(H)) == ALIAS and bwd(dv=hm(I)) == ALIAS
    assert bwd(lse=None) == INV and bwd(cq=None) == INV and bwd(ck=None) == INV and bwd(ws=None) == INV
    need = tar.attn_bwd_workspace(10, 12, 2, 8, 2, 128)
    assert bwd(wb=need - 1) == INV and bwd(ws=14 * G + 8) == ALIGN
    assert tar.attn_bwd_workspace(2 ** 31, 12, 2, 8, 2, 128) == 0 and tar.attn_bwd_workspace(10, 12, 2, 8, 3, 128) == 0


# ------------------------------------------------------------------ bindings

BF16, F16, F32, U8, I32, I64 = torch.bfloat16, torch.float16, torch.float32, torch.uint8, torch.int32, torch.int64
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


class Fake(FakeTensor):
    """Contiguous, of any rank."""

    def stride(self, i):
        n = 1
        for s in self.shape[i + 1:]:
            n *= s
        return n


def calls():
    t = dict(q=Fake(A, (3, 8, 64), BF16), k=Fake(B, (3, 2, 64), BF16), v=Fake(C, (3, 2, 64), BF16), out=Fake(D, (3, 8, 64), BF16),
             kc=Fake(E, (8, 16, 2, 64), BF16), vc=Fake(F, (8, 16, 2, 64), BF16), table=Fake(H, (3, 4), I32), lens=Fake(I, (3,), I32),
             cu=Fake(J, (2,), I32), cs=Fake(K, (9, 64), F32), pos=Fake(11 * G, (3,), I32), slots=Fake(12 * G, (3,), I64),
             lse=Fake(13 * G, (3, 8), F32), go=Fake(14 * G, (3, 8, 64), BF16), ks=Fake(15 * G, (8, 16, 2), F32), vs=Fake(16 * G, (8, 16, 2), F32))
    return t, {
        "rope": lambda t: tar.ar_rope_kv(t["q"], t["k"], t["v"], t["cs"], t["pos"], q_out=t["out"], cache=(t["kc"], t["vc"]), slots=t["slots"], stream=0),
        "decode": lambda t: tar.ar_attn_decode(t["q"], (t["kc"], t["vc"]), t["table"], t["lens"], t["out"], lse=t["lse"], stream=0),
        "paged": lambda t: tar.ar_attn_paged(t["q"], (t["kc"], t["vc"]), t["table"], t["lens"], t["cu"], t["out"], stream=0),
        "attn": lambda t: tar.ar_attn(t["q"], t["k"], t["v"], t["cu"], t["cu"], t["out"], lse=t["lse"], stream=0),
        "bwd": lambda t: tar.ar_attn_bwd(t["q"], t["k"], t["v"], t["out"], t["lse"], t["go"], t["cu"], t["cu"], dk=t["kc"], dv=t["vc"], stream=0),
    }


WRONG = [("rope", "q", F16), ("rope", "k", F32), ("rope", "v", F16), ("rope", "cs", I32), ("rope", "pos", F32), ("rope", "pos", I64),
         ("rope", "slots", I32), ("rope", "kc", F16), ("rope", "out", F16), ("decode", "q", F16), ("decode", "vc", F16),
         ("decode", "kc", E4M3), ("decode", "table", F32), ("decode", "table", I64), ("decode", "lens", I64), ("decode", "out", F32),
         ("decode", "lse", I32), ("paged", "cu", F32), ("paged", "lens", F32), ("attn", "k", F16), ("attn", "cu", I64), ("attn", "lse", BF16),
         ("bwd", "go", F16), ("bwd", "lse", I32), ("bwd", "out", F16)]


@pytest.mark.parametrize("call,name,dtype", WRONG)
def test_bindings_refuse_types(call, name, dtype):
    t, c = calls()
    t[name].dtype = dtype
    with pytest.raises(ValueError):
        c[call](t)


SHAPES = [("rope", "k", (3, 2, 32)), ("rope", "v", (2, 2, 64)), ("rope", "out", (3, 7, 64)), ("rope", "pos", (4,)), ("rope", "slots", (3, 1)),
          ("rope", "cs", (64,)), ("decode", "out", (3, 8, 32)), ("decode", "kc", (8, 16, 2, 32)), ("decode", "vc", (8, 16, 3, 64)),
          ("decode", "table", (2, 4)), ("decode", "lens", (2,)), ("decode", "lse", (8, 3)), ("paged", "cu", (2, 1)), ("attn", "v", (3, 3, 64)),
          ("attn", "k", (3, 2, 32)), ("attn", "cu", (2, 2)), ("bwd", "go", (3, 8, 32)), ("bwd", "out", (2, 8, 64)), ("bwd", "lse", (3, 7))]


@pytest.mark.parametrize("call,name,shape", SHAPES)
def test_bindings_refuse_shapes(call, name, shape):
    t, c = calls()
    t[name].shape = shape
    with pytest.raises(ValueError):
        c[call](t)


def test_bindings_refuse_the_rest():
    t, c = calls()
    q, k, v, out = (torch.zeros(3, 2, 64, dtype=BF16) for _ in range(4))
    with pytest.raises(ValueError):                                  # not on a device
        tar.ar_attn(q, k, v, torch.zeros(2, dtype=I32), torch.zeros(2, dtype=I32), out)
    for kw in (dict(window=-1), dict(sinks=-1)):
        with pytest.raises(ValueError):
            tar.ar_attn_decode(t["q"], (t["kc"], t["vc"]), t["table"], t["lens"], t["out"], stream=0, **kw)
    with pytest.raises(ValueError):                                  # codes without scales, scales without codes
        tar.ar_attn_decode(t["q"], (t["kc"], t["vc"], t["ks"]), t["table"], t["lens"], t["out"], stream=0)
    with pytest.raises(ValueError):
        tar.ar_attn_decode(t["q"], (t["kc"], t["vc"], t["ks"], t["vs"]), t["table"], t["lens"], t["out"], stream=0)
    with pytest.raises(ValueError):
        tar.ar_rope_kv(t["q"], t["k"], t["v"], t["cs"], t["pos"], cache=(t["kc"], t["vc"]), slots=t["slots"])
    with pytest.raises(ValueError):
        tar.ar_rope_kv(t["q"], t["k"], t["v"], t["cs"], t["pos"], q_out=t["out"], cache=(t["kc"], t["vc"]))
    with pytest.raises(ValueError):
        tar.ar_rope_kv(None, None, None, t["cs"], t["pos"])


# ------------------------------------------------------- the plain form itself

def test_reference_against_direct_sums():
    """attn_ref against the softmax written out, and its gradients against
    automatic ones."""
    g = torch.Generator().manual_seed(3)
    q, k, v, go = (torch.randn(n, 8, generator=g, dtype=torch.float64) for n in (6, 9, 9, 6))
    for window, sinks in ((0, 0), (3, 0), (3, 2), (1, 9)):
        leaves = [x.clone().requires_grad_() for x in (q, k, v)]
        rows = []
        for i in range(6):
            p = 3 + i
            seen = [j for j in range(9) if j <= p and (not window or j > p - window or j < sinks)]
            w = torch.exp(0.4 * torch.stack([leaves[0][i] @ leaves[1][j] for j in seen]))
            rows.append(sum(w[x] * leaves[2][j] for x, j in enumerate(seen)) / w.sum())
        out = torch.stack(rows)
        (out * go).sum().backward()
        r = ref.attend(q, k, v, 0.4, window, sinks, go)
        assert torch.allclose(r["out"], out.detach(), atol=1e-13)
        for x, y in zip(("dq", "dk", "dv"), leaves):
            assert torch.allclose(r[x], y.grad, atol=1e-12), x


def test_a_bound_notices_a_wrong_mask():
    """A window one key too wide, in the reference alone, is far beyond the bounds."""
    g = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn(40, 64, generator=g).to(BF16) for _ in range(3))
    want = ref.attend(q, k, v, 0.125, 8, 1)
    with pytest.raises(AssertionError):
        ref.close(ref.attend(q, k, v, 0.125, 9, 1)["out"], want["out"], want["out_t"], "out")
    ref.close(want["out"].to(BF16), want["out"], want["out_t"], "rounded")


def test_page_division():
    """The multiplier by which kernels divide positions by page sizes: exact for
    every position below 2^31 (around multiples, where it could fail)."""
    for d in (2, 3, 5, 7, 16, 48, 100, 511, 512, 12345, 2 ** 20 - 1, 2 ** 20, 2 ** 30 + 1, 2 ** 31 - 1):
        lg = 1
        while 1 << lg < d:
            lg += 1
        m = ((1 << (31 + lg)) + d - 1) // d
        assert m < 2 ** 32
        for n in (0, 1, 2, 3, 1000, (2 ** 31 - 1) // d - 1, (2 ** 31 - 1) // d):
            for x in (n * d - 1, n * d, n * d + 1):
                if 0 <= x < 2 ** 31:
                    assert (x * m >> 32) >> (lg - 1) == x // d
