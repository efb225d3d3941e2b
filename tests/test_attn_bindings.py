"""The bindings' checks of the rotary append and of attention, each on a call
that is right but for the tensor in question (CPU only: calls are marshalled,
none is made)."""
import pytest

import tensor_all_reduce_amd as tar
from test_attn_abi import A, B, BF16, C, D, E, E4M3, E5M2, F, F16, F32, Fake, G, H, I, I32, I64, J, K, U8

Q, KV = (3, 8, 64), (3, 2, 64)
CACHE, SCALES = (8, 16, 2, 64), (8, 16, 2)


def tensors():
    at = iter(range(11, 40))
    new = lambda shape, dtype: Fake(next(at) * G, shape, dtype)      # noqa: E731
    return dict(q=Fake(A, Q, BF16), k=Fake(B, KV, BF16), v=Fake(C, KV, BF16), out=Fake(D, Q, BF16), kc=Fake(E, CACHE, BF16),
                vc=Fake(F, CACHE, BF16), table=Fake(H, (3, 4), I32), lens=Fake(I, (3,), I32), cu=Fake(J, (4,), I32), cs=Fake(K, (9, 64), F32),
                pos=new((3,), I32), slots=new((3,), I64), lse=new((3, 8), F32), go=new(Q, BF16), k8=new(CACHE, E4M3), v8=new(CACHE, E4M3),
                ks=new(SCALES, F32), vs=new(SCALES, F32), dq=new(Q, BF16), dk=new(KV, BF16), dv=new(KV, BF16), ko=new(KV, BF16),
                ck=new((4,), I32), ws=new((2 ** 20,), U8))


CALLS = {
    "rope": lambda t: tar.prepare(tar.ar_rope_kv, t["q"], t["k"], t["v"], t["cs"], t["pos"], q_out=t["out"], k_out=t["ko"],
                                  cache=(t["kc"], t["vc"]), slots=t["slots"], stream=0),
    "rope8": lambda t: tar.prepare(tar.ar_rope_kv, t["q"], t["k"], t["v"], t["cs"], t["pos"], q_out=t["out"],
                                   cache=(t["k8"], t["v8"], t["ks"], t["vs"]), slots=t["slots"], stream=0),
    "decode": lambda t: tar.prepare(tar.ar_attn_decode, t["q"], (t["kc"], t["vc"]), t["table"], t["lens"], t["out"], lse=t["lse"],
                                    workspace=t["ws"], stream=0),
    "decode8": lambda t: tar.prepare(tar.ar_attn_decode, t["q"], (t["k8"], t["v8"], t["ks"], t["vs"]), t["table"], t["lens"], t["out"],
                                     stream=0),
    "paged": lambda t: tar.prepare(tar.ar_attn_paged, t["q"], (t["kc"], t["vc"]), t["table"], t["lens"], t["cu"], t["out"], lse=t["lse"],
                                   stream=0),
    "attn": lambda t: tar.prepare(tar.ar_attn, t["q"], t["k"], t["v"], t["cu"], t["ck"], t["out"], lse=t["lse"], stream=0),
    "bwd": lambda t: tar.prepare(tar.ar_attn_bwd, t["q"], t["k"], t["v"], t["out"], t["lse"], t["go"], t["cu"], t["ck"], dq=t["dq"],
                                 dk=t["dk"], dv=t["dv"], workspace=t["ws"], stream=0),
}
# the tensors that a call takes, and what its errors call them
NAMES = {
    "rope": dict(q="q", k="k", v="v", cs="cos_sin", pos="positions", out="q_out", ko="k_out", kc="cache keys", vc="cache values", slots="slots"),
    "rope8": dict(k8="cache keys", v8="cache values", ks="cache k_scales", vs="cache v_scales"),
    "decode": dict(q="q", kc="cache keys", vc="cache values", table="table", lens="lens", out="out", lse="lse"),
    "decode8": dict(k8="cache keys", v8="cache values", ks="cache k_scales", vs="cache v_scales"),
    "paged": dict(q="q", kc="cache keys", vc="cache values", table="table", lens="lens", cu="cu_q", out="out", lse="lse"),
    "attn": dict(q="q", k="k", v="v", cu="cu_q", ck="cu_k", out="out", lse="lse"),
    "bwd": dict(q="q", k="k", v="v", out="out", lse="lse", go="d_out", cu="cu_q", ck="cu_k", dq="dq", dk="dk", dv="dv"),
}
WRONG = {BF16: (F16, F32, U8), F32: (I32, BF16), I32: (I64, F32), I64: (I32,), E4M3: (E5M2, BF16)}                # (codes may be bytes)


@pytest.mark.parametrize("call", CALLS)
def test_right_calls_are_taken(call):
    CALLS[call](tensors())


@pytest.mark.parametrize("call,name", [(c, n) for c in CALLS for n in NAMES[c]])
def test_types(call, name):
    for dtype in WRONG[tensors()[name].dtype]:
        t = tensors()
        t[name].dtype = dtype
        with pytest.raises(ValueError, match=f"^{NAMES[call][name]} must have elements of type"):
            CALLS[call](t)


# Shapes that the errors of this very tensor, or of the one that it sets the
# shape of, are about.
SHAPES = [("rope", "q", (2, 8, 64), "q_out"), ("rope", "k", (3, 2, 32), "k"), ("rope", "v", (3, 3, 64), "v"), ("rope", "out", (3, 7, 64), "q_out"),
          ("rope", "ko", (3, 2, 48), "k_out"), ("rope", "cs", (64,), "cos_sin"), ("rope", "pos", (4,), "positions"),
          ("rope", "slots", (3, 1), "slots"), ("rope", "kc", (8, 16, 128), "cache keys"), ("rope", "vc", (8, 16, 3, 64), "cache values"),
          ("rope8", "ks", (8, 16, 1), "cache k_scales"), ("rope8", "vs", (8, 16, 2, 1), "cache v_scales"),
          ("decode", "q", (3, 8), "q"), ("decode", "out", (3, 8, 32), "out"), ("decode", "vc", (8, 16, 2, 32), "cache values"),
          ("decode", "table", (2, 4), "table"), ("decode", "table", (3,), "table"), ("decode", "lens", (2,), "lens"),
          ("decode", "lse", (8, 3), "lse"), ("decode8", "ks", (8, 2, 16), "cache k_scales"), ("decode8", "vs", (8, 16), "cache v_scales"),
          ("paged", "cu", (4, 1), "cu_q"), ("paged", "cu", (3,), "table"), ("paged", "table", (4, 4), "table"), ("paged", "lens", (4,), "lens"),
          ("paged", "out", (2, 8, 64), "out"), ("paged", "lse", (3, 7), "lse"), ("attn", "k", (3, 2, 32), "k"), ("attn", "v", (3, 3, 64), "v"),
          ("attn", "out", (3, 8, 32), "out"), ("attn", "cu", (2, 2), "cu_q"), ("attn", "ck", (3,), "cu_k"), ("attn", "lse", (8, 3), "lse"),
          ("bwd", "k", (3, 2, 32), "k"), ("bwd", "v", (3, 2, 32), "v"), ("bwd", "go", (3, 8, 32), "d_out"), ("bwd", "out", (2, 8, 64), "out"), ("bwd", "lse", (3, 7), "lse"),
          ("bwd", "dq", (3, 2, 64), "dq"), ("bwd", "dk", (3, 8, 64), "dk"), ("bwd", "dv", (4, 2, 64), "dv"), ("bwd", "ck", (5,), "cu_k"),
          ("bwd", "cu", (1, 4), "cu_q")]


@pytest.mark.parametrize("call,name,shape,about", SHAPES)
def test_shapes(call, name, shape, about):
    t = tensors()
    t[name].shape = shape
    with pytest.raises(ValueError, match=f"^{about} must have"):
        CALLS[call](t)


@pytest.mark.parametrize("call,name", [(c, n) for c in CALLS for n in NAMES[c]])
def test_tensors_of_the_host(call, name):
    t = tensors()
    t[name].is_cuda = False
    with pytest.raises(ValueError, match=f"^{NAMES[call][name]} must be a device tensor"):
        CALLS[call](t)


def test_dims_and_masks_that_do_not_fit():
    t = tensors()
    for name in ("kc", "vc"):
        t[name].shape = (8, 16, 2, 32)
    for call in ("decode", "paged"):
        with pytest.raises(ValueError, match="^the cache's dim is 32, q's 64"):
            CALLS[call](t)
    t = tensors()
    t["k"].shape = (3, 2, 32)
    with pytest.raises(ValueError, match="^k must have heads of 64, not 32"):
        CALLS["attn"](t)
    t = tensors()
    for kw in (dict(window=-1), dict(sinks=-1)):
        with pytest.raises(ValueError, match="^window and sinks must not be negative"):
            tar.prepare(tar.ar_attn, t["q"], t["k"], t["v"], t["cu"], t["ck"], t["out"], stream=0, **kw)
        with pytest.raises(ValueError, match="^window and sinks must not be negative"):
            tar.prepare(tar.ar_attn_decode, t["q"], (t["kc"], t["vc"]), t["table"], t["lens"], t["out"], stream=0, **kw)
