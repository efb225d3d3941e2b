"""Calls of more work items than a launch has (2^32 a dimension) are refused,
not left to the launch (CPU only: nothing here gets past its checks)."""
import pytest

import tensor_all_reduce_amd as tar
from test_attn_abi import A, UNS, attn, bwd, decode, hm, kv, rope


@pytest.mark.parametrize("dim,lanes", [(128, 8), (80, 8), (64, 4), (48, 4), (32, 2)])
def test_rotation(dim, lanes):
    """A head has `lanes` work items."""
    heads = 10                                       # 8 of queries, 2 of keys
    tokens = -(-(2 ** 32 // lanes) // heads)
    step = heads * dim
    kw = dict(hq=8, hkv=2, dim=dim, rot=16, v=None, cache=None, slots=None)
    far = 2 ** 50
    kw.update(cs=3 * far, pos=4 * far)
    assert rope(tokens=tokens, q=hm(2 * far, step, dim), qo=hm(2 * far, step, dim), k=hm(far, step, dim), ko=hm(far, step, dim), **kw) == UNS


def test_prompts():
    step, far = 64 * 128, 2 ** 50
    assert attn(seqs=2 ** 17, rq=2 ** 17, hq=64, q=hm(A, step), out=hm(far, step), cq=3 * far, ck=4 * far, k=hm(2 * far), v=hm(5 * far)) == UNS
    rows = 2 ** 25
    assert attn(seqs=1, rq=rows, hq=64, q=hm(A, step), out=hm(far, step), cq=3 * far, ck=4 * far, k=hm(2 * far), v=hm(5 * far)) == UNS


def test_gradients():
    step, far = 64 * 128, 2 ** 50
    at = dict(q=hm(far, step), o=hm(2 * far, step), go=hm(3 * far, step), dq=hm(4 * far, step), lse=5 * far, cq=6 * far, ck=7 * far,
              k=hm(8 * far), v=hm(9 * far), dk=hm(10 * far), dv=hm(11 * far), ws=12 * far)
    assert bwd(seqs=2 ** 17, rq=2 ** 17, hq=64, **at) == UNS
    # of the join alone: few query heads, many keys
    few = dict(q=hm(far), o=hm(2 * far), go=hm(3 * far), dq=hm(4 * far))
    assert bwd(seqs=1, rq=10, rk=2 ** 26, hq=4, hkv=1, window=10, sinks=1, **{**at, **few, "k": hm(8 * far, 128), "v": hm(9 * far, 128),
               "dk": hm(10 * far, 128), "dv": hm(11 * far, 128)}) == UNS


def test_single_tokens_without_a_workspace():
    far = 2 ** 50
    seqs, cache = 2 ** 22, kv(k=2 * far, v=3 * far)  # 2 key heads
    kw = dict(cache=cache, seqs=seqs, q=hm(far), out=hm(4 * far), table=5 * far, lens=6 * far, tp=1, ts=1)
    assert decode(**kw) == UNS
    need = tar.attn_decode_workspace(seqs, 8, 2, 128)
    assert decode(**kw, ws=7 * far, wb=need - 1) == UNS
