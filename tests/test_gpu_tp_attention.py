"""The block's attention run together: projection, rotation and append, attention
and the way back, on simulated ranks."""
import pytest
import torch

import attn_ref as ref
import tensor_all_reduce_amd as tar
from gpu_util import note
from tensor_all_reduce_amd import tp_attention, tp_block
from test_gpu_attn_cache import spin

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def projected(a):
    """The projection's results once more, which are not overwritten."""
    res = [torch.empty_like(x) for x in a.qkv]
    tar.ar_gemm_fp8([a.normed[0]] * a.P, [a.normed[1]] * a.P, [m[0] for m in a.weights], [m[1] for m in a.weights], res,
                    workspace=a.gemm_workspace)
    return res


def turned(x, tol, a, sign=1):
    """x [tokens, heads, dim] rotated in 64 bits, with the bound that its own
    bound and one rounding leave."""
    rot = a.cos_sin.shape[1]
    y, mag = spin(x, a.cos_sin, a.positions, rot, False, sign)
    _, wide = spin(tol, a.cos_sin, a.positions, rot, False, sign)
    return y, wide + ref.U * (y.abs() + wide) + 3 * ref.E * mag


@pytest.mark.parametrize("window,sinks", [(0, 0), (24, 2)])
def test_training_step(window, sinks):
    note(f"train window {window} sinks {sinks}")
    a = tp_attention.random_attention(2, 120, 3, 256, 4, 2, 64, "train", window=window, sinks=sinks)
    raw = projected(a)
    for _ in range(2):                               # a step repeats
        a.forward()
        a.backward()
    torch.cuda.synchronize()
    cu = a.cu.tolist()
    for r in range(a.P):
        q, k, v = a.heads(a.qkv[r])
        q0, k0, v0 = a.heads(raw[r])
        for x, y in ((q, q0), (k, k0)):
            want, tol = turned(y, torch.zeros_like(y, dtype=torch.float64), a)
            ref.close(x, want, tol, "rotated")
        assert torch.equal(v, v0)
        go = a.d_attn[r].view(120, 4, 64)
        want = ref.ragged(q, k, v, cu, cu, 0.125, window, sinks, go)
        ref.close(a.attn[r].view(120, 4, 64), want["out"], want["out_t"], "attn")
        dq, dk, dv = a.heads(a.d_qkv[r])
        ref.close(dv, want["dv"], want["dv_t"], "dv")
        for x, name in ((dq, "dq"), (dk, "dk")):
            y, tol = turned(want[name], want[name + "_t"], a, -1)
            ref.close(x, y, tol, name)


@pytest.mark.parametrize("e4m3", [False, True])
def test_prompt_then_tokens(e4m3):
    """A prompt's chunks, then single tokens, over the same pages."""
    note(f"serve e4m3 {e4m3}")
    P, seqs, each, hidden, hq, hkv, dim, page = 2, 3, 20, 256, 4, 1, 128, 16
    a = tp_attention.random_attention(P, seqs * each, seqs, hidden, hq, hkv, dim, "prompt", 40, page_size=page, e4m3=e4m3)
    a.forward()
    torch.cuda.synchronize()

    def check(s, n):
        for r in range(P):
            q = s.heads(s.qkv[r])[0]
            for i in range(seqs):
                rows = slice(i * n, (i + 1) * n)
                k, v = ref.paged(s.caches[r], s.table[i], int(s.lens[i]))
                for h in range(hq):
                    want = ref.attend(q[rows, h], k[:, 0], v[:, 0], dim ** -0.5)
                    ref.close(s.attn[r].view(-1, hq, dim)[rows, h], want["out"], want["out_t"], f"rank {r} sequence {i} head {h}")
    check(a, each)
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    w = [torch.randn((hq + 2 * hkv) * dim, hidden, generator=g, device=DEV).to(torch.bfloat16) / 16 for _ in range(P)]
    t = tp_attention.TPAttention(w, hq, hkv, dim, seqs, seqs, "decode", pages=1, page_size=page, table_pages=a.table.shape[1],
                                 max_positions=200, e4m3=e4m3)
    t.caches, t.table = a.caches, a.table
    t.prepare()
    for i in range(3):
        pos = 60 + i
        tar.ar_quantize_block(torch.randn(seqs, hidden, generator=g, device=DEV).to(torch.bfloat16), *t.normed)
        t.positions.fill_(pos)
        t.lens.fill_(pos + 1)
        t.slots.copy_(t.table[:, pos // page].long() * page + pos % page)
        raw = projected(t)
        t.forward()
        torch.cuda.synchronize()
        check(t, 1)
        for r in range(P):                           # the token's own key and value are in their place
            q0, k0, v0 = t.heads(raw[r])
            want, tol = turned(k0, torch.zeros_like(k0, dtype=torch.float64), t)
            for s in range(seqs):
                k, v = ref.paged(t.caches[r], t.table[s], pos + 1)
                if e4m3:
                    step = 2.0 ** -4 + 8 * ref.E, float(want[s].abs().max()) / 448 * 2.0 ** -10
                    ref.close(k[-1], want[s], want[s].abs() * step[0] + step[1] + tol[s], "key")
                else:
                    ref.close(k[-1], want[s], tol[s], "key")
                    assert torch.equal(v[-1], v0[s].double())


def test_a_block_around_its_attention():
    """The attention fills a TPBlock's first buffers and its gradient comes from
    the block's; both steps run as one captured graph."""
    P, T, H, hq, hkv, dim, outer = 2, 48, 256, 2, 1, 64, 128
    block, _, _ = tp_block.random_block(P, T, H, hq * dim, outer, seed=2)
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    w = [torch.randn((hq + 2 * hkv) * dim, H, generator=g, device=DEV).to(torch.bfloat16) / 16 for _ in range(P)]
    a = tp_attention.TPAttention(w, hq, hkv, dim, T, 2, "train", max_positions=T, attn=block.attn)
    assert all(x is y for x, y in zip(a.attn, block.attn))
    a.positions.copy_(torch.arange(T, device=DEV) % 24)
    a.cu.copy_(torch.tensor([0, 24, 48], device=DEV))
    x = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
    tar.ar_quantize_block(x, *a.normed)

    def work():
        a.prepare()
        block.prepare()
        a.forward()
        block.forward()
    work()
    torch.cuda.synchronize()
    want = [t.clone() for t in (*block.outs, block.hidden_out, *a.attn)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    for _ in range(3):
        for t in (*block.outs, block.hidden_out, *a.attn):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for t, y in zip((*block.outs, block.hidden_out, *a.attn), want):
            assert torch.equal(t, y)


def test_refusals():
    w = [torch.zeros(256, 128, device=DEV, dtype=torch.bfloat16)]
    with pytest.raises(ValueError):
        tp_attention.TPAttention(w, 2, 1, 64, 4, 2, "decode", pages=4, table_pages=2)
    with pytest.raises(ValueError):
        tp_attention.TPAttention(w, 2, 1, 64, 4, 2, "serve")
    a = tp_attention.TPAttention(w, 2, 1, 64, 2, 2, "decode", pages=4, table_pages=2, max_positions=64)
    with pytest.raises(ValueError):
        a.backward()


@pytest.mark.parametrize("step", ["decode", "prompt", "train"])
def test_command(step, capsys):
    assert tp_attention.main(["--step", step, "--tokens", "6", "--keys", "50", "--hidden", "256", "--heads", "2", "--dim", "64",
                              "--ranks", "2", "--steps", "2", "--window", "30", "--sinks", "1"]) == 0
    assert "forward" in capsys.readouterr().out
