"""Cases and plain forms of the attention between two projections.

The operators take a block from the result of its query, key and value
projection to the input of its output projection:

  append  queries and keys rotated by their positions, keys and values put
          into the pages of a cache, as bf16 or as E4M3 with a scale for each
          token and head
  decode  attention of one new token a sequence over that cache
  attn    attention of ragged prompts, over matrices of keys and values or
          over the cache; a sliding window and a few first tokens that stay
          visible (sinks)
  train   the same with its gradients: of queries, keys and values

``own`` selects what ``run`` computes: False the plain form in elementary
torch operations, True the framework's kernels.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
TINY = 2.0 ** -126
THETA = 10000.0


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one token of a decode step, all heads of a block of hidden size 8192: the smallest call
        dict(name="append decode 1", op="append", tokens=1, hq=64, hkv=8, dim=128, rot=128, pairs=False, fmt="bf16",
             page=16, skip=0.0),
        # odd sizes: part of each head rotated in neighbouring pairs, padded rows, pages of 48 tokens in 8 bits
        dict(name="append ragged", op="append", tokens=1003, hq=12, hkv=4, dim=96, rot=64, pairs=True, fmt="e4m3",
             page=48, skip=0.1),
        # a 16k-token prompt
        dict(name="append prompt", op="append", tokens=16384, hq=64, hkv=8, dim=128, rot=128, pairs=False, fmt="bf16",
             page=16, skip=0.0),
        # one sequence early in its answer: latency counts
        dict(name="decode 1", op="decode", seqs=1, least=700, most=700, hq=64, hkv=8, dim=128, fmt="bf16", page=16,
             window=0, sinks=0),
        # a served batch of very different lengths
        dict(name="decode batch", op="decode", seqs=48, least=100, most=16384, hq=64, hkv=8, dim=128, fmt="bf16", page=16,
             window=0, sinks=0),
        # few long contexts in an 8-bit cache
        dict(name="decode long", op="decode", seqs=8, least=120000, most=131072, hq=64, hkv=8, dim=128, fmt="e4m3",
             page=64, window=0, sinks=0),
        # next chunks of ragged prompts, earlier tokens in an 8-bit cache, window and sinks
        dict(name="attn chunks", op="attn", seqs=7, least=1, most=700, past=1500, hq=16, hkv=4, dim=64, fmt="e4m3",
             page=48, window=512, sinks=4),
        # a 16k-token prompt, causal, all heads of a block
        dict(name="attn prompt", op="attn", seqs=1, least=16384, most=16384, past=0, hq=64, hkv=8, dim=128, fmt="rows",
             page=0, window=0, sinks=0),
        # a long document with a window and sinks, the heads of one rank of eight
        dict(name="attn window", op="attn", seqs=1, least=32768, most=32768, past=0, hq=8, hkv=1, dim=128, fmt="rows",
             page=0, window=4096, sinks=4),
        # training on a few short sequences, odd lengths
        dict(name="train ragged", op="train", seqs=5, least=1, most=511, hq=6, hkv=2, dim=64, window=128, sinks=2),
        # training on two long sequences, causal, all heads of a block
        dict(name="train long", op="train", seqs=2, least=4096, most=4096, hq=64, hkv=8, dim=128, window=0, sinks=0),
        # a long document with a window and sinks, the heads of one rank of eight
        dict(name="train window", op="train", seqs=1, least=16384, most=16384, hq=8, hkv=1, dim=128, window=2048, sinks=4),
    ]


def _size(rng, lo, hi):
    """Log-uniform in [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "attn", "train"])
    dim = rng.choice([64, 64, 80, 96, 112, 128, 128, 128, 128])
    hkv = rng.choice([1, 2, 3, 4, 8, 8])
    hq = hkv * rng.choice([1, 2, 4, 5, 8, 8])
    page = rng.choice([16, 16, 32, 48, 64, 128])
    fmt = rng.choice(["bf16", "bf16", "e4m3"])
    windowed = rng.random() < 0.5
    window, sinks = (_size(rng, 64, 4096), rng.choice([0, 1, 4, 4, 16])) if windowed else (0, 0)
    if op == "append":
        rot = rng.choice([dim, dim, 32, 64])
        return dict(op=op, tokens=_size(rng, 1, 16384), hq=hq, hkv=hkv, dim=dim, rot=rot, pairs=rng.random() < 0.4,
                    fmt=fmt, page=page, skip=rng.choice([0.0, 0.1]))
    if op == "decode":
        seqs = _size(rng, 1, 64)
        most = _size(rng, 64, min(131072, 1048576 // seqs))
        return dict(op=op, seqs=seqs, least=_size(rng, 1, most), most=most, hq=hq, hkv=hkv, dim=dim, fmt=fmt, page=page,
                    window=window, sinks=sinks)
    if op == "attn":
        tokens = _size(rng, 16, 16384)
        seqs = min(_size(rng, 1, 8), tokens)
        most = tokens // seqs
        fmt = rng.choice(["rows", "rows", "bf16", "e4m3"])
        return dict(op=op, seqs=seqs, least=_size(rng, 1, most), most=most, past=0 if fmt == "rows" else _size(rng, 1, 4096),
                    hq=hq, hkv=hkv, dim=dim, fmt=fmt, page=0 if fmt == "rows" else page, window=window, sinks=sinks)
    tokens = _size(rng, 16, 8192)
    seqs = min(_size(rng, 1, 8), tokens)
    most = tokens // seqs
    return dict(op=op, seqs=seqs, least=_size(rng, 1, most), most=most, hq=hq, hkv=hkv, dim=dim, window=window, sinks=sinks)


def _lengths(case):
    """Lengths of the sequences, spread evenly over the logarithm from `least`
    to `most`, longest neither first nor last."""
    n, lo, hi = case["seqs"], case["least"], case["most"]
    if n == 1:
        return [hi]
    v = [int(round(lo * (hi / lo) ** (i / (n - 1)))) for i in range(n)]
    return v[1::2] + v[0::2][::-1]


def _up(a, b):
    return -(-a // b)


# --------------------------------------------------- what a program has in hand

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _heads(g, tokens, heads, dim, gain=0.0):
    """[tokens, heads, dim]: normal values, channel gains spread log-normally."""
    x = _normal(g, tokens, heads, dim)
    if gain:
        x *= torch.exp(gain * _normal(g, heads, dim))
    return x.to(torch.bfloat16)


def _offsets(lengths):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return torch.tensor(at, device=DEV, dtype=torch.int32)


def _table(g, lengths, page):
    """Pages of the sequences: every page once, in no order; (page table, pages)."""
    need = [_up(n, page) for n in lengths]
    order = torch.randperm(sum(need), generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lengths), max(need)), -1, device=DEV, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return table, sum(need)


def _cache(g, pages, page, heads, dim, fmt):
    """(keys, values) [pages, page, heads, dim], and in 8 bits their scales."""
    if fmt == "bf16":
        return tuple((_normal(g, pages, page, heads, dim)).to(torch.bfloat16) for _ in range(2))
    codes = tuple((100 * _normal(g, pages, page, heads, dim)).clamp(-448, 448).to(torch.float8_e4m3fn) for _ in range(2))
    scales = tuple(0.01 * torch.exp(0.3 * _normal(g, pages, page, heads)) for _ in range(2))
    return codes + scales


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case)
    op, hq, hkv, dim = case["op"], case["hq"], case["hkv"], case["dim"]
    s["scale"] = dim ** -0.5
    if op == "append":
        n, page = case["tokens"], case["page"]
        # one projection's result: the heads of a token lie side by side
        rows = _heads(g, n, hq + 2 * hkv, dim, 0.5)
        s["q"], s["k"], s["v"] = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
        s["q_out"] = torch.empty(n, hq, dim, device=DEV, dtype=torch.bfloat16)
        pages = _up(n, page) + 3
        s["cache"] = _cache(g, pages, page, hkv, dim, case["fmt"])
        slots = torch.randperm(pages * page, generator=g, device=DEV)[:n] if n < 2 * page else torch.arange(n, device=DEV) + page
        s["slots"] = torch.where(torch.rand(n, generator=g, device=DEV) < case["skip"], -1, slots)
        far = 32768
        s["positions"] = torch.randint(0, far - n, (1,), generator=g, device=DEV).to(torch.int32) + torch.arange(
            n, device=DEV, dtype=torch.int32)
        freq = THETA ** (-torch.arange(0, case["rot"], 2, device=DEV, dtype=torch.float64) / case["rot"])
        angle = torch.arange(far, device=DEV, dtype=torch.float64)[:, None] * freq
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    elif op == "decode":
        lengths = _lengths(case)
        s["q"] = _heads(g, case["seqs"], hq, dim, 0.5)
        s["table"], pages = _table(g, lengths, case["page"])
        s["cache"] = _cache(g, pages, case["page"], hkv, dim, case["fmt"])
        s["lens"] = torch.tensor(lengths, device=DEV, dtype=torch.int32)
        s["out"] = torch.empty(case["seqs"], hq, dim, device=DEV, dtype=torch.bfloat16)
    else:
        lengths = _lengths(case)
        n = sum(lengths)
        s["q"] = _heads(g, n, hq, dim, 0.5)
        s["cu_q"] = _offsets(lengths)
        s["out"] = torch.empty(n, hq, dim, device=DEV, dtype=torch.bfloat16)
        if case.get("fmt", "rows") == "rows":
            s["k"], s["v"] = _heads(g, n, hkv, dim), _heads(g, n, hkv, dim)
        else:
            lens = [v + case["past"] for v in lengths]
            s["table"], pages = _table(g, lens, case["page"])
            s["cache"] = _cache(g, pages, case["page"], hkv, dim, case["fmt"])
            s["lens"] = torch.tensor(lens, device=DEV, dtype=torch.int32)
        if op == "train":
            s["d_out"] = (0.1 * _normal(g, n, hq, dim)).to(torch.bfloat16)
            s["lse"] = torch.empty(hq, n, device=DEV, dtype=torch.float32).t()
            s["dq"], s["dk"], s["dv"] = (torch.empty_like(s[x]) for x in "qkv")
    if own:
        s["calls"] = _calls(s)
    return s


def _calls(s):
    """The prepared calls of the framework that a step loop keeps."""
    import tensor_all_reduce_amd as tar
    op, hq, hkv, dim = s["op"], s["hq"], s["hkv"], s["dim"]
    if op == "append":
        return [tar.prepare(tar.ar_rope_kv, s["q"], s["k"], s["v"], s["cos_sin"], s["positions"], q_out=s["q_out"],
                            cache=s["cache"], slots=s["slots"], pairs=s["pairs"])]
    mask = dict(scale=s["scale"], window=s["window"], sinks=s["sinks"])
    if op == "decode":
        ws = torch.zeros(tar.attn_decode_workspace(s["seqs"], hq, hkv, dim), device=DEV, dtype=torch.uint8)
        return [tar.prepare(tar.ar_attn_decode, s["q"], s["cache"], s["table"], s["lens"], s["out"], workspace=ws, **mask)]
    if op == "attn":
        if s["fmt"] != "rows":
            return [tar.prepare(tar.ar_attn_paged, s["q"], s["cache"], s["table"], s["lens"], s["cu_q"], s["out"], **mask)]
        return [tar.prepare(tar.ar_attn, s["q"], s["k"], s["v"], s["cu_q"], s["cu_q"], s["out"], **mask)]
    n = s["q"].shape[0]
    ws = torch.empty(tar.attn_bwd_workspace(n, n, s["seqs"], hq, hkv, dim, window=s["window"], sinks=s["sinks"]),
                     device=DEV, dtype=torch.uint8)
    return [tar.prepare(tar.ar_attn, s["q"], s["k"], s["v"], s["cu_q"], s["cu_q"], s["out"], lse=s["lse"], **mask),
            tar.prepare(tar.ar_attn_bwd, s["q"], s["k"], s["v"], s["out"], s["lse"], s["d_out"], s["cu_q"], s["cu_q"],
                        dq=s["dq"], dk=s["dk"], dv=s["dv"], workspace=ws, **mask)]


# ------------------------------------------------------------------- one pass

def run(s):
    op = s["op"]
    if own:
        for call in s["calls"]:
            call()
        if op == "append":
            return {"q_out": s["q_out"], "cache": s["cache"]}
        if op == "train":
            return {x: s[x] for x in ("out", "lse", "dq", "dk", "dv")}
        return {"out": s["out"]}
    if op == "append":
        return _append_plain(s)
    if op == "decode":
        return {"out": _decode_plain(s)}
    return _attn_plain(s)


def _rotate(x, s, dtype):
    """[tokens, heads, dim] rotated by the positions' angles."""
    rot, half = s["rot"], s["rot"] // 2
    rows = s["cos_sin"][s["positions"].long()].to(dtype)
    c, n = rows[:, None, :half], rows[:, None, half:]
    x = x.to(dtype)
    y = x.clone()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if s["pairs"] else (x[..., :half], x[..., half:rot])
    u, w = a * c - b * n, b * c + a * n
    if s["pairs"]:
        y[..., 0:rot:2], y[..., 1:rot:2] = u, w
    else:
        y[..., :half], y[..., half:rot] = u, w
    return y


def _append_plain(s):
    page, cache = s["page"], s["cache"]
    kept = s["slots"] >= 0
    at = s["slots"][kept]
    at = (at // page, at % page)
    for i, x in enumerate((_rotate(s["k"], s, torch.float32), s["v"].float())):
        x = x[kept]
        if s["fmt"] == "bf16":
            cache[i].index_put_(at, x.to(torch.bfloat16))
            continue
        scale = torch.clamp(x.abs().amax(2) / E4M3_MAX, min=TINY)
        codes = (x / scale[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        cache[i].view(torch.uint8).index_put_(at, codes.view(torch.uint8))
        cache[2 + i].index_put_(at, scale)
    return {"q_out": _rotate(s["q"], s, torch.float32).to(torch.bfloat16), "cache": cache}


def _gather(s, i, dtype):
    """Keys and values of sequence i out of the cache, [heads, length, dim]."""
    n, page = int(s["lengths"][i]), s["page"]
    pages = s["table"][i, :_up(n, page)].long()
    res = []
    for j in range(2):
        x = s["cache"][j][pages].to(dtype)
        if s["fmt"] == "e4m3":
            x = x * s["cache"][2 + j][pages].to(dtype)[..., None]
        res.append(x.flatten(0, 1)[:n].transpose(0, 1))
    return res


def _visible(first, count, keys, s):
    """[count, keys]: which keys the queries at positions first ... see."""
    p = torch.arange(first, first + count, device=DEV)[:, None]
    j = torch.arange(keys, device=DEV)[None, :]
    seen = j <= p
    if s["window"]:
        seen &= (j > p - s["window"]) | (j < s["sinks"])
    return seen


def _decode_plain(s):
    """The softmax of one query over a whole sequence, sequence by sequence."""
    out = torch.empty_like(s["out"])
    group = s["hq"] // s["hkv"]
    s["lengths"] = _lengths(s)
    for i, n in enumerate(s["lengths"]):
        k, v = _gather(s, i, torch.float32)
        q = s["q"][i].float().view(s["hkv"], group, s["dim"])
        x = (q @ k.transpose(1, 2)) * s["scale"]
        x = x.masked_fill(~_visible(n - 1, 1, n, s), -math.inf)
        x = torch.exp(x - x.amax(2, keepdim=True))
        out[i] = ((x @ v) / x.sum(2, keepdim=True)).view(s["hq"], s["dim"]).to(torch.bfloat16)
    return out


def _attn_plain(s):
    """Sequence by sequence, head by head, a few thousand queries at a time;
    with gradients for a training step."""
    train = s["op"] == "train"
    group, lengths = s["hq"] // s["hkv"], _lengths(s)
    s["lengths"] = [n + s.get("past", 0) for n in lengths]
    out = torch.empty_like(s["out"])
    res = {"out": out}
    if train:
        lse = torch.empty_like(s["lse"])
        dq = torch.empty_like(s["q"])
        dk, dv = (torch.zeros(s[x].shape, device=DEV, dtype=torch.float32) for x in "kv")
    at = 0
    for i, n in enumerate(lengths):
        total = s["lengths"][i]
        rows = slice(at, at + n)
        if s.get("fmt", "rows") == "rows":
            keys, values = (s[x][rows].float().transpose(0, 1) for x in "kv")
        else:
            keys, values = _gather(s, i, torch.float32)
        for c in range(0, n, 4096):
            m = min(4096, n - c)
            piece = slice(at + c, at + c + m)
            hidden = ~_visible(total - n + c, m, total, s)
            for h in range(s["hq"]):
                k, v = keys[h // group], values[h // group]
                q = s["q"][piece, h].float()
                x = ((q @ k.t()) * s["scale"]).masked_fill_(hidden, -math.inf)
                top = x.amax(1, keepdim=True)
                x = x.sub_(top).exp_()
                total_x = x.sum(1, keepdim=True)
                x /= total_x
                o = x @ v
                out[piece, h] = o.to(torch.bfloat16)
                if train:
                    lse[piece, h] = (top + total_x.log())[:, 0]
                    do = s["d_out"][piece, h].float()
                    d = (do @ v.t()).sub_((do * o).sum(1, keepdim=True)).mul_(x)
                    dq[piece, h] = ((d @ k) * s["scale"]).to(torch.bfloat16)
                    dk[rows, h // group] += (d.t() @ q) * s["scale"]
                    dv[rows, h // group] += x.t() @ do
        at += n
    if train:
        res.update(lse=lse, dq=dq, dk=dk.to(torch.bfloat16), dv=dv.to(torch.bfloat16))
    return res


# ------------------------------------------------------------ work of one pass

def _pairs(first, count, window, sinks):
    """How many keys the queries at positions first ... first + count - 1 see."""
    def upto(p):                                     # of positions 0 ... p - 1
        if not window or p <= window:
            return p * (p + 1) // 2
        far = p - window                             # queries with keys out of their window
        most = min(sinks, far)                       # sinks among those: 1, 2, ... then all
        return window * (window + 1) // 2 + far * window + most * (most + 1) // 2 + (far - most) * most
    return upto(first + count) - upto(first)


def work(case):
    op, hq, hkv, dim = case["op"], case["hq"], case["hkv"], case["dim"]
    small = case.get("fmt") == "e4m3"
    key = 2 * hkv * (dim + 4) if small else 4 * hkv * dim     # a token's keys and values in the cache
    if op == "append":
        n = case["tokens"]
        return {"bytes": n * (4 * hq * dim + 4 * hkv * dim + key + 4 * case["rot"] + 12), "flops": 3 * n * case["rot"] * (hq + hkv)}
    lengths = _lengths(case)
    window, sinks = case["window"], case["sinks"]
    if op == "decode":
        seen = sum(_pairs(n - 1, 1, window, sinks) for n in lengths)
        pages = sum(_up(n, case["page"]) for n in lengths)
        return {"bytes": seen * key + 4 * pages + case["seqs"] * (4 * hq * dim + 4), "flops": 4 * seen * hq * dim}
    past, n = case.get("past", 0), sum(lengths)
    pairs = sum(_pairs(past, m, window, sinks) for m in lengths)
    if op == "attn":
        # of the earlier tokens, those that a first query of the chunk sees
        if not window or past + 1 <= window:
            seen = sum(past + m for m in lengths)
        else:
            seen = sum(m + window - 1 + min(sinks, past + 1 - window) for m in lengths)
        return {"bytes": 4 * n * hq * dim + seen * key, "flops": 4 * pairs * hq * dim}
    # forward: q, k, v read, out and lse written; backward: those and d_out read, the gradients written
    return {"bytes": n * (hq * (14 * dim + 8) + hkv * 12 * dim), "flops": 14 * pairs * hq * dim}


# --------------------------------------------------------- the same in 64 bits

def _exact_codes(x):
    scale = torch.maximum(x.abs().amax(2) / 448, torch.full_like(x[:, :, 0], TINY))
    return x / scale[:, :, None], scale


def _exact_append(s):
    tokens, rot, page = s["tokens"], s["rot"], s["page"]
    half = rot // 2
    turn = s["cos_sin"][s["positions"].long()].double()
    turn = torch.complex(turn[:, :half], turn[:, half:])[:, None]

    def spin(x):
        x = x.double().clone()
        if s["pairs"]:
            z = torch.view_as_complex(x[..., :rot].reshape(tokens, -1, half, 2).contiguous()) * turn
            x[..., :rot] = torch.view_as_real(z).flatten(2)
        else:
            z = torch.complex(x[..., :half], x[..., half:rot]) * turn
            x[..., :rot] = torch.cat([z.real, z.imag], 2)
        return x

    cache = [c.double() for c in s["cache"]]
    flat = [c.view(-1, *c.shape[2:]) for c in cache]
    rows = torch.nonzero(s["slots"] >= 0)[:, 0]
    slots = s["slots"][rows]
    for i, x in enumerate((spin(s["k"]), s["v"].double())):
        if s["fmt"] == "bf16":
            flat[i][slots] = x[rows]
        else:
            flat[i][slots], flat[2 + i][slots] = _exact_codes(x[rows])
    return {"q_out": spin(s["q"]), "cache": tuple(cache)}


def exact(case, seed):
    s = prepare(case, seed)
    op, hkv, dim = case["op"], case["hkv"], case["dim"]
    if op == "append":
        return _exact_append(s)
    group = case["hq"] // hkv
    lengths = _lengths(case)
    past = case.get("past", 0)
    if op == "decode":
        lengths, past, starts = [1] * len(lengths), [n - 1 for n in lengths], range(len(lengths))
    else:
        starts, past = [sum(lengths[:i]) for i in range(len(lengths))], [past] * len(lengths)
    q_all = s["q"].double()
    out = torch.zeros_like(q_all)
    train = op == "train"
    if train:
        lse = torch.zeros(q_all.shape[:2], device=DEV, dtype=torch.float64)
        grads = [torch.zeros(s[x].shape, device=DEV, dtype=torch.float64) for x in "qkv"]
    for i, n in enumerate(lengths):
        a, total = starts[i], past[i] + n
        for h in range(hkv):
            # keys and values of the head, each looked up by its position
            if "cache" in s:
                j = torch.arange(total, device=DEV)
                at = (s["table"][i].long()[j // case["page"]], j % case["page"])
                k, v = (s["cache"][x][:, :, h][at].double() for x in range(2))
                if case["fmt"] == "e4m3":
                    k, v = (y * s["cache"][2 + x][:, :, h][at].double()[:, None] for x, y in enumerate((k, v)))
            else:
                k, v = (s[x][a:a + n, h].double() for x in "kv")
            for c in range(0, n, 2048):
                m = min(2048, n - c)
                w0 = 0 if not case["window"] or case["sinks"] else max(0, past[i] + c - case["window"] + 1)
                w1 = past[i] + c + m                     # keys w0 ... w1 - 1 are looked at
                p = torch.arange(past[i] + c, past[i] + c + m, device=DEV)
                j = torch.arange(w0, w1, device=DEV)
                away = p[:, None] - j[None, :]
                ok = away >= 0
                if case["window"]:
                    ok = ok & ((away < case["window"]) | (j < case["sinks"])[None, :])
                for head in range(h * group, (h + 1) * group):
                    q = q_all[a + c:a + c + m, head]
                    e = torch.matmul(q, k[w0:w1].t()) * s["scale"]
                    e = torch.where(ok, e, torch.full_like(e, -math.inf))
                    z = torch.logsumexp(e, 1)
                    e = torch.exp(e - z[:, None])
                    o = torch.matmul(e, v[w0:w1])
                    out[a + c:a + c + m, head] = o
                    if train:
                        lse[a + c:a + c + m, head] = z
                        do = s["d_out"][a + c:a + c + m, head].double()
                        grads[2][a + w0:a + w1, h] += torch.matmul(e.t(), do)
                        # d softmax: e (de - sum of e de)
                        de = torch.matmul(do, v[w0:w1].t())
                        e = s["scale"] * e * (de - (e * de).sum(1, keepdim=True))
                        grads[0][a + c:a + c + m, head] = torch.matmul(e, k[w0:w1])
                        grads[1][a + w0:a + w1, h] += torch.matmul(e.t(), q)
    if train:
        return {"out": out, "lse": lse, "dq": grads[0], "dk": grads[1], "dv": grads[2]}
    return {"out": out}
