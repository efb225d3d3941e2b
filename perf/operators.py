"""Cases and plain forms of the tensor-parallel block operators.

The four operators are the steps on either side of a tensor-parallel
all-reduce:

  norm   rank contributions summed, residual added, root-mean-square norm,
         result in bf16 and / or in 8 bits with a scale for each 128 elements
  bwd    gradients of that norm: of its input and of its gain
  quant  a bf16 matrix to 8 bits, a scale for each 1 x 128 or 128 x 128
         block, as it stands or transposed
  gemm   product of two such 8-bit matrices, for one or several ranks at once

``own`` selects what ``run`` computes: False the plain form in elementary
torch operations, True the framework's kernels.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128
EPS = 1e-6
E4M3_MAX = 448.0
TINY = 2.0 ** -126


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one token of a decode step, eight ranks: the smallest message of a served model
        dict(name="norm decode 1", op="norm", P=8, rows=1, hidden=8192, out="fp8", fmt="f32"),
        # odd sizes: three contributions, rows that start on no vector boundary, the gain's bf16 result only
        dict(name="norm ragged", op="norm", P=3, rows=1001, hidden=5003, out="bf16", fmt="f32"),
        # a 16k-token prefill on eight ranks, result in 8 bits for the next projection
        dict(name="norm prefill", op="norm", P=8, rows=16384, hidden=8192, out="fp8", fmt="f32"),
        # training: a short batch, where the launches count
        dict(name="bwd short", op="bwd", rows=128, hidden=8192),
        # training: 16k tokens of the widest hidden size in use here
        dict(name="bwd long", op="bwd", rows=16384, hidden=16384),
        # activations of a ragged batch, transposed for the gradient of a weight
        dict(name="quant transposed", op="quant", rows=4097, cols=8192, brows=1, turn=True, fmt="e8m0"),
        # a weight matrix, a scale for each 128 x 128 block
        dict(name="quant weight", op="quant", rows=8192, cols=8192, brows=128, turn=False, fmt="f32"),
        # one token through a row-parallel projection, the shards of eight ranks in one call
        dict(name="gemm decode 1", op="gemm", G=8, M=1, N=8192, K=1024, brows=128, out="bf16", fmt="f32"),
        # a decode batch through a column-parallel projection
        dict(name="gemm decode 48", op="gemm", G=1, M=48, N=4096, K=8192, brows=128, out="bf16", fmt="f32"),
        # gradient of a weight: row scales on both sides, an odd number of tokens, binary32 result
        dict(name="gemm weight grad", op="gemm", G=1, M=1024, N=8192, K=4097, brows=1, out="f32", fmt="e8m0"),
        # a 16k-token prefill through a projection, binary32 scales
        dict(name="gemm prefill", op="gemm", G=1, M=16384, N=8192, K=8192, brows=128, out="bf16", fmt="f32"),
        # the same with power-of-two scales
        dict(name="gemm prefill e8m0", op="gemm", G=1, M=16384, N=8192, K=8192, brows=128, out="bf16", fmt="e8m0"),
    ]


def _size(rng, lo, hi, step=1):
    """Log-uniform in [lo, hi]; a multiple of `step` two times in three."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if step > 1 and rng.random() < 0.67:
        v = (v + step // 2) // step * step
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["norm", "bwd", "quant", "gemm", "gemm"])
    fmt = rng.choice(["f32", "e8m0"])
    if op == "norm":
        P, hidden = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 8]), _size(rng, 512, 16384, 128)
        return dict(op=op, P=P, rows=_size(rng, 1, 16384 * 8192 // hidden), hidden=hidden,
                    out=rng.choice(["bf16", "fp8", "fp8", "both"]), fmt=fmt)
    if op == "bwd":
        hidden = _size(rng, 512, 16384, 128)
        return dict(op=op, rows=_size(rng, 1, 16384), hidden=hidden)
    if op == "quant":
        return dict(op=op, rows=_size(rng, 1, 16384, 128), cols=_size(rng, 128, 8192, 128), brows=rng.choice([1, 128]),
                    turn=rng.random() < 0.5, fmt=fmt)
    M, G = _size(rng, 1, 16384), 1
    if M <= 128:
        G = rng.choice([1, 1, 8])
    N, K = _size(rng, 256, 8192, 128), _size(rng, 256, 8192, 128)
    grad = rng.random() < 0.25
    return dict(op=op, G=G, M=M, N=N, K=K, brows=1 if grad else 128, out="f32" if grad else "bf16", fmt=fmt)


def _up(a, b):
    return -(-a // b)


# --------------------------------------------------- what a program has in hand

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _acts(g, rows, cols):
    """Activations: normal values, channel gains spread log-normally (a few
    channels far above the rest)."""
    gain = torch.exp(0.7 * _normal(g, cols))
    return (_normal(g, rows, cols) * gain).to(torch.bfloat16)


def _codes_like(rows, cols):
    """An uninitialised code matrix whose rows start on 16-byte boundaries."""
    return torch.empty(rows, _up(cols, 16) * 16, device=DEV, dtype=torch.float8_e4m3fn)[:, :cols]


def _scales_like(rows, cols, brows, fmt):
    """Scales of a [rows x cols] matrix, stored block column by block column."""
    dt = torch.float32 if fmt == "f32" else torch.float8_e8m0fnu
    return torch.empty(_up(cols, BLOCK), _up(rows, brows), device=DEV, dtype=dt).t()


def _quantised(x, brows, fmt):
    """(codes, scales) of a bf16 matrix, in buffers as a program keeps them."""
    c, s = _quant_plain(x, brows, fmt)
    codes, scales = _codes_like(*x.shape), _scales_like(*x.shape, brows, fmt)
    codes.view(torch.uint8).copy_(c.view(torch.uint8))
    if fmt == "f32":
        scales.copy_(s)
    else:
        scales.view(torch.uint8).copy_(s.view(torch.uint8))
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op == "norm":
        rows, hidden = case["rows"], case["hidden"]
        s["ins"] = [(0.5 * _normal(g, rows, hidden)).to(torch.bfloat16) for _ in range(case["P"])]
        s["residual"] = _acts(g, rows, hidden)
        s["weight"] = (1 + 0.1 * _normal(g, hidden)).to(torch.bfloat16)
        s["res_out"] = torch.empty_like(s["residual"])
        s["y"] = torch.empty_like(s["residual"]) if case["out"] != "fp8" else None
        s["codes"] = _codes_like(rows, hidden) if case["out"] != "bf16" else None
        s["scales"] = _scales_like(rows, hidden, 1, case["fmt"]) if case["out"] != "bf16" else None
    elif op == "bwd":
        rows, hidden = case["rows"], case["hidden"]
        s["h"] = _acts(g, rows, hidden)
        s["dy"] = (1e-2 * _normal(g, rows, hidden)).to(torch.bfloat16)
        s["dres"] = (1e-2 * _normal(g, rows, hidden)).to(torch.bfloat16)
        s["weight"] = (1 + 0.1 * _normal(g, hidden)).to(torch.bfloat16)
        s["dx"] = torch.empty_like(s["h"])
        s["dweight"] = torch.empty(hidden, device=DEV, dtype=torch.float32)
    elif op == "quant":
        s["x"] = _acts(g, case["rows"], case["cols"])
        shape = (case["cols"], case["rows"]) if case["turn"] else (case["rows"], case["cols"])
        s["codes"] = _codes_like(*shape)
        s["scales"] = _scales_like(*shape, case["brows"], case["fmt"])
    else:
        M, N, K, G = case["M"], case["N"], case["K"], case["G"]
        a = [_quantised(_acts(g, M, K), 1, case["fmt"]) for _ in range(G)]
        b = [_quantised((0.02 * _normal(g, N, K)).to(torch.bfloat16), case["brows"], case["fmt"]) for _ in range(G)]
        s["a"], s["sa"] = [v[0] for v in a], [v[1] for v in a]
        s["b"], s["sb"] = [v[0] for v in b], [v[1] for v in b]
        dt = torch.bfloat16 if case["out"] == "bf16" else torch.float32
        s["outs"] = [torch.empty(M, N, device=DEV, dtype=dt) for _ in range(G)]
    if own:
        s["call"] = _call(s)
    return s


def _call(s):
    """The prepared call of the framework that a step loop keeps."""
    import tensor_all_reduce_amd as tar
    op = s["op"]
    if op == "norm":
        return tar.prepare(tar.ar_reduce_norm, s["ins"], s["weight"], residual=s["residual"], res_out=s["res_out"],
                           y=s["y"], codes=s["codes"], scales=s["scales"], eps=EPS)
    if op == "bwd":
        ws = torch.empty(tar.norm_bwd_workspace(s["rows"], s["hidden"]), device=DEV, dtype=torch.uint8)
        return tar.prepare(tar.ar_norm_bwd, s["dy"], s["h"], s["weight"], s["dx"], dres=s["dres"],
                           dweight=s["dweight"], workspace=ws, eps=EPS)
    if op == "quant":
        return tar.prepare(tar.ar_quantize_block, s["x"], s["codes"], s["scales"], block_rows=s["brows"],
                           transpose=s["turn"])
    ws = torch.zeros(tar.gemm_fp8_workspace(s["M"], s["N"], s["K"], s["G"]), device=DEV, dtype=torch.uint8)
    return tar.prepare(tar.ar_gemm_fp8, s["a"], s["sa"], s["b"], s["sb"], s["outs"], b_block_rows=s["brows"],
                       workspace=ws)


# ------------------------------------------------------------------- one pass

def run(s):
    op = s["op"]
    if own:
        s["call"]()
        if op == "norm":
            return {"res_out": s["res_out"], "y": s["y"], "codes": s["codes"], "scales": s["scales"]}
        if op == "bwd":
            return {"dx": s["dx"], "dweight": s["dweight"]}
        if op == "quant":
            return {"codes": s["codes"], "scales": s["scales"]}
        return s["outs"]
    if op == "norm":
        return _norm_plain(s)
    if op == "bwd":
        return _bwd_plain(s)
    if op == "quant":
        x = s["x"].t() if s["turn"] else s["x"]
        codes, scales = _quant_plain(x, s["brows"], s["fmt"])
        return {"codes": codes, "scales": scales}
    dt = s["outs"][0].dtype
    return [(_values(a, sa, 1) @ _values(b, sb, s["brows"]).t()).to(dt)
            for a, sa, b, sb in zip(s["a"], s["sa"], s["b"], s["sb"])]


def _scale_plain(amax, fmt):
    """(scale as kept, its binary32 value) from a block's largest magnitude."""
    if fmt == "f32":
        v = torch.clamp(amax / E4M3_MAX, min=TINY)
        return v, v
    # the smallest power of two 2^k, k >= -127, with amax <= 448 * 2^k
    m, e = torch.frexp(amax)                                     # amax = m * 2^e, 0.5 <= m < 1
    k = torch.where(m > 0.875, e - 8, e - 9)
    k = torch.where(amax > 0, k, torch.full_like(k, -127)).clamp(-127, 127)
    return (k + 127).to(torch.uint8).view(torch.float8_e8m0fnu), torch.ldexp(torch.ones_like(amax), k)


def _quant_plain(x, brows, fmt):
    """Codes and scales of a finite matrix, in 32 bits, rounded once."""
    rows, cols = x.shape
    R, C = _up(rows, brows), _up(cols, BLOCK)
    f = torch.zeros(R * brows, C * BLOCK, device=x.device, dtype=torch.float32)
    f[:rows, :cols] = x
    f = f.view(R, brows, C, BLOCK)
    scales, v = _scale_plain(f.abs().amax(dim=(1, 3)), fmt)
    q = (f / v[:, None, :, None]).view(R * brows, C * BLOCK)[:rows, :cols]
    return q.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scales


def _values(codes, scales, brows):
    """The binary32 matrix that codes and scales stand for."""
    rows, cols = codes.shape
    v = scales.to(torch.float32).repeat_interleave(BLOCK, 1)[:, :cols]
    if brows > 1:
        v = v.repeat_interleave(brows, 0)[:rows]
    return codes.to(torch.float32) * v


def _norm_plain(s):
    h = torch.stack(s["ins"]).sum(0, dtype=torch.float32) + s["residual"]
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["weight"]
    codes = scales = None
    if s["out"] != "bf16":
        codes, scales = _quant_plain(y, 1, s["fmt"])
    return {"res_out": h.to(torch.bfloat16), "y": y.to(torch.bfloat16) if s["out"] != "fp8" else None,
            "codes": codes, "scales": scales}


def _bwd_plain(s):
    h, dy = s["h"].float(), s["dy"].float()
    r = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    x = h * r
    g = dy * s["weight"]
    dx = s["dres"] + r * (g - x * (g * x).mean(1, keepdim=True))
    return {"dx": dx.to(torch.bfloat16), "dweight": (dy * x).sum(0)}


# ------------------------------------------------------------ work of one pass

def work(case):
    op = case["op"]
    sb = 4 if case.get("fmt") == "f32" else 1
    if op == "norm":
        n = case["rows"] * case["hidden"]
        b = 2 * n * (case["P"] + 2) + 2 * case["hidden"]
        if case["out"] != "fp8":
            b += 2 * n
        if case["out"] != "bf16":
            b += n + sb * case["rows"] * _up(case["hidden"], BLOCK)
        return {"bytes": b, "flops": n * (case["P"] + 7)}
    if op == "bwd":
        n = case["rows"] * case["hidden"]
        return {"bytes": 2 * n * 4 + 6 * case["hidden"], "flops": 12 * n}
    if op == "quant":
        n = case["rows"] * case["cols"]
        rows, cols = (case["cols"], case["rows"]) if case["turn"] else (case["rows"], case["cols"])
        return {"bytes": 3 * n + sb * _up(rows, case["brows"]) * _up(cols, BLOCK), "flops": 3 * n}
    M, N, K, G = case["M"], case["N"], case["K"], case["G"]
    kb = _up(K, BLOCK)
    b = M * K + N * K + sb * kb * (M + _up(N, case["brows"])) + (2 if case["out"] == "bf16" else 4) * M * N
    return {"bytes": G * b, "flops": 2 * G * M * N * K}


# --------------------------------------------------------- the same in 64 bits

def _exact_codes(y, brows, fmt):
    """What codes and scales would be without rounding: y / s and s."""
    rows, cols = y.shape
    R, C = _up(rows, brows), _up(cols, BLOCK)
    pad = torch.nn.functional.pad(y.abs(), (0, C * BLOCK - cols, 0, R * brows - rows))
    amax = pad.unflatten(1, (C, BLOCK)).amax(2).unflatten(0, (R, brows)).amax(1)
    if fmt == "f32":
        scale = torch.maximum(amax / 448, torch.full_like(amax, TINY))
    else:
        scale = torch.exp2(torch.ceil(torch.log2(amax / 448)).clamp(-127, 127))
    whole = scale[torch.arange(rows, device=y.device) // brows][:, torch.arange(cols, device=y.device) // BLOCK]
    return y / whole, scale


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "norm":
        h = s["residual"].double()
        for x in s["ins"]:
            h += x.double()
        y = h / torch.sqrt(h.pow(2).sum(1, keepdim=True) / case["hidden"] + EPS)
        y *= s["weight"].double()
        out = {"res_out": h, "y": y if case["out"] != "fp8" else None, "codes": None, "scales": None}
        if case["out"] != "bf16":
            out["codes"], out["scales"] = _exact_codes(y, 1, case["fmt"])
        return out
    if op == "bwd":
        # d/dh of  sum(dy * w * h / rms) + sum(dres * h)
        dx = torch.empty_like(s["h"], dtype=torch.float64)
        dw = torch.zeros(case["hidden"], device=DEV, dtype=torch.float64)
        for a in range(0, case["rows"], 2048):
            at = slice(a, a + 2048)
            h, dy = s["h"][at].double(), s["dy"][at].double()
            rms = torch.sqrt(h.pow(2).sum(1, keepdim=True) / case["hidden"] + EPS)
            gw = dy * s["weight"].double()
            dx[at] = s["dres"][at].double() + gw / rms - h * (gw * h).sum(1, keepdim=True) / (case["hidden"] * rms ** 3)
            dw += (dy * h / rms).sum(0)
        return {"dx": dx, "dweight": dw}
    if op == "quant":
        x = s["x"].double()
        codes, scales = _exact_codes(x.t() if case["turn"] else x, case["brows"], case["fmt"])
        return {"codes": codes, "scales": scales}
    res = []
    for a, sa, b, sb in zip(s["a"], s["sa"], s["b"], s["sb"]):
        acc = torch.zeros(case["M"], case["N"], device=DEV, dtype=torch.float64)
        wide = sb.to(torch.float32).double()[torch.arange(case["N"], device=DEV) // case["brows"]]
        for j in range(0, case["K"], BLOCK):
            part = a[:, j:j + BLOCK].to(torch.float32).double() @ b[:, j:j + BLOCK].to(torch.float32).double().t()
            acc += part * sa[:, j // BLOCK].to(torch.float32).double()[:, None] * wide[:, j // BLOCK][None, :]
        res.append(acc)
    return res
