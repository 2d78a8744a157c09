"""The 8-bit integer operators, as cases that can be timed and compared.

  quantize    int8_quantize: rows of a matrix to int8 codes with one fp32 scale a row (the
              tokens of an activation, the output channels of a weight)
  matmul      int8_matmul: tokens times a weight of 8-bit rows, a scale for each token and channel
  input_grad  int8_matmul_backward: the gradient of that product for its tokens
  checkpoint  backward on Int8Rows: the NF4 layer's backward with the layer's input kept in 8 bits

A row of codes: a = max|x|, scale s = RN32(a / 127), code = the integer nearest to x / s (exact
quotient, ties to even, at most 127 in magnitude); 0 where s is 0.

`own` chooses between the elementary torch form below and the framework's calls.
"""
import math
import os
import sys

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
WEIGHT_MOST = 8192 * 28672          # weights of the largest projection
PRODUCT_MOST = 4096 * 4096 * 11008  # multiply-adds of the largest product


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the activation of one decoded token, on its way into an 8-bit product: latency
        dict(name="quantize_token", op="quantize", rows=1, cols=4096, dtype="bf16"),
        # a ragged batch kept for the backward pass, odd row length, rows inside a wider matrix
        dict(name="quantize_ragged", op="quantize", rows=1531, cols=4099, dtype="fp16", stride=4160),
        # a merged projection weight brought to 8 bits for deployment: the largest
        dict(name="quantize_weight", op="quantize", rows=28672, cols=8192, dtype="bf16"),
        # one token through a square projection: the smallest product, bound by the weight's bytes
        dict(name="matmul_decode1", op="matmul", M=1, K=4096, N=4096, dtype="bf16", rows_given=False, bias=False),
        # a decode batch through the largest up-projection
        dict(name="matmul_decode16", op="matmul", M=16, K=8192, N=28672, dtype="bf16", rows_given=False, bias=False),
        # odd in every extent, with a bias: a short ragged prompt
        dict(name="matmul_odd", op="matmul", M=333, K=1999, N=1003, dtype="fp16", rows_given=False, bias=True),
        # a training-sized batch through an up-projection whose input is already in 8 bits
        dict(name="matmul_batch", op="matmul", M=4096, K=4096, N=11008, dtype="bf16", rows_given=True, bias=False),
        # the input gradient of a short batch
        dict(name="input_grad_short", op="input_grad", M=48, K=4096, N=1000, dtype="fp16"),
        # the input gradient of the training-sized batch
        dict(name="input_grad_batch", op="input_grad", M=4096, K=4096, N=11008, dtype="bf16"),
        # the layer's backward from an 8-bit checkpoint: a small square projection, T recomputed
        dict(name="checkpoint_square", op="checkpoint", M=512, K=2048, N=2048, r=16, pool=1, dtype="fp16", saved_T=False),
        # the pooled adapter on a ragged batch
        dict(name="checkpoint_pooled", op="checkpoint", M=1000, K=4096, N=4096, r=24, pool=64, dtype="bf16", saved_T=True),
        # the training-sized up-projection
        dict(name="checkpoint_batch", op="checkpoint", M=4096, K=4096, N=11008, r=64, pool=1, dtype="bf16", saved_T=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "matmul", "matmul", "input_grad", "checkpoint"])
    if op == "quantize":
        cols = _log(rng, 64, 28672)
        rows = _log(rng, 1, max(1, min(28672, WEIGHT_MOST // cols)))
        return dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    if op == "checkpoint":
        K, N = 64 * _log(rng, 4, 172), 8 * _log(rng, 32, 1376)
        M = _log(rng, 1, max(1, min(4096, PRODUCT_MOST // (K * N))))
        return dict(op=op, M=M, K=K, N=N, r=_log(rng, 4, 128), pool=rng.choice([1, 1, 64]),
                    dtype=rng.choice(["bf16", "fp16"]), saved_T=rng.random() < 0.5)
    K = _log(rng, 128, 28672)
    N = _log(rng, 128, max(128, min(28672, WEIGHT_MOST // K)))
    if rng.random() < 0.5:
        K, N = K // 16 * 16, N // 16 * 16
    M = _log(rng, 1, max(1, min(8192, PRODUCT_MOST // (K * N))))
    if op == "input_grad":
        return dict(op=op, M=M, K=K, N=N, dtype=rng.choice(["bf16", "fp16"]))
    return dict(op=op, M=M, K=K, N=N, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                rows_given=rng.random() < 0.3, bias=rng.random() < 0.3)


def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (e + 1) + 4 * case["rows"], "flops": 3 * n}
    M, K, N = case["M"], case["K"], case["N"]
    if case["op"] == "matmul":
        x = M * (K + 4) if case["rows_given"] else e * M * K
        return {"bytes": x + N * (K + 4) + e * M * N + (e * N if case["bias"] else 0), "flops": 2 * M * N * K}
    if case["op"] == "input_grad":
        return {"bytes": e * M * (K + N) + N * (K + 4), "flops": 2 * M * N * K}
    r, Ka = case["r"], K // case["pool"]
    nb = N * K // 64
    weight = N * K // 2 + nb + 4 * ((nb + 255) // 256)
    adapters = (Ka + N) * r
    flops = 2 * M * N * K + 2 * M * r * (2 * N + 2 * Ka + (0 if case["saved_T"] else Ka))
    return {"bytes": M * (K + 4) + e * M * (K + N) + weight + e * adapters + 4 * adapters
            + (4 * M * r if case["saved_T"] else 0), "flops": flops}


# ------------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 11)
    return g


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _activation(g, rows, cols, dtype):
    """Normal features, some of them an order of magnitude larger, as hidden states have them,
    under a level of each token's own; one token is all zero where there are many."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= 1 + 9 * (torch.rand(cols, generator=g, device="cuda") < 0.003)
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=g, device="cuda"))
    if rows > 64:
        x[rows // 3] = 0
    return x.to(dtype)


def _quantize_rows(x):
    """(codes int8 with rows padded to 16 bytes, scales fp32) by the definition."""
    rows, cols = x.shape
    codes = torch.zeros(rows, (cols + 15) // 16 * 16, dtype=torch.int8, device=x.device)
    v = x.float()
    scale = v.abs().amax(1) / torch.full((1,), 127.0, device=x.device)
    # the quotient in 64 bits: x / s of two fp32 numbers is never nearer than 2^-33 (relative) to a
    # border between two codes without being on it
    q = v.double() / scale.double()[:, None]
    q = torch.where(scale[:, None] > 0, q, torch.zeros_like(q)).round().clamp(-127, 127)
    codes[:, :cols] = q.to(torch.int8)
    return codes[:, :cols], scale


def _nf4_levels():
    d = 1 - (1 / 32 + 1 / 30) / 2
    inv = lambda p: torch.special.ndtri(torch.tensor(p, dtype=torch.float64))  # noqa: E731
    top = inv(d)
    neg = [-inv(d + (0.5 - d) * i / 7) / top for i in range(7)]
    pos = [inv(d + (0.5 - d) * i / 8) / top for i in range(7, -1, -1)]
    return torch.stack(neg + [torch.zeros((), dtype=torch.float64)] + pos).float()


def _nf4_weight(g, rows, cols, levels):
    """(packed nibbles, 8-bit codes of the block scales, one fp32 step for 256 of them)."""
    w = _randn(g, rows * cols // 64, 64) * 0.02
    a = w.abs().amax(1)
    lev = levels.cuda()
    idx = torch.bucketize(w / a[:, None], (lev[1:] + lev[:-1]) / 2).to(torch.uint8).reshape(-1, 2)
    packed = (idx[:, 0] << 4) | idx[:, 1]
    nb = a.numel()
    groups = torch.zeros((nb + 255) // 256 * 256, device="cuda")
    groups[:nb] = a
    step = groups.reshape(-1, 256).amax(1) / torch.full((1,), 255.0, device="cuda")
    codes = (a / step.repeat_interleave(256)[:nb]).round().to(torch.uint8)
    return packed, codes, step


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=dict(case))
    dt = DTYPES[case["dtype"]]
    if case["op"] == "quantize":
        wide = _activation(g, case["rows"], case.get("stride", case["cols"]), dt)
        s["x"] = wide[:, :case["cols"]]
        return s
    M, K, N = case["M"], case["K"], case["N"]
    if case["op"] == "checkpoint":
        r, Ka = case["r"], K // case["pool"]
        s["levels"] = _nf4_levels()
        s["packed"], s["codes"], s["step"] = _nf4_weight(g, N, K, s["levels"])
        s["alpha"] = 2.0 * r
        x = _activation(g, M, K, dt)
        s["x8"], s["xs"] = _quantize_rows(x)
        s["dy"] = _randn(g, M, N, dtype=dt)
        s["A"] = (_randn(g, Ka, r) / math.sqrt(r)).to(dt)
        s["B"] = (_randn(g, r, N) * 0.01).to(dt)
        u = x.float().reshape(M, Ka, case["pool"]).mean(2)
        s["T"] = u @ s["A"].float() if case["saved_T"] else None
        return s
    s["w8"], s["ws"] = _quantize_rows(_randn(g, N, K) * 0.02)
    if case["op"] == "input_grad":
        s["dy"] = _activation(g, M, N, dt)
        return s
    x = _activation(g, M, K, dt)
    s["x"] = x
    if case["rows_given"]:
        s["x8"], s["xs"] = _quantize_rows(x)
    s["bias"] = _randn(g, N, dtype=dt) if case["bias"] else None
    return s


# ------------------------------------------------------------------------------------ one pass
def _framework():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    if root not in sys.path:
        sys.path.insert(0, root)
    import bit_nf4_quantized_22_b200 as q
    return q


def _run_own(s):
    q = _framework()
    case = s["case"]
    if case["op"] == "quantize":
        r = q.int8_quantize(s["x"])
        return {"codes": r.codes, "scales": r.scales}
    if case["op"] == "matmul":
        w = q.Int8Rows(s["w8"], s["ws"])
        x = q.Int8Rows(s["x8"], s["xs"]) if case["rows_given"] else s["x"]
        return {"y": q.int8_matmul(x, w, bias=s["bias"], dtype=s["x"].dtype)}
    if case["op"] == "input_grad":
        return {"dx": q.int8_matmul_backward(s["dy"], q.Int8Rows(s["w8"], s["ws"]))}
    w = q.NF4Weight(case["N"], case["K"], True, s["packed"], codes=s["codes"], steps=s["step"],
                    compute_dtype=DTYPES[case["dtype"]])
    dx, da, db = q.backward(q.Int8Rows(s["x8"], s["xs"]), s["dy"], w, s["A"], s["B"], s["alpha"],
                            pool_group=case["pool"], T=s["T"], codebook=s["levels"])
    return {"dx": dx, "dA": da, "dB": db}


def _run_plain(s):
    case = s["case"]
    if case["op"] == "quantize":
        codes, scales = _quantize_rows(s["x"])
        return {"codes": codes, "scales": scales}
    dt = DTYPES[case["dtype"]]
    if case["op"] == "matmul":
        x8, xs = (s["x8"], s["xs"]) if case["rows_given"] else _quantize_rows(s["x"])
        y = (x8.float() @ s["w8"].float().t()) * xs[:, None] * s["ws"][None, :]
        if s["bias"] is not None:
            y = y + s["bias"].float()
        return {"y": y.to(dt)}
    if case["op"] == "input_grad":
        return {"dx": (s["dy"].float() @ (s["w8"].float() * s["ws"][:, None])).to(dt)}
    K, N, g = case["K"], case["N"], case["pool"]
    byte = s["packed"]
    idx = torch.stack([byte >> 4, byte & 15], 1).reshape(-1, 64).long()
    scale = s["codes"].float() * s["step"].repeat_interleave(256)[:s["codes"].numel()]
    # the layer's weight is the dequantized one in the compute dtype
    w = (s["levels"].cuda()[idx] * scale[:, None]).to(dt).reshape(N, K).float()
    dy, A, B = s["dy"].float(), s["A"].float(), s["B"].float()
    u = (s["x8"].float() * s["xs"][:, None]).reshape(-1, K // g, g).mean(2)
    T = s["T"] if s["T"] is not None else u @ A
    f = s["alpha"] / case["r"]
    G = dy @ B.t()
    dx = dy @ w + (f / g) * (G @ A.t()).repeat_interleave(g, 1)
    return {"dx": dx.to(dt), "dA": f * (u.t() @ G), "dB": f * (T.t() @ dy)}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------------------ 64 bits
def _codes64(x):
    """Codes by comparison with the borders between them, apart from _quantize_rows: the number of
    half-odd multiples of the scale below |x|, the even code on a border."""
    v = x.double()
    top = v.abs().amax(1)
    s = (top / torch.full((1,), 127.0, dtype=torch.float64, device=x.device)).float().double()
    m, s1 = v.abs(), s[:, None]
    c = torch.floor(m / torch.where(s1 > 0, s1, torch.ones_like(s1)))
    rest = m - c * s1
    up = (2 * rest > s1) | ((2 * rest == s1) & (c % 2 == 1))
    c = torch.where(s1 > 0, torch.clamp(c + up, max=127.0), torch.zeros_like(c))
    return torch.sign(v) * c, s


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        return {"codes": None, "scales": _codes64(s["x"])[1]}
    if case["op"] == "matmul":
        if case["rows_given"]:
            x = torch.einsum("mk,m->mk", s["x8"].double(), s["xs"].double())
        else:
            c, sc = _codes64(s["x"])
            x = torch.einsum("mk,m->mk", c, sc)
        y = torch.einsum("mk,nk->mn", x, torch.einsum("nk,n->nk", s["w8"].double(), s["ws"].double()))
        return {"y": y if s["bias"] is None else y + s["bias"].double()[None]}
    if case["op"] == "input_grad":
        return {"dx": torch.einsum("mn,nk->mk", torch.einsum("mn,n->mn", s["dy"].double(), s["ws"].double()),
                                   s["w8"].double())}
    K, N, g, r = case["K"], case["N"], case["pool"], case["r"]
    level = s["levels"].cuda()
    nib = torch.empty(N * K, dtype=torch.int64, device="cuda")
    nib[0::2] = s["packed"].long() // 16
    nib[1::2] = s["packed"].long() % 16
    block = torch.arange(N * K // 64, device="cuda")
    a = s["codes"].float() * s["step"][block // 256]
    w = torch.take(level, nib).reshape(-1, 64).mul_(a[:, None]).to(DTYPES[case["dtype"]]).double().reshape(N, K)
    del nib
    A = s["A"].double().repeat_interleave(g, 0) / g      # the pooled adapter, one row a feature
    B, dy = s["B"].double(), s["dy"].double()
    x = torch.einsum("mk,m->mk", s["x8"].double(), s["xs"].double())
    f = s["alpha"] / r
    G = torch.einsum("mn,jn->mj", dy, B)
    T = torch.einsum("mk,kj->mj", x, A) if s["T"] is None else s["T"].double()
    dx = torch.einsum("mn,nk->mk", dy, w).add_(torch.einsum("mj,kj->mk", G, A), alpha=f)
    dA = f * torch.einsum("mk,mj->kj", x, G).reshape(K // g, g, r).mean(1)
    return {"dx": dx, "dA": dA, "dB": f * torch.einsum("mj,mn->jn", T, dy)}
