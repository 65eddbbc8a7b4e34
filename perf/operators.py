"""Measured cases of the operators on block-scaled 8-bit matrices.

An 8-bit matrix here is e4m3 codes with one scale for each block of 128: for activations a
block is 128 consecutive values of one row, for weights 128 x 128.  The operators make such a
matrix (quant_block), give its values back (dequant_block), multiply two of them
(gemm_block_scaled, and grouped_gemm_block_scaled with one weight matrix per group of rows),
and form a weight's gradient from activations that were kept in 8 bits (weight_grad,
grouped_weight_grad).

With ``own`` false, run() computes them from elementary torch operations in 32 bits; with
``own`` true it calls block_swizzle_tile_amd.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases ---
def listed():
    return [
        # one token's activations before an 8-bit product: latency
        dict(name="quant_token", op="quant", rows=1, cols=4096, block_rows=1, dtype="bf16"),
        # a layer's input kept for the backward pass: 16k tokens, wide
        dict(name="quant_checkpoint", op="quant", rows=16384, cols=8192, block_rows=1,
             dtype="bf16"),
        # a small restored activation with odd edges
        dict(name="dequant_small", op="dequant", rows=200, cols=136, block_rows=1, dtype="fp16"),
        # a layer's input restored in the backward pass
        dict(name="dequant_checkpoint", op="dequant", rows=8192, cols=8192, block_rows=1,
             dtype="bf16"),
        # one token through a linear layer (weights with 32-bit scales, as published)
        dict(name="gemm_token", op="gemm", M=1, N=4096, K=4096, trans_b=True, scales="f32",
             out="bf16"),
        # a few drafted tokens of several requests, odd sizes, weights stored K x N
        dict(name="gemm_drafts", op="gemm", M=33, N=4112, K=2056, trans_b=False,
             scales="mixed", out="bf16"),
        # a prompt of 1024 tokens
        dict(name="gemm_prompt", op="gemm", M=1024, N=2048, K=4096, trans_b=False,
             scales="e8m0", out="bf16"),
        # a training step's product, 32-bit scales
        dict(name="gemm_train", op="gemm", M=8192, N=8192, K=4096, trans_b=True, scales="f32",
             out="bf16"),
        # 64 tokens over 16 experts: a serving step of a mixture of experts
        dict(name="grouped_serving", op="grouped", G=16, M=64, N=2048, K=4096, trans_b=True,
             scales="mixed", out="bf16", spread=1.0),
        # 8192 tokens over 8 experts of uneven load
        dict(name="grouped_train", op="grouped", G=8, M=8192, N=4096, K=2048, trans_b=False,
             scales="e8m0", out="bf16", spread=0.5),
        # a short ragged batch in fp16: gradient of a narrow weight
        dict(name="grad_small", op="grad", G=0, M=200, K=256, N=136, dtype="fp16", out="fp32",
             accumulate=False, spread=0.0),
        # a training step's weight gradient, added to the accumulated one
        dict(name="grad_train", op="grad", G=0, M=8192, K=4096, N=4096, dtype="bf16",
             out="fp32", accumulate=True, spread=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(n, m):
    return max(m, n // m * m)


def draw(rng):
    op = rng.choice(["quant", "dequant", "gemm", "gemm", "grouped", "grad", "grad"])
    if op in ("quant", "dequant"):
        cols = _log(rng, 16, 16384)
        rows = _log(rng, 1, min(65536, 16384 * 4096 // cols))
        return dict(op=op, rows=rows, cols=cols, block_rows=rng.choice([1, 1, 128]),
                    dtype=rng.choice(["bf16", "fp16", "fp32"] if op == "quant" else
                                     ["bf16", "fp16"]))
    if op == "gemm":
        M = rng.choice([_log(rng, 1, 64), _log(rng, 1, 8192)])
        N, K = _log(rng, 64, 8192), _log(rng, 64, 8192)
        if rng.random() < 0.7:
            N, K = _mult(N, 16), _mult(K, 16)
        return dict(op=op, M=M, N=N, K=min(K, 4096), trans_b=rng.choice([True, False]),
                    scales=rng.choice(["e8m0", "f32", "mixed"]),
                    out=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    if op == "grouped":
        return dict(op=op, G=_log(rng, 1, 64), M=_log(rng, 1, 8192), N=_mult(_log(rng, 64, 4096), 8),
                    K=_mult(_log(rng, 64, 2048), 8), trans_b=rng.choice([True, False]),
                    scales=rng.choice(["e8m0", "f32", "mixed"]),
                    out=rng.choice(["bf16", "fp16"]), spread=round(rng.uniform(0, 1.5), 2))
    return dict(op=op, G=rng.choice([0, 0, _log(rng, 1, 16)]), M=_log(rng, 1, 8192),
                K=_mult(_log(rng, 64, 4096), 8), N=_mult(_log(rng, 64, 4096), 8),
                dtype=rng.choice(["bf16", "bf16", "fp16"]), out=rng.choice(["fp32", "bf16"]),
                accumulate=rng.choice([True, False]), spread=round(rng.uniform(0, 1.5), 2))


# ----------------------------------------------------------------- inputs ---
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _acts(rows, cols, g, dtype=torch.float32):
    """Activations: normal values, per-channel sizes that spread over a factor of some tens, and
    now and then a row of zeros."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= torch.exp(torch.randn(cols, generator=g, device="cuda"))
    if rows > 8:
        x[torch.randint(rows, (rows // 64 + 1,), generator=g, device="cuda")] = 0
    return x.to(dtype)


def _pad16(t):
    """The same matrix with rows of whole 16-byte chunks, as an 8-bit operand is kept."""
    p = -t.shape[-1] % 16
    if p == 0:
        return t
    v = t.view(torch.uint8)
    big = torch.zeros(*t.shape[:-1], t.shape[-1] + p, dtype=torch.uint8, device=t.device)
    big[..., : t.shape[-1]] = v
    return big.view(t.dtype)[..., : t.shape[-1]]


def _power(e):
    """2^e in 32 bits, exactly, for whole e from -126 to 127."""
    return ((e + 127) << 23).view(torch.float32)


def _codes(x, block_rows, kind):
    """8-bit codes and scales of x (2-D, or 3-D with a leading group axis)."""
    lead, (rows, cols) = x.shape[:-2], x.shape[-2:]
    rb, cb = -(-rows // block_rows), -(-cols // 128)
    p = torch.zeros(*lead, rb * block_rows, cb * 128, device=x.device)
    p[..., :rows, :cols] = x
    b = p.view(*lead, rb, block_rows, cb, 128)
    top = b.abs().amax(dim=(-3, -1), keepdim=True)
    if kind == "f32":
        s = torch.where(top > 0, top / 448, torch.ones_like(top))
    else:
        e = torch.ceil(torch.log2(torch.clamp(top, min=1e-30) / 448)).to(torch.int32)
        s = _power(e)
    q = torch.clamp(b / s, -448, 448).to(torch.float8_e4m3fn)
    q = q.view(torch.uint8).reshape(*lead, rb * block_rows, cb * 128)[..., :rows, :cols]
    s = s.reshape(*lead, rb, cb)
    if kind != "f32":
        s = (e.reshape(*lead, rb, cb) + 127).to(torch.uint8)
    return _pad16(q.contiguous().view(torch.float8_e4m3fn)), s.contiguous()


def _group_sizes(G, M, spread, seed):
    """Row counts of G groups that add up to M: loads that differ by the spread."""
    r = torch.Generator().manual_seed(int(seed) + 77)
    w = torch.exp(spread * torch.randn(G, generator=r, dtype=torch.float64))
    pick = torch.multinomial(w, M, replacement=True, generator=r)
    return torch.bincount(pick, minlength=G)


def _groups(case, seed):
    n = _group_sizes(case["G"], case["M"], case["spread"], seed)
    return n.to(torch.int32).cuda(), int(n.max())


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case=dict(case))
    if op == "quant":
        s["x"] = _acts(case["rows"], case["cols"], g, DT[case["dtype"]])
        return s
    if op == "dequant":
        s["q"], s["s"] = _codes(_acts(case["rows"], case["cols"], g), case["block_rows"], "e8m0")
        return s
    M, K, N, G = case["M"], case["K"], case["N"], case.get("G", 0)
    if op == "grad":
        s["q"], s["s"] = _codes(_acts(M, K, g), 1, "e8m0")
        n_pad = -(-N // 8) * 8
        s["dy"] = (0.01 * torch.randn(M, n_pad, generator=g, device="cuda")).to(
            DT[case["dtype"]])[:, :N]
        if G:
            s["group_m"], s["most"] = _groups(case, seed)
        if case["accumulate"]:
            shape = (G, K, N) if G else (K, N)
            s["dw"] = torch.randn(shape, generator=g, device="cuda").to(DT[case["out"]])
        return s
    sa, sb = {"e8m0": ("e8m0",) * 2, "f32": ("f32",) * 2, "mixed": ("e8m0", "f32")}[case["scales"]]
    s["a"], s["sa"] = _codes(_acts(M, K, g), 1, sa)
    shape = (N, K) if case["trans_b"] else (K, N)
    if op == "grouped":
        shape = (G,) + shape
        s["group_m"], s["most"] = _groups(case, seed)
    s["b"], s["sb"] = _codes(torch.randn(shape, generator=g, device="cuda") / math.sqrt(K), 128,
                             sb)
    return s


# ------------------------------------------------------------- plain form ---
def _scale32(s):
    return s if s.dtype == torch.float32 else s.view(torch.float8_e8m0fnu).float()


def _values(q, s, block_rows):
    """codes x scales in 32 bits."""
    rows, cols = q.shape[-2:]
    f = _scale32(s)
    if block_rows > 1:
        f = f.repeat_interleave(block_rows, -2)[..., :rows, :]
    return q.float() * f.repeat_interleave(128, -1)[..., :cols]


def _plain_quant(x, block_rows):
    rows, cols = x.shape
    rb, cb = -(-rows // block_rows), -(-cols // 128)
    p = torch.nn.functional.pad(x.float(), (0, cb * 128 - cols, 0, rb * block_rows - rows))
    b = p.view(rb, block_rows, cb, 128)
    top = torch.where(b.isfinite(), b.abs(), 0.0).amax(dim=(1, 3), keepdim=True)
    m, e = torch.frexp(top)                  # top = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(top > 0, (e - 9 + (m > 0.875)).clamp(min=-127), -127)
    q = (b * _power(-e)).to(torch.float8_e4m3fn)
    q = q.view(rb * block_rows, cb * 128)[:rows, :cols]
    return q, (e + 127).to(torch.uint8).view(rb, cb)


def _padded_rows(x, group_m, most):
    """The groups' rows as [G][most][...], zeros past a group's end, and each row's place."""
    n = group_m.long()
    first = n.cumsum(0) - n
    at = torch.arange(most, device=x.device)[None, :]
    idx = (first[:, None] + at).clamp(max=x.shape[0] - 1)
    live = at < n[:, None]
    return torch.where(live[..., None], x[idx], 0.0), idx, live


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "quant":
        q, e = _plain_quant(s["x"], c["block_rows"])
        return dict(q=q, scale=e.view(torch.float8_e8m0fnu))
    if op == "dequant":
        return dict(x=_values(s["q"], s["s"], c["block_rows"]).to(DT[c["dtype"]]))
    if op == "gemm":
        b = _values(s["b"], s["sb"], 128)
        b = b.t() if c["trans_b"] else b
        return dict(c=(_values(s["a"], s["sa"], 1) @ b).to(DT[c["out"]]))
    if op == "grouped":
        a, idx, live = _padded_rows(_values(s["a"], s["sa"], 1), s["group_m"], s["most"])
        b = _values(s["b"], s["sb"], 128)
        b = b.transpose(1, 2) if c["trans_b"] else b
        y = torch.bmm(a, b)
        out = torch.zeros(c["M"] + 1, c["N"], device=a.device)     # the last row: places past a group's end
        out[torch.where(live, idx, c["M"])] = y
        return dict(c=out[:-1].to(DT[c["out"]]))
    x, dy = _values(s["q"], s["s"], 1), s["dy"].float()
    if c["G"]:
        x = _padded_rows(x, s["group_m"], s["most"])[0]
        dy = _padded_rows(dy, s["group_m"], s["most"])[0]
        dw = torch.bmm(x.transpose(1, 2), dy)
    else:
        dw = x.t() @ dy
    if c["accumulate"]:
        dw = s["dw"].float() + dw
    return dict(dw=dw.to(DT[c["out"]]))


def _calls(s):
    import block_swizzle_tile_amd as bst
    c = s["case"]
    op = c["op"]
    if op == "quant":
        q, e = bst.quant_block(s["x"], block_rows=c["block_rows"])
        return dict(q=q, scale=e.view(torch.float8_e8m0fnu))
    if op == "dequant":
        return dict(x=bst.dequant_block(s["q"], s["s"], block_rows=c["block_rows"],
                                        out_dtype=DT[c["dtype"]]))
    if op == "gemm":
        return dict(c=bst.gemm_block_scaled(s["a"], s["b"], s["sa"], s["sb"],
                                            trans_b=c["trans_b"], out_dtype=DT[c["out"]]))
    if op == "grouped":
        return dict(c=bst.grouped_gemm_block_scaled(s["a"], s["b"], s["group_m"], s["sa"],
                                                    s["sb"], trans_b=c["trans_b"],
                                                    out_dtype=DT[c["out"]]))
    # an accumulated gradient is added into a copy, so that a pass can be called again
    kw = dict(out_dtype=DT[c["out"]])
    if c["accumulate"]:
        kw = dict(add=s["dw"])
    if c["G"]:
        return dict(dw=bst.grouped_weight_grad(s["q"], s["s"], s["dy"], s["group_m"], **kw))
    return dict(dw=bst.weight_grad(s["q"], s["s"], s["dy"], **kw))


def run(state):
    return _calls(state) if own else _plain(state)


# ------------------------------------------------------------------- work ---
def work(case):
    op = case["op"]
    es = {"bf16": 2, "fp16": 2, "fp32": 4}
    if op in ("quant", "dequant"):
        n = case["rows"] * case["cols"]
        scales = -(-case["rows"] // case["block_rows"]) * -(-case["cols"] // 128)
        return dict(bytes=n * (1 + es[case["dtype"]]) + scales, flops=2 * n)
    M, N, K, G = case["M"], case["N"], case["K"], max(1, case.get("G", 0))
    kb, nb = -(-K // 128), -(-N // 128)
    if op == "grad":
        return dict(bytes=M * K + M * kb + M * N * es[case["dtype"]]
                    + G * K * N * es[case["out"]] * (2 if case["accumulate"] else 1),
                    flops=2 * M * N * K)
    sa, sb = {"e8m0": (1, 1), "f32": (4, 4), "mixed": (1, 4)}[case["scales"]]
    used = min(G, M)    # groups that hold rows, at most
    return dict(bytes=M * K + M * kb * sa + used * (K * N + kb * nb * sb)
                + M * N * es[case["out"]], flops=2 * M * N * K)


# ------------------------------------------------------------------ exact ---
def _two_to(e):
    """2^e in 64 bits, exactly, for whole e (of any type) from -1022 to 1023."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _wide(q, s, block_rows):
    """The matrix that codes and scales stand for, in 64 bits: each element's own block looked up."""
    rows = torch.arange(q.shape[-2], device=q.device) // block_rows
    cols = torch.arange(q.shape[-1], device=q.device) // 128
    w = s.double() if s.dtype == torch.float32 else _two_to(s.long() - 127)
    return q.to(torch.float64) * w[..., rows[:, None], cols[None, :]]


def _e4m3_nearest(v):
    """The e4m3 value nearest to v (64 bits, |v| <= 448), ties to the even code."""
    a = v.abs()
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6)))
    e = torch.where(_two_to(e) > a, e - 1, e)
    e = torch.where(_two_to(e + 1) <= a, e + 1, e).clamp(min=-6)
    step = _two_to(e - 3)
    return torch.sign(v) * torch.round(a / step) * step


def _exact_quant(x, block_rows):
    rows, cols = x.shape
    rb, cb = -(-rows // block_rows), -(-cols // 128)
    v = x.double()
    mag = torch.zeros(rb * block_rows, cb * 128, dtype=torch.float64, device=x.device)
    mag[:rows, :cols] = v.abs()
    top = mag.view(rb, block_rows, cb, 128).amax(3).amax(1)
    # the smallest power of two 2^e, e >= -127, with top <= 448 2^e
    e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -200) / 448)).clamp(min=-127)
    e = torch.where(top > 448 * _two_to(e), e + 1, e)
    e = torch.where((top <= 448 * _two_to(e - 1)) & (e > -127), e - 1, e)
    scale = _two_to(e)
    r = torch.arange(rows, device=x.device) // block_rows
    k = torch.arange(cols, device=x.device) // 128
    return dict(q=_e4m3_nearest(v / scale[r[:, None], k[None, :]]), scale=scale)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "quant":
        return _exact_quant(s["x"], case["block_rows"])
    if op == "dequant":
        return dict(x=_wide(s["q"], s["s"], case["block_rows"]))
    if op == "gemm":
        b = _wide(s["b"], s["sb"], 128)
        return dict(c=torch.matmul(_wide(s["a"], s["sa"], 1), b.t() if case["trans_b"] else b))
    if op == "grouped":
        a, at, parts = _wide(s["a"], s["sa"], 1), 0, []
        for g, n in enumerate(s["group_m"].tolist()):
            b = _wide(s["b"][g], s["sb"][g], 128)
            parts.append(torch.matmul(a[at:at + n], b.t() if case["trans_b"] else b))
            at += n
        return dict(c=torch.cat(parts))
    x, dy = _wide(s["q"], s["s"], 1), s["dy"].double()
    if case["G"]:
        at, parts = 0, []
        for n in s["group_m"].tolist():
            parts.append(torch.matmul(x[at:at + n].t(), dy[at:at + n]))
            at += n
        dw = torch.stack(parts)
    else:
        dw = torch.matmul(x.t(), dy)
    return dict(dw=dw + s["dw"].double() if case["accumulate"] else dw)
