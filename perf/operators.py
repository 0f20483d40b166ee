"""Cases of the gradient-clipping and microscaled 4-bit operators: what is
timed, on which inputs, and what every result has to be.

Three groups, the order in which a training or serving program meets them:

  linear / train / factors   the products of microscaled 4-bit operands (MXFP4:
        OCP E2M1 values in blocks of 32 along the summed axis, one E8M0 power
        of two per block): a linear layer's forward on weights that are laid
        out once, a whole training pass of such a layer (forward, the input's
        gradient, the weight's gradient), and the reconstruction of a gradient
        matrix from two 4-bit low-rank factors
  quant                      quantisation of a gradient or a factor, with the
        values that the codes stand for (what error feedback subtracts)
  clip                       the global norm over many tensors and the clipped
        gradients, written into the flat buffer that the compression reads

The scale of a block is 2^k with k the smallest integer for which the block's
largest magnitude is at most 6 * 2^k (k >= -127); a value becomes the nearest
of 0, 0.5, 1, 1.5, 2, 3, 4, 6 times 2^k, ties to the even code, or, with one
random byte r per value, the upper neighbour where the fraction between its
neighbours, times 256, is above r + 0.5.
"""
from __future__ import annotations

import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2}
_BLOCK = 32


# ------------------------------------------------------------------ the cases
def _lstm_sizes():
    s = [33278 * 650]
    for _ in range(3):
        s += [2600 * 650, 2600 * 650, 2600, 2600]
    return s + [33278]


def _transformer_sizes(layers):
    s = [32000 * 4096]
    for _ in range(layers):
        s += [4096 * 4096] * 4 + [11008 * 4096] * 3 + [4096, 4096]
    return s + [32000 * 4096]


def _text(sizes):
    """A list of tensor sizes as a case holds it."""
    return ",".join(str(n) for n in sizes)


def _sizes(case):
    return [int(n) for n in case["sizes"].split(",")]


def listed():
    return [
        # One generated token through the widest projection of the 7B-shaped set.
        dict(name="linear_token", op="linear", m=1, k=4096, n=11008, dtype="bf16"),
        # A handful of sequences decoded together, the down projection (long sum).
        dict(name="linear_batch", op="linear", m=24, k=11008, n=4096, dtype="bf16"),
        # A prompt, or one forward micro-batch, of 4096 tokens.
        dict(name="linear_prompt", op="linear", m=4096, k=4096, n=11008, dtype="bf16"),
        # Training pass of one LSTM gate matrix: 35 steps of 20 sequences, every
        # size off the tiles' multiples, fp32.
        dict(name="train_lstm", op="train", m=700, k=650, n=2600, dtype="f32", stochastic=False),
        # Training pass of a 7B-shaped projection on 2048 tokens, the incoming
        # gradient rounded stochastically.
        dict(name="train_proj", op="train", m=2048, k=4096, n=11008, dtype="bf16", stochastic=True),
        # Receiver's side of a 4-bit payload: the dense gradient from rank-64
        # and from rank-4 factors (a write of the matrix, hardly a product).
        dict(name="factors_r64", op="factors", m=11008, n=4096, rank=64),
        dict(name="factors_r4", op="factors", m=33278, n=650, rank=4),
        # Payload of one rank-4 factor: four columns, the smallest call.
        dict(name="quant_factor", op="quant", rows=4, cols=11008, dtype="f32", stochastic=False),
        # A whole gradient matrix in 4 bits: the LSTM's embedding (rows that are
        # no multiple of a block or of 16 bytes) and the 7B embedding.
        dict(name="quant_embed_lstm", op="quant", rows=33278, cols=650, dtype="f32", stochastic=True),
        dict(name="quant_embed_7b", op="quant", rows=32000, cols=4096, dtype="bf16", stochastic=False),
        # Global norm and clipping: the LSTM's set (clipping is part of its
        # training recipe), and two layers plus both embeddings of the 7B set
        # with bf16 gradients gathered into the fp32 flat buffer.
        dict(name="clip_lstm", op="clip", sizes=_text(_lstm_sizes()), dtype="f32", out="f32"),
        dict(name="clip_7b", op="clip", sizes=_text(_transformer_sizes(2)), dtype="bf16", out="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _dim(rng, lo, hi):
    """A size in [lo, hi], spread over its logarithm: odd, or one of the sizes
    that the model sets have."""
    if rng.random() < 0.4:
        known = [s for s in (32, 64, 128, 512, 576, 650, 1152, 2304, 2600, 4096, 4608, 11008) if lo <= s <= hi]
        if known:
            return rng.choice(known)
    return min(max(_log(rng, lo, hi) | 1, lo), hi)


def draw(rng):
    op = rng.choice(["linear", "linear", "train", "factors", "quant", "quant", "clip", "clip"])
    if op == "linear":
        m = _log(rng, 1, 4096)
        return dict(op=op, m=m, k=_dim(rng, 16, 11008), n=_dim(rng, 16, 11008),
                    dtype=rng.choice(["bf16", "f32", "f16"]))
    if op == "train":
        while True:
            c = dict(op=op, m=_log(rng, 1, 2048), k=_dim(rng, 16, 11008), n=_dim(rng, 16, 11008),
                     dtype=rng.choice(["bf16", "f32"]), stochastic=rng.random() < 0.5)
            if c["m"] * c["k"] * c["n"] <= 2048 * 4096 * 11008:
                return c
    if op == "factors":
        return dict(op=op, m=_dim(rng, 64, 11008), n=_dim(rng, 27, 4608), rank=rng.randint(1, 64))
    if op == "quant":
        return dict(op=op, rows=_log(rng, 1, 32000), cols=_dim(rng, 1, 4608),
                    dtype=rng.choice(["f32", "bf16", "f16"]), stochastic=rng.random() < 0.4)
    total = _log(rng, 1000, 300_000_000)
    n = rng.randint(1, 80)
    cuts = [rng.random() ** 3 + 1e-4 for _ in range(n)]
    sizes = [max(1, int(total * c / sum(cuts))) for c in cuts]
    return dict(op=op, sizes=_text(sizes), dtype=rng.choice(["f32", "bf16", "f16"]), out=rng.choice(["f32", "bf16"]))


def work(case):
    op = case["op"]
    if op == "linear":
        # activations read, 4-bit weights and their scales read, result written
        m, n, k, e = case["m"], case["n"], case["k"], _SIZE[case["dtype"]]
        return {"bytes": e * m * k + n * k / 2 + n * k / _BLOCK + e * m * n, "flops": 2 * m * n * k}
    if op == "train":
        # x, w and dy read, y and both gradients written; three products
        m, n, k, e = case["m"], case["n"], case["k"], _SIZE[case["dtype"]]
        b = e * (m * k + n * k + m * n) + e * (m * n + m * k) + 4 * n * k
        return {"bytes": b + (m * n if case["stochastic"] else 0), "flops": 6 * m * n * k}
    if op == "factors":
        m, n, r = case["m"], case["n"], case["rank"]
        return {"bytes": 4 * r * (m + n) + 4 * m * n, "flops": 2 * m * n * r}
    if op == "quant":
        n, e = case["rows"] * case["cols"], _SIZE[case["dtype"]]
        codes = case["rows"] * (-(-case["cols"] // _BLOCK)) * 17
        return {"bytes": 2 * e * n + codes + (n if case["stochastic"] else 0), "flops": 4 * n}
    n = sum(_sizes(case))
    return {"bytes": n * (_SIZE[case["dtype"]] + _SIZE[case["out"]]), "flops": 3 * n}


# ----------------------------------------------------------------- the inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(0x5EED + 7919 * int(seed))
    return g


def _gradient_like(rows, cols, dtype, g):
    """Normal entries whose rows differ in scale, a few entries far out, as a
    gradient's or an activation's do."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= torch.exp(torch.randn(rows, 1, generator=g, device="cuda"))
    far = torch.rand(rows, cols, generator=g, device="cuda") < 1e-3
    return torch.where(far, 20.0 * x, x).to(dtype)


def _bytes(rows, cols, g):
    return torch.randint(0, 256, (rows, cols), generator=g, device="cuda", dtype=torch.uint8)


def _inputs(case, seed):
    """The tensors of a case, from the seed alone."""
    g = _gen(seed)
    op = case["op"]
    if op in ("linear", "train"):
        m, k, n, dt = case["m"], case["k"], case["n"], _DT[case["dtype"]]
        d = dict(x=_gradient_like(m, k, dt, g), w=(0.02 * torch.randn(n, k, generator=g, device="cuda")).to(dt))
        if op == "train":
            d["dy"] = (1e-3 * _gradient_like(m, n, torch.float32, g)).to(dt)
            d["rand"] = _bytes(m, n, g) if case["stochastic"] else None
        return d
    if op == "factors":
        m, n, r = case["m"], case["n"], case["rank"]
        # P_hat has orthonormal columns (entries of order m^-1/2); Q's columns fall off
        fall = torch.arange(1, r + 1, device="cuda", dtype=torch.float32) ** -1.5
        return dict(p=torch.randn(m, r, generator=g, device="cuda") / math.sqrt(m),
                    q=torch.randn(n, r, generator=g, device="cuda") * fall)
    if op == "quant":
        rows, cols = case["rows"], case["cols"]
        x = (1e-3 * _gradient_like(rows, cols, torch.float32, g)).to(_DT[case["dtype"]])
        return dict(x=x, rand=_bytes(rows, cols, g) if case["stochastic"] else None)
    dt = _DT[case["dtype"]]
    return dict(grads=[(1e-3 * torch.randn(s, generator=g, device="cuda")).to(dt) for s in _sizes(case)])


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    op = case["op"]
    if op == "linear":
        # serving: the weights were laid out when the model was loaded
        if own:
            from rank_gradient_compression_amd import torch_api as T
            s["w"] = T.mx_quantize(s["w"])
        else:
            s["w"] = _round_blocks(s["w"])
    elif op == "quant":
        s["values"] = torch.empty_like(s["x"])
    elif op == "clip":
        # the flat buffer of the compression: every tensor starts at a multiple of 64 elements
        offs, end = [], 0
        for n in _sizes(case):
            offs.append(end)
            end += -(-n // 64) * 64
        flat = torch.zeros(end, dtype=_DT[case["out"]], device="cuda")
        s["outs"] = [flat[o:o + n] for o, n in zip(offs, _sizes(case))]
        s["max_norm"] = 0.5 * 1e-3 * math.sqrt(sum(_sizes(case)))
        if own:
            from rank_gradient_compression_amd import torch_api as T
            s["clip"] = T.GradientClip(s["grads"], s["outs"])
    return s


# -------------------------------------------------------------- the plain form
def _pow2(k):
    """2^k in fp32, exactly, for -126 <= k <= 127."""
    return ((k.to(torch.int32) + 127) << 23).view(torch.float32)


def _round_blocks(x, rand=None):
    """The 4-bit values of x in fp32, blocks of 32 along the last axis."""
    rows, cols = x.shape
    pad = -cols % _BLOCK
    v = torch.nn.functional.pad(x.float(), (0, pad)).view(rows, -1, _BLOCK)
    amax = v.abs().amax(dim=2, keepdim=True)
    f, e = torch.frexp(amax)
    k = torch.where(f <= 0.75, e - 3, e - 2)
    k = torch.where(amax > 0, k, torch.full_like(k, -127)).clamp(min=-127)
    a = v.abs() * _pow2(-k)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    if rand is None:
        r = torch.round(a / step)  # ties to even
    else:
        u = torch.nn.functional.pad(rand.float(), (0, pad)).view(rows, -1, _BLOCK)
        low = torch.floor(a / step)
        r = low + ((a / step - low) * 256 > u + 0.5).float()
    v = torch.copysign(r * step * 0.5 * _pow2(k + 1), v)  # 2^-127 alone is no normal number
    return v.view(rows, cols + pad)[:, :cols].contiguous()


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "linear":
        return torch.matmul(_round_blocks(s["x"]), s["w"].t()).to(s["x"].dtype)
    if op == "train":
        x, w, dy, rand = s["x"], s["w"], s["dy"], s["rand"]
        y = torch.matmul(_round_blocks(x), _round_blocks(w).t())
        wt = _round_blocks(w.t())
        dx = torch.matmul(_round_blocks(dy, rand), wt.t())
        dyt = _round_blocks(dy.t(), None if rand is None else rand.t())
        dw = torch.matmul(dyt, _round_blocks(x.t()).t())
        return y.to(x.dtype), dx.to(x.dtype), dw
    if op == "factors":
        return torch.matmul(_round_blocks(s["p"]), _round_blocks(s["q"]).t())
    if op == "quant":
        s["values"].copy_(_round_blocks(s["x"], s["rand"]))
        return s["values"]
    sq = torch.stack([g.float().square().sum() for g in s["grads"]])
    norm = sq.sum().sqrt()
    coef = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    for g, o in zip(s["grads"], s["outs"]):
        o.copy_(g.float() * coef)
    return [torch.cat([norm.view(1), coef.view(1), sq.sqrt()])] + s["outs"]


# ------------------------------------------------------ the framework's calls
def _run_own(s):
    from rank_gradient_compression_amd import torch_api as T
    op = s["case"]["op"]
    if op == "linear":
        return T.mx_linear(s["x"], s["w"])
    if op == "train":
        y, saved = T.mx_linear_forward(s["x"], s["w"])
        dx, dw = T.mx_linear_backward(s["dy"], saved, rand=s["rand"])
        return y, dx, dw
    if op == "factors":
        return T.mx_product(T.mx_quantize(s["p"]), T.mx_quantize(s["q"]))
    if op == "quant":
        T.mx_quantize(s["x"], rand=s["rand"], values=s["values"])
        return s["values"]
    return [s["clip"].clip(s["max_norm"])] + s["outs"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# --------------------------------------------------- the definition in 64 bits
def _mx64(x, axis, rand=None):
    """Microscaled values of a matrix in float64, blocks along `axis`, straight
    from the definition: the block's exponent from its largest magnitude, then
    a search among the eight magnitudes."""
    if axis == 0:
        return _mx64(x.t(), 1, None if rand is None else rand.t()).t()
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=x.device)
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    per = max(1, (1 << 25) // max(1, x.shape[1]))  # rows at a time
    for r0 in range(0, x.shape[0], per):
        blk = x[r0:r0 + per].double()
        rnd = None if rand is None else rand[r0:r0 + per].double()
        rows, cols = blk.shape
        nb = (cols + _BLOCK - 1) // _BLOCK
        full = torch.zeros(rows, nb * _BLOCK, dtype=torch.float64, device=x.device)
        full[:, :cols] = blk
        top = full.view(rows, nb, _BLOCK).abs().max(dim=2).values
        k = torch.ceil(torch.log2(top.clamp(min=2.0 ** -200) / 6.0))
        # the logarithm may be off by one next to a power of two
        k = torch.where(top <= 6.0 * torch.exp2(k - 1), k - 1, k)
        k = torch.where(top > 6.0 * torch.exp2(k), k + 1, k).clamp(min=-127.0)
        unit = torch.exp2(k).repeat_interleave(_BLOCK, dim=1)[:, :cols]
        a = blk.abs() / unit
        hi = torch.searchsorted(grid, a.contiguous()).clamp(max=7)  # first magnitude >= a
        lo = (hi - 1).clamp(min=0)
        glo, ghi = grid[lo], grid[hi]
        frac = torch.where(hi > 0, (a - glo) / (ghi - glo).clamp(min=0.5), torch.ones_like(a))
        if rnd is None:
            even_hi = (hi % 2) == 0
            up = (frac > 0.5) | ((frac == 0.5) & even_hi)
        else:
            up = (frac * 256.0 > rnd + 0.5) | (a == ghi)
        out[r0:r0 + per] = torch.where(up, ghi, glo) * unit * torch.sign(blk)
    return out


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "linear":
        return _mx64(s["x"], 1) @ _mx64(s["w"], 1).t()
    if op == "train":
        y = _mx64(s["x"], 1) @ _mx64(s["w"], 1).t()
        dx = _mx64(s["dy"], 1, s["rand"]) @ _mx64(s["w"], 0)
        dw = _mx64(s["dy"], 0, s["rand"]).t() @ _mx64(s["x"], 0)
        return y, dx, dw
    if op == "factors":
        return _mx64(s["p"], 1) @ _mx64(s["q"], 1).t()
    if op == "quant":
        return _mx64(s["x"], 1, s["rand"])
    sq = [float((g.double() ** 2).sum()) for g in s["grads"]]
    norm = math.sqrt(math.fsum(sq))
    limit = 0.5 * 1e-3 * math.sqrt(sum(_sizes(case)))
    coef = min(1.0, limit / (norm + 1e-6))
    stats = torch.tensor([norm, coef] + [math.sqrt(v) for v in sq], dtype=torch.float64, device="cuda")
    return [stats] + [g.double() * coef for g in s["grads"]]
