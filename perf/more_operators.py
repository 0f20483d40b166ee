"""Cases of the operators at the two ends of a compressed training step: what is
timed, on which inputs, and what every result has to be.

  xent / xent_train   softmax cross entropy over a large vocabulary from hidden
        states and output weights, without keeping the logits: every token's
        loss and logarithm of the sum alone (scoring, evaluation, one token of
        a serving program), or with the gradients of the hidden states, the
        weights and the bias, scaled for the mean over the tokens that are not
        ignored
  ortho / muon        a matrix orthogonalised by five Newton-Schulz steps of a
        quintic, and the optimiser step around it over a list of matrices:
        momentum (Nesterov), orthogonalised update, decay, new weights

loss_t = log sum_v exp(x_t . w_v + b_v) - (x_t . w_y + b_y);
G_tv = softmax(l_t)_v - [v = y_t]; dx = G w / n, dw = G^T x / n, db = sum_t G_t / n
for the n tokens whose target is not -100 (the others' loss and G are zero).

X_0 = u / (||u|| + 1e-7), then five times X <- a X + (b A + c A^2) X with
A = X X^T, (a, b, c) = (3.4445, -4.7750, 2.0315).  A step: m <- mu m + g,
u = g + mu m, p <- (1 - lr wd) p - lr s X with s = sqrt(max(1, rows / cols)).
"""
from __future__ import annotations

import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2}
_ABC = (3.4445, -4.7750, 2.0315)
_STEPS = 5
_MU, _LR, _WD = 0.95, 0.02, 0.01


# ------------------------------------------------------------------ the cases
def _conv_set():
    """The matrix views (out, in * k * k) of ResNet18's weights for 32 x 32 images."""
    shapes, cin = [(64, 27)], 64
    for i, c in enumerate((64, 128, 256, 512)):
        shapes += [(c, 9 * cin), (c, 9 * c)] + ([(c, cin)] if i else []) + [(c, 9 * c)] * 2
        cin = c
    return shapes


def _text(shapes):
    """A list of matrix shapes as a case holds it."""
    return ",".join("%dx%d" % s for s in shapes)


def _shapes(case):
    return [tuple(int(n) for n in s.split("x")) for s in case["shapes"].split(",")]


def listed():
    return [
        # One token scored against the 7B-shaped set's vocabulary, as a serving
        # program does with each candidate: a reading of the weights.
        dict(name="xent_token", op="xent", t=1, v=32000, d=4096, dtype="bf16", bias=False, ignored=0.0),
        # A handful of sequences scored together.
        dict(name="xent_batch", op="xent", t=24, v=32000, d=4096, dtype="bf16", bias=False, ignored=0.0),
        # Evaluation on a micro-batch of 2048 tokens: perplexity, no gradient.
        dict(name="xent_eval", op="xent", t=2048, v=32000, d=4096, dtype="bf16", bias=False, ignored=0.0),
        # The LSTM's decoder on one of its 35 steps of 20 sequences in 16 bits:
        # rows of 650 values, the smallest training call.
        dict(name="xent_train_step", op="xent_train", t=20, v=33278, d=650, dtype="f16", bias=True, ignored=0.0),
        # The same decoder on a whole batch, 35 steps of 20 sequences, fp32.
        dict(name="xent_train_lstm", op="xent_train", t=700, v=33278, d=650, dtype="f32", bias=True, ignored=0.0),
        # The 7B-shaped head on a micro-batch of 4096 tokens, a tenth of them
        # prompt or padding.
        dict(name="xent_train_7b", op="xent_train", t=4096, v=32000, d=4096, dtype="bf16", bias=False, ignored=0.1),
        # One small matrix, the first convolution of ResNet18: launches count.
        dict(name="ortho_conv", op="ortho", rows=64, cols=27, dtype="f32"),
        # A square projection of the 7B-shaped set.
        dict(name="ortho_proj", op="ortho", rows=4096, cols=4096, dtype="bf16"),
        # The optimiser's step over ResNet18's convolutions: many small
        # matrices, wide ones, few launches.
        dict(name="muon_conv_set", op="muon", shapes=_text(_conv_set()), dtype="f32"),
        # Over the LSTM's six gate matrices: tall, sizes off every tile.
        dict(name="muon_lstm", op="muon", shapes=_text([(2600, 650)] * 6), dtype="f32"),
        # Over one layer of the 7B-shaped set, 16-bit gradients and weights.
        dict(name="muon_layer", op="muon", shapes=_text([(4096, 4096)] * 4 + [(11008, 4096)] * 2 + [(4096, 11008)]),
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _dim(rng, lo, hi):
    """A size in [lo, hi], spread over its logarithm: odd, or one of the sizes
    that the model sets have."""
    if rng.random() < 0.4:
        known = [s for s in (27, 64, 128, 512, 576, 650, 1152, 2304, 2600, 4096, 4608, 11008, 32000, 33278)
                 if lo <= s <= hi]
        if known:
            return rng.choice(known)
    return min(max(_log(rng, lo, hi) | 1, lo), hi)


def draw(rng):
    op = rng.choice(["xent", "xent_train", "xent_train", "ortho", "muon", "muon"])
    if op in ("xent", "xent_train"):
        while True:
            c = dict(op=op, t=_log(rng, 1, 4096), v=_dim(rng, 64, 33278), d=_dim(rng, 16, 4096),
                     dtype=rng.choice(["bf16", "f32", "f16"]), bias=rng.random() < 0.4,
                     ignored=rng.choice([0.0, 0.1, 0.5]))
            if c["t"] * c["v"] * c["d"] <= (1 << 36) and (c["dtype"] != "f32" or c["t"] * c["v"] * c["d"] <= (1 << 34)):
                return c
    if op == "ortho":
        return dict(op=op, rows=_dim(rng, 8, 4096), cols=_dim(rng, 8, 4608), dtype=rng.choice(["bf16", "f32", "f16"]))
    shapes, left = [], 1e12
    for _ in range(rng.randint(1, 12)):
        r, c = _dim(rng, 8, 2600), _dim(rng, 8, 4608)
        left -= min(r, c) ** 2 * max(r, c) * 2
        if left > 0:
            shapes.append((r, c))
    return dict(op=op, shapes=_text(shapes or [(33, 65)]), dtype=rng.choice(["bf16", "f32"]))


def _products(r, c):
    """Operations of the five steps: the symmetric products by half."""
    k, n = min(r, c), max(r, c)
    return _STEPS * (k * k * n + k ** 3 + 2 * k * k * n)


def work(case):
    op = case["op"]
    if op in ("xent", "xent_train"):
        t, v, d, e = case["t"], case["v"], case["d"], _SIZE[case["dtype"]]
        b = e * (t * d + v * d + (v if case["bias"] else 0)) + 16 * t
        if op == "xent":
            return {"bytes": b, "flops": 2 * t * v * d}
        return {"bytes": b + e * (t * d + v * d + (v if case["bias"] else 0)), "flops": 6 * t * v * d}
    e = _SIZE[case["dtype"]]
    if op == "ortho":
        r, c = case["rows"], case["cols"]
        return {"bytes": 2 * e * r * c, "flops": _products(r, c)}
    # gradients read, momentum and weights read and written
    n = sum(r * c for r, c in _shapes(case))
    return {"bytes": n * (e + 8 + 2 * e), "flops": sum(_products(r, c) for r, c in _shapes(case))}


# ----------------------------------------------------------------- the inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(0xC0DE + 7919 * int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _gradient_like(g, rows, cols):
    """A signal of rank 16 at most with falling singular values under noise of
    about its norm, as the compression's model sets have."""
    k = min(16, rows, cols)
    fall = torch.arange(1, k + 1, device="cuda", dtype=torch.float32) ** -1.0
    signal = (_randn(g, rows, k) * fall) @ _randn(g, k, cols)
    noise = _randn(g, rows, cols)
    return signal / signal.norm() + noise / noise.norm()


def _inputs(case, seed):
    """The tensors of a case, from the seed alone."""
    g = _gen(seed)
    op, dt = case["op"], _DT[case["dtype"]]
    if op in ("xent", "xent_train"):
        t, v, d = case["t"], case["v"], case["d"]
        # hidden states of unit variance, weights that give logits of about 2,
        # targets that the logits prefer for some of the tokens
        x = _randn(g, t, d)
        w = _randn(g, v, d) * (2.0 / math.sqrt(d))
        y = torch.randint(0, v, (t,), generator=g, device="cuda")
        x = x + (torch.rand(t, 1, generator=g, device="cuda") < 0.5) * w[y] * 1.5
        gone = torch.rand(t, generator=g, device="cuda") < case["ignored"]
        y = torch.where(gone, torch.full_like(y, -100), y)
        b = 0.5 * _randn(g, v) if case["bias"] else None
        return dict(x=x.to(dt), w=w.to(dt), y=y, b=None if b is None else b.to(dt))
    if op == "ortho":
        return dict(x=_gradient_like(g, case["rows"], case["cols"]).to(dt))
    s = dict(grads=[], momentum=[], params=[])
    for r, c in _shapes(case):
        s["grads"].append(_gradient_like(g, r, c).to(dt))
        s["momentum"].append(5.0 * _gradient_like(g, r, c))
        s["params"].append((_randn(g, r, c) / math.sqrt(c)).to(dt))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if case["op"] == "muon" and own:
        from rank_gradient_compression_amd import torch_api as T
        s["muon"] = T.Muon(s["params"], s["grads"], lr=_LR, momentum=_MU, nesterov=True, weight_decay=_WD,
                           momentum_buffers=s["momentum"])
    return s


# -------------------------------------------------------------- the plain form
def _plain_xent(s, grads):
    x, w, y, b = s["x"], s["w"], s["y"], s["b"]
    xf, wf = x.float(), w.float()
    logits = torch.matmul(xf, wf.t())
    if b is not None:
        logits += b.float()
    top = logits.max(dim=1, keepdim=True).values
    e = torch.exp(logits - top)
    total = e.sum(dim=1, keepdim=True)
    lse = (top + torch.log(total)).view(-1)
    valid = y >= 0
    at = y.clamp(min=0).view(-1, 1)
    loss = torch.where(valid, lse - logits.gather(1, at).view(-1), torch.zeros_like(lse))
    if not grads:
        return loss, lse
    scale = valid.float() / valid.sum().clamp(min=1)
    e /= total
    e.scatter_add_(1, at, torch.full_like(lse, -1.0).view(-1, 1))
    e *= scale.view(-1, 1)
    dx, dw = torch.matmul(e, wf), torch.matmul(e.t(), xf)
    out = [loss, lse, dx.to(x.dtype), dw.to(x.dtype)]
    return out if b is None else out + [e.sum(dim=0).to(x.dtype)]


def _plain_steps(u):
    a, b, c = _ABC
    x = u.float()
    x = x / (x.square().sum().sqrt() + 1e-7)
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    for _ in range(_STEPS):
        g = torch.matmul(x, x.t())
        x = a * x + torch.matmul(b * g + c * torch.matmul(g, g), x)
    return x.t() if tall else x


def _run_plain(s):
    op = s["case"]["op"]
    if op in ("xent", "xent_train"):
        return _plain_xent(s, op == "xent_train")
    if op == "ortho":
        return _plain_steps(s["x"]).to(s["x"].dtype)
    for g, m, p in zip(s["grads"], s["momentum"], s["params"]):
        gf = g.float()
        m.mul_(_MU).add_(gf)
        o = _plain_steps(gf + _MU * m)
        scale = math.sqrt(max(1.0, p.shape[0] / p.shape[1]))
        p.copy_(p.float() * (1.0 - _LR * _WD) - _LR * scale * o)
    return s["params"] + s["momentum"]


# ------------------------------------------------------ the framework's calls
def _run_own(s):
    from rank_gradient_compression_amd import torch_api as T
    op = s["case"]["op"]
    if op == "xent":
        return T.cross_entropy(s["x"], s["w"], s["y"], bias=s["b"])
    if op == "xent_train":
        loss, lse, dx, dw, db = T.cross_entropy_train(s["x"], s["w"], s["y"], bias=s["b"], reduction="mean")
        return [loss, lse, dx, dw] if s["b"] is None else [loss, lse, dx, dw, db]
    if op == "ortho":
        return T.orthogonalize(s["x"])
    s["muon"].step()
    return s["params"] + s["momentum"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# --------------------------------------------------- the definition in 64 bits
def _steps64(u):
    """The five steps as one polynomial of the Gram matrix on the shorter side:
    X_k = P_k X_0, A_k = P_k S P_k with S = X_0 X_0^T, and P_k commutes with S."""
    if u.shape[0] > u.shape[1]:
        return _steps64(u.t()).t()
    a, b, c = _ABC
    x0 = u / (torch.linalg.vector_norm(u) + 1e-7)
    s = x0 @ x0.t()
    eye = torch.eye(s.shape[0], dtype=torch.float64, device=u.device)
    p = eye
    for _ in range(_STEPS):
        g = p @ s @ p
        p = (a * eye + b * g + c * (g @ g)) @ p
    return p @ x0


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "ortho":
        return _steps64(s["x"].double())
    if op == "muon":
        params, momentum = [], []
        for g, m, p in zip(s["grads"], s["momentum"], s["params"]):
            m = _MU * m.double() + g.double()
            o = _steps64(g.double() + _MU * m)
            params.append((1.0 - _LR * _WD) * p.double() - _LR * max(1.0, p.shape[0] / p.shape[1]) ** 0.5 * o)
            momentum.append(m)
        return params + momentum
    x, w, y = s["x"].double(), s["w"].double(), s["y"]
    b = torch.zeros(w.shape[0], dtype=torch.float64, device=w.device) if s["b"] is None else s["b"].double()
    n = max(1, int((y != -100).sum()))
    losses, sums, dxs = [], [], []
    dw, db = torch.zeros_like(w), torch.zeros_like(b)
    for t0 in range(0, x.shape[0], 512):  # tokens at a time
        xs, ys = x[t0:t0 + 512], y[t0:t0 + 512]
        l = torch.addmm(b, xs, w.t())
        lse = torch.logsumexp(l, dim=1)
        keep = (ys != -100).double()
        hot = torch.nn.functional.one_hot(ys.clamp(min=0), w.shape[0]).double()
        losses.append(keep * (lse - (l * hot).sum(dim=1)))
        sums.append(lse)
        if op == "xent":
            continue
        g = (torch.exp(l - lse[:, None]) - hot) * keep[:, None] / n
        dxs.append(g @ w)
        dw += g.t() @ xs
        db += g.sum(dim=0)
    out = [torch.cat(losses), torch.cat(sums)]
    if op == "xent":
        return out
    return out + [torch.cat(dxs), dw] + ([] if s["b"] is None else [db])
