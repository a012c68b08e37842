"""The GPT output head, as it is measured: cases, inputs, plain forms, 64-bit values.

The head of a GPT model is a LayerNorm without a residual (the final norm), the
projection onto the vocabulary by the embedding matrix W [V, h] and the softmax
cross entropy of every token, with the gradients of all three.  Four calls:

  ln_forward     y = (x - mean) rstd gamma + beta, mean and rstd per row
  ln_backward    dx, dgamma, dbeta from dy
  loss_forward   lse[t] = log sum_v exp(z[t, v]), loss[t] = lse[t] - z[t, target[t]],
                 z = X W^T; a negative target is an ignored token, whose loss is 0
  loss_backward  dz[t, v] = dloss[t] (exp(z[t, v] - lse[t]) - [v == target[t]]),
                 0 for an ignored token; dX = dz W, dW = dz^T X

``own`` false: elementary torch operations in 32 bits.  ``own`` true: this
repository's kernels, through the calls that its users make.
"""

import math

import torch

own = False

EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}

# Hidden sizes and token counts are those of the repository's own layer
# configurations (1024 and 20480 wide, 8192 and 2048 tokens; 4096 in the
# sweep); 50257 tokens is the vocabulary of its GPT models, 51200 the same
# padded for even shards.
_LISTED = [
    # one row: the final norm of a single scored token, where latency is all
    {"name": "ln_fwd_token", "op": "ln_forward", "T": 1, "h": 4096, "dtype": "bf16"},
    # a training batch of 8 x 1024 tokens
    {"name": "ln_fwd_batch", "op": "ln_forward", "T": 8192, "h": 1024, "dtype": "bf16"},
    # rows that start at odd addresses, half precision
    {"name": "ln_fwd_odd", "op": "ln_forward", "T": 3001, "h": 2047, "dtype": "fp16"},
    # the same training batch, backward
    {"name": "ln_bwd_batch", "op": "ln_backward", "T": 8192, "h": 1024, "dtype": "bf16"},
    # the widest model's rows
    {"name": "ln_bwd_wide", "op": "ln_backward", "T": 2048, "h": 20480, "dtype": "bf16"},
    # a ragged batch kept in single precision
    {"name": "ln_bwd_fp32", "op": "ln_backward", "T": 1031, "h": 4100, "dtype": "fp32"},
    # scoring one token: the whole vocabulary matrix is read for one row
    {"name": "loss_fwd_token", "op": "loss_forward", "T": 1, "h": 1024, "V": 50257, "weights": "mean"},
    # a training batch
    {"name": "loss_fwd_batch", "op": "loss_forward", "T": 8192, "h": 1024, "V": 50257, "weights": "mean"},
    # a ragged evaluation batch over an odd vocabulary
    {"name": "loss_fwd_ragged", "op": "loss_forward", "T": 333, "h": 4096, "V": 32003, "weights": "mean"},
    # a short fine-tuning sample with a weight of its own for every token
    {"name": "loss_bwd_few", "op": "loss_backward", "T": 7, "h": 1024, "V": 50257, "weights": "tokens"},
    # a training batch
    {"name": "loss_bwd_batch", "op": "loss_backward", "T": 8192, "h": 1024, "V": 50257, "weights": "mean"},
    # the widest model's head
    {"name": "loss_bwd_wide", "op": "loss_backward", "T": 2048, "h": 20480, "V": 51200, "weights": "mean"},
]

# No drawn case does more than the largest listed one of its kind.
_LN_MOST = 2048 * 20480
_LOSS_MOST = 2048 * 20480 * 51200


def listed():
    return [dict(c) for c in _LISTED]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["ln_forward", "ln_backward", "loss_forward", "loss_backward"])
    if op.startswith("ln"):
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        h = _log_int(rng, 32, 24576)
        if rng.random() < 0.5:  # half of the widths keep whole 16-byte pieces
            h = 8 * max(1, h // 8)
        T = _log_int(rng, 1, max(1, min(32768, _LN_MOST // h)))
        return {"op": op, "T": T, "h": h, "dtype": dtype}
    h = 8 * _log_int(rng, 2, 2560)
    V = _log_int(rng, 500, 131072)
    T = _log_int(rng, 1, max(1, min(16384, _LOSS_MOST // (h * V))))
    return {"op": op, "T": T, "h": h, "V": V, "weights": rng.choice(["mean", "tokens"])}


def _ln_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, h, dt = case["T"], case["h"], DTYPES[case["dtype"]]
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    # a residual stream: rows of different size, with an offset of their own
    x = (randn(T, h) * (0.5 + 2.0 * torch.rand(T, 1, generator=g, device="cuda")) + 0.3 * randn(T, 1)).to(dt)
    gamma = (1.0 + 0.1 * randn(h)).to(dt)
    beta = (0.1 * randn(h)).to(dt)
    state = {"case": case, "x": x, "gamma": gamma, "beta": beta}
    if case["op"] == "ln_backward":
        state["dy"] = (randn(T, h) / math.sqrt(h)).to(dt)
        x64 = x.double()
        state["mean"] = x64.mean(-1).float()
        state["rstd"] = (1.0 / torch.sqrt(x64.var(-1, unbiased=False) + EPS)).float()
    return state


def _lse64(X, W):
    """log sum exp of the logits in 64 bits, some rows at a time."""
    W64, out = W.double(), []
    step = max(1, (1 << 27) // W.shape[0])
    for r in range(0, X.shape[0], step):
        out.append(torch.logsumexp(X[r:r + step].double() @ W64.t(), dim=1))
    return torch.cat(out)


def _loss_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, h, V = case["T"], case["h"], case["V"]
    std = 0.64 / math.sqrt(h)
    W = torch.empty(V, h, dtype=torch.bfloat16, device="cuda")
    W.copy_(torch.randn(V, h, generator=g, device="cuda", dtype=torch.bfloat16).mul_(std))
    targets = torch.randint(0, V, (T,), generator=g, device="cuda")
    # normalised activations that lean towards their target's row, from
    # tokens that the model knows nothing of to ones that it is sure of
    lean = torch.rand(T, 1, generator=g, device="cuda") * 20.0
    Wt = W[targets].float()
    X = torch.randn(T, h, generator=g, device="cuda") + lean * Wt / (Wt * Wt).sum(-1, keepdim=True)
    X = X.to(torch.bfloat16)
    # padding and prompt tokens do not count
    skip = torch.rand(T, generator=g, device="cuda") < 0.05
    skip[0] = False
    targets = torch.where(skip, torch.full_like(targets, -1), targets)
    state = {"case": case, "X": X, "W": W, "targets": targets}
    if case["op"] == "loss_backward":
        counted = (targets >= 0).float()
        w = counted
        if case["weights"] == "tokens":
            w = torch.rand(T, generator=g, device="cuda") * counted
        state["dloss"] = w / counted.sum()
        # what the forward pass saved
        z_lse = []
        W32 = W.float()
        step = max(1, (1 << 28) // V)
        for r in range(0, T, step):
            z_lse.append(torch.logsumexp((X[r:r + step].float() @ W32.t()).double(), dim=1))
        state["lse"] = torch.cat(z_lse).float()
    return state


def prepare(case, seed):
    return _ln_inputs(case, seed) if case["op"].startswith("ln") else _loss_inputs(case, seed)


# ------------------------------------------------------------- plain forms

def _plain_ln_forward(s):
    x = s["x"].float()
    mean = x.mean(-1)
    c = x - mean[:, None]
    rstd = torch.rsqrt((c * c).mean(-1) + EPS)
    y = c * rstd[:, None] * s["gamma"].float() + s["beta"].float()
    return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _plain_ln_backward(s):
    dy = s["dy"].float()
    rstd = s["rstd"][:, None]
    xhat = (s["x"].float() - s["mean"][:, None]) * rstd
    g = dy * s["gamma"].float()
    dx = rstd * (g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True))
    return {"dx": dx.to(s["x"].dtype), "dgamma": (dy * xhat).sum(0), "dbeta": dy.sum(0)}


def _plain_loss_forward(s):
    # loss = log(1 + sum_{v != target} exp(z_v - z_target)): where the model is
    # sure of its token, lse - z_target would be a difference of near equals
    z = s["X"].float() @ s["W"].float().t()
    counted = s["targets"] >= 0
    col = s["targets"].clamp(min=0)[:, None]
    zt = z.gather(1, col)[:, 0]
    z.scatter_(1, col, torch.where(counted, torch.full_like(zt, -math.inf), zt)[:, None])
    m = z.amax(-1, keepdim=True)
    others = m[:, 0] + torch.log(torch.exp(z - m).sum(-1))
    d = others - zt
    loss = d.clamp(min=0.0) + torch.log1p(torch.exp(-d.abs()))
    return {"loss": torch.where(counted, loss, torch.zeros_like(loss)),
            "lse": torch.where(counted, zt + loss, others)}


def _plain_loss_backward(s):
    X, W = s["X"].float(), s["W"].float()
    dz = torch.exp(X @ W.t() - s["lse"][:, None])
    rows = torch.arange(dz.shape[0], device=dz.device)
    dz[rows, s["targets"].clamp(min=0)] -= 1.0
    dz *= torch.where(s["targets"] >= 0, s["dloss"], torch.zeros_like(s["dloss"]))[:, None]
    return {"dX": (dz @ W).to(s["X"].dtype), "dW": (dz.t() @ X).to(s["W"].dtype)}


# --------------------------------------------------- this repository's calls

def _own_run(s):
    from tensor_transformer_mlp_forward_gb300 import binding

    op = s["case"]["op"]
    if op == "ln_forward":
        y, mean, rstd = binding.tp_ln_forward(s["x"], s["gamma"], s["beta"], EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "ln_backward":
        dx, dgamma, dbeta = binding.tp_ln_backward(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"])
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    if op == "loss_forward":
        loss, lse = binding.tp_head_loss_forward(s["X"], s["W"], s["targets"])
        return {"loss": loss, "lse": lse}
    dX, dW = binding.tp_head_loss_backward(s["dloss"], s["X"], s["W"], s["targets"], s["lse"])
    return {"dX": dX, "dW": dW}


_PLAIN = {"ln_forward": _plain_ln_forward, "ln_backward": _plain_ln_backward,
          "loss_forward": _plain_loss_forward, "loss_backward": _plain_loss_backward}


def run(state):
    if own:
        return _own_run(state)
    return _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("ln"):
        x = s["x"].double()
        if op == "ln_forward":
            var, mean = torch.var_mean(x, dim=1, unbiased=False)
            y = torch.addcmul(s["beta"].double(), (x - mean.unsqueeze(1)) / torch.sqrt(var + EPS).unsqueeze(1),
                              s["gamma"].double())
            return {"y": y, "mean": mean, "rstd": 1.0 / torch.sqrt(var + EPS)}
        # the chain rule through the saved mean and rstd
        n = x.shape[1]
        dy, r = s["dy"].double(), s["rstd"].double()
        c = x - s["mean"].double().unsqueeze(1)
        g = dy * s["gamma"].double()
        inner = torch.einsum("th,th->t", g, c) * r.pow(3) / n
        dx = g * r.unsqueeze(1) - (g.sum(1) * r / n).unsqueeze(1) - c * inner.unsqueeze(1)
        return {"dx": dx, "dgamma": torch.einsum("th,th,t->h", dy, c, r), "dbeta": dy.sum(0)}
    X, W, y = s["X"].double(), s["W"], s["targets"]
    T, V = X.shape[0], W.shape[0]
    counted = y >= 0
    if op == "loss_forward":
        lse = _lse64(s["X"], W)
        z_t = (X * W[y.clamp(min=0)].double()).sum(1)
        return {"loss": torch.where(counted, lse - z_t, torch.zeros_like(lse)), "lse": lse}
    # pieces of the vocabulary: softmax part by part, the target's row apart
    w = torch.where(counted, s["dloss"], torch.zeros_like(s["dloss"])).double()
    lse = s["lse"].double()
    dX = torch.zeros_like(X)
    dW = torch.empty(V, X.shape[1], dtype=torch.float64, device=X.device)
    step = max(1, (1 << 27) // T)
    for v in range(0, V, step):
        Wv = W[v:v + step].double()
        p = torch.exp(X @ Wv.t() - lse.unsqueeze(1)) * w.unsqueeze(1)
        dX += p @ Wv
        dW[v:v + step] = p.t() @ X
    wX = w.unsqueeze(1) * X
    dX -= w.unsqueeze(1) * W[y.clamp(min=0)].double()
    dW.index_add_(0, y.clamp(min=0), -wX)
    return {"dX": dX, "dW": dW}


def work(case):
    T, h = case["T"], case["h"]
    if case["op"].startswith("ln"):
        e = 4 if case["dtype"] == "fp32" else 2
        if case["op"] == "ln_forward":  # x in, y out, gamma and beta, mean and rstd
            return {"bytes": e * (2 * T * h + 2 * h) + 8 * T, "flops": 8 * T * h}
        # x and dy in, dx out, gamma, mean and rstd, dgamma and dbeta
        return {"bytes": e * (3 * T * h + h) + 8 * T + 8 * h, "flops": 14 * T * h}
    V = case["V"]
    if case["op"] == "loss_forward":  # X, W and targets in, loss and lse out; the logits
        return {"bytes": 2 * (T * h + V * h) + 8 * T + 8 * T, "flops": 2 * T * V * h}
    # X, W, targets, lse and dloss in, dX and dW out; the logits again, dX and dW
    return {"bytes": 2 * (2 * T * h + 2 * V * h) + 16 * T, "flops": 6 * T * V * h}
