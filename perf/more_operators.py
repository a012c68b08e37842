"""Packed attention with grouped heads, normed and rotated queries and keys, and
gradient clipping, as they are measured: cases, inputs, plain forms, 64-bit values.

What a training step of a GPT model with grouped key/value heads adds to a
layer whose sequences all have one length.  Five calls:

  qk_forward    y = R(p) (x rstd gamma), rstd = 1 / sqrt(mean(x^2) + eps) over
                each head of the queries and keys; R(p) turns the pairs
                (i, i + rot / 2) by the angle p theta^(-2 i / rot)
  qk_backward   its gradients dQ, dK, dgamma_q, dgamma_k
  attn_forward  causal softmax attention of every sequence of a packed batch;
                query head j reads key/value head j / (nh / nkv); O and lse =
                log2 sum_k exp(scale q.k)
  attn_backward dQ, dK, dV from dO and the saved O and lse
  clip          the norm of all gradients together, and each gradient times
                min(1, max_norm / (norm + 1e-6))

``own`` false: elementary torch operations in 32 bits (angles in 64).  ``own``
true: this repository's kernels, through the calls that its users make.
"""

import math
import random

import torch

own = False

EPS = 1e-5
THETA = 10000.0
MAX_NORM = 1.0
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}

# Head dims are those of the repository's attention block (64, 96, 128, 160);
# token counts those of its layer configurations (8 x 1024 and 2048) and
# longer; the clipped layers are 4096 wide, as in its sweep.
_LISTED = [
    # a prompt of one token
    {"name": "attn_fwd_token", "op": "attn_forward", "T": 1, "nb": 1, "cut": 0, "nh": 32, "nkv": 8, "d": 128},
    # a training batch of 8 x 1024 tokens
    {"name": "attn_fwd_batch", "op": "attn_forward", "T": 8192, "nb": 8, "cut": 0, "nh": 32, "nkv": 8, "d": 128},
    # documents of every length packed into one row of tokens, a head of its own for every query head
    {"name": "attn_fwd_packed", "op": "attn_forward", "T": 8191, "nb": 37, "cut": 1, "nh": 20, "nkv": 20, "d": 64},
    # one long document
    {"name": "attn_fwd_long", "op": "attn_forward", "T": 16384, "nb": 1, "cut": 0, "nh": 16, "nkv": 2, "d": 128},
    # the training batch, backward
    {"name": "attn_bwd_batch", "op": "attn_backward", "T": 8192, "nb": 8, "cut": 0, "nh": 32, "nkv": 8, "d": 128},
    # packed documents, backward, the widest heads
    {"name": "attn_bwd_packed", "op": "attn_backward", "T": 6007, "nb": 23, "cut": 2, "nh": 16, "nkv": 4, "d": 160},
    # one token, where latency is all
    {"name": "qk_fwd_token", "op": "qk_forward", "T": 1, "nb": 1, "cut": 0, "nh": 32, "nkv": 8, "d": 128,
     "rot": 128, "dtype": "bf16"},
    # the training batch
    {"name": "qk_fwd_batch", "op": "qk_forward", "T": 8192, "nb": 8, "cut": 0, "nh": 32, "nkv": 8, "d": 128,
     "rot": 128, "dtype": "bf16"},
    # the training batch, backward
    {"name": "qk_bwd_batch", "op": "qk_backward", "T": 8192, "nb": 8, "cut": 0, "nh": 32, "nkv": 8, "d": 128,
     "rot": 128, "dtype": "bf16"},
    # a ragged batch in half precision, heads turned in part
    {"name": "qk_bwd_odd", "op": "qk_backward", "T": 3001, "nb": 5, "cut": 3, "nh": 20, "nkv": 5, "d": 96,
     "rot": 64, "dtype": "fp16"},
    # the norms and biases of one layer
    {"name": "clip_vectors", "op": "clip", "tensors": 12, "largest": 4097, "cut": 4},
    # every gradient of the embedding and two layers
    {"name": "clip_layers", "op": "clip", "tensors": 31, "largest": 0, "cut": 0},
]

_ATTN_MOST = 16384 * 16385 // 2 * 16 * 128  # pairs x heads x head dim of the longest case
_QK_MOST = 8192 * 40 * 128
_CLIP_MOST = 550_000_000


def listed():
    return [dict(c) for c in _LISTED]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _lengths(case):
    """Lengths of the packed sequences: equal ones (cut 0), or T cut at nb - 1
    places, among them sequences of no token and of one."""
    T, nb = case["T"], case["nb"]
    if case["cut"] == 0:
        return [T // nb] * nb
    rng = random.Random(case["cut"])
    at = sorted(rng.randint(0, T) for _ in range(nb - 1))
    if len(at) > 1:
        at[1] = at[0]
    if len(at) > 3:
        at[3] = min(T, at[2] + 1)
        at.sort()
    at = [0] + at + [T]
    return [b - a for a, b in zip(at, at[1:])]


def _pairs(case):
    return sum(n * (n + 1) // 2 for n in _lengths(case))


def _sizes(case):
    """Sizes and types of the clipped tensors."""
    if case["largest"] == 0:
        h, F, qkv = 4096, 16384, (32 + 2 * 8) * 128
        layer = [(h * qkv, "bf16"), (h * h, "bf16"), (h * F, "bf16"), (F * h, "bf16"), (qkv, "fp32"), (h, "fp32"),
                 (F, "fp32"), (h, "fp32"), (h, "fp32"), (h, "fp32"), (h, "fp32"), (h, "fp32"), (128, "fp32"),
                 (128, "fp32")]
        return layer * 2 + [(50257 * h, "bf16"), (h, "fp32"), (h, "fp32")]
    rng = random.Random(case["cut"])
    return [(_log_int(rng, 1, case["largest"]), rng.choice(["bf16", "bf16", "fp32", "fp16"]))
            for _ in range(case["tensors"])]


def draw(rng):
    op = rng.choice(["attn_forward", "attn_backward", "qk_forward", "qk_backward", "clip"])
    if op == "clip":
        tensors = _log_int(rng, 1, 60)
        # a draw is log-uniform between 1 and the largest, whose sum stays below the largest listed case
        largest = _log_int(rng, 16, min(1 << 26, _CLIP_MOST // tensors))
        return {"op": op, "tensors": tensors, "largest": largest, "cut": rng.randint(1, 1 << 30)}
    d = rng.choice([64, 96, 128, 128, 160])
    nkv = rng.choice([1, 2, 3, 4, 8, 16])
    nh = nkv * rng.choice([1, 1, 2, 3, 4, 5, 8])
    case = {"op": op, "nh": nh, "nkv": nkv, "d": d}
    if op.startswith("qk"):
        T = _log_int(rng, 1, min(32768, _QK_MOST // ((nh + nkv) * d)))
        case["rot"] = rng.choice([d, d, d // 2])
        case["dtype"] = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    else:
        T = _log_int(rng, 1, 16384)
    nb = _log_int(rng, 1, max(1, min(64, T)))
    case.update(T=T, nb=nb, cut=rng.randint(1, 1 << 30) if nb > 1 else 0)
    if not op.startswith("qk"):
        while _pairs(case) * nh * d > _ATTN_MOST // (2 if op == "attn_backward" else 1):
            case["T"] //= 2
            case["nb"] = nb = min(nb, case["T"])
    return case


def _qkv(case, g, dt):
    """Queries, keys and values as the projection leaves them: [T, heads, d]
    parts of rows [Q | K | V]."""
    T, nh, nkv, d = case["T"], case["nh"], case["nkv"], case["d"]
    rows = torch.empty(T, nh + 2 * nkv, d, dtype=dt, device="cuda")
    rows.copy_(torch.randn(T, nh + 2 * nkv, d, generator=g, device="cuda"))
    return rows[:, :nh], rows[:, nh:nh + nkv], rows[:, nh + nkv:]


def _softmax_rows(q, k, scale):
    """P and lse (log2) of one head of one sequence, fp32."""
    n = q.shape[0]
    z = (q @ k.t()) * scale
    z.masked_fill_(torch.ones(n, n, dtype=torch.bool, device=z.device).triu_(1), -math.inf)
    m = z.amax(-1, keepdim=True)
    p = z.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    return p.div_(total), ((m + torch.log(total)) * math.log2(math.e))[:, 0]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    state = {"case": case}
    if case["op"] == "clip":
        sizes = _sizes(case)
        grads = []
        total = sum(n for n, _ in sizes)
        for n, kind in sizes:
            # gradients of very different size, together about three times the clipping norm
            size = 3.0 / math.sqrt(total) * math.exp(random.Random(seed + n).uniform(-1.0, 1.0))
            x = torch.empty(n, dtype=DTYPES[kind], device="cuda")
            grads.append(x.copy_(torch.randn(n, generator=g, device="cuda").mul_(size)))
        state["grads"] = grads
        state["out"] = [torch.empty_like(x) for x in grads]
        return state
    nh, nkv, d, T = case["nh"], case["nkv"], case["d"], case["T"]
    lens = _lengths(case)
    if case["op"].startswith("qk"):
        dt = DTYPES[case["dtype"]]
        q, k, _ = _qkv(case, g, dt)
        # tokens count from the start of their sequence, some of them parts of a long one
        start = random.Random(seed).choice([0, 0, 4096, 131072, 1 << 20])
        positions = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens]).add_(start).cuda()
        gq = (1.0 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(dt)
        gk = (1.0 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(dt)
        state.update(q=q, k=k, gq=gq, gk=gk, positions=positions)
        if case["op"] == "qk_backward":
            state["dq"], state["dk"], _ = _qkv(case, g, dt)
            x = torch.cat([q, k], 1).double()
            state["rstd"] = (1.0 / torch.sqrt((x * x).mean(-1) + EPS)).float()
        return state
    q, k, v = _qkv(case, g, torch.bfloat16)
    cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32)
    state.update(q=q, k=k, v=v, lens=lens, cu=cu.cuda(), scale=1.0 / math.sqrt(d))
    if case["op"] == "attn_backward":
        state["do"] = torch.randn(T, nh, d, generator=g, device="cuda").to(torch.bfloat16)
        # what the forward pass saved
        out = _plain_attn_forward(state)
        state["o"], state["lse"] = out["O"], out["lse"]
    return state


# ------------------------------------------------------------- plain forms

def _turns(s, back):
    """cos and sin [T, 1, rot / 2] of the rotation (or of its inverse)."""
    rot = s["case"]["rot"]
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    a = s["positions"].double()[:, None, None] * torch.pow(torch.tensor(THETA, dtype=torch.float64), -2.0 * i / rot)
    return torch.cos(a).float(), (-torch.sin(a) if back else torch.sin(a)).float()


def _rotate(x, cos, sin):
    r = 2 * cos.shape[-1]
    a, b, rest = x[..., :r // 2], x[..., r // 2:r], x[..., r:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)


def _plain_qk_forward(s):
    cos, sin = _turns(s, False)
    out = {}
    rs = []
    for name, gamma in (("q", "gq"), ("k", "gk")):
        x = s[name].float()
        rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        out[name.upper()] = _rotate(x * rstd * s[gamma].float(), cos, sin).to(s[name].dtype)
        rs.append(rstd[..., 0])
    out["rstd"] = torch.cat(rs, 1)
    return out


def _plain_qk_backward(s):
    cos, sin = _turns(s, True)
    nh = s["case"]["nh"]
    out = {}
    for name, gamma, rstd in (("q", "gq", s["rstd"][:, :nh]), ("k", "gk", s["rstd"][:, nh:])):
        x, r = s[name].float(), rstd[..., None]
        g = _rotate(s["d" + name].float(), cos, sin)
        gg = g * s[gamma].float()
        xhat = x * r
        out["d" + name.upper()] = (r * (gg - xhat * (gg * xhat).mean(-1, keepdim=True))).to(s[name].dtype)
        out["dgamma_" + name] = (g * xhat).sum((0, 1))
    return out


def _heads(s):
    """(rows, query head, key/value head) of the batch."""
    at, each = 0, s["case"]["nh"] // s["case"]["nkv"]
    for n in s["lens"]:
        if n:
            for j in range(s["case"]["nh"]):
                yield slice(at, at + n), j, j // each
        at += n


def _plain_attn_forward(s):
    q, k, v = s["q"], s["k"], s["v"]
    O = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    lse = torch.empty(q.shape[1], q.shape[0], device=q.device)
    for rows, j, c in _heads(s):
        p, lse[j, rows] = _softmax_rows(q[rows, j].float(), k[rows, c].float(), s["scale"])
        O[rows, j] = (p @ v[rows, c].float()).to(O.dtype)
    return {"O": O, "lse": lse}


def _plain_attn_backward(s):
    q, k, v, do = s["q"], s["k"], s["v"], s["do"]
    dQ = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    dK = torch.zeros(k.shape, device=q.device)
    dV = torch.zeros(v.shape, device=q.device)
    for rows, j, c in _heads(s):
        qj, kc, vc, gj = q[rows, j].float(), k[rows, c].float(), v[rows, c].float(), do[rows, j].float()
        z = (qj @ kc.t()) * s["scale"] - s["lse"][j, rows, None] * math.log(2.0)
        p = torch.exp(z).tril_()
        delta = (gj * s["o"][rows, j].float()).sum(-1, keepdim=True)
        ds = (gj @ vc.t()).sub_(delta).mul_(p)
        dQ[rows, j] = (ds @ kc * s["scale"]).to(dQ.dtype)
        dK[rows, c] += ds.t() @ qj * s["scale"]
        dV[rows, c] += p.t() @ gj
    return {"dQ": dQ, "dK": dK.to(k.dtype), "dV": dV.to(v.dtype)}


def _plain_clip(s):
    squares = torch.stack([(x.float() * x.float()).sum() for x in s["grads"]])
    norm = torch.sqrt(squares.sum())
    coef = torch.clamp(MAX_NORM / (norm + 1e-6), max=1.0)
    return {"norm": norm, "grads": [(x.float() * coef).to(x.dtype) for x in s["grads"]]}


# --------------------------------------------------- this repository's calls

def _own_run(s):
    from tensor_transformer_mlp_forward_gb300 import binding

    op = s["case"]["op"]
    if op == "qk_forward":
        Q, K, rstd = binding.tp_qk_norm_rope_forward(s["q"], s["k"], s["gq"], s["gk"], s["positions"],
                                                     rot=s["case"]["rot"], theta=THETA, eps=EPS)
        return {"Q": Q, "K": K, "rstd": rstd}
    if op == "qk_backward":
        dQ, dK, dgq, dgk = binding.tp_qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["gq"], s["gk"],
                                                            s["positions"], s["rstd"], rot=s["case"]["rot"],
                                                            theta=THETA)
        return {"dQ": dQ, "dgamma_q": dgq, "dK": dK, "dgamma_k": dgk}
    if op == "attn_forward":
        O, lse = binding.tp_attn_packed_forward(s["q"], s["k"], s["v"], s["cu"], scale=s["scale"])
        return {"O": O, "lse": lse}
    if op == "attn_backward":
        dQ, dK, dV = binding.tp_attn_packed_backward(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], s["cu"],
                                                     scale=s["scale"])
        return {"dQ": dQ, "dK": dK, "dV": dV}
    norm, grads = binding.tp_grad_clip(s["grads"], MAX_NORM, out=s["out"])
    return {"norm": norm, "grads": grads}


_PLAIN = {"qk_forward": _plain_qk_forward, "qk_backward": _plain_qk_backward, "attn_forward": _plain_attn_forward,
          "attn_backward": _plain_attn_backward, "clip": _plain_clip}


def run(state):
    if own:
        return _own_run(state)
    return _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------- 64 bits

def _turn64(x, positions, rot, sign):
    """Each pair as a complex number, times e^(sign i p theta^(-2 i / rot))."""
    half = rot // 2
    freq = torch.exp(torch.arange(half, device=x.device, dtype=torch.float64) * (-2.0 * math.log(THETA) / rot))
    angle = sign * torch.outer(positions.double(), freq)
    z = torch.complex(x[..., :half], x[..., half:rot]) * torch.polar(torch.ones_like(angle), angle).unsqueeze(1)
    return torch.cat([z.real, z.imag, x[..., rot:]], dim=2)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        flat = [x.double() for x in s["grads"]]
        norm = math.sqrt(math.fsum(torch.dot(x, x).item() for x in flat))
        coef = min(1.0, MAX_NORM / (norm + 1e-6))
        return {"norm": torch.tensor(norm, dtype=torch.float64, device="cuda"), "grads": [x.mul_(coef) for x in flat]}
    if op == "qk_forward":
        out, inv = {}, []
        for key, x, gamma in (("Q", s["q"], s["gq"]), ("K", s["k"], s["gk"])):
            x = x.double()
            inv.append((torch.einsum("thd,thd->th", x, x) / x.shape[2] + EPS).pow(-0.5))
            out[key] = _turn64(torch.einsum("thd,th,d->thd", x, inv[-1], gamma.double()), s["positions"], case["rot"], 1)
        out["rstd"] = torch.cat(inv, dim=1)
        return out
    if op == "qk_backward":
        out = {}
        inv = s["rstd"].double().split([case["nh"], case["nkv"]], dim=1)
        for key, x, dy, gamma, r in (("q", s["q"], s["dq"], s["gq"], inv[0]), ("k", s["k"], s["dk"], s["gk"], inv[1])):
            x = x.double()
            e = _turn64(dy.double(), s["positions"], case["rot"], -1)
            out["dgamma_" + key] = torch.einsum("thd,thd,th->d", e, x, r)
            e = e * gamma.double()
            along = torch.einsum("thd,thd->th", e, x) * r.pow(3) / x.shape[2]
            out["d" + key.upper()] = e * r.unsqueeze(2) - x * along.unsqueeze(2)
        return out
    each, scale = case["nh"] // case["nkv"], s["scale"]
    if _pairs(case) * case["nh"] * case["d"] > 5e11:
        return None  # 64-bit products of this size take too long
    q, k, v = (s[n].double() for n in "qkv")
    first = 0
    if op == "attn_forward":
        O, lse = torch.zeros_like(q), torch.zeros(case["nh"], case["T"], dtype=torch.float64, device="cuda")
        for n in s["lens"]:
            sl, first = slice(first, first + n), first + n
            for c in range(case["nkv"] if n else 0):
                for lo in range(0, n, 2048):  # some queries at a time, and the keys up to them
                    hi = min(n, lo + 2048)
                    qs = q[sl][lo:hi, c * each:(c + 1) * each]
                    z = torch.einsum("qjd,kd->jqk", qs, k[sl][:hi, c]) * scale
                    late = torch.arange(hi, device="cuda") > torch.arange(lo, hi, device="cuda").unsqueeze(1)
                    z[:, late] = -math.inf
                    total = torch.logsumexp(z, dim=2)
                    O[sl][lo:hi, c * each:(c + 1) * each] = torch.einsum(
                        "jqk,kd->qjd", torch.exp(z - total.unsqueeze(2)), v[sl][:hi, c])
                    lse[c * each:(c + 1) * each, sl][:, lo:hi] = total / math.log(2.0)
        return {"O": O, "lse": lse}
    dQ, dK, dV = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    do, o, lse = s["do"].double(), s["o"].double(), s["lse"].double()
    for n in s["lens"]:
        sl, first = slice(first, first + n), first + n
        for c in range(case["nkv"] if n else 0):
            hs = slice(c * each, (c + 1) * each)
            for lo in range(0, n, 2048):
                hi = min(n, lo + 2048)
                qs, gs = q[sl][lo:hi, hs], do[sl][lo:hi, hs]
                ks, vs = k[sl][:hi, c], v[sl][:hi, c]
                z = torch.einsum("qjd,kd->jqk", qs, ks) * scale
                p = torch.pow(2.0, z / math.log(2.0) - lse[hs, sl][:, lo:hi].unsqueeze(2))
                late = torch.arange(hi, device="cuda") > torch.arange(lo, hi, device="cuda").unsqueeze(1)
                p[:, late] = 0.0
                inner = torch.einsum("qjd,qjd->jq", gs, o[sl][lo:hi, hs])
                ds = p * (torch.einsum("qjd,kd->jqk", gs, vs) - inner.unsqueeze(2)) * scale
                dV[sl][:hi, c] += torch.einsum("jqk,qjd->kd", p, gs)
                dK[sl][:hi, c] += torch.einsum("jqk,qjd->kd", ds, qs)
                dQ[sl][lo:hi, hs] = torch.einsum("jqk,kd->qjd", ds, ks)
    return {"dQ": dQ, "dK": dK, "dV": dV}


def work(case):
    op = case["op"]
    if op == "clip":  # every gradient in, its clipped form out, the norm
        size = sum(n * (4 if kind == "fp32" else 2) for n, kind in _sizes(case))
        return {"bytes": 2 * size + 4, "flops": 3 * sum(n for n, _ in _sizes(case))}
    T, nh, nkv, d = case["T"], case["nh"], case["nkv"], case["d"]
    if op.startswith("qk"):
        e = 4 if case["dtype"] == "fp32" else 2
        values, small = T * (nh + nkv) * d, 4 * T + 4 * T * (nh + nkv) + 2 * e * d
        if op == "qk_forward":  # Q and K in and out, positions, gammas, rstd
            return {"bytes": 2 * e * values + small, "flops": 8 * values}
        # x and dy in, dx out, positions, gammas, rstd, two dgammas
        return {"bytes": 3 * e * values + small + 8 * d, "flops": 14 * values}
    small = 4 * T * nh + 4 * (case["nb"] + 1)
    if op == "attn_forward":  # Q, K, V in, O and lse out; S and P V
        return {"bytes": 2 * d * T * (2 * nh + 2 * nkv) + small, "flops": 4 * d * nh * _pairs(case)}
    # Q, K, V, O, dO, lse in, dQ, dK, dV out; S again, dP, dV, dQ and dK
    return {"bytes": 2 * d * T * (4 * nh + 4 * nkv) + small, "flops": 10 * d * nh * _pairs(case)}
