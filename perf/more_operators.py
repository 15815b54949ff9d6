"""Gated layers, log probabilities and distillation, in plain torch and through the library.

Operators of a language model around the products of its FC path:

* ``glu``: the gated feed-forward layer Y = act(G) * U with [G | U] = X.[Wg | Wu] + b, and ``glu_grad``, the
  gradient through the down projection and the gate, dH = dY.W^T, dG = dH * U * act'(G), dU = dH * act(G), with Y
  computed again for the down projection's weight gradient and the biases' gradients;
* ``logprob``: log probabilities of given tokens under softmax(X.W / T), the entropy, and the most likely
  alternatives (ties go to the lowest index);
* ``distill``: the divergence of softmax(X.W / T) from a teacher's distribution over its top tokens, and
  ``distill_grad``, its gradients with respect to both operands. No logits are kept between the two.

``own`` picks the library's calls; otherwise ``run`` computes the same formulas in elementary torch operations in
32 bits.
"""
import math

import torch

own = False

ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}  # the library's numbers of them
IGNORED = -100  # the target of a row that takes no part


def listed():
    return [
        # decoding: one token through the gated layer of a block of hidden size 2048, weights as nn.Linear keeps them
        {"name": "glu_token", "op": "glu", "M": 1, "K": 2048, "N": 8192, "act": "silu", "order": "col", "bias": False,
         "keep": False, "f32": False},
        # training: that layer over 8192 tokens, gate and up values kept for the backward pass
        {"name": "glu_up", "op": "glu", "M": 8192, "K": 2048, "N": 8192, "act": "silu", "order": "row", "bias": False,
         "keep": True, "f32": False},
        # odd sizes everywhere (no aligned vectors), biases and an fp32 output: a pruned layer
        {"name": "glu_odd", "op": "glu", "M": 777, "K": 1001, "N": 1531, "act": "gelu_tanh", "order": "row",
         "bias": True, "keep": True, "f32": True},
        # training: the gradient through the down projection into gate and up values
        {"name": "glu_grad", "op": "glu_grad", "M": 8192, "K": 8192, "N": 2048, "act": "silu", "order": "row",
         "bias": False},
        # the same direction at odd sizes, with the biases' gradients
        {"name": "glu_grad_odd", "op": "glu_grad", "M": 333, "K": 1531, "N": 611, "act": "gelu", "order": "col",
         "bias": True},
        # serving: the token just sampled, with 20 alternatives
        {"name": "logprob_token", "op": "logprob", "M": 1, "K": 2048, "N": 32000, "order": "col", "k": 20, "T": 1.0,
         "start": 0, "ignored": 0.0},
        # scoring a batch of prompts with five alternatives for each position; padding has no target
        {"name": "logprob_prompt", "op": "logprob", "M": 2500, "K": 2048, "N": 50001, "order": "col", "k": 5, "T": 1.0,
         "start": 0, "ignored": 0.1},
        # a teacher's pass over a training batch: its 64 most likely tokens at every position, at temperature 2
        {"name": "logprob_teacher", "op": "logprob", "M": 8192, "K": 2048, "N": 32000, "order": "row", "k": 64,
         "T": 2.0, "start": 0, "ignored": 0.0},
        # the student's loss against that teacher
        {"name": "distill", "op": "distill", "M": 8192, "K": 2048, "N": 32000, "order": "row", "k": 64, "T": 2.0,
         "start": 0, "absent": 0.05},
        # few rows, odd sizes, and a teacher that gives a different number of tokens for each position
        {"name": "distill_odd", "op": "distill", "M": 61, "K": 1030, "N": 10007, "order": "col", "k": 21, "T": 1.0,
         "start": 0, "absent": 0.4},
        # training: the gradients of the student's loss
        {"name": "distill_grad", "op": "distill_grad", "M": 8192, "K": 2048, "N": 32000, "order": "row", "k": 64,
         "T": 2.0, "start": 0, "absent": 0.05},
        # the gradients at odd sizes with many absent tokens
        {"name": "distill_grad_odd", "op": "distill_grad", "M": 1021, "K": 1030, "N": 10007, "order": "col", "k": 21,
         "T": 1.0, "start": 0, "absent": 0.4},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A size over the logarithm of its range: about half of them multiples of 64, the others as they come."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.5 else max(lo, min(hi, n // 64 * 64))


def draw(rng):
    op, order = rng.choice(["glu", "glu_grad", "logprob", "distill", "distill_grad"]), rng.choice(["row", "col"])
    if op in ("glu", "glu_grad"):
        c = {"op": op, "M": _log(rng, 1 if op == "glu" else 16, 8192), "K": _size(rng, 256, 8192),
             "N": _size(rng, 256, 8192), "act": rng.choice(list(ACTS)), "order": order, "bias": rng.random() < 0.4}
        return c | ({"keep": rng.random() < 0.5, "f32": rng.random() < 0.3} if op == "glu" else {})
    M, K = _log(rng, {"logprob": 1, "distill": 16, "distill_grad": 64}[op], 8192), _size(rng, 512, 4096)
    N = max(4096, min(_size(rng, 4096, 65536), 530_000_000_000 // (M * K)))
    c = {"op": op, "M": M, "K": K, "N": N, "order": order, "T": rng.choice([1.0, 1.0, 0.7, 2.0]),
         "start": rng.choice([0, 0, N])}
    if op == "logprob":
        return c | {"k": rng.choice([0, 1, 5, 20, _log(rng, 1, 128)]), "ignored": rng.choice([0.0, 0.1])}
    return c | {"k": _log(rng, 1, 128), "absent": rng.choice([0.0, 0.05, 0.4])}


def _teacher(case, g):
    """A teacher's listed tokens and their logits, most likely first, and how many of them count in each row: some
    positions have none (padding). A shard's tokens lie in the whole vocabulary."""
    M, N, k = case["M"], case["N"], case["k"]
    whole = N if case["start"] == 0 else 2 * N
    gap = torch.randint(1, whole // k + 1, (M, k), device="cuda", generator=g)
    ids = (gap.cumsum(1) + torch.randint(0, whole, (M, 1), device="cuda", generator=g)) % whole  # all different
    ids = ids.gather(1, torch.rand((M, k), device="cuda", generator=g).argsort(1))
    fall = torch.rand((M, k), device="cuda", generator=g) / torch.arange(1, k + 1, device="cuda")
    logits = 8.0 - 4.0 * fall.cumsum(1)
    count = torch.where(torch.rand((M, 1), device="cuda", generator=g) < case["absent"],
                        torch.randint(0, k, (M, 1), device="cuda", generator=g), k)
    return torch.where(torch.arange(k, device="cuda") < count, ids, -1), logits


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(5000 + seed)
    op, M, K, N = case["op"], case["M"], case["K"], case["N"]
    st = {"case": case}

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, device="cuda", generator=g) * scale).to(torch.bfloat16)

    def grid(*shape, scale, step):
        """Normal values on a grid, so that a logit is the same sum in any order and equal logits are real ties."""
        x = torch.randn(shape, device="cuda", generator=g) * (scale / step)
        return (torch.clamp(torch.round(x), -64, 64) * step).to(torch.bfloat16)

    def matrix(rows, cols):
        return (rows, cols) if case["order"] == "row" else (cols, rows)

    if op == "glu":
        return st | {"X": normal(M, K), "W": normal(*matrix(K, 2 * N), scale=0.02),
                     "b": normal(2 * N, scale=0.5) if case["bias"] else None}
    if op == "glu_grad":
        return st | {"dY": normal(M, N, scale=1e-3), "W": normal(*matrix(K, N), scale=0.02), "Z": normal(M, 2 * K)}
    if op == "logprob":
        st |= {"X": grid(M, K, scale=1.0, step=2.0 ** -4), "W": grid(*matrix(K, N), scale=0.04, step=2.0 ** -8)}
        t = torch.randint(0, N if case["start"] == 0 else 2 * N, (M,), device="cuda", generator=g)
        drop = torch.rand(M, device="cuda", generator=g) < case["ignored"]
        return st | {"targets": torch.where(drop, IGNORED, t)}
    st |= {"X": normal(M, K), "W": normal(*matrix(K, N), scale=0.04)}
    st["ids"], st["tlogits"] = _teacher(case, g)
    if op == "distill_grad":  # what the forward pass left, and the mean over the rows that count
        W = st["W"].float()
        z = st["X"].float() @ (W if case["order"] == "row" else W.t())
        st["lse"] = torch.logsumexp(z / case["T"], 1)
        at = st["ids"] - case["start"]
        here = (at >= 0) & (at < N)
        st["slogits"] = torch.where(here, z.gather(1, torch.where(here, at, 0)), 0.0)
        rows = max(1, int((st["ids"] >= 0).any(1).sum()))
        st["g"] = torch.full((M,), case["T"] ** 2 / rows, device="cuda")
    return st


# ---- the library's calls

def _run_own(st):
    from sharded_fc_layer_amd import fcshard as F
    case, op = st["case"], st["case"]["op"]
    order = F.ROW if case["order"] == "row" else F.COL
    if op == "glu":
        return F.fc_fwd_glu(st["X"], st["W"], bias=st["b"], act=ACTS[case["act"]], w_order=order, keep_z=case["keep"],
                            out_dtype=F.OUT_F32 if case["f32"] else F.OUT_BF16)
    if op == "glu_grad":
        return F.fc_bwd_data_glu(st["dY"], st["W"], st["Z"], ACTS[case["act"]], w_order=order, keep_y=True,
                                 bias_grad=case["bias"])
    if op == "logprob":
        return F.fc_logprob(st["X"], st["W"], st["targets"], w_order=order, vocab_start=case["start"],
                            ignore_index=IGNORED, temperature=case["T"], top_k=case["k"])
    if op == "distill":
        return F.fc_distill_fwd(st["X"], st["W"], st["ids"], st["tlogits"], w_order=order, vocab_start=case["start"],
                                temperature=case["T"])
    return F.fc_distill_bwd(st["X"], st["W"], st["ids"], st["tlogits"], st["slogits"], st["lse"], st["g"],
                            w_order=order, vocab_start=case["start"], temperature=case["T"])


# ---- the plain forms

def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    return torch.ones_like(z)


def _weight32(st):
    W = st["W"].float()
    return W if st["case"]["order"] == "row" else W.t()


def _lse(z):
    top = z.max(1).values
    return top + torch.log(torch.exp(z - top[:, None]).sum(1))


def _teacher32(st):
    """The teacher's probabilities (zeros where a token is absent) and their logarithms (zeros there too)."""
    there = st["ids"] >= 0
    t = torch.where(there, st["tlogits"] / st["case"]["T"], -math.inf)
    t = t - torch.where(there.any(1), t.max(1).values, 0.0)[:, None]
    e = torch.exp(t)
    s = torch.where(there.any(1), e.sum(1), 1.0)[:, None]
    return there, e / s, torch.where(there, t - torch.log(s), 0.0)


def _run_plain(st):
    case, op = st["case"], st["case"]["op"]
    W = _weight32(st)
    if op == "glu":
        z = st["X"].float() @ W
        if st["b"] is not None:
            z = z + st["b"].float()
        y = _act(z[:, :case["N"]], case["act"]) * z[:, case["N"]:]
        y = y if case["f32"] else y.to(torch.bfloat16)
        return (y, z.to(torch.bfloat16)) if case["keep"] else y
    if op == "glu_grad":
        h = st["dY"].float() @ W.t()
        G, U = st["Z"].float().chunk(2, 1)
        a = _act(G, case["act"])
        d = torch.cat([h * U * _act_slope(G, case["act"]), h * a], 1)
        out = d.to(torch.bfloat16), (a * U).to(torch.bfloat16)
        return out + (d.sum(0),) if case["bias"] else out
    z = st["X"].float() @ W
    if op == "logprob":
        at = st["targets"] - case["start"]
        here = (at >= 0) & (at < case["N"])
        hit = torch.where(here, z.gather(1, torch.where(here, at, 0)[:, None])[:, 0], -math.inf)
        ids = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :case["k"]] if case["k"] else at[:, None][:, :0]
        values = z.gather(1, ids)
        s = z / case["T"]
        lse = _lse(s)
        p = torch.exp(s - lse[:, None])
        entropy = -(p * (s - lse[:, None])).sum(1)
        logp = torch.where(st["targets"] != IGNORED, hit / case["T"] - lse, 0.0)
        return logp, entropy, lse, values / case["T"] - lse[:, None], ids + case["start"]
    there, p, logp = _teacher32(st)
    at = st["ids"] - case["start"]
    here = there & (at >= 0) & (at < case["N"])
    at = torch.where(here, at, 0)
    if op == "distill":
        lse = _lse(z / case["T"])
        own_logits = torch.where(here, z.gather(1, at), 0.0)
        loss = (p * (logp - own_logits / case["T"])).sum(1) + torch.where(there.any(1), lse, 0.0)
        return loss, lse, own_logits
    d = torch.exp(z / case["T"] - st["lse"][:, None])
    d.scatter_add_(1, at, -torch.where(here, p, 0.0))
    d = d * torch.where(there.any(1), st["g"] / case["T"], 0.0)[:, None]
    return (d @ W.t()).to(torch.bfloat16), (st["X"].float().t() @ d).to(torch.bfloat16)


def run(st):
    return _run_own(st) if own else _run_plain(st)


def work(case):
    op, M, K, N = case["op"], case["M"], case["K"], case["N"]
    if op == "glu":
        outs = M * N * ((4 if case["f32"] else 2) + (4 if case["keep"] else 0))
        return {"bytes": 2 * (M * K + 2 * K * N + (2 * N if case["bias"] else 0)) + outs, "flops": 4 * M * K * N}
    if op == "glu_grad":
        return {"bytes": 2 * (M * N + K * N + 5 * M * K) + (8 * K if case["bias"] else 0), "flops": 2 * M * K * N}
    ins = 2 * (M * K + K * N)
    if op == "logprob":
        return {"bytes": ins + M * (20 + 12 * case["k"]), "flops": 2 * M * K * N}
    if op == "distill":
        return {"bytes": ins + M * (8 + 16 * case["k"]), "flops": 2 * M * K * N}
    # the logits once more (they are not kept), and two products with their gradient
    return {"bytes": 2 * ins + M * (8 + 16 * case["k"]), "flops": 6 * M * K * N}


# ---- the definitions in 64 bits

def _exact_act(z, act):
    f = torch.nn.functional
    return {"none": lambda: z, "relu": lambda: f.relu(z), "gelu": lambda: f.gelu(z),
            "gelu_tanh": lambda: f.gelu(z, approximate="tanh"), "silu": lambda: f.silu(z)}[act]()


def exact(case, seed):
    st, op, M, N, T = prepare(case, seed), case["op"], case["M"], case["N"], case.get("T")
    W = st["W"].double()
    W = W if case["order"] == "row" else W.mT
    if op == "glu":
        z = torch.mm(st["X"].double(), W)
        z = z if st["b"] is None else z + st["b"].double()
        y = _exact_act(z[:, :N], case["act"]) * z[:, N:]
        return (y, z) if case["keep"] else y
    if op == "glu_grad":
        z = st["Z"].double().requires_grad_()
        gate, up = z.split(case["K"], 1)
        y = _exact_act(gate, case["act"]) * up
        (d,) = torch.autograd.grad(y, z, torch.mm(st["dY"].double(), W.mT))
        return (d, y.detach(), d.sum(0)) if case["bias"] else (d, y.detach())
    if op != "logprob":
        p = torch.where(st["ids"] >= 0, st["tlogits"].double() / T, -torch.inf).softmax(1)
        p = torch.where(st["ids"] >= 0, p, 0.0)
        counts = (st["ids"] >= 0).any(1)
    parts, dW = [], torch.zeros_like(W) if op == "distill_grad" else None
    for rows in torch.arange(M, device="cuda").split(1024):
        X = st["X"][rows].double()
        z, n = X @ W, len(rows)
        s = z / T
        at = (st["targets"][rows][:, None] if op == "logprob" else st["ids"][rows]) - case["start"]
        mine = (at >= 0) & (at < N)
        picked = z[torch.arange(n, device="cuda")[:, None], at.clamp(0, N - 1)]
        if op == "logprob":
            q = s.log_softmax(1)
            logp = torch.where(mine, picked, -torch.inf)[:, 0] / T - torch.logsumexp(s, 1)
            logp = logp.masked_fill(st["targets"][rows] == IGNORED, 0.0)
            best = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :case["k"]]
            parts.append((logp, -(q.exp() * q).sum(1), torch.logsumexp(s, 1), q.gather(1, best), best + case["start"]))
        elif op == "distill":
            lse = torch.logsumexp(s, 1)
            own_logits = torch.where(mine & (st["ids"][rows] >= 0), picked, 0.0)
            loss = torch.special.xlogy(p[rows], p[rows]) - p[rows] * (own_logits / T - lse[:, None])
            parts.append((loss.sum(1), lse, own_logits))
        else:
            d = (s - st["lse"][rows].double()[:, None]).exp()
            d.scatter_add_(1, at.clamp(0, N - 1), torch.where(mine, -p[rows], 0.0))
            d *= (st["g"][rows].double() / T * counts[rows])[:, None]
            parts.append((d @ W.mT,))
            dW += X.mT @ d
    out = tuple(torch.cat(x) for x in zip(*parts))
    return out if op != "distill_grad" else (out[0], dW)
