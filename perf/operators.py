"""The fused operators of the FC layer, in plain torch and through the library.

Three operators of a language model's FC path, each with its gradient:

* ``act``: Y = act(X.W + b) + R with the pre-activation kept for training, and
  its gradient dX = (dY.W^T) * act'(Z) with the bias gradient (the columns' sums);
* ``xent``: the softmax cross entropy of a vocabulary projection, whose logits
  are never kept, and its gradients with respect to both operands;
* ``grouped``: the products of an expert layer, whose rows are sorted by
  expert, with ragged groups, and their gradients.

``own`` picks the library's calls; otherwise ``run`` computes the same
formulas in elementary torch operations in 32 bits.
"""
import math

import numpy as np
import torch

own = False

ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}  # the library's numbers of them
IGNORED = -100  # the target of a row that takes no part in the loss


def listed():
    return [
        # decoding: one token through the up projection of the GPT block (hidden 2048), weight as nn.Linear keeps it
        {"name": "act_token", "op": "act", "M": 1, "K": 2048, "N": 8192, "act": "gelu_tanh", "order": "col",
         "bias": True, "residual": False, "keep": False, "f32": False},
        # training: the up projection of the GPT block over 8192 tokens, pre-activation kept for the backward pass
        {"name": "act_up", "op": "act", "M": 8192, "K": 2048, "N": 8192, "act": "gelu_tanh", "order": "row",
         "bias": True, "residual": False, "keep": True, "f32": False},
        # odd sizes everywhere (no aligned vectors), residual and fp32 output: a projection out of a pruned layer
        {"name": "act_odd", "op": "act", "M": 777, "K": 1001, "N": 1531, "act": "silu", "order": "row",
         "bias": True, "residual": True, "keep": False, "f32": True},
        # training: the gradient through the down projection of the GPT block into the up projection's pre-activation
        {"name": "act_grad", "op": "act_grad", "M": 8192, "K": 8192, "N": 2048, "act": "gelu_tanh", "order": "row"},
        # the same direction at odd sizes
        {"name": "act_grad_odd", "op": "act_grad", "M": 333, "K": 1531, "N": 611, "act": "gelu", "order": "col"},
        # scoring a short continuation: few rows against a whole vocabulary
        {"name": "xent_few", "op": "xent", "M": 64, "K": 2048, "N": 50001, "order": "col", "start": 0, "ignored": 0.0},
        # the vocabulary shard of the 405B-like layer: the second of eight, so most targets lie in other shards
        {"name": "xent_shard", "op": "xent", "M": 8192, "K": 16384, "N": 16032, "order": "row", "start": 16032,
         "ignored": 0.05},
        # training: the gradients of a whole vocabulary's loss over 8192 tokens
        {"name": "xent_grad", "op": "xent_grad", "M": 8192, "K": 2048, "N": 32000, "order": "row", "start": 0,
         "ignored": 0.05},
        # the same at odd sizes with many rows without a target (padding)
        {"name": "xent_grad_odd", "op": "xent_grad", "M": 1021, "K": 1030, "N": 10007, "order": "col", "start": 0,
         "ignored": 0.4},
        # decoding with experts: a few tokens a step, each expert has none to a handful of them
        {"name": "grouped_token", "op": "grouped", "T": 48, "E": 16, "K": 2048, "N": 6144, "order": "row"},
        # training: the up projection of 16 experts over 16384 routed rows
        {"name": "grouped_up", "op": "grouped", "T": 16384, "E": 16, "K": 2048, "N": 8192, "order": "row"},
        # training: both gradients of that layer at the attention width
        {"name": "grouped_grad", "op": "grouped_grad", "T": 16384, "E": 16, "K": 2048, "N": 6144, "order": "row"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A size over the logarithm of its range: about half of them multiples of 64, the others as they come."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.5 else max(lo, min(hi, n // 64 * 64))


def draw(rng):
    op = rng.choice(["act", "act_grad", "xent", "xent_grad", "grouped", "grouped_grad"])
    order = rng.choice(["row", "col"])
    if op == "act":
        return {"op": op, "M": _log(rng, 1, 8192), "K": _size(rng, 256, 8192), "N": _size(rng, 256, 8192),
                "act": rng.choice(list(ACTS)), "order": order, "bias": rng.random() < 0.7,
                "residual": rng.random() < 0.4, "keep": rng.random() < 0.4, "f32": rng.random() < 0.3}
    if op == "act_grad":
        return {"op": op, "M": _log(rng, 16, 8192), "K": _size(rng, 256, 8192), "N": _size(rng, 256, 8192),
                "act": rng.choice(list(ACTS)), "order": order}
    if op in ("xent", "xent_grad"):
        M, K = _log(rng, 16 if op == "xent" else 64, 8192), _size(rng, 512, 8192)
        N = _size(rng, 4096, 65536)
        N = max(4096, min(N, 1600_000_000_000 // (M * K)))  # within the largest listed case's work
        if op == "xent_grad":
            N = max(4096, min(N, 530_000_000_000 // (M * K)))
        return {"op": op, "M": M, "K": K, "N": N, "order": order, "start": rng.choice([0, 0, N]),
                "ignored": rng.choice([0.0, 0.05, 0.4])}
    T = _log(rng, 8, 16384) if op == "grouped" else _log(rng, 256, 16384)
    return {"op": op, "T": T, "E": _log(rng, 4, 64), "K": _size(rng, 256, 4096), "N": _size(rng, 256, 4096),
            "order": order}


def _cap(case):
    """The most rows an expert takes: the capacity that a padded layer would be built for."""
    return min(case["T"], 2 * -(-case["T"] // case["E"]) + 2)


def _counts(case, seed):
    """Rows of each expert: uneven, some experts without any, none over the capacity."""
    rng = np.random.default_rng([seed, case["T"], case["E"]])
    T, E, cap = case["T"], case["E"], _cap(case)
    p = np.exp(0.5 * rng.standard_normal(E))
    if E >= 8:
        p[rng.choice(E, E // 8, replace=False)] = 0.0
    counts = np.minimum(rng.multinomial(T, p / p.sum()), cap)
    for e in np.argsort(counts, kind="stable"):  # what the full ones could not take
        counts[e] += min(cap - counts[e], T - counts.sum())
    return counts


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(1000 + seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, device="cuda", generator=g) * scale).to(torch.bfloat16)

    def weight(*lead):
        K, N = case["K"], case["N"]
        return normal(*lead, *((K, N) if case["order"] == "row" else (N, K)), scale=0.02)

    op, st = case["op"], {"case": case}
    if op == "act":
        M, K, N = case["M"], case["K"], case["N"]
        st |= {"X": normal(M, K), "W": weight(), "b": normal(N, scale=0.5) if case["bias"] else None,
               "R": normal(M, N) if case["residual"] else None}
    elif op == "act_grad":
        M, K, N = case["M"], case["K"], case["N"]
        st |= {"dY": normal(M, N, scale=1e-3), "W": weight(), "Z": normal(M, K)}
    elif op in ("xent", "xent_grad"):
        M, K, N = case["M"], case["K"], case["N"]
        whole = N if case["start"] == 0 else 8 * N  # a shard's targets lie in the whole vocabulary
        t = torch.randint(0, whole, (M,), device="cuda", generator=g)
        drop = torch.rand(M, device="cuda", generator=g) < case["ignored"]
        st |= {"X": normal(M, K), "W": weight(), "targets": torch.where(drop, IGNORED, t)}
        if op == "xent_grad":  # what the forward pass left, and the mean over the rows that count
            X, W = st["X"].float(), st["W"].float()
            z = X @ (W if case["order"] == "row" else W.t())
            st["lse"] = torch.logsumexp(z, 1)
            st["g"] = torch.full((M,), 1.0 / max(1, int((~drop).sum())), device="cuda")
    else:
        counts = _counts(case, seed)
        st["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int64, device="cuda")
        st["W"] = weight(case["E"])
        if op == "grouped":
            st["X"] = normal(case["T"], case["K"])
        else:
            st |= {"X": normal(case["T"], case["K"]), "dY": normal(case["T"], case["N"], scale=1e-3)}
    return st


# ---- the library's calls

def _run_own(st):
    from sharded_fc_layer_amd import fcshard as F
    case, op = st["case"], st["case"]["op"]
    order = F.ROW if case["order"] == "row" else F.COL
    if op == "act":
        return F.fc_fwd_act(st["X"], st["W"], bias=st["b"], act=ACTS[case["act"]], residual=st["R"], w_order=order,
                            keep_z=case["keep"], out_dtype=F.OUT_F32 if case["f32"] else F.OUT_BF16)
    if op == "act_grad":
        return F.fc_bwd_data_act(st["dY"], st["W"], st["Z"], ACTS[case["act"]], w_order=order, bias_grad=True)
    if op == "xent":
        return F.fc_xent_fwd(st["X"], st["W"], st["targets"], w_order=order, vocab_start=case["start"],
                             ignore_index=IGNORED)
    if op == "xent_grad":
        return F.fc_xent_bwd(st["X"], st["W"], st["targets"], st["lse"], st["g"], w_order=order,
                             vocab_start=case["start"], ignore_index=IGNORED)
    if op == "grouped":
        return F.fc_grouped_fwd(st["X"], st["W"], st["offsets"], w_order=order)
    return (F.fc_grouped_bwd_data(st["dY"], st["W"], st["offsets"], w_order=order),
            F.fc_grouped_bwd_weight(st["X"], st["dY"], st["offsets"]))


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
    """The weight in 32 bits as the K x N matrix (one for each expert) that it stands for."""
    W = st["W"].float()
    return W if st["case"]["order"] == "row" else W.transpose(-1, -2)


def _padded(x, offsets, cap):
    """Each expert's rows, filled up with rows of zeros: experts x cap x columns, in 32 bits."""
    at = torch.arange(cap, device=x.device)
    rows = offsets[:-1, None] + at
    inside = rows < offsets[1:, None]
    return x.float()[torch.where(inside, rows, 0)] * inside[:, :, None]


def _unpadded(y, offsets, T):
    """The rows of _padded's layout back in their order."""
    t = torch.arange(T, device=y.device)
    e = torch.searchsorted(offsets[1:], t, right=True)
    return y[e, t - offsets[e]]


def _run_plain(st):
    case, op = st["case"], st["case"]["op"]
    W = _weight32(st)
    if op == "act":
        z = st["X"].float() @ W
        if st["b"] is not None:
            z = z + st["b"].float()
        y = _act(z, case["act"])
        if st["R"] is not None:
            y = y + st["R"].float()
        y = y if case["f32"] else y.to(torch.bfloat16)
        return (y, z.to(torch.bfloat16)) if case["keep"] else y
    if op == "act_grad":
        d = (st["dY"].float() @ W.t()) * _act_slope(st["Z"].float(), case["act"])
        return d.to(torch.bfloat16), d.sum(0)
    if op in ("xent", "xent_grad"):
        z = st["X"].float() @ W
        at = st["targets"] - case["start"]
        here = (st["targets"] != IGNORED) & (at >= 0) & (at < case["N"])
        at = torch.where(here, at, 0)[:, None]
        if op == "xent":
            top = z.max(1).values
            lse = top + torch.log(torch.exp(z - top[:, None]).sum(1))
            own_logit = torch.where(here, z.gather(1, at)[:, 0], 0.0)
            return torch.where(st["targets"] != IGNORED, lse - own_logit, 0.0), lse, own_logit
        d = torch.exp(z - st["lse"][:, None])
        d.scatter_add_(1, at, -here[:, None].to(d.dtype))
        d = d * torch.where(st["targets"] != IGNORED, st["g"], 0.0)[:, None]
        return (d @ W.t()).to(torch.bfloat16), (st["X"].float().t() @ d).to(torch.bfloat16)
    off, cap = st["offsets"], _cap(case)
    if op == "grouped":
        return _unpadded(torch.bmm(_padded(st["X"], off, cap), W), off, case["T"]).to(torch.bfloat16)
    d = _padded(st["dY"], off, cap)
    dX = _unpadded(torch.bmm(d, W.transpose(1, 2)), off, case["T"])
    dW = torch.bmm(_padded(st["X"], off, cap).transpose(1, 2), d)
    return dX.to(torch.bfloat16), dW.to(torch.bfloat16)


def run(st):
    return _run_own(st) if own else _run_plain(st)


def work(case):
    op, K, N = case["op"], case["K"], case["N"]
    if op == "act":
        M = case["M"]
        outs = M * N * ((4 if case["f32"] else 2) + (2 if case["keep"] else 0))
        ins = 2 * (M * K + K * N + (N if case["bias"] else 0) + (M * N if case["residual"] else 0))
        return {"bytes": ins + outs, "flops": 2 * M * K * N}
    if op == "act_grad":
        M = case["M"]
        return {"bytes": 2 * (M * N + K * N + 2 * M * K) + 4 * K, "flops": 2 * M * K * N}
    if op == "xent":
        M = case["M"]
        return {"bytes": 2 * (M * K + K * N) + 8 * M + 12 * M, "flops": 2 * M * K * N}
    if op == "xent_grad":  # the logits once more (they are not kept), and two products with their gradient
        M = case["M"]
        return {"bytes": 2 * (2 * M * K + 2 * K * N) + 16 * M, "flops": 6 * M * K * N}
    T, E = case["T"], case["E"]
    hit = min(E, T)  # experts without rows need not be read
    if op == "grouped":
        return {"bytes": 2 * (T * K + hit * K * N + T * N) + 8 * (E + 1), "flops": 2 * T * K * N}
    return {"bytes": 2 * (2 * T * K + T * N + hit * K * N + E * K * N) + 8 * (E + 1), "flops": 4 * T * K * N}


# ---- the definitions in 64 bits

def _exact_act(z, act):
    f = torch.nn.functional
    return {"none": lambda: z, "relu": lambda: f.relu(z), "gelu": lambda: f.gelu(z),
            "gelu_tanh": lambda: f.gelu(z, approximate="tanh"), "silu": lambda: f.silu(z)}[act]()


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    W = st["W"].double()
    W = W if case["order"] == "row" else W.mT
    if op == "act":
        z = torch.mm(st["X"].double(), W)
        z = z if st["b"] is None else z + st["b"].double()
        y = _exact_act(z, case["act"])
        y = y if st["R"] is None else y + st["R"].double()
        return (y, z) if case["keep"] else y
    if op == "act_grad":
        z = st["Z"].double().requires_grad_()
        up = torch.mm(st["dY"].double(), W.mT)
        (d,) = torch.autograd.grad(_exact_act(z, case["act"]), z, up)
        return d, d.sum(0)
    if op in ("xent", "xent_grad"):
        X, t = st["X"].double(), st["targets"]
        counts, at = t != IGNORED, t - case["start"]
        mine = counts & (at >= 0) & (at < case["N"])
        lse, hit = [], []
        dX, dW = [], torch.zeros_like(W) if op == "xent_grad" else None
        for rows in torch.split(torch.arange(len(t), device="cuda"), 1024):
            z = X[rows] @ W
            if op == "xent":
                lse.append(torch.logsumexp(z, 1))
                hit.append(torch.where(mine[rows], z[torch.arange(len(rows)), at[rows].clamp(0, case["N"] - 1)], 0.0))
                continue
            p = torch.exp(z - st["lse"][rows].double()[:, None])
            sel = torch.nonzero(mine[rows])[:, 0]
            p[sel, at[rows][sel]] -= 1.0
            p = p * (st["g"][rows].double() * counts[rows])[:, None]
            dX.append(p @ W.mT)
            dW += X[rows].mT @ p
        if op == "xent":
            lse, hit = torch.cat(lse), torch.cat(hit)
            return torch.where(counts, lse - hit, torch.zeros_like(lse)), lse, hit
        return torch.cat(dX), dW
    off = st["offsets"].tolist()
    spans = [slice(a, b) for a, b in zip(off[:-1], off[1:])]
    if op == "grouped":
        return torch.cat([st["X"][s].double() @ W[e] for e, s in enumerate(spans)])
    d = st["dY"].double()
    return (torch.cat([d[s] @ W[e].mT for e, s in enumerate(spans)]),
            torch.stack([st["X"][s].double().mT @ d[s] for s in spans]))
