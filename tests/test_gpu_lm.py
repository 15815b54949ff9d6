"""Gated layers, log probabilities and distillation on the GPU against plain
implementations in 64 bits.

Tolerances are bounds, derived from the arithmetic as in test_gpu_fused.py (u =
2^-24, h = 2^-8): a product of K terms errs by (K + 16) u (|A| |B|)_ij, an
activation passes on 1.13 times its argument's error and errs by 2^-20 (1 +
z^2) itself, an exponential of d by 2^-22 (1 + |d|) relative, a sum of n terms
by (n + 16) u times the sum of their sizes.

Inputs on a coarse grid, whose products and sums fit fp32, give logits that
are exact in any order, with many equal ones: there the alternatives' indices
are compared as they are.
"""
from __future__ import annotations

import pytest

from sharded_fc_layer_amd import fcshard as F

torch = pytest.importorskip("torch")

from test_gpu_fused import (ACT_NAMES, ACTS, COL, H, ROW, U, act64, among_nans, gen, integers, log, normal,  # noqa: E402
                            same, shifted, slope64, stored, within)

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

INF = float("inf")

# one row to several tiles, odd and aligned; reductions of one value, of several slices, of whole and partial stages
SHAPES = [(1, 1, 1), (1, 2048, 520), (3, 31, 7), (16, 512, 384), (32, 264, 136), (33, 129, 130), (100, 1001, 77),
          (130, 72, 259), (257, 520, 300), (300, 40, 1032), (520, 776, 264)]
# enough tiles for the 256 x 256 ones: reductions of 8 and 10 stages of 64, a partial last stage, odd rows
WIDE = [(4096, 512, 2048), (4000, 640, 2056), (2600, 100, 1304), (4001, 600, 2051), (4100, 640, 760)]


# the 256 x 256 tiles with a partial last stage; the tiles of 64 rows (the lower ones would be too many, the reduction
# is too short to split)
LARGE_GLU = [(4096, 600, 2048), (4104, 200, 2056)]
LARGE_GRAD = [(4096, 512, 4096), (4000, 640, 4104), (4096, 600, 4096)]
LOW = [(250, 72, 3200), (256, 71, 3201)]


# ---- gated layers

def glu64(z, ez, N, act):
    """(Y, its error bound) of [G | U] = z with errors ez."""
    G, Up, eG, eU = z[:, :N], z[:, N:], ez[:, :N], ez[:, N:]
    a = act64(G, act)
    ea = 1.13 * eG + 2.0 ** -20 * (1 + G * G)
    y = a * Up
    return y, ea * (Up.abs() + eU) + a.abs() * eU + U * y.abs()


@pytest.mark.parametrize("shape", SHAPES + WIDE + LARGE_GLU + LOW)
@pytest.mark.parametrize("wo", [ROW, COL])
def test_fwd_glu(shape, wo):
    M, K, N = shape
    g = gen(M * 7 + K * 3 + N)
    X, W, b = normal(g, M, K), normal(g, K, 2 * N, scale=K ** -0.5), normal(g, 2 * N)
    ws = stored(W, wo)
    z0 = X.double() @ W.double()
    e0 = X.double().abs() @ W.double().abs()
    for act in ACTS:
        for bias, keep, f32 in ((None, False, False), (b, True, True), (None, True, False), (b, False, True)):
            out = F.fc_fwd_glu(X, ws, bias=bias, act=act, w_order=wo, keep_z=keep,
                               out_dtype=F.OUT_F32 if f32 else F.OUT_BF16)
            Y, Z = out if keep else (out, None)
            z = z0 if bias is None else z0 + b.double()
            ez = (K + 16) * U * (e0 if bias is None else e0 + b.double().abs())
            y, tol = glu64(z, ez, N, act)
            what = f"{shape} {wo} {ACT_NAMES[act]}"
            within(Y, y, tol if f32 else tol + H * (y.abs() + tol), what)
            if keep:
                within(Z, z, ez + H * (z.abs() + ez), what + " Z")


@pytest.mark.parametrize("shape", SHAPES + WIDE + [(700, 2050, 513)])
@pytest.mark.parametrize("wo", [ROW, COL])
def test_fwd_glu_integers_are_exact(shape, wo):
    M, K, N = shape
    g = gen(5)
    X, W, b = integers(g, M, K), integers(g, K, 2 * N), integers(g, 2 * N)
    z = (X.double() @ W.double() + b.double()).float()
    for act in (F.ACT_NONE, F.ACT_RELU):
        y = act64(z[:, :N], act) * z[:, N:]
        for align in (lambda t: t, shifted):
            Y, Z = F.fc_fwd_glu(align(X), align(stored(W, wo)), bias=align(b), act=act, w_order=wo,
                                out_dtype=F.OUT_F32, keep_z=True)
            assert torch.equal(Y, y) and torch.equal(Z, z.to(torch.bfloat16)), f"{shape} {wo}"
            out, kept = shifted(Y.to(torch.bfloat16)), shifted(Z)  # outputs at addresses that are not aligned
            F.fc_fwd_glu(X, stored(W, wo), bias=b, act=act, w_order=wo, out=out, z=kept)
            assert torch.equal(out, y.to(torch.bfloat16)) and torch.equal(kept, Z)


def glu_grad64(d, ed, Z, act):
    """(dZ, Y and their error bounds) for a gradient d of Y with errors ed."""
    K = d.shape[1]
    G, Up = Z.double().split(K, 1)
    a, s = act64(G, act), slope64(G, act)
    own = 2.0 ** -20 * (1 + G * G)  # of the activation and of its slope
    dG, dU = d * Up * s, d * a
    tG = ed * Up.abs() * 1.13 + (d.abs() + ed) * Up.abs() * own + 2 * U * dG.abs()
    tU = ed * a.abs() + (d.abs() + ed) * own + U * dU.abs()
    return torch.cat([dG, dU], 1), torch.cat([tG, tU], 1), a * Up, Up.abs() * own + U * (a * Up).abs()


def check_glu_grad(dZ, Y, db, want, tol, y, ty, M, what):
    within(dZ, want, tol + H * (want.abs() + tol), what + " dZ")
    if Y is not None:
        within(Y, y, ty + H * (y.abs() + ty), what + " Y")
    if db is not None:
        within(db, want.sum(0), tol.sum(0) + (M + 16) * U * (want.abs() + tol).sum(0), what + " db")


@pytest.mark.parametrize("shape", SHAPES + [(m, n, k) for m, k, n in WIDE] + [(4096, 100, 4096), (4100, 1100, 4104)] +
                         LARGE_GRAD + [(m, k, 2 * n) for m, k, n in LOW])
@pytest.mark.parametrize("wo", [ROW, COL])
def test_bwd_data_glu(shape, wo):
    M, N, K = shape  # the reduction runs over the layer's outputs N
    g = gen(M + K * 5 + N * 11)
    dY, W, Z = normal(g, M, N, scale=1e-3), normal(g, K, N, scale=0.02), normal(g, M, 2 * K)
    ws = stored(W, wo)
    up = dY.double() @ W.double().t()
    e_up = (N + 16) * U * (dY.double().abs() @ W.double().abs().t())
    for act in ACTS:
        want, tol, y, ty = glu_grad64(up, e_up, Z, act)
        what = f"{shape} {wo} {ACT_NAMES[act]}"
        dZ, Y, db = F.fc_bwd_data_glu(dY, ws, Z, act, w_order=wo, keep_y=True, bias_grad=True)
        check_glu_grad(dZ, Y, db, want, tol, y, ty, M, what)
        assert torch.equal(F.fc_bwd_data_glu(dY, ws, Z, act, w_order=wo), dZ)
        got = F.fc_bwd_data_glu(shifted(dY), shifted(ws), shifted(Z), act, w_order=wo, out=shifted(dZ), y=shifted(Y))
        check_glu_grad(got[0], got[1], None, want, tol, y, ty, M, what + " shifted")


@pytest.mark.parametrize("shape", [(1, 1), (1, 300), (5, 7), (33, 256), (700, 130), (4100, 264), (64, 5000)])
def test_bwd_glu(shape):
    M, N = shape
    g = gen(M + N)
    dY, Z = normal(g, M, N), normal(g, M, 2 * N, scale=2.0)
    for act in ACTS:
        want, tol, y, ty = glu_grad64(dY.double(), torch.zeros((M, N), device="cuda"), Z, act)
        for align in (lambda t: t, shifted):
            dZ, Y, db = F.fc_bwd_glu(align(dY), align(Z), act, keep_y=True, bias_grad=True)
            check_glu_grad(dZ, Y, db, want, tol, y, ty, M, f"{shape} {ACT_NAMES[act]}")
        none, Y2, none2 = F.fc_bwd_glu(dY, Z, act, keep_dz=False, keep_y=True)
        assert none is None and none2 is None and torch.equal(Y2, Y)
        none, none2, db2 = F.fc_bwd_glu(dY, Z, act, keep_dz=False, bias_grad=True)
        assert none is None and none2 is None and torch.equal(db2, db)


def test_glu_gradient_by_differences():
    """Directional differences of the layer's own fp32 output."""
    M, K, N = 24, 40, 72
    g = gen(3)
    X, W = normal(g, M, K), normal(g, K, 2 * N, scale=0.2)
    R = normal(g, M, N)  # the loss: sum of R * Y
    for act in ACTS:
        Y, Z = F.fc_fwd_glu(X, W, act=act, keep_z=True, out_dtype=F.OUT_F32)
        dZ, _, _ = F.fc_bwd_glu(R, Z, act)
        dX = F.fc_bwd_data(dZ, W, out_dtype=F.OUT_F32)
        V = torch.where(torch.rand((M, K), device="cuda", generator=g) < 0.5, -1.0, 1.0) * 2.0 ** -5
        Xa, Xb = (X.float() + V).to(torch.bfloat16), (X.float() - V).to(torch.bfloat16)
        step = Xa.double() - Xb.double()
        ya, yb = (F.fc_fwd_glu(x, W, act=act, out_dtype=F.OUT_F32).double() for x in (Xa, Xb))
        diff, ours = (R.double() * (ya - yb)).sum().item(), (step * dX.double()).sum().item()
        # the slope in the middle of the step differs from the mean one by third derivatives (a bounded
        # multiple of the swing's cube; relu's kink: by the swing itself, where the gate changes its sign)
        z, swing = X.double() @ W.double(), (step @ W.double()).abs()
        big = 1 + z[:, N:].abs() + swing[:, N:]
        third = swing[:, :N] ** 2 * (swing[:, :N] * big + swing[:, N:])
        if act == F.ACT_RELU:
            third = torch.where(z[:, :N].abs() <= swing[:, :N], swing[:, :N] * big, 0.0)
        # the middle of the rounded steps is off X by at most 2^-8 |X|, dZ and Z are rounded to bf16
        mid = (H * X.double().abs()) @ W.double().abs()
        slack = (swing[:, :N] * (mid[:, :N] * big + mid[:, N:]) + swing[:, N:] * mid[:, :N]) * 2
        zs = 3 * H * (swing[:, :N] * (1 + z[:, N:].abs()) * (1 + z[:, :N].abs()) + swing[:, N:] * (1 + z[:, :N].abs()))
        assert abs(diff - ours) <= (R.double().abs() * (third + slack + zs)).sum().item() + 1e-4, ACT_NAMES[act]


def test_glu_values_at_the_ends():
    """Infinities and NaN in gate and up columns stay in their place."""
    M, K, N = 4, 1, 40
    X = torch.ones((M, K), dtype=torch.bfloat16, device="cuda")
    W = torch.linspace(-30, 30, 2 * N, device="cuda").to(torch.bfloat16)[None].repeat(K, 1)
    W[0, 3], W[0, N + 5], W[0, 7] = float("nan"), INF, 3e38
    for act in ACTS:
        Y, Z = F.fc_fwd_glu(X, W, act=act, keep_z=True, out_dtype=F.OUT_F32)
        z = X.double() @ W.double()
        want = act64(z[:, :N], act) * z[:, N:]
        rest = [i for i in range(N) if i not in (3, 5, 7)]
        assert bool(torch.isnan(Y[:, 3]).all()) and bool(torch.isnan(Z[:, 3]).all())
        assert torch.equal(Z[:, N + 5].float(), torch.full((M,), INF, device="cuda"))
        G, Up = z[:, :N][:, rest], z[:, N:][:, rest]
        within(Y[:, rest], want[:, rest], Up.abs() * 2.0 ** -20 * (1 + G * G) + U * want[:, rest].abs(), ACT_NAMES[act])


@pytest.mark.parametrize("shape", [(4000, 640, 2056), (4001, 640, 2051), (333, 611, 531), (40, 512, 264), (5, 2048, 40)])
@pytest.mark.parametrize("wo", [ROW, COL])
def test_glu_bias_gradient_of_infinite_weights(shape, wo):
    """An infinite weight's column of dZ is infinite or NaN, and no other."""
    M, N, K = shape
    g = gen(2)
    dY, W, Z = integers(g, M, N), integers(g, K, N), normal(g, M, 2 * K)
    dY[:, 0] = 1.0
    W[K // 2, 0] = INF
    _, db = F.fc_bwd_data_glu(dY, stored(W, wo), Z, F.ACT_SILU, w_order=wo, bias_grad=True)
    bad = torch.zeros(2 * K, dtype=torch.bool, device="cuda")
    bad[K // 2] = bad[K + K // 2] = True
    assert bool(torch.isfinite(db[~bad]).all()) and not bool(torch.isfinite(db[bad]).any())


# ---- log probabilities

VOCAB = [(1, 8, 1), (1, 64, 1000), (1, 2048, 5000), (5, 33, 130), (32, 128, 129), (33, 100, 999), (64, 264, 4001),
         (130, 72, 520), (300, 65, 2050), (600, 96, 3000), (40, 4104, 700), (96, 2001, 300), (1500, 64, 1000)]
VOCAB_WIDE = [(4096, 512, 4096), (4000, 640, 4104), (2309, 131, 3001), (4001, 600, 4099), (2600, 100, 2600)]


def grid(g, *shape, top=3):
    """Multiples of a quarter: products of up to 4096 of them sum exactly in fp32."""
    return integers(g, *shape, top=top) * 0.25


def logprob64(X, W, targets, v0, T, ignore=-100):
    z = X.double() @ W.double()
    s = z / T
    lse = torch.logsumexp(s, 1)
    at = targets - v0
    here = (at >= 0) & (at < W.shape[1])
    hit = torch.where(here, s.gather(1, torch.where(here, at, 0)[:, None])[:, 0], -INF)
    logp = torch.where(targets == ignore, 0.0, hit - lse)
    p = torch.exp(s - lse[:, None])
    entropy = -(torch.where(p > 0, p * (s - lse[:, None]), 0.0)).sum(1)
    return z, s, lse, logp, p, entropy


def check_logprob(X, ws, W, wo, t, v0, T, k, ez=0.0, ids=True, what=""):
    N = W.shape[1]
    z, s, lse, logp, p, entropy = logprob64(X, W, t, v0, T)
    got = F.fc_logprob(X, ws, t, w_order=wo, vocab_start=v0, temperature=T, top_k=k)
    # exponentials' errors weighted by p (|d| e^d <= 1 where it is negative), the sum's, the scaling's by 1 / T
    e_s = ez / T + 3 * U * s.abs().max(1).values
    e_lse = e_s + 2.0 ** -20 + (N + 16) * U + 4 * U * lse.abs()
    within(got[2], lse, e_lse, what + " lse")
    fin = torch.isfinite(logp)
    assert torch.equal(torch.isfinite(got[0]), fin) and bool((got[0][~fin] == -INF).all())
    within(got[0][fin], logp[fin], (2 * e_lse + 2 * U * logp.abs())[fin], what + " logp")
    # log s - w / s: the mean distance from the maximum, and the weights' relative errors of each term
    far = (p * (s.max(1).values[:, None] - s)).sum(1)
    e_ent = 2 * e_s * (1 + entropy) + (2.0 ** -20 + (N + 16) * U) * (2 + entropy.abs() + 4 * far) + \
        2.0 ** -21 * (p * (s.max(1).values[:, None] - s) ** 2).sum(1)
    within(got[1], entropy, e_ent, what + " entropy")
    best = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]
    if ids:
        assert torch.equal(got[4], best + v0), what + " ids"
    want = s.gather(1, best) - lse[:, None]
    within(got[3], want, (2 * e_lse)[:, None] + 2 * U * want.abs(), what + " top")
    if not ids and k:  # the indices belong to the values, each once
        own = s.gather(1, got[4] - v0) - lse[:, None]
        within(got[3], own, (2 * e_lse)[:, None] + 2 * U * own.abs(), what + " values at ids")
        assert bool((torch.sort(got[4], 1).values.diff(dim=1) > 0).all())
    return got


@pytest.mark.parametrize("shape", VOCAB + VOCAB_WIDE)
@pytest.mark.parametrize("wo", [ROW, COL])
def test_logprob(shape, wo):
    M, K, N = shape
    g = gen(M + 3 * K + N)
    X, W = grid(g, M, K), grid(g, K, N)
    for v0, T, k in ((0, 1.0, 5), (N, 0.5, min(N, 64)), (7, 2.0, min(N, 128)), (0, 1.0, 0), (0, 64.0, 1)):
        t = torch.randint(v0, v0 + N + N // 4 + 1, (M,), device="cuda", generator=g)
        t[::4] = -100
        check_logprob(X, stored(W, wo), W, wo, t, v0, T, min(k, N), what=f"{shape} {wo} {v0} {T} {k}")


@pytest.mark.parametrize("shape", VOCAB + VOCAB_WIDE)
def test_logprob_normal_inputs(shape):
    M, K, N = shape
    g = gen(M + K + N)
    X, W = normal(g, M, K), normal(g, K, N, scale=0.3)
    ez = (K + 16) * U * (X.double().abs() @ W.double().abs()).max(1).values
    t = torch.randint(0, N, (M,), device="cuda", generator=g)
    for wo in (ROW, COL):
        check_logprob(X, stored(W, wo), W, wo, t, 0, 1.0, min(N, 20), ez=ez, ids=False, what=f"{shape} {wo}")
        x, w = shifted(X), shifted(stored(W, wo))
        check_logprob(x, w, W, wo, t, 0, 0.7, min(N, 100), ez=ez, ids=False, what=f"{shape} {wo} shifted")


@pytest.mark.parametrize("shape", [(1, 16, 3000), (70, 64, 1000), (700, 520, 4000), (4096, 512, 4096), (2050, 64, 2000)])
@pytest.mark.parametrize("k", [1, 64, 65, 128])
def test_logprob_ties(shape, k):
    """Rows of equal logits, of two values, and whose largest all lie in one place."""
    M, K, N = shape
    X = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    W = torch.zeros((K, N), dtype=torch.bfloat16, device="cuda")
    W[1] = (torch.arange(N, device="cuda") % 3 == 1).to(torch.bfloat16)
    W[2, N - 200:] = torch.arange(200, device="cuda") // 2
    W[3] = -(torch.arange(N, device="cuda") // 256).to(torch.bfloat16)
    W[4] = (torch.arange(N, device="cuda") // 256).to(torch.bfloat16)
    for r in range(M):
        if r % 5:
            X[r, r % 5] = 1.0
    t = torch.arange(M, device="cuda") % N
    for wo in (ROW, COL):
        check_logprob(X, stored(W, wo), W, wo, t, 0, 1.0, k, what=f"{shape} {wo} {k}")
    X[:] = 0.0
    _, entropy, lse, top, ids = F.fc_logprob(X, W, top_k=k)
    assert torch.equal(ids, torch.arange(k, device="cuda").repeat(M, 1))
    log_n = torch.log(torch.tensor(float(N), dtype=torch.float64)).cuda()
    for x, s in ((entropy, 1), (lse, 1), (top, -1)):
        within(x, (s * log_n).expand(x.shape), torch.full_like(x, 2.0 ** -19 + (N + 16) * U, dtype=torch.float64), "log N")


@pytest.mark.parametrize("shape", [(40, 3000), (1100, 4096), (4200, 4000), (9, 40000)])
@pytest.mark.parametrize("k", [5, 64, 128])
def test_logprob_of_sorted_rows(shape, k):
    """Rising, falling and interleaved rows of different values, and steps: what comes first is not what counts."""
    M, N = shape
    i = torch.arange(N, device="cuda")
    orders = torch.stack([i, N - 1 - i, (i * 7919) % N, i // 150, (N - 1 - i) // 150, i % 2 * 1000 + i // 300])
    W = torch.cat([orders // 128, orders % 128]).to(torch.bfloat16)  # exact: under 256 each
    X = torch.zeros((M, 12), dtype=torch.bfloat16, device="cuda")
    r = torch.arange(M, device="cuda")
    X[r, r % 6], X[r, 6 + r % 6] = 1.0, 2.0 ** -7
    if N > 32768:
        W[:6] = W[:6] * (W[:6] < 256)  # (bf16 holds these, but no more digits)
    t = r % N
    for wo in (ROW, COL):
        check_logprob(X, stored(W, wo), W, wo, t, 0, 1.0, k, what=f"{shape} {wo} {k}")


def test_logprob_of_rows_that_are_not_finite():
    """NaN and infinities: their own rows alone, and indices that are columns."""
    for M, K, N in ((6, 16, 300), (2600, 72, 2600), (600, 16, 1000)):
        X, W = normal(gen(4), M, K), normal(gen(5), K, N, scale=0.1)
        X[0], X[3], X[M - 1] = float("nan"), INF, -INF
        W[:, 5] = 0.0
        bad = torch.zeros(M, dtype=torch.bool, device="cuda")
        bad[[0, 3, M - 1]] = True
        t = torch.arange(M, device="cuda") % N
        ez = (K + 16) * U * (X[~bad].double().abs() @ W.double().abs()).max(1).values
        z, s, lse, logp, p, entropy = logprob64(X[~bad], W, t[~bad], 0, 1.0)
        for wo in (ROW, COL):
            got = F.fc_logprob(X, stored(W, wo), t, w_order=wo, top_k=100)
            assert bool(((got[4] >= 0) & (got[4] < N)).all())
            assert bool((torch.sort(got[4], 1).values.diff(dim=1) > 0).all())  # each once
            assert bool(torch.isnan(got[2][0]).all())
            within(got[2][~bad], lse, ez + 2.0 ** -20 + (N + 16) * U + 4 * U * lse.abs(), "lse")
            want = torch.sort(z, 1, descending=True).values[:, :100] - lse[:, None]
            within(got[3][~bad], want, (2 * ez + 2.0 ** -18)[:, None] + 4 * U * want.abs(), "top")
    one = torch.tensor([[INF], [-INF]], device="cuda").to(torch.bfloat16)  # K = 1: no zero times infinity
    logp, entropy, lse, top, ids = F.fc_logprob(one, torch.ones((1, 300), dtype=torch.bfloat16, device="cuda"),
                                                torch.zeros(2, dtype=torch.int64, device="cuda"), top_k=3)
    assert lse[0].item() == INF and lse[1].item() == -INF and logp[1].item() == -INF
    assert ids.tolist() == [[0, 1, 2], [0, 1, 2]]
    # logits at the type's ends: one that has all the probability
    W = torch.full((1, 400), -3e38, device="cuda").to(torch.bfloat16)
    W[0, 77] = 3e38
    for T in (1.0, 2.0 ** -10, 2.0 ** 10):
        logp, entropy, lse, top, ids = F.fc_logprob(torch.ones((1, 1), dtype=torch.bfloat16, device="cuda"), W,
                                                    torch.tensor([77], device="cuda"), temperature=T, top_k=2)
        assert logp.item() == 0 and entropy.item() == 0 and ids.tolist() == [[77, 0]] and top[0, 0].item() == 0


def test_logprob_shards_join_to_the_whole():
    M, K, N = 70, 136, 1000
    g = gen(8)
    X, W = grid(g, M, K), grid(g, K, N)
    t = torch.randint(0, N, (M,), device="cuda", generator=g)
    logp, entropy, lse, top, ids = F.fc_logprob(X, W, t, top_k=30)
    cuts = [0, 40, 301, 640, 1000]
    parts = [F.fc_logprob(X, W[:, a:b].contiguous(), t, vocab_start=a, top_k=30) for a, b in zip(cuts, cuts[1:])]
    L = torch.logsumexp(torch.stack([p[2].double() for p in parts]), 0)
    within(lse, L, 2.0 ** -18 * (1 + L.abs()), "lse")
    best = torch.stack([p[0].double() + p[2].double() for p in parts]).max(0).values - L
    within(logp, best, 2.0 ** -17 * (1 + L.abs()), "logp")
    ent = sum(torch.exp(p[2].double() - L) * (p[1].double() + L - p[2].double()) for p in parts)
    within(entropy, ent, 2.0 ** -15 * (1 + L.abs()), "entropy")
    values = torch.cat([p[3].double() + p[2].double()[:, None] for p in parts], 1)
    order = torch.sort(values, dim=1, descending=True, stable=True)
    within(top, order.values[:, :30] - L[:, None], 2.0 ** -17 * (1 + L.abs())[:, None], "top")


def test_logprob_of_rows_in_several_chunks():
    """A vocabulary whose rows of logits do not fit the workspace at once."""
    M, K, N = 530, 40, 530001
    g = gen(12)
    X, W = grid(g, M, K), grid(g, K, N, top=7)
    t = torch.randint(0, N, (M,), device="cuda", generator=g)
    need = F.lib().fc_logprob_ws_bytes(M, K, N, ROW, 40, 1)
    assert need < 3 * 256 * N * 4  # fewer rows at once than there are
    logp, entropy, lse, top, ids = F.fc_logprob(X, W, t, top_k=40)
    n_ids, teacher = ids[:, :9].contiguous(), top[:, :9].contiguous()
    loss, lse2, sl = F.fc_distill_fwd(X, W, n_ids, teacher)
    for r in torch.split(torch.arange(M, device="cuda"), 100):
        z = X[r].double() @ W.double()
        want = torch.logsumexp(z, 1)
        tol = 2.0 ** -20 + (N + 16) * U + 4 * U * want.abs()
        # (the two calls may join the parts of a row in another order: each is within the bound of any order)
        within(lse[r], want, tol, "lse")
        within(lse2[r], want, tol, "lse of the distillation")
        best = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :40]
        assert torch.equal(ids[r], best)
        assert torch.equal(sl[r].double(), z.gather(1, n_ids[r]))


# rows whose parts' maxima fit a block's LDS with 16 rows to it, or do not (896 parts of 128 columns), or with one
# row (14336 parts of 32); and of more rows than one chunk has
@pytest.mark.parametrize("shape", [(2100, 24, 100003), (2304, 16, 115008), (3, 24, 530001), (1100, 16, 260000)])
@pytest.mark.parametrize("k", [5, 128])
def test_logprob_of_wide_rows(shape, k):
    M, K, N = shape
    g = gen(N)
    X, W = grid(g, M, K), grid(g, K, N, top=7)
    t = torch.randint(0, N, (M,), device="cuda", generator=g)
    ws = stored(W, COL)
    logp, entropy, lse, top, ids = F.fc_logprob(X, ws, t, w_order=COL, top_k=k)
    for r in torch.split(torch.arange(M, device="cuda"), 200):
        z, s, want, wl, p, ent = logprob64(X[r], W, t[r], 0, 1.0)
        tol = 2.0 ** -20 + (N + 16) * U + 4 * U * want.abs()
        within(lse[r], want, tol, f"{shape} lse")
        within(logp[r], wl, 2 * tol + 2 * U * wl.abs(), "logp")
        assert torch.equal(ids[r], torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k])


# ---- distillation

def teacher(g, M, n, low, high, absent=0.3):
    """Listed tokens low .. high - 1, some twice in a row, some absent, some rows without any."""
    ids = torch.randint(low, high, (M, n), device="cuda", generator=g)
    if n > 2:
        ids[:, n - 1] = ids[:, 0]  # the same token twice
    drop = torch.rand((M, n), device="cuda", generator=g) < absent
    ids[drop] = -1 - torch.randint(0, 5, (int(drop.sum()),), device="cuda", generator=g)
    ids[1::7] = -1
    tl = torch.randn((M, n), device="cuda", generator=g) * 3
    tl[2::9, 0] = -INF  # absent too
    return ids, tl


def distill64(X, W, ids, tl, v0, T):
    z = X.double() @ W.double()
    there = (ids >= 0) & (tl != -INF)
    any_ = there.any(1)
    t = torch.where(there, tl.double() / T, -INF)
    t = torch.where(any_[:, None], t, 0.0)
    p = torch.where(there, torch.softmax(t, 1), 0.0)
    logp = torch.where(there, torch.log_softmax(t, 1), 0.0)
    at = ids - v0
    here = there & (at >= 0) & (at < W.shape[1])
    at = torch.where(here, at, 0)
    sl = torch.where(here, z.gather(1, at), 0.0)
    return z, there, any_, p, logp, here, at, sl


LISTED = [1, 2, 21, 64, 65, 128]


@pytest.mark.parametrize("shape", VOCAB + VOCAB_WIDE)
@pytest.mark.parametrize("wo", [ROW, COL])
def test_distill_fwd(shape, wo):
    M, K, N = shape
    g = gen(M + 3 * K + N)
    X, W = normal(g, M, K), normal(g, K, N, scale=0.3)
    ez = (K + 16) * U * (X.double().abs() @ W.double().abs())
    for i, (v0, whole, T) in enumerate(((0, N, 1.0), (N, 3 * N, 2.0), (5, N + 5, 0.5))):
        n = LISTED[(M + N + i) % 6]
        ids, tl = teacher(g, M, n, 0, whole)
        z, there, any_, p, logp, here, at, sl = distill64(X, W, ids, tl, v0, T)
        loss, lse, slogits = F.fc_distill_fwd(X, stored(W, wo), ids, tl, w_order=wo, vocab_start=v0, temperature=T)
        what = f"{shape} {wo} {v0} {T} {n}"
        want = torch.logsumexp(z / T, 1)
        e_lse = (ez.max(1).values + 3 * U * z.abs().max(1).values) / T + 2.0 ** -20 + (N + 16) * U + 4 * U * want.abs()
        within(lse, want, e_lse, what + " lse")
        e_sl = torch.where(here, ez.gather(1, at), 0.0)
        within(slogits, sl, e_sl, what + " slogits")
        term = logp - sl / T + want[:, None]
        size = logp.abs() + sl.abs() / T + want.abs()[:, None]
        # p's relative error: its exponential's, the scaled logits' rounding, the normaliser's
        ep = 2.0 ** -20 * (1 + logp.abs()) + 4 * U * (tl.double() / T).abs().where(there, 0.0).amax(1, keepdim=True)
        e_term = e_sl / T + e_lse[:, None] + 4 * U * size + ep
        tol = (p * (ep * term.abs() + e_term)).sum(1) + (n + 16) * U * (p * term.abs()).sum(1)
        within(loss, torch.where(any_, (p * term).sum(1), 0.0), tol + 2.0 ** -126, what + " loss")
        assert bool((loss[~any_] == 0).all()) and bool((slogits[~here] == 0).all())


def test_one_listed_token_is_the_cross_entropy():
    M, K, N = 130, 136, 1000
    g = gen(8)
    X, W = normal(g, M, K), normal(g, K, N, scale=0.3)
    t = torch.randint(0, N, (M,), device="cuda", generator=g)
    t[::5] = -100
    loss, lse, tl = F.fc_xent_fwd(X, W, t)
    got, lse2, sl = F.fc_distill_fwd(X, W, t[:, None].contiguous(), torch.randn((M, 1), device="cuda", generator=g))
    within(got, loss.double(), 2.0 ** -18 * (1 + lse.double().abs()), "loss")
    within(lse2, lse.double(), 2.0 ** -18 * (1 + lse.double().abs()), "lse")
    w = torch.rand(M, device="cuda", generator=g)
    a = F.fc_xent_bwd(X, W, t, lse, w, dx_dtype=F.OUT_F32, dw_dtype=F.OUT_F32)
    b = F.fc_distill_bwd(X, W, t[:, None].contiguous(), torch.zeros((M, 1), device="cuda"), tl[:, None].contiguous(),
                         lse, w, dx_dtype=F.OUT_F32, dw_dtype=F.OUT_F32)
    assert same(a, b)  # the same gradient of the logits, bit for bit


def check_distill_bwd(shape, wo, v0, whole, T, n, seed):
    M, K, N = shape
    g = gen(seed)
    X, W = normal(g, M, K), normal(g, K, N, scale=0.3)
    ids, tl = teacher(g, M, n, 0, whole)
    z, there, any_, p, logp, here, at, sl = distill64(X, W, ids, tl, v0, T)
    ez = (K + 16) * U * (X.double().abs() @ W.double().abs())
    s = z / T
    lse = (torch.logsumexp(s, 1) + (1.0 if v0 else 0.0)).float()  # a shard's probabilities sum to less than 1
    w = torch.rand(M, device="cuda", generator=g) - 0.3
    q = torch.exp(s - lse.double()[:, None])
    eq = q * torch.expm1(ez / T + 2.0 ** -22 * (1 + s.abs() + lse.double().abs()[:, None]))
    hot, ehot = torch.zeros_like(q), torch.zeros_like(q)
    ep = 2.0 ** -20 * (1 + logp.abs()) + 4 * U * (tl.double() / T).abs().where(there, 0.0).amax(1, keepdim=True)
    hot.scatter_add_(1, at, torch.where(here, p, 0.0))
    ehot.scatter_add_(1, at, torch.where(here, p * (ep + n * U), 0.0))
    wc = torch.where(any_, w.double() / T, 0.0)[:, None]
    D = wc * (q - hot)
    eD = wc.abs() * (eq + ehot + 4 * U * (q + hot))
    eD = eD + H * (D.abs() + eD)
    # numbers under 2^-126 may be flushed to zero: a probability (the logits at T = 1 / 2 spread over 200), its
    # product with the weight, and D where the matrix units read it
    eD = eD + (wc.abs() + 2) * 2.0 ** -126
    aX, aW, aD = X.double().abs(), W.double().abs(), D.abs() + eD
    # ... and each product of a sum
    tx = eD @ aW.t() + (N + 16) * U * (aD @ aW.t()) + (N + 16) * 2.0 ** -126
    tw = aX.t() @ eD + (M + 16) * U * (aX.t() @ aD) + (M + 16) * 2.0 ** -126
    wx, ww = D @ W.double().t(), X.double().t() @ D
    what = f"{shape} {wo} {v0} {T} {n}"
    sls = sl.float()
    dX, dW = F.fc_distill_bwd(X, stored(W, wo), ids, tl, sls, lse, w, w_order=wo, vocab_start=v0, temperature=T)
    within(dX, wx, tx + H * (wx.abs() + tx), what + " dX")
    within(dW, ww, tw + H * (ww.abs() + tw), what + " dW")
    assert bool((dX[~any_] == 0).all())
    acc = torch.ones((K, N), device="cuda")
    dX, dW = F.fc_distill_bwd(X, stored(W, wo), ids, tl, sls, lse, w, w_order=wo, vocab_start=v0, temperature=T,
                              dx_dtype=F.OUT_F32, dW=acc, dw_dtype=F.OUT_F32_ACC)
    within(dX, wx, tx, what + " dX fp32")
    within(dW, ww + 1, tw + U * (ww.abs() + tw + 1), what + " dW accumulated")


@pytest.mark.parametrize("shape", VOCAB + VOCAB_WIDE + [(4096, 2048, 4096), (4099, 2049, 4103)])
@pytest.mark.parametrize("wo", [ROW, COL])
def test_distill_bwd(shape, wo):
    M, K, N = shape
    for i, (v0, whole, T) in enumerate(((0, N, 1.0), (N, 3 * N, 2.0), (3, N + 9, 0.5))):
        check_distill_bwd(shape, wo, v0, whole, T, LISTED[(M + N + i) % 6], M + 5 * K + N + i)


def test_distill_bwd_in_several_pieces():
    """A vocabulary of more columns than one piece of the logits' gradient holds: tokens of one row lie in several."""
    M, K, N = 16500, 40, 17001  # pieces of 7936 columns
    g = gen(12)
    X, W = normal(g, M, K), normal(g, K, N, scale=0.3)
    ids, tl = teacher(g, M, 12, 0, N)
    for wo in (ROW, COL):
        loss, lse, sl = F.fc_distill_fwd(X, stored(W, wo), ids, tl, w_order=wo, temperature=2.0)
        w = torch.full((M,), 1.0 / M, device="cuda")
        dX, dW = F.fc_distill_bwd(X, stored(W, wo), ids, tl, sl, lse, w, w_order=wo, temperature=2.0)
        wW, tW = (torch.zeros((K, N), dtype=torch.float64, device="cuda") for _ in range(2))
        for r in torch.split(torch.arange(M, device="cuda"), 4096):
            z, there, any_, p, logp, here, at, _ = distill64(X[r], W, ids[r], tl[r], 0, 2.0)
            D = torch.exp(z / 2 - lse[r].double()[:, None])
            q = D.clone()
            D.scatter_add_(1, at, torch.where(here, -p, 0.0))
            D *= torch.where(any_, 0.5 / M, 0.0)[:, None]
            # D errs by its rounding, by 2^-16 of the probabilities on either side (|z| + |lse| below 40)
            hot = torch.zeros_like(q).scatter_add_(1, at, torch.where(here, p, 0.0))
            eD = H * D.abs() + 2.0 ** -16 / M * (q + hot)
            wX, tX = D @ W.double().t(), (eD + (N + 16) * U * D.abs()) @ W.double().abs().t()
            within(dX[r], wX, tX + H * (wX.abs() + tX), f"{wo} dX")
            wW += X[r].double().t() @ D
            tW += X[r].double().abs().t() @ (eD + (M + 16) * U * D.abs())
        within(dW, wW, tW + H * (wW.abs() + tW), f"{wo} dW")


def test_distill_rows_that_do_not_count():
    """Rows of NaN and infinities without tokens: no loss, no gradient, no other row disturbed."""
    for M, K, N in ((130, 72, 520), (4096, 512, 4096), (4001, 600, 4099)):
        g = gen(K)
        X, W = normal(g, M, K), normal(g, K, N, scale=0.1)
        ids, tl = teacher(g, M, 9, 0, N, absent=0.0)
        out = torch.tensor([5, 128, M // 2, M - 2, M - 1], device="cuda")
        X[out[::2]], X[out[1::2]] = float("nan"), INF
        ids[out] = -1
        tl[out] = float("nan")
        any_ = (ids >= 0).any(1)
        w = torch.ones(M, device="cuda")
        w[out] = float("nan")
        for wo in (ROW, COL):
            loss, lse, sl = F.fc_distill_fwd(X, stored(W, wo), ids, tl, w_order=wo)
            assert bool((loss[~any_] == 0).all()) and bool(torch.isfinite(loss).all())
            dX, _ = F.fc_distill_bwd(X, stored(W, wo), ids, tl, sl, lse, w, w_order=wo)
            assert bool((dX[~any_] == 0).all()) and bool(torch.isfinite(dX).all())


def test_distill_gradient_by_differences():
    """Directional differences of the library's own loss."""
    M, K, N, n, T = 40, 64, 500, 9, 2.0
    g = gen(31)
    X, W = normal(g, M, K), normal(g, K, N, scale=0.2)
    ids, tl = teacher(g, M, n, 0, N)
    _, lse, sl = F.fc_distill_fwd(X, W, ids, tl, temperature=T)
    dX, _ = F.fc_distill_bwd(X, W, ids, tl, sl, lse, torch.ones(M, device="cuda"), temperature=T, dx_dtype=F.OUT_F32)
    V = torch.where(torch.rand((M, K), device="cuda", generator=g) < 0.5, -1.0, 1.0) * 2.0 ** -4
    Xa, Xb = (X.float() + V).to(torch.bfloat16), (X.float() - V).to(torch.bfloat16)
    step, mid = Xa.double() - Xb.double(), (Xa.double() + Xb.double()) / 2
    a, b = (F.fc_distill_fwd(x, W, ids, tl, temperature=T)[0].double() for x in (Xa, Xb))
    swing = (step @ W.double()).abs().max(1).values / T
    off = ((mid - X.double()) @ W.double()).abs().max(1).values / T
    # the third derivative along the step is at most 2 swing^3, the second 2 swing x off (softmax's moments);
    # the gradient's own error: D's rounding
    z, there, any_, p, logp, here, at, _ = distill64(X, W, ids, tl, 0, T)
    q = torch.softmax(z / T, 1)
    hot = torch.zeros_like(q).scatter_add_(1, at, torch.where(here, p, 0.0))
    own = (step.abs() * (H * ((q + hot) @ W.double().abs().t()) / T)).sum(1)
    bound = (swing ** 3 / 12 + 2 * swing * off + own + 2.0 ** -16).sum().item()
    assert abs((a - b).sum().item() - (step * dX.double()).sum().item()) <= bound


@pytest.mark.parametrize("shape", [(3, 256, 4000), (300, 64, 4100), (1200, 64, 2900), (2304, 64, 16032), (4096, 64, 1000)])
@pytest.mark.parametrize("wo", [ROW, COL])
def test_alternatives_of_about_as_many_parts(shape, wo):
    """Alternatives for fewer, as many and more than the parts of a row; values that repeat, and that do not."""
    M, K, N = shape
    g = gen(M + N)
    X, W = grid(g, M, K), grid(g, K, N)
    Xn, Wn = normal(g, M, K), normal(g, K, N, scale=0.3)
    ez = (K + 16) * U * (Xn.double().abs() @ Wn.double().abs()).max(1).values
    t = torch.randint(0, N, (M,), device="cuda", generator=g)
    for k in (7, 8, 23, 32, 72, 100, 101, 125, 128):
        check_logprob(X, stored(W, wo), W, wo, t, 0, 1.0, k, what=f"{shape} {wo} {k}")
        check_logprob(Xn, stored(Wn, wo), Wn, wo, t, 0, 1.0, k, ez=ez, ids=False, what=f"{shape} {wo} {k} normal")


# ---- few rows, W with its reduction contiguous: parts of 32 columns, many and few blocks, K at its least, partial pieces

FEW = [(1, 256, 1), (1, 2048, 8200), (3, 264, 31), (5, 2048, 33), (8, 2056, 1000), (9, 258, 9000), (16, 320, 20001),
       (16, 2048, 65), (8, 4090, 300)]


@pytest.mark.parametrize("shape", FEW)
def test_few_rows_of_logits(shape):
    test_logprob(shape, COL)
    test_logprob_normal_inputs(shape)
    test_distill_fwd(shape, COL)


@pytest.mark.parametrize("shape", [(3, 512, 4100), (20, 512, 4096)])
def test_few_rows_of_a_wide_gated_layer(shape):
    """Blocks of eight waves, for up to 16 and up to 32 rows."""
    test_fwd_glu(shape, COL)
    test_fwd_glu_integers_are_exact(shape, COL)


@pytest.mark.parametrize("k", [1, 64, 128])
def test_few_equal_rows(k):
    """All logits equal, and blocks of equal ones: the lowest indices."""
    M, K, N = 3, 256, 10000
    X, W = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda"), torch.zeros((K, N), dtype=torch.bfloat16, device="cuda")
    X[1:, 0] = 1.0
    W[0] = (torch.arange(N, device="cuda") // 50 % 7).to(torch.bfloat16)
    want = torch.sort(X.float() @ W.float(), dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(F.fc_logprob(X, stored(W, COL), w_order=COL, top_k=k)[4], want)


def test_few_rows_that_are_not_finite():
    M, K, N = 6, 256, 3000
    X, W = normal(gen(4), M, K), normal(gen(5), K, N, scale=0.1)
    X[0], X[3], X[5] = float("nan"), INF, -INF
    W[:, 5] = 0.0
    good = torch.tensor([1, 2, 4], device="cuda")
    ez = (K + 16) * U * (X[good].double().abs() @ W.double().abs()).max(1).values
    z, s, lse, logp, p, entropy = logprob64(X[good], W, good, 0, 1.0)
    got = F.fc_logprob(X, stored(W, COL), torch.arange(M, device="cuda"), w_order=COL, top_k=100)
    assert bool(((got[4] >= 0) & (got[4] < N)).all())
    assert bool((torch.sort(got[4], 1).values.diff(dim=1) > 0).all())  # each once
    assert bool(torch.isnan(got[2][0]))
    within(got[2][good], lse, ez + 2.0 ** -20 + (N + 16) * U + 4 * U * lse.abs(), "lse")
    want = torch.sort(z, 1, descending=True).values[:, :100] - lse[:, None]
    within(got[3][good], want, (2 * ez + 2.0 ** -18)[:, None] + 4 * U * want.abs(), "top")
    # one infinite logit, one of -inf, the others finite
    X, W = torch.zeros((2, K), dtype=torch.bfloat16, device="cuda"), torch.zeros((K, N), dtype=torch.bfloat16, device="cuda")
    X[:, 0] = 1.0
    W[0, 40], W[0, 41] = -INF, 1.0
    logp, entropy, lse, top, ids = F.fc_logprob(X, stored(W, COL), torch.tensor([40, 41], device="cuda"), w_order=COL,
                                                top_k=2)
    full = torch.log(torch.tensor(N - 2 + 2.718281828459045, dtype=torch.float64)).item()
    within(lse, torch.full((2,), full, device="cuda").double(), (N + 16) * U + 2.0 ** -20 + 4 * U * full, "lse")
    assert logp[0].item() == -INF and ids.tolist() == [[41, 0]] * 2


@pytest.mark.parametrize("shape", [(4096, 512, 2048), (3, 512, 2048), (300, 520, 264)])
def test_glu_bias_at_any_element(shape):
    """Operands on 16-byte boundaries, the bias alone at odd elements."""
    M, K, N = shape
    g = gen(6)
    X, W, b = integers(g, M, K), integers(g, K, 2 * N), integers(g, 2 * N)
    z = (X.double() @ W.double() + b.double()).float()
    y = act64(z[:, :N], F.ACT_RELU) * z[:, N:]
    for wo in (ROW, COL):
        for bias in (b, shifted(b)):
            Y, Z = F.fc_fwd_glu(X, stored(W, wo), bias=bias, act=F.ACT_RELU, w_order=wo, out_dtype=F.OUT_F32, keep_z=True)
            assert torch.equal(Y, y) and torch.equal(Z, z.to(torch.bfloat16))
            Y = F.fc_fwd_glu(X, stored(W, wo), bias=bias, act=F.ACT_RELU, w_order=wo)
            assert torch.equal(Y, y.to(torch.bfloat16))


# ---- memory, streams, graphs

@pytest.mark.parametrize("shape", [(1, 1, 1), (2, 9, 2), (65, 7, 3), (129, 33, 1), (70, 39, 5), (16, 264, 24),
                                   (33, 2051, 35), (100, 1000, 136), (2600, 70, 1285)])
@pytest.mark.parametrize("offset", [0, 1, 4])
def test_nothing_past_the_operands_counts(shape, offset):
    M, K, N = shape
    g = gen(M + K + N)
    X, W, b, dY = integers(g, M, K), integers(g, K, 2 * N), integers(g, 2 * N), integers(g, M, 2 * N)
    z = X.float() @ W.float() + b.float()
    y = torch.clamp(z[:, :N], min=0) * z[:, N:]
    up = dY.float() @ W.float().t()
    Z = integers(g, M, 2 * K)
    G, Up = Z[:, :K].float(), Z[:, K:].float()
    dZ = torch.cat([up * Up * (G > 0), up * torch.clamp(G, min=0)], 1)
    small = 2.0 ** -4
    t = torch.randint(0, 2 * N, (M,), device="cuda", generator=g)
    ids, tl = teacher(g, M, 3, 0, 2 * N)
    for wo in (ROW, COL):
        x, w = among_nans(X, offset), among_nans(stored(W, wo), offset)
        Y = F.fc_fwd_glu(x, w, bias=among_nans(b, offset), act=F.ACT_RELU, w_order=wo, out_dtype=F.OUT_F32)
        assert torch.equal(Y, y)
        got, Y2, db = F.fc_bwd_data_glu(among_nans(dY, offset), w, among_nans(Z, offset), F.ACT_RELU, w_order=wo,
                                        keep_y=True, bias_grad=True)
        assert torch.equal(got, dZ.to(torch.bfloat16)) and bool(torch.isfinite(db).all())
        assert torch.equal(Y2, (torch.clamp(G, min=0) * Up).to(torch.bfloat16))
        x, w = among_nans(X * small, offset), among_nans(stored(W * small, wo), offset)
        k = min(2 * N, 4)
        zs = (X.double() @ W.double()) * small * small
        logp, entropy, lse, top, tids = F.fc_logprob(x, w, t, w_order=wo, top_k=k)
        want = torch.logsumexp(zs, 1)
        within(lse, want, 2.0 ** -20 + (2 * N + 16) * U + 4 * U * want.abs(), f"{shape} lse")
        assert torch.equal(tids, torch.sort(zs, dim=1, descending=True, stable=True).indices[:, :k])
        loss, lse2, sl = F.fc_distill_fwd(x, w, ids, tl, w_order=wo)
        within(lse2, want, 2.0 ** -20 + (2 * N + 16) * U + 4 * U * want.abs(), f"{shape} lse of the distillation")
        assert bool(torch.isfinite(loss).all())
        dX1, dW1 = F.fc_distill_bwd(x, w, ids, tl, sl, lse, torch.ones(M, device="cuda"), w_order=wo)
        assert bool(torch.isfinite(dX1).all()) and bool(torch.isfinite(dW1).all())


def guarded(shape, dtype):
    """An output between bytes that must not change, and a check of them."""
    n = 1
    for s in shape:
        n *= s
    buf = torch.full((n + 64,), 7, dtype=dtype, device="cuda")
    return buf[32:32 + n].view(shape), lambda: bool((buf[:32] == 7).all()) and bool((buf[32 + n:] == 7).all())


@pytest.mark.parametrize("shape", [(3, 40, 5), (33, 129, 130), (257, 520, 300), (4001, 600, 2051), (4096, 512, 2048)])
def test_nothing_past_the_outputs_is_written(shape):
    M, K, N = shape
    g = gen(1)
    X, W, dY, Z = normal(g, M, K), normal(g, K, 2 * N, scale=0.1), normal(g, M, K), normal(g, M, 4 * N)
    for wo in (ROW, COL):
        y, ok1 = guarded((M, N), torch.bfloat16)
        z, ok2 = guarded((M, 2 * N), torch.bfloat16)
        F.fc_fwd_glu(X, stored(W, wo), w_order=wo, out=y, z=z)
        dz, ok3 = guarded((M, 4 * N), torch.bfloat16)
        h, ok4 = guarded((M, 2 * N), torch.bfloat16)
        db, ok5 = guarded((4 * N,), torch.float32)
        V = W.t().contiguous()  # 2N x K
        F.fc_bwd_data_glu(dY, stored(V, wo), Z, w_order=wo, out=dz, y=h, db=db)
        assert ok1() and ok2() and ok3() and ok4() and ok5()


def _all_calls(seed, M=96, K=200, N=328):
    g = gen(seed)
    X, W, b = normal(g, M, K), normal(g, K, 2 * N, scale=0.1), normal(g, 2 * N)
    dY, Z, d2 = normal(g, M, 2 * N), normal(g, M, 2 * K), normal(g, M, N)
    t = torch.randint(0, 2 * N, (M,), device="cuda", generator=g)
    ids, tl = teacher(g, M, 21, 0, 2 * N)
    _, lse, sl = F.fc_distill_fwd(X, W, ids, tl)
    w = torch.rand(M, device="cuda", generator=g)
    return {
        "fwd_glu": lambda **k: F.fc_fwd_glu(X, W, bias=b, keep_z=True, **k),
        "bwd_data_glu": lambda **k: F.fc_bwd_data_glu(dY, W, Z, keep_y=True, bias_grad=True, **k),
        "bwd_glu": lambda **k: F.fc_bwd_glu(d2, dY, keep_y=True, bias_grad=True, **k),
        "logprob": lambda **k: F.fc_logprob(X, W, t, top_k=70, **k),
        "distill_fwd": lambda **k: F.fc_distill_fwd(X, W, ids, tl, **k),
        "distill_bwd": lambda **k: F.fc_distill_bwd(X, W, ids, tl, sl, lse, w, **k),
    }


SIZES = [(96, 200, 328), (33, 1001, 131), (3, 2048, 264), (1, 512, 600), (520, 264, 520), (2304, 512, 1400)]


@pytest.mark.parametrize("size", SIZES)
def test_calls_are_deterministic_on_other_streams_and_at_once(size):
    calls, others = _all_calls(1, *size), _all_calls(2, *size)
    want = {n: c() for n, c in calls.items()}
    want2 = {n: c() for n, c in others.items()}
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for n in calls:
        got = [calls[n](stream=a) if r % 2 == 0 else others[n](stream=b) for r in range(6)]
        torch.cuda.synchronize()
        for r, o in enumerate(got):
            assert same(o, (want, want2)[r % 2][n]), f"{n} round {r}"


@pytest.mark.parametrize("size", SIZES)
def test_graph_replays_match_eager(size):
    """All operators captured into two graphs whose workspaces live on at once,
    replayed in turn with eager calls between."""
    sets = [_all_calls(1, *size), _all_calls(2, *size)]
    want = [{n: c() for n, c in s.items()} for s in sets]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in sets:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append({n: c() for n, c in s.items()})
        graphs.append(gr)
    for r in range(3):
        for i in (0, 1):
            for o in outs[i].values():
                for t in o:
                    t.zero_()
            graphs[i].replay()
            eager = {n: c() for n, c in sets[1 - i].items()}
            torch.cuda.synchronize()
            for n in sets[i]:
                assert same(outs[i][n], want[i][n]), f"replay {r} of graph {i}: {n}"
                assert same(eager[n], want[1 - i][n]), f"eager {n}"


def test_binding_refusals():
    g = gen(1)
    X, W = normal(g, 8, 16), normal(g, 16, 24)
    t = torch.zeros(8, dtype=torch.int64, device="cuda")
    ids, tl = torch.zeros((8, 3), dtype=torch.int64, device="cuda"), torch.zeros((8, 3), device="cuda")
    v = torch.zeros(8, device="cuda")
    with pytest.raises(ValueError, match="inner"):
        F.fc_fwd_glu(X, W.t().contiguous())
    with pytest.raises(ValueError, match="up projection"):
        F.fc_fwd_glu(X, W[:, :23].contiguous())
    with pytest.raises(TypeError, match="bias"):
        F.fc_fwd_glu(X, W, bias=normal(g, 12))
    with pytest.raises(ValueError, match="OUT_BF16"):
        F.fc_fwd_glu(X, W, out_dtype=F.OUT_F32_ACC)
    with pytest.raises(F.FcError):
        F.fc_fwd_glu(X, W, act=9)
    with pytest.raises(F.FcError):
        F.fc_fwd_glu(X, W, z=(z := normal(g, 8, 24)), out=z.view(-1)[:96].view(8, 12))  # one output on the other
    with pytest.raises(TypeError, match="Z"):
        F.fc_bwd_data_glu(normal(g, 8, 24), W, normal(g, 8, 16))
    with pytest.raises(ValueError, match="dY"):
        F.fc_bwd_data_glu(normal(g, 8, 16), W, normal(g, 8, 32))
    with pytest.raises(F.FcError):
        F.fc_bwd_glu(X, normal(g, 8, 32), keep_dz=False)
    for k in (-1, 25, 129):
        with pytest.raises(ValueError, match="top_k"):
            F.fc_logprob(X, W, t, top_k=k)
    for T in (0.0, -1.0, float("nan"), INF, 2.0 ** -11, 2.0 ** 11):
        with pytest.raises(F.FcError):
            F.fc_logprob(X, W, t, temperature=T)
        with pytest.raises(F.FcError):
            F.fc_distill_fwd(X, W, ids, tl, temperature=T)
        with pytest.raises(F.FcError):
            F.fc_distill_bwd(X, W, ids, tl, tl, v, v, temperature=T)
    with pytest.raises(TypeError, match="targets"):
        F.fc_logprob(X, W, t.int())
    with pytest.raises(F.FcError):
        F.fc_logprob(X, W, t, vocab_start=-1)
    with pytest.raises(TypeError, match="ids"):
        F.fc_distill_fwd(X, W, ids.int(), tl)
    with pytest.raises(TypeError, match="tlogits"):
        F.fc_distill_fwd(X, W, ids, tl.double())
    with pytest.raises(ValueError, match="1 .. 128"):
        F.fc_distill_fwd(X, W, ids.repeat(1, 43), tl.repeat(1, 43))
    with pytest.raises(TypeError, match="slogits"):
        F.fc_distill_bwd(X, W, ids, tl, tl[:, :2].contiguous(), v, v)
    with pytest.raises(ValueError, match="accumulating"):
        F.fc_distill_bwd(X, W, ids, tl, tl, v, v, dw_dtype=F.OUT_F32_ACC)
    far = torch.cuda.Stream(stream_id=0, device_index=X.get_device() + 1, device_type=torch.cuda.current_stream().device_type)
    for call in (lambda: F.fc_fwd_glu(X, W, stream=far), lambda: F.fc_logprob(X, W, t, stream=far),
                 lambda: F.fc_distill_fwd(X, W, ids, tl, stream=far)):
        with pytest.raises(ValueError, match="stream"):
            call()


# ---- together

def test_a_distillation_step_of_all_of_them():
    """One training step of a student with a gated layer against a teacher's top
    tokens, forward and backward with these calls, against the same model in 64
    bits.

    The step rounds to bf16 after each operator: 6 roundings lie between the
    inputs and any of its outputs. In the Frobenius norm a rounding changes a
    tensor by at most h = 2^-8 relative, and every map in between passes a
    relative change on by at most the bound below: 16 h."""
    M, K, N, V, n, T = 192, 128, 320, 1000, 20, 2.0
    g = gen(55)
    X = normal(g, M, K)
    W1, b1 = normal(g, K, 2 * N, scale=K ** -0.5), normal(g, 2 * N, scale=0.1)
    W2, E = normal(g, N, K, scale=N ** -0.5), normal(g, K, V, scale=K ** -0.5)
    teacher_X, teacher_E = normal(g, M, K), normal(g, K, V, scale=2 * K ** -0.5)

    _, _, _, tl, ids = F.fc_logprob(teacher_X, teacher_E, temperature=1.0, top_k=n)
    ids[::6] = -1  # padding
    w = torch.where(ids[:, 0] >= 0, T * T / (ids[:, 0] >= 0).sum(), 0.0).float()
    Y, Z = F.fc_fwd_glu(X, W1, bias=b1, act=F.ACT_SILU, keep_z=True)
    C = F.fc_fwd_act(Y, W2, residual=X)
    loss, lse, sl = F.fc_distill_fwd(C, E, ids, tl, temperature=T)
    dC, dE = F.fc_distill_bwd(C, E, ids, tl, sl, lse, w, temperature=T)
    dZ, again, db1 = F.fc_bwd_data_glu(dC, W2, Z, F.ACT_SILU, keep_y=True, bias_grad=True)
    dW2, dW1 = F.fc_bwd_weight(again, dC), F.fc_bwd_weight(X, dZ)
    dX = F.fc_bwd_data(dZ, W1)

    x, w1, bb, w2, e = (q.double().requires_grad_() for q in (X, W1, b1, W2, E))
    G, Up = (x @ w1 + bb).split(N, 1)
    c = (torch.nn.functional.silu(G) * Up) @ w2 + x
    logq = torch.log_softmax((c @ e) / T, 1)
    there = ids >= 0
    at = torch.where(there, ids, 0)
    p = torch.softmax(tl.double() / T, 1)
    each = torch.where(there[:, 0], (p * (p.log() - logq.gather(1, at))).sum(1), 0.0)
    (each * w.double()).sum().backward()
    for name, got, want in (("loss", loss, each.detach()), ("dE", dE, e.grad), ("dW2", dW2, w2.grad),
                            ("dW1", dW1, w1.grad), ("db1", db1, bb.grad),
                            ("dX", dX.double() + dC.double(), x.grad)):
        rel = ((got.double() - want).norm() / want.norm()).item()
        log(f"  {name}: {rel:.3g}")
        assert rel <= 16 * H, name


def test_a_decoding_step():
    """One token through a gated layer and the vocabulary, weights as nn.Linear keeps them, captured and replayed."""
    K, N, V = 512, 1024, 4000
    g = gen(6)
    W1, W2, E = normal(g, 2 * N, K, scale=K ** -0.5), normal(g, K, N, scale=N ** -0.5), normal(g, V, K, scale=0.1)
    x, t = normal(g, 1, K), torch.tensor([17], device="cuda")

    def step():
        y = F.fc_fwd_act(F.fc_fwd_glu(x, W1, w_order=COL), W2, w_order=COL, residual=x)
        return F.fc_logprob(y, E, t, w_order=COL, top_k=20)

    step()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = step()
    for r in range(3):
        x.copy_(normal(g, 1, K))
        t.fill_(r)
        gr.replay()
        torch.cuda.synchronize()
        assert same(out, step())
        G, Up = (x.double() @ W1.double().t()).split(N, 1)
        y = (torch.nn.functional.silu(G) * Up).to(torch.bfloat16).double() @ W2.double().t() + x.double()
        want = torch.log_softmax(y.to(torch.bfloat16).double() @ E.double().t(), 1)
        # two roundings to bf16 on the way, of values that reach each logit through |W2| and |E|
        off = H * 2 * ((torch.nn.functional.silu(G) * Up).abs() @ W2.double().abs().t() + y.abs()) @ E.double().abs().t()
        assert abs(out[0].item() - want[0, r].item()) <= 2 * off.max().item()
        assert bool((want[0, out[4][0]] >= want.max() - 4 * off.max() - (out[3].max() - out[3].min()).double()).all())


# ---- a teacher's logits and temperatures at their ends

@pytest.mark.parametrize("T", [0.7, 2.0 ** -10, 0.5, 1.0, 2.0 ** 10])
@pytest.mark.parametrize("n", [5, 64, 100])
@pytest.mark.parametrize("wo", [ROW, COL])
def test_distill_of_teacher_logits_at_the_ends(n, T, wo):
    """A finite teacher's logit is there, however it scales: the type's lowest value as a mask, and large ones whose
    quotient by T leaves the type. All differences are zero or more than T x 10^30, so the largest ones of a row share
    its probability. Only -inf and negative ids are absent."""
    M, K, N = 70, 24, 1000
    low, high = torch.finfo(torch.float32).min, torch.finfo(torch.float32).max
    g = gen(n)
    X, W = grid(g, M, K), grid(g, K, N)  # exact logits
    ids = torch.rand((M, N), device="cuda", generator=g).argsort(1)[:, :n].contiguous()
    tl = torch.full((M, n), low, device="cuda")  # rows 0, 6, ..: masked tokens alone
    tl[1::6, 0] = 0.0                            # one token that is not masked
    tl[2::6, 1:3] = high
    tl[3::6] = torch.where(torch.arange(n, device="cuda") % 3 == 0, 1e38, 5e37)
    tl[4::6] = torch.where(torch.arange(n, device="cuda") % 2 == 0, -1e36, -2e36)
    tl[::2, n - 1] = -INF
    ids[1::5, n - 2] = -1
    there = (ids >= 0) & (tl != -INF)
    best = there & (tl == torch.where(there, tl, -INF).max(1, keepdim=True).values)
    p = best.double() / best.sum(1, keepdim=True)
    z = X.double() @ W.double()
    sl = torch.where(there, z.gather(1, torch.where(there, ids, 0)), 0.0)
    lse = torch.logsumexp(z / T, 1)
    loss, got_lse, slogits = F.fc_distill_fwd(X, stored(W, wo), ids, tl, w_order=wo, temperature=T)
    e_lse = 3 * U * z.abs().max(1).values / T + 2.0 ** -20 + (N + 16) * U + 4 * U * lse.abs()
    within(got_lse, lse, e_lse, f"{T} lse")
    assert torch.equal(slogits.double(), sl), f"{T} slogits"
    logp = torch.where(best, torch.log(p), 0.0)
    term, size = logp - sl / T + lse[:, None], logp.abs() + sl.abs() / T + lse.abs()[:, None]
    ep = 2.0 ** -20 * (1 + logp.abs())
    tol = (p * (ep * term.abs() + e_lse[:, None] + 4 * U * size + ep)).sum(1) + (n + 16) * U * (p * term.abs()).sum(1)
    within(loss, (p * term).sum(1), tol, f"{T} loss")

    w = torch.rand(M, device="cuda", generator=g) - 0.3
    lse32 = lse.float()
    dX, _ = F.fc_distill_bwd(X, stored(W, wo), ids, tl, sl.float(), lse32, w, w_order=wo, temperature=T,
                             dx_dtype=F.OUT_F32)
    s = z / T
    q = torch.exp(s - lse32.double()[:, None])
    hot = torch.zeros_like(q).scatter_add_(1, torch.where(there, ids, 0), p)
    wc = (w.double() / T)[:, None]
    D = wc * (q - hot)
    eq = q * torch.expm1(2.0 ** -22 * (1 + s.abs() + lse.abs()[:, None]))
    eD = wc.abs() * (eq + hot * (ep.amax(1, keepdim=True) + n * U) + 4 * U * (q + hot))
    eD = eD + H * (D.abs() + eD) + (wc.abs() + 2) * 2.0 ** -126  # numbers under 2^-126 may be flushed to zero
    aW = W.double().abs().t()
    within(dX, D @ W.double().t(), eD @ aW + (N + 16) * U * ((D.abs() + eD) @ aW) + (N + 16) * 2.0 ** -126, f"{T} dX")


@pytest.mark.parametrize("T", [2.0 ** -10, 2.0 ** -9, 0.0013])
@pytest.mark.parametrize("shape", [(40, 500), (3, 900), (2304, 1400)])
@pytest.mark.parametrize("wo", [ROW, COL])
def test_distill_loss_at_low_temperatures(shape, T, wo):
    """z / T is of the order of 1e4 here and the loss of tokens near the maximum of the order of one: its error goes by
    the distances from the maximum, not by z / T and the logarithm of the normaliser, which differ by as little."""
    (M, N), K, n = shape, 256, 8
    g = gen(N)
    X = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    W = torch.zeros((K, N), dtype=torch.bfloat16, device="cuda")
    X[:, 0] = (1 + (torch.arange(M, device="cuda") % 100) / 128).to(torch.bfloat16)  # logits 16 .. 29, and up to
    X[:, 1] = 1.0                                                                   # 255 / 1024 more: exact
    W[0] = 16.0
    W[1] = (torch.randint(0, 256, (N,), device="cuda", generator=g) / 1024).to(torch.bfloat16)
    z = X.double() @ W.double()
    assert torch.equal(z, (X.float() @ W.float()).double()) and z.min() >= 16
    ids = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :n].contiguous()
    tl = torch.randn((M, n), device="cuda", generator=g) * T
    loss, lse, slogits = F.fc_distill_fwd(X, stored(W, wo), ids, tl, w_order=wo, temperature=T)
    sl, top = z.gather(1, ids), z.max(1).values[:, None]
    assert torch.equal(slogits.double(), sl)
    want = torch.logsumexp(z / T, 1)
    e_log = 2.0 ** -20 + (N + 16) * U  # of the logarithm of the sum, relative to the maximum
    within(lse, want, 3 * U * z.max(1).values / T + e_log + 4 * U * want.abs(), "lse")
    logp = torch.log_softmax(tl.double() / T, 1)
    p, far, ls = logp.exp(), (top - sl) / T, torch.log(torch.exp((z - top) / T).sum(1))[:, None]
    term, size = logp + far + ls, logp.abs() + far + ls.abs()
    ep = 2.0 ** -20 * (1 + logp.abs()) + 4 * U * (tl.double() / T).abs().amax(1, keepdim=True)
    tol = (p * (ep * term.abs() + ep + e_log + 7 * U * size)).sum(1) + (n + 16) * U * (p * term.abs()).sum(1)
    within(loss, (p * term).sum(1), tol, f"{shape} {T} loss")


@pytest.mark.parametrize("wo", [ROW, COL])
def test_distill_loss_of_logits_at_the_ends(wo):
    """Logits whose distance is more than fp32 holds, its quotient by T not."""
    N, T = 400, 2.0 ** 10
    W = torch.full((1, N), 1.0, device="cuda").to(torch.bfloat16)
    W[0, 7], W[0, 50] = 3e38, -3e38
    ids, tl = torch.tensor([[50, 7]], device="cuda"), torch.zeros((1, 2), device="cuda")
    loss, lse, slogits = F.fc_distill_fwd(torch.ones((1, 1), dtype=torch.bfloat16, device="cuda"), stored(W, wo), ids, tl,
                                          w_order=wo, temperature=T)
    z = W.double()[0]
    assert torch.equal(slogits.double(), z[ids])
    within(lse, z[7:8] / T, 4 * U * z[7:8] / T, "lse")
    want = (z[7:8] - z[50:51]) / T / 2
    within(loss, want, 2.0 ** -20 * want, "loss")


# ---- gradients against differences, row by row

def glu_line(act):
    """Rows of the gated layer with their gradients in 64 bits, and steps of 2^-7 along the signs of these gradients:
    (X, W, R, step, differences of sum_j R_ij Y_ij over the step, gradient of Z, change of Z). X, X + step and X - step
    are bf16 numbers and their products with W are exact in fp32. No gate lies near relu's kink where R is not zero."""
    M, K, N = 24, 256, 40
    g = torch.Generator().manual_seed(3)
    X = torch.clamp(torch.round(torch.randn((M, K), generator=g) * 8), -28, 28).double() / 16  # within 1.75
    W = torch.clamp(torch.round(torch.randn((K, 2 * N), generator=g) * 4), -16, 16).double() / 32
    R = torch.randint(0, 2, (M, N), generator=g).double() * 2 - 1
    z = X @ W
    R = torch.where(z[:, :N].abs() > 0.5, R, 0.0)

    def loss(x):
        q = x @ W
        return (R * act64(q[:, :N], act) * q[:, N:]).sum(1)

    G, Up = z[:, :N], z[:, N:]
    dZ = torch.cat([R * Up * slope64(G, act), R * act64(G, act)], 1)
    step = torch.where(dZ @ W.t() >= 0, 1.0, -1.0).double() * 2.0 ** -7
    return X, W, R, step, loss(X + step) - loss(X - step), dZ, step @ W


def glu_line_bound(X, W, R, act, dZ, d):
    """How far the difference of the library's losses and its gradient's product with twice the step may lie apart, for
    each row."""
    N = R.shape[1]
    G, Up = (X @ W).split(N, 1)
    dg, du = d.abs().split(N, 1)
    a = act64(G, act)
    # the differences: third derivatives (|act''| <= 2, |act'''| <= 2), and two fp32 outputs of exact Z
    third = (2 * dg ** 3 * (Up.abs() + du) + 6 * dg ** 2 * du) / 3
    big = (G.abs() + dg, Up.abs() + du)
    e_y = 2 * (2.0 ** -20 * (1 + big[0] ** 2) * big[1] + U * (a.abs() + 1.13 * dg) * big[1])
    # the gradient: Z rounded to bf16 (the slope of a slope is 2 at most), the functions' own errors, dZ rounded
    e_dg = R.abs() * Up.abs() * (1.13 * H + 2 * H * G.abs()) * (1 + H) + R.abs() * Up.abs() * 2.0 ** -20 * (1 + G * G)
    e_du = R.abs() * (1.13 * H * G.abs() + 2.0 ** -20 * (1 + G * G))
    e = torch.cat([e_dg, e_du], 1)
    e = e + H * (dZ.abs() + e)
    # ... and the fp32 product over 2 N columns
    e = e + (2 * N + 16) * U * (dZ.abs() + e)
    return (R.abs() * (third + e_y)).sum(1) + 2 * (d.abs() * e).sum(1)


@pytest.mark.parametrize("act", ACTS)
def test_glu_gradient_against_differences_of_each_row(act):
    """The difference of each row's loss along its gradient is the gradient's size, which the errors are a small part
    of: a gradient without one of its halves, or with another sign, is told from the right one in every row."""
    X, W, R, step, want, dZ64, d = glu_line(act)
    N = R.shape[1]
    bound = glu_line_bound(X, W, R, act, dZ64, d)
    cut = bound / want.abs()
    assert bool((cut < 0.05).all())
    halves = [torch.cat([dZ64[:, :N] * i, dZ64[:, N:] * j], 1) for i, j in ((0, 1), (1, 0), (0, 0), (-1, 1), (1, -1), (-1, -1))]
    for wrong in halves:
        assert bool((((2 * d * wrong).sum(1) - want).abs() > 2 * bound).all())

    dev = [t.cuda() for t in (X, X + step, X - step, W, R)]
    x, xa, xb, w, r = (t.to(torch.bfloat16) for t in dev)
    assert all(torch.equal(t.double(), s) for t, s in zip((x, xa, xb, w, r), dev))  # all are bf16 numbers
    for wo in (ROW, COL):
        ws = stored(w, wo)
        ya, yb = (F.fc_fwd_glu(t, ws, act=act, w_order=wo, out_dtype=F.OUT_F32).double() for t in (xa, xb))
        diff = (dev[4] * (ya - yb)).sum(1).cpu()
        _, Z = F.fc_fwd_glu(x, ws, act=act, w_order=wo, keep_z=True)
        dZ, _, _ = F.fc_bwd_glu(r, Z, act)
        dX = F.fc_bwd_data(dZ, ws, w_order=wo, out_dtype=F.OUT_F32)
        ours = (2 * step * dX.double().cpu()).sum(1)
        log(f"  {ACT_NAMES[act]}: bound / difference up to {cut.max().item():.3g}, "
            f"error / bound {((diff - ours).abs() / bound).max().item():.3g}")
        assert bool(((diff - ours).abs() <= bound).all()), ACT_NAMES[act]


def distill_line(T):
    """Rows with a teacher's tokens, their losses' gradients in 64 bits, and steps of 2^-7 along the signs of these
    gradients: X, X + step and X - step are bf16 numbers and their products with W are exact in fp32."""
    M, K, N, n = 40, 256, 500, 9
    g = torch.Generator().manual_seed(31)
    X = torch.clamp(torch.round(torch.randn((M, K), generator=g) * 8), -28, 28).double() / 16  # within 1.75
    W = torch.clamp(torch.round(torch.randn((K, N), generator=g) * 4), -16, 16).double() / 8 * min(T, 1.0)
    ids = torch.rand((M, N), generator=g).argsort(1)[:, :n].contiguous()
    ids[torch.rand((M, n), generator=g) < 0.3] = -1
    ids[:, 0], ids[:, 1] = ids[:, 0].abs(), ids[:, 0].abs()  # the first token twice
    ids[1::7] = -1
    tl = torch.randn((M, n), generator=g)
    there = ids >= 0
    any_ = there.any(1)
    t = torch.where(there, tl.double() / T, -INF)
    p = torch.where(there, torch.softmax(torch.where(any_[:, None], t, 0.0), 1), 0.0)
    hot = torch.zeros((M, N), dtype=torch.float64).scatter_add_(1, torch.where(there, ids, 0), p)

    def loss(x):
        logq = torch.log_softmax((x @ W) / T, 1)
        return -(hot * logq).sum(1) + torch.special.xlogy(p, p).sum(1)

    q = torch.softmax((X @ W) / T, 1)
    D = torch.where(any_[:, None], (q - hot) / T, 0.0)
    step = torch.where(D @ W.t() >= 0, 1.0, -1.0).double() * 2.0 ** -7
    want = torch.where(any_, loss(X + step) - loss(X - step), 0.0)
    return X, W, ids, tl, any_, p, hot, q, D, step, want


def distill_line_bound(X, W, T, tl, p, hot, q, D, step):
    """As glu_line_bound, of the loss and dX = D . W^T."""
    N, n = W.shape[1], p.shape[1]
    z, d = X @ W, step @ W
    # the third cumulant of a variable within a range r is at most r^3 / (6 sqrt 3)
    third = ((d.max(1).values - d.min(1).values) / T) ** 3 / (18 * 3 ** 0.5)
    # a loss: the normaliser's error and its rounding, each term's, p's relative error (as in test_distill_fwd; the
    # logits are exact)
    lse = torch.logsumexp(z / T, 1).abs() + (d / T).abs().max(1).values
    far = (z.abs() + d.abs()).max(1).values / T
    logp = torch.where(p > 0, torch.log(p), 0.0)
    e_lse = 3 * U * far + 2.0 ** -20 + (N + 16) * U + 4 * U * lse
    size = logp.abs() + (far + lse)[:, None]
    ep = 2.0 ** -20 * (1 + logp.abs()) + 4 * U * (tl.double() / T).abs().amax(1, keepdim=True)
    e_loss = (p * (ep * size + e_lse[:, None] + 4 * U * size + ep)).sum(1) + (n + 16) * U * (p * size).sum(1)
    # the gradient: probabilities on either side, D rounded to bf16, the fp32 product
    eq = q * 2.0 ** -21 * (1 + far + lse)[:, None]
    eh = hot * (ep + n * U).amax(1, keepdim=True)
    e_d = (eq + eh + 4 * U * (q + hot)) / T
    e_d = e_d + H * (D.abs() + e_d)
    e_d = e_d + (N + 16) * U * (D.abs() + e_d)
    return third + 2 * e_loss + 2 * (e_d * (step.abs() @ W.abs())).sum(1)


@pytest.mark.parametrize("T", [1.0, 2.0, 0.5])
def test_distill_gradient_against_differences_of_each_row(T):
    """As for the gated layer: without the teacher's share, without the student's, at another temperature or with the
    other sign the gradient lies outside the bound in every row."""
    X, W, ids, tl, any_, p, hot, q, D, step, want = distill_line(T)
    bound = distill_line_bound(X, W, T, tl, p, hot, q, D, step)
    d = step @ W
    cut = (bound / want.abs())[any_]
    assert bool((cut < 0.05).all())
    for wrong in (q / T, -hot / T, -D, 0 * D, 2 * D, D / 2):
        assert bool((((2 * d * wrong).sum(1) - want).abs() > 2 * bound)[any_].all())

    dev = [t.cuda() for t in (X, X + step, X - step, W)]
    x, xa, xb, w = (t.to(torch.bfloat16) for t in dev)
    assert all(torch.equal(t.double(), s) for t, s in zip((x, xa, xb, w), dev))  # all are bf16 numbers
    ids, tl = ids.cuda(), tl.cuda()
    for wo in (ROW, COL):
        ws = stored(w, wo)
        a, b = (F.fc_distill_fwd(t, ws, ids, tl, w_order=wo, temperature=T)[0].double() for t in (xa, xb))
        diff = (a - b).cpu()
        _, lse, sl = F.fc_distill_fwd(x, ws, ids, tl, w_order=wo, temperature=T)
        dX, _ = F.fc_distill_bwd(x, ws, ids, tl, sl, lse, torch.ones(len(X), device="cuda"), w_order=wo, temperature=T,
                                 dx_dtype=F.OUT_F32)
        ours = (2 * step * dX.double().cpu()).sum(1)
        log(f"  T {T}: bound / difference up to {cut.max().item():.3g}, "
            f"error / bound {((diff - ours).abs() / bound).max().item():.3g}")
        assert bool(((diff - ours).abs() <= bound).all())
        assert bool((diff[~any_] == 0).all()) and bool((ours[~any_] == 0).all())


# ---- the largest sizes: outputs whose columns or rows run into the millions

@pytest.mark.parametrize("shape", [(2, 8, 1 << 22), (3, 256, 1 << 21), (1 << 20, 16, 48)])
@pytest.mark.parametrize("wo", [ROW, COL])
def test_largest_vocabularies_and_rows(shape, wo):
    test_logprob(shape, wo)
    test_distill_fwd(shape, wo)
    check_distill_bwd(shape, wo, 0, shape[2], 1.0, 21, 3)


@pytest.mark.parametrize("shape", [(2, 64, 1 << 21), (2, 260, 1 << 21), (1 << 20, 32, 24)])
@pytest.mark.parametrize("wo", [ROW, COL])
def test_largest_gated_layers(shape, wo):
    M, K, N = shape
    test_fwd_glu_integers_are_exact(shape, wo)
    test_bwd_data_glu((M, K, N), wo)


@pytest.mark.parametrize("shape", [(1 << 20, 40), (1 << 22, 3), (3, 1 << 21), (3, (1 << 21) - 1)])
def test_largest_elementwise_gradients(shape):
    test_bwd_glu(shape)
