"""The fused operators on the GPU against plain implementations in 64 bits.

Tolerances are bounds, derived from the arithmetic: u = 2^-24 is the rounding
of one fp32 operation, h = 2^-8 that of a store to bf16.

* A product of K terms accumulated in fp32: (K + 16) u (|A| |B|)_ij, which
  holds for every order of summation.
* An activation: its slope is at most 1.13 in size, so it passes on 1.13
  times its argument's error, and its own evaluation (an exponential or erf
  of a few u, a division) errs by at most 2^-20 (1 + |z|).
* A softmax probability p = exp(z - lse): relative error e_z + 2^-22 (1 +
  |z - lse|), e_z being the logit's error.
* Sums of n terms in fp32: (n + 16) u times the sum of the terms' sizes.

Integer inputs, whose products and sums fit fp32, are compared bit for bit.
"""
from __future__ import annotations

import math
import sys

import pytest

from sharded_fc_layer_amd import fcshard as F

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

U, H = 2.0 ** -24, 2.0 ** -8
ROW, COL = F.ROW, F.COL
ACT_NAMES = {F.ACT_NONE: "none", F.ACT_RELU: "relu", F.ACT_GELU: "gelu", F.ACT_GELU_TANH: "gelu_tanh",
             F.ACT_SILU: "silu"}
ACTS = list(ACT_NAMES)


def log(msg):
    print(msg, file=sys.stderr, flush=True)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, scale=1.0):
    return (torch.randn(shape, device="cuda", generator=g) * scale).to(torch.bfloat16)


def integers(g, *shape, top=3):
    return torch.randint(-top, top + 1, shape, device="cuda", generator=g).to(torch.bfloat16)


def stored(w, order):
    """The storage of matrix w (or of each matrix of a stack) in an order."""
    return w if order == ROW else w.transpose(-1, -2).contiguous()


def shifted(t):
    """The same values at an address that is 2 bytes past a 16-byte boundary."""
    buf = torch.empty(t.numel() + 8, dtype=t.dtype, device=t.device)
    out = buf[1:1 + t.numel()].view(t.shape)
    out.copy_(t)
    assert out.data_ptr() % 16 == 2
    return out


def within(got, want, tol, what):
    err = (got.double() - want).abs()
    ok = err <= tol
    same = torch.isnan(got) & torch.isnan(want) | (got.double() == want)
    ratio = torch.where(same, 0.0, err / tol).max().item() if got.numel() else 0.0
    log(f"  {what}: largest error / bound = {ratio:.3g}")
    assert bool((ok | same).all()), f"{what}: {int((~(ok | same)).sum())} of {got.numel()} outside the bound"


def act64(z, act):
    f = torch.nn.functional
    return {F.ACT_NONE: lambda: z, F.ACT_RELU: lambda: f.relu(z), F.ACT_GELU: lambda: f.gelu(z),
            F.ACT_GELU_TANH: lambda: f.gelu(z, approximate="tanh"), F.ACT_SILU: lambda: f.silu(z)}[act]()


def slope64(z, act):
    z = z.clone().requires_grad_()
    (s,) = torch.autograd.grad(act64(z, act).sum(), z)
    return s


# from one row to several tiles, odd and aligned, reductions from one value to
# several slices of a split one
# ... and enough tiles for the 256 x 256 ones, with reductions of a partial
# stage after a whole one, 2 and 4 stages past a period of 6, and whole periods
WIDE = [(2600, 100, 2600), (2570, 512, 2700), (4100, 640, 1500), (2600, 384, 2560), (2309, 1001, 3001)]
SHAPES = [(1, 1, 1), (1, 2048, 520), (3, 31, 7), (16, 512, 384), (32, 264, 136), (33, 129, 130), (100, 1001, 77),
          (128, 64, 128), (130, 72, 259), (257, 520, 300), (300, 40, 1032), (520, 776, 264)]


@pytest.mark.parametrize("shape", SHAPES + WIDE)
@pytest.mark.parametrize("xo, wo", [(ROW, ROW), (ROW, COL), (COL, ROW), (COL, COL)])
def test_fwd_act(shape, xo, wo):
    M, K, N = shape
    g = gen(M * 7 + K * 3 + N)
    X, W = normal(g, M, K), normal(g, K, N, scale=K ** -0.5)
    b, R = normal(g, N), normal(g, M, N)
    z = X.double() @ W.double() + b.double()
    ez = (K + 16) * U * (X.double().abs() @ W.double().abs() + b.double().abs())
    xs, ws = stored(X, xo), stored(W, wo)
    for act in ACTS:
        for res, keep, f32 in ((None, False, False), (R, True, True), (R, False, False)):
            out = F.fc_fwd_act(xs, ws, bias=b, act=act, residual=res, x_order=xo, w_order=wo, keep_z=keep,
                               out_dtype=F.OUT_F32 if f32 else F.OUT_BF16)
            Y, Z = out if keep else (out, None)
            a = act64(z, act)
            y = a if res is None else a + res.double()
            tol = 1.13 * ez + 2.0 ** -20 * (1 + z.abs()) + U * y.abs()
            what = f"{shape} {xo}{wo} {ACT_NAMES[act]}"
            within(Y, y, tol if f32 else tol + H * (y.abs() + tol), what)
            if keep:
                within(Z, z, ez + H * (z.abs() + ez), what + " Z")


@pytest.mark.parametrize("shape", SHAPES + WIDE + [(700, 2050, 513)])
@pytest.mark.parametrize("wo", [ROW, COL])
def test_fwd_act_integers_are_exact(shape, wo):
    M, K, N = shape
    g = gen(5)
    X, W, b, R = integers(g, M, K), integers(g, K, N), integers(g, N), integers(g, M, N)
    want = X.double() @ W.double() + b.double()
    for act in (F.ACT_NONE, F.ACT_RELU):
        y = act64(want, act) + R.double()
        for align in (lambda t: t, shifted):
            Y, Z = F.fc_fwd_act(align(X), align(stored(W, wo)), bias=align(b), act=act, residual=align(R), w_order=wo,
                                out_dtype=F.OUT_F32, keep_z=True)
            assert torch.equal(Y.double(), y), f"{shape} {wo}"
            assert torch.equal(Z, want.float().to(torch.bfloat16))
    # neither bias nor residual: the plain product's bits
    assert torch.equal(F.fc_fwd_act(X, stored(W, wo), w_order=wo), (X.double() @ W.double()).float().to(torch.bfloat16))


@pytest.mark.parametrize("shape", SHAPES + [(m, n, k) for m, k, n in WIDE])
@pytest.mark.parametrize("wo", [ROW, COL])
def test_bwd_data_act(shape, wo):
    M, N, K = shape  # the reduction runs over the layer's outputs N
    g = gen(M + K * 5 + N * 11)
    dY, W, Z = normal(g, M, N, scale=1e-3), normal(g, K, N, scale=0.02), normal(g, M, K)
    up = dY.double() @ W.double().t()
    e_up = (N + 16) * U * (dY.double().abs() @ W.double().abs().t())
    for act in ACTS:
        s = slope64(Z.double(), act)
        want = up * s
        tol = 1.13 * e_up + 2.0 ** -20 * up.abs()
        what = f"{shape} {wo} {ACT_NAMES[act]}"
        for f32 in (False, True):
            dX, db = F.fc_bwd_data_act(dY, stored(W, wo), Z, act, w_order=wo, bias_grad=True,
                                       out_dtype=F.OUT_F32 if f32 else F.OUT_BF16)
            within(dX, want, tol if f32 else tol + H * (want.abs() + tol), what)
            within(db, want.sum(0), tol.sum(0) + (M + 16) * U * (want.abs() + tol).sum(0), what + " db")
        only = F.fc_bwd_data_act(dY, stored(W, wo), Z, act, w_order=wo, out_dtype=F.OUT_F32)
        assert torch.equal(only, dX)


@pytest.mark.parametrize("shape", [(1, 1), (1, 300), (5, 7), (33, 256), (700, 130), (4100, 264), (64, 5000)])
def test_bwd_act(shape):
    M, N = shape
    g = gen(M + N)
    dY, Z = normal(g, M, N), normal(g, M, N, scale=2.0)
    for act in ACTS:
        want = dY.double() * slope64(Z.double(), act)
        tol = 2.0 ** -20 * dY.double().abs()
        for align in (lambda t: t, shifted):
            dZ, db = F.fc_bwd_act(align(dY), align(Z), act)
            within(dZ, want, tol + H * (want.abs() + tol), f"{shape} {ACT_NAMES[act]}")
            within(db, want.sum(0), tol.sum(0) + (M + 16) * U * (want.abs() + tol).sum(0), "db")
    dZ, db = F.fc_bwd_act(dY, keep_dz=False)  # no activation: the bias gradient alone
    assert dZ is None
    within(db, dY.double().sum(0), (M + 16) * U * dY.double().abs().sum(0), "db alone")
    dZ, db = F.fc_bwd_act(dY, Z, F.ACT_SILU, bias_grad=False)
    assert db is None and dZ.shape == dY.shape


def test_slopes_by_differences_and_at_the_ends():
    """The slopes against central differences of the library's own forward
    activation, and at values where a formula could overflow or lose itself."""
    z = torch.linspace(-8, 8, 4097, device="cuda").to(torch.bfloat16)
    one = torch.ones((1, 1), dtype=torch.bfloat16, device="cuda")
    h = 2.0 ** -7  # z +- h is exact in the fp32 sum z + bias
    for act in (F.ACT_GELU, F.ACT_GELU_TANH, F.ACT_SILU):
        up, down = (F.fc_fwd_act(z[:, None].contiguous(), one, act=act, out_dtype=F.OUT_F32,
                                 bias=torch.full((1,), d, dtype=torch.bfloat16, device="cuda"))[:, 0].double()
                    for d in (h, -h))
        diff = (up - down) / (2 * h)
        s = F.fc_bwd_data_act(torch.ones((z.numel(), 1), dtype=torch.bfloat16, device="cuda"), one, z[:, None], act,
                              out_dtype=F.OUT_F32)[:, 0].double()
        # third derivatives are at most 3: h^2 / 6 of them; the values' errors over 2 h
        tol = h * h / 2 + 2 * 2.0 ** -20 * (1 + z.double().abs()) / (2 * h) + 2.0 ** -20
        within(s.float(), diff, tol, f"slope of {ACT_NAMES[act]}")
    ends = torch.tensor([-float("inf"), -3e38, -1e20, -300.0, -50.0, 50.0, 300.0, 1e20, 3e38, float("inf")],
                        device="cuda").to(torch.bfloat16)
    g1 = torch.ones((1, ends.numel()), dtype=torch.bfloat16, device="cuda")
    for act in (F.ACT_RELU, F.ACT_GELU, F.ACT_GELU_TANH, F.ACT_SILU):
        dZ, _ = F.fc_bwd_act(g1, ends[None], act)
        # 0 or 1 but for tails of (1 + |z|) e^-|z| at most, largest at |z| = 50: 51 e^-50 < 1e-20
        assert bool(((dZ[0].float() - (ends.float() > 0).float()).abs() <= 1e-20).all()), (ACT_NAMES[act], dZ)
    nan = torch.full((1, 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    for act in (F.ACT_GELU, F.ACT_GELU_TANH, F.ACT_SILU):
        assert bool(torch.isnan(F.fc_bwd_act(g1[:, :8].contiguous(), nan, act)[0]).all())


# ---- cross entropy

XENT = [(1, 8, 1), (1, 64, 1000), (5, 33, 130), (32, 128, 129), (33, 100, 999), (64, 264, 4001), (130, 72, 520),
        (257, 520, 1032), (300, 65, 2050),
        (2600, 100, 2600), (2570, 512, 2700), (4100, 640, 1500), (2309, 131, 3001),
        (96, 2001, 300), (40, 4104, 700)]  # (split reductions)


def xent64(X, W, t, v0, ignore, lse=None):
    """(z, its error bound, hits, counted rows) of the definition."""
    z = X.double() @ W.double()
    ez = (X.shape[1] + 16) * U * (X.double().abs() @ W.double().abs())
    counts = t != ignore
    at = t - v0
    here = counts & (at >= 0) & (at < W.shape[1])
    return z, ez, counts, here, torch.where(here, at, 0)


@pytest.mark.parametrize("shape", XENT)
@pytest.mark.parametrize("wo", [ROW, COL])
def test_xent_fwd(shape, wo):
    M, K, N = shape
    g = gen(M + 3 * K + N)
    X, W = normal(g, M, K), normal(g, K, N, scale=0.3)
    for v0, whole in ((0, N), (N, 3 * N), (5, N + 5)):
        t = torch.randint(0, whole, (M,), device="cuda", generator=g)
        t[::4] = -100
        if M > 2:
            t[1] = t[2]  # the same index twice
        z, ez, counts, here, at = xent64(X, W, t, v0, -100)
        loss, lse, tl = F.fc_xent_fwd(X, stored(W, wo), t, w_order=wo, vocab_start=v0)
        want = torch.logsumexp(z, 1)
        hit = torch.where(here, z.gather(1, at[:, None])[:, 0], 0.0)
        e_hit = torch.where(here, ez.gather(1, at[:, None])[:, 0], 0.0)
        # the sum's relative error: its terms' (2^-22 (1 + |z - max|) with |z - max| e^(z - max) <= 1) and N + 16 u
        e_lse = ez.max(1).values + 2.0 ** -20 + (N + 16) * U + 4 * U * want.abs()
        within(lse, want, e_lse, f"{shape} {wo} {v0} lse")
        within(tl, hit, e_hit, "tlogit")
        within(loss, torch.where(counts, want - hit, 0.0), e_lse + e_hit + U * (want.abs() + hit.abs()), "loss")
        assert bool((loss[~counts] == 0).all()) and bool((tl[~here] == 0).all())


def test_xent_shards_join_to_the_whole():
    M, K, N = 70, 136, 1000
    g = gen(8)
    X, W = normal(g, M, K), normal(g, K, N, scale=0.3)
    t = torch.randint(0, N, (M,), device="cuda", generator=g)
    loss, lse, tl = F.fc_xent_fwd(X, W, t)
    cuts = [0, 8, 301, 640, 1000]
    parts = [F.fc_xent_fwd(X, W[:, a:b].contiguous(), t, vocab_start=a) for a, b in zip(cuts, cuts[1:])]
    joined = torch.logsumexp(torch.stack([p[1].double() for p in parts]), 0)
    within(lse, joined, 2.0 ** -18 * (1 + joined.abs()), "lse")
    assert torch.allclose(sum(p[2] for p in parts), tl, rtol=1e-6, atol=1e-6)


def test_xent_extreme_logits():
    """Logits at infinity and far apart: what the definition gives, and nothing else is disturbed."""
    inf = float("inf")
    K, N = 16, 300
    X = torch.zeros((6, K), dtype=torch.bfloat16, device="cuda")
    W = torch.zeros((K, N), dtype=torch.bfloat16, device="cuda")
    W[0], W[1, :], W[2, 7] = 1.0, -1.0, 1.0
    W[3] = torch.linspace(-3e4, 3e4, N, device="cuda").to(torch.bfloat16)
    X[0, 0] = inf      # every logit +inf
    X[1, 1] = inf      # every logit -inf
    X[2, 2] = 1000.0   # one far above the others
    X[3, 3] = 1.0      # spread over 6e4
    X[4, 0] = float("nan")
    X[5, 2] = -3e38    # one at the type's lowest value
    t = torch.full((6,), 7, dtype=torch.int64, device="cuda")
    # rows with infinities have NaN products with W's zeros: keep those out
    W[0, :], W[1, :] = 1.0, -1.0
    X2 = X.clone()
    z = X2.double() @ W.double()
    z[0], z[1], z[4] = inf, -inf, float("nan")
    one = torch.zeros((2, 1), dtype=torch.bfloat16, device="cuda")
    one[0, 0], one[1, 0] = inf, -inf  # K = 1: no zero times infinity
    _, lse1, _ = F.fc_xent_fwd(one, torch.ones((1, N), dtype=torch.bfloat16, device="cuda"), t[:2])
    assert lse1[0].item() == inf and lse1[1].item() == -inf
    loss, lse, tl = F.fc_xent_fwd(X[2:], W, t[2:])
    want = torch.logsumexp(z[2:], 1)
    within(lse, want, 2.0 ** -18 * (1 + want.abs()), "lse")
    assert torch.isnan(lse[2]) and tl[0].item() == 1000.0
    dX, dW = F.fc_xent_bwd(X[2:4], W, t[2:4], lse[:2].contiguous(), torch.ones(2, device="cuda"))
    p = torch.softmax(z[2:4], 1)
    p[:, 7] -= 1
    within(dX, p @ W.double().t(), H * 4 * (p.abs() @ W.double().abs().t()) + 1e-30, "dX")
    # a row that does not count is zero, whatever its logits are
    t[4] = -100
    dX, dW = F.fc_xent_bwd(X[2:], W, t[2:], torch.nan_to_num(lse), torch.ones(4, device="cuda"))
    assert bool((dX[2] == 0).all())
    # the same where the 256 x 256 tiles are taken
    X, W = normal(gen(4), 2600, 72), normal(gen(5), 72, 2600, scale=0.1)
    X[5], X[2599] = float("nan"), inf
    t = torch.arange(2600, device="cuda")
    t[5] = t[2599] = -100
    for wo in (ROW, COL):
        loss, lse, _ = F.fc_xent_fwd(X, stored(W, wo), t, w_order=wo)
        assert loss[5].item() == 0 and loss[2599].item() == 0 and bool(torch.isfinite(loss).all())
        dX, _ = F.fc_xent_bwd(X, stored(W, wo), t, lse, torch.ones(2600, device="cuda"), w_order=wo)
        assert bool((dX[5] == 0).all()) and bool((dX[2599] == 0).all()) and bool(torch.isfinite(dX).all())


@pytest.mark.parametrize("shape", XENT)
@pytest.mark.parametrize("wo", [ROW, COL])
def test_xent_bwd(shape, wo):
    M, K, N = shape
    g = gen(M + 5 * K + N)
    X, W = normal(g, M, K), normal(g, K, N, scale=0.3)
    for v0, whole, ignore in ((0, N, -100), (N, 3 * N, -100), (0, N, 0)):
        t = torch.randint(0, whole, (M,), device="cuda", generator=g)
        t[::3] = ignore
        z, ez, counts, here, at = xent64(X, W, t, v0, ignore)
        lse = (torch.logsumexp(z, 1) + (1.0 if v0 else 0.0)).float()  # a shard's probabilities sum to less than 1
        w = torch.rand(M, device="cuda", generator=g) - 0.3
        p = torch.exp(z - lse.double()[:, None])
        # the fp32 subtraction and exponential: 2^-22 (1 + |z| + |lse|) relative
        ep = p * torch.expm1(ez + 2.0 ** -22 * (1 + z.abs() + lse.double().abs()[:, None]))
        hot = torch.zeros_like(p)
        hot[here, at[here]] = 1.0
        wc = torch.where(counts, w.double(), 0.0)[:, None]
        D = wc * (p - hot)
        eD = wc.abs() * (ep + 2 * U * (p + hot))
        eD = eD + H * (D.abs() + eD)
        aX, aW, aD = X.double().abs(), W.double().abs(), D.abs() + eD
        tx = eD @ aW.t() + (N + 16) * U * (aD @ aW.t()) + 2.0 ** -126
        tw = aX.t() @ eD + (M + 16) * U * (aX.t() @ aD) + 2.0 ** -126
        wx, ww = D @ W.double().t(), X.double().t() @ D
        what = f"{shape} {wo} {v0} {ignore}"
        dX, dW = F.fc_xent_bwd(X, stored(W, wo), t, lse, w, w_order=wo, vocab_start=v0, ignore_index=ignore)
        within(dX, wx, tx + H * (wx.abs() + tx), what + " dX")
        within(dW, ww, tw + H * (ww.abs() + tw), what + " dW")
        assert bool((dX[~counts] == 0).all())
        acc = torch.ones((K, N), device="cuda")
        dX, dW = F.fc_xent_bwd(X, stored(W, wo), t, lse, w, w_order=wo, vocab_start=v0, ignore_index=ignore,
                               dx_dtype=F.OUT_F32, dW=acc, dw_dtype=F.OUT_F32_ACC)
        within(dX, wx, tx, what + " dX fp32")
        within(dW, ww + 1, tw + U * (ww.abs() + tw + 1), what + " dW accumulated")


def test_xent_bwd_in_several_pieces():
    """A vocabulary of more columns than one piece holds (256 MB of the logits' gradient)."""
    M, K, N = 16500, 40, 17001  # pieces of 7936 columns
    g = gen(12)
    X, W = normal(g, M, K), normal(g, K, N, scale=0.3)
    t = torch.randint(0, N, (M,), device="cuda", generator=g)
    t[:100] = torch.arange(100, device="cuda") * 170  # targets in every piece
    for wo in (ROW, COL):
        loss, lse, _ = F.fc_xent_fwd(X, stored(W, wo), t, w_order=wo)
        w = torch.full((M,), 1.0 / M, device="cuda")
        dX, dW = F.fc_xent_bwd(X, stored(W, wo), t, lse, w, w_order=wo)
        wX = torch.empty((M, K), dtype=torch.float64, device="cuda")
        wW, tW = (torch.zeros((K, N), dtype=torch.float64, device="cuda") for _ in range(2))
        tX = torch.empty_like(wX)
        for r in torch.split(torch.arange(M, device="cuda"), 4096):
            D = torch.exp(X[r].double() @ W.double() - lse[r].double()[:, None])
            D[torch.arange(len(r)), t[r]] -= 1
            D /= M
            # D errs by its rounding and by 2^-16 of the probability (|z| + |lse| below 40)
            eD = (H + 2.0 ** -16) * D.abs() + 2.0 ** -16 / M * D.abs().clamp(max=1)
            wX[r], tX[r] = D @ W.double().t(), eD @ W.double().abs().t()
            wW += X[r].double().t() @ D
            tW += X[r].double().abs().t() @ eD
        tX += (N + 16) * U / H * tX
        tW += (M + 16) * U / H * tW
        within(dX, wX, tX + H * (wX.abs() + tX), f"{wo} dX")
        within(dW, wW, tW + H * (wW.abs() + tW), f"{wo} dW")


def test_xent_gradient_by_differences():
    """Directional differences of the library's own loss."""
    M, K, N = 40, 64, 500
    g = gen(31)
    X, W = normal(g, M, K), normal(g, K, N, scale=0.2)
    t = torch.randint(0, N, (M,), device="cuda", generator=g)
    _, lse, _ = F.fc_xent_fwd(X, W, t)
    dX, dW = F.fc_xent_bwd(X, W, t, lse, torch.ones(M, device="cuda"), dx_dtype=F.OUT_F32, dw_dtype=F.OUT_F32)
    vX = torch.where(torch.rand((M, K), device="cuda", generator=g) < 0.5, -1.0, 1.0)
    h = 2.0 ** -3

    def loss_at(x):
        return F.fc_xent_fwd(x.to(torch.bfloat16), W, t)[0].double().sum().item()

    Xa, Xb = (X.float() + h * vX).to(torch.bfloat16), (X.float() - h * vX).to(torch.bfloat16)
    # what the rounded steps really were; the mean slope between two points differs from
    # the middle's by h^2 / 6 of the third derivative, which is at most |v.W|^3 a row
    step = (Xa.double() - Xb.double())
    mid = (Xa.double() + Xb.double()) / 2
    _, lse_m, _ = F.fc_xent_fwd(X, W, t)
    diff = loss_at(Xa) - loss_at(Xb)
    z = (mid @ W.double()).requires_grad_()
    torch.nn.functional.cross_entropy(z, t, reduction="sum").backward()
    slope = (step * (z.grad @ W.double().t())).sum().item()
    swing = (step @ W.double()).abs().max(1).values
    assert abs(diff - slope) <= (swing ** 3).sum().item() / 24 + M * 2.0 ** -18 * 20
    # and the analytic gradient at X itself is the library's
    ours = (step * dX.double()).sum().item()
    z0 = (X.double() @ W.double()).requires_grad_()
    torch.nn.functional.cross_entropy(z0, t, reduction="sum").backward()
    ref = z0.grad @ W.double().t()
    bound = (step.abs() * (2 * H * (z0.grad.abs() @ W.double().abs().t()))).sum().item()
    assert abs(ours - (step * ref).sum().item()) <= bound


# ---- experts

def offsets_of(counts, first=0):
    return torch.tensor([first] + counts, device="cuda").cumsum(0)


GROUPED = [  # rows of each expert, first row, rows behind the last, K, N
    ([1], 0, 0, 8, 8), ([0, 5, 0], 0, 3, 33, 7), ([3, 0, 130, 1], 2, 9, 64, 136), ([300, 17, 0, 64], 0, 0, 136, 264),
    ([0, 0, 0], 4, 1, 16, 24), ([1] * 70 + [0] * 30 + [5] * 33, 0, 2, 40, 130), ([260, 255, 257], 1, 0, 520, 100),
    ([33, 31, 32, 129], 0, 40, 72, 520), ([700, 0, 30, 1500, 63, 64, 65, 257], 3, 5, 1200, 1300),
    ([1100, 900, 0, 1], 0, 0, 1032, 2570), ([2600], 0, 1, 640, 2600), ([700], 0, 0, 264, 300), ([40] * 8, 0, 0, 1001, 129)]


# few rows against long reductions, which are split
GROUPED_LONG = [([1], 2, 3, 2000, 136), ([5, 0, 12], 1, 4, 1560, 77), ([40, 0, 61], 3, 2, 4104, 257),
                ([1, 0, 1], 0, 0, 777, 4100), ([64, 30], 5, 5, 8001, 130)]


@pytest.mark.parametrize("case", GROUPED + GROUPED_LONG, ids=lambda c: f"{len(c[0])}x{c[3]}x{c[4]}")
@pytest.mark.parametrize("wo", [ROW, COL])
def test_grouped_integers_are_exact(case, wo):
    counts, first, behind, K, N = case
    E, T = len(counts), first + sum(counts) + behind
    g = gen(T + K + N)
    X, dY, W = integers(g, T, K), integers(g, T, N), integers(g, E, K, N)
    off = offsets_of(counts, first)
    lo = off.tolist()
    for align in (lambda t: t, shifted):
        x, d, w = align(X), align(dY), align(stored(W, wo))
        for dt, od in ((torch.bfloat16, F.OUT_BF16), (torch.float32, F.OUT_F32)):
            Y = torch.full((T, N), 77.0, dtype=dt, device="cuda")
            dX = torch.full((T, K), 77.0, dtype=dt, device="cuda")
            wantY, wantX = Y.double(), dX.double()
            for e in range(E):
                s = slice(lo[e], lo[e + 1])
                wantY[s] = (X[s].double() @ W[e].double()).to(dt).double()
                wantX[s] = (dY[s].double() @ W[e].double().t()).to(dt).double()
            assert F.fc_grouped_fwd(x, w, off, w_order=wo, out=Y, out_dtype=od) is Y
            F.fc_grouped_bwd_data(d, w, off, w_order=wo, out=dX, out_dtype=od)
            assert torch.equal(Y.double(), wantY) and torch.equal(dX.double(), wantX)
        wantW = torch.stack([X[a:b].double().t() @ dY[a:b].double() for a, b in zip(lo, lo[1:])])
        assert torch.equal(F.fc_grouped_bwd_weight(x, d, off, out_dtype=F.OUT_F32).double(), wantW)
        assert torch.equal(F.fc_grouped_bwd_weight(x, d, off), wantW.float().to(torch.bfloat16))
        acc = torch.full((E, K, N), 2.0, device="cuda")
        F.fc_grouped_bwd_weight(x, d, off, out=acc, out_dtype=F.OUT_F32_ACC)
        assert torch.equal(acc.double(), wantW + 2)


@pytest.mark.parametrize("case", [([200, 0, 57, 300], 0, 0, 520, 264), ([3, 1, 0, 9] * 4, 0, 0, 1024, 384)],
                         ids=["rows", "few"])
def test_grouped_normal_inputs(case):
    counts, _, _, K, N = case
    E, T = len(counts), sum(counts)
    g = gen(77)
    X, dY, W = normal(g, T, K), normal(g, T, N, scale=1e-3), normal(g, E, K, N, scale=0.02)
    off = offsets_of(counts)
    lo = off.tolist()
    Y, dX = F.fc_grouped_fwd(X, W, off), F.fc_grouped_bwd_data(dY, W, off)
    dW = F.fc_grouped_bwd_weight(X, dY, off)
    for e in range(E):
        s = slice(lo[e], lo[e + 1])
        x, d, w = X[s].double(), dY[s].double(), W[e].double()
        for got, a, b in ((Y[s], x, w), (dX[s], d, w.t()), (dW[e], x.t(), d)):
            want, tol = a @ b, (a.shape[1] + 16) * U * (a.abs() @ b.abs())
            within(got, want, tol + H * (want.abs() + tol), f"expert {e}")


def test_grouped_bad_offsets_stay_inside():
    """Offsets outside the rows, or decreasing, are clamped: rows that no
    expert can name keep their values, and neighbouring memory too."""
    T, E, K, N = 50, 3, 24, 40
    g = gen(3)
    X, W = integers(g, T, K), integers(g, E, K, N)
    big = torch.full((T + 20, N), 9.0, dtype=torch.bfloat16, device="cuda")
    Y = big[10:10 + T]
    for bad in ([-5, 10, 30, 1 << 40], [60, 70, 80, 90], [40, 20, 10, 5], [-(1 << 62), -3, -2, -1]):
        big.fill_(9.0)
        off = torch.tensor(bad, device="cuda")
        F.fc_grouped_fwd(X, W, off, out=Y)
        torch.cuda.synchronize()
        assert bool((big[:10] == 9).all()) and bool((big[10 + T:] == 9).all()), bad
        F.fc_grouped_bwd_weight(X, X, off)
    torch.cuda.synchronize()


# ---- neighbouring memory

def among_nans(t, offset):
    """The same values, `offset` elements past a 16-byte boundary, between NaNs."""
    buf = torch.full((t.numel() + 1024,), float("nan"), dtype=t.dtype, device=t.device)
    out = buf[256 + offset:256 + offset + t.numel()].view(t.shape)
    out.copy_(t)
    return out


@pytest.mark.parametrize("shape", [(1, 1, 1), (2, 9, 2), (65, 7, 3), (129, 33, 1), (200, 1, 1), (70, 39, 5), (16, 264, 24),
                                   (33, 2051, 35), (100, 1000, 136), (2600, 70, 2570)])
@pytest.mark.parametrize("offset", [0, 1, 4])
def test_nothing_past_the_operands_counts(shape, offset):
    M, K, N = shape
    g = gen(M + K + N)
    X, W, dY = integers(g, M, K), integers(g, K, N), integers(g, M, N)
    Y, dX = X.float() @ W.float(), dY.float() @ W.float().t()
    Z = torch.ones((M, K), dtype=torch.bfloat16, device="cuda")
    t = torch.randint(0, N, (M,), device="cuda", generator=g)
    small = 2.0 ** -4  # logits of a few units
    z = Y.double() * small * small
    for wo in (ROW, COL):
        w = among_nans(stored(W, wo), offset)
        for xo in (ROW, COL):
            x = among_nans(stored(X, xo), offset)
            assert torch.equal(F.fc_fwd_act(x, w, x_order=xo, w_order=wo, out_dtype=F.OUT_F32), Y), (xo, wo)
        got, db = F.fc_bwd_data_act(among_nans(dY, offset), w, Z, F.ACT_RELU, w_order=wo, out_dtype=F.OUT_F32,
                                    bias_grad=True)
        assert torch.equal(got, dX) and bool(torch.isfinite(db).all())
        x, ws = among_nans(X * small, offset), among_nans(stored(W * small, wo), offset)
        loss, lse, _ = F.fc_xent_fwd(x, ws, t, w_order=wo)
        want = torch.logsumexp(z, 1)
        # |z| <= 9 K 2^-8 exactly held (integers over 256); see test_xent_fwd for the sum
        within(lse, want, 2.0 ** -20 + (N + 16) * U + 4 * U * want.abs(), f"{shape} lse")
        dX1, dW1 = F.fc_xent_bwd(x, ws, t, lse, torch.ones(M, device="cuda"), w_order=wo)
        assert bool(torch.isfinite(dX1).all()) and bool(torch.isfinite(dW1).all())


@pytest.mark.parametrize("shape", [(48, 1000, 20000), (5, 2056, 28008), (20, 776, 32000), (64, 1544, 16392)])
def test_few_rows_wide_and_long(shape):
    """A few rows against a wide W whose rows are the reduction, with nothing but NaN around it."""
    M, K, N = shape
    g = gen(M + N)
    X, W = among_nans(integers(g, M, K), 0), integers(g, K, N)
    Y = X.float() @ W.float()
    assert torch.equal(F.fc_fwd_act(X, among_nans(W, 0), out_dtype=F.OUT_F32), Y)
    # the gradient of the layer with K outputs and N inputs, W column-major: the same product
    Z = torch.ones((M, N), dtype=torch.bfloat16, device="cuda")
    Z[:, ::3] = -1.0
    dX, db = F.fc_bwd_data_act(X, among_nans(W, 0), Z, F.ACT_RELU, w_order=COL, out_dtype=F.OUT_F32, bias_grad=True)
    want = torch.where(Z > 0, Y, 0.0)
    assert torch.equal(dX, want) and torch.equal(db, want.sum(0))
    t = torch.randint(0, N, (M,), device="cuda", generator=g)
    z = Y.double() / 256
    _, lse, tl = F.fc_xent_fwd((X / 16).contiguous(), (W / 16).contiguous(), t)
    want = torch.logsumexp(z, 1)
    within(lse, want, 2.0 ** -20 + (N + 16) * U + 4 * U * want.abs(), f"{shape} lse")
    assert torch.equal(tl.double(), z.gather(1, t[:, None])[:, 0])


@pytest.mark.parametrize("case", [([3, 0, 70, 1], 2, 9, 40, 136), ([300, 17, 0, 64], 5, 3, 135, 264),
                                  ([1, 2], 3, 2, 1501, 40), ([700, 0, 30, 1500], 3, 5, 1200, 1300)],
                         ids=lambda c: f"{len(c[0])}x{c[3]}x{c[4]}")
@pytest.mark.parametrize("wo", [ROW, COL])
def test_rows_and_experts_do_not_meet(case, wo):
    """Rows that no expert has, and the matrices of experts without rows, are NaN."""
    counts, first, behind, K, N = case
    E, T = len(counts), first + sum(counts) + behind
    g = gen(T)
    X, dY, W = integers(g, T, K), integers(g, T, N), integers(g, E, K, N)
    nan = float("nan")
    for v in (X, dY):
        v[:first], v[T - behind:] = nan, nan
    for e in range(E):
        if counts[e] == 0:
            W[e] = nan
    off = offsets_of(counts, first)
    lo = off.tolist()
    x, d, w = among_nans(X, 0), among_nans(dY, 0), among_nans(stored(W, wo), 0)
    Y, dX = torch.zeros((T, N), device="cuda"), torch.zeros((T, K), device="cuda")
    F.fc_grouped_fwd(x, w, off, w_order=wo, out=Y, out_dtype=F.OUT_F32)
    F.fc_grouped_bwd_data(d, w, off, w_order=wo, out=dX, out_dtype=F.OUT_F32)
    dW = F.fc_grouped_bwd_weight(x, d, off, out_dtype=F.OUT_F32)
    wantY, wantX, wantW = torch.zeros_like(Y), torch.zeros_like(dX), torch.zeros_like(dW)
    for e in range(E):
        s = slice(lo[e], lo[e + 1])
        if counts[e]:
            wantY[s], wantX[s] = X[s].float() @ W[e].float(), dY[s].float() @ W[e].float().t()
            wantW[e] = X[s].float().t() @ dY[s].float()
    assert torch.equal(Y, wantY) and torch.equal(dX, wantX) and torch.equal(dW, wantW)


# ---- streams, graphs, several calls at once

def _all_calls(seed, M=96, K=200, N=328, E=3):
    """One call of each operator on inputs of a seed: the calls, by name."""
    g = gen(seed)
    X, W, b, R = normal(g, M, K), normal(g, K, N, scale=0.1), normal(g, N), normal(g, M, N)
    dY, Z = normal(g, M, N), normal(g, M, K)
    t = torch.randint(0, N, (M,), device="cuda", generator=g)
    lse, w = torch.full((M,), 6.0, device="cuda"), torch.rand(M, device="cuda", generator=g)
    We, off = normal(g, E, K, N, scale=0.1), offsets_of([M // 2, 0, M - M // 2])
    return {
        "fwd_act": lambda **k: F.fc_fwd_act(X, W, bias=b, act=F.ACT_GELU, residual=R, keep_z=True, **k),
        "bwd_data_act": lambda **k: F.fc_bwd_data_act(dY, W, Z, F.ACT_SILU, bias_grad=True, **k),
        "bwd_act": lambda **k: F.fc_bwd_act(dY, R, F.ACT_GELU_TANH, **k),
        "xent_fwd": lambda **k: F.fc_xent_fwd(X, W, t, **k),
        "xent_bwd": lambda **k: F.fc_xent_bwd(X, W, t, lse, w, **k),
        "grouped_fwd": lambda **k: (F.fc_grouped_fwd(X, We, off, **k),),
        "grouped_bwd_data": lambda **k: (F.fc_grouped_bwd_data(dY, We, off, **k),),
        "grouped_bwd_weight": lambda **k: (F.fc_grouped_bwd_weight(X, dY, off, **k),),
    }


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


# odd sizes (copies, element stores), few rows (split reductions), and plain ones
SIZES = [(96, 200, 328), (33, 1001, 131), (3, 2048, 264), (520, 264, 520)]


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
    X, W, b = normal(g, 8, 16), normal(g, 16, 24), normal(g, 24)
    t = torch.zeros(8, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError, match="inner"):
        F.fc_fwd_act(X, W.t().contiguous())
    with pytest.raises(TypeError, match="bias"):
        F.fc_fwd_act(X, W, bias=b[:23])
    with pytest.raises(TypeError, match="residual"):
        F.fc_fwd_act(X, W, residual=X)
    with pytest.raises(ValueError, match="contiguous"):
        F.fc_fwd_act(X, W[:, ::2])
    with pytest.raises(ValueError, match="OUT_BF16"):
        F.fc_fwd_act(X, W, out_dtype=F.OUT_F32_ACC)
    with pytest.raises(F.FcError):
        F.fc_fwd_act(X, W, act=9)
    with pytest.raises(F.FcError):
        F.fc_fwd_act(X, W, residual=(R := normal(g, 8, 24)), out=R)  # the output on an input
    with pytest.raises(TypeError, match="targets"):
        F.fc_xent_fwd(X, W, t.int())
    with pytest.raises(TypeError, match="targets"):
        F.fc_xent_fwd(X, W, t[:7])
    with pytest.raises(F.FcError):
        F.fc_xent_fwd(X, W, t, vocab_start=-1)
    with pytest.raises(ValueError, match="accumulating"):
        F.fc_xent_bwd(X, W, t, torch.zeros(8, device="cuda"), torch.zeros(8, device="cuda"),
                      dw_dtype=F.OUT_F32_ACC)
    with pytest.raises(TypeError, match="offsets"):
        F.fc_grouped_fwd(X, W[None], torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="accumulating"):
        F.fc_grouped_bwd_weight(X, X, torch.zeros(2, dtype=torch.int64, device="cuda"), out_dtype=F.OUT_F32_ACC)


# ---- together

def test_a_step_of_all_of_them():
    """One training step of a small model: an MLP with bias, activation and
    residual, an expert layer, and the vocabulary's loss; forward and backward
    with these calls, against the same model in 64 bits.

    The step rounds to bf16 after each operator: 7 roundings lie between the
    inputs and any of its outputs. In the Frobenius norm a rounding changes a
    tensor by at most h = 2^-8 relative, and every map in between passes a
    relative change on by at most the bound below: 16 h."""
    M, K, Hd, N, E = 192, 128, 320, 1000, 4
    g = gen(55)
    X = normal(g, M, K)
    W1, b1 = normal(g, K, Hd, scale=K ** -0.5), normal(g, Hd, scale=0.1)
    W2 = normal(g, Hd, K, scale=Hd ** -0.5)
    We, V = normal(g, E, K, K, scale=K ** -0.5), normal(g, K, N, scale=K ** -0.5)
    off = offsets_of([70, 0, 90, 32])
    t = torch.randint(0, N, (M,), device="cuda", generator=g)
    t[::5] = -100
    w = (t != -100).float() / (t != -100).sum()

    A, Z = F.fc_fwd_act(X, W1, bias=b1, act=F.ACT_GELU_TANH, keep_z=True)
    B = F.fc_fwd_act(A, W2, residual=X)
    C = F.fc_grouped_fwd(B, We, off)
    loss, lse, _ = F.fc_xent_fwd(C, V, t)
    dC, dV = F.fc_xent_bwd(C, V, t, lse, w)
    dB, dWe = F.fc_grouped_bwd_data(dC, We, off), F.fc_grouped_bwd_weight(B, dC, off)
    dZ, db1 = F.fc_bwd_data_act(dB, W2, Z, F.ACT_GELU_TANH, bias_grad=True)
    dW2 = F.fc_bwd_weight(A, dB)
    dW1 = F.fc_bwd_weight(X, dZ)

    x, w1, bb, w2, we, v = (q.double().requires_grad_() for q in (X, W1, b1, W2, We, V))
    a = torch.nn.functional.gelu(x @ w1 + bb, approximate="tanh")
    bq = a @ w2 + x
    lo = off.tolist()
    c = torch.cat([bq[p:q] @ we[e] for e, (p, q) in enumerate(zip(lo, lo[1:]))])
    each = torch.nn.functional.cross_entropy(c @ v, t, reduction="none")
    (each * w).sum().backward()
    for name, got, want in (("loss", loss, each), ("dV", dV, v.grad), ("dWe", dWe, we.grad), ("dW2", dW2, w2.grad),
                            ("dW1", dW1, w1.grad), ("db1", db1, bb.grad)):
        rel = ((got.double() - want).norm() / want.norm()).item()
        log(f"  {name}: {rel:.3g}")
        assert rel <= 16 * H, name


# ---- values at the ends of the types

@pytest.mark.parametrize("shape", [(4000, 640, 4104), (4001, 640, 4099), (333, 611, 1531), (40, 512, 264)])
@pytest.mark.parametrize("wo", [ROW, COL])
def test_bias_gradient_of_infinite_weights(shape, wo):
    """Column sums of infinities are infinities: a tile's rows past the last one, whose products of zeros
    with infinite weights are NaN, are not in them."""
    M, N, K = shape
    g = gen(M)
    dY = torch.randint(1, 4, (M, N), device="cuda", generator=g).to(torch.bfloat16)
    W, Z = integers(g, K, N), torch.ones((M, K), dtype=torch.bfloat16, device="cuda")
    up = dY.double() @ W.double().t()
    W[3, 5], W[K - 1, 0] = float("inf"), -float("inf")
    up[:, 3], up[:, K - 1] = float("inf"), -float("inf")  # dY is positive
    for act in ACTS:  # every slope is positive at 1
        dX, db = F.fc_bwd_data_act(dY, stored(W, wo), Z, act, w_order=wo, out_dtype=F.OUT_F32, bias_grad=True)
        assert db[3].item() == float("inf") and db[K - 1].item() == -float("inf"), ACT_NAMES[act]
        assert bool(torch.isfinite(db[4:K - 1]).all()) and bool(torch.isfinite(db[:3]).all()), ACT_NAMES[act]
        if act in (F.ACT_NONE, F.ACT_RELU):  # sums of integers below 2^24
            assert torch.equal(dX.double(), up) and torch.equal(db.double(), up.sum(0))


@pytest.mark.parametrize("shape", [(4100, 640, 1500), (130, 72, 520), (96, 2001, 300)])
@pytest.mark.parametrize("wo", [ROW, COL])
def test_xent_logits_of_any_size(shape, wo):
    """Logits up to the type's largest and lowest values (a mask's), in some columns or in all."""
    M, K, N = shape
    g = gen(N)
    X, W = normal(g, M, K), normal(g, K, N, scale=0.3)
    X[:, 0] = (1 + torch.arange(M, device="cuda") % 128 / 128.0).to(torch.bfloat16)  # 1 <= x < 2, held exactly
    t = torch.randint(0, N, (M,), device="cuda", generator=g)
    for big in (-1e6, -1e10, -3e37, -1.6e38):
        W[0] = 0.0
        W[0, N // 4:N // 2 + 3] = big
        W[0, N - 1] = big
        rest = W[0] == 0
        z = X.double() @ W.double()
        _, lse, tl = F.fc_xent_fwd(X, stored(W, wo), t, w_order=wo)
        want = torch.logsumexp(z, 1)  # of the columns that are not masked: the others' terms are below e^-10^5
        ez = (K + 16) * U * (X.double().abs() @ W[:, rest].double().abs()).max(1).values
        within(lse, want, ez + 2.0 ** -20 + (N + 16) * U + 4 * U * want.abs(), f"{shape} {wo} {big:g} in places")
        hit = z.gather(1, t[:, None])[:, 0]
        assert bool(((tl.double() - hit).abs() <= (K + 16) * U * (X.double().abs() @ W.double().abs()).max(1).values).all())
    # one value in all columns: lse = z + log N, whose two additions round
    Xs = torch.zeros_like(X)
    Xs[:, 0] = X[:, 0]
    for big in (-1.6e38, -1e10, -1e6, -30.0, 0.0, 30.0, 1e6, 1e10, 1.6e38):
        W[0] = big
        z = Xs[:, 0].double() * W[0, 0].double()
        _, lse, _ = F.fc_xent_fwd(Xs, stored(W, wo), t, w_order=wo)
        want = z + math.log(N)
        within(lse, want, 2.0 ** -20 + (N + 16) * U + 4 * U * want.abs(), f"{shape} {wo} {big:g} everywhere")


@pytest.mark.parametrize("shape", [(20, 1, 1), (30, 256, 72), (4096, 512, 4096)])
def test_gelu_of_negative_values(shape):
    """The negative tail of z Phi(z) and its slope against erfc, relative to the value. exp(-z^2 / 2)
    comes from an argument with three roundings, 1.5 z^2 u relative; the fit, its evaluation, the reciprocal,
    the exponential and the products 16 u."""
    M, K, N = shape
    zs = torch.linspace(-12.5, -0.25, 4001, device="cuda").to(torch.bfloat16)
    for z in zs.split(M) if M < 64 else (zs,):
        m = z.numel()
        X, W = torch.zeros((m, K), dtype=torch.bfloat16, device="cuda"), torch.zeros((K, N), dtype=torch.bfloat16, device="cuda")
        X[:, 0], W[0] = z, 1.0
        zd = z.double()
        cdf, pdf = 0.5 * torch.special.erfc(-zd * 0.5 ** 0.5), torch.exp(-0.5 * zd * zd) / (2 * math.pi) ** 0.5
        rel = 16 * U + 2 * zd * zd * U
        Y = F.fc_fwd_act(X, W, act=F.ACT_GELU, out_dtype=F.OUT_F32)
        within(Y, (zd * cdf)[:, None].expand(m, N), (rel * (zd * cdf).abs())[:, None], f"{shape} gelu")
        # dX = (dY W^T) slope(Z), dY W^T = 1
        dY, Wd = X[:, :1].clone().fill_(1.0), torch.ones((N, 1), dtype=torch.bfloat16, device="cuda")
        Z = z[:, None].expand(m, N).contiguous()
        dX = F.fc_bwd_data_act(dY, Wd, Z, F.ACT_GELU, out_dtype=F.OUT_F32)
        within(dX, (cdf + zd * pdf)[:, None].expand(m, N), (rel * (cdf + zd.abs() * pdf))[:, None], f"{shape} slope")


@pytest.mark.parametrize("other", [False, True])
def test_expert_layers_without_rows(other):
    """A step in which no row came: empty outputs, weight gradients of zeros (or left as they were)."""
    E, K, N = 3, 24, 40
    g = gen(6)
    X, dY = torch.empty((0, K), dtype=torch.bfloat16, device="cuda"), torch.empty((0, N), dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    k = {"stream": torch.cuda.Stream()} if other else {}
    torch.cuda.synchronize()
    for wo in (ROW, COL):
        W = stored(normal(g, E, K, N), wo)
        for od, dt in ((F.OUT_BF16, torch.bfloat16), (F.OUT_F32, torch.float32)):
            Y, dX = F.fc_grouped_fwd(X, W, off, w_order=wo, out_dtype=od, **k), F.fc_grouped_bwd_data(dY, W, off, w_order=wo, out_dtype=od, **k)
            assert Y.shape == (0, N) and dX.shape == (0, K) and Y.dtype == dX.dtype == dt
            dW = torch.full((E, K, N), 5.0, dtype=dt, device="cuda")
            torch.cuda.synchronize()
            assert F.fc_grouped_bwd_weight(X, dY, off, out=dW, out_dtype=od, **k) is dW
            torch.cuda.synchronize()
            assert bool((dW == 0).all())
    acc = torch.full((E, K, N), 5.0, device="cuda")
    F.fc_grouped_bwd_weight(X, dY, off, out=acc, out_dtype=F.OUT_F32_ACC, **k)
    torch.cuda.synchronize()
    assert bool((acc == 5).all())
    with pytest.raises(TypeError, match="offsets"):  # checked as with rows
        F.fc_grouped_fwd(X, W, off[:2], w_order=COL)
    with pytest.raises(ValueError, match="accumulating"):
        F.fc_grouped_bwd_weight(X, dY, off, out_dtype=F.OUT_F32_ACC)


def test_expert_layers_without_rows_in_a_graph():
    E, K, N = 2, 16, 24
    X, dY = torch.empty((0, K), dtype=torch.bfloat16, device="cuda"), torch.empty((0, N), dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        dW = F.fc_grouped_bwd_weight(X, dY, off)
    for _ in range(3):
        dW.fill_(1.0)
        gr.replay()
        torch.cuda.synchronize()
        assert bool((dW == 0).all())


def test_a_stream_of_another_device_is_refused():
    g = gen(1)
    X, W = normal(g, 8, 16), normal(g, 16, 24)
    far = torch.cuda.Stream(stream_id=0, device_index=X.get_device() + 1, device_type=torch.cuda.current_stream().device_type)
    with pytest.raises(ValueError, match="stream"):
        F.fc_fwd_act(X, W, stream=far)


# ---- the 256 x 256 tiles: shapes that the planner sends there (test_fused_cpu.py asks it)

# whole reductions of 8 and 10 stages of 64 (2 and 4 past a period of 6), a partial last stage, and
# rows of 8 values' multiples or not
RING = [(4096, 512, 4096), (4000, 640, 4104), (4000, 600, 4104), (4001, 600, 4099)]
RING_XENT_BWD = [(4096, 2048, 4096), (4352, 2048, 4352), (4100, 2056, 4104), (4099, 2049, 4103)]
RING_GROUPED = [([1100, 900, 0, 2000], 0, 0, 1024, 4096), ([1600, 0, 70, 1800, 513], 3, 14, 2056, 4104),
                ([1103, 900, 1500, 497], 1, 2, 1031, 4103), ([1100, 900, 0, 2000], 0, 0, 512, 4096)]


@pytest.mark.parametrize("shape", RING)
@pytest.mark.parametrize("xo, wo", [(ROW, ROW), (ROW, COL), (COL, ROW), (COL, COL)])
def test_fwd_act_in_large_tiles(shape, xo, wo):
    test_fwd_act(shape, xo, wo)


@pytest.mark.parametrize("shape", RING + [(4096, 100, 4096)])
@pytest.mark.parametrize("wo", [ROW, COL])
def test_bwd_data_act_in_large_tiles(shape, wo):
    test_bwd_data_act(shape, wo)


@pytest.mark.parametrize("shape", RING)
@pytest.mark.parametrize("wo", [ROW, COL])
def test_xent_fwd_in_large_tiles(shape, wo):
    test_xent_fwd(shape, wo)


@pytest.mark.parametrize("shape", RING_XENT_BWD)
@pytest.mark.parametrize("wo", [ROW, COL])
def test_xent_bwd_in_large_tiles(shape, wo):
    test_xent_bwd(shape, wo)


@pytest.mark.parametrize("case", RING_GROUPED, ids=lambda c: f"{len(c[0])}x{c[3]}x{c[4]}")
@pytest.mark.parametrize("wo", [ROW, COL])
def test_grouped_in_large_tiles(case, wo):
    test_grouped_integers_are_exact(case, wo)


@pytest.mark.parametrize("shape", [RING[0], RING[3]])
@pytest.mark.parametrize("wo", [ROW, COL])
def test_xent_rows_that_do_not_count_in_large_tiles(shape, wo):
    """Rows of NaN and infinities whose targets are to be ignored: no loss, no gradient, no other row disturbed."""
    M, K, N = shape
    g = gen(K)
    X, W = normal(g, M, K), normal(g, K, N, scale=0.1)
    t = torch.arange(M, device="cuda") % N
    out = torch.tensor([5, 128, 255, 256, M - 1], device="cuda")
    X[out[::2]], X[out[1::2]] = float("nan"), float("inf")
    t[out] = -100
    counts = t != -100
    z = X[counts].double() @ W.double()
    ez = (K + 16) * U * (X[counts].double().abs() @ W.double().abs()).max(1).values
    loss, lse, _ = F.fc_xent_fwd(X, stored(W, wo), t, w_order=wo)
    want = torch.logsumexp(z, 1)
    within(lse[counts], want, ez + 2.0 ** -20 + (N + 16) * U + 4 * U * want.abs(), f"{shape} lse")
    assert bool((loss[~counts] == 0).all()) and bool(torch.isfinite(loss).all())
    dX, _ = F.fc_xent_bwd(X, stored(W, wo), t, lse, torch.ones(M, device="cuda"), w_order=wo)
    assert bool((dX[~counts] == 0).all()) and bool(torch.isfinite(dX).all())


# pieces of 7936 columns, the last of 33
LAST_PIECE = [(16500, 40, 15905), (16500, 128, 15905)]


@pytest.mark.parametrize("shape", LAST_PIECE)
def test_xent_bwd_with_a_short_last_piece(shape):
    """A last piece of fewer columns than a stage of the large tiles' reduction."""
    M, K, N = shape
    g = gen(9)
    X, W = normal(g, M, K), normal(g, K, N, scale=0.3)
    t = torch.randint(0, N, (M,), device="cuda", generator=g)
    t[:40] = torch.arange(N - 40, N, device="cuda")
    lse = torch.full((M,), 12.0, device="cuda")
    w = torch.full((M,), 1.0 / M, device="cuda")
    for wo in (ROW, COL):
        dX, dW = F.fc_xent_bwd(X, stored(W, wo), t, lse, w, w_order=wo, dx_dtype=F.OUT_F32, dw_dtype=F.OUT_F32)
        wW, tW = (torch.zeros((K, N), dtype=torch.float64, device="cuda") for _ in range(2))
        for r in torch.split(torch.arange(M, device="cuda"), 4096):
            z = X[r].double() @ W.double()
            p = torch.exp(z - 12.0)
            ez = (K + 16) * U * (X[r].double().abs() @ W.double().abs())
            ep = p * torch.expm1(ez + 2.0 ** -22 * (13 + z.abs()))
            p[torch.arange(len(r)), t[r]] -= 1
            D = p / M
            eD = (ep + 2 * U * (p.abs() + 1)) / M
            eD = eD + H * (D.abs() + eD)
            aD, aW, aX = D.abs() + eD, W.double().abs(), X[r].double().abs()
            within(dX[r], D @ W.double().t(), (eD + (N + 16) * U * aD) @ aW.t(), f"{shape} {wo} dX")
            wW += X[r].double().t() @ D
            tW += aX.t() @ (eD + (M + 16) * U * aD)
        within(dW, wW, tW, f"{shape} {wo} dW")


# tiles of 32 and 64 rows whose operands go straight into LDS, and the few-row kernel with more than 256
# blocks of columns (16 rows and 32)
@pytest.mark.parametrize("shape", [(20, 128, 520), (64, 72, 520), (5, 264, 5000), (30, 264, 5000)])
@pytest.mark.parametrize("wo", [ROW, COL])
def test_fwd_act_of_few_rows(shape, wo):
    test_fwd_act(shape, ROW, wo)


@pytest.mark.parametrize("wo", [ROW, COL])
def test_xent_of_few_rows(wo):
    test_xent_fwd((64, 72, 4000), wo)
    test_xent_bwd((64, 72, 4000), wo)


@pytest.mark.parametrize("shape", [(4096, 640, 4096), (130, 72, 520), (96, 2001, 300), (700, 40, 4001)])
@pytest.mark.parametrize("wo", [ROW, COL])
def test_xent_bwd_with_equal_weights(shape, wo):
    """Rows of one weight (a mean over the rows that count): the targets' values of the logits' gradient, w (p - 1),
    which make up nearly all of it, are held as p - 1, whose rounding is at most p, instead of all erring by
    the weight's rounding. Most rows, the first ones among them, do not count and have another weight."""
    M, K, N = shape
    g = gen(M + N)
    X, W = normal(g, M, K), normal(g, K, N, scale=0.1 * K ** -0.5)
    t = torch.randint(0, N, (M,), device="cuda", generator=g)
    t[:M // 2], t[::3] = -100, -100
    counts = t != -100
    z = X.double() @ W.double()
    ez = (K + 16) * U * (X.double().abs() @ W.double().abs())
    lse = torch.logsumexp(z, 1).float()
    p = torch.exp(z - lse.double()[:, None])
    ep = p * torch.expm1(ez + 2.0 ** -22 * (1 + z.abs() + lse.double().abs()[:, None]))
    hot = torch.zeros_like(p)
    hot[counts, t[counts]] = 1.0
    aX, aW = X.double().abs(), W.double().abs()
    for weight in (1.0 / 7782, 1.0 / 3, -0.7, 1.9921875):
        w = torch.where(counts, torch.tensor(weight, device="cuda"), 1.0)
        wd = torch.where(counts, w.double(), 0.0)[:, None]
        D = wd * (p - hot)
        # p rounds by H p; p - 1 by H (1 - p), but by no more than p where -1 is nearest; the factor and its use by 8 u
        eD = wd.abs() * (ep + torch.where(hot > 0, torch.minimum(H * (1 - p + ep), p + ep), H * (p + ep)) + 8 * U * (p + hot))
        aD = D.abs() + eD
        tx = (eD + (N + 16) * U * aD) @ aW.t() + 2.0 ** -126
        tw = aX.t() @ (eD + (M + 16) * U * aD) + 2.0 ** -126
        dX, dW = F.fc_xent_bwd(X, stored(W, wo), t, lse, w, w_order=wo, dx_dtype=F.OUT_F32, dw_dtype=F.OUT_F32)
        within(dX, D @ W.double().t(), tx, f"{shape} {wo} {weight:.3g} dX")
        within(dW, X.double().t() @ D, tw, f"{shape} {wo} {weight:.3g} dW")
        acc = torch.ones((K, N), device="cuda")
        F.fc_xent_bwd(X, stored(W, wo), t, lse, w, w_order=wo, dW=acc, dw_dtype=F.OUT_F32_ACC)
        within(acc, X.double().t() @ D + 1, tw + U * (2 + tw), "dW accumulated")
    # no row counts, weights of zero, infinite weights of rows that do not count
    for w, t2 in ((torch.ones(M, device="cuda"), torch.full_like(t, -100)), (torch.zeros(M, device="cuda"), t),
                  (torch.where(counts, 0.0, math.inf), t)):
        dX, dW = F.fc_xent_bwd(X, stored(W, wo), t2, lse, w, w_order=wo)
        assert bool((dX == 0).all()) and bool((dW == 0).all())


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("wo", [ROW, COL])
def test_one_unaligned_operand_is_copied_alone(which, wo):
    """Of two operands whose rows fit the large tiles, one at an odd address: the other's part of the
    workspace stays untouched."""
    M, K, N = RING[0]
    g = gen(which)
    X, W = integers(g, M, K), stored(integers(g, K, N), wo)
    want = X.double() @ (W if wo == ROW else W.t()).double()
    x, w = (shifted(X), W) if which == 0 else (X, shifted(W))
    L = F.lib()
    need = L.fc_fwd_act_ws_bytes(M, K, N, ROW, wo, 0)
    assert need == 2 * (M * K + K * N)  # a copy of each
    ws = torch.full((need,), 171, dtype=torch.uint8, device="cuda")
    Y = torch.empty((M, N), device="cuda")
    assert L.fc_fwd_act(x.data_ptr(), ROW, w.data_ptr(), wo, None, None, F.ACT_NONE, None, Y.data_ptr(), F.OUT_F32,
                        M, K, N, ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream) == F.FC_OK
    torch.cuda.synchronize()
    assert torch.equal(Y.double(), want)
    copies = ws[:2 * M * K], ws[2 * M * K:]
    assert not bool((copies[which] == 171).all()) and bool((copies[1 - which] == 171).all())


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("wo", [ROW, COL])
def test_one_unaligned_operand(which, wo):
    """The same in the other operators, where both operands' copies serve several products."""
    move = (shifted, lambda t: t) if which == 0 else (lambda t: t, shifted)
    M, K, N = RING[1]
    g = gen(which + 2)
    dY, W = integers(g, M, N), integers(g, K, N)
    Z = torch.ones((M, K), dtype=torch.bfloat16, device="cuda")
    dX = F.fc_bwd_data_act(move[0](dY), move[1](stored(W, wo)), Z, F.ACT_RELU, w_order=wo, out_dtype=F.OUT_F32)
    assert torch.equal(dX.double(), dY.double() @ W.double().t())
    M, K, N = RING_XENT_BWD[1]
    X, W = normal(g, M, K), stored(normal(g, K, N, scale=0.02), wo)
    t = torch.randint(0, N, (M,), device="cuda", generator=g)
    w = torch.rand(M, device="cuda", generator=g)
    fwd = F.fc_xent_fwd(X, W, t, w_order=wo)
    assert same(F.fc_xent_fwd(move[0](X), move[1](W), t, w_order=wo), fwd)  # the same kernels, the same bits
    assert same(F.fc_xent_bwd(move[0](X), move[1](W), t, fwd[1], w, w_order=wo),
                F.fc_xent_bwd(X, W, t, fwd[1], w, w_order=wo))
    counts, first, behind, K, N = RING_GROUPED[1]
    T, off = first + sum(counts) + behind, offsets_of(counts, first)
    X, dY, W = integers(g, T, K), integers(g, T, N), stored(integers(g, len(counts), K, N), wo)
    rows = slice(first, T - behind)
    assert torch.equal(F.fc_grouped_fwd(move[0](X), move[1](W), off, w_order=wo)[rows], F.fc_grouped_fwd(X, W, off, w_order=wo)[rows])
    assert torch.equal(F.fc_grouped_bwd_data(move[0](dY), move[1](W), off, w_order=wo)[rows],
                       F.fc_grouped_bwd_data(dY, W, off, w_order=wo)[rows])
    assert torch.equal(F.fc_grouped_bwd_weight(move[0](X), move[1](dY), off), F.fc_grouped_bwd_weight(X, dY, off))
