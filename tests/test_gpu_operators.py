"""Layer norm, the dense linear layer and the vocabulary cross entropy on MI355X against
float64.

Tolerances are derived, element by element, from the arithmetic the calls document:
  - a value rounded to a type is off by at most u(type) = finfo.eps / 2 of itself;
  - a float32 sum of K terms, in any order, is off by at most about K 2^-24 of the sum of
    their magnitudes (a product's K is its inner width, `acc(K)` below, with 8 more for the
    steps around it);
  - bf16 products of the backward read dp or dl rounded to bf16: u(bf16) of each term;
  - erf, tanh, exp and log in float32: a few units in the last place, taken as 2^-20 of the
    activation's argument scale.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
U = {F32: 2.0 ** -24, BF16: 2.0 ** -8}
FN = 2.0 ** -20
TINY = 1e-30


def acc(k):
    return (k + 8) * 2.0 ** -24


@pytest.fixture(scope="module")
def B():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from orthogonal_reparameterized_amd import binding
    return binding


def rand(seed, *shape, dtype=F32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g, dtype=F32) * scale).to(dtype)


def dev(t):
    return None if t is None else t.cuda()


def within(got, ref, tol, what):
    """|got - ref| <= tol everywhere (float64), NaN where and only where ref is NaN."""
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, what
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), what
    d = (got - ref).abs()
    tol = torch.as_tensor(tol, dtype=torch.float64).expand_as(d)
    bad = (d > tol + TINY) & ~torch.isnan(d)
    if bad.any():
        i = int(torch.nonzero(bad.reshape(-1))[0])
        pytest.fail(f"{what}: {int(bad.sum())} of {bad.numel()} off, first {i}: got {got.reshape(-1)[i].item():.9g} "
                    f"ref {ref.reshape(-1)[i].item():.9g} tol {tol.reshape(-1)[i].item():.3g}")


def off(got, ref):
    """2-norm of the difference over that of the reference."""
    return float((got.detach().cpu().double() - ref).norm() / ref.norm().clamp(min=TINY))


# ------------------------------------------------------------------------ layer norm ----

NORM_SHAPES = [(1, 1), (3, 7), (5, 8), (1, 5120), (70, 64), (33, 513), (1500, 1000), (9, 1024), (7, 1025),
               (300, 2048), (40, 4096), (11, 4100), (6, 8192), (5, 9001), (3, 16384)]


def norm_ref(x, gamma, beta, eps):
    x = x.double()
    mu = x.mean(1, keepdim=True)
    var = ((x - mu) ** 2).mean(1, keepdim=True)
    r = (var + eps) ** -0.5
    xh = (x - mu) * r
    g = torch.ones(x.shape[1], dtype=torch.float64) if gamma is None else gamma.double()
    b = torch.zeros(x.shape[1], dtype=torch.float64) if beta is None else beta.double()
    return mu, r, xh, g, b


@pytest.mark.parametrize("n,d", NORM_SHAPES)
@pytest.mark.parametrize("dtype,pdtype", [(BF16, F32), (BF16, BF16), (F32, F32), (BF16, None)])
def test_layernorm(B, n, d, dtype, pdtype):
    eps = 1e-5
    x = (rand(1, n, d) * torch.exp(rand(2, n, 1)) + rand(3, n, 1)).to(dtype)
    dy, dres = rand(4, n, d, dtype=dtype), rand(5, n, d, dtype=dtype)
    gamma = None if pdtype is None else rand(6, d, dtype=pdtype, scale=0.2) + 1
    beta = None if pdtype is None else rand(7, d, dtype=pdtype)
    mu, r, xh, g, b = norm_ref(x, gamma, beta, eps)
    y, mean, rstd = B.poetx_layernorm_forward(dev(x), dev(gamma), dev(beta), eps)
    mag = x.double().abs().mean(1, keepdim=True)
    e_mu = acc(d) * mag                       # the mean's error
    # r depends on the variance v as v^(-1/2): half its relative error, and e_mu enters the
    # variance squared; x - mu is off by e_mu and its own rounding
    e_r = (0.5 * acc(d) + 4 * 2.0 ** -24) * r + 0.5 * r ** 3 * e_mu ** 2
    e_c = e_mu + U[F32] * ((x.double() - mu).abs() + mu.abs())
    e_xh = e_c * r + xh.abs() * (e_r / r + 4 * 2.0 ** -24)
    within(mean, mu[:, 0], e_mu[:, 0], "mean")
    within(rstd, r[:, 0], e_r[:, 0] + r[:, 0] ** 2 * e_mu[:, 0] * acc(d), "rstd")
    ref = xh * g + b
    within(y, ref, U[dtype] * ref.abs() + 1.01 * (e_xh * g.abs() + 4 * U[F32] * (ref.abs() + b.abs())), "y")

    for with_res in (False, True):
        got = B.poetx_layernorm_backward(dev(x), dev(dy), dev(gamma), mean, rstd, dres=dev(dres) if with_res else None)
        gy = dy.double() * g
        m1, m2 = gy.mean(1, keepdim=True), (gy * xh).mean(1, keepdim=True)
        dx = r * (gy - m1 - xh * m2)
        # the backward takes the forward's float32 statistics: e_xh and e_r again
        e_m1 = acc(d) * gy.abs().mean(1, keepdim=True)
        e_m2 = acc(d) * (gy * xh).abs().mean(1, keepdim=True) + (gy.abs() * e_xh).mean(1, keepdim=True)
        e = r * (e_m1 + xh.abs() * e_m2 + e_xh * m2.abs() + 6 * U[F32] * (gy.abs() + m1.abs() + (xh * m2).abs()))
        e = e + dx.abs() * (e_r / r)
        if with_res:
            dx = dx + dres.double()
        within(got["dx"], dx, U[dtype] * dx.abs() + 1.01 * (e + U[F32] * dx.abs()), f"dx {with_res}")
        dyd = dy.double()
        within(got["dgamma"], (dyd * xh).sum(0), acc(n) * (dyd * xh).abs().sum(0) + (dyd.abs() * e_xh).sum(0),
               "dgamma")
        within(got["dbeta"], dyd.sum(0), acc(n) * dyd.abs().sum(0), "dbeta")
    only = B.poetx_layernorm_backward(dev(x), dev(dy), dev(gamma), mean, rstd, dres=dev(dres), want_params=False)
    assert set(only) == {"dx"} and torch.equal(only["dx"], got["dx"])


def test_layernorm_degenerate_rows(B):
    """Constant rows (variance 0), rows with an infinity or a NaN beside clean ones, no rows."""
    d = 300
    x = rand(11, 4, d, dtype=BF16)
    x[0] = 3.0
    x[1, 5] = float("inf")
    x[2, 299] = float("nan")
    y, mean, rstd = B.poetx_layernorm_forward(dev(x), None, None, 1e-5)
    assert torch.equal(y[0].cpu(), torch.zeros(d, dtype=BF16))
    assert abs(float(rstd[0]) * 1e-5 ** 0.5 - 1) < 1e-6
    assert torch.isnan(y[1]).all() and torch.isnan(y[2]).all() and torch.isfinite(y[3]).all()
    alone, _, _ = B.poetx_layernorm_forward(dev(x[3:]), None, None, 1e-5)
    assert torch.equal(y[3:], alone)
    e = torch.empty(0, d, dtype=BF16, device="cuda")
    s = torch.empty(0, device="cuda")
    got = B.poetx_layernorm_backward(e, e, None, s, s)
    assert got["dx"].shape == (0, d) and not got["dgamma"].any() and not got["dbeta"].any()
    assert B.poetx_layernorm_forward(e)[0].shape == (0, d)


# ------------------------------------------------------------------------ dense linear ----

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def act_ref(p, act):
    """(value, slope) in float64."""
    if act == "none":
        return p, torch.ones_like(p)
    q = p.clone().requires_grad_(True)
    f = {"relu": torch.relu, "gelu": torch.nn.functional.gelu, "silu": torch.nn.functional.silu,
         "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh")}[act]
    v = f(q)
    s, = torch.autograd.grad(v.sum(), q)
    return v.detach(), s


def linear_case(seed, n, i, o, dtype):
    x, w = rand(seed, n, i, dtype=dtype), rand(seed + 1, o, i, dtype=dtype, scale=i ** -0.5)
    return x, w


def check_linear_fwd(B, n, i, o, dtype, act, bias, residual, save_pre, seed=20):
    x, w = linear_case(seed, n, i, o, dtype)
    b = rand(seed + 2, o, dtype=bias, scale=0.5) if bias else None
    res = rand(seed + 3, n, o, dtype=dtype) if residual else None
    y, pre = B.poetx_linear_forward(dev(x), dev(w), dev(b), dev(res), act, save_pre=save_pre)
    p = x.double() @ w.double().t()
    mag = x.double().abs() @ w.double().abs().t()
    if b is not None:
        p, mag = p + b.double(), mag + b.double().abs()
    e_p = acc(i) * mag
    v, _ = act_ref(p, act)
    ref = v if res is None else v + res.double()
    # |act'| <= 1.13 for every activation here
    e = 1.13 * e_p + FN * (p.abs() + v.abs()) * (act not in ("none", "relu")) + 2 * U[F32] * ref.abs()
    within(y, ref, U[dtype] * ref.abs() + 1.01 * e, f"y {n} {i} {o} {act}")
    assert (pre is not None) == save_pre
    if save_pre:
        within(pre, p, U[dtype] * p.abs() + 1.01 * e_p, "pre")
    return y


def check_linear_bwd(B, n, i, o, dtype, act, seed=40):
    x, w = linear_case(seed, n, i, o, dtype)
    dy, pre = rand(seed + 2, n, o, dtype=dtype), rand(seed + 3, n, o, dtype=dtype, scale=1.5)
    got = B.poetx_linear_backward(dev(x), dev(w), dev(dy), dev(pre) if act != "none" else None, act)
    _, slope = act_ref(pre.double(), act)
    dp = dy.double() * slope
    # dp: the slope's own error, then its rounding as an operand
    e_dp = (FN * dy.double().abs() * (1 + pre.double().abs()) + U[F32] * dp.abs()) * (act not in ("none", "relu"))
    e_op = e_dp + (U[dtype] * dp.abs() if act != "none" else 0)
    xd, wd = x.double(), w.double()
    for name, ref, mag, e_in, k in (
            ("dx", dp @ wd, dp.abs() @ wd.abs(), e_op @ wd.abs() if act != "none" else 0, o),
            ("dw", dp.t() @ xd, dp.abs().t() @ xd.abs(), e_op.t() @ xd.abs() if act != "none" else 0, n)):
        within(got[name], ref, U[dtype] * ref.abs() + 1.02 * (acc(k) * mag + e_in), f"{name} {n} {i} {o} {act}")
        if ref.numel() > 4096:
            # independent roundings of the operands and of the result, each at most u and
            # u / sqrt(3) in the mean square: sqrt(2 / 3) u together, below u
            assert off(got[name], ref) <= U[dtype] + acc(k), name
    within(got["dbias"], dp.sum(0), acc(n) * dp.abs().sum(0) + (e_dp.sum(0) if act != "none" else 0), "dbias")
    return got


LIN_SHAPES = [(1, 64, 64), (1, 1, 1), (2, 9, 5), (3, 7, 130), (1, 5120, 600), (16, 100, 33), (16, 4097, 48),
              (15, 2048, 17000), (17, 64, 128), (64, 513, 777), (130, 257, 300), (300, 1000, 2040), (257, 4096, 512),
              (2048, 256, 256), (40, 5000, 96)]


@pytest.mark.parametrize("n,i,o", LIN_SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_linear_forward(B, n, i, o, dtype):
    for k, act in enumerate(ACTS):
        check_linear_fwd(B, n, i, o, dtype, act, (None, F32, BF16)[k % 3], k % 2 == 1, k % 2 == 0, seed=20 + 10 * k)


@pytest.mark.parametrize("n,i,o", LIN_SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_linear_backward(B, n, i, o, dtype):
    for k, act in enumerate(ACTS[:1] + ACTS[2:] if n * i * o > 1 << 24 else ACTS):
        check_linear_bwd(B, n, i, o, dtype, act, seed=40 + 10 * k)


@pytest.mark.parametrize("n,i,o", [(4096, 200, 3584), (3500, 3400, 203), (3841, 129, 3329)])
def test_linear_many_tiles(B, n, i, o):
    """Enough 256 x 256 tiles for the large-tile kernels, with tails on every axis."""
    check_linear_fwd(B, n, i, o, BF16, "gelu", F32, True, True)
    check_linear_bwd(B, n, i, o, BF16, "silu")


@pytest.mark.parametrize("n,i,o", [(4100, 4097, 4352), (2100, 8300, 8448)])
def test_linear_shared_last_round(B, n, i, o):
    """More tiles than CUs by a few: the tiles of the last round share their k."""
    x = (torch.randn(n, i, generator=torch.Generator("cuda").manual_seed(1), device="cuda")).to(BF16)
    w = (torch.randn(o, i, generator=torch.Generator("cuda").manual_seed(2), device="cuda") * i ** -0.5).to(BF16)
    dy = torch.randn(n, o, generator=torch.Generator("cuda").manual_seed(3), device="cuda").to(BF16)
    y, pre = B.poetx_linear_forward(x, w, act="gelu", save_pre=True)
    p = x.double() @ w.double().t()
    # roundings of the results alone: at most u(bf16) each, u / sqrt(3) in the mean square
    assert off(pre, p.cpu()) <= U[BF16] and off(y, torch.nn.functional.gelu(p).cpu()) <= U[BF16]
    within(pre[-3:], p[-3:].cpu(), U[BF16] * p[-3:].abs().cpu() + acc(i) * (x[-3:].double().abs() @ w.double().abs().t()).cpu(),
           "last rows")
    g = B.poetx_linear_backward(x, w, dy)
    assert off(g["dx"], (dy.double() @ w.double()).cpu()) <= U[BF16]
    assert off(g["dw"], (dy.double().t().contiguous() @ x.double()).cpu()) <= U[BF16]


@pytest.mark.parametrize("n,i,o", [(203, 1100, 12300), (64, 1288, 12301)])
def test_linear_wide_weight_gradient(B, n, i, o):
    """Weight gradients with many rows, whose product takes a transposed copy of x."""
    check_linear_bwd(B, n, i, o, BF16, "gelu")
    check_linear_bwd(B, n, i, o, BF16, "none")


def test_linear_outputs_not_wanted_and_no_tokens(B):
    x, w = linear_case(60, 50, 72, 40, BF16)
    dy = rand(62, 50, 40, dtype=BF16)
    full = B.poetx_linear_backward(dev(x), dev(w), dev(dy))
    a = B.poetx_linear_backward(None, dev(w), dev(dy), want_dw=False, want_dbias=False)
    b = B.poetx_linear_backward(dev(x), None, dev(dy), want_dx=False)
    assert set(a) == {"dx"} and torch.equal(a["dx"], full["dx"])
    assert set(b) == {"dw", "dbias"} and torch.equal(b["dw"], full["dw"]) and torch.equal(b["dbias"], full["dbias"])
    e = torch.empty(0, 72, dtype=BF16, device="cuda")
    g = B.poetx_linear_backward(e, dev(w), torch.empty(0, 40, dtype=BF16, device="cuda"))
    assert not g["dw"].any() and not g["dbias"].any() and g["dx"].shape == (0, 72)
    assert B.poetx_linear_forward(e, dev(w))[0].shape == (0, 40)


@pytest.mark.parametrize("n", [3, 70])
def test_linear_nan_stays_in_its_row(B, n):
    """A NaN or an infinity in one token reaches that token's results only; widths that are
    padded inside and rows past the last one do not spread it."""
    x, w = linear_case(70, n, 77, 50, BF16)
    clean, _ = B.poetx_linear_forward(dev(x), dev(w), act="silu")
    x[1, 76] = float("nan")
    x[2, 0] = float("inf")
    y, _ = B.poetx_linear_forward(dev(x), dev(w), act="silu")
    assert torch.isnan(y[1]).all() and not torch.isfinite(y[2]).all()
    keep = [r for r in range(n) if r not in (1, 2)]
    assert torch.equal(y[keep], clean[keep])


def test_linear_leading_axes_and_strides(B):
    x, w = linear_case(80, 24, 64, 32, BF16)
    y3, _ = B.poetx_linear_forward(dev(x).view(2, 3, 4, 64), dev(w))
    y, _ = B.poetx_linear_forward(dev(x), dev(w))
    assert y3.shape == (2, 3, 4, 32) and torch.equal(y3.reshape(24, 32), y)
    with pytest.raises(ValueError):
        B.poetx_linear_forward(dev(x).t().contiguous().t(), dev(w))
    with pytest.raises(ValueError):  # a 2-byte offset breaks the 16-byte alignment
        B.poetx_linear_forward(torch.zeros(65, dtype=BF16, device="cuda")[1:].view(1, 64), dev(w))


# ------------------------------------------------------------------------ cross entropy ----

def xent_case(seed, n, d, v, dtype, ignored=0.2):
    h = rand(seed, n, d, dtype=dtype)
    w = rand(seed + 1, v, d, dtype=dtype, scale=2 * d ** -0.5)
    g = torch.Generator().manual_seed(seed + 2)
    t = torch.randint(0, v, (n,), generator=g, dtype=torch.int32)
    drop = torch.rand(n, generator=g) < ignored
    t[drop] = torch.where(torch.arange(n)[drop] % 2 == 0, -1, v).int()
    dl = torch.rand(n, generator=g) + 0.5
    return h, w, t, dl


def check_xent(B, n, d, v, dtype, ignored=0.2, seed=100):
    h, w, t, dl = xent_case(seed, n, d, v, dtype, ignored)
    loss, lse = B.poetx_xent_forward(dev(h), dev(w), dev(t))
    hd, wd, on = h.double(), w.double(), (t >= 0) & (t < v)
    logits = hd @ wd.t()
    e_l = acc(d) * (hd.abs() @ wd.abs().t()).amax(1)          # worst logit of a row
    z = torch.logsumexp(logits, 1)
    # the sum: a chain of at most v / 16 + 64 additions, exp off by 2^-22 and by its
    # argument's rounding (2^-23 of up to 2 max |l|)
    arg = 2 * logits.abs().amax(1) + 1
    e_z = e_l + (v / 16 + 64) * 2.0 ** -24 + 2.0 ** -22 + arg * 2.0 ** -22 + 4 * U[F32] * z.abs()
    within(lse, z, e_z, "lse")
    at = t.long().clamp(0, v - 1)[:, None]
    lt = logits.gather(1, at)[:, 0]
    ref = torch.where(on, z - lt, torch.zeros_like(z))
    within(loss, ref, torch.where(on, e_z + e_l + 4 * U[F32] * (z.abs() + lt.abs()), torch.zeros_like(z)), "loss")

    got = B.poetx_xent_backward(dev(h), dev(w), dev(t), lse, dev(dl))
    p = torch.exp(logits - z[:, None])
    one = torch.zeros_like(p).scatter_(1, at, 1.0)
    g = torch.where(on, dl.double(), torch.zeros_like(z))[:, None]
    dlog = (p - one) * g
    e_p = p * (e_l + e_z + arg * 2.0 ** -22 + 2.0 ** -21)[:, None]
    e_d = (e_p + 2 * U[F32] * (p + one)) * g + U[dtype] * dlog.abs()
    for name, r, mag, e, k in (("dh", dlog @ wd, dlog.abs() @ wd.abs(), e_d @ wd.abs(), v),
                               ("dw", dlog.t() @ hd, dlog.abs().t() @ hd.abs(), e_d.t() @ hd.abs(), n)):
        within(got[name], r, U[dtype] * r.abs() + 1.02 * (acc(k) * mag + e), f"{name} {n} {d} {v}")
        if r.numel() > 4096 and on.any():
            assert off(got[name], r) <= U[dtype] + acc(k) + 2.0 ** -18, name
    assert not got["dh"].cpu()[~on].any()


XENT_SHAPES = [(1, 64, 1000), (1, 1, 1), (3, 5, 2), (8, 4096, 3001), (16, 77, 20001), (15, 520, 128), (17, 64, 257),
               (64, 100, 5003), (301, 520, 1007), (130, 1000, 2049), (1025, 256, 4104), (28, 3330, 1301),
              (70, 2500, 513), (19, 5000, 7)]


@pytest.mark.parametrize("n,d,v", XENT_SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_xent(B, n, d, v, dtype):
    check_xent(B, n, d, v, dtype)


def test_xent_large_tiles(B):
    check_xent(B, 3400, 136, 3333, BF16)
    check_xent(B, 131, 1004, 12500, BF16)  # dW by way of a transposed copy of h


def test_xent_mean_keeps_its_digits(B):
    """The rows of a mean share one dloss, and their dl at the target is nearly -dloss for all of
    them: its rounding to bf16 must not become one common error of the gradients.  The dloss
    here would be off by 0.98 u(bf16), u = 2^-8.  Independent roundings of dl and of the results
    are 0.43 u each in the mean square (u / 2^e(x) / sqrt(3) over a uniform log x), 0.61 u
    together."""
    n, d, v = 700, 256, 6000
    h, w, t, _ = xent_case(160, n, d, v, BF16)
    dl = torch.full((n,), 2.0 ** -12 * (1 + 0.98 * 2.0 ** -8))
    loss, lse = B.poetx_xent_forward(dev(h), dev(w), dev(t))
    g = B.poetx_xent_backward(dev(h), dev(w), dev(t), lse, dev(dl))
    on = (t >= 0) & (t < v)
    p = torch.softmax(h.double() @ w.double().t(), 1)
    p[torch.arange(n), t.long().clamp(0, v - 1)] -= 1
    p = p * torch.where(on, dl.double(), torch.zeros(n, dtype=torch.float64))[:, None]
    assert off(g["dh"], p @ w.double()) <= 0.7 * U[BF16]
    assert off(g["dw"], p.t() @ h.double()) <= 0.7 * U[BF16]


def test_xent_every_row_masked_and_no_rows(B):
    h, w, t, dl = xent_case(130, 40, 64, 500, BF16)
    t[:] = -1
    loss, lse = B.poetx_xent_forward(dev(h), dev(w), dev(t))
    assert not loss.any() and torch.isfinite(lse).all()
    g = B.poetx_xent_backward(dev(h), dev(w), dev(t), lse, dev(dl))
    assert not g["dh"].any() and not g["dw"].any()
    e = torch.empty(0, 64, dtype=BF16, device="cuda")
    s, ti = torch.empty(0, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    assert B.poetx_xent_forward(e, dev(w), ti)[0].shape == (0,)
    assert not B.poetx_xent_backward(e, dev(w), ti, s, s)["dw"].any()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [12, 60])
def test_xent_masked_rows_hold_anything(B, n, dtype):
    """Infinities and NaN in the h, lse and dloss of tokens that take no part change nothing
    of the other tokens' losses and gradients."""
    h, w, t, dl = xent_case(140, n, 72, 700, dtype, ignored=0.0)
    t[[2, 5]] = -100
    a, lse = B.poetx_xent_forward(dev(h), dev(w), dev(t))
    ga = B.poetx_xent_backward(dev(h), dev(w), dev(t), lse, dev(dl))
    h2, dl2 = h.clone(), dl.clone()
    h2[2], h2[5, 3], dl2[2], dl2[5] = float("nan"), float("inf"), float("nan"), float("inf")
    b, lse2 = B.poetx_xent_forward(dev(h2), dev(w), dev(t))
    gb = B.poetx_xent_backward(dev(h2), dev(w), dev(t), lse2, dev(dl2))
    assert torch.equal(a, b) and torch.equal(ga["dh"], gb["dh"]) and torch.equal(ga["dw"], gb["dw"])


def test_xent_extreme_logits(B):
    """Logits of hundreds, one far above the rest: no overflow, the loss stays exact."""
    n, d, v = 20, 64, 300
    h = torch.zeros(n, d, dtype=BF16)
    w = torch.zeros(v, d, dtype=BF16)
    h[:, 0] = 16.0
    w[:, 0] = torch.linspace(-40, 40, v).to(BF16)
    t = torch.arange(n, dtype=torch.int32)
    loss, lse = B.poetx_xent_forward(dev(h), dev(w), dev(t))
    logits = h.double() @ w.double().t()
    z = torch.logsumexp(logits, 1)
    # products and their sum are exact here; exp's argument error is 2^-23 of 1280 and only
    # terms near the maximum count
    within(lse, z, z.abs() * 2.0 ** -23 + 2.0 ** -18, "lse")
    ref = z - logits.gather(1, t.long()[:, None])[:, 0]
    within(loss, ref, ref.abs() * 2.0 ** -22 + 2.0 ** -18, "loss")


def test_xent_pieces(B):
    """A vocabulary of several pieces (dl of one piece is held to 512 MB): the results of the
    tokens' first rows agree with a call of few tokens, which needs one piece."""
    n, d, v = 40000, 64, 20000
    g = torch.Generator(device="cuda").manual_seed(5)
    h = torch.randn(n, d, generator=g, device="cuda").to(BF16)
    w = (torch.randn(v, d, generator=g, device="cuda") * 0.25).to(BF16)
    t = torch.randint(0, v, (n,), generator=g, device="cuda", dtype=torch.int32)
    dl = torch.full((n,), 1.0, device="cuda")
    loss, lse = B.poetx_xent_forward(h, w, t)
    full = B.poetx_xent_backward(h, w, t, lse, dl)
    k = 300
    part = B.poetx_xent_backward(h[:k].contiguous(), w, t[:k].contiguous(), lse[:k].contiguous(), dl[:k].contiguous())
    hd, wd = h[:k].double().cpu(), w.double().cpu()
    p = torch.exp(hd @ wd.t() - lse[:k, None].double().cpu())
    p[torch.arange(k), t[:k].long().cpu()] -= 1
    ref = p @ wd
    assert off(full["dh"][:k], ref) <= 2.0 ** -8 and off(part["dh"], ref) <= 2.0 ** -8
    # dw over all tokens, in pieces of tokens, against float64 on the device
    dw = torch.zeros(v, d, dtype=torch.float64, device="cuda")
    for s in range(0, n, 4000):
        q = torch.exp(h[s:s + 4000].double() @ w.double().t() - lse[s:s + 4000, None].double())
        q[torch.arange(q.shape[0], device="cuda"), t[s:s + 4000].long()] -= 1
        dw += q.t().contiguous() @ h[s:s + 4000].double()
    assert off(full["dw"], dw.cpu()) <= 2.0 ** -8


# ------------------------------------------------------------------------ how they run ----

def run_all(B, x, w, bias, head, t, dl):
    """Every operator once, chained; a flat list of results."""
    y, mean, rstd = B.poetx_layernorm_forward(x, bias[:x.shape[1]], None)
    u, pre = B.poetx_linear_forward(y, w, bias, None, "gelu", save_pre=True)
    loss, lse = B.poetx_xent_forward(u, head, t)
    g = B.poetx_xent_backward(u, head, t, lse, dl)
    lb = B.poetx_linear_backward(y, w, g["dh"], pre, "gelu")
    nb = B.poetx_layernorm_backward(x, lb["dx"], bias[:x.shape[1]], mean, rstd)
    return [y, mean, rstd, u, pre, loss, lse, g["dh"], g["dw"], lb["dx"], lb["dw"], lb["dbias"], nb["dx"],
            nb["dgamma"], nb["dbeta"]]


def chain_inputs(seed, n, dtype, d=200, o=264, v=3001):
    h, head, t, dl = xent_case(seed, n, o, v, dtype)
    return [dev(a) for a in (rand(seed + 5, n, d, dtype=dtype), rand(seed + 6, o, d, dtype=dtype, scale=d ** -0.5),
                             rand(seed + 7, o), head, t, dl)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [9, 333])
def test_repeated_calls_are_bitwise_equal(B, n, dtype):
    a = chain_inputs(200, n, dtype)
    first = [r.clone() for r in run_all(B, *a)]
    other = chain_inputs(900, n + 3, dtype)
    run_all(B, *other)
    for p, q in zip(first, run_all(B, *a)):
        assert torch.equal(p, q)


@pytest.mark.parametrize("n", [9, 333])
def test_on_another_stream(B, n):
    a = chain_inputs(210, n, BF16)
    want = run_all(B, *a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run_all(B, *a)
    s.synchronize()
    for p, q in zip(want, got):
        assert torch.equal(p, q)


@pytest.mark.parametrize("n", [9, 333])
def test_captured_and_replayed(B, n):
    """Two captured graphs of the whole chain, replayed in turns with eager calls of other
    sizes between: every replay equals the eager result on the inputs of that moment."""
    sets = [chain_inputs(220, n, BF16), chain_inputs(230, n, BF16)]
    graphs = []
    for a in sets:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            run_all(B, *a)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run_all(B, *a)
        graphs.append((g, out))
    big = chain_inputs(240, 2 * n + 50, BF16, v=9001)
    for rep in range(4):
        for (g, out), a in zip(graphs, sets):
            a[0].copy_(dev(rand(250 + rep, *a[0].shape, dtype=BF16)))
            g.replay()
            torch.cuda.synchronize()
            got = [r.clone() for r in out]
            run_all(B, *big)
            for p, q in zip(run_all(B, *a), got):
                assert torch.equal(p, q), rep


def test_two_threads_on_one_stream(B):
    """Calls of two threads whose kernels interleave on one stream keep their own workspaces."""
    import threading
    sets = [chain_inputs(260, 333, BF16), chain_inputs(270, 210, BF16, v=5003)]
    want = [[r.clone() for r in run_all(B, *a)] for a in sets]
    bad = []

    def work(k):
        for _ in range(25):
            got = run_all(B, *sets[k])
            torch.cuda.current_stream().synchronize()
            if not all(torch.equal(p, q) for p, q in zip(want[k], got)):
                bad.append(k)

    ts = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not bad


def test_xent_wide_pieces(B):
    """Few tokens over more than 2^20 vocabulary entries: pieces of 2^20."""
    check_xent(B, 18, 16, (1 << 20) + 777, BF16, seed=280)


def test_block_step(B):
    """The operators with the POET-X layer between them, as a training step: loss and every
    gradient against float64 (autograd through the definitions, the layer's G from the oracle)."""
    from oracle import poetx_oracle as O
    from orthogonal_reparameterized_amd import workloads as WL
    from orthogonal_reparameterized_amd.step import BlockStep, LayerStep
    d, f, v, n, b = 256, 640, 1003, 96, 64
    wl = WL.Workload(98, "block", n, d, d, b, "f32", "f32", "f32", 0.02, d)
    inp = WL.make_layer_inputs(wl)
    layer = LayerStep(wl, inp, "fast")
    p = {"gamma1": 1 + rand(1, d, scale=0.2), "beta1": rand(2, d, scale=0.2), "w1": rand(3, f, d, scale=d ** -0.5),
         "b1": rand(4, f, scale=0.2), "w2": rand(5, d, f, scale=f ** -0.5), "b2": rand(6, d, scale=0.2),
         "gamma2": 1 + rand(7, d, scale=0.2), "beta2": rand(8, d, scale=0.2), "head": rand(9, v, d, scale=d ** -0.5)}
    x0, t = rand(10, n, d), torch.randint(0, v, (n,), generator=torch.Generator().manual_seed(3), dtype=torch.int32)
    t[::7] = -1
    on = t >= 0
    dl = on.float() / on.sum()
    step = BlockStep(layer, {k: dev(q) for k, q in p.items()}, act="gelu")
    loss, got = step.step(dev(x0), dev(t), dev(dl))

    import torch.nn.functional as F
    P = {k: q.double().requires_grad_(True) for k, q in p.items()}
    X = x0.double().requires_grad_(True)
    G, th = [], []
    for side in ("theta_r", "theta_p"):
        th.append(torch.from_numpy(inp[side].astype(np.float64)).requires_grad_(True))
        iu = torch.triu_indices(b, b, 1)
        Q = torch.zeros(th[-1].shape[0], b, b, dtype=torch.float64)
        Q = Q.index_put((torch.arange(Q.shape[0])[:, None], iu[0][None], iu[1][None]), th[-1])
        Q = Q - Q.transpose(1, 2)
        Q2 = Q @ Q
        G.append(torch.eye(b, dtype=torch.float64) + 2 * (Q + Q2 + Q2 @ Q) + Q2 @ Q2)
        np.testing.assert_allclose(G[-1].detach().numpy(), O.cnp_forward(inp[side].astype(np.float64), b), rtol=0,
                                   atol=1e-12)
    W = torch.from_numpy(inp["w"].astype(np.float64))
    pin, pout = (torch.from_numpy(inp[k].astype(np.int64)) for k in ("perm_in", "perm_out"))
    wm = W[pout][:, pin]
    a = F.layer_norm(X, (d,), P["gamma1"], P["beta1"], 1e-5)
    blocks = lambda m, g: torch.cat([m[:, j * b:(j + 1) * b] @ g[j] for j in range(d // b)], 1)  # noqa: E731
    zt = blocks(blocks(a[:, pin], G[0]) @ wm.t(), G[1])
    z = torch.zeros_like(zt).index_copy(1, pout, zt)
    y = F.linear(F.gelu(F.linear(z, P["w1"], P["b1"])), P["w2"], P["b2"]) + X
    h = F.layer_norm(y, (d,), P["gamma2"], P["beta2"], 1e-5)
    ref = F.cross_entropy(F.linear(h, P["head"]), t.long(), ignore_index=-1, reduction="none")
    leaves = dict(P, theta_r=th[0], theta_p=th[1], x0=X)
    grads = torch.autograd.grad((ref * dl.double()).sum(), list(leaves.values()))
    # float32 throughout: eight stages, each off by about sqrt(K) 2^-24 (K <= 1003 terms of
    # independent rounding) with condition numbers of a few: 8 * 32 * 2^-24 * 4 = 6e-5
    assert off(loss, ref.detach()) <= 6e-5
    for (k, _), r in zip(leaves.items(), grads):
        assert off(got[k].reshape(r.shape), r) <= 6e-5, k


def test_gradients_against_differences(B):
    """dL of small float32 steps along random directions against the gradients' projections."""
    n, d, o, v = 24, 48, 40, 101
    x, w, bias, head, t, dl = chain_inputs(300, n, F32, d=d, o=48, v=v)

    def loss_of(x_, w_, head_):
        y, _, _ = B.poetx_layernorm_forward(x_)
        u, _ = B.poetx_linear_forward(y, w_, bias, None, "gelu_tanh")
        return float((B.poetx_xent_forward(u, head_, t)[0].double() * dl.double()).sum())

    y, mean, rstd = B.poetx_layernorm_forward(x)
    u, pre = B.poetx_linear_forward(y, w, bias, None, "gelu_tanh", save_pre=True)
    _, lse = B.poetx_xent_forward(u, head, t)
    g = B.poetx_xent_backward(u, head, t, lse, dl)
    lb = B.poetx_linear_backward(y, w, g["dh"], pre, "gelu_tanh")
    nb = B.poetx_layernorm_backward(x, lb["dx"], None, mean, rstd)
    total = loss_of(x, w, head)
    for k, grad in enumerate((nb["dx"], lb["dw"], g["dw"])):
        # along the gradient itself: no cancellation in the projection
        direc = grad / grad.norm()
        eps = 2.0 ** -7
        lo, hi = ([[x, w, head][j] + (s * eps * direc if j == k else 0) for j in range(3)] for s in (-1, 1))
        diff = (loss_of(*hi) - loss_of(*lo)) / (2 * eps)
        want = float((grad.double() * direc.double()).sum())
        # loss_of is off by about 2^-22 of the total (24 float32 losses): 2^-22 total / eps; the
        # third derivative's term is eps^2 / 6 of order the gradient's own scale
        assert abs(diff - want) <= 2.0 ** -22 * abs(total) / eps + 50 * eps ** 2 * abs(want) / 6, (k, diff, want)


def test_linear_relu_slope_of_nan(B):
    """A NaN that went into relu comes out of its slope; infinities of dy at a slope of 0 are
    NaN as in the formula's product, and nothing spreads to other tokens."""
    x, w = linear_case(310, 4, 16, 24, BF16)
    dy, pre = rand(312, 4, 24, dtype=BF16), rand(313, 4, 24, dtype=BF16)
    pre[1, 3], pre[2, 5], dy[2, 5] = float("nan"), -1.0, float("inf")
    got = B.poetx_linear_backward(dev(x), dev(w), dev(dy), dev(pre), "relu")
    assert torch.isnan(got["dx"][1:3]).all() and torch.isfinite(got["dx"][[0, 3]]).all()
    assert sorted(torch.nonzero(torch.isnan(got["dbias"]))[:, 0].tolist()) == [3, 5]


def test_more_than_2_31_elements(B):
    """Results and operands whose offsets pass 32 bits: the last rows are right."""
    n, i, o = 33000, 8, 65600
    g = torch.Generator(device="cuda").manual_seed(320)
    x = torch.randn(n, i, generator=g, device="cuda").to(BF16)
    w = torch.randn(o, i, generator=g, device="cuda").to(BF16)
    y, _ = B.poetx_linear_forward(x, w)
    assert y.numel() > 1 << 31
    xd, wd = x.double(), w.double()
    ref, mag = xd[-3:] @ wd.t(), xd[-3:].abs() @ wd.abs().t()
    within(y[-3:], ref.cpu(), (U[BF16] * ref.abs() + 1.01 * acc(i) * mag).cpu(), "y")
    got = B.poetx_linear_backward(x, w, y)
    r, c = y[-3:].double(), y[:, -3:].double()
    for name, at, ref, mag, k in (("dx", got["dx"][-3:], r @ wd, r.abs() @ wd.abs(), o),
                                  ("dw", got["dw"][-3:], c.t() @ xd, c.abs().t() @ xd.abs(), n)):
        within(at, ref.cpu(), (U[BF16] * ref.abs() + 1.02 * acc(k) * mag).cpu(), name)
    within(got["dbias"][-3:], c.sum(0).cpu(), (acc(n) * c.abs().sum(0)).cpu(), "dbias")
    del got, y
    n, d = 140000, 16384
    x = torch.randn(n, d, generator=g, device="cuda", dtype=BF16)
    y, mean, rstd = B.poetx_layernorm_forward(x)
    dx = B.poetx_layernorm_backward(x, y, None, mean, rstd, want_params=False)["dx"]
    tail = x[-3:].clone()
    y3, mean3, rstd3 = B.poetx_layernorm_forward(tail)
    assert torch.equal(y[-3:], y3) and torch.equal(mean[-3:], mean3) and torch.equal(rstd[-3:], rstd3)
    assert torch.equal(dx[-3:], B.poetx_layernorm_backward(tail, y3, None, mean3, rstd3)["dx"])


@pytest.mark.parametrize("n,d,v", [(16, 1029, 8200), (5, 600, 50000), (2, 3333, 40), (1, 40, 8192)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_xent_few_tokens(B, n, d, v, dtype):
    """Few tokens over vocabularies of each way to share a group's k, with tails of k that end
    inside a turn of the waves."""
    check_xent(B, n, d, v, dtype, seed=330)


@pytest.mark.parametrize("n,d", [(600, 5121), (530, 6144), (270, 6150), (300, 12288), (280, 12289), (3, 15000)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_layernorm_wide_rows(B, n, d, dtype):
    """Each way to spread a wide row over threads, with more rows than workgroups."""
    test_layernorm(B, n, d, dtype, F32)


@pytest.mark.parametrize("n,i,o", [(1500, 4700, 5300), (7001, 2200, 2000), (600, 7001, 6008)])
def test_linear_large_tiles_over_ranges_of_k(B, n, i, o):
    """Products whose 256 x 256 tiles are split over k, and ones with tiles for half the GPU."""
    test_linear_shared_last_round(B, n, i, o)


def test_xent_large_tiles_over_ranges_of_k(B):
    check_xent(B, 1300, 4700, 4400, BF16, seed=340)


def test_wide_weight_gradients_of_more_tokens(B):
    """Weight gradients by way of a transposed copy, with a tail of the tokens."""
    check_linear_bwd(B, 413, 1100, 12300, BF16, "silu")
    check_xent(B, 421, 1004, 12500, BF16, seed=350)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_as_many_tokens_as_there_are_tiles_for(B, dtype):
    """2^21 + 1 tiles of 128 tokens with one result each: in float32 twice as many tiles of 64."""
    n, d = (1 << 28) + 1, 20
    x = torch.zeros(n, d, dtype=dtype, device="cuda")
    x[:, 3] = torch.arange(n, device="cuda", dtype=torch.int32).remainder_(251).to(dtype)
    w = torch.zeros(1, d, dtype=dtype, device="cuda")
    w[0, 3] = 2.0
    y, _ = B.poetx_linear_forward(x, w)
    assert torch.equal(y[:, 0], x[:, 3] * 2)  # exact in both types
    dx = B.poetx_linear_backward(None, w, y, want_dw=False, want_dbias=False)["dx"]
    assert torch.equal(dx[:, 3], y[:, 0] * 2) and not dx[:, 4].any()


def act_errors(p, act, dtype):
    """Bounds of an activation's and its slope's own errors at p (float64), from their steps.
    float32: the library's functions (exp and erfc to 4 units of 2^-24 and 8), divisions to 5, the
    rest one 2^-24 per operation.  bf16: hardware exp2 and reciprocal (2 units of 2^-24 each, exp's
    argument times log2 e another 1.5 2^-24 of it) and a polynomial to 2^-19."""
    e = 2.0 ** -24
    fast = dtype == BF16
    one = torch.ones_like(p)
    if act == "gelu":
        cdf, pdf = torch.special.erfc(-p * 0.5 ** 0.5) / 2, torch.exp(-p * p / 2) / (2 * np.pi) ** 0.5
        # the argument's rounding counts p^2 + 1 fold in erfc, p^2 / 2 fold in exp(-p^2 / 2)
        d_cdf = 2.0 ** -19 + 8 * e + 1.25 * e * p * p if fast else e * (1.5 * (p * p + 1) + 9)
        d_pdf = e * (1.25 * p * p + 7) if fast else e * (p * p / 2 + 7)
        slope = cdf * (d_cdf + e) + p.abs() * pdf * (d_pdf + 2 * e)
        return (p * cdf).abs() * (d_cdf + e), slope
    if act == "silu":
        u, du = p, one
        d = e * (1.5 * p.abs() * fast + 11)
    else:
        c = (2 / np.pi) ** 0.5
        u, du = 2 * c * (p + 0.044715 * p ** 3), 2 * c * (1 + 3 * 0.044715 * p * p)
        d = e * ((7 + 1.5 * fast) * u.abs() + 11)
    g = torch.sigmoid(u)
    rest = (1 - g) * d + g * d + e  # of 1 - g, which is a difference, and of its factor g
    return (p * g).abs() * (d + e), g * d + 2 * e * g + p.abs() * du * g * (rest + 8 * e * (1 - g))


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_activations_keep_their_digits(B, act, dtype):
    """Values and slopes of the activations alone, element by element, far into the negative
    tail: weights of 1 make p the input itself.  (f32: errors relative to the value, not to p.)"""
    p = torch.linspace(-11, 11, 5001, dtype=torch.float64).to(dtype)[:, None].contiguous()
    w = torch.ones(1, 1, dtype=dtype)
    pd = p.double()
    v, slope = act_ref(pd, act)
    if act == "gelu":  # 1 + erf and 1 + tanh cancel in the tail, even in 64 bits
        cdf = torch.special.erfc(-pd * 0.5 ** 0.5) / 2
        v, slope = pd * cdf, cdf + pd * torch.exp(-pd * pd / 2) / (2 * np.pi) ** 0.5
    if act == "gelu_tanh":
        c = (2 / np.pi) ** 0.5
        g, less = (torch.sigmoid(s * 2 * c * (pd + 0.044715 * pd ** 3)) for s in (1, -1))
        v, slope = pd * g, g + pd * g * less * 2 * c * (1 + 3 * 0.044715 * pd * pd)
    e_v, e_s = act_errors(pd, act, dtype)
    for rows in (slice(None), slice(0, 16), slice(700, 716)):
        y, _ = B.poetx_linear_forward(dev(p[rows]), dev(w), act=act)
        within(y, v[rows], U[dtype] * v[rows].abs() + 1.01 * e_v[rows], f"{act} {rows}")
    one = torch.ones_like(p)
    got = B.poetx_linear_backward(dev(p), dev(w), dev(one), dev(p), act, want_dw=False)
    within(got["dx"], slope, U[dtype] * slope.abs() + 1.01 * e_s, f"slope of {act}")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_xent_of_more_than_2_28_tokens(B, dtype):
    """More tokens than a grid has workgroups of 16 for: losses and dh of a batch that repeats
    753 rows."""
    n, d, v, period = 753 * 356500, 4, 3, 753
    assert n > 1 << 28
    h, w = rand(360, period, d, dtype=dtype), rand(361, v, d, dtype=dtype)
    t = torch.arange(period, dtype=torch.int32) % 4 - 1  # -1: takes no part
    logits = h.double() @ w.double().t()
    z = torch.logsumexp(logits, 1)
    on = t >= 0
    at = t.long().clamp(0)[:, None]
    ref = torch.where(on, z - logits.gather(1, at)[:, 0], torch.zeros_like(z))
    dl = (torch.exp(logits - z[:, None]) - torch.zeros_like(logits).scatter_(1, at, 1.0)) * on[:, None]
    dh = dl @ w.double()
    big, ts = dev(h).repeat(n // period, 1), dev(t).repeat(n // period)
    loss, lse = B.poetx_xent_forward(big, dev(w), ts)
    # as in check_xent: the products, exp with its argument's rounding, the sum of three, log
    arg = 2 * float(logits.abs().amax()) + 1
    e_l = acc(d) * float((h.double().abs() @ w.double().abs().t()).amax())
    e_z = e_l + 4 * 2.0 ** -24 + 2.0 ** -22 + arg * 2.0 ** -22 + 4 * U[F32] * arg
    for got, want, e in ((loss, ref, e_z + e_l + 8 * U[F32] * arg), (lse, z, e_z)):
        assert float((got.view(-1, period) - dev(want).float()).abs().amax()) <= e + U[F32] * arg
    g = B.poetx_xent_backward(big, dev(w), ts, lse, torch.ones(n, device="cuda"), want_dw=False)["dh"]
    # dl and dh rounded to the type, and the sum over the vocabulary
    e_p = e_l + e_z + arg * 2.0 ** -22 + 2.0 ** -21
    mag = dl.abs() @ w.double().abs()
    tol = dev((2.02 * U[dtype] + acc(v)) * mag + e_p * w.double().abs().sum(0)).float()
    for k in range(0, n // period, 1 << 16):
        rows = g[k * period:(k + (1 << 16)) * period].float().view(-1, period, d)
        assert bool(((rows - dev(dh).float()).abs() <= tol).all()), k


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,d,v", [(12, 72, 700), (60, 77, 700), (3000, 392, 1200), (3300, 4100, 520)])
def test_xent_masked_rows_are_zero_whatever_w_holds(B, n, d, v, dtype):
    """A row of W that is not finite reaches the tokens that take part, not the others' dh."""
    h, w, t, dl = xent_case(370, n, d, v, dtype)
    w[3, 5], w[v - 1, 7] = float("inf"), float("nan")
    w[4] = float("-inf")
    t[0], t[1], t[n - 1] = -1, v, 5
    on = (t >= 0) & (t < v)
    z = torch.zeros(n)  # any statistics: the masked rows do not depend on them
    g = B.poetx_xent_backward(dev(h), dev(w), dev(t), dev(z), dev(dl))["dh"].cpu()
    assert not g[~on].any()  # (a NaN would count as true)
    assert torch.isnan(g[on][:, 7]).all()


def test_xent_masked_rows_are_zero_over_pieces(B):
    """The same where dh is summed over several pieces of the vocabulary."""
    n, d, v = 40000, 64, 20000
    g = torch.Generator(device="cuda").manual_seed(380)
    h = torch.randn(n, d, generator=g, device="cuda").to(BF16)
    w = (torch.randn(v, d, generator=g, device="cuda") * 0.25).to(BF16)
    w[11] = float("inf")
    t = torch.randint(0, v, (n,), generator=g, device="cuda", dtype=torch.int32)
    t[::3] = -1
    got = B.poetx_xent_backward(h, w, t, torch.zeros(n, device="cuda"), torch.ones(n, device="cuda"), want_dw=False)
    assert not got["dh"][::3].any() and torch.isnan(got["dh"][1::3]).any()


def test_calls_that_need_no_workspace(B):
    """A requirement of 0: the call runs with any aligned ws and 0 bytes; with ws == NULL it is
    the size query and leaves the outputs alone."""
    import ctypes
    n, d = 4, 64
    x, w, dy = (dev(rand(390 + k, r, d, dtype=BF16)) for k, r in enumerate((n, d, n)))
    _, mean, rstd = B.poetx_layernorm_forward(x)
    s = torch.cuda.current_stream().cuda_stream
    y, dx, dw = torch.full_like(x, 7.0), torch.full_like(x, 7.0), torch.full_like(w, 7.0)
    ws = torch.full((64,), 5, dtype=torch.uint8, device="cuda")
    calls = [(y, B.raw.poetx_linear_forward, (n, d, d, 1, x.data_ptr(), w.data_ptr(), None, 0, None, 0, y.data_ptr(),
                                              None)),
             (dx, B.raw.poetx_layernorm_backward, (n, d, 1, x.data_ptr(), dy.data_ptr(), None, 0, mean.data_ptr(),
                                                   rstd.data_ptr(), None, dx.data_ptr(), None, None)),
             (dw, B.raw.poetx_linear_backward, (0, d, d, 1, None, None, None, None, 0, None, dw.data_ptr(), None))]
    for out, f, args in calls:
        size = ctypes.c_size_t(99)
        assert f(*args, None, ctypes.byref(size), s) == B.POETX_OK and size.value == 0
        assert bool((out == 7).all())
        assert f(*args, ws.data_ptr(), ctypes.byref(size), s) == B.POETX_OK
    assert torch.equal(y, B.poetx_linear_forward(x, w)[0]) and not dw.any() and bool((ws == 5).all())
    assert torch.equal(dx, B.poetx_layernorm_backward(x, dy, None, mean, rstd, want_params=False)["dx"])


def test_release_drops_every_threads_workspaces(B):
    """release_workspace() frees the workspaces of threads that are alive and idle, and a thread
    whose workspace went gets another."""
    import threading
    h, w, t, dl = (dev(a) for a in xent_case(400, 400, 64, 50000, BF16))
    loss, lse = B.poetx_xent_forward(h, w, t)
    want = B.poetx_xent_backward(h, w, t, lse, dl)
    need = 400 * 50000 * 2  # dl alone
    done, go, bad = threading.Event(), threading.Event(), []

    def work():
        torch.cuda.set_device(h.device)
        for _ in range(2):
            got = B.poetx_xent_backward(h, w, t, lse, dl)
            torch.cuda.synchronize()
            bad.extend(k for k in want if not torch.equal(got[k], want[k]))
            del got
            done.set()
            go.wait(60)

    B.release_workspace()
    before = torch.cuda.memory_allocated()
    th = threading.Thread(target=work)
    th.start()
    assert done.wait(60)
    held = torch.cuda.memory_allocated()
    B.release_workspace()
    after = torch.cuda.memory_allocated()
    go.set()
    th.join()
    assert held - before >= need and after <= before and not bad


def test_a_threads_workspaces_go_with_it(B):
    import gc
    import threading
    h, w, t, dl = (dev(a) for a in xent_case(410, 400, 64, 50000, BF16))
    _, lse = B.poetx_xent_forward(h, w, t)
    B.release_workspace()
    before = torch.cuda.memory_allocated()
    th = threading.Thread(target=lambda: B.poetx_xent_backward(h, w, t, lse, dl))
    th.start()
    th.join()
    gc.collect()
    assert torch.cuda.memory_allocated() <= before


def test_current_stream_lookup(B):
    """The stream handle that the calls launch on is torch's current one, by either way of asking."""
    s = torch.cuda.Stream()
    for ctx in (torch.cuda.stream(s), torch.cuda.stream(torch.cuda.default_stream())):
        with ctx:
            assert B._raw_stream(0) == torch.cuda.current_stream(0).cuda_stream


# ---------------------------------------------------------- the large tiles, element by element ----
# The launch labels say which way a product went, so that these cases cannot drift off the paths
# they are for: "_large" is the larger tile (bf16 256 x 256, float32 128 x 128), "mm_join" a k split
# of all its tiles, "mm_tail" of the last round's, "pack_rows_t" a transposed copy for dW.

def labelled(B, f):
    """(f(), the labels of the kernels it launched)."""
    torch.cuda.synchronize()
    B.prof_read()
    B.prof_enable(True)
    try:
        r = f()
        torch.cuda.synchronize()
        return r, set(B.prof_read())
    finally:
        B.prof_enable(False)


def within_dev(got, ref, tol, what):
    """`within` on the device, for results of millions of elements."""
    d = (got.double() - ref).abs()
    bad = ~(d <= tol + TINY)
    if bad.any():
        i = int(torch.nonzero(bad.reshape(-1))[0])
        pytest.fail(f"{what}: {int(bad.sum())} of {bad.numel()} off, first {i}: got {got.reshape(-1)[i].item():.9g} "
                    f"ref {ref.reshape(-1)[i].item():.9g} tol {tol.reshape(-1)[i].item():.3g}")


def drand(seed, *shape, dtype=F32, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda") * scale).to(dtype)


def check_linear_large(B, n, i, o, dtype, act, bias, fwd, bwd, seed=420):
    """Forward with bias, residual and the kept pre-activation, and backward, against float64 with
    the bounds of check_linear_fwd and check_linear_bwd; fwd, bwd: the labels they must have."""
    x, w = drand(seed, n, i, dtype=dtype), drand(seed + 1, o, i, dtype=dtype, scale=i ** -0.5)
    b, res = drand(seed + 2, o, dtype=bias, scale=0.5), drand(seed + 3, n, o, dtype=dtype)
    (y, pre), ran = labelled(B, lambda: B.poetx_linear_forward(x, w, b, res, act, save_pre=True))
    assert fwd <= ran and ran & {"mm_join", "mm_tail"} <= fwd, ran
    xd, wd = x.double(), w.double()
    p, mag = xd @ wd.t() + b.double(), xd.abs() @ wd.abs().t() + b.double().abs()
    e_p = acc(i) * mag
    within_dev(pre, p, U[dtype] * p.abs() + 1.01 * e_p, "pre")
    v, _ = act_ref(p, act)
    ref = v + res.double()
    e = 1.13 * e_p + FN * (p.abs() + v.abs()) * (act not in ("none", "relu")) + 2 * U[F32] * ref.abs()
    within_dev(y, ref, U[dtype] * ref.abs() + 1.01 * e, "y")
    del y, p, mag, e_p, v, ref, e, res

    dy = drand(seed + 4, n, o, dtype=dtype)
    got, ran = labelled(B, lambda: B.poetx_linear_backward(x, w, dy, pre, act))
    assert bwd <= ran and ran & {"mm_join", "mm_tail", "pack_rows_t"} <= bwd, ran
    _, slope = act_ref(pre.double(), act)
    dp = dy.double() * slope
    e_dp = (FN * dy.double().abs() * (1 + pre.double().abs()) + U[F32] * dp.abs()) * (act not in ("none", "relu"))
    e_op = e_dp + (U[dtype] * dp.abs() if act != "none" else 0)
    for name, ref, mag, e_in, k in (("dx", dp @ wd, dp.abs() @ wd.abs(), e_op @ wd.abs(), o),
                                    ("dw", dp.t() @ xd, dp.abs().t() @ xd.abs(), e_op.t() @ xd.abs(), n)):
        within_dev(got[name], ref, U[dtype] * ref.abs() + 1.02 * (acc(k) * mag + (e_in if act != "none" else 0)), name)
    within_dev(got["dbias"], dp.sum(0), acc(n) * dp.abs().sum(0) + e_dp.sum(0), "dbias")


LARGE_FWD, LARGE_BWD = {"linear_fwd_large"}, {"linear_dx_large", "linear_dw_large"}


@pytest.mark.parametrize("n,i,o,act,bias,fwd,bwd", [
    (3500, 3400, 3593, "gelu", F32, set(), set()),                       # whole, widths that are padded
    (3593, 3401, 3528, "none", BF16, set(), set()),
    (4100, 4097, 4352, "silu", F32, {"mm_tail"}, {"mm_tail"}),           # a shared last round
    (1500, 4700, 5300, "gelu_tanh", BF16, {"mm_join"}, {"mm_join"}),     # split over k
    (3500, 1100, 12300, "gelu", F32, set(), {"pack_rows_t", "mm_join"}),  # dW by way of x transposed, dx split
])
def test_linear_large_tiles(B, n, i, o, act, bias, fwd, bwd):
    check_linear_large(B, n, i, o, BF16, act, bias, LARGE_FWD | fwd, LARGE_BWD | bwd)


@pytest.mark.parametrize("n,tail", [(413, 29), (64 * 7, 0)])
def test_linear_wide_weight_gradient_transposed(B, n, tail):
    """Few tokens, of which the last k step holds `tail` (0: all of it is full)."""
    assert n % 64 == tail
    x, w = drand(430, n, 1100, dtype=BF16), drand(431, 12300, 1100, dtype=BF16)
    dy = drand(432, n, 12300, dtype=BF16)
    got, ran = labelled(B, lambda: B.poetx_linear_backward(x, w, dy, want_dx=False))
    assert {"pack_rows_t", "linear_dw_large"} <= ran, ran
    ref, mag = dy.double().t() @ x.double(), dy.double().abs().t() @ x.double().abs()
    within_dev(got["dw"], ref, U[BF16] * ref.abs() + 1.02 * acc(n) * mag, "dw")


def test_linear_large_tiles_float32(B):
    check_linear_large(B, 4093, 4087, 4090, F32, "gelu", F32, LARGE_FWD, LARGE_BWD, seed=440)


def check_xent_large(B, n, d, v, dtype, bwd, ignored=0.2, seed=450):
    """check_xent on the device: whole products of the larger tile in the forward, those of `bwd`
    in the backward."""
    h, w = drand(seed, n, d, dtype=dtype), drand(seed + 1, v, d, dtype=dtype, scale=2 * d ** -0.5)
    gen = torch.Generator("cuda").manual_seed(seed + 2)
    t = torch.randint(0, v, (n,), generator=gen, device="cuda", dtype=torch.int32)
    drop = torch.rand(n, generator=gen, device="cuda") < ignored
    t = torch.where(drop, torch.where(torch.arange(n, device="cuda") % 2 == 0, -1, v), t).int()
    dl = torch.rand(n, generator=gen, device="cuda") + 0.5
    (loss, lse), ran = labelled(B, lambda: B.poetx_xent_forward(h, w, t))
    assert "xent_fwd_large" in ran and "xent_parts" not in ran, ran
    hd, wd, on = h.double(), w.double(), ~drop
    logits = hd @ wd.t()
    e_l = acc(d) * (hd.abs() @ wd.abs().t()).amax(1)
    z = torch.logsumexp(logits, 1)
    arg = 2 * logits.abs().amax(1) + 1
    e_z = e_l + (v / 16 + 64) * 2.0 ** -24 + 2.0 ** -22 + arg * 2.0 ** -22 + 4 * U[F32] * z.abs()
    within_dev(lse, z, e_z, "lse")
    at = t.long().clamp(0, v - 1)[:, None]
    lt = logits.gather(1, at)[:, 0]
    none = torch.zeros_like(z)
    within_dev(loss, torch.where(on, z - lt, none),
               torch.where(on, e_z + e_l + 4 * U[F32] * (z.abs() + lt.abs()), none), "loss")

    got, ran = labelled(B, lambda: B.poetx_xent_backward(h, w, t, lse, dl))
    every = {"xent_dlogits_large", "xent_dh_large", "xent_dw_large"}
    assert every | bwd <= ran and ran & {"mm_join", "mm_tail", "pack_rows_t"} <= bwd, ran
    p = torch.exp(logits - z[:, None])
    del logits
    one = torch.zeros_like(p).scatter_(1, at, 1.0)
    g = torch.where(on, dl.double(), none)[:, None]
    dlog = (p - one) * g
    e_d = p * (e_l + e_z + arg * 2.0 ** -22 + 2.0 ** -21)[:, None]
    e_d = (e_d + 2 * U[F32] * (p + one)) * g + U[dtype] * dlog.abs()
    del p, one
    for name, r, mag, e, k in (("dh", dlog @ wd, dlog.abs() @ wd.abs(), e_d @ wd.abs(), v),
                               ("dw", dlog.t() @ hd, dlog.abs().t() @ hd.abs(), e_d.t() @ hd.abs(), n)):
        within_dev(got[name], r, U[dtype] * r.abs() + 1.02 * (acc(k) * mag + e), f"{name} {n} {d} {v}")
    assert not got["dh"][drop].any()


@pytest.mark.parametrize("n,d,v,bwd", [
    (3400, 3401, 3333, set()),                        # whole, padded d, tails on every axis
    (3340, 3528, 3593, set()),
    (4100, 4097, 4352, {"mm_tail"}),                  # a shared last round in all three
    (40000, 700, 15000, {"mm_join"}),                 # three pieces, dh whole, dW split over the tokens
    (40000, 392, 15000, {"mm_join", "mm_tail"}),      # and with dh's last round shared
    (16384, 1100, 25000, {"pack_rows_t", "mm_tail"}),  # two pieces, dW by way of h transposed
])
def test_xent_whole_large_tiles(B, n, d, v, bwd):
    check_xent_large(B, n, d, v, BF16, bwd)


def test_xent_large_tiles_float32(B):
    check_xent_large(B, 4093, 4087, 4090, F32, set(), seed=460)


@pytest.mark.parametrize("n,d,v", [(12, 72, 700), (60, 77, 700), (301, 520, 1007), (3400, 3401, 3333),
                                   (421, 1004, 12500)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_xent_one_gradient_alone(B, n, d, v, dtype):
    """A frozen head (dh alone) and dW alone.  Each is right element by element, and leaves no
    key of the other; where both are wanted the products may share a launch, so the sums' order
    may differ between the calls."""
    h, w = drand(470, n, d, dtype=dtype), drand(471, v, d, dtype=dtype, scale=2 * d ** -0.5)
    t = (torch.arange(n, device="cuda", dtype=torch.int32) * 7919) % v
    t[::4] = -1
    dl = drand(472, n)
    _, lse = B.poetx_xent_forward(h, w, t)
    a = B.poetx_xent_backward(h, w, t, lse, dl, want_dw=False)
    b = B.poetx_xent_backward(h, w, t, lse, dl, want_dh=False)
    assert set(a) == {"dh"} and set(b) == {"dw"}
    hd, wd, on = h.double(), w.double(), t >= 0
    logits = hd @ wd.t()
    z = torch.logsumexp(logits, 1)
    e_l = acc(d) * (hd.abs() @ wd.abs().t()).amax(1)
    arg = 2 * logits.abs().amax(1) + 1
    e_z = e_l + (v / 16 + 64) * 2.0 ** -24 + 2.0 ** -22 + arg * 2.0 ** -22 + 4 * U[F32] * z.abs()
    p = torch.exp(logits - z[:, None])
    one = torch.zeros_like(p).scatter_(1, t.long().clamp(0)[:, None], 1.0)
    g = torch.where(on, dl.double(), torch.zeros_like(z))[:, None]
    dlog = (p - one) * g
    e_d = p * (e_l + e_z + arg * 2.0 ** -22 + 2.0 ** -21)[:, None]
    e_d = (e_d + 2 * U[F32] * (p + one)) * g.abs() + U[dtype] * dlog.abs()
    for got, r, mag, e, k in ((a["dh"], dlog @ wd, dlog.abs() @ wd.abs(), e_d @ wd.abs(), v),
                              (b["dw"], dlog.t() @ hd, dlog.abs().t() @ hd.abs(), e_d.t() @ hd.abs(), n)):
        within_dev(got, r, U[dtype] * r.abs() + 1.02 * (acc(k) * mag + e), f"{n} {d} {v}")
    assert not a["dh"][~on].any()


@pytest.mark.parametrize("variant", ["fast", "mem"])
@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_block_step_bf16(B, act, variant):
    """test_block_step in bf16, both variants of the layer: loss and every gradient against
    float64 on the same bf16 inputs."""
    import torch.nn.functional as F
    from orthogonal_reparameterized_amd import workloads as WL
    from orthogonal_reparameterized_amd.step import BlockStep, LayerStep
    d, f, v, n, b = 512, 1160, 2003, 333, 64
    wl = WL.Workload(97, "block", n, d, d, b, "bf16", "bf16", "bf16", 0.02, d)
    inp = WL.make_layer_inputs(wl)
    p = {"gamma1": 1 + rand(1, d, scale=0.2), "beta1": rand(2, d, scale=0.2),
         "w1": rand(3, f, d, dtype=BF16, scale=d ** -0.5), "b1": rand(4, f, scale=0.2),
         "w2": rand(5, d, f, dtype=BF16, scale=f ** -0.5), "b2": rand(6, d, dtype=BF16, scale=0.2),
         "gamma2": (1 + rand(7, d, scale=0.2)).to(BF16), "beta2": rand(8, d, dtype=BF16, scale=0.2),
         "head": rand(9, v, d, dtype=BF16, scale=d ** -0.5)}
    x0 = rand(10, n, d, dtype=BF16)
    t = torch.randint(0, v, (n,), generator=torch.Generator().manual_seed(3), dtype=torch.int32)
    t[::7] = -1
    on = t >= 0
    dl = on.float() / on.sum()
    step = BlockStep(LayerStep(wl, inp, variant), {k: dev(q) for k, q in p.items()}, act=act)
    loss, got = step.step(dev(x0), dev(t), dev(dl))

    P = {k: q.double().requires_grad_(True) for k, q in p.items()}
    X = x0.double().requires_grad_(True)
    G, th = [], []
    for side in ("theta_r", "theta_p"):
        th.append(torch.from_numpy(inp[side].astype(np.float64)).requires_grad_(True))
        iu = torch.triu_indices(b, b, 1)
        Q = torch.zeros(th[-1].shape[0], b, b, dtype=torch.float64)
        Q = Q.index_put((torch.arange(Q.shape[0])[:, None], iu[0][None], iu[1][None]), th[-1])
        Q = Q - Q.transpose(1, 2)
        Q2 = Q @ Q
        G.append(torch.eye(b, dtype=torch.float64) + 2 * (Q + Q2 + Q2 @ Q) + Q2 @ Q2)
    W = torch.from_numpy(np.ascontiguousarray(inp["w"]).view(np.int16)).view(BF16).double()
    pin, pout = (torch.from_numpy(inp[k].astype(np.int64)) for k in ("perm_in", "perm_out"))
    wm = W[pout][:, pin]
    a = F.layer_norm(X, (d,), P["gamma1"], P["beta1"], 1e-5)
    blocks = lambda m, g: torch.cat([m[:, j * b:(j + 1) * b] @ g[j] for j in range(d // b)], 1)  # noqa: E731
    zt = blocks(blocks(a[:, pin], G[0]) @ wm.t(), G[1])
    z = torch.zeros_like(zt).index_copy(1, pout, zt)
    y = F.linear(getattr(F, act)(F.linear(z, P["w1"], P["b1"])), P["w2"], P["b2"]) + X
    h = F.layer_norm(y, (d,), P["gamma2"], P["beta2"], 1e-5)
    ref = F.cross_entropy(F.linear(h, P["head"]), t.long(), ignore_index=-1, reduction="none")
    leaves = dict(P, theta_r=th[0], theta_p=th[1], x0=X)
    grads = torch.autograd.grad((ref * dl.double()).sum(), list(leaves.values()))
    # about twenty tensors are rounded to bf16 on the way (eight forward, ten backward, both G), each
    # by at most u = 2^-8 of an element and u / sqrt(3) in the mean square, independently, with
    # condition numbers of a few as in test_block_step: sqrt(20 / 3) u 4
    most = (20 / 3) ** 0.5 * U[BF16] * 4
    assert off(loss, ref.detach()) <= most
    for (k, _), r in zip(leaves.items(), grads):
        assert off(got[k].reshape(r.shape), r) <= most, (k, off(got[k].reshape(r.shape), r))
