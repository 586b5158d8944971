"""Cases of the training operators around the POET-X layer: layer norm, the dense linear
layer with its epilogue, and the softmax cross entropy of a language-model head.

Each case names one call, or one pair of calls, that a training or scoring program makes.
`run` computes it either in elementary float32 torch operations (own = False) or through
this package's entry points (own = True); `exact` is the same in float64.
"""

import math

import torch

own = False

EPS = 1e-5
_T = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # pre-norm of a training batch at the attention-projection width, and its backward
        # with the gradient of the residual stream added
        {"name": "norm_fwd 8192x4096", "op": "norm_fwd", "n": 8192, "d": 4096, "dtype": "bf16", "params": "f32"},
        {"name": "norm_bwd 8192x4096", "op": "norm_bwd", "n": 8192, "d": 4096, "dtype": "bf16", "params": "f32",
         "dres": True},
        # one token of a decoding loop: a call's latency
        {"name": "norm_fwd 1x5120", "op": "norm_fwd", "n": 1, "d": 5120, "dtype": "bf16", "params": "bf16"},
        # float32 rows of an odd width, which no vector load fits
        {"name": "norm_bwd 1000x1001", "op": "norm_bwd", "n": 1000, "d": 1001, "dtype": "f32", "params": "f32",
         "dres": False},
        # MLP up-projection of a training batch: bias and activation, the pre-activation kept
        {"name": "linear_fwd 8192 4096-14336", "op": "linear_fwd", "n": 8192, "d_in": 4096, "d_out": 14336,
         "dtype": "bf16", "params": "f32", "act": "gelu", "bias": True, "residual": False, "pre": True},
        # its backward, at the square projection
        {"name": "linear_bwd 8192 4096-4096", "op": "linear_bwd", "n": 8192, "d_in": 4096, "d_out": 4096,
         "dtype": "bf16", "params": "f32", "act": "silu", "bias": True},
        # one token of a decoding loop: the weight is read once
        {"name": "linear_fwd 1 5120-13824", "op": "linear_fwd", "n": 1, "d_in": 5120, "d_out": 13824,
         "dtype": "bf16", "params": "bf16", "act": "none", "bias": True, "residual": True, "pre": False},
        # a ragged float32 batch at widths that nothing divides
        {"name": "linear_bwd f32 513 1001-777", "op": "linear_bwd", "n": 513, "d_in": 1001, "d_out": 777,
         "dtype": "f32", "params": "f32", "act": "gelu_tanh", "bias": True},
        # loss of an evaluation batch
        {"name": "xent_fwd 8192 4096 32768", "op": "xent_fwd", "n": 8192, "d": 4096, "v": 32768, "dtype": "bf16",
         "ignored": 0.0},
        # a few tokens scored against a large vocabulary: the head's weight is read once
        {"name": "xent_fwd 8 4096 131072", "op": "xent_fwd", "n": 8, "d": 4096, "v": 131072, "dtype": "bf16",
         "ignored": 0.0},
        # the last step of a training pass: loss and both gradients, padding rows among the tokens
        {"name": "xent_step 4096 4096 65536", "op": "xent_step", "n": 4096, "d": 4096, "v": 65536, "dtype": "bf16",
         "ignored": 0.1},
        # the same in float32, at sizes that no tile divides
        {"name": "xent_step f32 301 520 10007", "op": "xent_step", "n": 301, "d": 520, "v": 10007, "dtype": "f32",
         "ignored": 0.3},
    ]


def _size(rng, lo, hi, fine=None):
    """A size between lo and hi, even over its logarithm; half of them multiples of `fine`."""
    s = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if fine and s > fine and rng.random() < 0.5:
        s -= s % fine
    return max(lo, min(hi, s))


def draw(rng):
    op = rng.choice(("norm_fwd", "norm_bwd", "linear_fwd", "linear_fwd", "linear_bwd", "xent_fwd", "xent_step"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    params = rng.choice(("f32", "bf16")) if dtype == "bf16" else "f32"
    # a bound on tokens x width x width, so that no drawn case outweighs the largest listed one
    most = 2.0 ** 38 if dtype == "bf16" else 2.0 ** 34
    while True:
        if op.startswith("norm"):
            c = {"op": op, "n": _size(rng, 1, 16384, 64), "d": _size(rng, 64, 16384, 64), "dtype": dtype,
                 "params": params}
            if op == "norm_bwd":
                c["dres"] = rng.random() < 0.5
            if c["n"] * c["d"] <= 2 ** 26:
                return c
        elif op.startswith("linear"):
            act = rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu"))
            c = {"op": op, "n": _size(rng, 1 if op == "linear_fwd" else 16, 8192, 64),
                 "d_in": _size(rng, 64, 8192, 128), "d_out": _size(rng, 64, 14336, 128), "dtype": dtype,
                 "params": params, "act": act, "bias": rng.random() < 0.7}
            if op == "linear_fwd":
                c["residual"] = rng.random() < 0.5
                c["pre"] = act != "none" and rng.random() < 0.5
            if c["n"] * c["d_in"] * c["d_out"] <= most:
                return c
        else:
            c = {"op": op, "n": _size(rng, 1 if op == "xent_fwd" else 16, 8192, 64), "d": _size(rng, 64, 8192, 128),
                 "v": _size(rng, 1000, 131072, 128), "dtype": dtype, "ignored": rng.choice((0.0, 0.1, 0.5))}
            if c["n"] * c["d"] * c["v"] <= most:
                return c


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = _T[case["dtype"]]
    pt = _T[case["params"]] if "params" in case else torch.float32

    def randn(*shape, std=1.0, mean=0.0):
        return torch.randn(shape, generator=gen, device="cuda") * std + mean

    s = {"op": case["op"]}
    n = case["n"]
    if case["op"].startswith("norm"):
        d = case["d"]
        # rows of a residual stream: a scale and an offset of their own
        s["x"] = (randn(n, d) * torch.exp(randn(n, 1, std=0.5)) + randn(n, 1, std=0.5)).to(dt)
        s["gamma"] = randn(d, std=0.2, mean=1.0).to(pt)
        s["beta"] = randn(d, std=0.2).to(pt)
        if case["op"] == "norm_bwd":
            s["dy"] = randn(n, d).to(dt)
            s["dres"] = randn(n, d).to(dt) if case["dres"] else None
            # what the forward left behind: the rows' statistics
            x = s["x"].double()
            mean = x.sum(1) / d
            s["mean"] = mean.float()
            s["rstd"] = (((x - mean[:, None]).square().sum(1) / d + EPS) ** -0.5).float()
    elif case["op"].startswith("linear"):
        d_in, d_out = case["d_in"], case["d_out"]
        s["act"] = case["act"]
        s["x"] = randn(n, d_in).to(dt)
        s["w"] = randn(d_out, d_in, std=d_in ** -0.5).to(dt)
        s["bias"] = randn(d_out, std=0.2).to(pt) if case["bias"] else None
        if case["op"] == "linear_fwd":
            s["residual"] = randn(n, d_out).to(dt) if case["residual"] else None
            s["pre"] = case["pre"]
        else:
            s["dy"] = randn(n, d_out).to(dt)
            # what the forward left behind: the pre-activation (its distribution is that of the
            # product of these inputs)
            s["pre"] = randn(n, d_out, std=1.02).to(dt) if case["act"] != "none" else None
    else:
        d, v = case["d"], case["v"]
        s["w"] = randn(v, d, std=2.0 * d ** -0.5).to(dt)
        target = torch.randint(0, v, (n,), generator=gen, device="cuda", dtype=torch.int32)
        # hidden states that point towards their target's row, as a partly trained model's do
        lean = 2.0 * torch.rand((n, 1), generator=gen, device="cuda")
        s["h"] = (randn(n, d) + lean * s["w"][target.long()].float()).to(dt)
        drop = torch.rand((n,), generator=gen, device="cuda") < case["ignored"]
        s["target"] = torch.where(drop, torch.full_like(target, -1), target)
        if case["op"] == "xent_step":
            # the gradient of the mean over the rows that count
            s["dloss"] = torch.full((n,), 1.0, device="cuda") / (~drop).sum().clamp(min=1)
    return s


# ---------------------------------------------------------------- plain forms, float32 ----

def _plain_act(pre, act):
    if act == "relu":
        return torch.where(pre > 0, pre, torch.zeros_like(pre))
    if act == "gelu":
        return 0.5 * pre * (1.0 + torch.erf(pre * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * pre * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (pre + 0.044715 * pre * pre * pre)))
    if act == "silu":
        return pre / (1.0 + torch.exp(-pre))
    return pre


def _plain_act_grad(pre, act):
    if act == "relu":
        return (pre > 0).to(pre.dtype)
    if act == "gelu":
        phi = torch.exp(-0.5 * pre * pre) * (1.0 / math.sqrt(2.0 * math.pi))
        return 0.5 * (1.0 + torch.erf(pre * math.sqrt(0.5))) + pre * phi
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (pre + 0.044715 * pre * pre * pre))
        return 0.5 * (1.0 + t) + 0.5 * pre * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * pre * pre)
    sg = 1.0 / (1.0 + torch.exp(-pre))
    return sg * (1.0 + pre * (1.0 - sg))


def _plain_norm_fwd(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    c = x - mean
    rstd = torch.rsqrt((c * c).mean(1, keepdim=True) + EPS)
    y = c * rstd * s["gamma"].float() + s["beta"].float()
    return {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _plain_norm_bwd(s):
    x, dy = s["x"].float(), s["dy"].float()
    rstd = s["rstd"][:, None]
    xhat = (x - s["mean"][:, None]) * rstd
    g = dy * s["gamma"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(s["x"].dtype), "dgamma": (dy * xhat).sum(0), "dbeta": dy.sum(0)}


def _plain_linear_fwd(s):
    pre = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        pre = pre + s["bias"].float()
    y = _plain_act(pre, s["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    dt = s["x"].dtype
    return {"y": y.to(dt), "pre": pre.to(dt) if s["pre"] else None}


def _plain_linear_bwd(s):
    dt = s["x"].dtype
    dpre = s["dy"].float()
    if s["act"] != "none":
        dpre = dpre * _plain_act_grad(s["pre"].float(), s["act"])
    dx = dpre @ s["w"].float()
    dw = dpre.t() @ s["x"].float()
    return {"dx": dx.to(dt), "dw": dw.to(dt), "dbias": dpre.sum(0) if s["bias"] is not None else None}


def _plain_xent(s):
    h, w, target = s["h"].float(), s["w"].float(), s["target"].long()
    logits = h @ w.t()
    top = logits.amax(1, keepdim=True)
    e = torch.exp(logits - top)
    total = e.sum(1, keepdim=True)
    lse = (top + torch.log(total))[:, 0]
    counts = (target >= 0) & (target < w.shape[0])
    at = torch.where(counts, target, torch.zeros_like(target))[:, None]
    loss = torch.where(counts, lse - logits.gather(1, at)[:, 0], torch.zeros_like(lse))
    out = {"loss": loss, "lse": lse}
    if s["op"] == "xent_step":
        p = e / total
        p.scatter_add_(1, at, torch.full_like(lse, -1.0)[:, None])
        dlogits = p * torch.where(counts, s["dloss"], torch.zeros_like(lse))[:, None]
        out["dh"] = (dlogits @ w).to(s["h"].dtype)
        out["dw"] = (dlogits.t() @ h).to(s["w"].dtype)
    return out


_PLAIN = {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "linear_fwd": _plain_linear_fwd,
          "linear_bwd": _plain_linear_bwd, "xent_fwd": _plain_xent, "xent_step": _plain_xent}


# ------------------------------------------------------------------ the package's calls ----

def _own(s):
    from orthogonal_reparameterized_amd import binding as B
    op = s["op"]
    if op == "norm_fwd":
        y, mean, rstd = B.poetx_layernorm_forward(s["x"], s["gamma"], s["beta"], EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_bwd":
        return B.poetx_layernorm_backward(s["x"], s["dy"], s["gamma"], s["mean"], s["rstd"], dres=s["dres"])
    if op == "linear_fwd":
        y, pre = B.poetx_linear_forward(s["x"], s["w"], s["bias"], s["residual"], s["act"], save_pre=s["pre"])
        return {"y": y, "pre": pre}
    if op == "linear_bwd":
        return B.poetx_linear_backward(s["x"], s["w"], s["dy"], s["pre"], s["act"],
                                       want_dbias=s["bias"] is not None)
    loss, lse = B.poetx_xent_forward(s["h"], s["w"], s["target"])
    out = {"loss": loss, "lse": lse}
    if op == "xent_step":
        out.update(B.poetx_xent_backward(s["h"], s["w"], s["target"], lse, s["dloss"]))
    return out


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["op"]](state)


def work(case):
    """Each input read once, each output written once; the products of the definition."""
    e = 2 if case["dtype"] == "bf16" else 4
    p = 4 if case.get("params") == "f32" else 2
    n, op = case["n"], case["op"]
    if op == "norm_fwd":
        d = case["d"]
        return {"bytes": 2 * n * d * e + 2 * d * p + 8 * n, "flops": 8 * n * d}
    if op == "norm_bwd":
        d = case["d"]
        return {"bytes": (4 if case["dres"] else 3) * n * d * e + d * p + 8 * d + 8 * n, "flops": 14 * n * d}
    if op.startswith("linear"):
        i, o = case["d_in"], case["d_out"]
        if op == "linear_fwd":
            return {"bytes": (n * i + i * o) * e + (o * p if case["bias"] else 0)
                    + n * o * e * (1 + case["residual"] + case["pre"]), "flops": 2 * n * i * o}
        return {"bytes": (2 * n * i + 2 * i * o + n * o * (1 + (case["act"] != "none"))) * e
                + (4 * o if case["bias"] else 0), "flops": 4 * n * i * o}
    d, v = case["d"], case["v"]
    step = op == "xent_step"
    return {"bytes": (n * d + v * d) * e * (2 if step else 1) + n * (16 if step else 12),
            "flops": (6 if step else 2) * n * d * v}


# ------------------------------------------------------------------- float64 definition ----

def exact(case, seed):
    import torch.nn.functional as F
    s = prepare(case, seed)
    op = s["op"]
    if op == "norm_fwd":
        x = s["x"].double()
        y = F.layer_norm(x, (case["d"],), s["gamma"].double(), s["beta"].double(), EPS)
        return {"y": y, "mean": x.mean(1), "rstd": 1.0 / torch.sqrt(x.var(1, unbiased=False) + EPS)}
    if op == "norm_bwd":
        # the derivative through x, with the statistics as functions of it
        x = s["x"].double().requires_grad_(True)
        gamma = s["gamma"].double().requires_grad_(True)
        beta = s["beta"].double().requires_grad_(True)
        y = F.layer_norm(x, (case["d"],), gamma, beta, EPS)
        dx, dg, db = torch.autograd.grad(y, (x, gamma, beta), s["dy"].double())
        if s["dres"] is not None:
            dx = dx + s["dres"].double()
        return {"dx": dx, "dgamma": dg, "dbeta": db}
    act = {"none": lambda t: t, "relu": F.relu, "gelu": F.gelu, "silu": F.silu,
           "gelu_tanh": lambda t: F.gelu(t, approximate="tanh")}
    if op == "linear_fwd":
        pre = F.linear(s["x"].double(), s["w"].double(), None if s["bias"] is None else s["bias"].double())
        y = act[s["act"]](pre)
        if s["residual"] is not None:
            y = y + s["residual"].double()
        return {"y": y, "pre": pre if s["pre"] else None}
    if op == "linear_bwd":
        dpre = s["dy"].double()
        if s["act"] != "none":
            pre = s["pre"].double().requires_grad_(True)
            dpre, = torch.autograd.grad(act[s["act"]](pre), pre, dpre)
        return {"dx": torch.mm(dpre, s["w"].double()), "dw": torch.mm(s["x"].double().t(), dpre).t().contiguous(),
                "dbias": dpre.sum(0) if s["bias"] is not None else None}
    # cross entropy over pieces of the tokens; the head's gradient summed over the pieces
    step = op == "xent_step"
    w = s["w"].double().requires_grad_(step)
    target = s["target"].long()
    target = torch.where((target < 0) | (target >= case["v"]), torch.full_like(target, -1), target)
    piece = max(1, 2 ** 28 // case["v"])
    out = {"loss": [], "lse": []}
    dh, dw = [], None
    for k in range(0, case["n"], piece):
        h = s["h"][k:k + piece].double().requires_grad_(step)
        logits = F.linear(h, w)
        loss = F.cross_entropy(logits, target[k:k + piece], ignore_index=-1, reduction="none")
        out["loss"].append(loss.detach())
        out["lse"].append(torch.logsumexp(logits.detach(), 1))
        if step:
            gh, gw = torch.autograd.grad((loss * s["dloss"][k:k + piece].double()).sum(), (h, w))
            dh.append(gh)
            dw = gw if dw is None else dw + gw
    out = {k: torch.cat(v) for k, v in out.items()}
    if step:
        out.update({"dh": torch.cat(dh), "dw": dw})
    return out
