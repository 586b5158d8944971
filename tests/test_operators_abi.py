"""Refusals and workspace queries of the operators around the layer (layer norm, dense
linear layer, vocabulary cross entropy).  No GPU: every call fails validation, or only asks
for its workspace, before anything is launched."""

import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def B():
    from orthogonal_reparameterized_amd import binding
    return binding


A, C, D, E = 0x10000, 0x20000, 0x30000, 0x40000  # distinct addresses, never dereferenced
BIG = 1 << 50


def size(n=0):
    return ctypes.byref(ctypes.c_size_t(n))


def norm_fwd(B, n=4, d=64, dt=1, x=A, gamma=None, beta=None, pdt=0, eps=1e-5, y=C, mean=None, rstd=None):
    return B.raw.poetx_layernorm_forward(n, d, dt, x, gamma, beta, pdt, eps, y, mean, rstd, None)


def norm_bwd(B, n=4, d=64, dt=1, x=A, dy=C, gamma=None, pdt=0, mean=D, rstd=E, dres=None, dx=0x50000, dg=0x60000,
             db=0x70000, ws=0x80000, nb=BIG):
    return B.raw.poetx_layernorm_backward(n, d, dt, x, dy, gamma, pdt, mean, rstd, dres, dx, dg, db, ws, size(nb),
                                          None)


def lin_fwd(B, n=4, i=64, o=64, dt=1, x=A, w=C, bias=None, bdt=0, res=None, act=0, y=D, pre=None, ws=E, nb=BIG):
    return B.raw.poetx_linear_forward(n, i, o, dt, x, w, bias, bdt, res, act, y, pre, ws, size(nb), None)


def lin_bwd(B, n=4, i=64, o=64, dt=1, x=A, w=C, dy=D, pre=None, act=0, dx=E, dw=0x50000, db=0x60000, ws=0x70000,
            nb=BIG):
    return B.raw.poetx_linear_backward(n, i, o, dt, x, w, dy, pre, act, dx, dw, db, ws, size(nb), None)


def xent_fwd(B, n=4, d=64, v=1000, dt=1, h=A, w=C, t=D, loss=E, lse=0x50000, ws=0x60000, nb=BIG):
    return B.raw.poetx_xent_forward(n, d, v, dt, h, w, t, loss, lse, ws, size(nb), None)


def xent_bwd(B, n=4, d=64, v=1000, dt=1, h=A, w=C, t=D, lse=E, dl=0x50000, dh=0x60000, dw=0x70000, ws=0x80000,
             nb=BIG):
    return B.raw.poetx_xent_backward(n, d, v, dt, h, w, t, lse, dl, dh, dw, ws, size(nb), None)


def test_layernorm_refusals(B):
    bad = B.POETX_ERR_INVALID_ARG
    for kw in (dict(n=-1), dict(dt=2), dict(dt=7), dict(pdt=2), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(x=None), dict(y=None), dict(x=A + 8), dict(y=A), dict(gamma=A + 2),
               dict(mean=E, rstd=E), dict(beta=C)):
        assert norm_fwd(B, **kw) == bad, kw
    assert norm_fwd(B, d=0) == B.POETX_ERR_SHAPE
    assert norm_fwd(B, d=16385) == B.POETX_ERR_UNSUPPORTED
    assert norm_fwd(B, n=0, x=None, y=None) == B.POETX_OK
    for kw in (dict(n=-1), dict(dt=2), dict(x=None), dict(dy=None), dict(mean=None), dict(rstd=None), dict(dx=None),
               dict(dx=A), dict(dx=C), dict(dres=0x50000), dict(dg=0x70000), dict(dy=C + 4), dict(ws=0x80008)):
        assert norm_bwd(B, **kw) == bad, kw
    assert norm_bwd(B, d=0) == B.POETX_ERR_SHAPE
    assert norm_bwd(B, nb=64) == B.POETX_ERR_WORKSPACE
    assert B.raw.poetx_layernorm_backward(4, 64, 1, A, C, None, 0, D, E, None, A, C, None, None, None, None) == bad


def test_linear_refusals(B):
    bad = B.POETX_ERR_INVALID_ARG
    for kw in (dict(n=-1), dict(dt=2), dict(bdt=2), dict(act=-1), dict(act=5), dict(x=None), dict(w=None),
               dict(y=None), dict(x=A + 8), dict(res=D), dict(y=A), dict(pre=D), dict(bias=C + 4), dict(pre=C)):
        assert lin_fwd(B, **kw) == bad, kw
    for kw in (dict(i=0), dict(o=0), dict(i=-3)):
        assert lin_fwd(B, **kw) == B.POETX_ERR_SHAPE, kw
        assert lin_bwd(B, **kw) == B.POETX_ERR_SHAPE, kw
    for kw in (dict(i=(1 << 20) + 1), dict(o=(1 << 20) + 1), dict(n=1 << 41), dict(n=1 << 30, o=1 << 20)):
        assert lin_fwd(B, **kw) == B.POETX_ERR_UNSUPPORTED, kw
        assert lin_bwd(B, **kw) == B.POETX_ERR_UNSUPPORTED, kw
    assert lin_fwd(B, n=0, x=None, w=None, y=None) == B.POETX_OK
    for kw in (dict(n=-1), dict(dt=2), dict(act=9), dict(dy=None), dict(w=None), dict(x=None),
               dict(dx=None, dw=None, db=None), dict(act=B.POETX_ACT_GELU), dict(dx=A), dict(dw=C), dict(db=D),
               dict(dx=0x50000)):
        assert lin_bwd(B, **kw) == bad, kw


def test_xent_refusals(B):
    bad = B.POETX_ERR_INVALID_ARG
    for kw in (dict(n=-1), dict(dt=2), dict(h=None), dict(w=None), dict(t=None), dict(loss=None), dict(lse=None),
               dict(h=A + 8), dict(loss=0x50000), dict(loss=A), dict(t=D + 4)):
        assert xent_fwd(B, **kw) == bad, kw
    for kw in (dict(d=0), dict(v=0)):
        assert xent_fwd(B, **kw) == B.POETX_ERR_SHAPE, kw
        assert xent_bwd(B, **kw) == B.POETX_ERR_SHAPE, kw
    for kw in (dict(d=(1 << 20) + 1), dict(v=1 << 31), dict(n=1 << 22, v=1 << 24)):
        assert xent_fwd(B, **kw) == B.POETX_ERR_UNSUPPORTED, kw
        assert xent_bwd(B, **kw) == B.POETX_ERR_UNSUPPORTED, kw
    for kw in (dict(n=-1), dict(lse=None), dict(dl=None), dict(dh=None, dw=None), dict(dh=A), dict(dw=C),
               dict(dh=0x70000)):
        assert xent_bwd(B, **kw) == bad, kw
    assert xent_fwd(B, nb=16) == B.POETX_ERR_WORKSPACE
    assert xent_bwd(B, nb=16) == B.POETX_ERR_WORKSPACE


def query(f, *args):
    nb = ctypes.c_size_t(0)
    assert f(*args, None, ctypes.byref(nb), None) == 0
    return nb.value


def test_workspace_queries(B):
    r = B.raw
    none = [None] * 4
    # no parameter gradients, no workspace
    assert query(r.poetx_layernorm_backward, 4, 64, 1, None, None, None, 0, *none, None, None) == 0
    assert query(r.poetx_layernorm_backward, 4, 64, 1, None, None, None, 0, *none, A, C) >= 2 * 64 * 4
    # the frozen weight's copy of x is not made: dw costs workspace only where it is wanted
    odd = (100, 77, 64, 1, None, None, None, None, 0)
    assert query(r.poetx_linear_backward, *odd, A, None, None) < query(r.poetx_linear_backward, *odd, A, C, None)
    # no tokens: every query answers
    assert query(r.poetx_layernorm_backward, 0, 64, 1, None, None, None, 0, *none, A, C) == 0
    assert query(r.poetx_linear_forward, 0, 64, 64, 1, *none[:3], 0, None, 0, None, None) == 0
    assert query(r.poetx_linear_backward, 0, 64, 64, 1, *none, 0, A, C, D) >= 0
    assert query(r.poetx_xent_forward, 0, 64, 100, 1, *none, None) == 0
    assert query(r.poetx_xent_backward, 0, 64, 100, 1, *none, None, A, C) == 0
    # logits are never kept: far less than n x v values, and pieces of dl at most 512 MB
    n, d, v = 16384, 1024, 131072
    fwd = query(r.poetx_xent_forward, n, d, v, 1, *none, None)
    assert n * 8 < fwd < n * v // 8
    bwd = query(r.poetx_xent_backward, n, d, v, 1, *none, None, A, C)
    assert bwd < (600 << 20) + n * d * 8


def test_weight_gradient_of_very_many_tokens_makes_no_transposed_copy(B):
    """The transposed copy of x has the tokens as its row stride, and a tile's 256 rows of it
    are reached by 32-bit offsets: 2^20 tokens at most."""
    d_in, d_out = 4096, 8192
    args = (d_in, d_out, 1, None, None, None, None, 0, None, A, None)
    f = B.raw.poetx_linear_backward
    assert query(f, 1 << 20, *args) >= d_in * 2 << 20
    for n in ((1 << 20) + 1, 1 << 22, (1 << 23) - 8):
        assert query(f, n, *args) < d_in * 2 * n


def test_binding_refusals(B):
    """The binding refuses shapes, dtypes and layouts before it touches a device."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(32, 64, dtype=torch.bfloat16)
    s = torch.zeros(4)
    t = torch.zeros(4, dtype=torch.int32)
    cases = [
        lambda: B.poetx_layernorm_forward(x.half()),
        lambda: B.poetx_layernorm_forward(x, torch.zeros(63)),
        lambda: B.poetx_layernorm_forward(x, torch.zeros(64), torch.zeros(64, dtype=torch.bfloat16)),
        lambda: B.poetx_layernorm_forward(x[:, ::2]),
        lambda: B.poetx_layernorm_forward(x),  # on the CPU
        lambda: B.poetx_layernorm_backward(x, x.float(), None, s, s),
        lambda: B.poetx_layernorm_backward(x, x, None, s[:3], s),
        lambda: B.poetx_linear_forward(x, w.float()),
        lambda: B.poetx_linear_forward(x, w[:, :32]),
        lambda: B.poetx_linear_forward(x, w, act="swish"),
        lambda: B.poetx_linear_forward(x, w, residual=x),
        lambda: B.poetx_linear_forward(x, w, torch.zeros(31)),
        lambda: B.poetx_linear_forward(x, w),  # on the CPU
        lambda: B.poetx_linear_backward(x, None, x[:, :32].contiguous()),
        lambda: B.poetx_linear_backward(x, w, x[:, :32].contiguous(), act="gelu"),
        lambda: B.poetx_linear_backward(x, w, x),
        lambda: B.poetx_xent_forward(x, w, t.long()),
        lambda: B.poetx_xent_forward(x, w, t[:3]),
        lambda: B.poetx_xent_forward(x, w[:, :63].contiguous(), t),
        lambda: B.poetx_xent_backward(x, w, t, s, s, want_dh=False, want_dw=False),
        lambda: B.poetx_xent_backward(x, w, t, s.double(), s),
    ]
    for k, f in enumerate(cases):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"case {k} was accepted")


def test_a_null_workspace_is_the_query_also_where_none_is_needed(B):
    """With every buffer given and a requirement of 0, ws == NULL still asks for the size and
    launches nothing (a launch on these addresses, or without a GPU, would not return OK)."""
    for f, kw in ((norm_bwd, dict(dg=None, db=None)), (lin_fwd, dict(n=4)), (lin_fwd, dict(n=0)),
                  (norm_bwd, dict(n=0, dg=None, db=None)), (lin_bwd, dict(n=0, db=None))):
        assert f(B, ws=None, nb=1 << 30, **kw) == B.POETX_OK, (f, kw)
    r, none = B.raw, [None] * 4
    assert query(r.poetx_linear_forward, 4, 64, 64, 1, A, C, None, 0, None, 0, D, None) == 0
    assert query(r.poetx_layernorm_backward, 4, 64, 1, A, C, None, 0, D, E, None, 0x50000, None, None) == 0
    assert query(r.poetx_linear_backward, 0, 64, 64, 1, *none, 0, A, C, None) == 0


def test_binding_imports_without_torchs_internal_functions():
    """The binding takes torch's internal stream lookup where it is there and does without
    otherwise."""
    import subprocess
    import sys
    code = ("import torch\n"
            "for name in ('_cuda_getCurrentRawStream', '_cuda_isCurrentStreamCapturing'):\n"
            "    if hasattr(torch._C, name): delattr(torch._C, name)\n"
            "from orthogonal_reparameterized_amd import binding\n"
            "assert callable(binding._raw_stream) and callable(binding._capturing)\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
