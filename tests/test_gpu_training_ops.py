"""The training operators on the GPU against plain 64-bit forms.

Tolerances are error bounds worked out from the operations: a BF16 rounding is
off by at most 2^-8 of the value, an fp32 operation by 2^-24, a tensor-core sum
over K by at most 2^-23 of the sum of magnitudes for each 16-wide step.
"""
import math
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import rank_gradient_sketching_philox_gb300 as rgs
from rank_gradient_sketching_philox_gb300 import binding, synth

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__ as g
    g.build()
    binding.lib()


@pytest.fixture(autouse=True)
def no_timeouts():
    yield
    assert binding.read_device_errors() == 0


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape, std=1.0, dtype=F32):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def rows(t, ld, offset=0):
    """The same values with row stride ld, ``offset`` elements into a buffer filled with NaN."""
    buf = torch.full((offset + t.shape[0] * ld,), float("nan"), dtype=t.dtype, device=DEV)
    view = buf[offset:].view(t.shape[0], ld)[:, :t.shape[1]]
    view.copy_(t)
    return view


def within(got, want, bound):
    """Every element within its bound; NaN nowhere."""
    err = (got.to(F64) - want).abs()
    assert not torch.isnan(err).any()
    over = err - bound
    assert (over <= 0).all(), "worst excess %.3g at error %.3g" % (over.max().item(), err.flatten()[over.argmax()].item())


# ---- layer norm -----------------------------------------------------------------

def norm64(X, gamma, beta, eps):
    x = X.to(F64)
    mean = x.mean(1, keepdim=True)
    rstd = ((x - mean).square().mean(1, keepdim=True) + eps).rsqrt()
    y = (x - mean) * rstd
    if gamma is not None:
        y = y * gamma.to(F64)
    return (y if beta is None else y + beta.to(F64)), mean[:, 0], rstd[:, 0]


def norm_bounds(X, eps, sums):
    """Bounds on the errors of mean, of xh and of rstd (relative): sums of k terms of which a thread adds
    at most ``sums`` in a row, fp32."""
    x = X.to(F64)
    _, mean, rstd = norm64(X, None, None, eps)
    n = (sums + 16) * 2.0 ** -24
    dmean = n * x.abs().mean(1)
    # var's error: n of itself, and the square of mean's error
    drel = 0.5 * (n + (dmean * rstd) ** 2) + 2.0 ** -22
    return dmean, drel


NORM_SHAPES = [(1, 1), (1, 2), (3, 7), (2, 8), (5, 31), (4, 32), (7, 257), (33, 512), (130, 1000), (1021, 1001),
               (64, 1024), (17, 2048), (300, 4096), (9, 5000), (3, 8192), (5, 8200), (2, 16384), (3, 16387), (2, 40000)]


@pytest.mark.parametrize("x,w", [(BF, F32), (BF, BF), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("T,k", NORM_SHAPES)
def test_norm_forward(T, k, x, w):
    g = gen(T * 100003 + k)
    X = randn(g, T, k, dtype=x) + 0.5
    gamma, beta = randn(g, k, dtype=w), randn(g, k, dtype=w)
    Y, mean, rstd = torch.full_like(X, float("nan")), torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    rgs.layer_norm_forward(X, gamma, beta, Y, mean, rstd, eps=1e-5)
    y, m, r = norm64(X, gamma, beta, 1e-5)
    dmean, drel = norm_bounds(X, 1e-5, k)
    within(mean, m, dmean + 1e-30)
    within(rstd, r, drel * r)
    xh = (X.to(F64) - m[:, None]).abs() * r[:, None]
    bound = ((dmean * r)[:, None] + xh * (drel[:, None] + 2.0 ** -22)) * gamma.to(F64).abs() + y.abs() * 2.0 ** -23
    bound = bound + beta.to(F64).abs() * 2.0 ** -23
    within(Y, y, bound * 1.01 + (y.abs() * 2.0 ** -8 if x == BF else 0.0) + 1e-30)


@pytest.mark.parametrize("x", [BF, F32])
@pytest.mark.parametrize("T,k,ld,offset", [(5, 64, 64, 1), (5, 64, 67, 0), (33, 1000, 1008, 0), (33, 1001, 1004, 3),
                                           (8, 4096, 4104, 0), (8, 4096, 4097, 5)])
def test_norm_rows_of_any_stride_and_alignment(T, k, ld, offset, x):
    """Strided and unaligned rows give the bits of contiguous ones, and nothing outside them is written."""
    g = gen(k)
    X, dY = randn(g, T, k, dtype=x), randn(g, T, k, dtype=x)
    gamma, beta = randn(g, k), randn(g, k)
    out = {}
    for name, place in (("plain", lambda t: t.clone()), ("strided", lambda t: rows(t, ld, offset))):
        Xp, dYp = place(X), place(dY)
        Y, dX = place(torch.zeros_like(X)), place(torch.zeros_like(X))
        mean, rstd, dg, db = (torch.empty(n, device=DEV) for n in (T, T, k, k))
        rgs.layer_norm_forward(Xp, gamma, beta, Y, mean, rstd)
        rgs.layer_norm_backward(dYp, Xp, gamma, mean, rstd, dX, dg, db, overwrite=True)
        out[name] = (Y, mean, rstd, dX, dg, db)
        for t in (Y, dX):
            base = t._base if t._base is not None else t
            kept = torch.zeros(base.numel(), dtype=torch.bool, device=DEV)
            torch.as_strided(kept, t.shape, t.stride(), t.storage_offset()).fill_(True)
            assert torch.isnan(base.reshape(-1)[~kept]).all()
    y, m, r = norm64(X, gamma, beta, 1e-5)
    for a, b in zip(out["plain"], out["strided"]):
        assert torch.isfinite(b).all()
        # the two may add in another order: fp32 sums of k or T terms, then perhaps one BF16 step
        step = 2.0 ** -7 if a.dtype == BF else 0.0
        within(b, a.to(F64), a.to(F64).abs() * step + (k + T) * 2.0 ** -23 * (1 + a.to(F64).abs().max()))


def test_norm_without_weights_in_place_and_special_rows():
    g = gen(5)
    X = randn(g, 6, 100)
    X[1] = 3.0                 # no variance: rstd = 1/sqrt(eps), y = 0
    X[2] *= 1e18               # squares up to 1e38 / 100
    X[3] *= 1e-30
    X[4, 7] = float("nan")     # stays in its own row
    X[5, 9] = float("inf")
    want, m, r = norm64(X, None, None, 1e-5)
    mean, rstd = torch.empty(6, device=DEV), torch.empty(6, device=DEV)
    Y = X.clone()
    rgs.layer_norm_forward(Y, None, None, Y, mean, rstd)
    assert torch.equal(Y[1], torch.zeros(100, device=DEV))
    assert abs(rstd[1].item() - 1e-5 ** -0.5) < 1e-4
    for i in (0, 2, 3):
        within(Y[i], want[i], 1e-5 * want[i].abs().max() + 1e-30)
    assert torch.isnan(Y[4]).all() and torch.isnan(Y[5]).any()
    assert torch.isfinite(Y[:4]).all()


def norm_grads64(dY, X, gamma, eps):
    x, dy = X.to(F64), dY.to(F64)
    xh, _, r = norm64(X, None, None, eps)
    d = dy if gamma is None else dy * gamma.to(F64)
    dx = r[:, None] * (d - d.mean(1, keepdim=True) - xh * (d * xh).mean(1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0), xh, d, r


@pytest.mark.parametrize("x,w", [(BF, F32), (BF, BF), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("T,k", NORM_SHAPES + [(2000, 64), (5000, 40)])
def test_norm_backward(T, k, x, w):
    g = gen(T * 7 + k)
    X, dY, gamma = randn(g, T, k, dtype=x), randn(g, T, k, dtype=x), randn(g, k, dtype=w)
    eps = 1e-3 if k > 1 else 1.0
    _, m, r = norm64(X, None, None, eps)
    mean, rstd = m.float(), r.float()
    dx, dg, db, xh, d, r = norm_grads64(dY, X, gamma, eps)
    dX, dgamma, dbeta = torch.full_like(X, float("nan")), torch.ones(k, device=DEV), torch.ones(k, device=DEV)
    rgs.layer_norm_backward(dY, X, gamma, mean, rstd, dX, dgamma, dbeta, overwrite=True)
    # xh from fp32 mean and rstd: 2^-24 of |x - m| and |m|, three operations
    exh = 2.0 ** -22 * (xh.abs() + (m.abs() * r)[:, None])
    n = (k + 16) * 2.0 ** -24
    e0 = n * d.abs().mean(1, keepdim=True)
    e1 = n * (d * xh).abs().mean(1, keepdim=True) + (d.abs() * exh).mean(1, keepdim=True)
    s1 = (d * xh).mean(1, keepdim=True).abs()
    ex = r[:, None] * (e0 + exh * s1 + xh.abs() * e1 + 2.0 ** -21 * (d.abs() + d.mean(1, keepdim=True).abs() + xh.abs() * s1))
    within(dX, dx, ex * 1.01 + (dx.abs() * 2.0 ** -8 if x == BF else 0.0) + 1e-30)
    nt = (T + 16) * 2.0 ** -24
    within(dgamma, dg, nt * (dY.to(F64) * xh).abs().sum(0) + (dY.to(F64).abs() * exh).sum(0) + 1e-30)
    within(dbeta, db, nt * dY.to(F64).abs().sum(0) + 1e-30)
    # adding to gradients, each output alone, the same bits; dX in dY's place
    twice = [dgamma.clone(), dbeta.clone()]
    rgs.layer_norm_backward(dY, X, gamma, mean, rstd, dgamma=twice[0])
    rgs.layer_norm_backward(dY, X, gamma, mean, rstd, dbeta=twice[1])
    assert torch.equal(twice[0], dgamma + dgamma) and torch.equal(twice[1], dbeta + dbeta)
    inplace = dY.clone()
    rgs.layer_norm_backward(inplace, X, gamma, mean, rstd, dX=inplace)
    assert torch.equal(inplace, dX)


LONG_SHAPES = [(40000, 24), (9000, 100), (3000, 520), (2500, 4096), (2500, 4100), (2011, 4099), (900, 8192),
               (700, 8200), (400, 8201), (500, 12288), (400, 12289), (330, 16384), (330, 16383)]


@pytest.mark.parametrize("x", [BF, F32])
@pytest.mark.parametrize("T,k", LONG_SHAPES)
def test_norm_many_rows_of_every_width(T, k, x):
    """More rows than the blocks in flight: each block walks over several sets of them."""
    g = gen(T + k)
    X, dY = randn(g, T, k, dtype=x) + 0.25, randn(g, T, k, dtype=x)
    gamma, beta = randn(g, k), randn(g, k)
    eps = 1e-5
    Y, dX = torch.full_like(X, float("nan")), torch.full_like(X, float("nan"))
    mean, rstd, dg, db = (torch.full((n,), float("nan"), device=DEV) for n in (T, T, k, k))
    rgs.layer_norm_forward(X, gamma, beta, Y, mean, rstd, eps=eps)
    rgs.layer_norm_backward(dY, X, gamma, mean, rstd, dX, dg, db, overwrite=True)
    y, m, r = norm64(X, gamma, beta, eps)
    dmean, drel = norm_bounds(X, eps, k)
    within(mean, m, dmean)
    within(rstd, r, drel * r)
    xh = (X.to(F64) - m[:, None]).abs() * r[:, None]
    bound = ((dmean * r)[:, None] + xh * (drel[:, None] + 2.0 ** -22)) * gamma.to(F64).abs()
    bound = bound + (y.abs() + beta.to(F64).abs()) * 2.0 ** -23
    half = 2.0 ** -8 if x == BF else 0.0
    within(Y, y, bound * 1.01 + y.abs() * half)
    # the gradients of the formula at the kernel's own mean and rstd
    m, r = mean.to(F64), rstd.to(F64)
    xs, dy = X.to(F64), dY.to(F64)
    xh = (xs - m[:, None]) * r[:, None]
    d = dy * gamma.to(F64)
    s0, s1 = d.mean(1, keepdim=True), (d * xh).mean(1, keepdim=True)
    dx = r[:, None] * (d - s0 - xh * s1)
    exh = 2.0 ** -22 * (xh.abs() + (m.abs() * r)[:, None])
    n = (k + 16) * 2.0 ** -24
    e0 = n * d.abs().mean(1, keepdim=True)
    e1 = n * (d * xh).abs().mean(1, keepdim=True) + (d.abs() * exh).mean(1, keepdim=True)
    ex = r[:, None] * (e0 + exh * s1.abs() + xh.abs() * e1 + 2.0 ** -21 * (d.abs() + s0.abs() + xh.abs() * s1.abs()))
    within(dX, dx, ex * 1.01 + dx.abs() * half)
    nt = (T + 16) * 2.0 ** -24
    within(dg, (dy * xh).sum(0), nt * (dy * xh).abs().sum(0) + (dy.abs() * exh).sum(0))
    within(db, dy.sum(0), nt * dy.abs().sum(0))


@pytest.mark.parametrize("x", [BF, F32])
@pytest.mark.parametrize("ox,oy,pad_x,pad_y", [(1, 1, 0, 0), (3, 3, 9, 17), (0, 1, 0, 0), (2, 1, 1, 4), (5, 0, 3, 0)])
@pytest.mark.parametrize("T,k", [(3, 1), (40, 5), (9000, 33), (3000, 259), (700, 2050), (40, 4098), (330, 6001), (9, 16384)])
def test_norm_forward_rows_on_any_place(T, k, ox, oy, pad_x, pad_y, x):
    """X and Y may start on the same place between two 16-byte boundaries or on different ones, rows too."""
    g = gen(T + 7 * k)
    X = randn(g, T, k, dtype=x) + 0.25
    gamma, beta = randn(g, k), randn(g, k)
    eps = 1e-5
    mean, rstd = (torch.full((T,), float("nan"), device=DEV) for _ in range(2))
    Xp = rows(X, k + pad_x, ox)
    buf = torch.full((oy + T * (k + pad_y) + 16,), 7.0, dtype=x, device=DEV)
    Y = torch.as_strided(buf, (T, k), (k + pad_y, 1), oy)
    rgs.layer_norm_forward(Xp, gamma, beta, Y, mean, rstd, eps=eps)
    y, m, r = norm64(X, gamma, beta, eps)
    dmean, drel = norm_bounds(X, eps, k)
    within(mean, m, dmean + 1e-30)
    within(rstd, r, drel * r)
    xh = (X.to(F64) - m[:, None]).abs() * r[:, None]
    bound = ((dmean * r)[:, None] + xh * (drel[:, None] + 2.0 ** -22)) * gamma.to(F64).abs()
    bound = bound + (y.abs() + beta.to(F64).abs()) * 2.0 ** -23
    within(Y, y, bound * 1.01 + y.abs() * (2.0 ** -8 if x == BF else 0.0) + 1e-30)
    kept = torch.zeros(buf.numel(), dtype=torch.bool, device=DEV)
    torch.as_strided(kept, Y.shape, Y.stride(), oy).fill_(True)
    assert (buf[~kept] == 7.0).all()


@pytest.mark.parametrize("x", [BF, F32])
@pytest.mark.parametrize("offsets,pads", [((1, 1, 1), (0, 0, 0)), ((3, 3, 3), (1, 9, 17)), ((0, 1, 0), (0, 0, 0)),
                                          ((2, 2, 1), (3, 3, 2)), ((0, 0, 0), (2, 2, 10))])
@pytest.mark.parametrize("T,k", [(7, 33), (8, 16), (9000, 37), (3000, 261), (700, 2051), (400, 4098), (330, 6001),
                                 (17, 16381)])
def test_norm_backward_rows_on_any_place(T, k, offsets, pads, x):
    """dY, X and dX may start on the same place between two 16-byte boundaries or on different ones, rows too."""
    g = gen(T + 11 * k)
    X, dY, gamma = randn(g, T, k, dtype=x), randn(g, T, k, dtype=x), randn(g, k)
    eps = 1e-3
    _, m, r = norm64(X, None, None, eps)
    mean, rstd = m.float(), r.float()
    dx, dg, db, xh, d, r = norm_grads64(dY, X, gamma, eps)
    bufs, views = [], []
    for t, o, p in zip((X, dY, torch.zeros_like(X)), offsets, pads):
        buf = torch.full((o + T * (k + p) + 16,), float("nan"), dtype=x, device=DEV)
        view = torch.as_strided(buf, (T, k), (k + p, 1), o)
        view.copy_(t)
        bufs.append(buf)
        views.append(view)
    Xp, dYp, dX = views
    dgamma, dbeta = torch.empty(k, device=DEV), torch.empty(k, device=DEV)
    rgs.layer_norm_backward(dYp, Xp, gamma, mean, rstd, dX, dgamma, dbeta, overwrite=True)
    exh = 2.0 ** -22 * (xh.abs() + (m.abs() * r)[:, None])
    n = (k + 16) * 2.0 ** -24
    e0 = n * d.abs().mean(1, keepdim=True)
    e1 = n * (d * xh).abs().mean(1, keepdim=True) + (d.abs() * exh).mean(1, keepdim=True)
    s1 = (d * xh).mean(1, keepdim=True).abs()
    ex = r[:, None] * (e0 + exh * s1 + xh.abs() * e1 + 2.0 ** -21 * (d.abs() + d.mean(1, keepdim=True).abs() + xh.abs() * s1))
    within(dX, dx, ex * 1.01 + (dx.abs() * 2.0 ** -8 if x == BF else 0.0) + 1e-30)
    nt = (T + 16) * 2.0 ** -24
    within(dgamma, dg, nt * (dY.to(F64) * xh).abs().sum(0) + (dY.to(F64).abs() * exh).sum(0) + 1e-30)
    within(dbeta, db, nt * dY.to(F64).abs().sum(0) + 1e-30)
    kept = torch.zeros(bufs[2].numel(), dtype=torch.bool, device=DEV)
    torch.as_strided(kept, dX.shape, dX.stride(), offsets[2]).fill_(True)
    assert torch.isnan(bufs[2][~kept]).all()


def test_norm_gradient_against_differences():
    """<dX, u>, <dgamma, a> and <dbeta, b> against central differences of sum(dY * LN(X)) in 64 bits."""
    g = gen(11)
    T, k, eps = 5, 48, 1e-3
    X, dY, gamma, beta = randn(g, T, k), randn(g, T, k), randn(g, k), randn(g, k)
    mean, rstd = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    Y, dX, dg, db = torch.empty_like(X), torch.empty_like(X), torch.empty(k, device=DEV), torch.empty(k, device=DEV)
    rgs.layer_norm_forward(X, gamma, beta, Y, mean, rstd, eps=eps)
    rgs.layer_norm_backward(dY, X, gamma, mean, rstd, dX, dg, db, overwrite=True)
    for t, grad in ((X, dX), (gamma, dg), (beta, db)):
        u = randn(g, *t.shape).to(F64)
        h = 1e-5

        def f(s):
            a = [v.to(F64) + s * u if v is t else v.to(F64) for v in (X, gamma, beta)]
            return (dY.to(F64) * norm64(a[0], a[1], a[2], eps)[0]).sum().item()

        diff = (f(h) - f(-h)) / (2 * h)
        # differences: h^2 of the third derivative, 1e-16 / h of f; the gradient: 2^-20 of its terms
        assert abs(diff - (grad.to(F64) * u).sum().item()) < 1e-7 * abs(f(0)) + 2.0 ** -18 * (grad.to(F64) * u).abs().sum().item()


def test_norm_passes_2_to_31_elements():
    T, k = 1_100_000, 2048
    X = torch.empty(T, k, dtype=BF, device=DEV).normal_(generator=gen(3))
    Y, mean, rstd = torch.empty_like(X), torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    gamma = randn(gen(4), k)
    rgs.layer_norm_forward(X, gamma, None, Y, mean, rstd)
    dg = torch.empty(k, device=DEV)
    dX = torch.empty_like(X)
    rgs.layer_norm_backward(Y, X, gamma, mean, rstd, dX, dg, overwrite=True)
    for at in (slice(0, 3), slice(T // 2, T // 2 + 3), slice(T - 3, T)):
        y, _, _ = norm64(X[at], gamma, None, 1e-5)
        within(Y[at], y, y.abs() * 2.0 ** -8 + 1e-4)
        dx = norm_grads64(Y[at], X[at], gamma, 1e-5)[0]
        within(dX[at], dx, dx.abs() * 2.0 ** -8 + 1e-3)
    assert torch.isfinite(dg).all()


# ---- cross entropy ------------------------------------------------------------------

def ce_inputs(T, k, V, seed=0, ignored=0.2):
    g = gen(seed * 1000003 + T * 101 + k * 7 + V)
    W = randn(g, V, k, std=0.05, dtype=BF)
    targets = torch.randint(0, V, (T,), generator=g, device=DEV)
    X = (randn(g, T, k) + 4.0 / (k * 0.05 ** 2) ** 0.5 * W[targets].float()).to(BF)
    targets = torch.where(torch.rand(T, generator=g, device=DEV) < ignored, torch.full_like(targets, -100), targets)
    up = randn(g, T, std=1.0 / T)
    return X, W, targets, up


def ce64(X, W, targets, scale):
    """Logits, lse, loss and the bound on a logit's error: each 16-wide step of the sum over k."""
    x, w = X.to(F64), W.to(F64)
    logits = scale * (x @ w.t())
    elog = scale * (X.shape[1] / 16 + 4) * 2.0 ** -23 * (x.abs() @ w.abs().t())
    lse = torch.logsumexp(logits, 1)
    hit = logits.gather(1, targets.clamp(min=0)[:, None])[:, 0]
    return logits, elog, lse, torch.where(targets >= 0, lse - hit, 0.0)


CE_SHAPES = [(1, 8, 1), (1, 8, 2), (2, 64, 127), (5, 72, 128), (3, 64, 129), (16, 128, 1000), (127, 64, 257),
             (128, 256, 256), (129, 64, 255), (200, 200, 515), (255, 512, 777), (257, 136, 3000), (300, 1024, 2049),
             (1000, 64, 5003)]


@pytest.mark.parametrize("scale", [1.0, 0.7])
@pytest.mark.parametrize("T,k,V", CE_SHAPES)
def test_cross_entropy_forward(T, k, V, scale):
    X, W, targets, _ = ce_inputs(T, k, V)
    loss, lse = torch.full((T,), float("nan"), device=DEV), torch.full((T,), float("nan"), device=DEV)
    status = torch.full((1,), -1, dtype=torch.int32, device=DEV)
    rgs.cross_entropy_forward(X, W, targets, loss, lse, scale=scale, dev_status=status)
    logits, elog, want, want_loss = ce64(X, W, targets, scale)
    bound = elog.amax(1) + 2.0 ** -20 * (1 + want.abs() + logits.abs().amax(1)) + V * 2.0 ** -24
    within(lse, want, bound)
    within(loss, want_loss, 2 * bound)
    assert torch.equal(loss[targets < 0], torch.zeros_like(loss[targets < 0]))
    assert status.item() == 0


def ce_grads64(X, W, targets, up, lse, scale):
    """dX, dW and elementwise bounds on D = g scale (softmax - onehot), 64-bit, from the given lse."""
    x, w = X.to(F64), W.to(F64)
    logits, elog, _, _ = ce64(X, W, targets, scale)
    p = torch.exp(logits - lse.to(F64)[:, None])
    kept = targets >= 0
    d = p.clone()
    d[torch.arange(len(x), device=DEV), targets.clamp(min=0)] -= 1.0
    weight = (up.to(F64) * scale).abs()[:, None]
    d = d * (up.to(F64) * scale)[:, None]
    # the exponential: the logit's error, 2^-21 of it and of lse; the subtraction and product: 2^-23; BF16: 2^-8
    ed = weight * (p * (torch.expm1(elog) + 2.0 ** -21 * (1 + logits.abs() + lse.to(F64).abs()[:, None])) + 2.0 ** -22)
    ed = ed + (d.abs() + ed) * 2.0 ** -8
    d, ed = (torch.where(kept[:, None], t, 0.0) for t in (d, ed))
    return d, ed, x, w


def product_bound(da, ea, b):
    """Error of a product whose left factor is off by ea, summed in steps of 16 in fp32."""
    n = (da.shape[1] / 16 + 8) * 2.0 ** -23
    return (ea + n * da.abs()) @ b.abs()


@pytest.mark.parametrize("dw", [BF, F32])
@pytest.mark.parametrize("T,k,V", CE_SHAPES)
def test_cross_entropy_backward(T, k, V, dw):
    X, W, targets, up = ce_inputs(T, k, V, seed=1)
    scale = 0.8
    _, _, lse, _ = ce64(X, W, targets, scale)
    lse = lse.float()
    d, ed, x, w = ce_grads64(X, W, targets, up, lse, scale)
    dX, dW = torch.full_like(X, float("nan")), torch.full((V, k), float("nan"), dtype=dw, device=DEV)
    status = torch.full((1,), -1, dtype=torch.int32, device=DEV)
    rgs.cross_entropy_backward(X, W, targets, lse, up, dX=dX, dW=dW, overwrite=True, scale=scale, dev_status=status)
    assert status.item() == 0
    want = d @ w
    bx = product_bound(d, ed, w) + 1e-30
    within(dX, want, bx * 1.01 + want.abs() * 2.0 ** -8)
    assert (dX[targets < 0] == 0).all()
    wantw = d.t() @ x
    bw = product_bound(d.t(), ed.t(), x) + 1e-30
    within(dW, wantw, bw * 1.01 + (wantw.abs() * 2.0 ** -8 if dw == BF else wantw.abs() * 2.0 ** -22))
    # each gradient alone: the same bits; an fp32 dW can be added to
    alone = torch.empty_like(dX)
    rgs.cross_entropy_backward(X, W, targets, lse, up, dX=alone, scale=scale)
    assert torch.equal(alone, dX)
    again = dW.clone()
    rgs.cross_entropy_backward(X, W, targets, lse, up, dW=again, scale=scale)
    assert torch.equal(again, dW if dw == BF else dW + dW)


def test_cross_entropy_head_sketch():
    """C (+)= D^T XP: against D in 64 bits, and the same bits from repeated calls."""
    T, k, V, r = 300, 256, 1500, 24
    X, W, targets, up = ce_inputs(T, k, V, seed=2)
    XP = randn(gen(9), T, 32, dtype=BF)[:, :r]
    _, _, lse, _ = ce64(X, W, targets, 1.0)
    lse = lse.float()
    d, ed, _, _ = ce_grads64(X, W, targets, up, lse, 1.0)
    C, dX = torch.full((V, r), float("nan"), device=DEV), torch.empty_like(X)
    rgs.cross_entropy_backward(X, W, targets, lse, up, dX=dX, XP=XP, C=C, overwrite=True)
    want = d.t() @ XP.to(F64)
    within(C, want, product_bound(d.t(), ed.t(), XP.to(F64)) * 1.01 + 1e-30)
    twice = C.clone()
    rgs.cross_entropy_backward(X, W, targets, lse, up, XP=XP, C=twice)
    assert torch.equal(twice, C + C)
    only = torch.empty_like(X)
    rgs.cross_entropy_backward(X, W, targets, lse, up, dX=only)
    assert torch.equal(only, dX)


@pytest.mark.parametrize("V", [20000, 70001])
@pytest.mark.parametrize("T", [3, 48])
def test_cross_entropy_equal_weights_keep_the_targets_entries(T, V):
    """The mean over tokens: -g (1 - p) of a target keeps its value to p or 2^-9 of g, whatever g's last bits are."""
    k, r, up = 128, 16, 1.0 / 3.0
    g = gen(T + V)
    X, W, XP = randn(g, T, k, dtype=BF), randn(g, V, k, std=0.02, dtype=BF), randn(g, T, r, dtype=BF)
    targets = torch.randint(0, V, (T,), generator=g, device=DEV)
    ups = torch.full((T,), up, device=DEV)
    x, w = X.to(F64), W.to(F64)
    logits = x @ w.t()
    lse = torch.logsumexp(logits, 1)
    p = torch.exp(logits - lse[:, None])
    hit = torch.zeros(T, V, dtype=torch.bool, device=DEV)
    hit[torch.arange(T, device=DEV), targets] = True
    d = (p - hit.to(F64)) * float(ups[0])
    # p from fp32 logits (magnitudes below 64) and fp32 exponentials: 2^-15; BF16: 2^-8 of p, of 1 - p at most p or 2^-9
    ed = float(ups[0]) * (p * 2.0 ** -15 + torch.where(hit, p.clamp(max=2.0 ** -9), p * 2.0 ** -8) + 2.0 ** -22)
    dX, dW, C = torch.empty_like(X), torch.empty(V, k, device=DEV), torch.empty(V, r, device=DEV)
    rgs.cross_entropy_backward(X, W, targets, lse.float(), ups, dX=dX, dW=dW, overwrite=True)
    rgs.cross_entropy_backward(X, W, targets, lse.float(), ups, XP=XP, C=C, overwrite=True)
    for got, b in ((dW, x), (C, XP.to(F64))):
        want = d.t() @ b
        within(got, want, product_bound(d.t(), ed.t(), b) * 1.01 + want.abs() * 2.0 ** -22 + 1e-30)
    want = d @ w
    within(dX, want, product_bound(d, ed, w) * 1.01 + want.abs() * 2.0 ** -8)


@pytest.mark.parametrize("T,V", [(1, 40), (3, 700), (128, 1300), (129, 700), (2, 140001)])
def test_cross_entropy_gradients_beyond_bf16_logit_gradients(T, V):
    """dX has its tokens' target entries in fp32; up to 128 tokens, dW and C have every entry in two BF16 terms."""
    k, r = 136, 24
    X, W, targets, up = ce_inputs(T, k, V, seed=8, ignored=0.2 if T > 3 else 0.0)
    XP = randn(gen(9), T, r, dtype=BF)
    _, elog, lse, _ = ce64(X, W, targets, 1.0)
    lse = lse.float()
    d, _, x, w = ce_grads64(X, W, targets, up, lse, 1.0)
    kept = targets >= 0
    p = torch.exp(x @ w.t() - lse.to(F64)[:, None])
    logits = x @ w.t()
    # as ce_grads64 has it, before the rounding to BF16
    ed = up.to(F64).abs()[:, None] * (p * (torch.expm1(elog) + 2.0 ** -21 * (1 + logits.abs() + lse.to(F64).abs()[:, None]))
                                      + 2.0 ** -22)
    ed = torch.where(kept[:, None], ed, 0.0)
    hit = torch.zeros(T, V, dtype=torch.bool, device=DEV)
    hit[torch.arange(T, device=DEV), targets.clamp(min=0)] = True
    hit &= kept[:, None]
    dX, dW, C = torch.empty_like(X), torch.empty(V, k, device=DEV), torch.empty(V, r, device=DEV)
    rgs.cross_entropy_backward(X, W, targets, lse, up, dX=dX, dW=dW, overwrite=True)
    again = torch.empty_like(X)
    rgs.cross_entropy_backward(X, W, targets, lse, up, dX=again, XP=XP, C=C, overwrite=True)
    assert torch.equal(dX, again)
    want = d @ w
    ex = ed + torch.where(hit, 2.0 ** -20, 2.0 ** -8) * (d.abs() + ed)
    within(dX, want, product_bound(d, ex, w) * 1.01 + want.abs() * 2.0 ** -8 + 1e-30)
    if T > 128:
        return
    ew = ed + 2.0 ** -16 * (d.abs() + ed)
    for got, b in ((dW, x), (C, XP.to(F64))):
        want = d.t() @ b
        within(got, want, product_bound(d.t(), ew.t(), b) * 1.01 + want.abs() * 2.0 ** -22 + 1e-30)


def test_cross_entropy_weights_of_every_size():
    """Zero, tiny, huge, infinite and NaN weights: each token's dX follows its own weight."""
    T, k, V = 6, 64, 700
    X, W, targets, _ = ce_inputs(T, k, V, seed=6)
    targets = targets.clamp(min=0)
    _, _, lse, _ = ce64(X, W, targets, 1.0)
    lse = lse.float()
    nan, inf = float("nan"), float("inf")
    zero = torch.zeros(T, device=DEV)
    dX, dW = torch.full_like(X, nan), torch.full_like(W, nan)
    rgs.cross_entropy_backward(X, W, targets, lse, zero, dX=dX, dW=dW, overwrite=True)
    assert (dX == 0).all() and (dW == 0).all()
    for weights in ([1e-30] * T, [1e30, 3e29, -1e30, 0.0, 7e28, 1e30], [1.0, inf, -0.5, 0.25, 0.0, 3.0],
                    [nan, 1.0, 1.0, nan, 2.0, 0.5]):
        up = torch.tensor(weights, device=DEV)
        fine = torch.isfinite(up)
        d, ed, x, w = ce_grads64(X, W, targets, torch.where(fine, up, 0.0), lse, 1.0)
        dX = torch.empty_like(X)
        rgs.cross_entropy_backward(X, W, targets, lse, up, dX=dX)
        want = d @ w
        within(dX[fine], want[fine], (product_bound(d, ed, w) * 1.01 + want.abs() * 2.0 ** -8 + 1e-37)[fine])
        assert not torch.isfinite(dX[~fine]).any()


def test_cross_entropy_in_pieces_of_the_vocabulary():
    """Sizes whose logit gradients take several pieces, the last one ragged."""
    T, k, V = 8200, 64, 40_003
    X, W, targets, up = ce_inputs(T, k, V, seed=3)
    pieces = binding.workspace_bytes(binding.OP_CROSS_ENTROPY_BACKWARD, T, V, k, 0)
    assert pieces < 2 * T * V  # in pieces, or it would hold all T x V BF16 values twice over
    loss, lse = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    rgs.cross_entropy_forward(X, W, targets, loss, lse)
    logits, elog, want, want_loss = ce64(X, W, targets, 1.0)
    bound = elog.amax(1) + 2.0 ** -20 * (1 + want.abs() + logits.abs().amax(1)) + V * 2.0 ** -24
    within(lse, want, bound)
    within(loss, want_loss, 2 * bound)
    del logits, elog
    d, ed, x, w = ce_grads64(X, W, targets, up, lse, 1.0)
    r = 16
    XP = randn(gen(10), T, r, dtype=BF)
    for out_type in (BF, F32):
        dX, dW = torch.empty_like(X), torch.empty(V, k, dtype=out_type, device=DEV)
        C = torch.empty(V, r, device=DEV)
        rgs.cross_entropy_backward(X, W, targets, lse, up, dX=dX, dW=dW, XP=XP, C=C, overwrite=True)
        want = d @ w
        within(dX, want, product_bound(d, ed, w) * 1.01 + want.abs() * 2.0 ** -8 + 1e-30)
        want = d.t() @ x
        within(dW, want, product_bound(d.t(), ed.t(), x) * 1.01 + want.abs() * (2.0 ** -8 if out_type == BF else 2.0 ** -22) + 1e-30)
        want = d.t() @ XP.to(F64)
        within(C, want, product_bound(d.t(), ed.t(), XP.to(F64)) * 1.01 + 1e-30)


@pytest.mark.parametrize("T,k,V", [(20001, 64, 300), (9000, 8, 1300), (640, 4096, 300), (40, 512, 70001)])
def test_cross_entropy_long_and_narrow(T, k, V):
    """Many tokens (blocks of the gather that take several rows a warp), wide rows, and a vocabulary split for dX."""
    X, W, targets, up = ce_inputs(T, k, V, seed=11, ignored=0.5)
    loss, lse = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    rgs.cross_entropy_forward(X, W, targets, loss, lse)
    logits, elog, want, want_loss = ce64(X, W, targets, 1.0)
    bound = elog.amax(1) + 2.0 ** -20 * (1 + want.abs() + logits.abs().amax(1)) + V * 2.0 ** -24
    within(lse, want, bound)
    within(loss, want_loss, 2 * bound)
    del logits, elog
    dX, dW = torch.full_like(X, float("nan")), torch.full_like(W, float("nan"))
    rgs.cross_entropy_backward(X, W, targets, lse, up, dX=dX, dW=dW)
    d, ed, x, w = ce_grads64(X, W, targets, up, lse, 1.0)
    want = d @ w
    within(dX, want, product_bound(d, ed, w) * 1.01 + want.abs() * 2.0 ** -8 + 1e-30)
    assert (dX[targets < 0] == 0).all()
    want = d.t() @ x
    within(dW, want, product_bound(d.t(), ed.t(), x) * 1.01 + want.abs() * 2.0 ** -8 + 1e-30)


@pytest.mark.parametrize("V", [100, 3000])
def test_cross_entropy_all_ignored_and_poisoned_rows(V):
    """No kept token: zero gradients.  NaN and infinities in ignored rows reach nothing."""
    T, k = 140, 64
    X, W, targets, up = ce_inputs(T, k, V, seed=4)
    none = torch.full_like(targets, -1)
    loss, lse = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    XP = randn(gen(1), T, 8, dtype=BF)
    nan = float("nan")
    bad = X.clone()
    bad[targets < 0] = nan
    bad[(targets < 0).nonzero()[0, 0]] = float("inf")
    bad_xp = XP.clone()
    bad_xp[targets < 0] = nan
    bad_lse_up = up.clone()
    bad_lse_up[targets < 0] = nan
    rgs.cross_entropy_forward(X, W, none, loss, lse)
    assert torch.equal(loss, torch.zeros_like(loss)) and torch.isfinite(lse).all()
    outs = []
    for x, xp, t, g in ((X, XP, none, up), (X, XP, targets, up), (bad, bad_xp, targets, bad_lse_up)):
        dX, dW, C = torch.full_like(X, nan), torch.full_like(W, nan), torch.full((V, 8), nan, device=DEV)
        rgs.cross_entropy_backward(x, W, t, lse, g, dX=dX, dW=dW, XP=xp, C=C, overwrite=True)
        outs.append((dX, dW, C))
    for t in outs[0]:
        assert (t == 0).all()
    for a, b in zip(outs[1], outs[2]):
        assert torch.isfinite(a).all() and torch.equal(a, b)
    rgs.cross_entropy_forward(bad, W, targets, loss, lse)
    assert torch.isfinite(loss).all() and torch.isfinite(lse[targets >= 0]).all()


def test_cross_entropy_flags_targets_past_the_vocabulary():
    T, k, V = 40, 64, 300
    X, W, targets, up = ce_inputs(T, k, V, seed=5, ignored=0.0)
    bad = targets.clone()
    bad[3], bad[39] = V, 1 << 40
    ok = torch.ones(T, dtype=torch.bool, device=DEV)
    ok[3] = ok[39] = False
    loss, lse, good, _ = (torch.empty(T, device=DEV) for _ in range(4))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    rgs.cross_entropy_forward(X, W, targets, good, lse)
    rgs.cross_entropy_forward(X, W, bad, loss, lse, dev_status=status)
    assert status.item() == binding.DEV_BAD_TARGET
    assert torch.isnan(loss[~ok]).all() and torch.equal(loss[ok], good[ok])
    masked = torch.where(ok, targets, -1)
    outs = []
    for t in (bad, masked):
        dX, dW = torch.empty_like(X), torch.empty_like(W)
        rgs.cross_entropy_backward(X, W, t, lse, up, dX=dX, dW=dW, dev_status=status)
        outs.append((dX, dW, status.item()))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert (outs[0][2], outs[1][2]) == (binding.DEV_BAD_TARGET, 0)


def test_cross_entropy_strided_rows_and_extreme_logits():
    """Row strides past the width; logits of +-3e4, whose exponentials overflow unshifted; a -inf column."""
    T, k, V = 70, 72, 500
    X, W, targets, up = ce_inputs(T, k, V, seed=6)
    X = (X.float() * 200).to(BF)
    W[7] = 0
    Xs, Ws = rows(X, 96), rows(W, 80)
    outs = []
    for x, w in ((X, W), (Xs, Ws)):
        loss, lse = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
        rgs.cross_entropy_forward(x, w, targets, loss, lse)
        dX, dW = rows(torch.zeros_like(X), 88), rows(torch.zeros_like(W), 104)
        rgs.cross_entropy_backward(x, w, targets, lse, up, dX=dX, dW=dW)
        assert torch.isnan(dX._base.view(T, 88)[:, k:]).all() and torch.isnan(dW._base.view(V, 104)[:, k:]).all()
        outs.append((loss, lse, dX, dW))
    for a, b in zip(*outs):
        assert torch.isfinite(a).all() and torch.equal(a, b)
    logits, elog, want, want_loss = ce64(X, W, targets, 1.0)
    bound = elog.amax(1) + 2.0 ** -20 * (1 + want.abs() + logits.abs().amax(1)) + V * 2.0 ** -24
    within(outs[0][1], want, bound)
    within(outs[0][0], want_loss, 2 * bound)


def test_cross_entropy_gradient_against_differences():
    """<dX, u> and <dW, u> against central differences of sum(g loss) in 64 bits, within the gradient's bounds."""
    T, k, V = 24, 64, 200
    X, W, targets, up = ce_inputs(T, k, V, seed=7)
    loss, lse = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    rgs.cross_entropy_forward(X, W, targets, loss, lse, scale=0.9)
    dX, dW = torch.empty_like(X), torch.empty(V, k, device=DEV)
    rgs.cross_entropy_backward(X, W, targets, lse, up, dX=dX, dW=dW, overwrite=True, scale=0.9)
    d, ed, x, w = ce_grads64(X, W, targets, up, lse, 0.9)
    else_ = (ce64(X, W, targets, 0.9)[2] - lse.to(F64)).abs().max().item()
    h = 1e-4
    for which, grad, bound in (("X", dX, product_bound(d, ed + d.abs() * else_, w) + dX.to(F64).abs() * 2.0 ** -8),
                               ("W", dW, product_bound(d.t(), (ed + d.abs() * else_).t(), x))):
        u = randn(gen(8), *grad.shape).to(F64)

        def f(s):
            a, b = (x + s * u, w) if which == "X" else (x, w + s * u)
            return (up.to(F64) * ce64(a, b, targets, 0.9)[3]).sum().item()

        diff = (f(h) - f(-h)) / (2 * h)
        assert abs(diff - (grad.to(F64) * u).sum().item()) < (bound * u.abs()).sum().item() + 1e-6


def test_cross_entropy_head_past_2_to_31_weights():
    T, k, V = 40, 2048, 1_100_000
    W = torch.empty(V, k, dtype=BF, device=DEV).normal_(std=0.02, generator=gen(1))
    X = randn(gen(2), T, k, dtype=BF)
    targets = torch.randint(V - 1000, V, (T,), generator=gen(3), device=DEV)
    loss, lse, up = torch.empty(T, device=DEV), torch.empty(T, device=DEV), randn(gen(4), T)
    rgs.cross_entropy_forward(X, W, targets, loss, lse)
    want = torch.stack([torch.logsumexp(X.to(F64) @ W[v:v + 100_000].to(F64).t(), 1) for v in range(0, V, 100_000)])
    want = torch.logsumexp(want, 0)
    hit = (X.to(F64) * W[targets].to(F64)).sum(1)
    # a logit is off by (k/16 + 4) 2^-23 sum|x||w|, here at most about 132 * 1.2e-7 * 30
    within(lse, want, 6e-4)
    within(loss, want - hit, 1.2e-3)
    dX, dW = torch.empty_like(X), torch.full_like(W, float("nan"))
    rgs.cross_entropy_backward(X, W, targets, lse, up, dX=dX, dW=dW)
    for at in (slice(0, 64), slice(V // 2, V // 2 + 64), slice(V - 64, V)):
        d = torch.exp(X.to(F64) @ W[at].to(F64).t() - lse.to(F64)[:, None])
        hits = (targets[:, None] == torch.arange(V, device=DEV)[at][None])
        d = (d - hits.to(F64)) * up.to(F64)[:, None]
        want = d.t() @ X.to(F64)
        within(dW[at], want, want.abs() * 2.0 ** -8 + (2.0 ** -8 + 1e-3) * (d.abs().t() @ X.to(F64).abs()))
    assert torch.isfinite(dX).all()


# ---- AdamW -----------------------------------------------------------------------

def value_bits(t):
    return t.view(torch.int16).to(torch.int32) & 0xFFFF


def random16(n, seed, layer, step, tag):
    """16 random bits a value: lane e % 8 of Philox4x32-10 block e // 8, counter (block, step, layer, tag)."""
    c = [np.arange((n + 7) // 8, dtype=np.uint64)] + [np.full((n + 7) // 8, v, np.uint64) for v in (step, layer, tag)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    mask = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        s = np.uint64(32)
        c = [(p1 >> s) ^ c[1] ^ np.uint64(k[0]), p1 & mask, (p0 >> s) ^ c[3] ^ np.uint64(k[1]), p0 & mask]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    words = np.stack(c, 1)
    lanes = np.stack([words & np.uint64(0xFFFF), words >> np.uint64(16)], 2).reshape(-1)[:n]
    return torch.from_numpy(lanes.astype(np.int64)).to(DEV)


LR, BETAS, EPS, DECAY = 2e-3, (0.9, 0.999), 1e-8, 0.1


def adam64(w, g, m, v, step, scale=1.0):
    g = g.to(F64) * scale
    t = step + 1
    m = BETAS[0] * m + (1 - BETAS[0]) * g
    v = BETAS[1] * v + (1 - BETAS[1]) * g * g
    upd = LR * (m / (1 - BETAS[0] ** t)) / ((v / (1 - BETAS[1] ** t)).sqrt() + EPS)
    return w.to(F64) * (1 - LR * DECAY) - upd, m, v, upd


SIZES = [1, 2, 7, 8, 9, 255, 256, 257, 1000, 2048, 4099, 0, 65537]


def adam_tensors(sizes, w, g, seed=0):
    r = gen(seed)
    Ws = [randn(r, n, std=0.05, dtype=w) for n in sizes]
    Gs = [(randn(r, n) * torch.exp(randn(r, n, std=2.0) - 8)).to(g) for n in sizes]
    return Ws, Gs


@pytest.mark.parametrize("w,g", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)])
def test_adamw_32(w, g):
    Ws, Gs = adam_tensors(SIZES, w, g)
    state = {"m": [randn(gen(i), n, std=1e-3) for i, n in enumerate(SIZES)],
             "v": [randn(gen(50 + i), n, std=1e-3).square() for i, n in enumerate(SIZES)]}
    old = [(a.clone(), b.to(F64), c.to(F64)) for a, b, c in zip(Ws, state["m"], state["v"])]
    layers = [3 * i + 1 for i in range(len(SIZES))]
    opt = rgs.AdamW(Ws, Gs, state=state, betas=BETAS, eps=EPS, weight_decay=DECAY, seed=(7 << 40) + 5, layers=layers)
    opt.step(LR, step=11)
    u = 2.0 ** -24
    for i, n in enumerate(SIZES):
        want, m, v, upd = adam64(old[i][0], Gs[i], old[i][1], old[i][2], 11)
        within(state["m"][i], m, 4 * u * (old[i][1].abs() + Gs[i].to(F64).abs()) + 1e-38)
        within(state["v"][i], v, 6 * u * v + 1e-38)
        # the update: sqrt, division and their factors, and m's own error over v's root
        em = 4 * u * (old[i][1].abs() + Gs[i].to(F64).abs()) / m.abs().clamp(min=1e-38)
        bound = 4 * u * want.abs() + 2 * u * old[i][0].to(F64).abs() + (32 * u + em) * upd.abs()
        if w == F32:
            within(Ws[i], want, bound)
            continue
        # stochastic rounding: the neighbour that the stream's bits choose; a value within its error of a carry may go either way
        lanes = random16(n, (7 << 40) + 5, layers[i], 11, 0)
        lo = (want - bound).float().view(torch.int32).to(torch.int64) & 0xFFFFFFFF
        hi = (want + bound).float().view(torch.int32).to(torch.int64) & 0xFFFFFFFF
        a, b = ((x + lanes) >> 16 for x in (lo, hi))
        got = value_bits(Ws[i])
        first, last = torch.minimum(a, b), torch.maximum(a, b)
        assert ((got >= first) & (got <= last) | ((want - bound) * (want + bound) < 0)).all()
        assert n == 0 or ((a == b).float().mean() > 0.99 or n < 100)  # the choice is fixed almost everywhere


def test_adamw_grad_scale_and_first_step():
    """step 0 of zero states: m / (1 - b1) = g, so that each weight moves by lr sign(g)."""
    Ws, Gs = adam_tensors([3000], F32, F32, seed=1)
    old = Ws[0].clone()
    scale = torch.full((1,), 0.25, device=DEV)
    opt = rgs.AdamW(Ws, Gs, betas=BETAS, eps=1e-30)
    opt.step(LR, step=0, grad_scale=scale)
    within(Ws[0], old.to(F64) - LR * torch.sign(Gs[0].to(F64)), 1e-5 * LR + old.to(F64).abs() * 2.0 ** -23)
    within(opt.state_dict()["m"][0], 0.1 * 0.25 * Gs[0].to(F64), 1e-6 * Gs[0].to(F64).abs() + 1e-38)


def codes64(t):
    return t.to(F32).to(F64)


def e4m3_code(y, lanes):
    """y >= 0 as an E4M3 code, rounded by 16 bits: steps of an eighth of y's power of two, of 2^-9 below 2^-6."""
    y = y.clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** -6))) - 3)
    k = torch.floor(y / step + lanes.to(F64) / 65536)
    return torch.round(torch.where(y < 2.0 ** -6, k, (torch.log2(step) + 9) * 8 + k)).to(torch.int64)


@pytest.mark.parametrize("w,g", [(BF, BF), (BF, F32), (F32, F32)])
def test_adamw_8_bit_states(w, g):
    Ws, Gs = adam_tensors(SIZES, w, g, seed=2)
    opt = rgs.AdamW(Ws, Gs, state_bits=8, betas=BETAS, eps=EPS, weight_decay=DECAY, seed=9)
    s = opt.state_dict()
    for step in range(3):
        held = []
        for i, n in enumerate(SIZES):
            per = [s[x][i].repeat_interleave(256)[:n].to(F64) for x in ("m_scale", "u_scale")]
            held.append((Ws[i].clone(), codes64(s["m"][i]) * per[0], (codes64(s["u"][i]) * per[1]).square()))
        opt.step(LR, step=step)
        for i, n in enumerate(SIZES):
            want, m, v, upd = adam64(held[i][0], Gs[i], held[i][1], held[i][2], step)
            bound = 1e-5 * upd.abs() + want.abs() * (2.0 ** -7 if w == BF else 2.0 ** -22) + 1e-12
            em = 1e-6 * upd.abs() * (held[i][1].abs() + Gs[i].to(F64).abs()) / m.abs().clamp(min=1e-38)
            within(Ws[i], want, bound + em)
            for name, x, sn in (("m", m, "m_scale"), ("u", v.sqrt(), "u_scale")):
                top = torch.zeros((n + 255) // 256 * 256, dtype=F64, device=DEV)
                top[:n] = x.abs()
                top = top.view(-1, 256).amax(1) / 448 if n else top
                within(s[sn][i], top, 1e-5 * top)
                scale = s[sn][i].to(F64).repeat_interleave(256)[:n]
                # the code that the stream's bits choose, for x a relative 4e-6 down and up
                y = torch.where(scale > 0, x.abs() / scale.clamp(min=1e-300), 0.0)
                lanes = random16(n, 9, i, step, 3 if name == "m" else 4)
                a, b = (e4m3_code(y * (1 + side), lanes) for side in (-4e-6, 4e-6))
                if name == "u":
                    a, b = (torch.where(v > 0, c.clamp(min=1), c) for c in (a, b))
                code = s[name][i].view(torch.uint8).to(torch.int64)
                assert ((code & 127 == a) | (code & 127 == b)).all()
                assert ((code >> 7 == 1) == (x < 0)).all()
                assert n < 1000 or (a == b).float().mean() > 0.99
            assert ((codes64(s["u"][i]) > 0) | (v == 0)).all()


def test_adamw_8_bit_rounding_is_unbiased():
    """One value of a state in every block, rounded in many blocks: the codes' mean is the value."""
    n = 256 * 20000
    G = torch.zeros(n, device=DEV)
    G.view(-1, 256)[:, 0] = 4.48          # m = 0.448: scale 1e-3
    x = torch.tensor([0.1234, 0.0317, 1.3e-3, 3.3e-5, 5e-7], device=DEV)
    for j in range(5):
        G.view(-1, 256)[:, 10 + 40 * j] = x[j] * 10
    W = torch.zeros(n, device=DEV)
    opt = rgs.AdamW([W], [G], state_bits=8, betas=(0.9, 0.999), seed=3)
    opt.step(0.0, step=0)
    s = opt.state_dict()
    got = (codes64(s["m"][0]) * s["m_scale"][0].repeat_interleave(256).to(F64)).view(-1, 256)
    for j in range(5):
        col, v = got[:, 10 + 40 * j], x[j].double().item()
        step = max(2.0 ** math.floor(math.log2(v / 1e-3)) / 8, 2.0 ** -9) * 1e-3
        # at most half a step of deviation, 20000 draws: five of their mean's deviations; 2^-16 of a step from the bits' number
        assert abs(col.mean().item() - v) < 5 * 0.5 * step / math.sqrt(20000) + step * 2.0 ** -15 + 1e-6 * v
        assert len(torch.unique(col)) <= 2


def test_adamw_8_bit_moments_follow_small_changes():
    """A second moment of constant gradients converges though each step moves it by less than a code's step."""
    n = 4096
    G = torch.exp(torch.linspace(-3, 3, n, device=DEV))
    W = torch.zeros(n, device=DEV)
    opt = rgs.AdamW([W], [G], state_bits=8, betas=(0.9, 0.99), seed=4)
    for step in range(600):
        opt.step(1e-4, step=step)
    s = opt.state_dict()
    u = codes64(s["u"][0]) * s["u_scale"][0].repeat_interleave(256).to(F64)
    want = G.to(F64) * math.sqrt(1 - 0.99 ** 600)
    # unbiased rounding of u every step, remembered for 1 / (1 - 0.99 / 2) = 200 of them at a relative deviation of at
    # most 1/16: mean over 4096 values of the relative error
    assert abs(((u / want) - 1).mean().item()) < 0.1
    # each step moves a weight by about lr: 600 lr in all
    assert abs((-W / (600 * 1e-4) - 1).mean().item()) < 0.1


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_non_finite_gradients_stay_their_own(bits):
    n = 1000
    Ws, Gs = adam_tensors([n], BF, F32, seed=5)
    bad = Gs[0].clone()
    bad[3], bad[300], bad[999] = float("nan"), float("inf"), float("-inf")
    hit = torch.zeros(n, dtype=torch.bool, device=DEV)
    hit[[3, 300, 999]] = True
    # without them, in the same places, nothing else may change: zeros there keep a block's largest value
    Gs[0][hit] = 0.0
    results = []
    for grad in (Gs[0], bad):
        W = Ws[0].clone()
        opt = rgs.AdamW([W], [grad], state_bits=bits, betas=BETAS, seed=6)
        opt.step(LR, step=0)
        opt.step(LR, step=1)
        results.append([W] + [t[0] for t in opt.state_dict().values()])
    for a, b in zip(*results):
        if a.numel() == n:
            assert torch.equal(a.float()[~hit], b.float()[~hit])
            assert not torch.isfinite(b.float()[hit]).any() or bits == 8 or b is results[1][0]
        else:
            assert torch.equal(a, b)
    assert torch.isnan(results[1][0].float()[hit]).all()


def test_adamw_many_tensors_and_no_others():
    """More tensors than one launch takes; values beside each tensor stay."""
    sizes = [(37 * i) % 600 for i in range(700)]
    starts, at = [], 0
    for n in sizes:
        starts.append(at)
        at += (n + 255) // 256 * 256 + 256
    flat = {d: torch.full((at,), 0.5, dtype=d, device=DEV) for d in (BF, F32)}
    G = randn(gen(1), at)
    state = {"m": torch.zeros(at, device=DEV), "v": torch.zeros(at, device=DEV)}
    part = lambda t: [t[a:a + n] for a, n in zip(starts, sizes)]  # noqa: E731
    held = torch.zeros(at, dtype=torch.bool, device=DEV)
    for a, n in zip(starts, sizes):
        held[a:a + n] = True
    before = binding.kernel_launches()
    rgs.AdamW(part(flat[F32]), part(G), state={k: part(v) for k, v in state.items()}, betas=BETAS).step(0.1, step=0)
    assert binding.kernel_launches() - before == 3
    assert torch.equal(flat[F32][~held], torch.full_like(flat[F32][~held], 0.5))
    g = G[held].to(F64)
    within(flat[F32][held], 0.5 - 0.1 * g / (g.abs() + 1e-8), 1e-5)  # m / (1 - b1) = g, v / (1 - b2) = g^2


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_passes_2_to_32_values(bits):
    n = (1 << 32) + 1000
    W = torch.zeros(n, dtype=BF, device=DEV)
    G = torch.zeros(n, dtype=BF, device=DEV)
    G[-1000:] = 1.0
    G[:1000] = -1.0
    opt = rgs.AdamW([W], [G], state_bits=bits, betas=BETAS, seed=1)
    opt.step(0.125, step=0)
    assert (W[-1000:].float() + 0.125).abs().max().item() <= 0.125 * 2.0 ** -7
    assert (W[:1000].float() - 0.125).abs().max().item() <= 0.125 * 2.0 ** -7
    assert (W[1000:1_000_000] == 0).all() and (W[-1_000_000:-1000] == 0).all()


# ---- all of them -----------------------------------------------------------------

def test_operators_on_another_stream_and_in_a_graph():
    """Calls on a side stream, and captured and replayed, give the bits of plain calls."""
    T, k, V = 200, 256, 1000
    X, W, targets, up = ce_inputs(T, k, V, seed=8)
    gamma, beta = randn(gen(1), k), randn(gen(2), k)

    def everything(stream=None):
        o = {n: torch.empty(T, device=DEV) for n in ("mean", "rstd", "loss", "lse")}
        o.update(Y=torch.empty_like(X), dY=torch.empty_like(X), dX=torch.empty_like(X), dW=torch.empty_like(W),
                 dg=torch.empty(k, device=DEV), db=torch.empty(k, device=DEV))
        ws = {op: torch.empty(binding.workspace_bytes(op, T, V, k, 0 if op == binding.OP_CROSS_ENTROPY_BACKWARD else 1),
                              dtype=torch.uint8, device=DEV)
              for op in (binding.OP_LAYER_NORM_BACKWARD, binding.OP_CROSS_ENTROPY_FORWARD, binding.OP_CROSS_ENTROPY_BACKWARD)}
        Wp, gp = W.clone(), gamma.clone()
        opt = rgs.AdamW([Wp, gp], [o["dW"], o["dg"]], state_bits=8, seed=2)

        def run(stream=None):
            rgs.layer_norm_forward(X, gamma, beta, o["Y"], o["mean"], o["rstd"], stream=stream)
            rgs.cross_entropy_forward(o["Y"], W, targets, o["loss"], o["lse"], ws=ws[binding.OP_CROSS_ENTROPY_FORWARD],
                                      stream=stream)
            rgs.cross_entropy_backward(o["Y"], W, targets, o["lse"], up, dX=o["dY"], dW=o["dW"],
                                       ws=ws[binding.OP_CROSS_ENTROPY_BACKWARD], stream=stream)
            rgs.layer_norm_backward(o["dY"], X, gamma, o["mean"], o["rstd"], o["dX"], o["dg"], o["db"], overwrite=True,
                                    ws=ws[binding.OP_LAYER_NORM_BACKWARD], stream=stream)
            opt.step(1e-3, step=0, stream=stream)
        return run, lambda: [t.clone() for t in o.values()] + [Wp.clone(), gp.clone()] + [
            t.view(torch.uint8).clone() if t.dtype == torch.float8_e4m3fn else t.clone() for ts in opt.state_dict().values() for t in ts]

    run, results = everything()
    run()
    torch.cuda.synchronize()
    want = results()
    run, results = everything()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    run(stream=side)
    side.synchronize()
    for a, b in zip(want, results()):
        assert torch.equal(a, b)
    run, results = everything()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, results()):
        assert torch.equal(a, b)


def test_operators_repeat_bit_for_bit():
    T, k, V = 1000, 520, 6001
    X, W, targets, up = ce_inputs(T, k, V, seed=9)
    runs = []
    for _ in range(3):
        loss, lse, mean, rstd = (torch.empty(T, device=DEV) for _ in range(4))
        dX, dW, dg, db = torch.empty_like(X), torch.empty(V, k, device=DEV), torch.empty(k, device=DEV), torch.empty(k, device=DEV)
        rgs.cross_entropy_forward(X, W, targets, loss, lse)
        rgs.cross_entropy_backward(X, W, targets, lse, up, dX=dX, dW=dW, overwrite=True)
        Y, dN = torch.empty_like(X), torch.empty_like(X)
        rgs.layer_norm_forward(X, None, None, Y, mean, rstd)
        rgs.layer_norm_backward(dX, X, None, mean, rstd, dN, dg, db, overwrite=True)
        runs.append((loss, lse, dX, dW, Y, mean, rstd, dN, dg, db))
    for other in runs[1:]:
        for a, b in zip(runs[0], other):
            assert torch.equal(a, b)


def test_synthetic_recipe_is_shared():
    """The operators take the framework's own activations: D of a head feeds the sketch of its weight."""
    X = synth.layer_x(64, 128, 0, 0, device=DEV)
    W = synth.layer_weight(96, 128, 0, device=DEV)
    targets = torch.arange(64, device=DEV)
    loss, lse = torch.empty(64, device=DEV), torch.empty(64, device=DEV)
    rgs.cross_entropy_forward(X, W, targets, loss, lse)
    assert torch.isfinite(loss).all() and (loss > 0).all()


def test_training_example_learns():
    """Sketched layers, norms, the head's loss and 8-bit AdamW together: a permutation of 1000 tokens is learnt.
    Guessing gives ln 1000 = 6.9."""
    from rank_gradient_sketching_philox_gb300 import train_example
    losses = train_example.main(["--steps", "60", "--tokens", "1024"])
    assert 6.0 < losses[0] < 9.0
    assert losses[-1] < 1.0


# ---- layer norm far from zero ---------------------------------------------------------

# how X's and the outputs' rows lie: contiguous, from an element off a 16-byte boundary alike, or on different places
PLACES = {"whole": (0, 0), "same": (1, 1), "different": (0, 1)}


def placed(t, offset):
    """t's values, contiguous, ``offset`` elements into a buffer."""
    buf = torch.empty(offset + t.numel(), dtype=t.dtype, device=DEV)
    view = buf[offset:].view(t.shape)
    view.copy_(t)
    return view


FAR_SHAPES = [(700, 24), (40, 128), (9, 1000), (300, 1001), (9, 1024), (40, 4096), (9, 5000), (40, 8192), (9, 8200),
              (9, 16384), (3, 16387)]


@pytest.mark.parametrize("x", [BF, F32])
@pytest.mark.parametrize("places", list(PLACES))
@pytest.mark.parametrize("T,k", FAR_SHAPES)
def test_norm_constant_rows_are_their_mean(T, k, places, x):
    """Sums of these values are exact below 2^24, so the mean is the value: xh = 0, Y = beta, dgamma = 0."""
    ox, oy = PLACES[places]
    g = gen(T + 13 * k)
    value = torch.tensor([37.0, 100.0, 255.0, 1000.0], device=DEV)[torch.arange(T, device=DEV) % 4]
    X = placed(value[:, None].expand(T, k).to(x), ox)
    gamma, beta = randn(g, k) + 2.0, randn(g, k)
    mean, rstd = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    Y = placed(torch.full_like(X, float("nan")), oy)
    rgs.layer_norm_forward(X, gamma, beta, Y, mean, rstd, eps=1e-5)
    assert torch.equal(mean, value)
    r = float(torch.tensor(1e-5)) ** -0.5
    within(rstd, torch.full_like(rstd, r).to(F64), r * 2.0 ** -22)
    assert torch.equal(Y, beta.to(x).expand(T, k))
    dY = placed(randn(g, T, k, dtype=x), oy)
    dX, dgamma, dbeta = torch.empty_like(dY), torch.empty(k, device=DEV), torch.empty(k, device=DEV)
    rgs.layer_norm_backward(dY, X, gamma, mean, rstd, dX, dgamma, dbeta, overwrite=True)
    assert torch.equal(dgamma, torch.zeros_like(dgamma))
    # dX = rstd (d - mean(d)): the product, the sum over k, the factors
    d = dY.to(F64) * gamma.to(F64)
    want = rstd.to(F64)[:, None] * (d - d.mean(1, keepdim=True))
    bound = rstd.to(F64)[:, None] * ((k + 16) * 2.0 ** -24 * d.abs().mean(1, keepdim=True) + 2.0 ** -22 * (
        d.abs() + d.mean(1, keepdim=True).abs()))
    within(dX, want, bound * 1.01 + (want.abs() * 2.0 ** -8 if x == BF else 0.0) + 1e-30)


@pytest.mark.parametrize("x,size,spread", [(F32, 1e3, 1.0), (F32, 1e4, 1.0), (BF, 1e3, 8.0)])
@pytest.mark.parametrize("places", list(PLACES))
@pytest.mark.parametrize("T,k", FAR_SHAPES)
def test_norm_rows_far_from_zero(T, k, places, x, size, spread):
    """Means of 100 to 10000 deviations: x - mean is exact, so xh's error stays relative to xh, whatever |mean|."""
    ox, oy = PLACES[places]
    g = gen(T + 17 * k)
    sign = torch.where(torch.arange(T, device=DEV) % 2 == 0, 1.0, -1.0)[:, None]
    X = placed((sign * size + spread * randn(g, T, k)).to(x), ox)
    gamma, beta = randn(g, k), randn(g, k)
    mean, rstd = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    Y = placed(torch.full_like(X, float("nan")), oy)
    rgs.layer_norm_forward(X, gamma, beta, Y, mean, rstd, eps=1e-5)
    _, m, r = norm64(X, None, None, 1e-5)
    dmean, drel = norm_bounds(X, 1e-5, k)
    within(mean, m, dmean)
    # of rstd: the variance around a mean that is off by dmean; a relative error of 2^-20 where that is small
    within(rstd, r, drel * r)
    # with the mean and rstd that the kernel gives: the difference, two products and a sum, each rounded once
    half = 2.0 ** -8 if x == BF else 0.0
    mk, rk = mean.to(F64)[:, None], rstd.to(F64)[:, None]
    xh = (X.to(F64) - mk) * rk
    want = xh * gamma.to(F64) + beta.to(F64)
    bound = 2.0 ** -22 * (xh * gamma.to(F64)).abs() + 2.0 ** -23 * want.abs()
    within(Y, want, bound * 1.01 + want.abs() * half + 1e-30)
    dY = placed(randn(g, T, k, dtype=x), oy)
    dX, dgamma, dbeta = torch.empty_like(dY), torch.empty(k, device=DEV), torch.empty(k, device=DEV)
    rgs.layer_norm_backward(dY, X, gamma, mean, rstd, dX, dgamma, dbeta, overwrite=True)
    dy = dY.to(F64)
    d = dy * gamma.to(F64)
    s0, s1 = d.mean(1, keepdim=True), (d * xh).mean(1, keepdim=True)
    want = rk * (d - s0 - xh * s1)
    n = (k + 16) * 2.0 ** -24
    exh = 2.0 ** -22 * xh.abs()
    e0 = n * d.abs().mean(1, keepdim=True)
    e1 = n * (d * xh).abs().mean(1, keepdim=True) + (d.abs() * exh).mean(1, keepdim=True)
    ex = rk * (e0 + exh * s1.abs() + xh.abs() * e1 + 2.0 ** -21 * (d.abs() + s0.abs() + xh.abs() * s1.abs()))
    within(dX, want, ex * 1.01 + want.abs() * half)
    nt = (T + 16) * 2.0 ** -24
    within(dgamma, (dy * xh).sum(0), nt * (dy * xh).abs().sum(0) + (dy.abs() * exh).sum(0))


# ---- confident tokens ---------------------------------------------------------------

@pytest.mark.parametrize("scale", [1.0, 0.7])
@pytest.mark.parametrize("T", [5, 300])
def test_cross_entropy_small_losses_keep_their_digits(T, scale):
    """Losses of 1e-3 to 1e-9: W has one-hot rows and X one value b, so a token's logits are b scale and zeros."""
    V = k = 1000
    W = torch.eye(V, dtype=BF, device=DEV)
    targets = (torch.arange(T, device=DEV) * 37) % V
    b = (14.0 + torch.arange(T, device=DEV) % 29 * 0.5) / scale
    X = torch.zeros(T, k, dtype=BF, device=DEV)
    X[torch.arange(T, device=DEV), targets] = b.to(BF)
    h = X[torch.arange(T, device=DEV), targets].to(F64) * float(np.float32(scale))
    want = torch.log1p((V - 1) * torch.exp(-h))
    assert want.min() < 2e-9 and want.max() > 5e-4 if T > 29 else want.max() > 5e-4
    loss, lse = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    rgs.cross_entropy_forward(X, W, targets, loss, lse, scale=scale)
    # the exponent h: two roundings and log2(e)'s own, 2.5 * 2^-24 of it; the exponential, logarithm and products 2^-20
    within(loss, want, want * (h * 2.0 ** -22 + 2.0 ** -20))
    within(lse, h + want, 2.0 ** -23 * (h + want))


@pytest.mark.parametrize("T,V", [(20, 300), (300, 300), (20, 5000)])
def test_cross_entropy_small_losses_of_wide_heads(T, V):
    """The same with dense rows over several blocks of columns: the others' logits are off by the sum over k."""
    k = 512
    g = gen(T + V)
    W = randn(g, V, k, std=0.05, dtype=BF)
    targets = torch.randint(0, V, (T,), generator=g, device=DEV)
    X = (W[targets].float() * torch.linspace(14, 22, T, device=DEV)[:, None] / (k * 0.05 ** 2)).to(BF)
    x, w = X.to(F64), W.to(F64)
    logits, elog, lse64, _ = ce64(X, W, targets, 1.0)
    hit = torch.arange(V, device=DEV)[None] == targets[:, None]
    h = logits[hit]
    others = torch.logsumexp(logits.masked_fill(hit, -math.inf), 1)
    want = torch.nn.functional.softplus(others - h)
    assert want.max() < 0.1
    loss, lse = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    rgs.cross_entropy_forward(X, W, targets, loss, lse)
    # the target's logit is an fp32 sum of k terms dealt over 32 lanes
    eh = (k / 32 + 8) * 2.0 ** -24 * (x.abs() * w[targets].abs()).sum(1) + h.abs() * 2.0 ** -22
    e = eh + elog.masked_fill(hit, 0.0).amax(1) + others.abs() * 2.0 ** -22 + V * 2.0 ** -24 + 2.0 ** -20
    within(loss, want, want * torch.expm1(e))
    within(lse, lse64, eh + want * torch.expm1(e) + 2.0 ** -23 * lse64.abs())


@pytest.mark.parametrize("T,V", [(24, 500), (200, 500), (24, 40000)])
def test_cross_entropy_backward_of_confident_tokens(T, V):
    """The target's entry of D is -g (1 - p) with p from the same logit as the forward call's lse: off by lse's own
    rounding, not by the tensor cores' sum over k (about 1.5e-6 of the logit), which for 1 - p of 1e-5 is more than it."""
    k = 4096
    g = gen(3 * T + V)
    W = randn(g, V, k, std=0.02, dtype=BF)
    targets = torch.randint(0, V, (T,), generator=g, device=DEV)
    top = math.log(V)
    X = (W[targets].float() * (top + torch.linspace(8, 12, T, device=DEV)[:, None]) / (k * 0.02 ** 2)).to(BF)
    up = torch.full((T,), 1.0 / T, device=DEV)
    loss, lse = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    rgs.cross_entropy_forward(X, W, targets, loss, lse)
    dX, dW = torch.empty_like(X), torch.empty(V, k, device=DEV)
    rgs.cross_entropy_backward(X, W, targets, lse, up, dX=dX, dW=dW, overwrite=True)
    x, w = X.to(F64), W.to(F64)
    logits, elog, lse64, want = ce64(X, W, targets, 1.0)
    hit = torch.arange(V, device=DEV)[None] == targets[:, None]
    others = torch.logsumexp(logits.masked_fill(hit, -math.inf), 1, keepdim=True)
    assert want.max() < 2e-3
    weight = up.to(F64)[:, None]
    p = torch.exp(logits - lse64[:, None])
    rest = -torch.expm1(-want)[:, None]  # 1 - p of the target
    d = torch.where(hit, -rest, p) * weight
    # p: its logit's error, and 2^-21 of the logit and lse.  The target: relative errors of the others' sum, and lse's
    # rounding (2^-24 of it in the forward call, once more in the difference)
    rel = torch.expm1(elog.masked_fill(hit, 0.0)) + 2.0 ** -21 * (1 + logits.abs() + lse64.abs()[:, None])
    ed = weight * torch.where(hit, rest * (rel.masked_fill(hit, 0.0).amax(1, keepdim=True) + others.abs() * 2.0 ** -20)
                              + 2.0 ** -23 * lse64.abs()[:, None], p * rel)
    ex = ed + torch.where(hit, 2.0 ** -20, 2.0 ** -8) * (d.abs() + ed)
    want = d @ w
    within(dX, want, product_bound(d, ex, w) * 1.01 + want.abs() * 2.0 ** -8 + 1e-30)
    ew = ed + 2.0 ** -8 * (d.abs() + ed)
    want = d.t() @ x
    within(dW, want, product_bound(d.t(), ew.t(), x) * 1.01 + want.abs() * 2.0 ** -22 + 1e-30)


# ---- calls of a fresh process ----------------------------------------------------------

FIRST_CALLS = """
import torch
import rank_gradient_sketching_philox_gb300 as rgs
failed = []
for T, k, offset, dtype in [(4, 768, 0, torch.float32), (64, 1536, 0, torch.bfloat16), (4, 192, 0, torch.bfloat16),
                            (4, 6112, 0, torch.bfloat16), (4, 6100, 0, torch.float32), (4, 6101, 1, torch.bfloat16),
                            (64, 755, 1, torch.bfloat16), (8, 379, 1, torch.float32)]:
    g = torch.Generator(device="cuda").manual_seed(T + k)
    def rows():
        buf = torch.empty(T * k + offset, dtype=dtype, device="cuda").normal_(generator=g)
        return buf[offset:].view(T, k)
    X, dY, Y, dX = rows(), rows(), rows(), rows()
    x, dy = X.double(), dY.double()
    m, r = x.mean(1, keepdim=True), (x.var(1, unbiased=False, keepdim=True) + 1e-5).rsqrt()
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dg, db = torch.empty(k, device="cuda"), torch.empty(k, device="cuda")
    xh = (x - m) * r
    dx = r * (dy - dy.mean(1, keepdim=True) - xh * (dy * xh).mean(1, keepdim=True))
    step = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    def check(*results):
        for got, want, e in results:
            assert ((got.double() - want).abs() <= e * want.abs() + 1e-4 * (1 + want.abs().max())).all(), (T, k)
    try:
        rgs.layer_norm_forward(X, None, None, Y, mean, rstd)
        check((Y, xh, step), (mean, m[:, 0], 0.0), (rstd, r[:, 0], 0.0))
    except rgs.SketchError as e:
        failed.append(("forward", T, k, str(e)))
    try:
        rgs.layer_norm_backward(dY, X, None, m[:, 0].float(), r[:, 0].float(), dX, dg, db, overwrite=True)
        check((dX, dx, step), (dg, (dy * xh).sum(0), 0.0), (db, dy.sum(0), 0.0))
    except rgs.SketchError as e:
        failed.append(("backward", T, k, str(e)))
assert not failed, failed
"""


def test_norm_sizes_whose_shared_memory_is_near_48_kb():
    """First launches of a process, with dynamic shared memory that passes 48 KB only together with the static part."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr[-3000:]


def test_norm_of_two_widths_from_several_threads():
    """Host threads launch one kernel with different amounts of shared memory, each on a stream of its own."""
    call, jobs = binding.lib().sketch_layer_norm_forward, []
    for i in range(8):
        k = (8192, 16384)[i & 1]  # one kernel, 64 and 128 KB
        X = randn(gen(i), 4, k, dtype=BF)
        out, stream = (torch.empty_like(X), torch.empty(4, device=DEV), torch.empty(4, device=DEV)), torch.cuda.Stream()
        args = (X.data_ptr(), binding.DTYPE_BF16, 4, k, k, None, None, binding.DTYPE_FP32, 1e-5, out[0].data_ptr(), k,
                out[1].data_ptr(), out[2].data_ptr(), stream.cuda_stream)
        jobs.append((X, out, args))
    torch.cuda.synchronize()
    start, refused = threading.Barrier(len(jobs)), [0] * len(jobs)

    def work(i):
        start.wait()
        for _ in range(5000):
            refused[i] += call(*jobs[i][2]) != binding.OK

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert refused == [0] * len(jobs)
    for X, out, _ in jobs:
        want, _, _ = norm64(X, None, None, 1e-5)
        within(out[0], want, want.abs() * 2.0 ** -8 + 1e-4)


def test_adamw_refuses_unaligned_tensors_when_it_is_built():
    buf = torch.zeros(72, device=DEV)
    good = lambda: torch.zeros(64, device=DEV)  # noqa: E731
    for bad in range(4):
        ts = [good() for _ in range(4)]
        ts[bad] = buf[1:65]
        with pytest.raises(ValueError, match="16-byte"):
            rgs.AdamW([ts[0]], [ts[1]], state={"m": [ts[2]], "v": [ts[3]]})
    rgs.AdamW([good()], [good()]).step(1e-3, step=0)


# ---- forms beside the usual ones -------------------------------------------------------

@pytest.mark.parametrize("T", [1, 40, 128])
@pytest.mark.parametrize("V", [100, 3000])
def test_cross_entropy_few_tokens_all_ignored(T, V):
    """At most 128 tokens, where every entry of D has two terms, and none is kept: zeros everywhere."""
    k, r = 64, 8
    X, W, _, up = ce_inputs(T, k, V, seed=12)
    none = torch.full((T,), -1, dtype=torch.int64, device=DEV)
    X[0, 0], nan = float("nan"), float("nan")
    XP = randn(gen(1), T, r, dtype=BF)
    lse = torch.zeros(T, device=DEV)
    dX, dW = torch.full_like(X, nan), torch.full((V, k), nan, device=DEV)
    C, status = torch.full((V, r), nan, device=DEV), torch.full((1,), -1, dtype=torch.int32, device=DEV)
    rgs.cross_entropy_backward(X, W, none, lse, up, dX=dX, dW=dW, XP=XP, C=C, overwrite=True, dev_status=status)
    assert (dX == 0).all() and (dW == 0).all() and (C == 0).all() and status.item() == 0
    dW.fill_(2.0)
    rgs.cross_entropy_backward(X, W, none, lse, up, dW=dW)
    assert (dW == 2.0).all()


def test_cross_entropy_forward_of_a_masked_out_entry():
    """A row of W that makes an entry's logit -inf for positive X: as if the entry were not there."""
    T, k, V = 70, 72, 500
    X, W, targets, _ = ce_inputs(T, k, V, seed=13)
    X = X.abs() + 0.25
    targets = torch.where(targets == 7, 8, targets)
    W[7] = -float("inf")
    loss, lse = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    rgs.cross_entropy_forward(X, W, targets, loss, lse)
    keep = torch.arange(V, device=DEV) != 7
    shifted = torch.where(targets > 7, targets - 1, targets)
    logits, elog, want, want_loss = ce64(X, W[keep], shifted, 1.0)
    bound = elog.amax(1) + 2.0 ** -20 * (1 + want.abs() + logits.abs().amax(1)) + V * 2.0 ** -24
    within(lse, want, bound)
    within(loss, want_loss, 2 * bound)


def test_cross_entropy_feeds_the_sketch_of_the_heads_weight():
    """C from the backward call is what accumulate makes of the same D, rounded to BF16, and the projected inputs."""
    T, k, V, r = 64, 128, 96, 16
    X = synth.layer_x(T, k, 0, 0, device=DEV)
    W = synth.layer_weight(V, k, 0, device=DEV)
    targets = torch.arange(T, device=DEV)
    loss, lse = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    rgs.cross_entropy_forward(X, W, targets, loss, lse)
    P = torch.empty(k, r, device=DEV)
    rgs.sample_projection(rgs.PROJ_GAUSSIAN_QR, 3, 0, 0, P)
    XP = torch.empty(T, r, dtype=BF, device=DEV)
    rgs.project_inputs(X, P, XP)
    up = torch.full((T,), 1.0 / T, device=DEV)
    C = torch.full((V, r), float("nan"), device=DEV)
    rgs.cross_entropy_backward(X, W, targets, lse, up, XP=XP, C=C, overwrite=True)
    d, ed, _, _ = ce_grads64(X, W, targets, up, lse, 1.0)
    want = d.t() @ XP.to(F64)
    within(C, want, product_bound(d.t(), ed.t(), XP.to(F64)) * 1.01 + 1e-30)
    D = d.to(F32).to(BF)
    S = torch.empty(V, r, device=DEV)
    rgs.accumulate(D, XP, S, overwrite=True)
    both = product_bound(d.t(), (ed + d.abs() * 2.0 ** -8).t(), XP.to(F64)) * 2.02 + 1e-30
    within(C, S.to(F64), both)


def test_adamw_8_bit_codes_of_values_that_are_not_finite():
    """NaN's code, apart from the sign, in both states: after the step that met the gradient and after the next."""
    n = 1000
    Ws, Gs = adam_tensors([n], BF, F32, seed=5)
    Gs[0][3], Gs[0][300], Gs[0][999] = float("nan"), float("inf"), float("-inf")
    hit = ~torch.isfinite(Gs[0])
    opt = rgs.AdamW(Ws, Gs, state_bits=8, betas=BETAS, seed=6)
    for step in range(2):
        opt.step(LR, step=step)
        for name in ("m", "u"):
            code = opt.state_dict()[name][0].view(torch.uint8).to(torch.int64) & 0x7F
            assert (code[hit] == 0x7F).all() and (code[~hit] < 0x7F).all()
            assert torch.isfinite(opt.state_dict()[name + "_scale"][0]).all()
        assert torch.isnan(Ws[0][hit]).all() and torch.isfinite(Ws[0][~hit]).all()


def test_operators_on_two_streams_at_once():
    """Calls of all operators on two streams side by side give the bits of calls on one."""
    def inputs(seed):
        T, k, V = 300, 512, 5000
        X, W, targets, up = ce_inputs(T, k, V, seed=seed)
        return X, W, targets, up, randn(gen(seed), k)

    def run(X, W, targets, up, gamma, stream=None):
        T, k = X.shape
        o = [torch.empty(T, device=DEV) for _ in range(4)] + [torch.empty_like(X) for _ in range(3)] + [
            torch.empty(W.shape, device=DEV), torch.empty(k, device=DEV), W.clone()]
        mean, rstd, loss, lse, Y, dY, dX, dW, dg, Wn = o
        opt = rgs.AdamW([Wn], [dW], state_bits=8, seed=1)

        def calls():
            rgs.layer_norm_forward(X, gamma, None, Y, mean, rstd, stream=stream)
            rgs.cross_entropy_forward(Y, W, targets, loss, lse, stream=stream)
            rgs.cross_entropy_backward(Y, W, targets, lse, up, dX=dY, dW=dW, overwrite=True, stream=stream)
            rgs.layer_norm_backward(dY, X, gamma, mean, rstd, dX, dg, overwrite=True, stream=stream)
            opt.step(1e-3, step=0, stream=stream)
        return calls, o

    sets = [inputs(s) for s in (21, 22)]
    want = []
    for s in sets:
        calls, o = run(*s)
        calls()
        torch.cuda.synchronize()
        want.append(o)
    streams = [torch.cuda.Stream() for _ in sets]
    made = [run(*s, stream=stream) for s, stream in zip(sets, streams)]
    torch.cuda.synchronize()
    for _ in range(3):  # the weights move on from call to call; the rest is the same each time
        for (calls, o), w in zip(made, want):
            calls()
    torch.cuda.synchronize()
    for (_, o), w in zip(made, want):
        for a, b in zip(o[:-1], w[:-1]):
            assert torch.equal(a, b)
