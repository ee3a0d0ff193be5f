"""The residual stream's norm, the 8-bit products and clipping on the GPU, against plain
64-bit implementations.

Tolerances.  A rounding to a type is off by at most half a step, eps / 2 of the value
(BF16 2^-8, fp32 2^-24, E4M3 2^-4, below 2^-6 2^-10).  A sum of n fp32 terms, added in any
order over at least 256 threads or 32 lanes, is off by at most (longest chain) 2^-24 of
the sum of its magnitudes; the chains below are counted generously.
"""
import math

import pytest
import torch

import rank_gradient_sketching_philox_gb300 as rgs

pytestmark = pytest.mark.gpu
BF, F32, F64, E4 = torch.bfloat16, torch.float32, torch.float64, torch.float8_e4m3fn
U = 2.0 ** -24
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(autouse=True)
def no_device_errors():
    yield
    torch.cuda.synchronize()
    assert rgs.read_device_errors() == 0


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * std


def padded(t, ld=None, before=0):
    """The matrix t with row stride ld, `before` elements behind an allocation's start; NaN around it."""
    T, k = t.shape
    ld = k if ld is None else ld
    store = torch.full((before + T * ld + 16,), math.nan, dtype=t.dtype, device=t.device)
    out = store[before:before + T * ld].view(T, ld)[:, :k]
    out.copy_(t)
    return out


def close(got, want, bound):
    """|got - want| <= bound, elementwise."""
    assert got.shape == want.shape
    over = (got.double() - want.double()).abs() - bound
    assert not torch.isnan(got.double()).any()
    assert float(over.max()) <= 0, "off by %g past the bound" % float(over.max())


def groups(n):
    return (n + 127) // 128


def tops(x, rows):
    """Largest magnitude of each block of `rows` rows and 128 columns (64 bits)."""
    T, k = x.shape
    full = torch.zeros(-(-T // rows) * rows, groups(k) * 128, dtype=F64, device=x.device)
    full[:T, :k] = x.abs()
    return full.view(-1, rows, groups(k), 128).amax((1, 3))


def wide(scale, rows, T, k):
    return scale.double().repeat_interleave(rows, 0)[:T].repeat_interleave(128, 1)[:, :k]


def check_codes(q, scale, y, rows, rel):
    """Codes and scales of y, which the kernel may have seen off by `rel` of a value."""
    T, k = y.shape
    want = (tops(y, rows) / 448.0).clamp(min=2.0 ** -126)
    close(scale, want, want * (rel + 4 * U))
    units = y / wide(want, rows, T, k)
    # half a step, and what the value and its scale may be off
    close(q.double(), units, (units.abs() * 2.0 ** -4).clamp(min=2.0 ** -10) + units.abs() * 2 * (rel + 4 * U))
    # the largest value of a block that is not zero has the largest code
    top = tops(q.double(), rows)
    assert bool(((top == 448.0) | (want == 2.0 ** -126)).all())


# ---- root-mean-square norm -----------------------------------------------------------

NORM_SHAPES = [(1, 1), (1, 64), (3, 127), (2, 128), (5, 129), (4, 1000), (33, 1001), (7, 2048), (70, 4096), (2, 4104),
               (3, 8192), (2, 10001), (2, 16384), (2, 16400), (1, 20001)]


def rms_reference(x, r, gamma, eps):
    s = x.double() + (r.double() if r is not None else 0.0)
    rstd = (s.square().mean(1) + eps).rsqrt()
    y = s * rstd[:, None] * (gamma.double() if gamma is not None else 1.0)
    return s, rstd, y


def chain(k):
    return k / 256 + 64


def check_forward(x, r, gamma, eps, S, Y, Q, scale, rstd):
    s, want_rstd, y = rms_reference(x, r, gamma, eps)
    rel = (chain(x.shape[1]) + 4) * U
    if rstd is not None:
        close(rstd, want_rstd, want_rstd * rel)
    if S is not None:
        close(S, s, s.abs() * HALF[S.dtype])
    if Y is not None:
        close(Y, y, y.abs() * (HALF[Y.dtype] + rel + 4 * U))
    if Q is not None:
        check_codes(Q, scale, y, 1, rel + 4 * U)


@pytest.mark.parametrize("T,k", NORM_SHAPES)
@pytest.mark.parametrize("dtype,w", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("res,quantized", [(True, True), (True, False), (False, True), (False, False)])
def test_rms_forward(T, k, dtype, w, res, quantized):
    g = gen(T * k)
    x = (normal(g, T, k) * torch.exp(normal(g, T, 1))).to(dtype)
    r = normal(g, T, k).to(dtype) if res else None
    gamma = (1 + normal(g, k, std=0.1)).to(w)
    S, Y = (torch.empty_like(x) if res else None), torch.empty_like(x)
    Q = rgs.code_rows(T, k) if quantized else None
    scale = torch.empty(T, groups(k), device="cuda") if quantized else None
    rstd = torch.empty(T, device="cuda")
    rgs.rms_norm_forward(x, gamma, rstd, R=r, S=S, Y=Y, Q=Q, scale=scale)
    check_forward(x, r, gamma, 1e-6, S, Y, Q, scale, rstd)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("k", [40, 264, 1001, 4096])
@pytest.mark.parametrize("place", [0, 1, 3, 8])
def test_rms_forward_any_stride_and_place(dtype, k, place):
    """Rows of every alignment, matrices on different ones; what lies beside them stays."""
    g, T = gen(5), 6
    x = padded(normal(g, T, k).to(dtype), k + place, place)
    r = padded(normal(g, T, k).to(dtype), k + 2 * place, 0)
    S = padded(torch.zeros(T, k, dtype=dtype, device="cuda"), k + place, place)
    Y = padded(torch.zeros(T, k, dtype=dtype, device="cuda"), k + 8, place)
    around = [(t, t.as_strided((T, t.stride(0) - k), t.stride(), t.storage_offset() + k)) for t in (S, Y) if t.stride(0) > k]
    Q = torch.full((T, (k + 15) // 16 * 16 + 16), 1.0, device="cuda").to(E4)
    scale = torch.empty(T, groups(k), device="cuda")
    rgs.rms_norm_forward(x, None, None, R=r, S=S, Y=Y, Q=Q[:, :k], scale=scale, eps=1e-3)
    check_forward(x, r, None, 1e-3, S, Y, Q[:, :k], scale, None)
    for _, beside in around:
        assert bool(torch.isnan(beside.double()).all())
    assert bool((Q[:, k:].double() == 1.0).all())


@pytest.mark.parametrize("k", [1000, 1001, 4096, 16392])
@pytest.mark.parametrize("which", ["S is X", "S is R", "Y is X", "Y is X, S is R"])
def test_rms_forward_in_place(k, which):
    g, T = gen(6), 19
    x, r = normal(g, T, k).to(BF), normal(g, T, k).to(BF)
    x0, r0 = x.clone(), r.clone()
    S = x if which == "S is X" else r if "S is R" in which else torch.empty_like(x)
    Y = x if "Y is X" in which else torch.empty_like(x)
    rgs.rms_norm_forward(x, None, None, R=r, S=S, Y=Y)
    check_forward(x0, r0, None, 1e-6, S, Y, None, None, None)


def test_rms_forward_many_rows():
    """More rows than the launch holds at once, and outputs in 8 bits alone."""
    g, T, k = gen(7), 5003, 264
    x = normal(g, T, k).to(BF)
    Q, scale = rgs.code_rows(T, k), torch.empty(T, groups(k), device="cuda")
    rgs.rms_norm_forward(x, None, None, Q=Q, scale=scale)
    check_forward(x, None, None, 1e-6, None, None, Q, scale, None)


@pytest.mark.parametrize("k", [256, 1001, 20000])
def test_rms_forward_zeros_and_values_that_are_not_finite(k):
    x = torch.ones(5, k, device="cuda")
    x[0] = 0.0                  # a row of zeros: rstd = 1 / sqrt(eps)
    x[1, 3] = math.nan
    x[2, 200] = math.inf
    Y, rstd = torch.empty_like(x), torch.empty(5, device="cuda")
    Q, scale = rgs.code_rows(5, k), torch.empty(5, groups(k), device="cuda")
    rgs.rms_norm_forward(x, None, rstd, Y=Y, Q=Q, scale=scale, eps=1e-4)
    assert float(rstd[0]) == pytest.approx(100.0, rel=1e-6) and bool((Y[0] == 0).all()) and bool((Q[0].float() == 0).all())
    assert bool((scale[0] == 2.0 ** -126).all())
    assert bool(torch.isnan(Y[1]).all()) and bool(torch.isnan(Q[1].float()).all()) and bool(torch.isnan(scale[1]).all())
    # an infinity leaves a rstd of zero: zeros, and a NaN in its own place and block
    assert float(rstd[2]) == 0.0 and bool(torch.isnan(Y[2, 200])) and int(torch.isnan(Y[2]).sum()) == 1
    assert bool(torch.isnan(scale[2, 1])) and bool(torch.isnan(Q[2, 128:min(256, k)].float()).all())
    assert bool((Q[2, :128].float() == 0).all())
    close(Y[3:], torch.ones(2, k, device="cuda"), 1e-4)


def backward_reference(dy, s, gamma, rstd, ds):
    rs = rstd.double()[:, None]
    xh = s.double() * rs
    dxh = dy.double() * (gamma.double() if gamma is not None else 1.0)
    c = (dxh * xh).mean(1, keepdim=True)
    dx = rs * (dxh - xh * c) + (ds.double() if ds is not None else 0.0)
    size = rs * (dxh.abs() + xh.abs() * (c.abs() + (dxh * xh).abs().mean(1, keepdim=True) * chain(s.shape[1])))
    return dx, size, (dy.double() * xh)


def check_backward(dy, s, gamma, rstd, ds, dX, dgamma, before=None):
    dx, size, terms = backward_reference(dy, s, gamma, rstd, ds)
    if dX is not None:
        close(dX, dx, dx.abs() * HALF[dX.dtype] + size * 8 * U + (ds.double().abs() * 2 * U if ds is not None else 0))
    if dgamma is not None:
        want = terms.sum(0) + (before.double() if before is not None else 0.0)
        close(dgamma, want, (terms.abs().sum(0) * (len(s) + 8) + want.abs()) * 2 * U)


@pytest.mark.parametrize("T,k", NORM_SHAPES + [(1021, 1001), (700, 64), (1500, 512)])
@pytest.mark.parametrize("dtype,w", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("res", [True, False])
def test_rms_backward(T, k, dtype, w, res):
    g = gen(T + k)
    s, dy = normal(g, T, k, std=2.0).to(dtype), normal(g, T, k, std=1e-3).to(dtype)
    ds = normal(g, T, k, std=1e-3).to(dtype) if res else None
    gamma = (1 + normal(g, k, std=0.1)).to(w)
    rstd = (s.double().square().mean(1) + 1e-6).rsqrt().float()
    dX, dgamma = torch.empty_like(s), torch.empty(k, device="cuda")
    rgs.rms_norm_backward(dy, s, gamma, rstd, dS=ds, dX=dX, dgamma=dgamma, overwrite=True)
    check_backward(dy, s, gamma, rstd, ds, dX, dgamma)
    before = dgamma.clone()  # added to, without dX
    rgs.rms_norm_backward(dy, s, gamma, rstd, dgamma=dgamma)
    check_backward(dy, s, gamma, rstd, ds, None, dgamma, before)


@pytest.mark.parametrize("dtype,k", [(F32, 16384), (F32, 16383), (BF, 16384), (BF, 16381)])
@pytest.mark.parametrize("res", [True, False])
def test_rms_backward_of_the_widest_rows_one_after_another(dtype, k, res):
    """Rows of which shared memory holds a single set (fp32 with the stream's gradient) or few, several to a block."""
    g, T = gen(k), 500
    s, dy, ds = (normal(g, T, k, std=std).to(dtype) for std in (2.0, 1e-3, 1e-3))
    ds = ds if res else None
    rstd = (s.double().square().mean(1) + 1e-6).rsqrt().float()
    dX, dgamma = torch.empty_like(s), torch.empty(k, device="cuda")
    rgs.rms_norm_backward(dy, s, None, rstd, dS=ds, dX=dX, dgamma=dgamma, overwrite=True)
    check_backward(dy, s, None, rstd, ds, dX, dgamma)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("k", [40, 264, 1001, 4096])
@pytest.mark.parametrize("place", [0, 1, 3, 8])
def test_rms_backward_any_stride_and_place(dtype, k, place):
    g, T = gen(8), 37
    s, dy, ds = (padded(normal(g, T, k).to(dtype), k + p, q) for p, q in ((place, place), (2 * place, 0), (8, place)))
    rstd = torch.rand(T, generator=g, device="cuda") + 0.5
    dX = padded(torch.zeros(T, k, dtype=dtype, device="cuda"), k + 3, place)
    beside = dX.as_strided((T, 3), dX.stride(), dX.storage_offset() + k)
    dgamma = torch.empty(k, device="cuda")
    rgs.rms_norm_backward(dy, s, None, rstd, dS=ds, dX=dX, dgamma=dgamma, overwrite=True)
    check_backward(dy, s, None, rstd, ds, dX, dgamma)
    assert bool(torch.isnan(beside.double()).all())


@pytest.mark.parametrize("k", [512, 1001, 4096, 16392])
@pytest.mark.parametrize("which", ["dX is dY", "dX is dS"])
def test_rms_backward_in_place(k, which):
    g, T = gen(9), 300
    s, dy, ds = (normal(g, T, k).to(BF) for _ in range(3))
    rstd = torch.rand(T, generator=g, device="cuda") + 0.5
    dy0, ds0, dgamma = dy.clone(), ds.clone(), torch.zeros(k, device="cuda")
    dX = dy if which == "dX is dY" else ds
    rgs.rms_norm_backward(dy, s, None, rstd, dS=ds, dX=dX, dgamma=dgamma)
    check_backward(dy0, s, None, rstd, ds0, dX, dgamma)


def test_rms_gradient_matches_differences():
    """The gradient against central differences of the forward pass, fp32."""
    g, T, k = gen(10), 3, 40
    x, gamma, w = normal(g, T, k), 1 + normal(g, k, std=0.1), normal(g, T, k)

    def loss(x, gamma):
        Y = torch.empty_like(x)
        rgs.rms_norm_forward(x, gamma, Y=Y)
        return float((Y.double() * w.double()).sum())

    rstd, dX, dgamma = torch.empty(T, device="cuda"), torch.empty_like(x), torch.zeros(k, device="cuda")
    rgs.rms_norm_forward(x, gamma, rstd, Y=torch.empty_like(x))
    rgs.rms_norm_backward(w, x, gamma, rstd, dX=dX, dgamma=dgamma)
    h = 2.0 ** -7
    for grad, at, other in ((dX, x, lambda t: loss(t, gamma)), (dgamma, gamma, lambda t: loss(x, t))):
        for i in (0, 7, at.numel() - 1):
            up, down = at.clone(), at.clone()
            up.view(-1)[i] += h
            down.view(-1)[i] -= h
            # the difference's own error: h^2 / 6 of a third derivative of some tens, and 2^-24 / h of the loss's terms
            assert (other(up) - other(down)) / (2 * h) == pytest.approx(float(grad.view(-1)[i]), abs=2e-3)


# ---- 8-bit matrices -------------------------------------------------------------------

QUANT_SHAPES = [(1, 1), (1, 128), (3, 129), (128, 128), (129, 127), (200, 1000), (257, 384), (16, 20001), (1000, 33)]


@pytest.mark.parametrize("T,k", QUANT_SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("place", [0, 1])
def test_quantize(T, k, dtype, rows, place):
    g = gen(T + 3 * k)
    x = padded((normal(g, T, k) * torch.exp(2 * normal(g, T, 1))).to(dtype), k + place, place)
    Q, scale = rgs.code_rows(T, k), torch.empty(-(-T // rows), groups(k), device="cuda")
    Qt = rgs.code_rows(k, T) if rows == 128 else None
    rgs.quantize_blocks(x, Q, scale, rows=rows, Qt=Qt)
    check_codes(Q, scale, x.double(), rows, 0.0)
    if Qt is not None:
        assert torch.equal(Qt.t().float(), Q.float())
        alone, again = rgs.code_rows(k, T), torch.empty_like(scale)
        rgs.quantize_blocks(x, None, again, rows=rows, Qt=alone)
        assert torch.equal(alone.float(), Qt.float()) and torch.equal(again, scale)


def test_quantize_rounds_to_nearest_even():
    """Every code and every border between two codes, in units of a scale of one."""
    codes = torch.arange(0x7F, dtype=torch.uint8, device="cuda").view(E4).float()
    borders = (codes[:-1] + codes[1:]) / 2
    values = torch.cat([codes, -codes, borders, borders * (1 + 2.0 ** -20), borders * (1 - 2.0 ** -20), -borders])
    x = torch.zeros(-(-len(values) // 127), 128, device="cuda")
    x[:, 127] = 448.0
    x[:, :127] = torch.cat([values, torch.zeros(x.shape[0] * 127 - len(values), device="cuda")]).view(-1, 127)
    Q, scale = rgs.code_rows(*x.shape), torch.empty(x.shape[0], 1, device="cuda")
    rgs.quantize_blocks(x, Q, scale)
    assert bool((scale == 1.0).all())
    assert torch.equal(Q.view(torch.uint8), x.to(E4).view(torch.uint8))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("size", [1.0, 1e-30, 1e-36, 1e-38, 1e30, 5e36])
def test_quantize_keeps_to_its_bounds(dtype, rows, size):
    """Scales within 2^-23 of the quotient; codes that are nearest to a number within 2^-22 of x / scale."""
    T, k = 1024, 1000
    g = gen(rows)
    x = (normal(g, T, k).clamp(-8, 8) * torch.exp(normal(g, T, 1)).clamp(max=4.0) * size).to(dtype)
    Q, scale = rgs.code_rows(T, k), torch.empty(-(-T // rows), groups(k), device="cuda")
    rgs.quantize_blocks(x, Q, scale, rows=rows)
    want = (tops(x.double(), rows) / 448.0).clamp(min=2.0 ** -126)
    close(scale, want, want * 2.0 ** -23)
    units = (x.double() / wide(scale, rows, T, k)).abs()
    # the conversions to fp32 here may bring the two ends 2^-24 nearer: the codes' bound is 3/4 of 2^-22
    low, high = ((units * (1 + f)).float().clamp(max=448.0).to(E4).float() for f in (-2.0 ** -22, 2.0 ** -22))
    q = Q.float().abs()
    assert bool(((low <= q) & (q <= high)).all())
    assert bool(((Q.float() * x.float()) >= 0).all())


@pytest.mark.parametrize("rows", [1, 128])
def test_quantize_extremes(rows):
    x = torch.zeros(128 * 5, 130, device="cuda")
    for block, v in enumerate((0.0, 2.0 ** -149, 3.0e38, math.inf, math.nan)):
        x[128 * block, 5] = v
    x[128 * 2, 6] = -1.0e38
    Q, scale = rgs.code_rows(*x.shape), torch.empty(len(x) // rows, 2, device="cuda")
    rgs.quantize_blocks(x, Q, scale, rows=rows)
    q, at = Q.float(), [128 * b // rows for b in range(5)]
    assert float(scale[at[0], 0]) == 2.0 ** -126 and bool((q[:128] == 0).all())
    assert float(scale[at[1], 0]) == 2.0 ** -126 and bool((q[128:256] == 0).all())
    assert float(scale[at[2], 0]) == pytest.approx(3.0e38 / 448, rel=1e-6) and float(q[256, 5]) == 448.0
    assert float(q[256, 6]) == -144.0  # -149.3 among codes 16 apart
    for b in (3, 4):
        assert bool(torch.isnan(scale[at[b], 0])) and bool(torch.isnan(q[128 * b, :128]).all())
        assert bool((q[128 * b, 128:] == 0).all())
        assert bool(torch.isnan(q[128 * b + 1, :128]).all()) == (rows == 128)


def operands(g, T, N, k, scales=True):
    A, B = rgs.code_rows(T, k), rgs.code_rows(N, k)
    A.copy_(normal(g, T, k, std=60.0).clamp(-448, 448).to(E4))
    B.copy_(normal(g, N, k, std=60.0).clamp(-448, 448).to(E4))
    sa = torch.exp(normal(g, T, groups(k))) / 64
    sb = torch.exp(normal(g, groups(N), groups(k))) / 64
    return A, sa, B, sb


def check_product(A, sa, B, sb, Y, before=None):
    T, k = A.shape
    N = len(B)
    a, b = A.double() * wide(sa, 1, T, k), B.double() * wide(sb, 128, N, k)
    want, size = a @ b.t(), a.abs() @ b.abs().t()
    if before is not None:
        want = want + before.double()
    # a block's 128 products are exact; each addition of the tensor cores may cut 2^-23 of
    # the sum: 128 2^-23 = 2^-16 of the block's magnitudes; the blocks' sums and scales in fp32
    close(Y, want, size * (2.0 ** -16 + (groups(k) + 3) * U) + want.abs() * (HALF[Y.dtype] + 2 * U))


TOKENS = [1, 2, 15, 16, 17, 32, 33, 64, 65, 100, 128, 129, 300, 700]


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("N,k", [(128, 128), (1, 1), (130, 16), (257, 384), (1027, 2100), (100, 1025)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_matmul(T, N, k, dtype):
    A, sa, B, sb = operands(gen(T + N + k), T, N, k)
    Y = torch.full((T, (N + 7) // 8 * 8 + 8), 7.0, dtype=dtype, device="cuda")
    rgs.matmul_blocks(A, sa, B, sb, Y[:, :N])
    check_product(A, sa, B, sb, Y[:, :N])
    assert bool((Y[:, N:] == 7.0).all())  # what lies behind a row stays
    again = torch.empty_like(Y)
    rgs.matmul_blocks(A, sa, B, sb, again[:, :N])
    assert torch.equal(again[:, :N], Y[:, :N])


@pytest.mark.parametrize("T,N,k", [(16, 4096, 4096), (3, 300, 16384), (600, 4096, 1024), (2500, 2056, 1000), (5000, 1000, 260),
                                   (20000, 40, 72), (40, 20000, 72), (5001, 5001, 2100), (300, 9000, 5000), (1999, 1021, 130),
                                   (256, 2048, 4096), (511, 1027, 3000), (513, 2049, 2500), (700, 300, 16384), (260, 520, 1300), (2560, 2100, 16400)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_matmul_larger(T, N, k, dtype):
    A, sa, B, sb = operands(gen(T), T, N, k)
    Y = torch.full((T, (N + 7) // 8 * 8), 7.0, dtype=dtype, device="cuda")
    rgs.matmul_blocks(A, sa, B, sb, Y[:, :N])
    check_product(A, sa, B, sb, Y[:, :N])
    assert bool((Y[:, N:] == 7.0).all())
    if dtype == F32:
        before = Y[:, :N].clone()
        rgs.matmul_blocks(A, sa, B, sb, Y[:, :N], overwrite=False)
        check_product(A, sa, B, sb, Y[:, :N], before)
        assert bool((Y[:, N:] == 7.0).all())


@pytest.mark.parametrize("T", [5, 24, 60, 300, 1500])
@pytest.mark.parametrize("a_exp,b_exp", [(-63, -63), (-126, 0), (0, -126), (-20, -106), (63, 64), (127, 0), (0, 127)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_matmul_scales_at_the_ends_of_their_products_range(T, a_exp, b_exp, dtype):
    """Scales whose products are fp32's smallest and largest normal powers of two: results are as exact as any, and
    rows of zeros give zeros."""
    N, k = 270, 500
    A, sa, B, sb = operands(gen(T), T, N, k)
    if a_exp + b_exp > 0:  # values of 2^-6 at most: 500 products of them add up to 2^-3, times 2^127 that is no infinity
        A.copy_(A.float() / 448 * 2.0 ** -6), B.copy_(B.float() / 448 * 2.0 ** -6)
    sa.fill_(2.0 ** a_exp), sb.fill_(2.0 ** b_exp)
    A[3], B[7], B[130:256] = 0, 0, 0
    Y = torch.full((T, 272), 7.0, dtype=dtype, device="cuda")[:, :N]
    rgs.matmul_blocks(A, sa, B, sb, Y)
    a, b = A.double() * wide(sa, 1, T, k), B.double() * wide(sb, 128, N, k)
    want, size = a @ b.t(), a.abs() @ b.abs().t()
    # as in check_product; below 2^-126 a step is 2^-149 (BF16 2^-133) whatever the value: half of it for the result's
    # rounding, and for each block's
    least = (groups(k) + 3) * 2.0 ** -150 + (2.0 ** -134 if dtype == BF else 0.0)
    close(Y, want, size * (2.0 ** -16 + (groups(k) + 3) * U) + want.abs() * (HALF[dtype] + 2 * U) + least)
    assert not Y[3].any() and not Y[:, 7].any() and not Y[:, 130:256].any()


@pytest.mark.parametrize("T", [3, 40, 300, 1000])
def test_matmul_adds_to_fp32(T):
    g = gen(T)
    A, sa, B, sb = operands(g, T, 300, 500)
    Y = normal(g, T, 304, std=5.0)[:, :300]
    before = Y.clone()
    rgs.matmul_blocks(A, sa, B, sb, Y, overwrite=False)
    check_product(A, sa, B, sb, Y, before)


@pytest.mark.parametrize("T", [5, 200, 1500])
def test_matmul_padding_and_values_that_are_not_finite(T):
    """Codes between rows reach no result; a NaN or an infinity stays in its row or column."""
    g, N, k = gen(11), 270, 200
    A, sa, B, sb = operands(g, T, N, k)
    for t in (A, B):
        t.as_strided((len(t), t.stride(0) - k), t.stride(), t.storage_offset() + k).view(torch.uint8).fill_(0x7F)
    Y = torch.empty(T, 272, device="cuda")[:, :N]
    rgs.matmul_blocks(A, sa, B, sb, Y)
    check_product(A, sa, B, sb, Y)
    A.view(torch.uint8)[1, 7] = 0x7F
    sa[2, 1] = math.inf
    B.view(torch.uint8)[5, 150] = 0x7F
    bad = torch.empty(T, 272, device="cuda")[:, :N]
    rgs.matmul_blocks(A, sa, B, sb, bad)
    keep = torch.ones(T, N, dtype=torch.bool, device="cuda")
    keep[1:3] = False
    keep[:, 5] = False
    assert bool(torch.isnan(bad[1]).all()) and bool(torch.isnan(bad[:, 5]).all())
    assert not bool(torch.isfinite(bad[2]).any())
    assert torch.equal(bad[keep], Y[keep])


@pytest.mark.parametrize("T,N,k", [(5, 100, 300), (70, 100, 300), (1501, 515, 130)])
def test_matmul_scales_of_any_strides_and_rows_behind(T, N, k):
    """a_scale with rows apart, b_scale one value for all blocks; Y's rows from T on stay."""
    g = gen(15)
    A, sa, B, _ = operands(g, T, N, k)
    apart = torch.full((T, groups(k) + 3), math.nan, device="cuda")
    apart[:, :groups(k)] = sa
    one = torch.full((1, 1), 0.25, device="cuda")
    for dtype in (BF, F32):
        Y = torch.full((T + 40, 520), 7.0, dtype=dtype, device="cuda")
        rgs.matmul_blocks(A, apart[:, :groups(k)], B, one.expand(groups(N), groups(k)), Y[:T, :N])
        check_product(A, sa, B, one.expand(groups(N), groups(k)).contiguous(), Y[:T, :N])
        assert bool((Y[T:] == 7.0).all()) and bool((Y[:, N:] == 7.0).all())


def test_offsets_past_32_bits():
    """Matrices and gradients of more than 2^31 values, looked at where they end."""
    T, N, k = 66000, 33000, 128
    A, sa, B, sb = operands(gen(16), T, N, k)
    Y = torch.empty(T, N, dtype=BF, device="cuda")
    rgs.matmul_blocks(A, sa, B, sb, Y)
    check_product(A[-300:], sa[-300:], B, sb, Y[-300:])
    del A, B
    X = Y.view(66000, 33000)
    Q, scale = rgs.code_rows(T, N), torch.empty(T, groups(N), device="cuda")
    rgs.quantize_blocks(X, Q, scale)
    check_codes(Q[-50:], scale[-50:], X[-50:].double(), 1, 0.0)
    tiles, Qt = torch.empty(groups(T), groups(N), device="cuda"), rgs.code_rows(N, T)
    rgs.quantize_blocks(X, Q, tiles, rows=128, Qt=Qt)
    check_codes(Q[-80:], tiles[-1:], X[-80:].double(), 128, 0.0)
    assert torch.equal(Qt[:, -80:].t().float(), Q[-80:].float())
    del Qt, Q
    for k in (16384, 33000):  # rows in registers; rows read twice
        T = Y.numel() // k
        X = Y.view(-1)[:T * k].view(T, k)
        O, rstd = torch.empty_like(X), torch.empty(T, device="cuda")
        rgs.rms_norm_forward(X, None, rstd, Y=O)
        check_forward(X[-9:], None, None, 1e-6, None, O[-9:], None, None, rstd[-9:])
        dX = torch.empty_like(X)
        rgs.rms_norm_backward(O, X, None, rstd, dX=dX)
        check_backward(O[-9:], X[-9:], None, rstd[-9:], None, dX[-9:], None)
        del dX, O
    X.fill_(0.5)
    X.view(-1)[-3:] = 4096.0
    clip = rgs.GradClip([X], 1.0, outs=[X])
    clip.step()
    want = math.sqrt(0.25 * (X.numel() - 3) + 3 * 4096.0 ** 2)
    assert float(clip.norm) == pytest.approx(want, rel=8 * U)
    assert float(X.view(-1)[-1]) == pytest.approx(4096.0 / want, rel=2.0 ** -8)


@pytest.mark.parametrize("T", [4, 500])
def test_layer_and_its_input_gradient(T):
    """The path as a layer uses it: norm into 8 bits, product; derivatives into 8 bits, product with the transposed weight."""
    g, k, d = gen(12), 384, 520
    x, r, gamma = normal(g, T, k).to(BF), normal(g, T, k).to(BF), (1 + normal(g, k, std=0.1)).to(BF)
    W = normal(g, d, k, std=0.05).to(BF)
    S, rstd = torch.empty_like(x), torch.empty(T, device="cuda")
    Q, qs = rgs.code_rows(T, k), torch.empty(T, groups(k), device="cuda")
    rgs.rms_norm_forward(x, gamma, rstd, R=r, S=S, Q=Q, scale=qs)
    Wq, Wt, ws = rgs.code_rows(d, k), rgs.code_rows(k, d), torch.empty(groups(d), groups(k), device="cuda")
    rgs.quantize_blocks(W, Wq, ws, rows=128, Qt=Wt)
    Y = torch.empty(T, d, dtype=BF, device="cuda")
    rgs.matmul_blocks(Q, qs, Wq, ws, Y)
    check_product(Q, qs, Wq, ws, Y)
    # against the unquantised product: two roundings of 2^-4 at most, independent over k terms
    want = rms_reference(x, r, gamma, 1e-6)[2] @ W.double().t()
    assert float((Y.double() - want).norm() / want.norm()) < 2.0 ** -4
    D = normal(g, T, d, std=1e-3).to(BF)
    Dq, ds = rgs.code_rows(T, d), torch.empty(T, groups(d), device="cuda")
    rgs.quantize_blocks(D, Dq, ds)
    dY = torch.empty(T, k, dtype=BF, device="cuda")
    rgs.matmul_blocks(Dq, ds, Wt, ws.t(), dY)
    check_product(Dq, ds, Wt, ws.t().contiguous(), dY)
    want = D.double() @ W.double()
    assert float((dY.double() - want).norm() / want.norm()) < 2.0 ** -4
    dX, dgamma = torch.empty_like(x), torch.zeros(k, device="cuda")
    rgs.rms_norm_backward(dY, S, gamma, rstd, dS=r, dX=dX, dgamma=dgamma)
    check_backward(dY, S, gamma, rstd, r, dX, dgamma)


# ---- clipping ---------------------------------------------------------------------------

def check_norm(Gs, norm, scale, max_norm):
    want = math.sqrt(sum(float(G.double().square().sum()) for G in Gs))
    # a thread's 32 squares in fp32 (chains of 8, three additions), halved by the root, and the result's rounding
    # a norm past fp32's largest value, (2 - 2^-23) 2^127, is an infinity: 6000 values of 1e37 have 7.75e38.  Its scale is
    # then below 2^-126, where half a step is 2^-150 whatever the value
    assert float(norm) == pytest.approx(float(torch.tensor(want, dtype=F64).float()), rel=8 * U, abs=0)
    assert float(scale) == pytest.approx(min(1.0, max_norm / want) if want else 1.0, rel=8 * U, abs=2.0 ** -150)


SIZES = [[1], [0, 5, 0], [8192], [8193, 1, 7], [100000, 3, 8191], [2048] * 114, [1] * 600, [3000001]]


@pytest.mark.parametrize("sizes", SIZES, ids=[str(len(s)) + "x" + str(s[0]) for s in SIZES])
@pytest.mark.parametrize("dtype", [BF, F32, "both"])
@pytest.mark.parametrize("place", [0, 1])
def test_grad_clip(sizes, dtype, place):
    g = gen(sum(sizes))
    Gs, outs = [], []
    for i, n in enumerate(sizes):
        t = dtype if dtype != "both" else (BF, F32)[i % 2]
        Gs.append(torch.empty(n + place, dtype=t, device="cuda")[place:])
        Gs[-1].copy_(normal(g, n) * torch.exp(normal(g, n)))
        outs.append(torch.full((n + place + 8,), 5.0, dtype=t, device="cuda")[place:])
    for max_norm in (0.5, 1e6):
        clip = rgs.GradClip(Gs, max_norm, outs=[o[:n] for o, n in zip(outs, sizes)])
        before = [G.clone() for G in Gs]
        scale = clip.step()
        check_norm(Gs, clip.norm, scale, max_norm)
        for G, b, o, n in zip(Gs, before, outs, sizes):
            assert torch.equal(G, b) and bool((o[n:] == 5.0).all())
            want = G.double() * float(scale)
            if n:
                close(o[:n], want, want.abs() * HALF[G.dtype] + 2.0 ** -134)
                if float(scale) == 1.0:
                    assert torch.equal(o[:n], G)
        clip.step()
        again = clip.norm.clone()
        clip.step()
        assert torch.equal(again, clip.norm)


def test_grad_clip_in_place_and_with_adamw():
    g = gen(13)
    W, G = normal(g, 5000).to(BF), normal(g, 5000)
    C = normal(g, 300, 64)  # a sketch, clipped with the gradients
    G0, C0 = G.clone(), C.clone()
    clip = rgs.GradClip([G, C], 1.0, outs=[G, C])
    scale = float(clip.step())
    check_norm([G0, C0], clip.norm, clip.scale, 1.0)
    close(C, C0.double() * scale, C0.double().abs() * scale * U)
    a, b = W.clone(), W.clone()
    rgs.AdamW([a], [G]).step(lr=1e-2, step=0)
    only = rgs.GradClip([G0, C0], 1.0)
    rgs.AdamW([b], [G0]).step(lr=1e-2, step=0, grad_scale=only.step())
    assert torch.equal(a, b)
    within = rgs.GradClip([G], 1e9, outs=[G])  # a scale of one in place leaves the values as they are
    kept = G.clone()
    within.step()
    assert float(within.scale) == 1.0 and torch.equal(G, kept)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("value", [0.0, 2.0 ** -126, 1e-30, 1e-22, 1e-19, 1e19, 1e30, 1e37])
def test_grad_norm_of_any_size(dtype, value):
    """Squares past fp32's range, either side, beside ones that are not."""
    G = torch.full((9000,), value, device="cuda").to(dtype)
    G[::3] = 0.0
    norm, scale = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    rgs.grad_norm_batched(rgs.grad_problems([G, torch.zeros(17, device="cuda")]), norm, scale, max_norm=1.0)
    check_norm([G], norm, scale, 1.0)


def test_grad_norm_of_values_that_are_not_finite():
    G = torch.ones(20000, device="cuda")
    norm, scale = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    probs = rgs.grad_problems([G])
    G[12345] = -math.inf
    rgs.grad_norm_batched(probs, norm, scale)
    assert float(norm) == math.inf and float(scale) == 0.0
    G[777] = math.nan
    rgs.grad_norm_batched(probs, norm, scale)
    assert math.isnan(float(norm)) and math.isnan(float(scale))
    rgs.grad_norm_batched(probs, norm)  # the norm alone
    assert math.isnan(float(norm))


# ---- streams, graphs, workspaces ----------------------------------------------------------

def a_step(s):
    """A run of the operators into buffers of its own; returns the outputs."""
    rgs.rms_norm_forward(s["x"], s["gamma"], s["rstd"], R=s["r"], S=s["S"], Y=s["Yn"], Q=s["Q"], scale=s["qs"], stream=s.get("stream"))
    rgs.quantize_blocks(s["W"], s["Wq"], s["ws"], rows=128, Qt=s["Wt"], stream=s.get("stream"))
    rgs.matmul_blocks(s["Q"], s["qs"], s["Wq"], s["ws"], s["Y"], stream=s.get("stream"))
    rgs.quantize_blocks(s["Y"], s["Dq"], s["ds"], stream=s.get("stream"))
    rgs.matmul_blocks(s["Dq"], s["ds"], s["Wt"], s["ws"].t(), s["dY"], stream=s.get("stream"))
    rgs.rms_norm_backward(s["dY"], s["S"], s["gamma"], s["rstd"], dS=s["r"], dX=s["dX"], dgamma=s["dgamma"], overwrite=True,
                          stream=s.get("stream"))
    s["clip"].step(stream=s.get("stream"))
    return [s[n].view(torch.uint8) if s[n].dtype == E4 else s[n]
            for n in ("S", "Yn", "Q", "qs", "Wq", "Wt", "ws", "Y", "Dq", "ds", "dY", "dX", "dgamma", "out")] + [s["clip"].norm]


def a_state(seed, T=70, k=272, d=400):
    g = gen(seed)
    s = {"x": normal(g, T, k).to(BF), "r": normal(g, T, k).to(BF), "gamma": normal(g, k).to(BF),
         "W": normal(g, d, k, std=0.05).to(BF)}
    like = {"S": (T, k, BF), "Yn": (T, k, BF), "Y": (T, d, BF), "dY": (T, k, BF), "dX": (T, k, BF), "qs": (T, groups(k), F32),
            "ws": (groups(d), groups(k), F32), "ds": (T, groups(d), F32)}
    s.update({n: torch.empty(a, b, dtype=t, device="cuda") for n, (a, b, t) in like.items()})
    s.update(Q=rgs.code_rows(T, k), Wq=rgs.code_rows(d, k), Wt=rgs.code_rows(k, d), Dq=rgs.code_rows(T, d))
    s.update(rstd=torch.empty(T, device="cuda"), dgamma=torch.empty(k, device="cuda"))
    s["out"] = torch.empty_like(s["dgamma"])
    s["clip"] = rgs.GradClip([s["dgamma"], s["dX"]], 0.01, outs=[s["out"], s["dX"]])
    torch.cuda.synchronize()
    return s


def test_on_two_streams_at_once():
    want = [[t.clone() for t in a_step(a_state(seed))] for seed in (1, 2)]
    states = [a_state(1), a_state(2)]
    for s in states:
        s["stream"] = torch.cuda.Stream()
    for _ in range(3):
        got = [a_step(s) for s in states]
    torch.cuda.synchronize()
    for w, o in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(w, o))


def test_products_on_many_streams_at_once():
    """Clusters of several sizes and pairs of CTAs beside each other, which share the SMs' TMEM."""
    shapes = [(8, 2048, 2048), (24, 1024, 4096), (48, 3000, 1000), (16, 300, 512), (200, 2048, 2048), (700, 1024, 1024)]
    work = []
    for i, (T, N, k) in enumerate(shapes):
        ops = operands(gen(30 + i), T, N, k)
        want = torch.empty(T, (N + 7) // 8 * 8, dtype=BF, device="cuda")[:, :N]
        rgs.matmul_blocks(*ops, want)
        work.append((ops, want, torch.zeros(T, (N + 7) // 8 * 8, dtype=BF, device="cuda")[:, :N], torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(40):
        for ops, _, Y, stream in work:
            rgs.matmul_blocks(*ops, Y, stream=stream)
    torch.cuda.synchronize()
    for _, want, Y, _ in work:
        assert torch.equal(Y, want)


def test_captured_and_replayed():
    a_step(a_state(3))
    s = a_state(3)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = a_step(s)
    for seed in (4, 5):
        other = a_state(seed)
        for n in ("x", "r", "gamma", "W"):
            s[n].copy_(other[n])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(a_step(other), out))


def test_the_example_runs_with_these_operators():
    from rank_gradient_sketching_philox_gb300 import train_example
    losses = train_example.main(["--steps", "3", "--tokens", "200", "--norm", "rms", "--products", "8bit", "--clip", "0.5"])
    assert len(losses) == 3 and all(math.isfinite(x) for x in losses)


@pytest.mark.parametrize("most", ["0", "-1", "nan"])
def test_the_example_refuses_a_norm_that_is_no_bound(most):
    """As GradClip does; 0 is not taken for no clipping."""
    from rank_gradient_sketching_philox_gb300 import train_example
    with pytest.raises(ValueError, match="max_norm"):
        train_example.main(["--steps", "1", "--tokens", "64", "--clip=" + most])


@pytest.mark.parametrize("products", ["bf16", "8bit"])
def test_the_examples_gradients(products):
    """A microbatch's gradients of the stream, through every norm and product, against autograd in 64 bits."""
    from rank_gradient_sketching_philox_gb300 import train_example
    model = train_example.Model(vocabulary=64, width=128, blocks=2, rank=16, norm="rms", products=products)
    g = gen(20)
    for n in model.norms:
        n.gamma.copy_(1 + normal(g, 128, std=0.2))
    rgs.sample_projection_batched(rgs.PROJ_GAUSSIAN_QR, 0, 0, [m.P for m in model.linears[:-1]], [m.layer for m in model.linears[:-1]])
    rgs.sample_projection(rgs.PROJ_GAUSSIAN_QR, 0, model.head.layer, 0, model.head.P)
    tokens = torch.randint(0, 64, (96,), generator=g, device="cuda")
    targets = torch.randint(0, 64, (96,), generator=g, device="cuda")
    losses = model.microbatch(tokens, targets, True, 1.0 / 96)
    leaf = lambda t: t.double().requires_grad_()  # noqa: E731
    E, gammas = leaf(model.embedding), [leaf(n.gamma) for n in model.norms]

    def rms(x, gamma):
        return x * (x.square().mean(1, keepdim=True) + 1e-6).rsqrt() * gamma

    x = E[tokens]
    for gamma, (up, down) in zip(gammas, model.pairs):
        # relu's pieces are the model's own: a value that a rounding moves across zero would change a whole term
        x = x + torch.where(up.active, rms(x, gamma) @ up.W.double().t(), 0.0) @ down.W.double().t()
    want = torch.nn.functional.cross_entropy(rms(x, gammas[-1]) @ model.head.W.double().t(), targets, reduction="none")
    want.mean().backward()
    # Roundings of activations and derivatives on the way: in BF16 some twenty of 2^-8 at most each; in 8 bits sixteen
    # more of 2^-4 (eight products, each with two operands).  As independent errors they add up as squares, a uniform
    # one of half-width e to e / sqrt(3): sqrt(20) 2^-8 / sqrt(3) = 0.010 and sqrt(16) 2^-4 / sqrt(3) = 0.144; doubled,
    # since not all are independent.
    most = 2 * (0.010 if products == "bf16" else 0.144)
    for got, exact in [(losses, want.detach()), (model.dembedding, E.grad)] + [(n.dgamma, q.grad) for n, q in zip(model.norms, gammas)]:
        assert float((got.double() - exact).norm() / exact.norm()) < most


def test_workspaces_are_checked_and_need_no_zeros():
    g, T, k = gen(14), 500, 264
    s, dy, rstd = normal(g, T, k).to(BF), normal(g, T, k).to(BF), torch.ones(T, device="cuda")
    n = rgs.workspace_bytes(rgs.binding.OP_RMS_NORM_BACKWARD, T, 0, k)
    want = torch.empty(k, device="cuda")
    rgs.rms_norm_backward(dy, s, None, rstd, dgamma=want, overwrite=True)
    got = torch.empty_like(want)
    rgs.rms_norm_backward(dy, s, None, rstd, dgamma=got, overwrite=True, ws=torch.full((n,), 255, dtype=torch.uint8, device="cuda"))
    assert torch.equal(want, got)
    with pytest.raises(ValueError):
        rgs.rms_norm_backward(dy, s, None, rstd, dgamma=got, ws=torch.empty(n - 1, dtype=torch.uint8, device="cuda"))
    norm = torch.empty(1, device="cuda")
    with pytest.raises(ValueError):
        rgs.grad_norm_batched(rgs.grad_problems([dy]), norm, ws=torch.empty(64, dtype=torch.uint8, device="cuda"))


def test_binding_refuses_mismatches():
    T, k, N = 6, 200, 70
    x, q = torch.zeros(T, k, dtype=BF, device="cuda"), rgs.code_rows(T, k)
    sc, b, sb = torch.zeros(T, 2, device="cuda"), rgs.code_rows(N, k), torch.zeros(1, 2, device="cuda")
    y = torch.zeros(T, 72, dtype=BF, device="cuda")
    before = rgs.kernel_launches()
    for call in (lambda: rgs.rms_norm_forward(x, None, Y=x.float()),
                 lambda: rgs.rms_norm_forward(x, None, Y=x.t()),
                 lambda: rgs.rms_norm_forward(x, torch.ones(k - 1, device="cuda"), Y=torch.empty_like(x)),
                 lambda: rgs.rms_norm_forward(x, None, Q=q, scale=sc[:, :1]),
                 lambda: rgs.rms_norm_forward(x, None, Q=q.float(), scale=sc),
                 lambda: rgs.quantize_blocks(x, q, sc[:1]),
                 lambda: rgs.quantize_blocks(x, q, sc, rows=0),
                 lambda: rgs.quantize_blocks(x[:, ::2], q[:, :100], sc[:, :1]),
                 lambda: rgs.matmul_blocks(q, sc, b[:, :100], sb, y[:, :N]),
                 lambda: rgs.matmul_blocks(q, sc[:5], b, sb, y[:, :N]),
                 lambda: rgs.matmul_blocks(q, sc, b, sb.t(), y[:, :N]),
                 lambda: rgs.matmul_blocks(q, sc, b, sb, y),
                 lambda: rgs.grad_problems([x.t()]),
                 lambda: rgs.grad_problems([x], outs=[x.float()])):
        with pytest.raises((ValueError, rgs.SketchError)):
            call()
    with pytest.raises(rgs.SketchError):  # rows of codes that do not start on 16 bytes
        rgs.quantize_blocks(x, torch.empty(T, k + 1, dtype=E4, device="cuda")[:, :k], sc)
    assert rgs.kernel_launches() == before


def test_grad_clip_refuses_what_it_would_write_twice():
    """A tensor that is listed twice counts twice in the norm, and is not scaled."""
    G, o = torch.full((4000,), 0.5, device="cuda"), torch.empty(4000, device="cuda")
    twice = rgs.GradClip([G, G], 1.0)
    twice.step()
    check_norm([G, G], twice.norm, twice.scale, 1.0)
    before = rgs.kernel_launches()
    for Gs, outs in (([G, G], [G, G]), ([G, G[:100]], [G, G[:100]]), ([G, G], [o, o]), ([G, o], [o, G]),
                     ([G[:100]], [G[50:150]])):
        with pytest.raises(ValueError):
            rgs.GradClip(Gs, 1.0, outs=outs)
        with pytest.raises(ValueError):
            rgs.grad_scale_batched(rgs.grad_problems(Gs, outs), twice.scale)
    assert rgs.kernel_launches() == before
    halves = rgs.GradClip([G, G], 1.0, outs=[o, torch.empty_like(o)])  # read twice, written apart
    halves.step()
    for out in halves.outs:
        close(out, G.double() * float(halves.scale), G.double().abs() * float(halves.scale) * U)


def test_borrowed_workspaces_are_given_back():
    """A call's own workspace belongs to the call's stream, or to the graph that is captured, and to nobody after it."""
    g, T, k = gen(21), 700, 1000
    s, dy, rstd = normal(g, T, k), normal(g, T, k), torch.ones(T, device="cuda")
    other_dy = normal(g, T, k)
    dgamma, other, norm = (torch.zeros(n, device="cuda") for n in (k, k, 1))
    probs = rgs.grad_problems([dy, s])

    def calls(d, into, stream=None):
        rgs.rms_norm_backward(d, s, None, rstd, dgamma=into, overwrite=True, stream=stream)
        rgs.grad_norm_batched(probs, norm, stream=stream)

    calls(dy, dgamma)
    calls(other_dy, other)
    torch.cuda.synchronize()
    want, want_other, want_norm = dgamma.clone(), other.clone(), norm.clone()
    before = torch.cuda.memory_allocated()
    for stream in (None, torch.cuda.Stream()):
        for _ in range(3):
            calls(dy, dgamma, stream)
    with pytest.raises(rgs.SketchError):  # refused after the workspace was lent
        rgs.rms_norm_backward(dy, s, None, rstd, dS=dy, dgamma=dgamma)
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() == before
    assert torch.equal(dgamma, want) and torch.equal(norm, want_norm)

    graphs, streams = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], [torch.cuda.Stream(), torch.cuda.Stream()]
    with torch.cuda.graph(graphs[0]):
        calls(dy, dgamma)
        held = torch.zeros(400_000, device="cuda")  # may lie where the workspaces were, after them
        calls(dy, dgamma)
    with torch.cuda.graph(graphs[1]):
        rgs.rms_norm_backward(other_dy, s, None, rstd, dgamma=other, overwrite=True)
    for _ in range(5):
        dgamma.zero_(), other.zero_()
        junk = [torch.full((T * k,), float("nan"), device="cuda") for _ in range(3)]
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        del junk
        assert torch.equal(dgamma, want) and torch.equal(other, want_other) and torch.equal(norm, want_norm)
        assert not held.any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [1, 7, 8191, 8192, 100_003, 3_000_001])
def test_grad_norm_does_not_depend_on_the_gradients_place(n, dtype):
    """Equal bits of the norm and of the scale, wherever a gradient starts between two 16-byte boundaries."""
    g = gen(n)
    values = (normal(g, n) * torch.exp(normal(g, n))).to(dtype)
    got = []
    for place in range(8 if dtype == BF else 4):
        G = torch.full((place + n + 8,), math.nan, dtype=dtype, device="cuda")[place:place + n]
        G.copy_(values)
        clip = rgs.GradClip([G], 0.25)
        clip.step()
        check_norm([G], clip.norm, clip.scale, 0.25)
        got.append((clip.norm, clip.scale))
    assert all(torch.equal(norm, got[0][0]) and torch.equal(scale, got[0][1]) for norm, scale in got)


def test_a_product_does_not_replace_what_it_is_to_add_to():
    """A sum in BF16 would lose its earlier terms: refused, and Y stays."""
    A, sa, B, sb = operands(gen(1), 4, 16, 128)
    Y = torch.full((4, 16), 3.0, dtype=BF, device="cuda")
    before = rgs.kernel_launches()
    with pytest.raises(ValueError, match="overwrite=False"):
        rgs.matmul_blocks(A, sa, B, sb, Y, overwrite=False)
    assert rgs.kernel_launches() == before and bool((Y == 3.0).all())
