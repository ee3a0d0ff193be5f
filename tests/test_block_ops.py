"""The residual stream's norm, the 8-bit products and clipping without a GPU: workspace
sizes and the refusals of the C ABI and of the binding (no call here reaches a kernel)."""
import ctypes

import pytest
import torch

from rank_gradient_sketching_philox_gb300 import GradClip, binding, code_rows

NULL = None
A = 1 << 20  # an address that is aligned and never read: every call below is refused first
BAD, UNSUPPORTED, WORKSPACE = binding.ERR_INVALID_ARG, binding.ERR_UNSUPPORTED, binding.ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build()
    return binding.lib()


@pytest.fixture(autouse=True)
def nothing_launched(lib):
    before = binding.kernel_launches()
    yield
    assert binding.kernel_launches() == before


def refused(lib, status, want, message):
    assert status == want
    assert message in lib.sketch_last_error().decode()


def rms_forward(lib, **kw):
    a = dict(X=A, x_type=1, T=4, k=10, ld_x=10, R=A, ld_r=10, S=A, ld_s=10, gamma=A, w_type=1, eps=1e-6, Y=A + 4096,
             ld_y=10, Q=A, ld_q=16, scale=A, rstd=A)
    a.update(kw)
    return lib.sketch_rms_norm_forward(*a.values(), NULL)


@pytest.mark.parametrize("kw,message", [
    (dict(T=0), "T=0"), (dict(k=0), "k=0"), (dict(T=1 << 31), "T="), (dict(x_type=2), "x_type"),
    (dict(w_type=-1), "w_type"), (dict(ld_x=9), "ld_x=9"), (dict(ld_r=9), "ld_r=9"), (dict(ld_s=9), "ld_s=9"),
    (dict(ld_y=9), "ld_y=9"), (dict(eps=-1.0), "eps"), (dict(eps=float("inf")), "eps"), (dict(X=NULL), "X is NULL"),
    (dict(X=A + 2), "X is not 4-byte aligned"), (dict(x_type=0, R=A + 1), "R is not 2-byte aligned"),
    (dict(R=NULL), "S is given without R"), (dict(Y=NULL, Q=NULL, scale=NULL), "both NULL"), (dict(Y=A), "one buffer"),
    (dict(Q=NULL), "together"), (dict(scale=NULL), "together"), (dict(ld_q=10), "ld_q=10"), (dict(ld_q=24), "ld_q=24"),
    (dict(k=20, ld_x=20, ld_r=20, ld_s=20, ld_y=20), "ld_q=16"), (dict(Q=A + 8), "Q is not 16-byte"),
    (dict(scale=A + 2), "scale is not 4-byte"), (dict(gamma=A + 2), "gamma is not"), (dict(rstd=A + 1), "rstd is not"),
])
def test_rms_forward_refuses(lib, kw, message):
    refused(lib, rms_forward(lib, **kw), BAD, message)


def rms_backward(lib, **kw):
    a = dict(dY=A, ld_dy=10, S=A, x_type=1, T=4, k=10, ld_s=10, gamma=A, w_type=1, rstd=A, dS=A, ld_ds=10, dX=A,
             ld_dx=10, dgamma=A, overwrite=1, ws=A, ws_bytes=1 << 20)
    a.update(kw)
    return lib.sketch_rms_norm_backward(*a.values(), NULL)


@pytest.mark.parametrize("kw,status,message", [
    (dict(T=0), BAD, "T=0"), (dict(ld_dy=9), BAD, "ld_dy"), (dict(ld_s=9), BAD, "ld_s"), (dict(ld_ds=9), BAD, "ld_ds"),
    (dict(ld_dx=9), BAD, "ld_dx"), (dict(overwrite=2), BAD, "overwrite"), (dict(dY=NULL), BAD, "dY is NULL"),
    (dict(S=NULL), BAD, "S is NULL"), (dict(rstd=NULL), BAD, "rstd is NULL"),
    (dict(dX=NULL, dgamma=NULL), BAD, "both NULL"), (dict(dX=NULL), BAD, "dS is given without dX"),
    (dict(dgamma=A + 2), BAD, "dgamma is not"), (dict(ws=NULL), WORKSPACE, "workspace"),
    (dict(ws_bytes=8), WORKSPACE, "workspace"), (dict(ws=A + 16), WORKSPACE, "256-byte"),
])
def test_rms_backward_refuses(lib, kw, status, message):
    refused(lib, rms_backward(lib, **kw), status, message)


def quantize(lib, **kw):
    a = dict(X=A, x_type=0, T=40, k=130, ld_x=130, rows=128, Q=A, ld_q=144, scale=A, Qt=A, ld_qt=48)
    a.update(kw)
    return lib.sketch_quantize_blocks(*a.values(), NULL)


@pytest.mark.parametrize("kw,status,message", [
    (dict(T=0), BAD, "T=0"), (dict(k=0), BAD, "k=0"), (dict(x_type=7), BAD, "x_type"), (dict(ld_x=129), BAD, "ld_x"),
    (dict(rows=0), BAD, "rows=0"), (dict(rows=64), BAD, "rows=64"), (dict(rows=1), BAD, "Qt needs rows=128"),
    (dict(Q=NULL, Qt=NULL), BAD, "both NULL"), (dict(ld_q=128), BAD, "ld_q"), (dict(ld_q=136), BAD, "ld_q"),
    (dict(ld_qt=32), BAD, "ld_qt"), (dict(ld_qt=40), BAD, "ld_qt"), (dict(X=NULL), BAD, "X is NULL"),
    (dict(X=A + 1), BAD, "X is not 2-byte"), (dict(Q=A + 4), BAD, "Q is not 16-byte"),
    (dict(Qt=A + 4), BAD, "Qt is not 16-byte"), (dict(scale=NULL), BAD, "scale is NULL"),
    (dict(T=(1 << 31) - 1, k=1 << 24, ld_x=1 << 24, ld_q=1 << 24, Qt=NULL), UNSUPPORTED, "2^31 blocks"),
])
def test_quantize_refuses(lib, kw, status, message):
    refused(lib, quantize(lib, **kw), status, message)


def matmul(lib, **kw):
    a = dict(A=A, T=4, k=130, ld_a=144, a_scale=A, ld_as=2, B=A, N=10, ld_b=144, b_scale=A, bs_row=2, bs_col=1, Y=A,
             y_type=0, ld_y=16, overwrite=1)
    a.update(kw)
    return lib.sketch_matmul_blocks(*a.values(), NULL)


@pytest.mark.parametrize("kw,status,message", [
    (dict(T=0), BAD, "T=0"), (dict(N=0), BAD, "N=0"), (dict(k=0), BAD, "k=0"),
    (dict(T=(1 << 24) + 1), UNSUPPORTED, "T="), (dict(N=(1 << 24) + 1), UNSUPPORTED, "N="),
    (dict(k=(1 << 24) + 1), UNSUPPORTED, "k="), (dict(T=1 << 24, N=1 << 24), UNSUPPORTED, "tiles"),
    (dict(ld_a=128), BAD, "ld_a"), (dict(ld_a=136), BAD, "ld_a"), (dict(ld_b=130), BAD, "ld_b"),
    (dict(ld_as=1), BAD, "ld_as"), (dict(bs_row=-1), BAD, "bs_row"), (dict(bs_col=-1), BAD, "bs_col"),
    (dict(ld_y=8), BAD, "ld_y"), (dict(ld_y=12), BAD, "ld_y"), (dict(y_type=3), BAD, "y_type"),
    (dict(A=NULL), BAD, "A is NULL"), (dict(A=A + 8), BAD, "A is not 16-byte"), (dict(B=A + 8), BAD, "B is not 16-byte"),
    (dict(a_scale=NULL), BAD, "a_scale is NULL"), (dict(b_scale=A + 2), BAD, "b_scale is not 4-byte"),
    (dict(Y=A + 8), BAD, "Y is not 16-byte"), (dict(overwrite=2), BAD, "overwrite"),
])
def test_matmul_refuses(lib, kw, status, message):
    refused(lib, matmul(lib, **kw), status, message)


def test_matmul_does_not_replace_what_it_is_to_add_to(lib):
    refused(lib, matmul(lib, overwrite=0), BAD, "overwrite=0 needs an fp32 Y")


def grads(**kw):
    a = dict(G=A, out=A, count=8, type=0)
    a.update(kw)
    return (binding.GradProblem * 1)(binding.GradProblem(*a.values()))


@pytest.mark.parametrize("kw,call,status,message", [
    (dict(), dict(n=0), BAD, "n=0"), (dict(), dict(problems=NULL), BAD, "problems is NULL"),
    (dict(count=-1), {}, BAD, "count=-1"), (dict(count=(1 << 40) + 1), {}, BAD, "count="), (dict(type=2), {}, BAD, "type"),
    (dict(G=NULL), {}, BAD, "G is NULL"), (dict(G=A + 1), {}, BAD, "G is not 2-byte"),
    (dict(type=1, G=A + 2), {}, BAD, "G is not 4-byte"), (dict(), dict(max_norm=0.0), BAD, "max_norm"),
    (dict(), dict(max_norm=float("nan")), BAD, "max_norm"), (dict(), dict(norm=NULL), BAD, "norm is NULL"),
    (dict(), dict(scale=A + 2), BAD, "scale is not"), (dict(), dict(ws=NULL), WORKSPACE, "workspace"),
    (dict(), dict(ws_bytes=100), WORKSPACE, "workspace"),
])
def test_grad_norm_refuses(lib, kw, call, status, message):
    a = dict(n=1, problems=grads(**kw), max_norm=1.0, norm=A, scale=A, ws=A, ws_bytes=1 << 20)
    a.update(call)
    refused(lib, lib.sketch_grad_norm_batched(*a.values(), NULL), status, message)


@pytest.mark.parametrize("kw,call,message", [
    (dict(), dict(n=0), "n=0"), (dict(out=NULL), {}, "out is NULL"), (dict(out=A + 1), {}, "out is not"),
    (dict(), dict(scale=NULL), "scale is NULL"),
])
def test_grad_scale_refuses(lib, kw, call, message):
    a = dict(n=1, problems=grads(**kw), scale=A)
    a.update(call)
    refused(lib, lib.sketch_grad_scale_batched(*a.values(), NULL), BAD, message)


def test_workspace_sizes(lib):
    ws = binding.workspace_bytes
    assert ws(binding.OP_RMS_NORM_BACKWARD, 1, 0, 7) >= 4 * 7
    assert ws(binding.OP_RMS_NORM_BACKWARD, 1 << 20, 0, 4096) == ws(binding.OP_RMS_NORM_BACKWARD, 1 << 21, 0, 4096)
    assert ws(binding.OP_RMS_NORM_BACKWARD, 0, 0, 7) == 0
    assert ws(binding.OP_GRAD_NORM, 1) % 256 == 0 and ws(binding.OP_GRAD_NORM, 1) > 0
    assert ws(binding.OP_GRAD_NORM, 257) == 2 * ws(binding.OP_GRAD_NORM, 256)
    assert ws(binding.OP_GRAD_NORM, 0) == 0


def test_code_rows_start_on_16_bytes():
    q = code_rows(5, 33, device="cpu")
    assert q.shape == (5, 33) and q.dtype == torch.float8_e4m3fn and q.stride() == (48, 1)


def test_binding_refuses_cpu_tensors(lib):
    x = torch.zeros(4, 16)
    with pytest.raises(ValueError):
        binding.rms_norm_forward(x, None, Y=torch.zeros(4, 16))
    with pytest.raises(ValueError):
        binding.rms_norm_backward(x, x, None, torch.zeros(4), dX=torch.zeros(4, 16))
    q = code_rows(4, 16, device="cpu")
    with pytest.raises(ValueError):
        binding.quantize_blocks(x, q, torch.zeros(4, 1))
    with pytest.raises(ValueError):
        binding.matmul_blocks(q, torch.zeros(4, 1), q, torch.zeros(1, 1), torch.zeros(4, 4))
    with pytest.raises(ValueError):
        binding.grad_problems([x])
    with pytest.raises(ValueError):
        binding.grad_problems([])
    with pytest.raises(ValueError):
        binding.grad_norm_batched((binding.GradProblem * 1)(), torch.zeros(1))
    with pytest.raises(ValueError):
        GradClip([x], float("inf"))
    with pytest.raises(ValueError):
        GradClip([x], 0.0)


def test_problem_layout_matches_the_header():
    """sketch_grad_problem is two pointers, an int64 and an enum."""
    assert ctypes.sizeof(binding.GradProblem) == 32
    assert binding.GradProblem.count.offset == 16 and binding.GradProblem.type.offset == 24


@pytest.mark.parametrize("spans,want", [
    ([], False),
    ([(0, 16, True), (16, 16, True), (32, 4, False)], False),
    ([(64, 16, True), (64, 16, True)], True),                    # one tensor listed twice
    ([(64, 16, False), (64, 16, False)], False),                 # read twice
    ([(64, 16, True), (79, 16, False)], True),                   # its last byte read by another
    ([(79, 16, False), (64, 16, True)], True),
    ([(79, 16, True), (64, 16, False)], True),                   # its first byte
    ([(0, 1000, True), (10, 10, False)], True),                  # inside
    ([(0, 1000, False), (10, 10, True), (2000, 8, True)], True),
    ([(0, 1000, False), (10, 10, False), (1000, 8, True)], False),
    ([(0, 0, True), (0, 0, True), (0, 8, True)], False),         # empty tensors have no place
    ([(0, 64, True), (8, 0, True)], False),
])
def test_tensors_that_a_scaling_would_write_twice(spans, want):
    assert binding._written_twice(spans) is want
