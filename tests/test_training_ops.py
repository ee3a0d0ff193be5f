"""The training operators without a GPU: workspace sizes and the refusals of the
C ABI and of the binding (no call here reaches a kernel)."""
import ctypes

import pytest
import torch

from rank_gradient_sketching_philox_gb300 import AdamW, binding

NULL = None
A = 1 << 20  # an address that is aligned and never read: every call below is refused first


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


def norm_forward(lib, **kw):
    a = dict(X=A, x_type=1, T=4, k=10, ld_x=10, gamma=A, beta=A, w_type=1, eps=1e-5, Y=A, ld_y=10, mean=A, rstd=A)
    a.update(kw)
    return lib.sketch_layer_norm_forward(*a.values(), NULL)


@pytest.mark.parametrize("kw,message", [
    (dict(T=0), "T=0"), (dict(k=0), "k=0"), (dict(T=1 << 31), "T="), (dict(x_type=2), "x_type"),
    (dict(w_type=-1), "w_type"), (dict(ld_x=9), "ld_x=9"), (dict(ld_y=9), "ld_y=9"), (dict(eps=-1.0), "eps"),
    (dict(eps=float("nan")), "eps"), (dict(X=NULL), "X is NULL"), (dict(Y=NULL), "Y is NULL"),
    (dict(mean=NULL), "mean is NULL"), (dict(rstd=NULL), "rstd is NULL"), (dict(X=A + 2), "X is not 4-byte aligned"),
    (dict(x_type=0, Y=A + 1), "Y is not 2-byte aligned"), (dict(beta=A + 2), "beta is not 4-byte aligned"),
])
def test_norm_forward_refuses(lib, kw, message):
    refused(lib, norm_forward(lib, **kw), binding.ERR_INVALID_ARG, message)


def norm_backward(lib, **kw):
    a = dict(dY=A, ld_dy=10, X=A, x_type=1, T=4, k=10, ld_x=10, gamma=A, w_type=1, mean=A, rstd=A, dX=A, ld_dx=10,
             dgamma=A, dbeta=A, overwrite=1, ws=A, ws_bytes=1 << 20)
    a.update(kw)
    return lib.sketch_layer_norm_backward(*a.values(), NULL)


@pytest.mark.parametrize("kw,status,message", [
    (dict(T=0), binding.ERR_INVALID_ARG, "T=0"), (dict(ld_dy=9), binding.ERR_INVALID_ARG, "ld_dy"),
    (dict(ld_dx=9), binding.ERR_INVALID_ARG, "ld_dx"), (dict(overwrite=2), binding.ERR_INVALID_ARG, "overwrite"),
    (dict(dY=NULL), binding.ERR_INVALID_ARG, "dY is NULL"), (dict(mean=NULL), binding.ERR_INVALID_ARG, "mean is NULL"),
    (dict(dX=NULL, dgamma=NULL, dbeta=NULL), binding.ERR_INVALID_ARG, "all NULL"),
    (dict(dgamma=A + 2), binding.ERR_INVALID_ARG, "dgamma is not"),
    (dict(ws=NULL), binding.ERR_WORKSPACE, "workspace"), (dict(ws_bytes=8), binding.ERR_WORKSPACE, "workspace"),
    (dict(ws=A + 16), binding.ERR_WORKSPACE, "256-byte"),
])
def test_norm_backward_refuses(lib, kw, status, message):
    refused(lib, norm_backward(lib, **kw), status, message)


def ce_forward(lib, **kw):
    a = dict(X=A, T=4, k=16, ld_x=16, W=A, V=10, ld_w=16, targets=A, scale=1.0, loss=A, lse=A, dev_status=NULL, ws=A,
             ws_bytes=1 << 20)
    a.update(kw)
    return lib.sketch_cross_entropy_forward(*a.values(), NULL)


@pytest.mark.parametrize("kw,status,message", [
    (dict(T=0), binding.ERR_INVALID_ARG, "T=0"), (dict(V=0), binding.ERR_INVALID_ARG, "V=0"),
    (dict(k=12), binding.ERR_INVALID_ARG, "k=12"), (dict(ld_x=20), binding.ERR_INVALID_ARG, "ld_x"),
    (dict(ld_w=8), binding.ERR_INVALID_ARG, "ld_w"), (dict(V=(1 << 24) + 1), binding.ERR_UNSUPPORTED, "V="),
    (dict(X=A + 8), binding.ERR_INVALID_ARG, "X is not 16-byte"), (dict(W=NULL), binding.ERR_INVALID_ARG, "W is NULL"),
    (dict(targets=NULL), binding.ERR_INVALID_ARG, "targets is NULL"),
    (dict(targets=A + 4), binding.ERR_INVALID_ARG, "targets is not 8-byte"),
    (dict(scale=0.0), binding.ERR_INVALID_ARG, "scale"), (dict(scale=-1.0), binding.ERR_INVALID_ARG, "scale"),
    (dict(scale=float("inf")), binding.ERR_INVALID_ARG, "scale"), (dict(loss=NULL), binding.ERR_INVALID_ARG, "loss"),
    (dict(dev_status=A + 2), binding.ERR_INVALID_ARG, "dev_status"), (dict(ws=NULL), binding.ERR_WORKSPACE, "workspace"),
    (dict(ws_bytes=4), binding.ERR_WORKSPACE, "workspace"),
])
def test_cross_entropy_forward_refuses(lib, kw, status, message):
    refused(lib, ce_forward(lib, **kw), status, message)


def ce_backward(lib, **kw):
    a = dict(X=A, T=4, k=16, ld_x=16, W=A, V=10, ld_w=16, targets=A, scale=1.0, lse=A, g=A, dX=A, ld_dx=16, dW=A,
             dw_type=0, ld_dw=16, XP=NULL, ld_xp=0, r=0, C=NULL, overwrite=1, dev_status=NULL, ws=A, ws_bytes=1 << 24)
    a.update(kw)
    return lib.sketch_cross_entropy_backward(*a.values(), NULL)


@pytest.mark.parametrize("kw,status,message", [
    (dict(lse=NULL), binding.ERR_INVALID_ARG, "lse is NULL"), (dict(g=NULL), binding.ERR_INVALID_ARG, "g is NULL"),
    (dict(overwrite=3), binding.ERR_INVALID_ARG, "overwrite"),
    (dict(dX=NULL, dW=NULL), binding.ERR_INVALID_ARG, "all NULL"),
    (dict(ld_dx=12), binding.ERR_INVALID_ARG, "ld_dx"), (dict(ld_dw=8), binding.ERR_INVALID_ARG, "ld_dw"),
    (dict(dw_type=5), binding.ERR_INVALID_ARG, "dw_type"), (dict(C=A), binding.ERR_INVALID_ARG, "together"),
    (dict(C=A, XP=A, r=0, ld_xp=8), binding.ERR_INVALID_ARG, "r=0"),
    (dict(C=A, XP=A, r=16, ld_xp=8), binding.ERR_INVALID_ARG, "ld_xp"),
    (dict(ws_bytes=100), binding.ERR_WORKSPACE, "workspace"), (dict(k=20), binding.ERR_INVALID_ARG, "k=20"),
])
def test_cross_entropy_backward_refuses(lib, kw, status, message):
    refused(lib, ce_backward(lib, **kw), status, message)


def adamw(lib, problems=None, count=None, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, decay=0.0, grad_scale=NULL, **kw):
    a = dict(W=A, G=A, m=A, v=A, m_scale=NULL, v_scale=NULL, n=8, layer=0, w_type=0, g_type=0)
    a.update(kw)
    if problems is None:
        problems = (binding.AdamWProblem * 1)(binding.AdamWProblem(*a.values()))
    return lib.sketch_adamw_batched(len(problems) if count is None else count, problems, lr, b1, b2, eps, decay, grad_scale, 0,
                                    0, NULL)


@pytest.mark.parametrize("kw,message", [
    (dict(W=NULL), "W is NULL"), (dict(G=A + 8), "G is not 16-byte"), (dict(m=NULL), "m is NULL"),
    (dict(n=0, lr=float("nan")), "lr"), (dict(decay=float("inf")), "weight_decay"), (dict(b1=1.0), "beta"),
    (dict(b2=-0.1), "beta"), (dict(b2=1.0 - 1e-12), "beta"), (dict(eps=0.0), "eps"), (dict(eps=1e-60), "eps"),
    (dict(w_type=2), "w_type"), (dict(g_type=7), "g_type"), (dict(m_scale=A), "for all tensors"),
    (dict(v_scale=A), "for all tensors"), (dict(m_scale=A + 2, v_scale=A), "m_scale is not 4-byte"),
    (dict(grad_scale=A + 1), "grad_scale"),
])
def test_adamw_refuses(lib, kw, message):
    refused(lib, adamw(lib, **kw), binding.ERR_INVALID_ARG, message)


def test_adamw_refuses_mixed_states_and_sizes(lib):
    P = binding.AdamWProblem
    mixed = (P * 2)(P(A, A, A, A, A, A, 8, 0, 0, 0), P(A, A, A, A, None, None, 8, 1, 0, 0))
    refused(lib, adamw(lib, problems=mixed), binding.ERR_INVALID_ARG, "for all tensors")
    negative = (P * 1)(P(A, A, A, A, None, None, -1, 0, 0, 0))
    refused(lib, adamw(lib, problems=negative), binding.ERR_INVALID_ARG, "n=-1")
    refused(lib, adamw(lib, problems=negative, count=0), binding.ERR_INVALID_ARG, "n=0")


def test_workspace_sizes(lib):
    ws = binding.workspace_bytes
    assert ws(binding.OP_CROSS_ENTROPY_FORWARD, 128, 1000) == 8 * 8 * 128  # a pair of floats for each of 8 blocks of 128 columns
    assert ws(binding.OP_CROSS_ENTROPY_FORWARD, 0, 1000) == 0
    assert ws(binding.OP_CROSS_ENTROPY_BACKWARD, 128, 1000, 12, 0) == 0  # k not a multiple of 8
    assert ws(binding.OP_CROSS_ENTROPY_BACKWARD, 128, 1000, 64, 300) == 0
    small, sketched = (ws(binding.OP_CROSS_ENTROPY_BACKWARD, 128, 1000, 64, r) for r in (0, 16))
    assert 0 < small < sketched
    # the logit gradients of a large head are bounded by its pieces, not by T x V
    assert ws(binding.OP_CROSS_ENTROPY_BACKWARD, 8192, 131072, 4096, 0) < 8192 * 131072 * 2 // 2
    assert ws(binding.OP_LAYER_NORM_BACKWARD, 1000, 0, 64) > 0
    assert ws(binding.OP_LAYER_NORM_BACKWARD, 0, 0, 64) == 0


def test_binding_refuses_wrong_tensors(lib):
    bf = torch.zeros(4, 8, dtype=torch.bfloat16)
    f = torch.zeros(4)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        binding.layer_norm_forward(bf.double(), None, None, bf, f, f)
    with pytest.raises(ValueError, match="CUDA"):
        binding.layer_norm_forward(bf, None, None, bf, f, f)
    with pytest.raises(ValueError, match="CUDA"):
        binding.layer_norm_backward(bf, bf, None, f, f, bf)
    with pytest.raises(ValueError, match="CUDA"):
        binding.cross_entropy_forward(bf, bf, torch.zeros(4, dtype=torch.int64), f, f)
    with pytest.raises(ValueError, match="CUDA"):
        AdamW([f], [f])
    with pytest.raises(ValueError, match="state_bits"):
        AdamW([f], [f], state_bits=16)
    with pytest.raises(ValueError, match="no tensors"):
        AdamW([], [])
    with pytest.raises(ValueError, match="states"):
        AdamW([f], [f], state={"m": [f]})
    with pytest.raises(ValueError, match="one length"):
        binding.adamw_problems([f], [], [f], [f])


def test_exports_list_the_operators(lib):
    for name in ("sketch_layer_norm_forward", "sketch_layer_norm_backward", "sketch_cross_entropy_forward",
                 "sketch_cross_entropy_backward", "sketch_adamw_batched"):
        assert name in binding.EXPORTS and hasattr(lib, name)
    assert ctypes.sizeof(binding.AdamWProblem) == 72


@pytest.mark.parametrize("where,contiguous,size", [("cuda:1", True, 1 << 20), ("cpu", True, 1 << 20), ("cuda:0", False, 1 << 20),
                                                   ("cuda:0", True, 1000)])
def test_callers_workspace_is_refused(lib, where, contiguous, size):
    """On another device, without storage of its own for every element (an expanded tensor), too small."""

    class Workspace:
        device, is_cuda = torch.device(where), where != "cpu"
        numel, element_size, data_ptr = lambda self: size, lambda self: 1, lambda self: A
        is_contiguous = lambda self: contiguous  # noqa: E731

    with pytest.raises(ValueError, match="workspace"):
        binding._scratch(binding.OP_CROSS_ENTROPY_FORWARD, 128, 1000, 64, 0, torch.device("cuda:0"), None, Workspace())


@pytest.mark.parametrize("scale", [torch.ones(1), torch.ones(2), torch.ones(1, dtype=torch.bfloat16), torch.tensor([1.0, 2.0])[:1]])
def test_adamw_batched_refuses_a_grad_scale_that_a_kernel_cannot_read(lib, scale):
    """The list function checks it as AdamW.step does (an empty tensor: nothing would be launched)."""

    class Stream:
        cuda_stream = 0

    probs = (binding.AdamWProblem * 1)(binding.AdamWProblem(NULL, NULL, NULL, NULL, NULL, NULL, 0, 0, 0, 0))
    call = lambda s: binding.adamw_batched(probs, 1e-3, (0.9, 0.999), 1e-8, 0.0, 0, 0, grad_scale=s,  # noqa: E731
                                           device=torch.device("cuda:0"), stream=Stream())
    call(None)
    with pytest.raises(ValueError, match="grad_scale"):
        call(scale)


@pytest.mark.parametrize("T,k,V", [(1 << 24, 16, 1 << 24), (1 << 24, 1 << 23, 256), (256, 1 << 24, 1 << 23)])
def test_cross_entropy_refuses_more_tiles_than_a_launch_counts(lib, T, k, V):
    """Sizes below 2^24 each, by either call, with any workspace; asked for one, the sizes are invalid too."""
    kw = dict(T=T, k=k, V=V, ld_x=k, ld_w=k, ws_bytes=1 << 62)
    refused(lib, ce_forward(lib, **kw), binding.ERR_UNSUPPORTED, "2^28 tiles")
    refused(lib, ce_backward(lib, ld_dx=k, ld_dw=k, **kw), binding.ERR_UNSUPPORTED, "2^28 tiles")
    assert binding.workspace_bytes(binding.OP_CROSS_ENTROPY_BACKWARD, T, V, k, 0) == 0
