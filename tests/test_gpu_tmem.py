"""Kernels in clusters that take tensor memory, beside each other on several streams: accumulations at the ranks
whose blocks have 256 columns, products of few tokens, projections and Gram matrices.  Results are those of each alone."""
import pytest
import torch

import rank_gradient_sketching_philox_gb300 as rgs

pytestmark = pytest.mark.gpu
BF, E4 = torch.bfloat16, torch.float8_e4m3fn


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * std


def product(seed, T, N, k):
    g = gen(seed)
    A, B = rgs.code_rows(T, k), rgs.code_rows(N, k)
    A.copy_(normal(g, T, k, std=60.0).clamp(-448, 448).to(E4))
    B.copy_(normal(g, N, k, std=60.0).clamp(-448, 448).to(E4))
    sa, sb = torch.rand(T, (k + 127) // 128, generator=g, device="cuda"), torch.rand((N + 127) // 128, (k + 127) // 128, generator=g, device="cuda")
    Y = torch.zeros(T, N, dtype=BF, device="cuda")
    return Y, lambda stream: rgs.matmul_blocks(A, sa, B, sb, Y, stream=stream)


def sketch(seed, T, d, r):
    g = gen(seed)
    D, XP = normal(g, T, d).to(BF), normal(g, T, r).to(BF)
    C = torch.zeros(d, r, device="cuda")
    return C, lambda stream: rgs.accumulate(D, XP, C, overwrite=True, stream=stream)


def projected(seed, T, k, r):
    g = gen(seed)
    X, P = normal(g, T, k).to(BF), normal(g, k, r)
    XP = torch.zeros(T, r, dtype=BF, device="cuda")
    return XP, lambda stream: rgs.project_inputs(X, P, XP, stream=stream)


def frame(seed, k, r):
    P = torch.zeros(k, r, device="cuda")
    return P, lambda stream: rgs.sample_projection(rgs.PROJ_GAUSSIAN_QR, seed, 0, 0, P, stream=stream)


@pytest.mark.parametrize("r", [136, 144, 160, 192])
def test_accumulations_beside_products_of_few_tokens(r):
    work = [sketch(1, 4096, 1024, r), sketch(2, 2048, 2048, r), sketch(3, 4096, 512, r), product(4, 8, 2048, 4096),
            product(5, 16, 1024, 4096), product(6, 24, 2048, 2048), product(7, 1, 4096, 2048), projected(8, 512, 2048, r),
            frame(9, 2048, 64), frame(10, 2048, r)]
    for _, call in work:
        call(None)
    torch.cuda.synchronize()
    want = [out.clone() for out, _ in work]
    for out, _ in work:
        out.zero_()
    streams = [torch.cuda.Stream() for _ in work]
    torch.cuda.synchronize()
    for _ in range(30):
        for (_, call), stream in zip(work, streams):
            call(stream)
    torch.cuda.synchronize()
    assert rgs.read_device_errors() == 0
    for (out, _), w in zip(work, want):
        assert torch.equal(out, w)
