"""oq_gemm_w8a8 of the most tokens that it takes, more than one launch does."""
import pytest
import torch

import rotated_bit_quantized_amd as oq

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("N", [8, 70])
def test_the_most_tokens(N):
    M, K = 1 << 30, 16
    g = torch.Generator(device=DEV).manual_seed(N)
    qa = torch.randint(-127, 128, (1 << 20, K), generator=g, device=DEV, dtype=torch.int32).to(torch.int8).repeat(M >> 20, 1)
    w = torch.randint(-127, 128, (N, K), generator=g, device=DEV, dtype=torch.int32).to(torch.int8)
    a_scale = torch.rand(M, generator=g, device=DEV) * 1e-4 + 1e-4
    w_scale, w1, bias = torch.rand(N, generator=g, device=DEV) + 0.1, torch.randn(N, generator=g, device=DEV), torch.randn(N, generator=g, device=DEV)
    mean = torch.rand(M, generator=g, device=DEV)
    y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    oq.oq_gemm_w8a8(qa, a_scale, w, w_scale, mean, w1, bias, y=y)
    acc = qa[: 1 << 20].double() @ w.double().t().contiguous()
    for m in range(0, M, 1 << 20):
        s = slice(m, m + (1 << 20))
        if N > 8 and 1 << 20 < m < M - (1 << 20):
            assert not torch.isnan(y[s]).any()
            continue
        p, q = acc * (a_scale[s].double()[:, None] * w_scale.double()), mean[s].double()[:, None] * w1.double()
        want = p + q + bias.double()
        tol = 2.0 ** -8 * want.abs() + 2.0 ** -21 * (p.abs() + q.abs() + bias.double().abs())  # as in test_gpu_w8a8.py
        assert ((y[s].double() - want).abs() <= tol).all()
    del qa, y, mean, a_scale
    torch.cuda.empty_cache()
