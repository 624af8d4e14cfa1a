"""Zeros of oq_gemm_w8a8: their sign does not depend on the kernel that the
sizes select."""
import pytest
import torch

import rotated_bit_quantized_amd as oq

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("epi", ["plain", "mean", "bias", "full"])
@pytest.mark.parametrize("K", [16, 528])
def test_bits_do_not_depend_on_the_batch(epi, K):
    """Rows of scale zero and weights of negative scale, so that products are -0."""
    g = torch.Generator().manual_seed(K)
    M, N = 700, 1000
    qa = torch.randint(-127, 128, (M, K), generator=g).to(torch.int8).to(DEV)
    w = torch.randint(-127, 128, (N, K), generator=g).to(torch.int8).to(DEV)
    a_s, w_s = torch.rand(M, generator=g).to(DEV), (torch.rand(N, generator=g) - 0.5).to(DEV)
    a_s[::3] = 0
    mean, w1 = torch.randn(M, generator=g).to(DEV), torch.randn(N, generator=g).to(DEV)
    mean[::2], bias = 0, torch.randn(N, generator=g).to(DEV)
    bias[::2] = -0.0
    w1[::5] = -0.0
    kw = dict(w1=w1 if epi in ("mean", "full") else None, bias=bias if epi in ("bias", "full") else None)

    def run(m):
        return oq.oq_gemm_w8a8(qa[:m], a_s[:m], w, w_s, mean=mean[:m] if kw["w1"] is not None else None, **kw)

    whole = run(M)
    for m in (1, 5, 16, 20, 33, 100, 300):
        assert torch.equal(run(m).view(torch.int16), whole[:m].view(torch.int16)), m
