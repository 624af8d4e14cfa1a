"""oq_residual_norm of more rows than the workgroups of one launch."""
import pytest
import torch

import rotated_bit_quantized_amd as oq

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("T", [(1 << 29) + 41])
def test_more_rows_than_a_launch_takes(T):
    d = 8
    g = torch.Generator(device=DEV).manual_seed(0)
    r = torch.empty(T, d, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    h = torch.full((T, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    w = 1 + 0.1 * torch.randn(d, generator=g, device=DEV)
    oq.oq_residual_norm(None, r, pre=oq.Norm(oq.OQ_NORM_RMS, d, w=w), h=h, want_r=False)
    step = 1 << 25
    for t in range(0, T, step):
        x = r[t:t + step].double()
        want = x / (x.square().mean(1, keepdim=True) + 1e-6).sqrt() * w.double()
        # the float32 part is off by less than 64 units of 2^-24, the result by half a step of bfloat16
        assert ((h[t:t + step].double() - want).abs() <= (2.0 ** -8 + 64 * 2.0 ** -24) * want.abs() + 2.0 ** -120).all()
    del r, h
    torch.cuda.empty_cache()
