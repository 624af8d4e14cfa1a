"""oq_gemm_w8a8_experts with more workgroups than one launch takes: short rows of
very many outputs."""
import pytest
import torch

import rotated_bit_quantized_amd as oq

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("each", [16, 65])
def test_more_tiles_than_a_launch_takes(each):
    """1024 experts of 2^20 weight rows of 16: 2^23 workgroups of 512 threads.  Every expert has `each` entries."""
    E, N, K = 1024, 1 << 20, 16
    n = E * each
    g = torch.Generator(device=DEV).manual_seed(each)
    w = torch.empty(E, N, K, dtype=torch.int8, device=DEV)
    for e in range(0, E, 64):
        w[e:e + 64] = torch.randint(-127, 128, (64, N, K), generator=g, device=DEV, dtype=torch.int16).to(torch.int8)
    qa = torch.randint(-127, 128, (n, K), generator=g, device=DEV, dtype=torch.int16).to(torch.int8)
    a_scale, w_scale = torch.rand(n, generator=g, device=DEV) * 1e-4 + 1e-4, torch.rand(E, N, generator=g, device=DEV) + 0.1
    order = torch.arange(n, dtype=torch.int32, device=DEV).view(each, E).t().contiguous().flatten()  # entry i has expert i % E
    offsets = torch.arange(E + 1, dtype=torch.int32, device=DEV) * each
    y = torch.full((n, N // 2), float("nan"), dtype=torch.bfloat16, device=DEV)
    oq.oq_gemm_w8a8_experts(qa, a_scale, w, w_scale, offsets, order, act=oq.OQ_ACT_SWIGLU, y=y)
    for i in range(0, n, 256):
        assert not torch.isnan(y[i:i + 256]).any(), f"rows {i} .. hold outputs that were not written"
    for i in [0, 1, E - 1, E, n // 2 + 5, n - E - 1, n - 2, n - 1] + torch.randint(0, n, (40,), generator=torch.Generator().manual_seed(1)).tolist():
        e = i % E
        v = a_scale[i].double() * w_scale[e].double() * (w[e].double() @ qa[i].double())
        gate, up = v.chunk(2)
        s = gate * torch.sigmoid(gate)
        mag_g, mag_u = gate.abs() * 2.0 ** -21, up.abs() * 2.0 ** -21
        tol = 2.0 ** -7.9 * (s * up).abs() + 2 * mag_g * up.abs() + s.abs() * mag_u + mag_g * mag_u
        assert ((y[i].double() - s * up).abs() <= tol).all()
    del y, w, w_scale
    torch.cuda.empty_cache()
