"""oq_gemm_w8a8_experts: SwiGLU of gates far from zero, whose sigmoid is below what
float32 holds as a normal number while its product with gate and up is not.

The codes are 0, so that the bias is the projections' value without an error.  In
units of 2^-24: the exponential's argument is off by 1.5 |gate|, exponential,
reciprocal and products add 16; the bfloat16 result 2^-8 of the value, and half a
step of 2^-133 where it is subnormal."""
import pytest
import torch

import rotated_bit_quantized_amd as oq

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("K,n", [(64, 5), (64, 300), (400, 200)])
@pytest.mark.parametrize("lo,hi,up", [(-95, -84, 1.0), (-95, -84, 3e20), (-95, -84, -1e38), (-120, -60, 1e30), (-170, -90, 1e37), (-170, -90, -3e38), (-12, 12, 3.0),
                                      (0, 90, 1e30), (0, 1, 3e38), (80, 100, -1e-3), (-1e-3, 1e-3, 1e-30)])
def test_far_gates(K, n, lo, hi, up):
    f = 160
    g = torch.Generator(device=DEV).manual_seed(n)
    gate = lo + (hi - lo) * torch.rand(f, generator=g, device=DEV)
    ups = up * (0.2 + 0.8 * torch.rand(f, generator=g, device=DEV))
    zero = lambda *s: torch.zeros(*s, dtype=torch.int8, device=DEV)  # noqa: E731
    one = lambda *s: torch.ones(*s, device=DEV)  # noqa: E731
    offsets = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    order = torch.arange(n, dtype=torch.int32, device=DEV)
    y = oq.oq_gemm_w8a8_experts(zero(n, K), one(n), zero(1, 2 * f, K), one(1, 2 * f), offsets, order, act=oq.OQ_ACT_SWIGLU,
                                bias=torch.cat((gate, ups))[None].contiguous())
    d = gate.double()
    s = torch.where(d < 0, torch.exp(d) / (1 + torch.exp(d)), 1 / (1 + torch.exp(-d)))
    want = (d * s * ups.double()).expand(n, f)
    tol = (2.0 ** -8 + (1.5 * d.abs() + 16) * 2.0 ** -24) * want.abs() + 2.0 ** -133
    off = (y.double() - want).abs()
    assert (off <= tol).all(), f"{int((off > tol).sum())} outside, got {y[off > tol][:3].tolist()}, want {want[off > tol][:3].tolist()}"


@pytest.mark.parametrize("K,n", [(64, 5), (400, 200)])
def test_gates_that_are_not_finite(K, n):
    inf, nan = float("inf"), float("nan")
    gate = torch.tensor([inf, -inf, nan, 0.0, 1.0, 1.0, -1.0, inf] * 4, device=DEV)
    ups = torch.tensor([2.0, 2.0, 2.0, inf, nan, inf, inf, 0.0] * 4, device=DEV)
    zero = lambda *s: torch.zeros(*s, dtype=torch.int8, device=DEV)  # noqa: E731
    one = lambda *s: torch.ones(*s, device=DEV)  # noqa: E731
    y = oq.oq_gemm_w8a8_experts(zero(n, K), one(n), zero(1, 64, K), one(1, 64), torch.tensor([0, n], dtype=torch.int32, device=DEV),
                                torch.arange(n, dtype=torch.int32, device=DEV), act=oq.OQ_ACT_SWIGLU, bias=torch.cat((gate, ups))[None].contiguous())
    want = torch.tensor([inf, nan, nan, nan, nan, inf, -inf, nan] * 4, device=DEV).bfloat16().expand(n, 32)
    assert torch.equal(torch.isnan(y), torch.isnan(want)) and torch.equal(y[~torch.isnan(y)], want[~torch.isnan(want)])
