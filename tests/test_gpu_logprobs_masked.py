"""oq_logprobs: rows that hold NaN beside logits of the type's lowest value."""
import pytest
import torch

import rotated_bit_quantized_amd as oq

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,V", [(4, 300), (4, 40000), (600, 9000)])
@pytest.mark.parametrize("scale", [1.0, 1.4])
def test_a_row_with_nan_gives_nan_for_masked_tokens_too(T, V, dtype, scale):
    g = torch.Generator(device=DEV).manual_seed(V)
    x = torch.randn(T, V, generator=g, device=DEV).to(dtype)
    x[:, V // 2:] = torch.finfo(dtype).min
    x[1, 5] = float("nan")
    x[2, V - 2] = float("nan")
    tok = torch.tensor([V - 1, V // 2, 0], dtype=torch.int32, device=DEV).repeat(T, 1)
    logprob, _, entropy, lse, _, top_logprob = oq.oq_logprobs(x, tok, top=min(V, 20), scale=scale)
    sound = [t for t in range(T) if t not in (1, 2)]
    for got in (logprob, entropy, lse, top_logprob):
        assert torch.isnan(got[1:3]).all() and not torch.isnan(got[sound]).any()
    assert (logprob[sound][:, :2] < -1e38).all()
