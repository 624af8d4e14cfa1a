"""oq_qk_norm_rope of more tokens than the workgroups of one launch."""
import pytest
import torch

import rotated_bit_quantized_amd as oq
from test_gpu_heads import _check, _exact, _tables

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


@pytest.mark.parametrize("T", [(1 << 29) + 77])
def test_head_norm_of_more_tokens_than_a_launch_takes(T):
    """One query head of 8 elements."""
    g = torch.Generator(device=DEV).manual_seed(0)
    q = torch.empty(T, 1, 8, dtype=BF, device=DEV).normal_(generator=g)
    w = 1 + 0.3 * torch.randn(8, generator=g, device=DEV)
    rope = oq.Rope(*_tables(100, 8))
    pos = torch.randint(0, 100, (T,), generator=g, device=DEV, dtype=torch.int32)
    out = torch.full_like(q, float("nan"))
    oq.oq_qk_norm_rope(q, None, w, None, 1e-6, rope, pos, q_out=out)
    step = 1 << 24
    for t in range(0, T, step):
        _check(out[t:t + step], *_exact(q[t:t + step], w, rope, pos[t:t + step]))
    del q, out, pos
    torch.cuda.empty_cache()
