"""oq_attn_prefix of more query rows than the workgroups of one launch join."""
import math

import pytest
import torch

import rotated_bit_quantized_amd as oq

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def test_attention_of_more_rows_than_a_launch_joins():
    """2^20 sequences of one token and 64 heads, a prefix and own keys: 2^26 rows in two parts."""
    B, H, D, page, prefix = (1 << 20) + 77, 64, 64, 16, 13
    g = torch.Generator(device=DEV).manual_seed(0)
    k, v = (torch.randn(64, 1, page, D, generator=g, device=DEV).to(BF) for _ in range(2))
    q = torch.empty(B, H, D, dtype=BF, device=DEV).normal_(generator=g)
    table = torch.randint(1, 64, (B, 1), generator=g, device=DEV, dtype=torch.int32)
    lens = torch.randint(0, page + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    o = torch.full_like(q, float("nan"))
    scale = 1 / math.sqrt(D)
    oq.oq_attn_prefix(q, 1, oq.PagedKV(k, v), torch.zeros(1, dtype=torch.int32, device=DEV), prefix, table, lens, scale, o=o)
    for b in range(0, B, 1 << 16):
        assert not torch.isnan(o[b:b + (1 << 16)]).any(), f"sequences {b} .. hold outputs that were not written"
    for b in (0, B // 3, (1 << 20) - 250, B - 300):
        s = slice(b, b + 300)
        keys, values = (torch.cat((c[0, 0, :prefix].double().expand(300, prefix, D), c[table[s, 0].long(), 0].double()), 1) for c in (k, v))
        seen = torch.cat((torch.ones(300, prefix, dtype=torch.bool, device=DEV), torch.arange(page, device=DEV) < lens[s, None]), 1)[:, None]
        at = keys.transpose(1, 2).contiguous()
        x = torch.bmm(q[s].double(), at).mul_(scale).masked_fill(~seen, -math.inf)
        mag = (torch.bmm(q[s].double().abs(), at.abs()) * scale).masked_fill(~seen, 0).amax(-1, keepdim=True)
        p = torch.softmax(x, -1)
        y, A = torch.bmm(p, values), torch.bmm(p, values.abs())
        tol = 2.0 ** -8 * y.abs() + A * (1.01 * 2.0 ** -8 + 2 * (D + 4) * 2.0 ** -24 * mag + 2.0 ** -18)  # as in test_gpu_attn_prefix.py
        assert ((o[s].double() - y).abs() <= tol).all()
    del q, o
    torch.cuda.empty_cache()
