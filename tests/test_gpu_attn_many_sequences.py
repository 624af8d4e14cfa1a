"""oq_attn_prefix of more sequences than the workgroups of one launch take."""
import math

import pytest
import torch

import rotated_bit_quantized_amd as oq

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def test_attention_of_more_sequences_than_a_launch_takes():
    """2^26 sequences of one token and one head with keys of their own, a wavefront each."""
    B, D, page = (1 << 26) + 77, 64, 16
    g = torch.Generator(device=DEV).manual_seed(0)
    k, v = (torch.randn(64, 1, page, D, generator=g, device=DEV).to(BF) for _ in range(2))
    q = torch.empty(B, 1, D, dtype=BF, device=DEV).normal_(generator=g)
    table = torch.randint(0, 64, (B, 1), generator=g, device=DEV, dtype=torch.int32)
    lens = torch.randint(1, page + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    o = torch.full_like(q, float("nan"))
    scale = 1 / math.sqrt(D)
    oq.oq_attn_prefix(q, 1, oq.PagedKV(k, v), None, 0, table, lens, scale, o=o)
    for b in range(0, B, 1 << 22):
        assert not torch.isnan(o[b:b + (1 << 22)]).any(), f"sequences {b} .. hold outputs that were not written"
    for b in (0, B // 3, (1 << 26) - 250, B - 300):
        s = slice(b, b + 300)
        keys, values = (c[table[s, 0].long(), 0].double() for c in (k, v))
        hidden = (torch.arange(page, device=DEV) >= lens[s, None])[:, None]
        at = keys.transpose(1, 2).contiguous()
        x = torch.bmm(q[s].double(), at).mul_(scale).masked_fill(hidden, -math.inf)
        mag = (torch.bmm(q[s].double().abs(), at.abs()) * scale).masked_fill(hidden, 0).amax(-1, keepdim=True)
        p = torch.softmax(x, -1)
        y, A = torch.bmm(p, values), torch.bmm(p, values.abs())
        tol = 2.0 ** -8 * y.abs() + A * (1.01 * 2.0 ** -8 + 2 * (D + 4) * 2.0 ** -24 * mag + 2.0 ** -18)  # as in test_gpu_attn_prefix.py
        assert ((o[s].double() - y).abs() <= tol).all()
    del q, o
    torch.cuda.empty_cache()
