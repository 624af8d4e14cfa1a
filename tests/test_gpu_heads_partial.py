"""Partly rotated heads (oq_qk_norm_rope, oq_kv_append): the elements that the
rotary embedding leaves alone."""
import pytest
import torch

import rotated_bit_quantized_amd as oq
from test_gpu_heads import EPS, _check, _exact, _tables, _x

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("d,dim,inter", [(128, 64, False), (128, 64, True), (80, 40, False), (80, 40, True), (64, 32, False),
                                         (64, 10, False), (64, 10, True), (256, 128, False), (512, 256, True), (64, 16, False)])
@pytest.mark.parametrize("T", [3, 9000])
def test_elements_past_the_rotation_stay(d, dim, inter, T):
    """Without a norm, elements dim .. d - 1 pass bit for bit, infinities, -0 and
    largest values among them, and nothing of them reaches the rotated ones."""
    H = 5 if T > 100 else 2
    q, k = _x(T, H, d, 1), _x(T, H, d, 2)
    for x in (q, k):
        x[0, 0, dim] = float("inf")
        x[0, 1, d - 1] = float("-inf")
        x[1, 0, dim : dim + 3] = -0.0
        x[1, 1, d - 2] = -3e38
        x[2, :, dim:] = float("inf")
        x[2, 0, dim + 1] = 0.0
    rope = oq.Rope(*_tables(100, dim), inter)
    pos = torch.randint(0, 100, (T,), generator=torch.Generator(device=DEV).manual_seed(3), device=DEV).int()
    qo, ko = oq.oq_qk_norm_rope(q, k, None, None, EPS, rope, pos)
    pages = -(-T // 16)
    kv = oq.PagedKV(*(torch.zeros(pages, H, 16, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)))
    slot = torch.arange(T, device=DEV)
    oq.oq_kv_append(k, q, slot, kv, None, EPS, rope, pos)
    for x, y in ((q, qo), (k, ko), (k, kv.k[slot // 16, :, slot % 16])):
        assert torch.equal(y[..., dim:].contiguous().view(torch.int16), x[..., dim:].contiguous().view(torch.int16))
        want, mag = _exact(x, None, rope, pos)
        _check(y[..., :dim], want[..., :dim], mag[..., :dim])


@pytest.mark.parametrize("dim,inter", [(64, False), (64, True), (10, True)])
def test_infinity_past_the_rotation_under_a_norm(dim, inter):
    """A head of infinite norm: zeros, and NaN in the infinity's own place alone."""
    q = _x(4, 3, 128, 1)
    q[1, 2, 101] = float("inf")
    w = torch.rand(128, device=DEV) + 0.5
    rope = oq.Rope(*_tables(4, dim), inter)
    qo, _ = oq.oq_qk_norm_rope(q, None, w, None, EPS, rope)
    head = qo[1, 2].float()
    assert torch.isnan(head[101]) and (head[torch.arange(128, device=DEV) != 101] == 0).all()
