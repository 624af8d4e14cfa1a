"""oq_route: weights of a softmax over logits that hold +inf.  The formula gives
NaN for every score of such a row, whether or not the infinite expert is chosen."""
import pytest
import torch

import rotated_bit_quantized_amd as oq

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("how", [dict(), dict(bias=True), dict(groups=4, top_groups=2, group_best=2), dict(groups=4, top_groups=1, group_best=2, bias=True),
                                 dict(groups=4, top_groups=2, group_best=1)])
@pytest.mark.parametrize("E", [64, 500])
def test_softmax_of_an_infinite_logit(dtype, renorm, how, E):
    how = dict(how)
    g = torch.Generator(device=DEV).manual_seed(E)
    x = torch.randn(40, E, generator=g, device=DEV).to(dtype)
    x[3, E - 1] = x[7, E // 2] = x[20, 0] = float("inf")
    x[9, E - 2], x[9, 1] = float("inf"), -float("inf")
    x[11, 5] = -float("inf")
    if how.get("bias"):
        how["bias"] = 0.1 * torch.randn(E, generator=g, device=DEV)
    ids, w, offsets, order = oq.oq_route(x, oq.Router(E, 8, renorm=renorm, **how))
    infinite = (x == float("inf")).any(1)
    assert int(infinite.sum()) == 4
    assert torch.isnan(w[infinite]).all()
    assert torch.isfinite(w[~infinite]).all()
    assert int(ids.min()) >= 0 and int(ids.max()) < E and all(len(set(r)) == 8 for r in ids.tolist())
    assert int(offsets[-1]) == 320 and torch.equal(order.sort().values.cpu(), torch.arange(320, dtype=torch.int32))


def test_sigmoid_of_an_infinite_logit_is_one():
    x = torch.zeros(2, 64, device=DEV)
    x[0, 9] = float("inf")
    ids, w, *_ = oq.oq_route(x, oq.Router(64, 3, score="sigmoid", renorm=False))
    assert ids[0].tolist() == [9, 0, 1] and w[0].tolist() == [1.0, 0.5, 0.5] and w[1].tolist() == [0.5] * 3
