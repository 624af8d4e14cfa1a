"""The example's sparse layer: the experts are the best of the float64 layer within
the rounding of the normed stream, and the alternatives are the head's largest logits.

The router reads h in bfloat16, each element off by 2^-8 of itself at most, so a
logit by 2^-8 sum |h w| and a float32 product's 2^-16 of that; h itself comes from
float32 sums, another 2^-16.  The float64 layer's stream is rounded nowhere, the
tested one's r is not rounded before h.  A softmax keeps the order of its logits; a
sigmoid's slope is at most a quarter."""
import pytest
import torch

from test_gpu_sparse_layer import ex, inputs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hidden,f,E,k,V,T", [(256, 128, 8, 2, 500, 5), (512, 256, 60, 4, 3001, 33), (1024, 384, 128, 8, 1000, 130)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_choices_and_alternatives(ex, hidden, f, E, k, V, T, score):  # noqa: F811
    bias = 0.05 * torch.randn(E, generator=torch.Generator().manual_seed(2)).cuda() if score == "sigmoid" else None
    layer, weights = ex.random_layer(hidden, f, E, k, V, seed=3, score=score, bias=bias)
    y, r = inputs(T, hidden, 4)
    r_out, h, ids, w = layer.forward(y, r)
    logits, answer = layer.answer(h, torch.zeros(T, 1, dtype=torch.int32, device="cuda"), 7)

    stream = y.double() + r.double()
    normed = stream / (stream.square().mean(1, keepdim=True) + 1e-6).sqrt() * weights[4].double()
    x = normed @ weights[0].double().t().contiguous()
    err = (2.0 ** -8 + 2.0 ** -15) * (normed.abs() @ weights[0].double().abs().t().contiguous())
    c = x if score == "softmax" else torch.sigmoid(x) + bias.double()
    if score == "sigmoid":
        err = err / 4 + 2.0 ** -20
    chosen = torch.zeros(T, E, dtype=torch.bool, device="cuda").scatter_(1, ids.long(), True)
    assert (chosen.sum(1) == k).all()
    worst = torch.where(chosen, c + err, torch.full_like(c, float("inf"))).amin(1)
    best_left = torch.where(chosen, torch.full_like(c, -float("inf")), c - err).amax(1)
    assert (worst >= best_left).all()
    assert float(err.mean()) < 0.15 * float(c.std())  # the bound tells experts apart
    # weights: a logit's error moves a score by as much of itself, and the sum likewise
    s = (torch.softmax(x, 1) if score == "softmax" else torch.sigmoid(x)).gather(1, ids.long())
    far = 2 * (2.0 ** -8 + 2.0 ** -15) * (normed.abs() @ weights[0].double().abs().t().contiguous()).amax(1, keepdim=True)
    want = s / s.sum(1, keepdim=True)
    assert ((w.double() - want).abs() <= torch.expm1(far) * want + 2.0 ** -20).all()

    assert torch.equal(answer[4].long(), torch.sort(logits.float(), dim=1, descending=True, stable=True).indices[:, :7])
    lp = torch.log_softmax(logits.double(), 1)
    assert float((answer[5] - lp.gather(1, answer[4].long())).abs().max()) < 1e-5
