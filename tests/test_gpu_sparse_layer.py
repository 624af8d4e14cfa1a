"""The example's sparse layer (residual stream and norms, routing, the experts'
products, the answer) against a float64 layer with the same experts.

Bound on the distance, as a part of the output's norm.  An int8 code is within
half a scale of its value; after the rotation the rms error is 0.8% of the rms
(largest value about 3.5 deviations, / 127 / sqrt(12)), for activations and
weights of a projection 1.1% together.  SwiGLU: gate and up 1.1% each, and the
gate's derivative next to its value at most doubles its share: 2.5%.  The down
projection 1.1% more, bfloat16 roundings 0.2% each: 3% of the experts' sum,
which the norm behind it passes on and the head's projection raises by 1.1%.
The bound is 6%."""
import importlib.util
import os

import pytest
import torch

import rotated_bit_quantized_amd as oq

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "sparse_layer.py")


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("sparse_layer", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def rel(got, want):
    return float((got.double() - want).norm() / want.norm())


def inputs(T, hidden, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return tuple(torch.randn(T, hidden, generator=g, device="cuda").bfloat16() for _ in range(2))


@pytest.mark.parametrize("hidden,f,E,k,V,T", [(256, 128, 8, 2, 500, 5), (512, 256, 60, 4, 3001, 33), (1024, 384, 128, 8, 1000, 130), (512, 256, 8, 2, 700, 600)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_against_float64(ex, hidden, f, E, k, V, T, score):
    bias = 0.05 * torch.randn(E, generator=torch.Generator().manual_seed(2)).cuda() if score == "sigmoid" else None
    layer, weights = ex.random_layer(hidden, f, E, k, V, seed=3, score=score, bias=bias)
    y, r = inputs(T, hidden, 4)
    r_out, h, ids, w = layer.forward(y, r)
    tokens = torch.arange(T, device="cuda", dtype=torch.int32)[:, None] % V
    logits, (logprob, rank, entropy, lse, top_id, top_logprob) = layer.answer(h, tokens, 3)
    some = torch.arange(0, T, max(1, T // 24), device="cuda")
    want_r, want_h, score_of, want_logits = ex.reference(weights, y[some], r[some], ids[some], score, bias)
    assert rel(r_out[some], want_r) < 0.06 and rel(h[some], want_h) < 0.06 and rel(logits[some], want_logits) < 0.06
    # the experts are the best ones but for the rounding of h (2^-8 of a logit of about 1)
    best = score_of.topk(k, 1).values
    assert float((best - score_of.gather(1, ids[some].long())).max()) < 0.05
    lp = torch.log_softmax(logits.double(), 1)
    assert float((logprob[:, 0] - lp.gather(1, tokens.long())[:, 0]).abs().max()) < 1e-4
    assert torch.equal(top_id, lp.topk(3, 1).indices.int()) or float((top_logprob - lp.topk(3, 1).values).abs().max()) < 1e-4


def test_padding_leaves_the_stream_alone(ex):
    layer, _ = ex.random_layer(256, 128, 8, 2, 300, seed=1)
    T = 40
    y, r = inputs(T, 256, 2)
    mask = (torch.arange(T, device="cuda") % 3 > 0).to(torch.uint8)
    y_bad, r_bad = y.clone(), r.clone()
    y_bad[mask == 0] = float("nan")
    full = layer.forward(y, r)
    part = layer.forward(y_bad, r_bad, mask)
    live = mask > 0
    for a, b in zip(full[:2], part[:2]):
        assert torch.equal(a[live], b[live])
    assert (part[2][~live] == -1).all() and (part[3][~live] == 0).all()
    assert torch.equal(full[2][live], part[2][live]) and torch.equal(full[3][live], part[3][live])


def test_graph_gives_the_eager_steps(ex):
    layer, _ = ex.random_layer(512, 256, 16, 4, 2000, seed=5)
    T = 50
    pairs = [inputs(T, 512, s) for s in range(4)]
    tokens = torch.arange(T, device="cuda", dtype=torch.int32)[:, None]

    def step(y, r):
        out = layer.forward(y, r)
        logits, answer = layer.answer(out[1], tokens, 4)
        return (*out, logits, *answer)

    want = [step(*p) for p in pairs]
    y, r = (torch.empty_like(t) for t in pairs[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(y, r)
    for i, p in enumerate(pairs):
        y.copy_(p[0]), r.copy_(p[1])
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want[i]))
        step(*pairs[3 - i])
        torch.cuda.synchronize()


def test_command(ex, capsys):
    ex.main(hidden=512, f=256, E=16, k=2, V=1000, T=8, steps=3)
    assert "us a step" in capsys.readouterr().out
