"""The example's attention layer (projections, norm and rotation, cache,
attention) against a float64 layer.

Bound on the distance, as a part of the output's norm.  An int8 code is within
half a scale of its value, a scale is the row's largest value / 127: after the
rotation the values are near normal, largest about 3.5 deviations, so the rms
error is 3.5 / 127 / sqrt(12) = 0.8% of the rms, for the activations and for
the weights of both projections, 2 sqrt(2) 0.8% = 2.3% where they only add.
Scores (norm about 1 after the softmax scale) off by the first projection's
1.1% on both sides move the weights by less than 2%; bfloat16 roundings add
0.2% each.  Root sum of squares about 3%; the bound is 6%."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_layer.py")


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("attention_layer", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def rel(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("hidden,heads,kv_heads,d,B,prompt_len", [(256, 4, 2, 64, 3, 37), (512, 8, 1, 128, 9, 200),
                                                                  (1024, 8, 8, 64, 40, 130)])
def test_decode_against_float64(ex, hidden, heads, kv_heads, d, B, prompt_len):
    steps = 19  # past the end of a page of 16
    layer, weights = ex.random_layer(hidden, heads, kv_heads, d, prompt_len + steps, seed=2)
    g = torch.Generator(device="cuda").manual_seed(3)
    prompt = torch.randn(prompt_len, hidden, generator=g, device="cuda").bfloat16()
    xs = torch.randn(steps, B, hidden, generator=g, device="cuda").bfloat16()
    dec = ex.Decoder(layer, prompt, B, steps, page=16)
    for t in (0, prompt_len // 2, prompt_len - 1):
        assert rel(dec.prompt_y[t], ex.reference(weights, heads, kv_heads, d, prompt[: t + 1])) < 0.06
    for i, x in enumerate(xs):
        dec.x.copy_(x)
        y = dec.step()
        if i in (0, 15, 16, steps - 1):
            for b in (0, B - 1):
                want = ex.reference(weights, heads, kv_heads, d, torch.cat((prompt, xs[: i + 1, b])))
                assert rel(y[b], want) < 0.06, (i, b)


def test_graph_gives_the_eager_steps(ex):
    layer, _ = ex.random_layer(256, 4, 2, 64, 200, seed=4)
    g = torch.Generator(device="cuda").manual_seed(5)
    prompt = torch.randn(100, 256, generator=g, device="cuda").bfloat16()
    xs = torch.randn(20, 6, 256, generator=g, device="cuda").bfloat16()
    eager, replayed = (ex.Decoder(layer, prompt, 6, 21, page=16) for _ in range(2))
    graph = replayed.capture()
    for x in xs:
        eager.x.copy_(x)
        want = eager.step()
        replayed.x.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(replayed.y, want)


def test_command(ex, capsys):
    ex.main(hidden=512, heads=8, kv_heads=2, d=64, B=4, prompt_len=256, steps=4)
    assert "us a step" in capsys.readouterr().out
