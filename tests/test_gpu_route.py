"""oq_route against float64: choices and lists exactly, weights within their
float32 errors.

Bound on a weight, relative, in units of 2^-24, with D the largest distance of a
chosen logit from the reference it is taken from (the largest logit, or 0): the
difference is off by D / 2, expf by 2 units of its last place (4), so a term by
D + 4; the sum adds at most E / 64 + 6 <= 22 roundings, the division, the factor
and the sigmoid's own addition and division one each.  Numerator and denominator
together: 2 D + 48."""
import math

import pytest
import torch

import rotated_bit_quantized_amd as oq

pytestmark = pytest.mark.gpu
DEV = "cuda"


def reference(logits, k, score="softmax", bias=None, groups=1, top_groups=None, group_best=1, renorm=True, factor=1.0, mask=None):
    """ids, weights (float64), offsets, order on the CPU, token by token."""
    x = logits.detach().cpu().double()
    T, E = x.shape
    s = torch.sigmoid(x) if score == "sigmoid" else torch.exp(x - torch.logsumexp(x, 1, keepdim=True))
    if score == "sigmoid":  # small ones keep their digits
        s = torch.where(x < 0, torch.exp(x) / (1 + torch.exp(x)), s)
    c = x if bias is None else s + bias.cpu().double()
    top_groups = groups if top_groups is None else top_groups
    each = E // groups
    ids = torch.full((T, k), -1, dtype=torch.int32)
    w = torch.zeros(T, k, dtype=torch.float64)

    def ranked(values, allowed, n):  # the n first by falling value, NaN last, ties by index
        keyed = [(1, 0.0, i) if math.isnan(values[i]) else (0, -values[i], i) for i in allowed]
        return [i for _, _, i in sorted(keyed)[:n]]

    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        cs, ss = c[t].tolist(), s[t].tolist()
        allowed = range(E)
        if groups > top_groups:
            by = ss if bias is None and group_best == 2 else cs
            score_of = []
            for g in range(groups):
                mine = sorted((-math.inf if math.isnan(v) else v for v in by[g * each:(g + 1) * each]), reverse=True)
                score_of.append(sum(mine[:group_best]))
            open_ = set(ranked(score_of, range(groups), top_groups))
            allowed = [e for e in range(E) if e // each in open_]
        ids[t] = torch.tensor(ranked(cs, allowed, k), dtype=torch.int32)
        chosen = s[t][ids[t].long()]
        w[t] = factor * (chosen / chosen.sum() if renorm else chosen)
    flat = ids.flatten().tolist()
    order = sorted((i for i in range(T * k) if flat[i] >= 0), key=lambda i: (flat[i], i))
    count = [0] * (E + 1)
    for e in flat:
        if e >= 0:
            count[e + 1] += 1
    offsets = torch.tensor(count).cumsum(0).int()
    return ids, w, offsets, torch.tensor(order + [-1] * (T * k - len(order)), dtype=torch.int32)


def check(logits, k, mask=None, runs=1, **how):
    r = oq.Router(logits.shape[1], k, **how)
    want = reference(logits, k, mask=mask, **how)
    for _ in range(runs):
        ids, w, offsets, order = oq.oq_route(logits, r, mask=mask)
        assert torch.equal(ids.cpu(), want[0])
        assert torch.equal(offsets.cpu(), want[2])
        assert torch.equal(order.cpu(), want[3])
        got = w.cpu().double()
        x = logits.cpu().double()
        ref = x.amax(1, keepdim=True) if how.get("score", "softmax") == "softmax" else torch.zeros(len(x), 1, dtype=torch.float64)
        D = (x - ref).gather(1, ids.cpu().long().clamp_min(0)).abs().clamp_max(1e4)
        bad = ~((got - want[1]).abs() <= (2 * D.amax(1, keepdim=True) + 48) * 2.0 ** -24 * want[1].abs() + 2.0 ** -126)
        bad &= ~(torch.isnan(got) & torch.isnan(want[1]))
        assert not bad.any(), (got[bad][:4], want[1][bad][:4])
    return ids, w, offsets, order


def logits_of(T, E, seed, dtype=torch.float32, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn(T, E, generator=g)).to(dtype).to(DEV)


def bias_of(E, seed):
    return (0.2 * torch.randn(E, generator=torch.Generator().manual_seed(seed + 77))).to(DEV)


@pytest.mark.parametrize("T", [1, 2, 15, 32, 33, 100, 513, 8209])
@pytest.mark.parametrize("E,k", [(8, 2), (128, 8), (60, 4)])
def test_softmax(T, E, k):
    check(logits_of(T, E, T + E), k)


@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (7, 7), (63, 3), (64, 32), (65, 1), (127, 8), (129, 8), (256, 10), (257, 5), (511, 8), (512, 32),
                                 (513, 8), (1000, 6), (1024, 32)])
@pytest.mark.parametrize("T,score,bias,dtype", [(5, "softmax", True, torch.bfloat16), (70, "sigmoid", True, torch.float32),
                                                (70, "sigmoid", False, torch.bfloat16), (40, "softmax", False, torch.float32)])
def test_experts(E, k, T, score, bias, dtype):
    check(logits_of(T, E, E, dtype), k, score=score, bias=bias_of(E, E) if bias else None, renorm=bool(E % 2), factor=2.5)


@pytest.mark.parametrize("groups,each,top_groups,k", [(8, 32, 4, 8), (2, 3, 1, 2), (3, 20, 2, 7), (4, 2, 3, 6), (8, 64, 1, 32), (16, 2, 5, 10),
                                                      (64, 8, 7, 9), (33, 15, 2, 8), (9, 56, 3, 8), (5, 64, 5, 8), (63, 2, 62, 32), (21, 24, 4, 8)])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("score,bias", [("sigmoid", True), ("softmax", False), ("softmax", True)])
def test_groups(groups, each, top_groups, k, best, score, bias):
    E = groups * each
    check(logits_of(50, E, E + best), k, score=score, bias=bias_of(E, E) if bias else None, groups=groups, top_groups=top_groups,
          group_best=best, factor=2.5)


def test_more_tokens_than_one_round_of_chunks():
    check(logits_of(20011, 40, 3, torch.bfloat16), 3)


@pytest.mark.parametrize("how", [dict(), dict(score="sigmoid"), dict(groups=4, top_groups=2, group_best=2),
                                 dict(groups=4, top_groups=2, score="sigmoid", bias=True)])
def test_equal_logits_go_to_the_lowest_index(how):
    how = dict(how)
    g = torch.Generator().manual_seed(0)
    x = torch.randint(-2, 3, (300, 64), generator=g).float()
    x[0], x[1] = 0.0, -0.0
    x[1, ::2] = 0.0  # -0 is 0
    if how.get("bias"):
        how["bias"] = torch.zeros(64, device=DEV)
    check(x.to(DEV), 8, runs=2, **how)
    check(x.bfloat16().to(DEV), 8, **how)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups", [1, 4])
def test_neighbours_that_float32_cannot_tell_apart(score, groups):
    """The bias undoes the scores up to its own rounding: sums differ by 1e-8 or less."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(1, 128, generator=g).expand(40, 128).contiguous()
    s = torch.sigmoid(x[0].double()) if score == "sigmoid" else torch.softmax(x[0].double(), 0)
    bias = (0.5 - s).float()
    c = (s + bias.double()).sort().values
    assert float((c[1:] - c[:-1]).median()) < 2e-8  # the case is what it says
    check(x.to(DEV), 8, score=score, bias=bias.to(DEV), groups=groups, top_groups=max(1, groups // 2), group_best=min(2, groups))


@pytest.mark.parametrize("how", [dict(), dict(renorm=False), dict(score="sigmoid"), dict(score="sigmoid", renorm=False)])
def test_scores_that_vanish(how):
    """Far negative logits: what is chosen among them still has weights."""
    x = torch.linspace(-95, -60, 64).repeat(3, 1)
    x[1] -= 20
    check(x.to(DEV), 6, **how)


def test_values_that_are_not_finite():
    x = logits_of(12, 64, 9)
    x[0, 3] = math.nan
    x[1, :] = -math.inf
    x[2, 5:] = -math.inf  # fewer finite ones than choices
    x[3, :] = math.nan
    x[4, 10] = math.inf
    x[5, :60] = math.nan
    check(x, 8)
    check(x, 8, score="sigmoid")
    check(x, 8, score="sigmoid", bias=bias_of(64, 1), groups=8, top_groups=3, group_best=2)
    for ids in (oq.oq_route(x, oq.Router(64, 8, bias=bias_of(64, 2)))[0], oq.oq_route(x, oq.Router(64, 8, groups=4, top_groups=2))[0]):
        assert int(ids.min()) >= 0 and int(ids.max()) < 64
        assert all(len(set(row.tolist())) == 8 for row in ids)


@pytest.mark.parametrize("T", [20, 700])
@pytest.mark.parametrize("kind", ["some", "none", "all"])
def test_mask(T, kind):
    g = torch.Generator().manual_seed(1)
    mask = {"some": torch.rand(T, generator=g) < 0.6, "none": torch.zeros(T, dtype=torch.bool), "all": torch.ones(T, dtype=torch.bool)}[kind].to(DEV)
    x = logits_of(T, 48, T)
    check(x, 5, mask=mask)
    check(x, 5, mask=mask.to(torch.uint8) * 200)


def test_strided_logits_and_outputs_inside_larger_buffers():
    T, E, k = 77, 60, 4
    wide = logits_of(T, 131, 2)
    x = wide[:, 3:63]  # rows 4-byte aligned only
    want = reference(x, k)
    big = [torch.full((n + 64,), -7, dtype=d, device=DEV) for n, d in ((T * k, torch.int32), (T * k, torch.float32), (E + 1, torch.int32), (T * k, torch.int32))]
    out = [b[32:-32] for b in big]
    oq.oq_route(x, oq.Router(E, k), None, out[0].view(T, k), out[1].view(T, k), out[2], out[3])
    for b in big:
        assert (b[:32] == -7).all() and (b[-32:] == -7).all()
    assert torch.equal(out[0].view(T, k).cpu(), want[0]) and torch.equal(out[3].cpu(), want[3])
    check(logits_of(T, 131, 2, torch.bfloat16)[:, 1:61], k)


def test_empty_and_without_lists():
    r = oq.Router(16, 2)
    ids, w, offsets, order = oq.oq_route(torch.empty(0, 16, device=DEV), r)
    assert ids.shape == (0, 2) and order.numel() == 0 and torch.equal(offsets.cpu(), torch.zeros(17, dtype=torch.int32))
    assert oq.oq_route(torch.empty(0, 16, device=DEV), r, lists=False)[2] is None
    big = oq.Router(1000, 2)  # no single-workgroup form
    assert not oq.oq_route(torch.empty(0, 1000, device=DEV), big)[2].any()
    x = logits_of(40, 16, 0)
    a, b = oq.oq_route(x, r), oq.oq_route(x, r, lists=False)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and b[2] is None and b[3] is None


def test_streams_graphs_and_a_shared_workspace():
    r = oq.Router(128, 8, score="sigmoid", bias=bias_of(128, 4), groups=8, top_groups=4, group_best=2)
    xs = [logits_of(600, 128, s) for s in range(4)]
    want = [oq.oq_route(x, r) for x in xs]
    ws = torch.empty(oq.oq_route_ws_bytes(600, r), dtype=torch.uint8, device=DEV)
    x = torch.empty_like(xs[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = oq.oq_route(xs[1], r, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want[1]))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = oq.oq_route(x, r, ws=ws)
        graphs.append((g, outs))
    for i in range(4):
        x.copy_(xs[i])
        for g, outs in graphs:
            g.replay()
            assert all(torch.equal(a, b) for a, b in zip(outs, want[i]))
        oq.oq_route(xs[3 - i], r, ws=ws)
        torch.cuda.synchronize()
