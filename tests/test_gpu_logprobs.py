"""oq_logprobs against float64: ranks and alternatives exactly, values within
their float32 errors.

In units of 2^-24, with z = scale x - (the row's largest): the factor scale
log2(e) is off by 1.5, so z by 1.5 |z| and its own rounding |z|; a term 2^z by
that and 2; a sum goes over at most 64 terms a thread and 20 further steps, so
s by 90 and sum p |z| = A; the logarithm and the factors back add 3 of what they
give.  A log probability: 4 |z| + 4 log V + 120, absolute.  lse: 4 |lse| more, and 4
of the largest logit.  The entropy also takes sum 2^z z, whose terms are off by
3 |z| + 4 of themselves: 8 B + 250 (1 + A), B = sum p z^2."""
import math

import pytest
import torch

import rotated_bit_quantized_amd as oq

pytestmark = pytest.mark.gpu
DEV, U = "cuda", 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
INF, NAN = math.inf, math.nan


def order_of(x):
    """Places of a row's elements by falling value, equal ones by index, NaN last."""
    x = torch.where(torch.isnan(x), torch.full_like(x, -INF), x.double())
    by_value = torch.sort(x, dim=1, descending=True, stable=True).indices
    return by_value


def ranked(x):
    """As order_of, with NaN behind -inf."""
    x = x.double()
    idx = order_of(x)
    nan_last = torch.sort(torch.isnan(x).gather(1, idx).int(), dim=1, stable=True).indices
    return idx.gather(1, nan_last)


def check(x, tokens=None, top=0, scale=1.0, plain_rows=None):
    """plain_rows: rows whose values are compared (others hold NaN or infinities)."""
    T, V = x.shape
    got = oq.oq_logprobs(x, tokens, top=top, scale=scale)
    logprob, rank, entropy, lse, top_id, top_logprob = got
    idx = ranked(x)
    assert torch.equal(top_id.long(), idx[:, :top])
    place = torch.empty_like(idx).scatter_(1, idx, torch.arange(V, device=DEV).expand(T, V).contiguous())
    rows = torch.ones(T, dtype=torch.bool, device=DEV) if plain_rows is None else plain_rows
    z = x.double() * scale
    m = z.amax(1, keepdim=True)
    total = torch.logsumexp(z, 1, keepdim=True)
    logp = z - total
    p = logp.exp()
    far = torch.where(p > 0, (z - m).abs(), torch.zeros_like(z))
    A, B = (p * far).sum(1), (p * far * far).sum(1)
    H = -torch.where(p > 0, p * logp, torch.zeros_like(p)).sum(1)
    base = 4 * math.log(V) + 120

    def close(got, want, tol, what):
        same = (got.double() == want) | (torch.isnan(got) & torch.isnan(want))
        bad = ~(((got.double() - want).abs() <= tol) | same) & rows.view(-1, *[1] * (got.dim() - 1))
        assert not bad.any(), f"{what}: {int(bad.sum())} outside, got {got[bad][:3].tolist()}, want {want[bad][:3].tolist()}"

    close(top_logprob, logp.gather(1, idx[:, :top]), U * (4 * (z - m).abs().gather(1, idx[:, :top]) + base), "top_logprob")
    close(lse, total[:, 0], U * (base + 4 * total[:, 0].abs() + 4 * m[:, 0].abs()), "lse")
    close(entropy, H, U * (8 * B + 250 * (1 + A)), "entropy")
    if tokens is not None:
        tok = tokens.long()
        inside = (tok >= 0) & (tok < V)
        at = tok.clamp(0, V - 1)
        assert torch.equal(rank.long(), torch.where(inside, place.gather(1, at), torch.full_like(at, -1)))
        want = torch.where(inside, logp.gather(1, at), torch.full_like(logp.gather(1, at), NAN))
        close(logprob, want, U * (4 * (z - m).abs().gather(1, at) + base), "logprob")
    else:
        assert logprob.shape == (T, 0) and rank.shape == (T, 0)
    return got


def logits_of(T, V, seed, dtype=F32, spread=2.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (spread * torch.randn(T, V, generator=g, device=DEV)).to(dtype)


def tokens_of(T, V, n, seed):
    g = torch.Generator(device=DEV).manual_seed(seed + 1000)
    return torch.randint(0, V, (T, n), generator=g, device=DEV, dtype=torch.int32)


@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 31, 64, 65, 500, 2047, 2049, 4095, 4096, 4097, 8200, 16384, 16385, 32768, 32769, 50021, 131072, 262147])
@pytest.mark.parametrize("T,dtype", [(1, F32), (3, BF), (17, F32)])
def test_widths(V, T, dtype):
    check(logits_of(T, V, V, dtype), tokens_of(T, V, 2, V), top=min(V, 7), scale=1.25)


@pytest.mark.parametrize("T,V", [(600, 5000), (600, 20000), (530, 33000), (260, 70000), (2000, 300), (130, 131072), (1700, 20000), (800, 33001)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_many_rows(T, V, dtype):
    """Every number of pieces a thread, one part a row and several."""
    check(logits_of(T, V, T, dtype), tokens_of(T, V, 1, V), top=5)


@pytest.mark.parametrize("top", [0, 1, 2, 20, 32])
@pytest.mark.parametrize("n", [0, 1, 5, 64])
@pytest.mark.parametrize("T,V", [(4, 3001), (4, 40000), (700, 4000)])
def test_counts(top, n, T, V):
    check(logits_of(T, V, top + n, BF if n % 2 else F32), tokens_of(T, V, n, V) if n else None, top=top, scale=0.7)


@pytest.mark.parametrize("offset,ld", [(0, 1003), (1, 1003), (5, 1010), (7, 1001), (3, 1024)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_rows_at_any_element(offset, ld, dtype):
    T, V = 40, 1000
    big = torch.full((T * ld + 64,), 1e4, dtype=dtype, device=DEV)  # large values around every row
    x = big.as_strided((T, V), (ld, 1), offset)
    x.copy_(logits_of(T, V, ld, dtype))
    check(x, tokens_of(T, V, 3, 1), top=9)


@pytest.mark.parametrize("V", [300, 9000, 33000])
@pytest.mark.parametrize("T", [3, 520])
def test_equal_logits(V, T):
    g = torch.Generator(device=DEV).manual_seed(V)
    x = torch.randint(-2, 3, (T, V), generator=g, device=DEV).float()
    x[0] = 1.5
    x[1] = -0.0
    x[1, 1::2] = 0.0
    tok = tokens_of(T, V, 4, 2)
    tok[0] = torch.tensor([0, 1, V - 1, V // 2])
    check(x, tok, top=32)
    check(x.bfloat16(), tok, top=20)
    check(x.bfloat16(), tok, top=8)


@pytest.mark.parametrize("V", [300, 9000, 40000])
@pytest.mark.parametrize("T", [2, 530])
@pytest.mark.parametrize("kept", [1, 3, 32, 200])
def test_masked_vocabulary(V, T, kept):
    """All but a few logits are -inf, or the type's lowest value."""
    g = torch.Generator(device=DEV).manual_seed(kept)
    for dtype in (F32, BF):
        for low in (-INF, torch.finfo(dtype).min):
            x = torch.full((T, V), low, dtype=dtype, device=DEV)
            keep = torch.rand(T, V, generator=g, device=DEV).topk(kept, 1).indices
            x.scatter_(1, keep, logits_of(T, kept, kept, dtype))
            tok = torch.cat((keep[:, :2].int(), torch.zeros(T, 1, dtype=torch.int32, device=DEV), torch.full((T, 1), V - 1, dtype=torch.int32, device=DEV)), 1)
            check(x, tok, top=20)
            check(x, tok, top=5)


@pytest.mark.parametrize("kind", ["rising", "falling", "one lane", "two values", "block"])
@pytest.mark.parametrize("T,V", [(3, 12000), (530, 32768), (530, 16000)])
def test_orders_that_fill_the_list(kind, T, V):
    """The largest values where one lane of every wavefront holds them, in a block, in order."""
    x = logits_of(T, V, 4, F32)
    i = torch.arange(V, device=DEV)
    if kind == "rising":
        x = (i.float() * 1e-3).expand(T, V).contiguous()
    elif kind == "falling":
        x = (i.flip(0).float() * 1e-3).expand(T, V).contiguous()
    elif kind == "two values":
        x = (i % 2).float().expand(T, V).contiguous()
    elif kind == "block":
        x[:, 1000:3500] += 40
    for dtype, ve in ((F32, 4), (BF, 8)):
        y = x.clone()
        if kind == "one lane":
            y[:, (i // ve) % 64 == 3] += 40
        y = y.to(dtype)
        check(y, tokens_of(T, V, 2, 3), top=20)
        check(y, tokens_of(T, V, 2, 3), top=6)  # parts of another size


@pytest.mark.parametrize("V", [200, 5000, 40000])
@pytest.mark.parametrize("T", [12, 540])
def test_values_that_are_not_finite(V, T):
    x = logits_of(T, V, 8)
    x[1] = -INF
    x[2, V // 3] = NAN
    x[3] = NAN
    x[4, V // 2] = INF
    x[5] = -INF
    x[5, :7] = NAN
    x[6, 3:] = NAN
    x[7, 11] = -INF
    plain = torch.ones(T, dtype=torch.bool, device=DEV)
    plain[1:7] = False
    tok = tokens_of(T, V, 5, 1)
    tok[:, 0], tok[:, 1] = V // 3, 3
    tok[7, 2] = 11
    for dtype in (F32, BF):
        check(x.to(dtype), tok, top=8, plain_rows=plain)
        logprob, rank, entropy, lse, top_id, top_logprob = check(x.to(dtype), tok, top=20, plain_rows=plain)
        assert float(lse[1]) == -INF and torch.isnan(lse[2:7]).all()
        assert torch.isnan(logprob[1:7]).all() and torch.isnan(entropy[1:7]).all() and torch.isnan(top_logprob[1:7]).all()
        assert float(logprob[7, 2]) == -INF


def test_parts_that_hold_nothing():
    """-inf over whole parts of a row, far negative and far positive logits."""
    V = 40000
    x = logits_of(6, V, 3)
    x[0, :20000] = -INF
    x[1, 20000:] = -INF
    x[2] -= 3000
    x[2, 100:] = -INF
    x[3] += 3000
    x[4, :39990] = -INF
    x[5, 1:] = -3.4e38
    check(x, tokens_of(6, V, 3, 2), top=6)


def test_tokens_outside_the_vocabulary():
    for T, V in ((9, 777), (9, 30000)):
        tok = tokens_of(T, V, 4, 5)
        tok[:, 1], tok[:, 2] = -1, V
        tok[0, 3], tok[1, 3] = -2 ** 31, 2 ** 31 - 1
        check(logits_of(T, V, 5), tok, top=2)


def test_the_widest_rows():
    """As many parts as there can be, one list a lane and several."""
    for T, V in ((1, 1 << 21), (2, 1200003)):
        check(logits_of(T, V, 1), tokens_of(T, V, 2, 1), top=32)
        check(logits_of(T, V, 2, BF), tokens_of(T, V, 2, 1), top=32)


def test_the_same_token_twice():
    tok = tokens_of(5, 3000, 1, 0).repeat(1, 6).contiguous()
    logprob, rank, *_ = check(logits_of(5, 3000, 0), tok)
    assert (logprob == logprob[:, :1]).all() and (rank == rank[:, :1]).all()


def test_a_nearly_certain_token():
    x = torch.zeros(4, 50000, device=DEV)
    tok = torch.tensor([[5], [600], [7000], [49999]], dtype=torch.int32, device=DEV)
    x.scatter_(1, tok.long(), torch.tensor([[12.0], [20.0], [40.0], [200.0]], device=DEV))
    check(x, tok, top=1)


def test_repeats_are_the_same_bits():
    x = logits_of(64, 60000, 1, BF)
    tok = tokens_of(64, 60000, 2, 1)
    a = oq.oq_logprobs(x, tok, top=20)
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(a, oq.oq_logprobs(x, tok, top=20)))


def test_given_outputs_inside_larger_buffers():
    T, V, n, top = 5, 9000, 3, 4
    x, tok = logits_of(T, V, 2), tokens_of(T, V, n, 2)
    want = oq.oq_logprobs(x, tok, top=top)
    sizes = [(T, n), (T, n), (T,), (T,), (T, top), (T, top)]
    types = [F32, torch.int32, F32, F32, torch.int32, F32]
    big = [torch.full((math.prod(s) + 32,), -9, dtype=d, device=DEV) for s, d in zip(sizes, types)]
    ws = torch.full((oq.oq_logprobs_ws_bytes(T, V, n, top) + 64,), 99, dtype=torch.uint8, device=DEV)
    oq.oq_logprobs(x, tok, top, 1.0, *[b[16:-16].view(s) for b, s in zip(big, sizes)], ws=ws[:-64])
    for b, w in zip(big, want):
        assert (b[:16] == -9).all() and (b[-16:] == -9).all() and torch.equal(b[16:-16], w.flatten())
    assert (ws[-64:] == 99).all()


def test_empty():
    out = oq.oq_logprobs(torch.empty(0, 100, device=DEV), torch.empty(0, 2, dtype=torch.int32, device=DEV), top=3)
    assert [tuple(o.shape) for o in out] == [(0, 2), (0, 2), (0,), (0,), (0, 3), (0, 3)]


@pytest.mark.parametrize("T,V", [(3, 30000), (900, 5000)])
def test_streams_graphs_and_a_shared_workspace(T, V):
    xs = [logits_of(T, V, s, BF) for s in range(4)]
    tok = tokens_of(T, V, 1, 0)
    want = [oq.oq_logprobs(x, tok, top=5) for x in xs]
    ws = torch.empty(max(16, oq.oq_logprobs_ws_bytes(T, V, 1, 5)), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = oq.oq_logprobs(xs[1], tok, top=5, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want[1]))
    x = torch.empty_like(xs[0])
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = oq.oq_logprobs(x, tok, top=5, ws=ws)
        graphs.append((g, outs))
    for i in range(4):
        x.copy_(xs[i])
        for g, outs in graphs:
            g.replay()
            assert all(torch.equal(a, b) for a, b in zip(outs, want[i]))
        oq.oq_logprobs(xs[3 - i], tok, top=5, ws=ws)
        torch.cuda.synchronize()
