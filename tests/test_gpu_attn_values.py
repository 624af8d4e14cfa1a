"""oq_attn_prefix where values, keys, queries or the scale are infinite, NaN or
zero: what a row does not see leaves no trace in it, what it sees arrives,
whichever plan of parts the sizes select.  Finite outputs within the bound of
test_gpu_attn_prefix.py."""
import math

import pytest
import torch

import rotated_bit_quantized_amd as oq
from test_gpu_attn_prefix import DIRECT, WIDE, Case

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN, INF = float("nan"), float("inf")


def _exact(c, b, i):
    """Output, lse, the bound's magnitude and score error of token i of sequence b, float64 [Hk][G][D] (lse [Hk][G])."""
    at = torch.tensor(c.places(b, i), device=DEV)
    q = c.q[b * c.n_q + i].double().view(c.Hk, c.G, c.D)
    k, v = (t[at[:, 0], :, at[:, 1]].double().transpose(0, 1) for t in (c.k, c.v))
    s = torch.matmul(q, k.transpose(1, 2).contiguous()) * c.scale
    ds = (c.D + 4) * 2.0 ** -24 * (torch.matmul(q.abs(), k.abs().transpose(1, 2).contiguous()) * abs(c.scale)).amax(-1)
    z = torch.logsumexp(s, -1)
    p = torch.exp(s - z[..., None])
    return torch.matmul(p, v), z, torch.matmul(p, v.abs()), ds


def _check(c, o, lse):
    for b in range(c.B):
        for i in range(c.n_q):
            t = b * c.n_q + i
            if not c.places(b, i):
                assert (o[t] == 0).all() and (lse[t] == -INF).all(), (b, i)
                continue
            y, z, A, ds = _exact(c, b, i)
            got = o[t].double().view(c.Hk, c.G, c.D)
            assert torch.equal(torch.isnan(got), torch.isnan(y)), (b, i)
            big = torch.isinf(y)
            assert torch.equal(got[big], y[big]), (b, i)
            ok = torch.isfinite(y)
            tol = 2.0 ** -8 * y.abs() + A * (1.01 * 2.0 ** -8 + 2 * ds[..., None] + 2.0 ** -18)
            assert ((got - y).abs()[ok] <= tol[ok]).all(), (b, i)
            got = lse[t].double().view(c.Hk, c.G)
            assert ((got - z).abs() <= ds + 2.0 ** -20 * (1 + z.abs())).all(), (b, i)


def _own(c, b, j):
    """(page, offset) of place j of sequence b's own keys."""
    return int(c.tables[b, j // c.page]), j % c.page


@pytest.mark.parametrize("prefix", [0, 211])
@pytest.mark.parametrize("D", [64, 128])
def test_tokens_before_the_first_key_give_zeros(prefix, D):
    """Two of four query tokens stand before their sequence's first key, whose value is not finite."""
    c = Case(3, 4, 2, 4, D, 16, prefix, [2, 1, 3], seed=40)
    for b, bad in ((0, NAN), (1, INF), (2, -INF)):
        p, off = _own(c, b, 0)
        c.v[p, :, off] = bad
    o, lse = c.run()
    if prefix == 0:
        assert oq.oq_attn_prefix_ws_bytes(3, 4, 8, oq.PagedKV(c.k, c.v), 0, c.S) == 0  # one part writes the output
        for t in (0, 1, 4, 5, 6, 8):
            assert (o[t] == 0).all() and (lse[t] == -INF).all(), t


@pytest.mark.parametrize("prefix,lens", [(0, [30, 30]), (30, [0, 0]), (30, [30, 30])])
@pytest.mark.parametrize("bad", [NAN, INF])
def test_keys_without_weight_alone(prefix, lens, bad):
    """Every key of a row scores -inf and its value is not finite: zeros, as for a row without keys."""
    c = Case(2, 1, 1, 2, 64, 16, prefix, lens, seed=41, width=2)
    c.q.abs_().add_(0.1)
    c.k[..., 0] = -INF
    c.v[:] = bad
    o, lse = c.run()
    assert (o == 0).all() and (lse == -INF).all()


@pytest.mark.parametrize("prefix,lens", [(37, [0, 0, 0]), (0, [5, 33, 70]), (37, [5, 33, 70]), (2211, [1, 2, 3])])
@pytest.mark.parametrize("B", [3, 192])
@pytest.mark.parametrize("D", [64, 128])
def test_infinite_value_at_the_last_place(prefix, lens, B, D):
    """The last key of a part ends inside a tile: its infinite value gives infinity, in its place, not NaN."""
    c = Case(B, 1, 8 if B > 3 else 2, 4, D, 16, prefix, (lens * B)[:B], seed=42, width=5)
    for bad, d in ((INF, 3), (-INF, 9)):
        if prefix:
            c.v[int(c.prefix_table[(prefix - 1) // 16]), 0, (prefix - 1) % 16, d] = bad
        for b in range(B):
            if int(c.lens[b]) > 0:
                p, off = _own(c, b, int(c.lens[b]) - 1)
                c.v[p, 1, off, d + 1] = bad
    _check(c, *c.run())


LATER = [
    # single wavefronts: a prefix beside the own keys, own keys alone, more tokens than one tile holds, tokens before the first key
    dict(B=3, n_q=4, Hk=2, G=4, D=64, page=16, prefix=211, lens=[4, 61, 33]),
    dict(B=3, n_q=4, Hk=2, G=4, D=128, page=16, prefix=211, lens=[2, 64, 32]),
    dict(B=4, n_q=5, Hk=1, G=3, D=64, page=32, prefix=0, lens=[5, 77, 3, 0]),
    dict(B=3, n_q=4, Hk=1, G=8, D=128, page=8, prefix=0, lens=[2, 40, 129]),
    dict(B=2, n_q=37, Hk=2, G=1, D=128, page=16, prefix=65, lens=[37, 200]),
    dict(B=1, n_q=60, Hk=1, G=1, D=64, page=64, prefix=0, lens=[500]),
    # wavefronts that share the keys, with a prefix and alone
    WIDE[4], WIDE[5], WIDE[6], DIRECT[4], DIRECT[5],
]


@pytest.mark.parametrize("n", range(len(LATER)))
@pytest.mark.parametrize("every", [False, True])
def test_later_tokens_values_stay_out_of_earlier_rows(n, every):
    """Values that are not finite at the query tokens' own places, a few of them
    or all: a row shows those that it sees, where they stand, and no others."""
    c = Case(seed=400 + n, **LATER[n])
    clean = c.v.clone()
    want = c.run()
    g = torch.Generator().manual_seed(n)
    first_bad = []
    for b in range(c.B):
        L = min(int(c.lens[b]), c.S * c.page)
        own = list(range(max(0, L - c.n_q + 1), L)) or [L - 1] * (L > 0)
        if not every:
            own = sorted({own[int(torch.randint(0, len(own), (1,), generator=g))] for _ in range(2)} | set(own[-1:])) if own else []
        for j in own:
            p, off = _own(c, b, j)
            h = int(torch.randint(0, c.Hk, (1,), generator=g))
            for bad in (NAN, INF, -INF):
                c.v[p, h, off, int(torch.randint(0, c.D, (1,), generator=g))] = bad
        first_bad.append(own[0] if own else L)
    assert not torch.equal(clean.view(torch.int16), c.v.view(torch.int16))
    o, lse = c.run()
    assert torch.equal(lse, want[1])  # no value enters it
    for b in range(c.B):
        for i in range(c.n_q):
            if int(c.lens[b]) - c.n_q + 1 + i <= first_bad[b]:
                t = b * c.n_q + i
                assert torch.equal(o[t], want[0][t]), (b, i)
    _check(c, o, lse)


@pytest.mark.parametrize("n", [0, 3, 6, 9])
@pytest.mark.parametrize("bad", [NAN, INF])
def test_whole_later_tokens_not_finite(n, bad):
    """Keys and values of each sequence's last place: only the last token's rows see them."""
    c = Case(seed=430 + n, **LATER[n])
    want = c.run()
    for b in range(c.B):
        if 0 < int(c.lens[b]) <= c.S * c.page:
            p, off = _own(c, b, int(c.lens[b]) - 1)
            c.k[p, :, off] = bad
            c.v[p, :, off] = bad
    o, lse = c.run()
    for b in range(c.B):
        last = (b + 1) * c.n_q - 1
        assert torch.equal(o[b * c.n_q : last], want[0][b * c.n_q : last]), b
        assert torch.equal(lse[b * c.n_q : last], want[1][b * c.n_q : last]), b
        if int(c.lens[b]) > 0:
            assert torch.isnan(o[last]).any(), b


@pytest.mark.parametrize("B,Hk,G", [(1, 1, 1), (1, 8, 4), (40, 8, 4), (192, 8, 4)])
@pytest.mark.parametrize("D", [64, 128])
def test_nan_in_a_part_of_vanishing_weight_shows(B, Hk, G, D):
    """A NaN value among keys whose whole part weighs less than float32 can tell beside another."""
    c = Case(B, 1, Hk, G, D, 16, 2000, [20] * B, seed=43)
    c.q[:] = 1.0
    c.k[c.tables.long()] = 4.0 * math.sqrt(D) * 16 / D  # scores 64, the prefix's below -192 of them
    c.k[c.prefix_table.long()] = -12.0 * math.sqrt(D) * 16 / D
    c.v[int(c.prefix_table[3]), Hk - 1, 5, 7] = NAN
    o, lse = c.run()
    nan = torch.zeros_like(o, dtype=torch.bool)
    nan[:, (Hk - 1) * G :, 7] = True
    assert torch.equal(torch.isnan(o), nan) and torch.isfinite(lse).all()


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("B,prefix", [(3, 100), (64, 2200)])
def test_scale_zero_keeps_what_is_not_finite(bad, B, prefix):
    """0 times a score that is not finite is NaN, for a query's element as for a key's."""
    c = Case(B, 1, 8, 8, 64, 16, prefix, [5 + b % 30 for b in range(B)], seed=44)
    c.scale = 0.0
    want = c.run()
    c.q[1, 3, 7] = bad
    c.q[2, 9, 60] = -3e38  # finite: no part in it
    p, off = _own(c, 2, 4)
    c.k[p, 7, off, 11] = bad
    o, lse = c.run()
    nan = torch.zeros(B, 64, dtype=torch.bool, device=DEV)
    nan[1, 3] = True
    nan[2, 56:] = True
    assert torch.isnan(o[nan]).all() and torch.isnan(lse[nan]).all()
    assert torch.equal(o[~nan], want[0][~nan]) and torch.equal(lse[~nan], want[1][~nan])
