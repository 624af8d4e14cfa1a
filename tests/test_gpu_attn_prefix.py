"""Shared-prefix attention over a paged cache (oq_attn_prefix) against a
64-bit softmax.

Bound on one output: with S_j = |scale| sum_e |q_e k_je| a score is within
(d + 4) 2^-24 S_j of the exact one (float32 sums of exact products, the
scale), so every softmax weight within twice the largest such error, plus
2^-8 for its rounding to bfloat16 and 2^-18 for the exponential, the running
sums and the join; the result is rounded once more to bfloat16.  With A =
sum_j p_j |v_j|:  |o - exact| <= 2^-8 |exact| + A (1.01 2^-8 + 2 (d + 4)
2^-24 max S + 2^-18).  lse is within (d + 4) 2^-24 max S + 2^-20 (1 + |lse|)."""
import math

import pytest
import torch

import rotated_bit_quantized_amd as oq

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


class Case:
    def __init__(self, B, n_q, Hk, G, D, page, prefix, lens, seed=0, width=None, q_scale=1.0, spare=3):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.B, self.n_q, self.Hk, self.G, self.D, self.page, self.prefix = B, n_q, Hk, G, D, page, prefix
        self.P, self.S = -(-prefix // page), -(-max(list(lens) + [0]) // page) if width is None else width
        self.pages = self.P + B * self.S + spare
        self.k = torch.randn(self.pages, Hk, page, D, generator=g, device=DEV).to(BF)
        self.v = torch.randn(self.pages, Hk, page, D, generator=g, device=DEV).to(BF)
        order = torch.randperm(self.pages, generator=g, device=DEV).int()
        self.prefix_table = order[: self.P].contiguous()
        self.tables = order[self.P : self.P + B * self.S].view(B, self.S).contiguous()
        self.lens = torch.tensor(list(lens), dtype=torch.int32, device=DEV)
        self.q = (torch.randn(B * n_q, Hk * G, D, generator=g, device=DEV) * q_scale).to(BF)
        self.scale = 1 / math.sqrt(D)

    def run(self, **kw):
        kv = oq.PagedKV(self.k, self.v)
        return oq.oq_attn_prefix(self.q, self.n_q, kv, self.prefix_table, self.prefix, self.tables if self.S else None,
                                 self.lens if self.S else None, self.scale, want_lse=True, **kw)

    def places(self, b, i):
        """(page, offset) of the keys that query token i of sequence b sees."""
        t = self.prefix_table.tolist()
        seen = [(t[j // self.page], j % self.page) for j in range(self.prefix)]
        t = self.tables[b].tolist()
        n = min(int(self.lens[b]) - self.n_q + 1 + i, self.S * self.page)
        seen += [(t[j // self.page], j % self.page) for j in range(max(0, n))]
        return [(p, o) for p, o in seen if 0 <= p < self.pages]

    def check(self, o, lse):
        for b in range(self.B):
            for i in range(self.n_q):
                at = self.places(b, i)
                t = b * self.n_q + i
                if not at:
                    assert (o[t] == 0).all() and (lse[t] == -math.inf).all()
                    continue
                idx = torch.tensor(at, device=DEV)
                k, v = (c[idx[:, 0], :, idx[:, 1]].double().transpose(0, 1) for c in (self.k, self.v))  # [Hk][n][D]
                q = self.q[t].double().view(self.Hk, self.G, self.D)
                s = torch.matmul(q, k.transpose(1, 2).contiguous()) * self.scale
                mag = (torch.matmul(q.abs(), k.abs().transpose(1, 2).contiguous()) * abs(self.scale)).amax(-1)
                z = torch.logsumexp(s, -1)
                p = torch.exp(s - z[..., None])
                y, A = torch.matmul(p, v), torch.matmul(p, v.abs())
                ds = (self.D + 4) * 2.0 ** -24 * mag
                tol = 2.0 ** -8 * y.abs() + A * (1.01 * 2.0 ** -8 + 2 * ds[..., None] + 2.0 ** -18)
                got = o[t].double().view(self.Hk, self.G, self.D)
                off = (got - y).abs()
                assert torch.isfinite(got).all(), (b, i)
                assert (off <= tol).all(), f"sequence {b}, token {i}: {float((off / tol).max()):.2f} of the bound"
                got = lse[t].double().view(self.Hk, self.G)
                assert ((got - z).abs() <= ds + 2.0 ** -20 * (1 + z.abs())).all(), (b, i, float((got - z).abs().max()))


CASES = [
    # one sequence, one token, one key
    dict(B=1, n_q=1, Hk=1, G=1, D=64, page=8, prefix=1, lens=[0]),
    dict(B=1, n_q=1, Hk=1, G=1, D=128, page=16, prefix=0, lens=[1]),
    dict(B=1, n_q=1, Hk=2, G=3, D=128, page=16, prefix=17, lens=[5]),
    # rows with a prefix alone, a suffix alone, nothing at all
    dict(B=3, n_q=1, Hk=2, G=4, D=128, page=16, prefix=100, lens=[0, 33, 7]),
    dict(B=4, n_q=1, Hk=2, G=4, D=64, page=32, prefix=0, lens=[0, 1, 31, 95]),
    dict(B=5, n_q=1, Hk=1, G=8, D=128, page=64, prefix=63, lens=[0, 0, 0, 0, 0]),
    # lengths around the tiles and pages
    dict(B=6, n_q=1, Hk=1, G=4, D=128, page=16, prefix=127, lens=[15, 16, 17, 31, 32, 33]),
    dict(B=6, n_q=1, Hk=1, G=4, D=128, page=64, prefix=128, lens=[63, 64, 65, 127, 128, 129]),
    dict(B=6, n_q=1, Hk=2, G=2, D=64, page=8, prefix=129, lens=[7, 8, 9, 255, 256, 257]),
    dict(B=2, n_q=1, Hk=1, G=1, D=64, page=1024, prefix=1025, lens=[1500, 3]),
    # several query tokens: causal at the end, some before the suffix begins
    dict(B=3, n_q=2, Hk=2, G=4, D=128, page=16, prefix=50, lens=[2, 40, 1]),
    dict(B=4, n_q=5, Hk=1, G=3, D=64, page=32, prefix=0, lens=[5, 77, 3, 0]),
    dict(B=2, n_q=37, Hk=2, G=1, D=128, page=16, prefix=65, lens=[37, 200]),
    dict(B=2, n_q=100, Hk=1, G=5, D=64, page=64, prefix=333, lens=[100, 150]),
    # head layouts: many query heads a key head, none shared
    dict(B=7, n_q=1, Hk=1, G=32, D=128, page=16, prefix=300, lens=[20, 1, 9, 64, 130, 11, 5]),
    dict(B=9, n_q=1, Hk=16, G=1, D=64, page=16, prefix=200, lens=[3] * 9),
    dict(B=3, n_q=1, Hk=3, G=5, D=128, page=128, prefix=511, lens=[100, 200, 128]),
    # tiles of rows full and ragged, splits of the prefix
    dict(B=64, n_q=1, Hk=2, G=4, D=128, page=64, prefix=2000, lens=[1 + 3 * b for b in range(64)]),
    dict(B=65, n_q=1, Hk=1, G=2, D=64, page=32, prefix=4097, lens=[b % 7 for b in range(65)]),
    dict(B=33, n_q=4, Hk=2, G=5, D=64, page=32, prefix=3000, lens=[4 + b for b in range(33)]),
    dict(B=130, n_q=1, Hk=2, G=8, D=128, page=16, prefix=700, lens=[5 + b % 40 for b in range(130)]),
    dict(B=2, n_q=1, Hk=2, G=4, D=128, page=64, prefix=20000, lens=[4000, 17]),
    dict(B=1, n_q=1, Hk=8, G=4, D=64, page=16, prefix=9001, lens=[9001]),
    dict(B=20, n_q=1, Hk=1, G=1, D=128, page=16, prefix=0, lens=[50 * b for b in range(20)]),
]


@pytest.mark.parametrize("n", range(len(CASES)))
def test_against_float64(n):
    c = Case(seed=n, **CASES[n])
    c.check(*c.run())


@pytest.mark.parametrize("D,B", [(64, 3), (128, 40)])
@pytest.mark.parametrize("q_scale", [0.0, 8.0, 60.0])
def test_flat_and_peaked_scores(D, B, q_scale):
    """All scores equal; scores far apart, so that nearly one key takes all."""
    c = Case(B, 1, 2, 4, D, 32, 1500, [40] * B, seed=1, q_scale=q_scale)
    c.check(*c.run())


@pytest.mark.parametrize("order", ["rising", "falling"])
@pytest.mark.parametrize("B", [2, 40])
def test_running_maximum(order, B):
    """Scores that rise (fall) along the prefix by some 200 in all."""
    c = Case(B, 1, 1, 4, 128, 16, 2048, [64] * B, seed=2)
    c.q[:] = 1.0
    ramp = torch.linspace(-1, 1, 2048, device=DEV) * (1 if order == "rising" else -1) * 8.8
    for j in range(2048):
        c.k[int(c.prefix_table[j // 16]), :, j % 16] = ramp[j].to(BF)
    c.check(*c.run())


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_scales(scale):
    c = Case(5, 1, 2, 4, 128, 16, 300, [10, 0, 33, 5, 100], seed=3)
    c.scale = scale
    c.check(*c.run())


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -3e38])
@pytest.mark.parametrize("B,n_q,D", [(3, 1, 128), (3, 4, 64), (50, 1, 64)])
def test_unseen_places_may_hold_anything(fill, B, n_q, D):
    """Places past each length, unused pages and the rest of the prefix's last page."""
    lens = [(7 * b) % 60 + n_q - 1 for b in range(B)]
    c = Case(B, n_q, 2, 4, D, 16, 211, lens, seed=4, width=6)
    want = c.run()
    seen = torch.zeros(c.pages, c.page, dtype=torch.bool, device=DEV)
    for b in range(B):
        for p, o in c.places(b, n_q - 1):
            seen[p, o] = True
    mask = ~seen[:, None, :, None]
    c.k.masked_fill_(mask, fill)
    c.v.masked_fill_(mask, fill)
    o, lse = c.run()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    c.check(o, lse)


def test_pages_outside_the_cache_are_left_out():
    c = Case(4, 1, 2, 4, 128, 16, 200, [70, 33, 5, 0], seed=5)
    c.prefix_table[3], c.prefix_table[12] = -1, c.pages
    c.tables[0, 1], c.tables[2, 0] = 2 ** 31 - 1, -(2 ** 31)
    c.check(*c.run())
    c.prefix_table[:] = -5  # nothing of the prefix, and one sequence without any key
    c.check(*c.run())


def test_lengths_past_the_table_read_the_table_only():
    c = Case(3, 1, 1, 4, 64, 16, 40, [10, 20, 30], seed=6, width=2)
    c.lens = torch.tensor([1000, 2 ** 31 - 1, -7], dtype=torch.int32, device=DEV)
    c.check(*c.run())


def test_scores_of_minus_infinity():
    """A seen key whose score is -inf has weight zero; a row of such keys alone counts as empty."""
    c = Case(2, 1, 1, 2, 64, 16, 20, [3, 0], seed=7)
    c.q.abs_().add_(0.1)
    for j in range(20):
        c.k[int(c.prefix_table[j // 16]), :, j % 16, 0] = float("-inf")
    o, lse = c.run()
    assert (o[1] == 0).all() and (lse[1] == -math.inf).all()
    c.prefix, c.B = 0, 1  # the first sequence: its suffix alone
    c.check(o[:1], lse[:1])


@pytest.mark.parametrize("B,n_q", [(3, 1), (40, 2)])
def test_strides_and_guard(B, n_q):
    """Queries inside wider rows, head-major outputs in a larger buffer, no lse."""
    c = Case(B, n_q, 2, 4, 128, 16, 500, [9 + n_q] * B, seed=8)
    want, _ = c.run()
    T, H, D = c.q.shape
    wide = torch.randn(T, (H + 3) * D, device=DEV).to(BF)
    wide[:, D : D + H * D] = c.q.flatten(1)
    out = torch.full((H + 1, T, D + 8), 3.0, dtype=BF, device=DEV)
    o = out[:H, :, :D].transpose(0, 1)
    kv = oq.PagedKV(c.k, c.v)
    got, lse = oq.oq_attn_prefix(wide[:, D : D + H * D].unflatten(1, (H, D)), n_q, kv, c.prefix_table, c.prefix, c.tables,
                                 c.lens, c.scale, o=o)
    assert lse is None and torch.equal(o, want)
    out[:H, :, :D] = 3.0
    assert (out == 3.0).all()


def test_interleaved_cache_and_deterministic():
    c = Case(30, 1, 2, 4, 128, 16, 3000, [50] * 30, seed=9)
    want = c.run()
    both = torch.stack((c.k, c.v), 1)
    c.k, c.v = both[:, 0], both[:, 1]
    for _ in range(3):
        o, lse = c.run()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_cache_past_4_gib():
    """Pages more than 2^32 bytes (and 2^31 elements) from the base."""
    c = Case(3, 1, 1, 4, 64, 16, 40, [5, 20, 16], seed=10)
    want = c.run()
    # pages of the same contents, page p at place p * stride
    n, stride = c.pages, 1 << 29
    k = torch.as_strided(torch.empty((n - 1) * stride + 16 * 64, dtype=BF, device=DEV), (n, 1, 16, 64), (stride, 1024, 64, 1))
    v = torch.as_strided(torch.empty((n - 1) * stride + 16 * 64, dtype=BF, device=DEV), (n, 1, 16, 64), (stride, 1024, 64, 1))
    for p in range(n):
        k[p], v[p] = c.k[p], c.v[p]
    assert (n - 1) * stride > 1 << 32
    o, lse = oq.oq_attn_prefix(c.q, 1, oq.PagedKV(k, v), c.prefix_table, c.prefix, c.tables, c.lens, c.scale, want_lse=True)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_empty_batch():
    c = Case(2, 1, 1, 4, 64, 16, 40, [5, 20], seed=11)
    o, _ = oq.oq_attn_prefix(c.q[:0], 1, oq.PagedKV(c.k, c.v), c.prefix_table, c.prefix, c.tables[:0], c.lens[:0], c.scale)
    assert o.shape == (0, 4, 64)


@pytest.mark.parametrize("B,prefix", [(2, 100), (40, 3000)])
def test_streams_and_graph(B, prefix):
    c = Case(B, 1, 2, 4, 128, 16, prefix, [50] * B, seed=12)
    want = c.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o, lse = c.run()
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(o, want[0])
    kv = oq.PagedKV(c.k, c.v)
    ws = torch.empty(oq.oq_attn_prefix_ws_bytes(B, 1, 8, kv, prefix, c.S), dtype=torch.uint8, device=DEV)
    ws.fill_(255)  # scratch needs no particular contents
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        oq.oq_attn_prefix(c.q, 1, kv, c.prefix_table, prefix, c.tables, c.lens, c.scale, o=o, lse=lse, ws=ws)
    for i in range(3):
        c.q.mul_(-1.25)
        c.lens.sub_(9)
        g.replay()
        torch.cuda.synchronize()
        want = c.run()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    c.check(o, lse)


MORE = [
    # so many small pages that a split's page numbers come in several rounds
    dict(B=1, n_q=1, Hk=1, G=4, D=64, page=8, prefix=70001, lens=[13]),
    dict(B=40, n_q=1, Hk=1, G=4, D=64, page=8, prefix=30000, lens=[b % 9 for b in range(40)]),
    dict(B=2, n_q=1, Hk=1, G=2, D=128, page=8, prefix=5, lens=[20000, 9001]),
    # prefix rows in several narrow tiles, the last one ragged
    dict(B=9, n_q=1, Hk=2, G=4, D=128, page=16, prefix=900, lens=[b for b in range(9)]),
    dict(B=31, n_q=1, Hk=2, G=4, D=64, page=32, prefix=1111, lens=[3 * b for b in range(31)]),
    dict(B=32, n_q=1, Hk=1, G=4, D=128, page=64, prefix=640, lens=[b for b in range(32)]),
    # just past them: one wide tile, two wide tiles
    dict(B=43, n_q=1, Hk=1, G=3, D=64, page=16, prefix=1500, lens=[b for b in range(43)]),
    dict(B=129, n_q=1, Hk=1, G=2, D=128, page=16, prefix=257, lens=[b % 50 for b in range(129)]),
    dict(B=57, n_q=3, Hk=2, G=3, D=128, page=32, prefix=65, lens=[3 + b for b in range(57)]),
    # a sequence's own rows fill a wide tile, beside a prefix and alone
    dict(B=2, n_q=130, Hk=2, G=2, D=64, page=16, prefix=777, lens=[400, 131]),
    dict(B=2, n_q=131, Hk=1, G=2, D=128, page=64, prefix=0, lens=[700, 60]),
    dict(B=1, n_q=300, Hk=1, G=4, D=128, page=128, prefix=333, lens=[300]),
]


@pytest.mark.parametrize("n", range(len(MORE)))
def test_tiles_and_splits_against_float64(n):
    c = Case(seed=100 + n, **MORE[n])
    c.check(*c.run())


def test_sequences_are_independent():
    """What a sequence returns does not depend on the contents of the others."""
    c = Case(40, 1, 2, 4, 128, 16, 1000, [30 + b for b in range(40)], seed=13)
    o, lse = c.run()
    c.q[1:] *= -3
    for b in range(1, 40):
        c.v[c.tables[b].long()] += 1
    p, lse2 = c.run()
    assert torch.equal(o[0], p[0]) and torch.equal(lse[0], lse2[0])


@pytest.mark.parametrize("n_q", [1, 3])
def test_other_rows_do_not_move_a_rows_maximum(n_q):
    """Rows of one tile whose scores rise at different places of the prefix: each keeps its bits."""
    c = Case(6, n_q, 1, 4, 64, 16, 2500, [20 + b for b in range(6)], seed=14)
    o, lse = c.run()
    for f in (0.0, 40.0):
        c.q[n_q:] *= f
        p, lse2 = c.run()
        assert torch.equal(o[:n_q], p[:n_q]) and torch.equal(lse[:n_q], lse2[:n_q])
    c.check(p, lse2)


def test_many_parts_and_few():
    """One row over a long prefix (all its parts joined together), and many rows over a short one."""
    c = Case(1, 1, 1, 1, 128, 16, 33000, [0], seed=15)
    c.check(*c.run())
    c = Case(700, 1, 1, 8, 64, 32, 40, [b % 4 for b in range(700)], seed=16)
    c.check(*c.run())


# Enough rows and keys that wavefronts share the keys (more than 64 rows and 16
# tiles of 32 rows x 64 keys a CU): the prefix's part, a suffix's, both.
WIDE = [
    dict(B=64, n_q=1, Hk=8, G=8, D=128, page=16, prefix=2200, lens=[b % 37 for b in range(64)]),
    dict(B=64, n_q=1, Hk=8, G=8, D=64, page=64, prefix=2177, lens=[0] * 64),
    dict(B=43, n_q=3, Hk=8, G=6, D=64, page=32, prefix=1500, lens=[3 + 5 * b for b in range(43)]),
    dict(B=43, n_q=3, Hk=8, G=6, D=128, page=1024, prefix=1409, lens=[b for b in range(43)]),
    dict(B=8, n_q=100, Hk=4, G=4, D=128, page=16, prefix=0, lens=[700, 640, 100, 99, 0, 650, 333, 401]),
    dict(B=8, n_q=100, Hk=4, G=4, D=64, page=64, prefix=700, lens=[660, 641, 100, 37, 0, 650, 512, 449]),
    dict(B=8, n_q=100, Hk=4, G=4, D=128, page=128, prefix=40, lens=[768, 700, 640, 100, 0, 650, 512, 449]),
    # chunks that hold as many page numbers as fit
    dict(B=64, n_q=1, Hk=8, G=32, D=64, page=8, prefix=17003, lens=[b % 11 for b in range(64)]),
    # more single wavefronts' work than shared work: half of it before, half after
    dict(B=100, n_q=1, Hk=16, G=2, D=64, page=32, prefix=2500, lens=[700 - 6 * b for b in range(100)]),
]


@pytest.mark.parametrize("n", range(len(WIDE)))
def test_shared_keys_against_float64(n):
    c = Case(seed=200 + n, **WIDE[n])
    c.check(*c.run())


def _wide(D=128, prefix=2200, seed=20, q_scale=1.0):
    return Case(64, 1, 8, 8, D, 16, prefix, [b % 37 for b in range(64)], seed=seed, width=3, q_scale=q_scale)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_scale", [0.0, 60.0])
def test_shared_keys_flat_and_peaked(D, q_scale):
    c = _wide(D, q_scale=q_scale)
    c.check(*c.run())


@pytest.mark.parametrize("order", ["rising", "falling"])
def test_shared_keys_running_maximum(order):
    c = _wide(128, 2208)
    c.q[:] = 1.0
    c.q[::2] = -0.5  # half of the rows see it the other way round
    ramp = (torch.linspace(-1, 1, 2208, device=DEV) * (1 if order == "rising" else -1) * 8.8).to(BF)
    c.k[c.prefix_table.long()] = ramp.view(-1, 1, 16, 1).expand(-1, 8, 16, 128)
    c.check(*c.run())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -3e38])
def test_shared_keys_unseen_places_may_hold_anything(D, fill):
    c = _wide(D, 2211)
    want = c.run()
    seen = torch.zeros(c.pages, c.page, dtype=torch.bool, device=DEV)
    for b in range(c.B):
        at = torch.tensor(c.places(b, 0), device=DEV)
        seen[at[:, 0], at[:, 1]] = True
    mask = ~seen[:, None, :, None]
    c.k.masked_fill_(mask, fill)
    c.v.masked_fill_(mask, fill)
    o, lse = c.run()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    c.check(o, lse)


def test_shared_keys_pages_outside_the_cache():
    c = _wide()
    c.prefix_table[3], c.prefix_table[77], c.prefix_table[137] = -1, c.pages, 2 ** 31 - 1
    c.k[0], c.v[0] = float("nan"), float("nan")  # page 0 is in no table then
    for t in (c.prefix_table, c.tables):
        t[t == 0] = -(2 ** 31)
    c.check(*c.run())


def test_shared_keys_strides_streams_and_graph():
    c = _wide(64)
    want, wlse = c.run()
    T, H, D = c.q.shape
    wide = torch.randn(T, (H + 3) * D, device=DEV).to(BF)
    wide[:, D : D + H * D] = c.q.flatten(1)
    q = wide[:, D : D + H * D].unflatten(1, (H, D))
    out = torch.full((H + 1, T, D + 8), 3.0, dtype=BF, device=DEV)
    o = out[:H, :, :D].transpose(0, 1)
    kv = oq.PagedKV(c.k, c.v)
    ws = torch.full((oq.oq_attn_prefix_ws_bytes(c.B, 1, H, kv, c.prefix, c.S),), 255, dtype=torch.uint8, device=DEV)
    lse = torch.empty(T, H, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        oq.oq_attn_prefix(q, 1, kv, c.prefix_table, c.prefix, c.tables, c.lens, c.scale, o=o, lse=lse, ws=ws)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(o, want) and torch.equal(lse, wlse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        oq.oq_attn_prefix(q, 1, kv, c.prefix_table, c.prefix, c.tables, c.lens, c.scale, o=o, lse=lse, ws=ws)
    for _ in range(3):
        wide.mul_(-1.25)
        c.q.mul_(-1.25)
        c.lens.sub_(5)
        g.replay()
        torch.cuda.synchronize()
        want, wlse = c.run()
        assert torch.equal(o, want) and torch.equal(lse, wlse)
    c.check(o.contiguous(), lse)
    o.fill_(3.0)
    assert (out == 3.0).all()


@pytest.mark.parametrize("B", [3, 64])
def test_nan_in_a_query_shows_in_its_row(B):
    c = Case(B, 1, 8, 8, 64, 16, 2200 if B == 64 else 100, [5 + b for b in range(B)], seed=30)
    want = c.run()
    c.q[1, 3, 7] = float("nan")
    o, lse = c.run()
    assert torch.isnan(o[1, 3]).all() and torch.isnan(lse[1, 3])
    keep = torch.ones(B, 64, dtype=torch.bool, device=DEV)
    keep[1, 3] = False
    assert torch.equal(o[keep], want[0][keep]) and torch.equal(lse[keep], want[1][keep])


def test_nan_in_a_seen_key_shows_in_the_rows_that_see_it():
    c = Case(3, 1, 2, 4, 128, 16, 100, [5, 20, 9], seed=31)
    want = c.run()
    c.k[int(c.tables[1, 0]), 1, 3] = float("nan")
    o, lse = c.run()
    assert torch.isnan(o[1, 4:]).all() and torch.isnan(lse[1, 4:]).all()
    keep = torch.ones(3, 8, dtype=torch.bool, device=DEV)
    keep[1, 4:] = False
    assert torch.equal(o[keep], want[0][keep]) and torch.equal(lse[keep], want[1][keep])


# One part of the keys alone, which writes the output itself: own keys or a
# prefix, single wavefronts and shared keys, rows without keys among them.
DIRECT = [
    dict(B=30, n_q=1, Hk=4, G=4, D=128, page=16, prefix=0, lens=[2 * b % 61 for b in range(30)]),
    dict(B=17, n_q=3, Hk=2, G=5, D=64, page=32, prefix=0, lens=[3 * b for b in range(17)]),
    dict(B=3, n_q=1, Hk=2, G=4, D=64, page=64, prefix=40, lens=[0, 0, 0]),
    dict(B=5, n_q=2, Hk=1, G=40, D=128, page=16, prefix=0, lens=[0, 1, 2, 64, 33]),
    dict(B=8, n_q=100, Hk=8, G=8, D=128, page=16, prefix=0, lens=[700, 640, 0, 50, 100, 650, 333, 401]),
    dict(B=8, n_q=100, Hk=8, G=8, D=64, page=64, prefix=0, lens=[0, 641, 700, 37, 0, 650, 512, 449]),
]


@pytest.mark.parametrize("n", range(len(DIRECT)))
def test_one_part_against_float64(n):
    c = Case(seed=300 + n, **DIRECT[n])
    assert oq.oq_attn_prefix_ws_bytes(c.B, c.n_q, c.Hk * c.G, oq.PagedKV(c.k, c.v), c.prefix, c.S) == 0
    c.check(*c.run())


@pytest.mark.parametrize("n", [1, 5])
def test_one_part_strides_and_guard(n):
    c = Case(seed=310 + n, **DIRECT[n])
    want, wlse = c.run()
    T, H, D = c.q.shape
    out = torch.full((H + 1, T + 1, D + 8), 3.0, dtype=BF, device=DEV)
    o = out[:H, :T, :D].transpose(0, 1)
    lse = torch.full((T + 1, H), 5.0, device=DEV)
    oq.oq_attn_prefix(c.q, c.n_q, oq.PagedKV(c.k, c.v), c.prefix_table, 0, c.tables, c.lens, c.scale, o=o, lse=lse[:T])
    assert torch.equal(o, want) and torch.equal(lse[:T], wlse) and (lse[T] == 5.0).all()
    out[:H, :T, :D] = 3.0
    assert (out == 3.0).all()
    oq.oq_attn_prefix(c.q, c.n_q, oq.PagedKV(c.k, c.v), c.prefix_table, 0, c.tables, c.lens, c.scale, o=o)
    assert torch.equal(o, want)
    c.q[0, 0, 0] = float("nan")
    c.lens[0] = c.n_q
    o2, lse2 = c.run()
    assert torch.isnan(o2[0, 0]).all() and torch.isnan(lse2[0, 0]) and torch.equal(o2[c.n_q :], want[c.n_q :])
