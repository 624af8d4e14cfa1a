"""The experts' int8 products (oq_gemm_w8a8_experts) against 64-bit results.

Bound on an output before SwiGLU, as for the plain product: 2^-8 |exact| (the
bfloat16 rounding) + 2^-21 (|a s acc| + |mean w1| + |bias|) = 2^-8 |v| + e(v).
SwiGLU: y = silu(g) u with |silu'| <= 1.1, so float32 values off by e(g), e(u)
move y by at most 1.1 e(g) |u| + |silu(g)| e(u) + e(g) e(u).  The exponential's
argument g log2(e) is off by 1.5 |g log2(e)| units of 2^-24, which moves y by 1.5
|g| units at most; the exponential, sum, reciprocal and products add 8; the result's
rounding 2^-8 |y|.  The bound takes 2 e(g) |u| and 2^-7.9 |y|, which leaves 4700
units for |g| (below 10 here, unless a test says otherwise)."""
import pytest
import torch

import rotated_bit_quantized_amd as oq

pytestmark = pytest.mark.gpu
DEV = "cuda"


def lists_of(ids, E):
    """offsets and order of choices [T][k] (-1: none) on the CPU."""
    flat = ids.flatten().tolist()
    order = sorted((i for i, e in enumerate(flat) if e >= 0), key=lambda i: (flat[i], i))
    offsets = [sum(1 for e in flat if 0 <= e < x) for x in range(E + 1)] if len(flat) < 4000 else None
    if offsets is None:
        count = torch.bincount(ids.flatten()[ids.flatten() >= 0].long(), minlength=E)
        offsets = [0] + count.cumsum(0).tolist()
    return torch.tensor(offsets, dtype=torch.int32), torch.tensor(order + [-1] * (len(flat) - len(order)), dtype=torch.int32)


def spread(v, pad, fill=77):
    """v inside a larger tensor: pad further elements a row."""
    big = torch.full((*v.shape[:-1], v.shape[-1] + pad), fill, dtype=v.dtype, device=v.device)
    big[..., : v.shape[-1]] = v
    return big[..., : v.shape[-1]]


class Case:
    def __init__(self, ids, E, K, N, act=False, per=None, center=False, bias=False, seed=0, lo=-127, hi=127, lda=0, ldw=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        T, k = ids.shape
        self.ids, self.E, self.N, self.act, self.n = ids, E, N, act, T * k
        self.per = k if per is None else per
        rows = -(-self.n // self.per)
        r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
        code = lambda *s: torch.randint(lo, hi + 1, s, generator=g, device=DEV, dtype=torch.int32).to(torch.int8)  # noqa: E731
        self.qa, self.w = code(rows, K), code(E, N, K)
        if lda:
            self.qa = spread(self.qa, lda)
        if ldw:
            self.w = spread(self.w, ldw)
        unit = 1 / (60 * K ** 0.5)
        self.a_scale, self.w_scale = (torch.rand(rows, generator=g, device=DEV) + 0.1) * unit, torch.rand(E, N, generator=g, device=DEV) + 0.1
        self.mean, self.w1 = (r(rows), r(E, N)) if center else (None, None)
        self.bias = r(E, N) if bias else None
        self.offsets, self.order = (t.to(DEV) for t in lists_of(ids, E))

    def run(self, y=None, offsets=None, order=None):
        return oq.oq_gemm_w8a8_experts(self.qa, self.a_scale, self.w, self.w_scale, self.offsets if offsets is None else offsets,
                                       self.order if order is None else order, per=self.per,
                                       act=oq.OQ_ACT_SWIGLU if self.act else oq.OQ_ACT_NONE, mean=self.mean, w1=self.w1, bias=self.bias, y=y)

    def exact(self):
        """(values, bounds) [n][out]; rows without expert are NaN."""
        v = torch.full((self.n, self.N), float("nan"), dtype=torch.float64, device=DEV)
        mag = v.clone()
        flat = self.ids.flatten().to(DEV)
        for e in range(self.E):
            i = (flat == e).nonzero()[:, 0]
            if len(i) == 0:
                continue
            row = i // self.per
            p = self.a_scale[row].double()[:, None] * self.w_scale[e].double() * (self.qa[row].double() @ self.w[e].double().t().contiguous())
            m = p.abs()
            if self.mean is not None:
                q = self.mean[row].double()[:, None] * self.w1[e].double()
                p, m = p + q, m + q.abs()
            if self.bias is not None:
                p, m = p + self.bias[e].double(), m + self.bias[e].double().abs()
            v[i], mag[i] = p, m * 2.0 ** -21
        if not self.act:
            return v, 2.0 ** -8 * v.abs() + mag
        (g, u), (eg, eu) = v.chunk(2, 1), mag.chunk(2, 1)
        s = g * torch.sigmoid(g)
        return s * u, 2.0 ** -7.9 * (s * u).abs() + 2 * eg * u.abs() + s.abs() * eu + eg * eu

    def check(self, y=None):
        y = self.run(y)
        want, tol = self.exact()
        listed = (self.ids.flatten() >= 0).to(DEV)
        off = (y.double() - want).abs()[listed]
        bad = ~(off <= tol[listed])
        assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside, first at {bad.nonzero()[0].tolist()}, {float((off / tol[listed].clamp_min(1e-30)).max()):.2f} of the bound"
        return y


def routed(T, E, k, seed=0, skew=0.7):
    """Choices as a router makes them: k different experts a token, some liked more."""
    g = torch.Generator().manual_seed(seed)
    return torch.topk(torch.randn(T, E, generator=g) + skew * torch.randn(E, generator=g), k, dim=1).indices.int()


@pytest.mark.parametrize("T,E,k", [(1, 8, 1), (1, 128, 8), (3, 60, 4), (16, 128, 8), (64, 8, 2), (100, 16, 4), (257, 8, 3), (600, 4, 2), (1000, 64, 6)])
@pytest.mark.parametrize("K,N,act", [(256, 96, True), (256, 97, False), (1040, 64, False), (2048, 130, True)])
def test_batches(T, E, k, K, N, act):
    Case(routed(T, E, k, T + E), E, K, N, act, seed=T).check()


@pytest.mark.parametrize("K", [16, 32, 48, 112, 128, 144, 1008, 1024, 1040, 4096, 4112, 14336])
@pytest.mark.parametrize("T", [9, 120, 700])
def test_widths(K, T):
    Case(routed(T, 6, 2, K), 6, K, 40, seed=K).check()
    Case(routed(T, 6, 2, K), 6, K, 40, act=True, per=1, seed=K + 1).check()


@pytest.mark.parametrize("N", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 257, 384, 513])
@pytest.mark.parametrize("T", [5, 150, 900])
def test_outputs(N, T):
    Case(routed(T, 5, 3, N), 5, 208, N, seed=N).check()
    Case(routed(T, 5, 3, N), 5, 208, 2 * N, act=True, seed=N).check()


@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("T", [7, 130, 1100])
def test_mean_and_bias(T, act):
    for center, bias in ((True, True), (True, False), (False, True)):
        Case(routed(T, 10, 2, 3), 10, 320, 144, act, center=center, bias=bias, seed=T).check()


@pytest.mark.parametrize("T", [1, 40, 300, 1500])
def test_all_entries_at_one_expert(T):
    Case(torch.full((T, 1), 11, dtype=torch.int32), 16, 512, 160, True).check()
    Case(torch.full((T, 1), 0, dtype=torch.int32), 1, 512, 160).check()


def test_expert_counts_at_the_tiles_borders():
    counts = [0, 1, 15, 16, 17, 0, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 0]
    ids = torch.repeat_interleave(torch.arange(len(counts), dtype=torch.int32), torch.tensor(counts))[:, None]
    g = torch.Generator().manual_seed(0)
    Case(ids[torch.randperm(len(ids), generator=g)], len(counts), 256, 200, True, seed=2).check()


@pytest.mark.parametrize("E", [63, 64, 65, 200, 1000, 1024])
def test_many_experts(E):
    Case(routed(150, E, 4, E), E, 64, 36, seed=E).check()


@pytest.mark.parametrize("T", [12, 400])
def test_strides(T):
    c = Case(routed(T, 6, 2), 6, 272, 80, True, lda=48, ldw=16, seed=1)
    big = torch.full((6, 90, 288), 55, dtype=torch.int8, device=DEV)  # experts further apart than their rows
    big[:, :80, :272] = c.w
    c.w = big[:, :80, :272]
    y = torch.full((c.n, 57), -3.0, dtype=torch.bfloat16, device=DEV)
    c.check(y[:, 5:45])
    assert (y[:, :5] == -3).all() and (y[:, 45:] == -3).all()


def test_the_largest_codes():
    Case(routed(60, 4, 2), 4, 131056, 16, lo=-128, hi=-128).check()


@pytest.mark.parametrize("T", [10, 200, 2000])
def test_rows_without_expert_stay(T):
    ids = routed(T, 12, 3, 5)
    g = torch.Generator().manual_seed(6)
    ids[torch.rand(T, 3, generator=g) < 0.3] = -1
    c = Case(ids, 12, 128, 64, True)
    y = torch.full((c.n, 32), 9.0, dtype=torch.bfloat16, device=DEV)
    c.check(y)
    assert (y[(ids.flatten() < 0).to(DEV)] == 9).all()


@pytest.mark.parametrize("T", [10, 500])
def test_list_values_outside_their_range_are_ignored(T):
    ids = routed(T, 4, 2, 5)
    c = Case(ids, 4, 128, 64)
    want = c.run()
    order = c.order.clone()
    hit = [0, c.n // 2, c.n - 1]
    lost = order[hit].tolist()
    order[hit] = torch.tensor([-5, c.n, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    y = torch.full_like(want, 9.0)
    c.run(y, order=order)
    for i in range(c.n):
        assert torch.equal(y[i], torch.full_like(y[i], 9.0) if i in lost else want[i])
    y = torch.full_like(want, 9.0)
    c.run(y, offsets=torch.tensor([-9, 0, 0, 0, 2 ** 31 - 1], dtype=torch.int32, device=DEV))  # all of them at the last expert
    last = Case(torch.full_like(ids, 3), 4, 128, 64)
    last.qa, last.w, last.a_scale, last.w_scale = c.qa, c.w, c.a_scale, c.w_scale
    assert torch.equal(y, last.run())
    y = torch.full_like(want, 9.0)
    c.run(y, offsets=torch.tensor([50, 7, 7, 3, 3], dtype=torch.int32, device=DEV))  # falling: empty
    assert (y == 9).all()


def test_a_rows_bits_do_not_depend_on_the_others():
    """Entry 0 .. 11 alone, among hundreds and among thousands."""
    E, K, N = 8, 528, 96
    ids = routed(2000, E, 2, 8)
    got = []
    for T in (6, 60, 400, 2000):
        c = Case(ids, E, K, N, True, center=True, bias=True, seed=4)
        c.ids, c.n = ids[:T], 2 * T
        c.offsets, c.order = (t.to(DEV) for t in lists_of(ids[:T], E))
        got.append(c.run()[:12])
    for y in got[1:]:
        assert torch.equal(y, got[0])


def test_empty():
    c = Case(routed(4, 4, 2), 4, 64, 32)
    y = oq.oq_gemm_w8a8_experts(c.qa[:0], c.a_scale[:0], c.w, c.w_scale, torch.zeros(5, dtype=torch.int32, device=DEV),
                                torch.empty(0, dtype=torch.int32, device=DEV))
    assert y.shape == (0, 32)


@pytest.mark.parametrize("T", [20, 800])
def test_streams_and_graphs(T):
    c = Case(routed(T, 8, 2), 8, 256, 128, True)
    other = Case(routed(T, 8, 2, 9), 8, 256, 128, True, seed=3)
    want, want_other = c.check(), other.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = c.run()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    y = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(y)
    for i in range(4):
        if i % 2:
            c.qa.copy_(other.qa)
            c.offsets.copy_(other.offsets), c.order.copy_(other.order)
        y.zero_()
        g.replay()
        assert torch.equal(oq.oq_gemm_w8a8_experts(c.qa, c.a_scale, c.w, c.w_scale, c.offsets, c.order, per=2, act=oq.OQ_ACT_SWIGLU), y)
        other.run()
        torch.cuda.synchronize()


def test_agrees_with_the_plain_product():
    """One expert, every row: the bits of oq_gemm_w8a8."""
    for M in (5, 20, 300):
        c = Case(torch.zeros(M, 1, dtype=torch.int32), 1, 640, 160, center=True, bias=True)
        y = oq.oq_gemm_w8a8(c.qa, c.a_scale, c.w[0], c.w_scale[0], c.mean, c.w1[0], c.bias[0])
        assert torch.equal(y, c.run())
