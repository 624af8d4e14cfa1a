"""oq_residual_norm against float64, within bounds that follow its float32
errors (units of 2^-24) through the formula.

u: k products and sums, (k + 2) sum |w y| (0 for a plain row).  A norm's sums go
over at most 16 elements a thread and 10 further steps: 26 of the mean of |x| for
the mean, 26 of the variance, half of that for the deviation, 3 for quotient and
root; 32 covers each.  An input error e moves the mean by mean(e) and the
deviation's relative error by mean(|x - m| e) / var.  R and h add 4 of their terms,
and a bfloat16 result 2^-8 of its value (a float32 one 1 unit)."""
import itertools

import pytest
import torch

import rotated_bit_quantized_amd as oq

pytestmark = pytest.mark.gpu
DEV, U = "cuda", 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def norm64(x, e, kind, w, b, eps):
    """The norm of x known within e: values and bounds."""
    if kind is None:
        return x, e
    m = x.mean(1, keepdim=True) if kind == oq.OQ_NORM_LAYER else 0 * x[:, :1]
    em = (e.mean(1, keepdim=True) + 32 * U * x.abs().mean(1, keepdim=True)) if kind == oq.OQ_NORM_LAYER else 0 * x[:, :1]
    c, ec = x - m, e + em + U * (x - m).abs()
    var = (c * c).mean(1, keepdim=True) + eps
    rel = (c.abs() * ec + ec * ec).mean(1, keepdim=True) / var + 32 * U
    w = torch.ones_like(x[0]) if w is None else w.double()
    v = c / var.sqrt() * w
    ev = (ec / var.sqrt()) * w.abs() * (1 + rel) + v.abs() * (rel + 4 * U)
    return (v, ev) if b is None else (v + b.double(), ev + U * (v.abs() + b.double().abs()))


def half(dtype):
    return 2.0 ** -8 if dtype is BF else U


def check(T, d, k=None, post=None, pre=oq.OQ_NORM_RMS, gate=False, scale=False, shift=False, r=BF, y=True, r_dtype=BF, rows=1, row=True,
          vectors=True, bias=False, y_scale=1.0, r_scale=1.0, pad=0, in_place=False, want_r=True, want_h=True, seed=0, eps=1e-6):
    g = torch.Generator(device=DEV).manual_seed(seed + d + T)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731

    def laid(v, dtype):
        big = torch.full((v.shape[0], v.shape[1] + pad), 7.0, dtype=dtype, device=DEV)
        big[:, : v.shape[1]] = v
        return big[:, : v.shape[1]]

    yt = laid(1.5 * rand(T * (k or 1), d) + 0.3, BF) if y else None
    mix = torch.softmax(rand(T, k), 1) * 1.3 if k else None
    rt = laid(3 * rand(T, d) - 0.4, r) if r else None
    if r is None and r_dtype is None:
        r_dtype = BF
    make = lambda kind: None if kind is None else oq.Norm(kind, d, eps, 1 + 0.2 * rand(d) if vectors else None, rand(d) if bias else None)  # noqa: E731
    n_post, n_pre = make(post), make(pre)
    table = laid(0.4 * rand(rows, 3 * d), BF)
    parts = [table[:, i * d:(i + 1) * d] if want else None for i, want in enumerate((gate, scale, shift))]
    at = torch.randint(0, rows, (T,), generator=g, device=DEV, dtype=torch.int32) if row else None
    index = at.long() if row else torch.zeros(T, dtype=torch.long, device=DEV) if rows == 1 else torch.arange(T, device=DEV)

    u, eu = torch.zeros(T, d, dtype=torch.float64, device=DEV), torch.zeros(T, d, dtype=torch.float64, device=DEV)
    if y:
        u = yt.double()
        if k:
            terms = u.reshape(T, k, d) * mix.double()[:, :, None]
            u, eu = terms.sum(1), (k + 2) * U * terms.abs().sum(1)
    take = lambda n, x, e, kind: norm64(x, e, kind, n.w if n else None, n.b if n else None, eps)  # noqa: E731
    v, ev = take(n_post, u, eu, post) if y else (u, eu)
    ga = parts[0].double()[index] * y_scale if gate else torch.full((1, 1), float(y_scale), dtype=torch.float64, device=DEV)
    R, eR = ga * v, ga.abs() * ev + 4 * U * (ga * v).abs()
    if r:
        R, eR = R + r_scale * rt.double(), eR + 4 * U * (r_scale * rt.double()).abs()
    h, eh = take(n_pre, R, eR, pre)
    s = parts[1].double()[index] if scale else torch.zeros(1, 1, dtype=torch.float64, device=DEV)
    b = parts[2].double()[index] if shift else torch.zeros(1, 1, dtype=torch.float64, device=DEV)
    eh = (1 + s).abs() * eh + 4 * U * (h.abs() * (1 + s).abs() + b.abs())
    h = h * (1 + s) + b
    eR, eh = eR + half(r or r_dtype) * R.abs(), eh + 2.0 ** -8 * h.abs()

    out_type = r or r_dtype
    r_out = rt if in_place else laid(torch.zeros(T, d, device=DEV), out_type) if pad else None
    h_out = laid(torch.zeros(T, d, device=DEV), BF) if pad else None
    got_r, got_h = oq.oq_residual_norm(yt, rt, mix, n_post, n_pre, *parts, row=at, y_scale=y_scale, r_scale=r_scale, r_out=r_out, h=h_out,
                                       want_r=want_r, want_h=want_h, r_dtype=r_dtype)
    for name, got, want, tol, on in (("r", got_r, R, eR, want_r), ("h", got_h, h, eh, want_h)):
        if not on:
            assert got is None
            continue
        off = (got.double() - want).abs()
        bad = ~(off <= 1.02 * tol)  # second-order terms
        assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} outside, first {bad.nonzero()[0].tolist()}, worst {float((off / tol.clamp_min(1e-30)).max()):.2f}"
        if pad:
            assert (got.as_strided((T, pad), got.stride(), got.storage_offset() + d) == 7).all(), "written past the rows"
    return got_r, got_h


WIDTHS = [8, 16, 64, 72, 128, 136, 256, 264, 512, 520, 1000, 1024, 1032, 1920, 2048, 2056, 4096, 4104, 8192, 8200, 16384]


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("T", [1, 2, 33])
def test_widths(d, T):
    check(T, d)
    check(T, d, k=3, post=oq.OQ_NORM_LAYER, pre=oq.OQ_NORM_LAYER, gate=True, scale=True, shift=True, rows=4, r=F32, bias=True)


@pytest.mark.parametrize("post,pre", itertools.product([None, oq.OQ_NORM_RMS, oq.OQ_NORM_LAYER], repeat=2))
@pytest.mark.parametrize("d", [96, 1920, 5000])
@pytest.mark.parametrize("r", [BF, F32])
def test_norms(post, pre, d, r):
    check(37, d, post=post, pre=pre, r=r)
    check(37, d, k=8, post=post, pre=pre, r=r, vectors=False, y_scale=0.22, r_scale=0.7)
    check(37, d, post=post, pre=pre, r=r, bias=True, gate=True, rows=3)


@pytest.mark.parametrize("gate,scale,shift", itertools.product([False, True], repeat=3))
@pytest.mark.parametrize("T,rows,row", [(50, 1, False), (50, 7, True), (50, 50, False), (5, 9, False)])
def test_modulation(gate, scale, shift, T, rows, row):
    check(T, 640, gate=gate, scale=scale, shift=shift, rows=rows, row=row, pre=oq.OQ_NORM_LAYER, vectors=False)


@pytest.mark.parametrize("k", [1, 2, 4, 5, 8, 13, 64])
@pytest.mark.parametrize("d", [40, 2048, 4200])
def test_weighted_sums(k, d):
    check(9, d, k=k)


@pytest.mark.parametrize("T", [300, 4100])
def test_more_rows(T):
    check(T, 256, k=2)
    check(T, 1920, gate=True, rows=2)


@pytest.mark.parametrize("d", [80, 1920, 4096])
def test_parts_of_the_formula(d):
    check(20, d, y=False)
    check(20, d, y=False, r=F32, r_scale=0.5, scale=True, shift=True, rows=20)
    check(20, d, r=None, r_dtype=F32, post=oq.OQ_NORM_RMS)
    check(20, d, r=None, k=4, pre=None)
    check(20, d, want_r=False)
    check(20, d, want_h=False, k=2, gate=True)


@pytest.mark.parametrize("d", [48, 1032, 6000])
@pytest.mark.parametrize("r", [BF, F32])
def test_strides_and_in_place(d, r):
    check(30, d, pad=24, r=r, gate=True, scale=True, shift=True, rows=5)
    check(30, d, pad=24, r=r, in_place=True, k=2)
    check(30, d, r=r, in_place=True)


def test_rows_without_weight_are_not_read():
    T, k, d = 21, 4, 328
    g = torch.Generator(device=DEV).manual_seed(0)
    y = torch.randn(T * k, d, generator=g, device=DEV).bfloat16()
    w = torch.rand(T, k, generator=g, device=DEV)
    w[torch.rand(T, k, generator=g, device=DEV) < 0.4] = 0.0
    w[3] = 0.0  # a token without any expert
    w[4, 0] = -0.0
    clean = torch.where((w == 0).view(-1, 1), torch.zeros_like(y), y)
    dirty = torch.where((w == 0).view(-1, 1), torch.full_like(y, float("nan")), y)
    r = torch.randn(T, d, generator=g, device=DEV).bfloat16()
    n = oq.Norm(oq.OQ_NORM_RMS, d)
    a, b = oq.oq_residual_norm(clean, r, w, pre=n), oq.oq_residual_norm(dirty, r, w, pre=n)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.equal(b[0][3], r[3])


def test_modulation_rows_out_of_range_give_nan():
    T, d = 12, 72
    y, r = torch.ones(T, d, dtype=BF, device=DEV), torch.ones(T, d, dtype=BF, device=DEV)
    table = torch.ones(3, d, dtype=BF, device=DEV)
    row = torch.tensor([0, 1, 2, 3, -1, 0, 2 ** 31 - 1, -2 ** 31, 1, 1, 1, 1], dtype=torch.int32, device=DEV)
    bad = (row < 0) | (row >= 3)
    for args in (dict(gate=table), dict(scale=table), dict(shift=table)):
        R, h = oq.oq_residual_norm(y, r, row=row, **args)
        assert torch.equal(torch.isnan(R).all(1), bad) and torch.equal(torch.isnan(h).all(1), bad)
        assert not torch.isnan(R[~bad]).any() and not torch.isnan(h[~bad]).any()


def test_values_that_are_not_finite_stay_in_their_row():
    T, d = 6, 2048
    y, r = torch.ones(T, d, dtype=BF, device=DEV), torch.ones(T, d, dtype=BF, device=DEV)
    y[1, 5], y[2, 6], r[3, 7] = float("nan"), float("inf"), float("-inf")
    R, h = oq.oq_residual_norm(y, r, pre=oq.Norm(oq.OQ_NORM_RMS, d))
    assert torch.isnan(h[1]).all() and int(torch.isnan(R[1]).sum()) == 1
    assert float(R[2, 6]) == float("inf") and float(R[3, 7]) == float("-inf") and int(torch.isinf(R).sum()) == 2
    for t in (0, 4, 5):
        assert torch.isfinite(R[t]).all() and torch.isfinite(h[t]).all()
    # nothing stands for what is not given: an infinity is not met by 0 x inf
    R, _ = oq.oq_residual_norm(None, r)
    assert not torch.isnan(R).any()
    R, _ = oq.oq_residual_norm(y[2:3], None)
    assert not torch.isnan(R).any()


def test_zero_rows_and_eps():
    z = torch.zeros(4, 512, dtype=BF, device=DEV)
    for kind in (oq.OQ_NORM_RMS, oq.OQ_NORM_LAYER):
        R, h = oq.oq_residual_norm(z, z, post=oq.Norm(kind, 512, 1e-5), pre=oq.Norm(kind, 512, 1e-5))
        assert not R.any() and not h.any()
    check(10, 512, eps=3.0, post=oq.OQ_NORM_LAYER)
    check(10, 512, eps=0.0)


def test_empty():
    e = torch.empty(0, 64, dtype=BF, device=DEV)
    R, h = oq.oq_residual_norm(e, e, post=oq.Norm(oq.OQ_NORM_RMS, 64), pre=oq.Norm(oq.OQ_NORM_RMS, 64))
    assert R.shape == h.shape == (0, 64)


def test_streams_and_graphs():
    T, k, d = 40, 4, 1024
    g = torch.Generator(device=DEV).manual_seed(0)
    ys = [torch.randn(T * k, d, generator=g, device=DEV).bfloat16() for _ in range(4)]
    w, r = torch.rand(T, k, generator=g, device=DEV), torch.randn(T, d, generator=g, device=DEV).bfloat16()
    n = oq.Norm(oq.OQ_NORM_RMS, d, w=torch.rand(d, generator=g, device=DEV))
    want = [oq.oq_residual_norm(y, r, w, pre=n) for y in ys]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = oq.oq_residual_norm(ys[1], r, w, pre=n)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[1], want[1][1])
    y = torch.empty_like(ys[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = oq.oq_residual_norm(y, r, w, pre=n)
    for i in range(4):
        y.copy_(ys[i])
        graph.replay()
        assert torch.equal(out[0], want[i][0]) and torch.equal(out[1], want[i][1])
        oq.oq_residual_norm(ys[3 - i], r, w, pre=n)
        torch.cuda.synchronize()
