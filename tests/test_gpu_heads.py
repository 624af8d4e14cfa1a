"""Head norm with rotary embedding (oq_qk_norm_rope) and the paged append
(oq_kv_append) against 64-bit results.

Bound on one output element: the norm's sum of squares, its mean, root and
reciprocal and the two products are at most 24 float32 roundings (the sum of
8 terms a lane and 6 cross-lane adds among them, halved by the root), each
rotary term 3 more, so the float32 value is within 32 * 2^-24 = 2^-19 of the
sum of the magnitudes of its terms; the bfloat16 rounding adds 2^-8 of the
result."""
import pytest
import torch

import rotated_bit_quantized_amd as oq

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-6


def _tables(rows, dim, seed=0):
    f = 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    a = torch.arange(rows, dtype=torch.float64)[:, None] * f
    return a.cos().float().to(DEV), a.sin().float().to(DEV)


def _exact(x, w, rope, pos, eps=EPS):
    """(value, sum of the magnitudes of its terms), float64 [T][H][d]."""
    x = x.double()
    if w is not None:
        x = x / ((x * x).mean(-1, keepdim=True) + eps).sqrt() * w.double()
    y, mag = x.clone(), x.abs()
    if rope is not None:
        dim = rope.c.dim
        at = torch.arange(x.shape[0], device=x.device) if pos is None else pos.long()
        ok = (at >= 0) & (at < rope.cos.shape[0])
        c, s = (t[at.clamp(0, rope.cos.shape[0] - 1)].double()[:, None] for t in (rope.cos, rope.sin))
        ia = torch.arange(dim // 2, device=x.device)
        ia, ib = (2 * ia, 2 * ia + 1) if rope.interleaved else (ia, ia + dim // 2)
        a, b = x[..., ia], x[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        mag[..., ia], mag[..., ib] = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
        y[~ok] = float("nan")
    return y, mag


def _check(got, y, mag):
    got = got.double()
    nan = torch.isnan(y)
    assert torch.equal(torch.isnan(got), nan)
    off = (got - y).abs()[~nan]
    tol = (2.0 ** -8 * y.abs() + 2.0 ** -19 * mag)[~nan]
    assert (off <= tol).all(), f"worst {float((off / tol.clamp_min(1e-30)).max()):.2f} of the bound"


def _x(T, H, d, seed, layout="rows"):
    """bfloat16 [T][H][d]: dense, a part of wider rows, or head-major."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    if layout == "rows":
        return torch.randn(T, H, d, generator=g, device=DEV).to(torch.bfloat16)
    if layout == "wide":
        return torch.randn(T, H * d + 2 * d + 8, generator=g, device=DEV).to(torch.bfloat16)[:, 8 : 8 + H * d].unflatten(1, (H, d))
    return torch.randn(H, T, d + 16, generator=g, device=DEV).to(torch.bfloat16)[:, :, 8 : 8 + d].transpose(0, 1)


WIDTHS = [  # d, rotary dim (0: none), pairs interleaved
    (8, 8, False), (8, 2, True), (16, 16, False), (16, 10, False), (40, 24, True), (64, 64, False), (64, 32, True),
    (64, 48, False), (72, 0, False), (80, 40, False), (80, 40, True), (80, 20, True), (96, 96, False), (128, 128, False),
    (128, 128, True), (128, 64, False), (136, 136, True), (256, 256, False), (256, 64, True), (264, 18, False),
    (512, 512, False), (512, 500, False), (512, 512, True),
]


@pytest.mark.parametrize("d,dim,inter", WIDTHS)
@pytest.mark.parametrize("norm", [True, False])
def test_widths_and_pairs(d, dim, inter, norm):
    for T, hq, hk in ((1, 1, 1), (3, 5, 2), (67, 9, 3)):
        q, k = _x(T, hq, d, 1), _x(T, hk, d, 2)
        g = torch.Generator(device=DEV).manual_seed(5)
        w = [1 + 0.3 * torch.randn(d, generator=g, device=DEV) for _ in range(2)] if norm else [None, None]
        rope = oq.Rope(*_tables(100, dim), inter) if dim else None
        pos = torch.randint(0, 100, (T,), generator=g, device=DEV).int()
        qo, ko = oq.oq_qk_norm_rope(q, k, w[0], w[1], EPS, rope, pos if rope else None)
        _check(qo, *_exact(q, w[0], rope, pos))
        _check(ko, *_exact(k, w[1], rope, pos))


@pytest.mark.parametrize("lay_in", ["rows", "wide", "heads"])
@pytest.mark.parametrize("lay_out", ["rows", "wide", "heads"])
@pytest.mark.parametrize("T,hq,hk,d", [(1, 32, 8, 128), (130, 24, 24, 64), (1000, 16, 2, 80), (5000, 7, 1, 128)])
def test_layouts(lay_in, lay_out, T, hq, hk, d):
    q, k = _x(T, hq, d, 1, lay_in), _x(T, hk, d, 2, lay_in)
    qo, ko = _x(T, hq, d, 3, lay_out), _x(T, hk, d, 4, lay_out)
    w = torch.rand(d, device=DEV) + 0.5
    rope = oq.Rope(*_tables(T, d))
    base = qo._base if qo._base is not None else qo
    rest = base.clone()
    oq.oq_qk_norm_rope(q, k, w, None, EPS, rope, None, q_out=qo, k_out=ko)
    _check(qo, *_exact(q, w, rope, None))
    _check(ko, *_exact(k, None, rope, None))
    if qo._base is not None:  # nothing else of the output's buffer has changed
        view = torch.as_strided(rest, qo.shape, qo.stride(), qo.storage_offset())
        view.copy_(qo)
        assert torch.equal(base, rest)


def test_in_place_and_one_side_only():
    x = _x(100, 48, 128, 1)
    rope = oq.Rope(*_tables(128, 128))
    w = torch.rand(128, device=DEV) + 0.5
    want, want_k = oq.oq_qk_norm_rope(x[:, :32], x[:, 32:40], w, w, EPS, rope)
    keep = x.clone()
    oq.oq_qk_norm_rope(x[:, :32], x[:, 32:40], w, w, EPS, rope, q_out=x[:, :32], k_out=x[:, 32:40])
    assert torch.equal(x[:, :32], want) and torch.equal(x[:, 32:40], want_k) and torch.equal(x[:, 40:], keep[:, 40:])
    only, none = oq.oq_qk_norm_rope(keep[:, :32], None, w, None, EPS, rope)
    assert none is None and torch.equal(only, want)
    none, only = oq.oq_qk_norm_rope(None, keep[:, 32:40], None, w, EPS, rope)
    assert none is None and torch.equal(only, want_k)


def test_positions_outside_the_table_give_nan():
    q, k = _x(6, 3, 64, 1), _x(6, 2, 64, 2)
    rope = oq.Rope(*_tables(50, 64))
    pos = torch.tensor([0, -1, 49, 50, -(2 ** 31), 2 ** 31 - 1], device=DEV, dtype=torch.int64).int()
    qo, ko = oq.oq_qk_norm_rope(q, k, None, None, EPS, rope, pos)
    _check(qo, *_exact(q, None, rope, pos))
    _check(ko, *_exact(k, None, rope, pos))


@pytest.mark.parametrize("scale", [1e-20, 1e-3, 1e4, 1e15])
def test_norm_over_the_range(scale):
    q = (_x(20, 4, 128, 1).float() * scale).to(torch.bfloat16)
    q[3] = 0
    w = torch.rand(128, device=DEV) + 0.5
    qo, _ = oq.oq_qk_norm_rope(q, None, w, None, EPS)
    _check(qo, *_exact(q, w, None, None))


def test_infinities_and_nan_stay_in_their_head():
    q = _x(4, 4, 64, 1)
    q[1, 2, 5], q[2, 1, 7] = float("inf"), float("nan")
    rope = oq.Rope(*_tables(4, 64))
    w = torch.ones(64, device=DEV)
    qo, _ = oq.oq_qk_norm_rope(q, None, w, None, EPS, rope)
    ok = torch.ones(4, 4, dtype=torch.bool)
    ok[1, 2] = ok[2, 1] = False
    y, mag = _exact(q, w, rope, None)
    _check(qo[ok], y[ok], mag[ok])
    assert torch.isnan(qo[2, 1]).any()


def test_empty_and_passthrough():
    q = _x(0, 4, 64, 1)
    qo, ko = oq.oq_qk_norm_rope(q, q, None, None)
    assert qo.shape == q.shape
    x = _x(33, 4, 64, 2)
    x[0, 0, 0] = float("nan")
    qo, _ = oq.oq_qk_norm_rope(x, None)
    assert torch.equal(qo.view(torch.int16), x.view(torch.int16))


@pytest.mark.parametrize("H,d,dim,inter,page,norm", [
    (8, 128, 128, False, 64, True), (1, 64, 64, True, 16, True), (30, 64, 32, True, 8, False), (3, 80, 40, False, 128, True),
    (2, 256, 128, False, 32, False), (5, 8, 0, False, 1024, True), (2, 512, 512, False, 16, True), (4, 96, 0, False, 32, False),
])
@pytest.mark.parametrize("T", [1, 7, 300])
def test_append(H, d, dim, inter, page, norm, T):
    g = torch.Generator(device=DEV).manual_seed(T + d)
    pages = -(-2 * T // page) + 2
    both = torch.randn(pages, 2, H, page, d, generator=g, device=DEV).to(torch.bfloat16)  # pages of k and v side by side
    before = both.clone()
    kv = oq.PagedKV(both[:, 0], both[:, 1])
    k, v = _x(T, H, d, 1, "wide"), _x(T, H, d, 2, "heads")
    v[0, 0, 0] = float("nan")  # values pass as they are
    w = torch.rand(d, device=DEV, generator=g) + 0.5 if norm else None
    rope = oq.Rope(*_tables(500, dim), inter) if dim else None
    pos = torch.randint(0, 500, (T,), generator=g, device=DEV).int()
    slot = torch.randperm(pages * page, generator=g, device=DEV)[:T]
    if T > 4:
        slot[1], slot[2], slot[3], slot[4] = -1, pages * page, -(2 ** 62), 2 ** 62
    oq.oq_kv_append(k, v, slot, kv, w, EPS, rope, pos if rope else None)
    ok = (slot >= 0) & (slot < pages * page)
    at, off = slot[ok] // page, slot[ok] % page
    y, mag = _exact(k, w, rope, pos)
    _check(both[at, 0, :, off], y[ok], mag[ok])
    assert torch.equal(both[at, 1, :, off].view(torch.int16), v[ok].contiguous().view(torch.int16))
    both[at, :, :, off] = before[at, :, :, off]
    assert torch.equal(both.view(torch.int16), before.view(torch.int16))


def test_append_past_4_gib():
    """Pages more than 2^32 bytes (and 2^31 elements) from the base of the cache."""
    pages, H, page, d, stride = 3, 2, 16, 64, 3 << 29
    caches = [torch.as_strided(torch.empty((pages - 1) * stride + H * page * d, dtype=torch.bfloat16, device=DEV),
                               (pages, H, page, d), (stride, page * d, d, 1)) for _ in range(2)]
    k, v = _x(3, H, d, 1), _x(3, H, d, 2)
    slot = torch.tensor([5, 17, 47], device=DEV)
    kv = oq.PagedKV(*caches)
    oq.oq_kv_append(k, v, slot, kv)
    for t, (p, o) in enumerate(((0, 5), (1, 1), (2, 15))):
        assert torch.equal(kv.k[p, :, o], k[t]) and torch.equal(kv.v[p, :, o], v[t])


def test_streams_and_graph():
    T, H, d, page = 40, 8, 128, 16
    k, v, q = _x(T, H, d, 1), _x(T, H, d, 2), _x(T, 32, d, 3)
    cache = [torch.zeros(8, H, page, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    kv = oq.PagedKV(*cache)
    w = torch.rand(d, device=DEV) + 0.5
    rope = oq.Rope(*_tables(64, d))
    pos = torch.arange(T, device=DEV).int()
    slot = torch.arange(T, device=DEV)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    oq.oq_qk_norm_rope(q, k, w, w, EPS, rope, pos, q_out=qo, k_out=ko)  # first use of the kernels outside the capture
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        oq.oq_kv_append(k, v, slot, kv, w, EPS, rope, pos)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(kv.k[0, :, 3], ko[3])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        oq.oq_qk_norm_rope(q, k, w, w, EPS, rope, pos, q_out=qo, k_out=ko)
        oq.oq_kv_append(k, v, slot, kv, w, EPS, rope, pos)
    for i in range(3):
        q.copy_(_x(T, 32, d, 10 + i))
        k.copy_(_x(T, H, d, 20 + i))
        pos.add_(5)
        slot.add_(7)
        g.replay()
        torch.cuda.synchronize()
        eq, ek = oq.oq_qk_norm_rope(q, k, w, w, EPS, rope, pos)
        assert torch.equal(eq, qo) and torch.equal(ek, ko)
        assert torch.equal(cache[0][slot // page, :, slot % page], ek)
        assert torch.equal(cache[1][slot // page, :, slot % page], v)


@pytest.mark.parametrize("T,hq,hk", [(9000, 5, 3), (3000, 16, 2), (2500, 7, 3), (30000, 1, 1), (12000, 2, 1)])
@pytest.mark.parametrize("d,dim,inter", [(80, 40, False), (80, 36, True), (128, 20, False), (64, 62, False), (128, 128, False), (64, 32, True)])
def test_several_heads_of_a_group(T, hq, hk, d, dim, inter):
    """Token counts at which a lane group takes one, two or four heads, every kind of pairs."""
    q, k = _x(T, hq, d, 1), _x(T, hk, d, 2)
    w = 1 + 0.3 * torch.randn(d, generator=torch.Generator(device=DEV).manual_seed(6), device=DEV)
    pos = torch.randint(0, 200, (T,), generator=torch.Generator(device=DEV).manual_seed(7), device=DEV).int()
    rope = oq.Rope(*_tables(200, dim), inter)
    qo, ko = oq.oq_qk_norm_rope(q, k, w, None, EPS, rope, pos)
    _check(qo, *_exact(q, w, rope, pos))
    _check(ko, *_exact(k, None, rope, pos))
