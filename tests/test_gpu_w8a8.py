"""int8 x int8 product (oq_gemm_w8a8) and its weights (oq_quant_weight_w8)
against 64-bit results.

Bound on one output: the int32 sum is exact; its float32 conversion, the
product of the two scales and their product are one rounding each (3 of
2^-24 relative), the rank-1 and bias terms one each, the bfloat16 result one
of 2^-8 relative.  So |y - exact| <= 2^-8 |exact| + 2^-21 (|a s acc| +
|mean w1| + |bias|), the second term also covering the float32 errors'
share of the bfloat16 rounding."""
import numpy as np
import pytest
import torch

import rotated_bit_quantized_amd as oq

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _codes(rows, cols, seed, lo=-127, hi=127):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(lo, hi + 1, (rows, cols), generator=g, dtype=torch.int32).to(torch.int8)


def _case(M, K, N, center, bias, seed=0, lda=None, ldw=None, lo=-127, hi=127):
    g = torch.Generator().manual_seed(seed + 99)
    qa, w = _codes(M, K, seed, lo, hi), _codes(N, K, seed + 1, lo, hi)
    a_s, w_s = torch.rand(M, generator=g) * 0.02 + 1e-3, torch.rand(N, generator=g) * 1e-3 + 1e-5
    mean = torch.randn(M, generator=g) * 3 if center else None
    w1 = torch.randn(N, generator=g) if center else None
    b = torch.randn(N, generator=g) if bias else None
    acc = (qa.to(DEV).double() @ w.to(DEV).double().t()).cpu()  # whole numbers below 2^53: exact
    p = a_s.double()[:, None] * w_s.double() * acc
    exact, mag = p.clone(), p.abs()
    if center:
        r = torch.outer(mean.double(), w1.double())
        exact, mag = exact + r, mag + r.abs()
    if bias:
        exact, mag = exact + b.double(), mag + b.double().abs()
    dev = [t.to(DEV) if t is not None else None for t in (a_s, w_s, mean, w1, b)]

    def laid(t, ld):
        if ld is None:
            return t.to(DEV)
        full = torch.full((t.shape[0], ld), 77, dtype=torch.int8, device=DEV)
        full[:, : t.shape[1]] = t.to(DEV)
        return full[:, : t.shape[1]]

    return laid(qa, lda), dev[0], laid(w, ldw), dev[1], dict(mean=dev[2], w1=dev[3], bias=dev[4]), exact, mag


def _check(y, exact, mag):
    y = y.double().cpu()
    tol = 2.0 ** -8 * exact.abs() + 2.0 ** -21 * mag
    off = (y - exact).abs()
    assert torch.isfinite(y).all()
    bad = off > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside, worst {float((off / tol.clamp_min(1e-30)).max()):.2f} of the bound, first at {bad.nonzero()[0].tolist()}"


SHAPES = [
    # single tokens and a few, every kind of K tail
    (1, 16, 1), (1, 32, 64), (1, 48, 33), (1, 4096, 6144), (2, 80, 17), (3, 1040, 129), (8, 1920, 1920), (15, 144, 31),
    (16, 2064, 257), (17, 272, 63), (31, 112, 96), (33, 4112, 100),
    # between, ragged
    (47, 1024, 1024), (64, 64, 64), (65, 528, 65), (77, 1936, 515), (100, 8208, 72), (127, 256, 129), (128, 128, 128),
    (129, 3072, 257), (200, 96, 1000), (256, 1024, 1024), (257, 1040, 383), (333, 1920, 770),
    # several tiles each way, odd remainders
    (511, 144, 513), (640, 2048, 1152), (1000, 1008, 1100), (1025, 528, 2049), (2049, 272, 777), (4096, 1040, 1100),
    # the widest tiles, ragged
    (4090, 400, 4085), (2030, 272, 4001), (1000, 144, 4099),
    # wide and tall
    (5, 64, 20001), (4097, 48, 3), (300, 16400, 40), (1, 131056, 5),
]


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("epi", ["plain", "full"])
def test_product(M, K, N, epi):
    qa, a_s, w, w_s, kw, exact, mag = _case(M, K, N, epi == "full", epi == "full", seed=M + 3 * K + 7 * N)
    _check(oq.oq_gemm_w8a8(qa, a_s, w, w_s, **kw), exact, mag)


@pytest.mark.parametrize("M,K,N", [(1, 144, 40), (20, 80, 300), (70, 1040, 130), (300, 528, 600), (1100, 272, 1300)])
def test_strides_and_guard(M, K, N):
    """Padded rows of codes, padding bytes that would change the sum, a y whose
    rows start at odd places; nothing outside [M][N] is written."""
    qa, a_s, w, w_s, kw, exact, mag = _case(M, K, N, False, True, seed=5, lda=K + 48, ldw=K + 16)
    full = torch.full((M + 2, N + 13), 3.0, dtype=torch.bfloat16, device=DEV)
    y = full[1:-1, 5 : 5 + N]
    oq.oq_gemm_w8a8(qa, a_s, w, w_s, y=y, **kw)
    _check(y, exact, mag)
    full[1:-1, 5 : 5 + N] = 3.0
    assert (full == 3.0).all()


@pytest.mark.parametrize("M", [1, 40, 200, 1030])
def test_extreme_codes_do_not_overflow(M):
    K, N = 131056, 24
    qa = torch.full((M, K), -128, dtype=torch.int8, device=DEV)
    w = torch.full((N, K), -128, dtype=torch.int8, device=DEV)
    w[1::2] = 127
    one = torch.ones(max(M, N), device=DEV)
    y = oq.oq_gemm_w8a8(qa, one[:M], w, one[:N]).double().cpu()
    want = torch.tensor([128.0 * 128 * K, -128.0 * 127 * K], dtype=torch.float64).repeat(N // 2).expand(M, N)
    assert ((y - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -21 * want.abs()).all()


@pytest.mark.parametrize("M", [1, 9, 50, 130, 400])
def test_small_sums_are_exact(M):
    """With unit scales and |acc| <= 256 every output is the integer itself."""
    K, N = 64, 200
    qa, w = _codes(M, K, 1, -2, 2), _codes(N, K, 2, -2, 2)
    one = torch.ones(max(M, N), device=DEV)
    y = oq.oq_gemm_w8a8(qa.to(DEV), one[:M], w.to(DEV), one[:N]).cpu().float()
    assert torch.equal(y, (qa.float() @ w.float().t()))


def test_rows_do_not_depend_on_the_batch():
    """The tile follows M, the result does not."""
    K, N = 1936, 1000
    qa, a_s, w, w_s, kw, _, _ = _case(700, K, N, True, True, seed=11)
    whole = oq.oq_gemm_w8a8(qa, a_s, w, w_s, **kw)
    for M in (1, 5, 16, 33, 100, 300):
        part = oq.oq_gemm_w8a8(qa[:M], a_s[:M], w, w_s, mean=kw["mean"][:M], w1=kw["w1"], bias=kw["bias"])
        assert torch.equal(part, whole[:M])


def test_empty():
    qa = torch.zeros((0, 64), dtype=torch.int8, device=DEV)
    w = torch.zeros((8, 64), dtype=torch.int8, device=DEV)
    y = oq.oq_gemm_w8a8(qa, torch.zeros(0, device=DEV), w, torch.ones(8, device=DEV))
    assert y.shape == (0, 8)
    y = oq.oq_gemm_w8a8(w, torch.ones(8, device=DEV), qa, torch.zeros(0, device=DEV))
    assert y.shape == (8, 0)


@pytest.mark.parametrize("M", [3, 60, 500])
def test_other_stream_and_graph(M):
    qa, a_s, w, w_s, kw, exact, mag = _case(M, 1040, 520, False, True, seed=21)
    y = torch.empty(M, 520, dtype=torch.bfloat16, device=DEV)
    oq.oq_gemm_w8a8(qa, a_s, w, w_s, y=y, **kw)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y2 = torch.empty_like(y)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        oq.oq_gemm_w8a8(qa, a_s, w, w_s, y=y2, **kw)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, y2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        oq.oq_gemm_w8a8(qa, a_s, w, w_s, y=y2, **kw)
    for i in range(3):
        y2.zero_()
        a_s.mul_(1.5)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y2, oq.oq_gemm_w8a8(qa, a_s, w, w_s, **kw))


@pytest.mark.parametrize("N,K,ldw", [(1, 16, 16), (33, 1920, 1924), (70, 3072, 3072), (5, 16384, 16384)])
def test_weight_codes(N, K, ldw):
    """Without a rotation: scale RN32(a / 127) and codes of the nearest integer
    of v RN32(127 / a); the row sums in float64."""
    g = torch.Generator().manual_seed(K)
    full = torch.randn(N, ldw, generator=g) * 0.02
    W = full[:, :K]
    got = oq.oq_quant_weight_w8(full.to(DEV)[:, :K], want_w1=True)
    a = np.maximum(np.abs(W.numpy()).max(1), np.float32(1e-10))
    assert np.array_equal(got["scales"].cpu().numpy(), a / np.float32(127))
    q = np.rint(W.numpy() * (np.float32(127) / a)[:, None])
    assert np.array_equal(got["codes"].cpu().numpy(), np.clip(q, -127, 127).astype(np.int8))
    s64 = W.double().sum(1)
    assert ((got["w1"].double().cpu() - s64).abs() <= 2.0 ** -24 * s64.abs() + 1e-12 * W.double().abs().sum(1)).all()


@pytest.mark.parametrize("kind", ["rpbh1", "rpbh2", "kron"])
def test_rotated_layer(kind):
    """Rotated activations (A8) times rotated weights: the unrotated product to
    the accuracy of 8-bit codes, and exactly what the codes say."""
    g = torch.Generator().manual_seed(3)
    M, K, N = 130, 1920, 257
    x = torch.randn(M, K, generator=g).to(torch.bfloat16).to(DEV)
    W = (torch.randn(N, K, generator=g) * 0.02).to(DEV)
    if kind == "kron":
        rot = oq.Rotation.kron(K)
    else:
        rounds = int(kind[-1])
        perm = torch.stack([torch.randperm(K, generator=g) for _ in range(rounds)]).to(DEV)
        signs = (torch.randint(0, 2, (rounds, K), generator=g) * 2 - 1).to(DEV)
        rot = oq.Rotation.rpbh(perm, signs, 128)
    wq = oq.oq_quant_weight_w8(W, rot, want_w1=True)
    act = oq.oq_quant_act(x, rot, oq.OQ_A8, center=True)
    bias = torch.randn(N, generator=g).to(DEV)
    y = oq.oq_gemm_w8a8(act["codes"], act["scale"], wq["codes"], wq["scales"], mean=act["mean"], w1=wq["w1"], bias=bias)
    p = act["scale"].double()[:, None] * wq["scales"].double() * (act["codes"].double() @ wq["codes"].double().t())
    r = torch.outer(act["mean"].double(), wq["w1"].double())
    exact = p + r + bias.double()
    _check(y, exact.cpu(), (p.abs() + r.abs() + bias.double().abs()).cpu())
    ref = x.double() @ W.double().t() + bias.double()
    assert float((y.double() - ref).norm() / ref.norm()) < 0.03


FEW_OUTPUTS = [
    # more tokens than one group of 16 or 32, few weight rows: k split over the wavefronts
    (33, 16, 5), (37, 4112, 50), (49, 1008, 16), (100, 14336, 500), (130, 2064, 31), (1000, 8208, 17), (4100, 32, 1), (250, 528, 255),
    # groups of 32, ragged, one or two rounds
    (48, 4096, 2000), (65, 272, 1500), (300, 1040, 700), (95, 16400, 1030),
    # long k, a chunk of which ends inside a KiB
    (17, 131056, 33), (40, 40016, 100), (64, 15376, 1000),
]


@pytest.mark.parametrize("M,K,N", FEW_OUTPUTS)
def test_few_outputs(M, K, N):
    qa, a_s, w, w_s, kw, exact, mag = _case(M, K, N, True, M % 2 == 0, seed=M + N, lda=K + 48, ldw=K + 16)
    _check(oq.oq_gemm_w8a8(qa, a_s, w, w_s, **kw), exact, mag)
