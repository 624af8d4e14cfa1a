"""oq_logprobs of nearly certain tokens: signs, and errors relative to the value.

With z = scale (x - the largest logit) and the others' sum r = sum 2^(z log2 e)
without the largest one's 1: log p = z - log1p(r), entropy = log1p(r) - sum e^z z
/ (1 + r); both parts of each have one sign, so nothing cancels.  In units of
2^-24: a distance and its product with the scale are off by 1 each; the factor
scale log2(e) by 1.5, so a term of r by 1.5 |z|, by |z| for its exponent's
rounding and 2 for the exponential; the sums over at most 64 terms a thread
and some 20 further steps 90, joining the parts of a row 2.5 |z| and 6 more:
(3 A + 110) log1p(r) with A = sum e^z |z| / r over the others (log1p passes on no
more than the relative error of r), and 4 of the value for log1p and the last steps.
Terms below 2^-126 may be lost."""
import pytest
import torch

import rotated_bit_quantized_amd as oq

pytestmark = pytest.mark.gpu
DEV, U = "cuda", 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
SHAPES = [(1, 32000, F32), (40, 32000, BF), (3, 100003, BF), (3, 50001, F32), (600, 20000, BF), (530, 4001, F32), (9, 300, BF), (9, 2, F32), (2, 1, F32),
          (2, 1 << 20, F32)]


def exact(x, scale):
    """log p, entropy and their bounds in float64."""
    z = x.double()
    at = z.argmax(1, keepdim=True)
    z = (z - z.gather(1, at)) * float(torch.tensor(scale, dtype=F32))
    e = torch.exp(z).scatter_(1, at, 0.0)
    far = torch.where(e > 0, z.abs(), torch.zeros_like(z))
    r = e.sum(1, keepdim=True)
    A = (e * far).sum(1, keepdim=True) / r.clamp_min(1e-300)
    L = torch.log1p(r)
    logp = z - L
    part = (e * far).sum(1, keepdim=True) / (1 + r)
    H = L + part
    lost = x.shape[1] * 2.0 ** -118
    tol_p = U * (4 * logp.abs() + 2 * z.abs() + (3 * A + 110) * L) + lost
    tol_h = U * (4 * H + (3 * A + 110) * L + (e * far * (3 * far + 110)).sum(1, keepdim=True) / (1 + r) + (3 * A + 110) * r / (1 + r) * part) + lost
    return logp, H[:, 0], tol_p, tol_h[:, 0]


def check(x, tok, top, scale):
    logp, H, tol_p, tol_h = exact(x, scale)
    logprob, _, entropy, _, top_id, top_logprob = oq.oq_logprobs(x, tok, top=top, scale=scale)
    for got, at in ((logprob, tok.long()), (top_logprob, top_id.long())):
        off, tol = (got.double() - logp.gather(1, at)).abs(), tol_p.gather(1, at)
        assert (off <= tol).all(), f"off by {float((off / tol).max()):.2f} of the bound"
        assert (got <= 0).all()
    off = (entropy.double() - H).abs()
    assert (off <= tol_h).all(), f"entropy off by {float((off / tol_h).max()):.2f} of the bound"
    assert (entropy >= 0).all()


@pytest.mark.parametrize("T,V,dtype", SHAPES)
@pytest.mark.parametrize("gap", [0.0, 6.0, 14.0, 18.0, 25.0, 60.0])
@pytest.mark.parametrize("level,scale", [(0.0, 1.0), (37.0, 1.25), (-500.0, 0.7), (3001.0, 1.0)])
def test_relative_errors_and_signs(T, V, dtype, gap, level, scale):
    g = torch.Generator(device=DEV).manual_seed(V + int(gap))
    x = torch.randn(T, V, generator=g, device=DEV)
    tok = torch.randint(0, V, (T, 2), generator=g, device=DEV, dtype=torch.int32)
    x.scatter_(1, tok[:, :1].long(), gap + torch.rand(T, 1, generator=g, device=DEV))
    check((x + level).to(dtype), tok, min(V, 5), scale)


@pytest.mark.parametrize("T,V", [(5, 1000), (5, 70000), (600, 9000)])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("low", [-float("inf"), "lowest", -2000.0])
def test_a_token_beside_which_all_vanish(T, V, dtype, low):
    """Log probability, entropy and loss are exactly 0, whatever the logit's bits."""
    low = torch.finfo(dtype).min if low == "lowest" else low
    g = torch.Generator(device=DEV).manual_seed(V)
    x = torch.full((T, V), low, dtype=dtype, device=DEV)
    tok = torch.randint(0, V, (T, 1), generator=g, device=DEV, dtype=torch.int32)
    x.scatter_(1, tok.long(), (50 * torch.randn(T, 1, generator=g, device=DEV)).to(dtype))
    logprob, rank, entropy, lse, _, top_logprob = oq.oq_logprobs(x, tok, top=1)
    assert not rank.any() and not logprob.any() and not entropy.any() and not top_logprob.any()
    assert torch.equal(lse, x.gather(1, tok.long())[:, 0].float())


@pytest.mark.parametrize("T,V", [(3, 9000), (3, 70000)])
def test_several_largest(T, V):
    """n equal largest logits in one thread, in several wavefronts, in several parts: log p = -log n."""
    for places in ([0, 1], [3, V // 2, V - 1], list(range(0, V, 97)), list(range(V))):
        x = torch.full((T, V), 17.3 - 900.0, device=DEV)
        x[:, places] = 17.3
        tok = torch.tensor([[places[-1]]] * T, dtype=torch.int32, device=DEV)
        check(x, tok, 2, 1.0)
        check(x.to(BF), tok, 2, 1.0)


@pytest.mark.parametrize("V", [300, 40000])
def test_distances_past_float32(V):
    """The largest logit is far past 2^31, and a difference of two is not a float32 while its product with the scale is one."""
    x = torch.zeros(3, V, device=DEV)
    x[:, 7], x[:, 9] = 3.3e38, -3.3e38
    tok = torch.tensor([[7, 9, 0]] * 3, dtype=torch.int32, device=DEV)
    logprob, _, entropy, lse, _, _ = oq.oq_logprobs(x, tok, scale=0.125)
    want = (x.double() - x.double().amax(1, keepdim=True)).gather(1, tok.long()) * 0.125
    assert ((logprob.double() - want).abs() <= 2.0 ** -21 * want.abs()).all()
    assert (entropy == 0).all() and torch.allclose(lse, x[:, 7] * 0.125, rtol=1e-6)
    assert (oq.oq_logprobs(x, tok)[0][:, 1] == -float("inf")).all()
