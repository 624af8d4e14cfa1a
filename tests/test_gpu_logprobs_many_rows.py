"""oq_logprobs of more rows than the workgroups of one launch."""
import pytest
import torch

import rotated_bit_quantized_amd as oq

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("T,V,top", [(1 << 24, 4, 1), ((1 << 23) + 3, 16, 9)])
def test_more_rows_than_a_launch_takes(T, V, top):
    g = torch.Generator(device=DEV).manual_seed(top)
    x = torch.randn(T, V, generator=g, device=DEV).bfloat16()
    tok = torch.randint(0, V, (T, 1), generator=g, device=DEV, dtype=torch.int32)
    logprob, rank, entropy, lse, top_id, top_logprob = oq.oq_logprobs(x, tok, top=top)
    places = torch.sort(x.float(), dim=1, descending=True, stable=True).indices
    assert torch.equal(top_id.long(), places[:, :top])
    assert torch.equal(places.gather(1, rank.long()), tok.long())
    logp = torch.log_softmax(x.double(), 1)
    # a handful of terms: far within 64 units of 2^-24 of values below 16
    tol = 64 * 2.0 ** -24 * 16
    assert float((logprob - logp.gather(1, tok.long())).abs().max()) < tol and float((top_logprob - logp.gather(1, places[:, :top])).abs().max()) < tol
    assert float((entropy + (logp.exp() * logp).sum(1)).abs().max()) < tol and float((lse - torch.logsumexp(x.double(), 1)).abs().max()) < tol
    del logp, places
    torch.cuda.empty_cache()
