"""oq_gemm_lm on canonical codes whose expansion is more than one launch takes."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
DEV = "cuda"


def test_more_codes_than_a_launch_expands():
    """2^21 rows of 16384: 2^32 threads and more.  4096 different rows in turn, so every turn has the same outputs."""
    import rotated_bit_quantized_amd as oq

    M, K, N, turn = (1 << 21) + 4096, 16384, 8, 4096
    g = torch.Generator(device=DEV).manual_seed(0)
    codes = torch.randint(0, 256, (turn, K // 2), generator=g, device=DEV, dtype=torch.int32).to(torch.uint8)
    levels = torch.linspace(-2, 2, 16, device=DEV).half()
    weights = torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.int32).to(torch.uint8)
    w16 = oq.oq_prepack_w16(weights, torch.rand(N, K // 64, generator=g, device=DEV) * 0.02 + 0.001, N, K, 64)
    scale = torch.rand(turn, generator=g, device=DEV) + 0.5
    want = oq.oq_gemm_lm(4, codes, scale, w16, N, levels=levels.view(torch.int16)).float()
    got = oq.oq_gemm_lm(4, codes.repeat(M // turn, 1), scale.repeat(M // turn), w16, N, levels=levels.view(torch.int16)).view(-1, turn, N)
    assert torch.equal(got, got[:1].expand_as(got))
    # the same float16 products; sums in another order are off by K units of 2^-24 of their terms, far below a step of bfloat16
    assert ((got[0].float() - want).abs() <= 2.0 ** -7 * want.abs() + 2.0 ** -24 * K * want.abs().amax()).all()
    del got
    torch.cuda.empty_cache()
