"""oq_gemm_w8a8_experts where it runs the persistent tiles: K above 384, and more
column tiles of 256 weight rows over the reached experts than half of the CUs, or
more than 32 entries an expert.  Bounds as in test_gpu_experts.py."""
import pytest
import torch

import rotated_bit_quantized_amd as oq
from test_gpu_experts import DEV, Case, lists_of, routed

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [400, 528, 1040])
@pytest.mark.parametrize("N", [1, 34, 130, 255, 256, 257, 513, 1026])
def test_outputs(K, N):
    """One expert has more than eight row tiles: bands with a short last one."""
    ids = torch.zeros(2300, 1, dtype=torch.int32)
    ids[:700] = routed(700, 4, 1, N)
    ids = ids[torch.randperm(len(ids), generator=torch.Generator().manual_seed(K))]
    Case(ids, 4, K, N, seed=N).check()
    Case(ids, 4, K, 2 * N, act=True, seed=N).check()


@pytest.mark.parametrize("K", [400, 496, 512, 640, 1008, 1040, 4112])
@pytest.mark.parametrize("act", [False, True])
def test_several_tiles_a_workgroup(K, act):
    """More than two tiles for each of 256 CUs, with every addend and padded strides."""
    N = 1540
    c = Case(routed(6000, 9, 2, K), 9, K, N, act, center=True, bias=True, seed=K, lda=48, ldw=16)
    out = N // 2 if act else N
    y = torch.full((c.n, out + 13), -3.0, dtype=torch.bfloat16, device=DEV)
    c.check(y[:, 5:5 + out])
    assert (y[:, :5] == -3).all() and (y[:, 5 + out:] == -3).all()
    y = c.check()
    order = [int(i) for i in torch.randperm(c.n, generator=torch.Generator().manual_seed(1))[:500]]
    assert torch.equal(y[order], c.run()[order])


@pytest.mark.parametrize("center,bias", [(True, False), (False, True), (False, False)])
def test_mean_or_bias_alone(center, bias):
    Case(routed(3000, 6, 2, 3), 6, 432, 1030, True, center=center, bias=bias, seed=5).check()


@pytest.mark.parametrize("E", [63, 64, 65, 127, 128, 129, 200, 1000, 1023, 1024])
def test_many_experts(E):
    """One expert a lane and several; every expert has some 35 entries, some none."""
    T = 9 * E
    ids = routed(T, E, 4, E, skew=0.3)
    ids[ids == E // 2] = -1
    Case(ids, E, 400, 36, seed=E).check()


@pytest.mark.parametrize("T,E,k,N", [(1, 64, 1, 40000), (1, 128, 8, 5000), (3, 60, 4, 3070), (70, 128, 1, 514), (16, 128, 8, 770), (5, 1000, 2, 4000)])
def test_few_entries_and_wide_weights(T, E, k, N):
    Case(routed(T, E, k, T), E, 416, N, seed=T, bias=True).check()
    Case(routed(T, E, k, T), E, 416, N, act=True, seed=T, per=1).check()


def test_counts_at_the_tiles_borders():
    counts = [0, 1, 31, 32, 33, 63, 64, 65, 95, 96, 97, 127, 128, 129, 0, 255, 256, 257, 383, 1023, 1024, 1025, 1153, 0]
    ids = torch.repeat_interleave(torch.arange(len(counts), dtype=torch.int32), torch.tensor(counts))[:, None]
    ids = ids[torch.randperm(len(ids), generator=torch.Generator().manual_seed(0))]
    Case(ids, len(counts), 464, 520, True, seed=2).check()
    Case(ids, len(counts), 464, 520, seed=2, center=True).check()


def test_the_largest_codes():
    Case(routed(80, 4, 2), 4, 131056, 16, lo=-128, hi=-128).check()


@pytest.mark.parametrize("act", [False, True])
def test_rows_without_expert_stay(act):
    ids = routed(4000, 7, 3, 5)
    ids[torch.rand(4000, 3, generator=torch.Generator().manual_seed(6)) < 0.4] = -1
    c = Case(ids, 7, 432, 1540, act, bias=True)
    y = torch.full((c.n, 770 if act else 1540), 9.0, dtype=torch.bfloat16, device=DEV)
    c.check(y)
    assert (y[(ids.flatten() < 0).to(DEV)] == 9).all()


def test_list_values_outside_their_range_are_ignored():
    ids = routed(3000, 4, 2, 5)
    c = Case(ids, 4, 400, 1032)
    want = c.check()
    order = c.order.clone()
    hit = list(range(0, c.n, 53)) + [c.n - 1]
    lost = order[hit].long()
    order[hit] = torch.tensor([-5, c.n, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=DEV).repeat(len(hit))[: len(hit)]
    y = torch.full_like(want, 9.0)
    c.run(y, order=order)
    kept = torch.ones(c.n, dtype=torch.bool, device=DEV)
    kept[lost] = False
    assert torch.equal(y[kept], want[kept]) and (y[~kept] == 9).all()
    y = torch.full_like(want, 9.0)
    c.run(y, offsets=torch.tensor([-9, 0, 0, 0, 2 ** 31 - 1], dtype=torch.int32, device=DEV))  # all of them at the last expert
    last = Case(torch.full_like(ids, 3), 4, 400, 1032)
    last.qa, last.w, last.a_scale, last.w_scale = c.qa, c.w, c.a_scale, c.w_scale
    assert torch.equal(y, last.run())
    y = torch.full_like(want, 9.0)
    c.run(y, offsets=torch.tensor([5000, 700, 700, 3, 3], dtype=torch.int32, device=DEV))  # falling: empty
    assert (y == 9).all()


def test_a_rows_bits_do_not_depend_on_the_others():
    """Entry 0 .. 11 alone and among a hundred (not the tiles), among hundreds and among thousands (the tiles)."""
    E, K, N = 8, 528, 1100
    ids = routed(9000, E, 2, 8)
    got = []
    for T in (6, 60, 400, 9000):
        c = Case(ids, E, K, N, True, center=True, bias=True, seed=4)
        c.ids, c.n = ids[:T], 2 * T
        c.offsets, c.order = (t.to(DEV) for t in lists_of(ids[:T], E))
        got.append(c.run()[:12])
    for y in got[1:]:
        assert torch.equal(y, got[0])


def test_agrees_with_the_plain_product():
    c = Case(torch.zeros(5000, 1, dtype=torch.int32), 1, 656, 3333, center=True, bias=True)
    y = oq.oq_gemm_w8a8(c.qa, c.a_scale, c.w[0], c.w_scale[0], c.mean, c.w1[0], c.bias[0])
    assert torch.equal(y, c.check())


def test_streams_and_graphs():
    c, other = Case(routed(5000, 8, 2), 8, 464, 1540, True), Case(routed(5000, 8, 2, 9), 8, 464, 1540, True, seed=3)
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
        if i == 2:
            c.qa.copy_(other.qa)
            c.offsets.copy_(other.offsets), c.order.copy_(other.order)
        y.zero_()
        g.replay()
        assert torch.equal(oq.oq_gemm_w8a8_experts(c.qa, c.a_scale, c.w, c.w_scale, c.offsets, c.order, per=2, act=oq.OQ_ACT_SWIGLU), y)
        assert i >= 2 or torch.equal(y, want)
        assert torch.equal(other.run(), want_other)
        torch.cuda.synchronize()


@pytest.mark.parametrize("T,k", [(6, 4), (500, 4)])
def test_weights_past_4_gib(T, k):
    """160 experts of 4096 x 7168: 4.7 GB, offsets past 32 bits."""
    E, N, K = 160, 4096, 7168
    g = torch.Generator(device=DEV).manual_seed(0)
    w = torch.empty(E, N, K, dtype=torch.int8, device=DEV)
    for e in range(0, E, 8):
        w[e:e + 8] = torch.randint(-127, 128, (8, N, K), generator=g, device=DEV, dtype=torch.int16).to(torch.int8)
    ids = routed(T, E, k, 3)
    ids[0] = torch.tensor([E - 1, E - 2, E // 2, 0], dtype=torch.int32)
    c = Case(ids, 2, K, 16)  # its activations; weights and lists of the wide ones instead
    c.E, c.N, c.w, c.w_scale = E, N, w, torch.rand(E, N, generator=g, device=DEV) + 0.1
    c.offsets, c.order = (t.to(DEV) for t in lists_of(ids, E))
    c.check()
    c.act = True
    c.check()
    del w, c
    torch.cuda.empty_cache()
