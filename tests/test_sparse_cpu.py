"""Refusals of the sparse layer's operators: nothing is launched, every bad
argument has its code (CPU only)."""
import ctypes

import pytest
import torch

import rotated_bit_quantized_amd as oq
from test_serve_cpu import ALN, INV, P, P1, P4, UNS, WS, _call

B = oq._binding
OK = B.OQ_OK
P2 = ctypes.c_void_p(0x100002)
f32 = ctypes.c_float
NAN, INF = f32(float("nan")), f32(float("inf"))


def _router(bias=None, experts=64, k=4, score=oq.OQ_SCORE_SOFTMAX, groups=1, top_groups=1, group_best=1, renorm=1, factor=1.0):
    return ctypes.byref(B.oq_router(bias, experts, k, score, groups, top_groups, group_best, renorm, factor))


ROUTE = dict(logits=P, dtype=oq.OQ_F32, ld=64, T=100, mask=None, r=_router(), ids=P, weights=P, offsets=P, order=P, ws=P, ws_bytes=1 << 30,
             stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(r=None), INV), (dict(T=-1), INV), (dict(r=_router(experts=0)), INV), (dict(r=_router(k=0)), INV), (dict(r=_router(experts=1025)), UNS),
    (dict(r=_router(experts=1000, k=33)), UNS), (dict(r=_router(score=0)), INV), (dict(r=_router(score=3)), INV), (dict(r=_router(groups=0)), INV),
    (dict(r=_router(groups=65, experts=65)), UNS), (dict(r=_router(groups=3)), INV), (dict(r=_router(groups=8, top_groups=0)), INV),
    (dict(r=_router(groups=8, top_groups=9)), INV), (dict(r=_router(groups=8, top_groups=8, group_best=0)), INV),
    (dict(r=_router(groups=8, top_groups=8, group_best=3)), INV), (dict(r=_router(groups=64, top_groups=8, group_best=2)), INV),
    (dict(r=_router(groups=8, top_groups=2, k=17)), INV), (dict(r=_router(experts=1024, groups=2, top_groups=1)), UNS),
    (dict(r=_router(factor=float("nan"))), INV), (dict(r=_router(factor=float("inf"))), INV), (dict(r=_router(bias=0x100001)), ALN),
    (dict(r=_router(k=65)), UNS), (dict(r=_router(experts=3, k=4)), INV), (dict(T=(1 << 26) + 1), UNS), (dict(T=(1 << 63) - 1), UNS),
    (dict(dtype=0), INV), (dict(dtype=3), INV), (dict(offsets=None), INV), (dict(order=None), INV), (dict(logits=None), INV), (dict(ids=None), INV),
    (dict(weights=None), INV), (dict(ld=63), INV), (dict(ld=(1 << 63) - 1), UNS), (dict(logits=P1), ALN), (dict(logits=P2), ALN), (dict(ids=P2), ALN),
    (dict(weights=P2), ALN), (dict(offsets=P2), ALN), (dict(order=P2), ALN), (dict(ws=P4), ALN), (dict(ws=None), WS), (dict(ws_bytes=0), WS)])
def test_route(change, code):
    assert _call("oq_route", ROUTE, change) == code and b"oq_route" in oq.lib().oq_last_error()


def test_route_workspace():
    need = oq.lib().oq_route_ws_bytes(100, _router())
    assert need > 0 and _call("oq_route", ROUTE, dict(ws_bytes=need - 1)) == WS
    assert oq.lib().oq_route_ws_bytes(-1, _router()) == 0 and oq.lib().oq_route_ws_bytes(100, None) == 0
    assert oq.lib().oq_route_ws_bytes(100, _router(k=0)) == 0
    assert _call("oq_route", ROUTE, dict(T=0, offsets=None, order=None, logits=None, ids=None, weights=None)) == OK


EX = dict(qa=P, lda=1024, a_scale=P, rows=10, K=1024, w=P, ldw=1024, w_stride=64 * 1024, w_scale=P, N=64, E=8, offsets=P, order=P, n=40, per=4,
          act=oq.OQ_ACT_NONE, mean=None, w1=None, bias=None, y=P, ldy=64, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), INV), (dict(n=-1), INV), (dict(N=-1), INV), (dict(E=0), INV), (dict(per=0), INV), (dict(act=2), INV), (dict(act=-1), INV),
    (dict(act=oq.OQ_ACT_SWIGLU, N=63), INV), (dict(K=0), UNS), (dict(K=8), UNS), (dict(K=1000), UNS), (dict(K=131072, lda=131072, ldw=131072), UNS),
    (dict(E=1025), UNS), (dict(N=(1 << 20) + 2), UNS), (dict(mean=P), INV), (dict(w1=P), INV), (dict(n=(1 << 28) + 1, rows=1 << 30), UNS),
    (dict(rows=9), INV), (dict(per=1), INV), (dict(n=(1 << 63) - 1, per=2), UNS), (dict(qa=None), INV), (dict(a_scale=None), INV), (dict(w=None), INV),
    (dict(w_scale=None), INV), (dict(offsets=None), INV), (dict(order=None), INV), (dict(y=None), INV), (dict(lda=1008), INV), (dict(ldw=1008), INV),
    (dict(lda=(1 << 23) + 16), UNS), (dict(ldw=1 << 24, w_stride=1 << 40), UNS), (dict(w_stride=64 * 1024 - 16), INV), (dict(w_stride=-(1 << 40)), INV),
    (dict(w_stride=(1 << 50) + 16), UNS), (dict(ldy=63), INV), (dict(ldy=(1 << 30) + 1), UNS), (dict(qa=P4), ALN), (dict(w=P4), ALN),
    (dict(lda=1032), ALN), (dict(ldw=1032, w_stride=64 * 1032), ALN), (dict(w_stride=64 * 1024 + 8), ALN), (dict(y=P1), ALN), (dict(a_scale=P1), ALN),
    (dict(w_scale=P2), ALN), (dict(mean=P1, w1=P), ALN), (dict(mean=P, w1=P1), ALN), (dict(bias=P2), ALN), (dict(offsets=P2), ALN), (dict(order=P2), ALN)])
def test_experts(change, code):
    assert _call("oq_gemm_w8a8_experts", EX, change) == code and b"oq_gemm_w8a8_experts" in oq.lib().oq_last_error()


@pytest.mark.parametrize("change", [dict(n=0), dict(N=0), dict(n=0, qa=None, y=None, order=None, rows=0)])
def test_experts_empty(change):
    assert _call("oq_gemm_w8a8_experts", EX, change) == OK


def _norm(w=P, b=None, kind=oq.OQ_NORM_RMS, eps=1e-6):
    at = lambda p: None if p is None else p.value  # noqa: E731
    return ctypes.byref(B.oq_norm(at(w), at(b), kind, eps))


def _mod(gate=P, scale=P, shift=P, row=P, ld=256, rows=3):
    at = lambda p: None if p is None else p.value  # noqa: E731
    return ctypes.byref(B.oq_mod(at(gate), at(scale), at(shift), at(row), ld, rows))


RN = dict(y=P, y_ld=256, k=2, weights=P, y_scale=f32(1), r=P, r_ld=256, r_scale=f32(1), r_type=oq.OQ_BF16, T=10, d=256, post=_norm(), pre=_norm(),
          mod=_mod(), r_out=P, ro_ld=256, h=P, h_ld=256, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(r_type=0), INV), (dict(r_type=4), INV), (dict(post=_norm(kind=0)), INV), (dict(pre=_norm(kind=3)), INV), (dict(pre=_norm(eps=-1.0)), INV),
    (dict(post=_norm(eps=float("nan"))), INV), (dict(post=_norm(eps=float("inf"))), INV), (dict(pre=_norm(w=P1)), ALN), (dict(pre=_norm(b=P2)), ALN),
    (dict(T=-1), INV), (dict(k=0), INV), (dict(k=65), UNS), (dict(T=1 << 30), UNS), (dict(d=0), UNS), (dict(d=4), UNS), (dict(d=260), UNS),
    (dict(d=16392), UNS), (dict(weights=None), INV), (dict(y_scale=NAN), INV), (dict(r_scale=INF), INV), (dict(y=None, mod=None), INV),
    (dict(y=None, post=None), INV), (dict(y=None, r=None, post=None, mod=None), INV), (dict(r_out=None, h=None), INV), (dict(y_ld=248), INV),
    (dict(r_ld=-256), INV), (dict(ro_ld=0), INV), (dict(h_ld=8), INV), (dict(y_ld=260), ALN), (dict(r=P4, r_out=P), ALN), (dict(h=P4), ALN),
    (dict(ro_ld=264), INV), (dict(r_type=oq.OQ_F32, r_ld=258, r_out=None), ALN), (dict(weights=P2), ALN), (dict(y_ld=(1 << 63) - 1), UNS),
    (dict(mod=_mod(rows=0)), INV), (dict(mod=_mod(rows=-1)), INV), (dict(mod=_mod(row=None)), INV), (dict(mod=_mod(ld=128)), INV), (dict(mod=_mod(ld=260)), ALN),
    (dict(mod=_mod(gate=P4)), ALN), (dict(mod=_mod(scale=P4)), ALN), (dict(mod=_mod(shift=P4)), ALN), (dict(mod=_mod(row=P2)), ALN)])
def test_residual_norm(change, code):
    assert _call("oq_residual_norm", RN, change) == code and b"oq_residual_norm" in oq.lib().oq_last_error()


def test_residual_norm_empty():
    assert _call("oq_residual_norm", RN, dict(T=0)) == OK
    assert _call("oq_residual_norm", RN, dict(T=0, y=None, r=None, r_out=None, h=None)) == OK


LP = dict(logits=P, dtype=oq.OQ_BF16, ld=1000, T=10, V=1000, scale=f32(1), tokens=P, n=2, top=5, logprob=P, rank=P, entropy=P, lse=P, top_id=P,
          top_logprob=P, ws=P, ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INV), (dict(V=0), INV), (dict(V=-5), INV), (dict(n=-1), INV), (dict(top=-1), INV), (dict(V=(1 << 21) + 1, ld=1 << 23), UNS),
    (dict(n=65), UNS), (dict(top=33), UNS), (dict(V=4, top=5), INV), (dict(T=(1 << 24) + 1), UNS), (dict(T=(1 << 63) - 1), UNS), (dict(dtype=7), INV),
    (dict(scale=f32(0)), INV), (dict(scale=f32(-1)), INV), (dict(scale=NAN), INV), (dict(scale=INF), INV), (dict(scale=f32(3e38)), INV), (dict(ld=999), INV),
    (dict(ld=(1 << 63) - 1), UNS), (dict(logits=None), INV), (dict(tokens=None), INV), (dict(logprob=None), INV), (dict(rank=None), INV),
    (dict(top_id=None), INV), (dict(top_logprob=None), INV), (dict(logits=P1), ALN), (dict(logits=P2, dtype=oq.OQ_F32), ALN), (dict(tokens=P2), ALN),
    (dict(logprob=P2), ALN), (dict(rank=P2), ALN), (dict(entropy=P2), ALN), (dict(lse=P2), ALN), (dict(top_id=P2), ALN), (dict(top_logprob=P2), ALN),
    (dict(ws=P4), ALN), (dict(V=100000, ld=100000, ws=None), WS), (dict(V=100000, ld=100000, ws_bytes=0), WS)])
def test_logprobs(change, code):
    assert _call("oq_logprobs", LP, change) == code and b"oq_logprobs" in oq.lib().oq_last_error()


def test_logprobs_workspace():
    lib = oq.lib()
    need = lib.oq_logprobs_ws_bytes(10, 100000, 2, 5)
    assert need > 0 and _call("oq_logprobs", LP, dict(V=100000, ld=100000, dtype=oq.OQ_F32, ws_bytes=16)) == WS
    for bad in ((-1, 10, 0, 0), (1, 0, 0, 0), (1, 10, 65, 0), (1, 10, 0, 11), (0, 10, 0, 0)):
        assert lib.oq_logprobs_ws_bytes(*bad) == 0
    assert _call("oq_logprobs", LP, dict(T=0, logits=None, tokens=None)) == OK


def test_binding_refuses_host_tensors_and_shapes():
    z = torch.zeros
    r = oq.Router(8, 2)
    i32 = torch.int32
    for bad in (lambda: oq.oq_route(z(4, 8), r), lambda: oq.Router(8, 2, score="relu"), lambda: oq.Router(8, 2, bias=z(8)),
                lambda: oq.Router(8, 1 << 32), lambda: oq.Norm(oq.OQ_NORM_RMS, 8, w=z(8)),
                lambda: oq.oq_gemm_w8a8_experts(z(4, 64, dtype=torch.int8), z(4), z(2, 8, 64, dtype=torch.int8), z(2, 8), z(3, dtype=i32), z(4, dtype=i32)),
                lambda: oq.oq_gemm_w8a8_experts(z(4, 64), z(4), z(2, 8, 64, dtype=torch.int8), z(2, 8), z(3, dtype=i32), z(4, dtype=i32)),
                lambda: oq.oq_residual_norm(z(4, 64, dtype=torch.bfloat16)), lambda: oq.oq_residual_norm(None, None),
                lambda: oq.oq_residual_norm(None, z(4, 64, dtype=torch.bfloat16), weights=z(4, 1)), lambda: oq.oq_logprobs(z(4, 100)),
                lambda: oq.oq_logprobs_ws_bytes(1, 1 << 32, 0, 0)):
        with pytest.raises(oq.OQError):
            bad()
