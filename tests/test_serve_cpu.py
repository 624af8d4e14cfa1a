"""Refusals of the serving operators: nothing is launched, every bad argument
has its code (CPU only)."""
import ctypes

import pytest

import rotated_bit_quantized_amd as oq

B = oq._binding
P = ctypes.c_void_p(0x100000)  # never dereferenced: validation fails first
P4, P1 = ctypes.c_void_p(0x100004), ctypes.c_void_p(0x100001)
INV, UNS, ALN, WS = oq.OQ_ERR_INVALID_ARG, oq.OQ_ERR_UNSUPPORTED, oq.OQ_ERR_ALIGNMENT, oq.OQ_ERR_WORKSPACE


def _call(fn, args, change):
    names = list(args)
    assert set(change) <= set(names)
    return getattr(oq.lib(), fn)(*[change.get(n, args[n]) for n in names])


GEMM = dict(qa=P, lda=1024, a_scale=P, M=4, K=1024, w=P, ldw=1024, w_scale=P, N=64, mean=None, w1=None, bias=None, y=P, ldy=64,
            stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(M=-1), INV), (dict(N=-1), INV), (dict(K=0), UNS), (dict(K=1000), UNS), (dict(K=131072, lda=131072, ldw=131072), UNS),
    (dict(K=-16), UNS), (dict(mean=P), INV), (dict(w1=P), INV), (dict(qa=None), INV), (dict(a_scale=None), INV), (dict(w=None), INV),
    (dict(w_scale=None), INV), (dict(y=None), INV), (dict(lda=1008), INV), (dict(ldw=1008), INV), (dict(ldy=63), INV),
    (dict(lda=1032), ALN), (dict(ldw=1032), ALN), (dict(qa=P4), ALN), (dict(w=P4), ALN), (dict(y=P1), ALN), (dict(a_scale=P1), ALN),
    (dict(bias=P1), ALN), (dict(M=(1 << 30) + 1), UNS),
    (dict(lda=(1 << 23) + 16), UNS), (dict(ldw=1 << 24), UNS)])
def test_gemm_w8a8(change, code):
    assert _call("oq_gemm_w8a8", GEMM, change) == code and b"oq_gemm_w8a8" in oq.lib().oq_last_error()


@pytest.mark.parametrize("change", [dict(M=0), dict(N=0), dict(M=0, qa=None, y=None)])
def test_gemm_w8a8_empty(change):
    assert _call("oq_gemm_w8a8", GEMM, change) == oq._binding.OQ_OK


QW = dict(w=P, N=4, K=1024, ldw=1024, rot=None, codes=P, ldc=1024, scales=P, w1=None, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(N=-1), INV), (dict(K=8), UNS), (dict(K=1000), UNS), (dict(K=16400, ldw=16400), UNS), (dict(ldw=1020), INV), (dict(w=None), INV),
    (dict(codes=None), INV), (dict(scales=None), INV), (dict(w=P4), ALN), (dict(ldw=1026), ALN), (dict(ldc=1030), ALN), (dict(ldc=1008), INV),
    (dict(rot=ctypes.byref(B.oq_rot(oq.OQ_ROT_DENSE32, 1024, 32, 1, P, P, P))), INV),
    (dict(rot=ctypes.byref(B.oq_rot(oq.OQ_ROT_RPBH, 1024, 96, 1, P, P, None))), UNS)])
def test_quant_weight_w8(change, code):
    assert _call("oq_quant_weight_w8", QW, change) == code


def _rope(cos=P, sin=P, rows=100, dim=128, inter=0):
    return ctypes.byref(B.oq_rope(cos, sin, rows, dim, inter))


QK = dict(q=P, q_ld=4096, q_hs=128, heads_q=32, k=P, k_ld=1024, k_hs=128, heads_k=8, T=10, d=128, w_q=P, w_k=P,
          eps=ctypes.c_float(1e-6), rope=_rope(), pos=P, q_out=P, qo_ld=4096, qo_hs=128, k_out=P, ko_ld=1024, ko_hs=128, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INV), (dict(T=1 << 31), UNS), (dict(heads_q=-1), INV), (dict(heads_k=65536), UNS), (dict(d=4), UNS), (dict(d=100), UNS),
    (dict(d=520), UNS), (dict(eps=ctypes.c_float(-1.0)), INV), (dict(eps=ctypes.c_float(float("nan"))), INV),
    (dict(eps=ctypes.c_float(float("inf"))), INV), (dict(rope=_rope(cos=None)), INV), (dict(rope=_rope(sin=None)), INV),
    (dict(rope=_rope(cos=P1)), ALN), (dict(rope=_rope(dim=127)), INV), (dict(rope=_rope(dim=0)), INV), (dict(rope=_rope(dim=130)), INV),
    (dict(rope=_rope(rows=0)), INV), (dict(rope=_rope(rows=9), pos=None), INV), (dict(pos=P1), ALN), (dict(q=None), INV), (dict(k=None), INV),
    (dict(q_out=None), INV), (dict(k_out=None), INV), (dict(q=P4), ALN), (dict(q_ld=4100), ALN), (dict(k_hs=132), ALN), (dict(q_hs=-128), INV),
    (dict(q_hs=120), INV), (dict(ko_ld=120), INV), (dict(k_out=P4), ALN), (dict(w_q=P1), ALN)])
def test_qk_norm_rope(change, code):
    assert _call("oq_qk_norm_rope", QK, change) == code


def _kv(k=P, v=P, stride=8 * 16 * 128, pages=4, page=16, heads=8, d=128):
    return ctypes.byref(B.oq_kv(k, v, stride, pages, page, heads, d))


AP = dict(k=P, k_ld=1024, k_hs=128, v=P, v_ld=1024, v_hs=128, T=10, w_k=P, eps=ctypes.c_float(1e-6), rope=_rope(), pos=P, slot=P, kv=_kv(),
          stream=None)
KV_BAD = [(dict(kv=None), INV), (dict(kv=_kv(pages=-1)), INV), (dict(kv=_kv(heads=0)), INV), (dict(kv=_kv(page=12)), UNS),
          (dict(kv=_kv(page=4)), UNS), (dict(kv=_kv(page=2048, stride=1 << 30)), UNS), (dict(kv=_kv(stride=16000)), INV), (dict(kv=_kv(k=None)), INV),
          (dict(kv=_kv(v=None)), INV), (dict(kv=_kv(k=P4)), ALN), (dict(kv=_kv(stride=8 * 16 * 128 + 4)), ALN)]


@pytest.mark.parametrize("change,code", KV_BAD + [
    (dict(T=-1), INV), (dict(kv=_kv(d=132, stride=1 << 20)), UNS), (dict(kv=_kv(d=520, stride=1 << 20)), UNS), (dict(slot=None), INV),
    (dict(slot=P4), ALN), (dict(k=None), INV), (dict(v=None), INV), (dict(v_hs=64), INV), (dict(k_ld=1020), ALN), (dict(rope=_rope(dim=200)), INV),
    (dict(eps=ctypes.c_float(-1.0)), INV)])
def test_kv_append(change, code):
    assert _call("oq_kv_append", AP, change) == code


AT = dict(q=P, q_ld=4096, q_hs=128, B=4, n_q=1, heads_q=32, kv=_kv(), prefix_table=P, prefix_len=60, tables=P, table_ld=2, lens=P,
          scale=ctypes.c_float(0.1), o=P, o_ld=4096, o_hs=128, lse=None, ws=P, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("change,code", KV_BAD + [
    (dict(kv=_kv(d=96)), UNS), (dict(B=-1), INV), (dict(n_q=0), INV), (dict(heads_q=0), INV), (dict(heads_q=30), INV), (dict(prefix_len=-1), INV),
    (dict(table_ld=-1), INV), (dict(table_ld=1 << 27), UNS), (dict(prefix_len=(1 << 31) - 1), UNS), (dict(B=1 << 20, n_q=1 << 10), UNS),
    (dict(scale=ctypes.c_float(float("nan"))), INV), (dict(scale=ctypes.c_float(float("inf"))), INV), (dict(q=None), INV), (dict(o=None), INV),
    (dict(q_ld=4100), ALN), (dict(o=P4), ALN), (dict(prefix_table=None), INV), (dict(tables=None), INV), (dict(lens=None), INV),
    (dict(tables=P1), ALN), (dict(lse=P1), ALN), (dict(ws=P4), ALN)])
def test_attn_prefix(change, code):
    assert _call("oq_attn_prefix", AT, change) == code


def test_attn_prefix_workspace_query():
    lib = oq.lib()
    assert lib.oq_attn_prefix_ws_bytes(4, 1, 32, None, 60, 2) == 0
    assert lib.oq_attn_prefix_ws_bytes(4, 1, 30, _kv(), 60, 2) == 0
    assert lib.oq_attn_prefix_ws_bytes(0, 1, 32, _kv(), 60, 2) == 0


def test_binding_refuses_host_tensors_and_shapes():
    import torch

    z = torch.zeros
    with pytest.raises(oq.OQError):
        oq.oq_gemm_w8a8(z(4, 64, dtype=torch.int8), z(4), z(8, 64, dtype=torch.int8), z(8))
    with pytest.raises(oq.OQError):
        oq.oq_gemm_w8a8(z(4, 64), z(4), z(8, 64, dtype=torch.int8), z(8))
    with pytest.raises(oq.OQError):
        oq.oq_quant_weight_w8(z(4, 64))
    with pytest.raises(oq.OQError):
        oq.oq_qk_norm_rope(z(4, 2, 64, dtype=torch.bfloat16), None)
    with pytest.raises(oq.OQError):
        oq.oq_qk_norm_rope(None, None)
    with pytest.raises(oq.OQError):
        oq.Rope(z(4, 32), z(4, 32))
    with pytest.raises(oq.OQError):
        oq.PagedKV(z(4, 2, 16, 64, dtype=torch.bfloat16), z(4, 2, 16, 64, dtype=torch.bfloat16))
