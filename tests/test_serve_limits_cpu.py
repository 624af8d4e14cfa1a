"""Refusals of the serving operators at the ends of their argument ranges (CPU only)."""
import ctypes

import pytest

import rotated_bit_quantized_amd as oq
from test_serve_cpu import AT, INV, QK, UNS, WS, _call, _kv


@pytest.mark.parametrize("B,n_q,heads_q", [(1 << 22, 1 << 21, 1 << 21), (1 << 30, 1 << 30, 8), ((1 << 31) - 1, (1 << 31) - 1, (1 << 31) - 8),
                                           (1 << 16, 1 << 16, 1 << 30), (1, 1, (1 << 30) + 8)])
def test_attn_prefix_row_counts_past_64_bits(B, n_q, heads_q):
    """Products of the three counts that pass 2^30, 2^63 and come back as small numbers modulo 2^64."""
    assert _call("oq_attn_prefix", AT, dict(B=B, n_q=n_q, heads_q=heads_q)) == UNS
    assert oq.lib().oq_attn_prefix_ws_bytes(B, n_q, heads_q, _kv(), 60, 2) == 0


@pytest.mark.parametrize("scale", [2.4e38, -3.4e38])
def test_attn_prefix_scale_past_float32(scale):
    """scale log2(e), by which the kernels multiply, is not finite: a score of 0 would become NaN."""
    assert _call("oq_attn_prefix", AT, dict(scale=ctypes.c_float(scale))) == INV


OVERLAPS = [  # token stride, head stride of 10 tokens and several heads of 128
    (128, 128), (1024, 512), (256, 1280), (1288, 640), (4096, 4096),
]


@pytest.mark.parametrize("ld,hs", OVERLAPS)
def test_outputs_that_overlap_are_refused(ld, hs):
    """Heads of different tokens on the same places: which one stays would be a matter of time."""
    assert _call("oq_qk_norm_rope", QK, dict(qo_ld=ld, qo_hs=hs)) == INV
    assert _call("oq_qk_norm_rope", QK, dict(ko_ld=ld, ko_hs=hs)) == INV
    assert _call("oq_attn_prefix", AT, dict(B=10, o_ld=ld, o_hs=hs)) == INV


@pytest.mark.parametrize("short", ["none", "empty", "one byte"])
def test_attn_prefix_workspace_too_small(short):
    need = oq.lib().oq_attn_prefix_ws_bytes(4, 1, 32, _kv(), 60, 2)
    assert need > 0
    change = dict(ws=None) if short == "none" else dict(ws_bytes=0 if short == "empty" else need - 1)
    assert _call("oq_attn_prefix", AT, change) == WS
