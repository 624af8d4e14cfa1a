"""Devices and sizes of the sparse layer's entry points in the binding, where no GPU is there (CPU only)."""
import pytest
import torch

import rotated_bit_quantized_amd as oq
from test_binding_cpu import F32, HUGE, I8, I32, U8, gpu

B = oq._binding
BF = torch.bfloat16
TENSORS = {  # entry point: its tensor arguments, as (shape, dtype)
    "oq_route": dict(logits=((4, 8), F32), bias=((8,), F32), mask=((4,), U8), ids=((4, 2), I32), weights=((4, 2), F32), offsets=((9,), I32),
                     order=((8,), I32), ws=((4096,), U8)),
    "oq_gemm_w8a8_experts": dict(qa=((4, 64), I8), a_scale=((4,), F32), w=((3, 8, 64), I8), w_scale=((3, 8), F32), offsets=((4,), I32), order=((8,), I32),
                                 mean=((4,), F32), w1=((3, 8), F32), bias=((3, 8), F32), y=((8, 8), BF)),
    "oq_residual_norm": dict(y=((8, 64), BF), r=((4, 64), F32), weights=((4, 2), F32), post_w=((64,), F32), pre_w=((64,), F32), pre_b=((64,), F32),
                             gate=((3, 64), BF), scale=((3, 64), BF), shift=((3, 64), BF), row=((4,), I32), r_out=((4, 64), F32), h=((4, 64), BF)),
    "oq_logprobs": dict(logits=((4, 100), BF), tokens=((4, 2), I32), logprob=((4, 2), F32), rank=((4, 2), I32), entropy=((4,), F32), lse=((4,), F32),
                        top_id=((4, 3), I32), top_logprob=((4, 3), F32), ws=((4096,), U8)),
}
SCALARS = {"oq_gemm_w8a8_experts": dict(per=2), "oq_logprobs": dict(top=3)}


def _call(entry, where, monkeypatch, change=None):
    reached = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: 4096 if name.endswith("_ws_bytes") else reached.append(name) or 0

    monkeypatch.setattr(B, "_lib", Lib())
    monkeypatch.setattr(B, "_raw_stream", lambda d: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    change = change or {}
    t = {n: gpu(*shape, dtype=dt, where=where.get(n, 0)) for n, (shape, dt) in {**TENSORS[entry], **{k: v for k, v in change.items() if isinstance(v, tuple)}}.items()}
    if entry == "oq_route":
        t["router"] = oq.Router(t["logits"].shape[1], 2, bias=t.pop("bias"))
    if entry == "oq_residual_norm":
        t["post"] = oq.Norm(oq.OQ_NORM_RMS, 64, w=t.pop("post_w"))
        t["pre"] = oq.Norm(oq.OQ_NORM_LAYER, 64, w=t.pop("pre_w"), b=t.pop("pre_b"))
    getattr(oq, entry)(**t, **{**SCALARS.get(entry, {}), **{k: v for k, v in change.items() if not isinstance(v, tuple)}})
    return reached


@pytest.mark.parametrize("entry", TENSORS)
def test_tensors_of_the_current_gpu_reach_the_library(entry, monkeypatch):
    assert _call(entry, {}, monkeypatch) == [entry]


@pytest.mark.parametrize("entry,name", [(e, n) for e, a in TENSORS.items() for n in a])
@pytest.mark.parametrize("where", [1, -1])
def test_every_tensor_has_to_live_on_the_current_gpu(entry, name, where, monkeypatch):
    with pytest.raises(oq.OQError):
        _call(entry, {name: where}, monkeypatch)


@pytest.mark.parametrize("names", [("bias",), ("post_w",), ("pre_w", "pre_b")])
def test_a_whole_handle_of_another_gpu(names, monkeypatch):
    with pytest.raises(oq.OQError):
        _call("oq_route" if names == ("bias",) else "oq_residual_norm", dict.fromkeys(names, 1), monkeypatch)


WRONG = [("oq_route", n, s, d) for n, s, d in [("logits", (4, 8), torch.float16), ("ids", (4, 1), I32), ("ids", (4, 2), torch.int64), ("mask", (3,), U8),
                                               ("mask", (4,), F32), ("offsets", (8,), I32), ("order", (7,), I32)]]
WRONG += [("oq_gemm_w8a8_experts", n, s, d) for n, s, d in [("y", (8, 7), BF), ("y", (7, 8), BF), ("w", (3, 8, 48), I8), ("w", (8, 64), I8), ("a_scale", (3,), F32),
                                                            ("w_scale", (2, 8), F32), ("offsets", (3,), I32), ("mean", (3,), F32), ("bias", (3, 7), F32)]]
WRONG += [("oq_residual_norm", n, s, d) for n, s, d in [("y", (7, 64), BF), ("r", (4, 56), F32), ("r", (4, 64), torch.float16), ("r_out", (4, 64), BF),
                                                        ("h", (4, 64), F32), ("weights", (4, 1), F32), ("weights", (8,), F32), ("gate", (3, 56), BF),
                                                        ("scale", (2, 64), BF), ("shift", (3, 64), F32), ("row", (3,), I32), ("post_w", (56,), F32)]]
WRONG += [("oq_logprobs", n, s, d) for n, s, d in [("logits", (4, 100), torch.float16), ("tokens", (3, 2), I32), ("tokens", (4, 2), torch.int64), ("tokens", (8,), I32),
                                                   ("logprob", (4, 1), F32), ("rank", (4, 2), F32), ("lse", (3,), F32), ("top_id", (4, 2), I32)]]


@pytest.mark.parametrize("entry,name,shape,dtype", WRONG)
def test_wrong_shapes_and_types_are_refused(entry, name, shape, dtype, monkeypatch):
    with pytest.raises(oq.OQError):
        _call(entry, {}, monkeypatch, {name: (shape, dtype)})


@pytest.mark.parametrize("entry,change", [
    ("oq_gemm_w8a8_experts", dict(qa=((4, HUGE), I8), w=((3, 8, HUGE), I8))), ("oq_gemm_w8a8_experts", dict(per=HUGE)),
    ("oq_gemm_w8a8_experts", dict(w=((3, HUGE, 64), I8), w_scale=((3, HUGE), F32), w1=((3, HUGE), F32), bias=((3, HUGE), F32), y=((8, HUGE), BF))),
    ("oq_gemm_w8a8_experts", dict(w=((HUGE, 8, 64), I8), w_scale=((HUGE, 8), F32), w1=((HUGE, 8), F32), bias=((HUGE, 8), F32), offsets=((HUGE + 1,), I32))),
    ("oq_residual_norm", dict(y=((4 * HUGE, 64), BF), weights=((4, HUGE), F32))),
    ("oq_logprobs", dict(logits=((4, HUGE), BF))), ("oq_logprobs", dict(top=HUGE)),
    ("oq_logprobs", dict(tokens=((4, HUGE), I32), logprob=((4, HUGE), F32), rank=((4, HUGE), I32)))])
def test_sizes_past_32_bits_are_refused(entry, change, monkeypatch):
    with pytest.raises(oq.OQError):
        _call(entry, {}, monkeypatch, change)


def test_modulations_of_different_strides_are_refused(monkeypatch):
    monkeypatch.setattr(B, "_raw_stream", lambda d: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    wide = gpu(3, 128, dtype=BF)
    with pytest.raises(oq.OQError):
        oq.oq_residual_norm(gpu(4, 64, dtype=BF), gate=gpu(3, 64, dtype=BF), scale=wide[:, :64], row=gpu(4, dtype=I32))
