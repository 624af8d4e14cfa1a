"""The binding where no GPU is there (CPU only)."""
import os
import subprocess
import sys

import pytest
import torch

import rotated_bit_quantized_amd as oq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_import_without_the_raw_stream_symbol():
    """A torch without GPU support lacks it; the library's host functions need no stream."""
    code = ("import torch\n"
            "if hasattr(torch._C, '_cuda_getCurrentRawStream'):\n"
            "    del torch._C._cuda_getCurrentRawStream\n"
            "import rotated_bit_quantized_amd as oq\n"
            "assert oq.oq_kron_plan(1920)[2] >= 1920\n"
            "torch.cuda.current_device = lambda: 3\n"
            "torch.cuda.current_stream = lambda d=None: type('S', (), dict(cuda_stream=70 + d))\n"
            "assert oq._binding._stream() == 73\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


class OnGpu(torch.Tensor):
    """A tensor without memory that says it lives on GPU `where`."""

    where = 0
    is_cuda = property(lambda self: self.where >= 0)

    def get_device(self):
        return self.where


def gpu(*shape, dtype=torch.bfloat16, where=0):
    t = torch.empty(*shape, dtype=dtype, device="meta").as_subclass(OnGpu)
    t.where = where
    return t


I8, I32, I64, F32, U8 = torch.int8, torch.int32, torch.int64, torch.float32, torch.uint8
TENSORS = {  # entry point: its tensor arguments, as (shape, dtype)
    "oq_quant_weight_w8": dict(w=((8, 64), F32), codes=((8, 64), I8), scales=((8,), F32), w1=((8,), F32)),
    "oq_gemm_w8a8": dict(qa=((4, 64), I8), a_scale=((4,), F32), w=((8, 64), I8), w_scale=((8,), F32), mean=((4,), F32), w1=((8,), F32),
                         bias=((8,), F32), y=((4, 8), torch.bfloat16)),
    "oq_qk_norm_rope": dict(q=((4, 2, 64),), k=((4, 1, 64),), w_q=((64,), F32), w_k=((64,), F32), cos=((9, 32), F32), sin=((9, 32), F32),
                            pos=((4,), I32), q_out=((4, 2, 64),), k_out=((4, 1, 64),)),
    "oq_kv_append": dict(k=((4, 1, 64),), v=((4, 1, 64),), slot=((4,), I64), k_cache=((5, 1, 16, 64),), v_cache=((5, 1, 16, 64),),
                         w_k=((64,), F32), cos=((9, 32), F32), sin=((9, 32), F32), pos=((4,), I32)),
    "oq_attn_prefix": dict(q=((4, 2, 64),), k_cache=((5, 1, 16, 64),), v_cache=((5, 1, 16, 64),), prefix_table=((2,), I32),
                           tables=((4, 1), I32), lens=((4,), I32), o=((4, 2, 64),), lse=((4, 2), F32), ws=((1 << 20,), U8)),
}

SCALARS = {"oq_attn_prefix": dict(n_q=1, prefix_len=20, scale=0.1)}


def _call(entry, where, monkeypatch):
    """Calls `entry` with the named arguments on GPU 1 (a host tensor: -1), all others on GPU 0; how often the library was reached."""
    reached = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: 4096 if name.endswith("_ws_bytes") else reached.append(name) or 0

    B = oq._binding
    monkeypatch.setattr(B, "_lib", Lib())
    monkeypatch.setattr(B, "_raw_stream", lambda d: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    t = {n: gpu(*s, where=where.get(n, 0)) if not dt else gpu(*s, dtype=dt[0], where=where.get(n, 0)) for n, (s, *dt) in TENSORS[entry].items()}
    if "cos" in t:
        t["rope"] = oq.Rope(t.pop("cos"), t.pop("sin"))
    if "k_cache" in t:
        t["kv"] = oq.PagedKV(t.pop("k_cache"), t.pop("v_cache"))
    getattr(oq, entry)(**t, **SCALARS.get(entry, {}))
    return reached


@pytest.mark.parametrize("entry", TENSORS)
def test_tensors_of_the_current_gpu_reach_the_library(entry, monkeypatch):
    assert _call(entry, {}, monkeypatch) == [entry]


@pytest.mark.parametrize("entry,name", [(e, n) for e, a in TENSORS.items() for n in a])
@pytest.mark.parametrize("where", [1, -1])
def test_every_tensor_has_to_live_on_the_current_gpu(entry, name, where, monkeypatch):
    """An address of another GPU or of the host would be read by the wrong device."""
    with pytest.raises(oq.OQError):
        _call(entry, {name: where}, monkeypatch)


@pytest.mark.parametrize("entry,pair", [("oq_qk_norm_rope", ("cos", "sin")), ("oq_kv_append", ("cos", "sin")), ("oq_kv_append", ("k_cache", "v_cache")),
                                        ("oq_attn_prefix", ("k_cache", "v_cache"))])
def test_a_whole_handle_of_another_gpu(entry, pair, monkeypatch):
    with pytest.raises(oq.OQError):
        _call(entry, dict.fromkeys(pair, 1), monkeypatch)


HUGE = (1 << 32) + 64  # 64 in 32 bits
LARGE = {
    "oq_quant_weight_w8": [dict(w=((1, HUGE), F32), codes=((1, HUGE), I8)), dict(w=((HUGE, 64), F32), codes=((HUGE, 64), I8), scales=((HUGE,), F32), w1=((HUGE,), F32))],
    "oq_gemm_w8a8": [dict(qa=((4, HUGE), I8), w=((8, HUGE), I8)),
                     dict(w=((HUGE, 64), I8), w_scale=((HUGE,), F32), w1=((HUGE,), F32), bias=((HUGE,), F32), y=((4, HUGE), torch.bfloat16))],
    "oq_qk_norm_rope": [dict(q=((4, HUGE, 64),), q_out=((4, HUGE, 64),)), dict(k=((4, HUGE, 64),), k_out=((4, HUGE, 64),)),
                        {n: (s[:-1] + (HUGE,),) for n, s in dict(q=(4, 2, 0), k=(4, 1, 0), q_out=(4, 2, 0), k_out=(4, 1, 0)).items()}
                        | dict(w_q=((HUGE,), F32), w_k=((HUGE,), F32))],
    "oq_kv_append": [dict(k=((4, HUGE, 64),), v=((4, HUGE, 64),), k_cache=((5, HUGE, 16, 64),), v_cache=((5, HUGE, 16, 64),)),
                     dict(k_cache=((HUGE, 1, 16, 64),), v_cache=((HUGE, 1, 16, 64),)), dict(cos=((9, HUGE // 2), F32), sin=((9, HUGE // 2), F32))],
    "oq_attn_prefix": [dict(prefix_len=HUGE, prefix_table=((HUGE // 16,), I32)), dict(tables=((4, HUGE), I32)),
                       dict(q=((4, HUGE, 64),), o=((4, HUGE, 64),), lse=((4, HUGE), F32)), dict(n_q=HUGE, q=((HUGE, 2, 64),), o=((HUGE, 2, 64),), tables=((1, 1), I32), lens=((1,), I32), lse=((HUGE, 2), F32)),
                       dict(q=((HUGE, 2, 64),), o=((HUGE, 2, 64),), tables=((HUGE, 1), I32), lens=((HUGE,), I32), lse=((HUGE, 2), F32))],
}


@pytest.mark.parametrize("entry,n", [(e, n) for e, a in LARGE.items() for n in range(len(a))])
def test_sizes_past_32_bits_are_refused(entry, n, monkeypatch):
    """The library's sizes are 32 bits: what they cannot hold must not arrive as its remainder."""
    change = dict(LARGE[entry][n])
    scalars = {k: change.pop(k) for k in list(change) if not isinstance(change[k], tuple)}
    monkeypatch.setitem(TENSORS, entry, {**TENSORS[entry], **change})
    monkeypatch.setitem(SCALARS, entry, {**SCALARS.get(entry, {}), **scalars})
    with pytest.raises(oq.OQError):
        _call(entry, {}, monkeypatch)


@pytest.mark.parametrize("at", range(5))
def test_workspace_sizes_past_32_bits_are_refused(at, monkeypatch):
    args = [4, 1, 32, 60, 2]
    args[at] = HUGE
    kv = oq.PagedKV(gpu(5, 1, 16, 64), gpu(5, 1, 16, 64))
    with pytest.raises(oq.OQError):
        oq.oq_attn_prefix_ws_bytes(*args[:3], kv, *args[3:])


def test_keys_of_another_rank_are_refused(monkeypatch):
    monkeypatch.setitem(TENSORS, "oq_qk_norm_rope", {**TENSORS["oq_qk_norm_rope"], "k": ((64,),)})
    with pytest.raises(oq.OQError):
        _call("oq_qk_norm_rope", {}, monkeypatch)
