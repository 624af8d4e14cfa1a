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
    """A host tensor that says it lives on GPU `where`."""

    where = 0
    is_cuda = property(lambda self: self.where >= 0)

    def get_device(self):
        return self.where


def gpu(*shape, dtype=torch.bfloat16, where=0):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)
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
    if entry == "oq_attn_prefix":
        t.update(n_q=1, prefix_len=20, scale=0.1)
    getattr(oq, entry)(**t)
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
