"""The binding where no GPU is there (CPU only)."""
import os
import subprocess
import sys

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
