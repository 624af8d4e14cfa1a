"""The sparse layer's entry points: argument validation, dispatch and plans,
built for the host alone under AddressSanitizer and UndefinedBehaviorSanitizer
and run on the CPU, as test_abi_sanitized.py does for the others.

abi_sparse.hip and sparse_plan.hip are compiled with --cuda-host-only beside
abi.hip; the launchers are replaced by the recording stand-ins of
tests/host_abi/sparse_stubs.hip, and tests/host_abi/sparse_driver.hip makes the
calls; any sanitizer report aborts the run."""
import os
import re
import subprocess

import pytest

from test_abi_sanitized import CLANG, CSRC, HERE, HIPCC, _compile


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)), reason="ROCm compilers not present")
def test_sparse_validation_under_sanitizers(tmp_path):
    objs = []
    for d, name in ((CSRC, "abi"), (CSRC, "lm_codebook"), (CSRC, "abi_sparse"), (CSRC, "sparse_plan"), (HERE, "stubs"),
                    (HERE, "sparse_stubs"), (HERE, "sparse_driver")):
        objs.append(str(tmp_path / f"{name}.o"))
        _compile(os.path.join(d, name + ".hip"), objs[-1], name)
    # stand-ins for the device images that host-only objects name, never read
    syms = set()
    for obj in objs:
        syms.update(re.findall(r"\b(__hip_fatbin_\w+)", subprocess.run(["nm", "-u", obj], capture_output=True, text=True, check=True).stdout))
    fat = tmp_path / "fatbin.cpp"
    fat.write_text("".join(f'extern "C" {{ unsigned char {s}[64] = {{0}}; }}\n' for s in sorted(syms)))
    exe = str(tmp_path / "sparse_check")
    r = subprocess.run([CLANG, "-fsanitize=address,undefined", "-o", exe, *objs, str(fat)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    # verify_asan_link_order=0: the environment may preload a library of its own
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:halt_on_error=1:verify_asan_link_order=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
    print(r.stdout[-2000:])
    assert r.returncode == 0, (r.stdout[-3000:], r.stderr[-3000:])
    assert "cases passed" in r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr[-3000:]
