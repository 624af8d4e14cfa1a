"""The plan of the experts' products: which kernel a call takes, and that every tile
has a workgroup, in host code built as test_sparse_sanitized.py does (CPU only)."""
import os
import re
import subprocess

import pytest

from test_abi_sanitized import CLANG, CSRC, HERE, HIPCC, _compile

pytestmark = pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)), reason="ROCm compilers not present")


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    tmp = tmp_path_factory.mktemp("expert_plan")
    objs = []
    for d, name in ((CSRC, "abi"), (CSRC, "lm_codebook"), (CSRC, "abi_sparse"), (CSRC, "sparse_plan"), (HERE, "stubs"), (HERE, "sparse_stubs"),
                    (HERE, "expert_plan_driver")):
        objs.append(str(tmp / f"{name}.o"))
        _compile(os.path.join(d, name + ".hip"), objs[-1], name)
    syms = set()
    for obj in objs:
        syms.update(re.findall(r"\b(__hip_fatbin_\w+)", subprocess.run(["nm", "-u", obj], capture_output=True, text=True, check=True).stdout))
    fat = tmp / "fatbin.cpp"
    fat.write_text("".join(f'extern "C" {{ unsigned char {s}[64] = {{0}}; }}\n' for s in sorted(syms)))
    exe = str(tmp / "expert_plan")
    r = subprocess.run([CLANG, "-fsanitize=address,undefined", "-o", exe, *objs, str(fat)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]

    def run(*args):
        env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:halt_on_error=1:verify_asan_link_order=0", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
        r = subprocess.run([exe, *map(str, args)], capture_output=True, text=True, env=env, timeout=120)
        assert r.returncode == 0 and "runtime error" not in r.stderr, (r.stdout[-3000:], r.stderr[-3000:])
        return r.stdout

    return run


def kernels(driver, calls):
    """(mt, ks) of calls (n, K, N, E, act); mt 0: the persistent tiles."""
    lines = driver(*[int(v) for c in calls for v in c]).split("\n")[: len(calls)]
    return [tuple(int(v) for v in line.split()[:2]) for line in lines]


def test_ranges(driver):
    assert "cases passed" in driver()


def test_calls_of_the_tiles_tests_reach_the_tiles(driver):
    """The sizes of test_gpu_experts_tiles.py."""
    calls = [(2300, K, f * N, 4, f - 1) for K in (400, 528, 1040) for N in (1, 34, 130, 255, 256, 257, 513, 1026) for f in (1, 2)]
    calls += [(12000, K, 1540, 9, act) for K in (400, 496, 512, 640, 1008, 1040, 4112) for act in (0, 1)] + [(6000, 432, 1030, 6, 1)]
    calls += [(36 * E, 400, 36, E, 0) for E in (63, 64, 65, 127, 128, 129, 200, 1000, 1023, 1024)]
    calls += [(T * k, 416, N, E, act) for T, E, k, N in ((1, 64, 1, 40000), (1, 128, 8, 5000), (3, 60, 4, 3070), (70, 128, 1, 514), (16, 128, 8, 770), (5, 1000, 2, 4000))
              for act in (0, 1)]
    calls += [(6000, 464, 520, 24, 1), (160, 131056, 16, 4, 0), (12000, 432, 1540, 7, 1), (6000, 400, 1032, 4, 0), (800, 528, 1100, 8, 1), (18000, 528, 1100, 8, 1), (5000, 656, 3333, 1, 0),
              (10000, 464, 1540, 8, 1), (2000, 7168, 4096, 160, 0), (24, 7168, 4096, 160, 0)]
    got = kernels(driver, calls)
    wrong = [c for c, kernel in zip(calls, got) if kernel[0] != 0]
    assert not wrong


def test_the_other_kernels_are_reached(driver):
    """Few entries with k over 8, 4, 2 and 1 wavefronts; short rows, few and many."""
    assert kernels(driver, [(4, 1408, 2048, 60, 0), (8, 2048, 1536, 128, 1), (16, 1408, 2048, 60, 0), (12, 528, 1100, 8, 1)]) == [(1, 8), (1, 4), (1, 2), (1, 8)]
    assert kernels(driver, [(1024, 384, 4096, 128, 0), (100000, 384, 1024, 64, 1), (16 * 1024, 16, 1 << 20, 1024, 1), (65 * 1024, 16, 1 << 20, 1024, 1)]) == [
        (1, 1), (4, 1), (1, 1), (4, 1)]
