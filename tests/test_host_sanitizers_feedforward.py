"""The feed-forward calls' host code under AddressSanitizer and
UndefinedBehaviorSanitizer, driven by tests/ffn_host_driver.cpp: the sources
are compiled with the sanitizers on their host half only (the device code is
built as usual and never runs here)."""

import glob
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from tests.test_host_sanitizers import CSRC, INCLUDE, ROCM, ROOT, SAN, _hipcc

pytestmark = pytest.mark.slow


def test_feedforward_host_code_is_clean(tmp_path):
    hipcc = _hipcc()
    objs, cmds = [], []
    for src in sorted(glob.glob(os.path.join(CSRC, "*.hip"))):
        obj = str(tmp_path / (os.path.basename(src)[:-4] + ".o"))
        objs.append(obj)
        cmds.append([hipcc, "--offload-arch=gfx950", "-O3", "-g", "-std=c++17", "-fPIC", *SAN,
                     "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", f"-I{INCLUDE}", f"-I{CSRC}",
                     "-c", src, "-o", obj])
    with ThreadPoolExecutor(8) as ex:
        for r in ex.map(lambda c: subprocess.run(c, capture_output=True, text=True), cmds):
            assert r.returncode == 0, r.stderr[-3000:]
    clang = os.path.join(ROCM, "llvm", "bin", "clang++")
    exe = str(tmp_path / "ffn_host_driver")
    r = subprocess.run([clang, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                        "-D__HIP_PLATFORM_AMD__", f"-I{INCLUDE}", f"-I{os.path.join(ROCM, 'include')}",
                        os.path.join(ROOT, "tests", "ffn_host_driver.cpp"), *objs,
                        f"-L{os.path.join(ROCM, 'lib')}", "-lamdhip64", f"-Wl,-rpath,{os.path.join(ROCM, 'lib')}",
                        "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    env.pop("LD_PRELOAD", None)
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=600)
    assert r.returncode == 0 and "host driver ok" in r.stdout, (r.returncode, r.stdout[-2000:], r.stderr[-4000:])
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr[-4000:]
