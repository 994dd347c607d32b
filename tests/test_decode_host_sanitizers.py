"""The host code of the entry points of decoding under AddressSanitizer and
UndefinedBehaviorSanitizer (no GPU needed): its sources are compiled with both
sanitizers on the host pass only and linked into tests/decode_host_check.cpp,
with the library as it is built for the rest.
"""

import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

from int8_quantized_matmul_amd import _native, build
from test_host_sanitizers import ROOT, SANITIZE

SOURCES = ["decode_api.cpp", "cache_kernels.hip", "attend_kernels.hip", "select_kernels.hip"]


def test_decoding_entry_points_under_host_sanitizers(tmp_path):
    if not os.path.exists(_native.LIB_PATH):
        build.build()
    hipcc = build._hipcc()
    flags = [*build.HIP_FLAGS, "-g", *SANITIZE]

    def compile_one(path):
        obj = str(tmp_path / (os.path.basename(path) + ".o"))
        res = subprocess.run([hipcc, *flags, "-x", "hip", "-c", path, "-o", obj], capture_output=True, text=True)
        assert res.returncode == 0, res.stdout + res.stderr
        return obj

    paths = [os.path.join(build.CSRC, s) for s in SOURCES] + [os.path.join(ROOT, "tests", "decode_host_check.cpp")]
    with ThreadPoolExecutor(max_workers=len(paths)) as ex:
        objs = list(ex.map(compile_one, paths))
    exe = str(tmp_path / "decode_host_check")
    res = subprocess.run([hipcc, "--offload-arch=gfx950", *SANITIZE, *objs, build.LIB_PATH,
                          f"-Wl,-rpath,{build.LIB_DIR}", "-o", exe], capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:halt_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    res = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    out = res.stdout + res.stderr
    assert res.returncode == 0, out[-4000:]
    assert "0 failed" in res.stdout, out[-4000:]
    assert "runtime error" not in out and "AddressSanitizer" not in out, out[-4000:]
