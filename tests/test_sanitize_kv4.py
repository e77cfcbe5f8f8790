"""The host side of the 4-bit cache's calls and of the append with rotation (argument checks, workspace sizes)
under AddressSanitizer and UndefinedBehaviorSanitizer: their HIP sources with only the
host passes instrumented, the packer (which holds the error state) and
tests/sanitize/kv4_driver.cpp; no launch is reached, so it runs without a GPU."""
import os
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "memory_bound_decode_amd", "csrc")
HIPCC = "/opt/rocm/bin/hipcc"
CLANG = "/opt/rocm/llvm/bin/clang++"


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)), reason="ROCm compilers not available")
def test_kv4_host_code_under_asan_ubsan():
    san = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all"]
    host_san = [x for f in san for x in ("-Xarch_host", f)]
    inc = ["-I", os.path.join(ROOT, "include"), "-I", CSRC]
    with tempfile.TemporaryDirectory() as td:
        cmds, objs = [], []
        for src in ("kv.hip", "kv_attn.hip"):
            objs.append(os.path.join(td, src + ".o"))
            cmds.append([HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-Xclang", "-target-feature", "-Xclang",
                         "-packed-fp32-ops", *host_san, *inc, "-c", os.path.join(CSRC, src), "-o", objs[-1]])
        for src in (os.path.join(CSRC, "packer.cpp"), os.path.join(ROOT, "tests", "sanitize", "kv4_driver.cpp")):
            objs.append(os.path.join(td, os.path.basename(src) + ".o"))
            cmds.append([CLANG, "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", *san, *inc, "-c", src, "-o", objs[-1]])
        with ThreadPoolExecutor(max_workers=4) as ex:
            for c, r in zip(cmds, ex.map(lambda c: subprocess.run(c, capture_output=True, text=True), cmds)):
                assert r.returncode == 0, (" ".join(c[-3:]), r.stderr[-3000:])
        exe = os.path.join(td, "kv4_driver")
        r = subprocess.run([HIPCC, *san, "-o", exe, *objs, "-lpthread"], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-3000:]
        env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
        env.pop("LD_PRELOAD", None)
        r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
        assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
        assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr[-4000:]
        assert r.stdout.strip() == "ok"
