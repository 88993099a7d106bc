"""The layer operators' host code (csrc/layer_api.hip) under AddressSanitizer and UndefinedBehaviorSanitizer (CPU
only), rebuilt with the sanitizers on the host pass and driven down its refusals by tests/abi_layer_driver.c."""
import os
import shutil
import subprocess

import pytest

from moe_grouped_gemm_sizes_amd import build as B

HERE = os.path.dirname(os.path.abspath(__file__))
OBJ = os.path.join(os.path.dirname(B.CSRC), "_build")


@pytest.mark.timeout(300)
def test_layer_api_host_code_under_asan_and_ubsan(tmp_path):
    objs = [os.path.join(OBJ, o) for o in ("route.o", "permute.o", "checkpoint.o")]
    if not all(os.path.exists(o) for o in objs):
        B.build(verbose=False)
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=undefined", "-Xarch_host", "-fno-omit-frame-pointer"]
    api_o, drv_o, exe = (str(tmp_path / n) for n in ("layer_api_san.o", "driver.o", "driver"))
    cc = shutil.which("gcc") or "cc"
    for cmd in ([B.hipcc(), *B.HIPFLAGS, *san, "-c", os.path.join(B.CSRC, "layer_api.hip"), "-o", api_o],
                [cc, "-std=c99", "-O1", "-g", "-Wall", "-c", os.path.join(HERE, "abi_layer_driver.c"), "-o", drv_o],
                [B.hipcc(), f"--offload-arch={B.ARCH}", *san, drv_o, api_o, *objs, "-o", exe]):
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", (r.stdout[-2000:], r.stderr[-3000:])
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr[-3000:]
