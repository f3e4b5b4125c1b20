"""Host code of the branching operators' entry points (branch_api.hip) under AddressSanitizer
and UBSan, driven by tests/sanitize/branch_driver.cpp without touching a device.  The
kernels' objects are the library's own, built without sanitizers."""
import os
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "clebsch_gordan_tensor_node_amd", "csrc")
BUILD = os.path.join(ROOT, "_build")
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
CLANG = "/opt/rocm/llvm/bin/clang++"


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)), reason="ROCm toolchain not found")
def test_branching_entry_points_under_asan_ubsan(tmp_path):
    built = [os.path.join(BUILD, n) for n in ["kernels_graph.o", "kernels_bwd.o", "kernels_norm.o", "kernels_optim.o", "train_api.o", "kernels_group.o",
                                                "kernels_route.o"] +
             [f"kernels_conv_c{c}.o" for c in range(9)]]
    if not all(os.path.exists(o) for o in built):
        pytest.skip("library objects not built (python -m clebsch_gordan_tensor_node_amd.build)")
    san = ["-fsanitize=address,undefined", "-fno-sanitize-recover=undefined", "-fno-omit-frame-pointer"]

    def compile_host(src):
        # host pass instrumented, device pass untouched: each sanitizer flag behind -Xarch_host
        out = str(tmp_path / (os.path.basename(src) + ".o"))
        if src.endswith(".cpp"):
            cmd = [CLANG, "-std=c++17", "-O1", "-g", *san, "-c", src, "-o", out]
        else:
            cmd = [HIPCC, "-std=c++17", "-O1", "-g", "--offload-arch=gfx950", "-fPIC", "-Xclang", "-target-feature",
                   "-Xclang", "-packed-fp32-ops",
                   "-Xarch_host", "-fsanitize=address,undefined",
                   "-Xarch_host", "-fno-sanitize-recover=undefined",
                   "-Xarch_host", "-fno-omit-frame-pointer",
                   "-c", src, "-o", out]
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-3000:]
        return out

    srcs = [os.path.join(CSRC, n) for n in ("cgtp_api.hip", "branch_api.hip")]
    srcs.append(os.path.join(ROOT, "tests", "sanitize", "branch_driver.cpp"))
    with ThreadPoolExecutor(max_workers=4) as ex:
        objs = list(ex.map(compile_host, srcs))
    exe = str(tmp_path / "branch_driver")
    r = subprocess.run([CLANG, *san, *objs, *built, "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib",
                        "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, (r.stdout[-2000:], r.stderr[-4000:])
    assert "all checks passed" in r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr[-4000:]
