"""The host-side validation of quantisation, products and routing under
AddressSanitizer and UndefinedBehaviorSanitizer: lh_api.hip rebuilt with
host-only sanitizers (-Xarch_host, so no GPU code is instrumented), linked with
the library's other objects, and the boundary tests of these entry points run
against it in a child process.  None of their calls reaches a kernel launch,
so this needs no GPU."""
import os
import shutil
import subprocess
import sys
import tempfile

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_host_sanitize import HIPCC, OTHERS, PKG, ROOT, _asan_runtime  # noqa: E402

TESTS = ["test_boundary_products.py", "test_boundary_routing.py", "test_boundary_empty.py", "test_boundary_tiles.py",
         "test_boundary_extremes.py"]


@pytest.mark.skipif(not os.path.exists(HIPCC) or _asan_runtime() is None, reason="hipcc or its ASan runtime missing")
def test_operators_validation_is_clean_under_sanitizers():
    objs = [os.path.join(PKG, "_build", o) for o in OTHERS]
    if not all(os.path.exists(o) for o in objs):
        pytest.skip("library objects not built (run __graft_entry__.build())")
    with tempfile.TemporaryDirectory() as d:
        api_o = os.path.join(d, "lh_api.o")
        flags = ["--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-ffp-contract=off",
                 "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
                 "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
                 "-Xarch_host", "-fno-sanitize-recover=undefined", "-Xarch_host", "-fno-omit-frame-pointer",
                 "-I", os.path.join(ROOT, "include"), "-I", os.path.join(PKG, "csrc")]
        subprocess.run([HIPCC, *flags, "-c", os.path.join(PKG, "csrc", "lh_api.hip"), "-o", api_o], check=True,
                       capture_output=True)
        pkg = os.path.join(d, "pkg", "nvfp4_scale_calibration_amd")
        os.makedirs(pkg)
        shutil.copy(os.path.join(PKG, "__init__.py"), pkg)
        subprocess.run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-Xarch_host", "-fsanitize=address",
                        "-Xarch_host", "-fsanitize=undefined", "-shared-libasan", "-o", os.path.join(pkg, "liblh.so"),
                        api_o, *objs], check=True, capture_output=True)
        env = dict(os.environ, PYTHONPATH=os.path.join(d, "pkg") + os.pathsep + ROOT, LD_PRELOAD=_asan_runtime(),
                   ASAN_OPTIONS="detect_leaks=0:halt_on_error=1", UBSAN_OPTIONS="print_stacktrace=1")
        r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider",
                            *(os.path.join(ROOT, "tests", t) for t in TESTS)], env=env, capture_output=True, text=True,
                           cwd=d, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
