"""CPU run of the host side of the operators around the core under AddressSanitizer and UBSan: ssd_layer_api.hip and
ssd_api.hip (argument checks, workspace layouts, product plans) built with the sanitizers on the host pass only,
linked against the built libssd.so for the launch code (tests/sanitize/layer_abi_check.cpp)."""
from __future__ import annotations

import os
import shutil

import pytest

from tests.test_sanitizers import HERE, LIBDIR, ROOT, SAN_ENV, _run


@pytest.mark.skipif(shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"),
                    reason="hipcc not available")
def test_layer_abi_under_asan_and_ubsan(tmp_path):
    if not os.path.exists(os.path.join(LIBDIR, "libssd.so")):
        pytest.skip("libssd.so is not built")
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    inc = ["-I" + os.path.join(ROOT, "include"), "-I" + os.path.join(LIBDIR, "csrc")]
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined"]
    objs = []
    for name in ("ssd_api", "ssd_layer_api"):
        objs.append(str(tmp_path / f"{name}.o"))
        _run([hipcc, "--offload-arch=gfx950", "-O1", "-g", "-fPIC", "-std=c++17", *inc, "-Xclang", "-target-feature",
              "-Xclang", "-packed-fp32-ops", *san, "-c", os.path.join(LIBDIR, "csrc", f"{name}.hip"), "-o", objs[-1]])
    drv, exe = str(tmp_path / "check.o"), str(tmp_path / "check")
    _run([hipcc, "--offload-host-only", "-O1", "-g", "-std=c++17", *inc, *san, "-c",
          os.path.join(HERE, "layer_abi_check.cpp"), "-o", drv])
    _run([hipcc, "--offload-arch=gfx950", *san, drv, *objs, "-L" + LIBDIR, "-lssd", "-Wl,-rpath," + LIBDIR, "-o", exe])
    # leak checking off: the HIP runtime's own start-up allocations are not ours
    out = _run([exe], env=dict(SAN_ENV, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1")).stdout
    assert "layer abi checks passed" in out
