"""The root-mean-square norm, 8-bit product and beam search entry points' host code under
AddressSanitizer and UndefinedBehaviorSanitizer (host_sanitizer_serve_driver.cpp), as
test_host_sanitizers.py does for the loss's. Runs where no GPU is visible."""
import os
import shutil

import pytest
import torch

from linear_cross_entropy_masked_amd import build as lce_build
from test_host_sanitizers import CSRC, HOST_SAN, ROOT, _run


@pytest.mark.timeout(900)
def test_serve_host_code_under_asan_and_ubsan(tmp_path):
    if torch.cuda.is_available():
        pytest.skip("runs where no GPU is visible (valid calls would reach the kernels)")
    hipcc = lce_build.hipcc()
    clangxx = os.path.join(os.path.dirname(os.path.realpath(hipcc)), "..", "llvm", "bin", "clang++")
    if not os.path.exists(clangxx):
        clangxx = shutil.which("clang++") or "/opt/rocm/llvm/bin/clang++"
    objs = {s: os.path.join(lce_build.BUILD_DIR, s.replace(".hip", ".o")) for s in lce_build.SOURCES}
    if not all(os.path.exists(o) for o in objs.values()):
        lce_build.build()
    out = str(tmp_path / "capi_serve_san.o")
    _run([hipcc, f"--offload-arch={lce_build.ARCH}", "-O1", "-std=c++17", "-fPIC", "-g",
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-I", os.path.join(ROOT, "include"), "-I", CSRC, *HOST_SAN, "-c",
          os.path.join(CSRC, "capi_serve.hip"), "-o", out])
    lib = str(tmp_path / "liblce_serve_san.so")
    _run([hipcc, f"--offload-arch={lce_build.ARCH}", "-shared", "-fPIC", out,
          *(o for s, o in objs.items() if s != "capi_serve.hip"), *HOST_SAN, "-o", lib])
    exe = str(tmp_path / "host_sanitizer_serve_driver")
    rocm_lib = os.path.join(os.path.dirname(os.path.realpath(hipcc)), "..", "lib")
    _run([clangxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined",
          "-fno-sanitize-recover=all", "-fno-omit-frame-pointer",
          "-I", os.path.join(ROOT, "include"),
          os.path.join(ROOT, "tests", "host_sanitizer_serve_driver.cpp"), lib,
          f"-Wl,-rpath,{tmp_path}", f"-L{rocm_lib}", "-lamdhip64", f"-Wl,-rpath,{rocm_lib}",
          "-o", exe])
    printed = _run([exe], sanitized_program=True)
    assert "0 failures" in printed or "skipped" in printed
