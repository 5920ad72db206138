"""The mixture-of-experts operators' and the tensor lists' entry points from C:
tests/native/experts_host_checks.c, a C99 program, against the regular library and
against the sources built with AddressSanitizer in their host code (-Xarch_host
-fsanitize=address).  Host logic only: sizes, overlaps and refusals."""

import os
import shutil

import pytest

native = pytest.importorskip("test_native_host")
INC, PKG, ROCM, ROOT = native.INC, native.PKG, native.ROCM, native.ROOT
_run, _asan_runtime = native._run, native._asan_runtime

SRC = os.path.join(ROOT, "tests", "native", "experts_host_checks.c")
INCLUDES = ["-D__HIP_PLATFORM_AMD__", f"-I{INC}", f"-I{ROCM}/include"]
PASSED = "experts' host checks passed"


@pytest.mark.skipif(shutil.which("gcc") is None, reason="no C compiler")
def test_c99_consumer_against_the_library(tmp_path):
    exe = tmp_path / "experts_host_checks"
    _run(["gcc", "-std=c99", "-Wall", "-Werror", "-O1", *INCLUDES, SRC, f"-L{PKG}", "-lgrz",
          f"-Wl,-rpath,{PKG}", f"-Wl,-rpath,{ROCM}/lib", "-o", str(exe)])
    assert PASSED in _run([str(exe)]).stdout


@pytest.mark.skipif(not os.path.exists(f"{ROCM}/bin/hipcc") or _asan_runtime() is None,
                    reason="hipcc or the clang ASan runtime missing")
def test_host_code_under_address_sanitizer(tmp_path):
    from gradient_reduce_zero_amd.build import EXPERTS_SRC, FLAGS, TENSORS_SRC
    lib = tmp_path / "libexperts.so"
    flags = [f for f in FLAGS if f != "-O3"] + ["-O1", "-g"]
    _run([f"{ROCM}/bin/hipcc", *flags, "-Xarch_host", "-fsanitize=address", "-shared-libsan",
          f"-I{INC}", EXPERTS_SRC, TENSORS_SRC, "-o", str(lib)])
    exe = tmp_path / "experts_host_checks_asan"
    rt = _asan_runtime()
    _run([f"{ROCM}/llvm/bin/clang", "-g", "-O1", "-fsanitize=address", "-shared-libsan",
          *INCLUDES, "-DWITHOUT_STEP", "-rdynamic", SRC, f"-L{tmp_path}", "-lexperts",
          f"-Wl,-rpath,{tmp_path}", f"-Wl,-rpath,{ROCM}/lib", f"-Wl,-rpath,{rt}",
          "-o", str(exe)])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0")
    assert PASSED in _run([str(exe)], env=env).stdout
