"""The operators around the recurrences used from plain C (tests/c/
layer_consumer.c, host-side paths only), built with the system compiler against
the library, and with the C ABI source rebuilt under AddressSanitizer and
UndefinedBehaviorSanitizer (host code; the other objects are the regular
build's). No GPU is used."""
import glob
import os
import shutil
import subprocess

import pytest

import delta_rule_recurrent_scan_amd as osdn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "delta_rule_recurrent_scan_amd", "csrc")
BUILD = os.path.join(ROOT, "_build")
HIPCC = "/opt/rocm/bin/hipcc"
CLANG = "/opt/rocm/llvm/bin/clang"
CLANGXX = "/opt/rocm/llvm/bin/clang++"
RUNTIME = (glob.glob("/opt/rocm/llvm/lib/clang/*/lib/linux") or [None])[0]
LIB = osdn.library_path()
SRC = os.path.join(ROOT, "tests", "c", "layer_consumer.c")


@pytest.mark.skipif(not os.path.exists(LIB), reason="libosdn.so not built")
@pytest.mark.skipif(shutil.which("gcc") is None, reason="no C compiler")
def test_layer_consumer(tmp_path):
    exe, libdir = str(tmp_path / "layer_consumer"), os.path.dirname(LIB)
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "include"), SRC, "-L", libdir, "-losdn",
                    "-Wl,-rpath," + libdir, "-o", exe], check=True)
    p = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert p.returncode == 0, p.stdout + p.stderr
    assert "all checks passed" in p.stdout


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG) and RUNTIME),
                    reason="ROCm clang toolchain with sanitizer runtimes not found")
@pytest.mark.skipif(not os.path.exists(os.path.join(BUILD, "mixer_api.cpp.o")),
                    reason="in-tree build objects (_build/) missing")
def test_layer_consumer_under_sanitizers(tmp_path):
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-fno-omit-frame-pointer"]
    src = "mixer_api.cpp"
    obj = str(tmp_path / (src + ".o"))
    subprocess.run([HIPCC, "-O1", "-g", "-std=c++17", "-fPIC", "-I",
                    os.path.join(ROOT, "include")] + san
                   + ["-c", os.path.join(CSRC, src), "-o", obj], check=True,
                   capture_output=True)
    rest = [os.path.join(BUILD, o) for o in sorted(os.listdir(BUILD))
            if o.endswith(".o") and o != src + ".o"]
    rt, lib = RUNTIME, str(tmp_path / "liblayer_san.so")
    subprocess.run([CLANGXX, "-shared", "-fPIC", "-fsanitize=address,undefined",
                    "-shared-libsan", "-o", lib, obj] + rest
                   + ["-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib",
                      "-Wl,-rpath," + rt], check=True, capture_output=True)
    exe = str(tmp_path / "layer_consumer_san")
    subprocess.run([CLANG, "-std=c99", "-Wall", "-Werror", "-O1", "-g",
                    "-fsanitize=address,undefined", "-shared-libsan",
                    "-fno-omit-frame-pointer", "-I", os.path.join(ROOT, "include"), SRC,
                    "-o", exe, "-L", str(tmp_path), "-llayer_san",
                    "-Wl,-rpath," + str(tmp_path), "-Wl,-rpath," + rt], check=True,
                   capture_output=True)
    env = dict(os.environ, ASAN_OPTIONS="halt_on_error=1:detect_leaks=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    p = subprocess.run([exe], capture_output=True, text=True, timeout=120, env=env)
    out = p.stdout + p.stderr
    assert p.returncode == 0, out
    assert "all checks passed" in p.stdout
    assert "runtime error" not in out and "AddressSanitizer" not in out, out
