"""The host checks of the attention and cache entry points (test_attention_abi_cpu.py)
with the C-ABI sources' host pass under AddressSanitizer and UBSan (CPU only)."""
import glob
import os
import shutil
import subprocess
import sys

import pytest

CHECKS = os.path.join(os.path.dirname(os.path.abspath(__file__)), "test_attention_abi_cpu.py")


def test_host_checks_under_sanitizers(tmp_path):
    """These checks again with the C-ABI sources' host pass under AddressSanitizer and UBSan."""
    from rotation_int4_weight_amd import build as b
    abi = [s for s in b.SOURCES if s.endswith(".cpp")]
    objs = [os.path.join(b.BUILD, s + ".o") for s in b.SOURCES if s not in abi]
    rt = sorted(glob.glob("/opt/rocm/llvm/lib/clang/*/lib/linux/libclang_rt.asan-x86_64.so"))
    clangxx = "/opt/rocm/llvm/bin/clang++"
    if not rt or not os.path.exists(clangxx) or not all(os.path.exists(o) for o in objs):
        pytest.skip("sanitizer runtime or kernel objects missing")
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    san = []
    for f in ("-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer"):
        san += ["-Xarch_host", f]
    built = []
    for s in abi:
        built.append(str(tmp_path / (s + ".o")))
        subprocess.run([hipcc, "-O1", "-g", "-std=c++17", "-fPIC", "--offload-arch=gfx950", *san, "-I",
                        os.path.join(b.ROOT, "include"), "-I", b.CSRC, "-c", os.path.join(b.CSRC, s), "-o", built[-1]],
                       check=True, capture_output=True)
    lib, rtdir = str(tmp_path / "libparo_san.so"), os.path.dirname(rt[-1])
    subprocess.run([clangxx, "-shared", "-fPIC", *built, *objs, "-L", rtdir, "-lclang_rt.asan-x86_64",
                    "-Wl,-rpath," + rtdir, "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", lib],
                   check=True, capture_output=True)
    env = dict(os.environ, PARO_LIB=lib, LD_PRELOAD=rt[-1], ASAN_OPTIONS="detect_leaks=0")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", CHECKS,
                        "-k", "not binding"], env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, f"exit {r.returncode}:\n{r.stdout[-3000:]}\n{r.stderr[-3000:]}"
