"""The dense operators' host code under host-only sanitizers, on the CPU: every
rejection and the plans of a grid of sizes (the kernel launchers are stubs that
abort, so any call that slipped past the checks would fail the test)."""
import os
import re
import shutil

import pytest

from test_sanitize_cpu import CSRC, HERE, ROOT, SAN_ENV, _run


def _launcher_stubs():
    """Definitions that abort for every launcher dense.h declares."""
    text = open(os.path.join(CSRC, "dense.h")).read()
    decls = re.findall(r"^hipError_t (launch_\w+\([^;]*\));", text, re.M)
    assert len(decls) >= 5
    body = "\n".join(f"hipError_t {d} {{ abort(); }}" for d in decls)
    return f'#include <stdlib.h>\n#include "dense.h"\nnamespace moe {{\n{body}\n}}\n'


@pytest.mark.skipif(not os.path.exists("/opt/rocm/bin/hipcc"), reason="needs hipcc")
def test_dense_host_checks_under_sanitizers(tmp_path):
    obj = str(tmp_path / "dense.o")
    _run(["/opt/rocm/bin/hipcc", "-O1", "-g", "-std=c++17", "-fPIC", "--offload-arch=gfx950", "-x", "hip",
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
          "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer",
          "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-c", os.path.join(CSRC, "dense.cpp"), "-o", obj], tmp_path)
    stubs = tmp_path / "stubs.cpp"
    stubs.write_text(_launcher_stubs())
    flags = ["-O1", "-g", "-std=c++17", "-fno-omit-frame-pointer", "-I", os.path.join(ROOT, "include")]
    _run(["/opt/rocm/llvm/bin/clang++", *flags, "-x", "hip", "--cuda-host-only", "-fsanitize=address,undefined",
          "-I", CSRC, "-c", str(stubs), "-o", str(tmp_path / "stubs.o")], tmp_path)
    exe = str(tmp_path / "dense_asan")
    _run([shutil.which("g++"), *flags, "-fsanitize=address,undefined", os.path.join(HERE, "dense_driver.cpp"), obj,
          str(tmp_path / "stubs.o"), "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", exe], tmp_path)
    import subprocess
    r = subprocess.run([exe], capture_output=True, text=True, env=SAN_ENV)
    assert r.returncode == 0 and "dense driver: ok" in r.stdout, r.stdout + r.stderr
