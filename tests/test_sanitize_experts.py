"""The host code of the operators around a MoE layer's own experts under
host-only sanitizers, on the CPU: rejections and plans (the kernel launchers
are stubs that abort, so a call that slipped past the checks fails)."""
import os
import re
import shutil
import subprocess

import pytest

from test_sanitize_cpu import CSRC, HERE, ROOT, SAN_ENV, _run

SOURCES = {"tokens.cpp": "tokens.h", "w4.cpp": "w4.h"}


def _launcher_stubs():
    """Definitions that abort for every launcher the headers declare."""
    text = ""
    for header in SOURCES.values():
        decls = re.findall(r"^hipError_t (launch_\w+\([^;]*\));", open(os.path.join(CSRC, header)).read(), re.M)
        assert decls
        body = "\n".join(f"hipError_t {d} {{ abort(); }}" for d in decls)
        text += f'#include <stdlib.h>\n#include "{header}"\nnamespace moe {{\n{body}\n}}\n'
    return text


@pytest.mark.skipif(not os.path.exists("/opt/rocm/bin/hipcc"), reason="needs hipcc")
def test_host_checks_under_sanitizers(tmp_path):
    objs = []
    for src in SOURCES:
        objs.append(str(tmp_path / (src + ".o")))
        _run(["/opt/rocm/bin/hipcc", "-O1", "-g", "-std=c++17", "-fPIC", "--offload-arch=gfx950", "-x", "hip",
              "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
              "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
              "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer",
              "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-c", os.path.join(CSRC, src), "-o", objs[-1]], tmp_path)
    stubs = tmp_path / "stubs.cpp"
    stubs.write_text(_launcher_stubs())
    flags = ["-O1", "-g", "-std=c++17", "-fno-omit-frame-pointer", "-I", os.path.join(ROOT, "include")]
    _run(["/opt/rocm/llvm/bin/clang++", *flags, "-x", "hip", "--cuda-host-only", "-fsanitize=address,undefined",
          "-I", CSRC, "-c", str(stubs), "-o", str(tmp_path / "stubs.o")], tmp_path)
    exe = str(tmp_path / "experts_asan")
    _run([shutil.which("g++"), *flags, "-fsanitize=address,undefined", os.path.join(HERE, "experts_driver.cpp"), *objs,
          str(tmp_path / "stubs.o"), "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", exe], tmp_path)
    r = subprocess.run([exe], capture_output=True, text=True, env=SAN_ENV)
    assert r.returncode == 0 and "experts driver: ok" in r.stdout, r.stdout + r.stderr
