"""The launches that the dense operators plan, on the CPU: their host code, built
with host-only sanitizers against recorders in place of the kernel launchers.
Every call of every test here also has the planner, its workspaces and its
partial tiles checked (tests/sanitize/dense_plan_driver.cpp)."""
import os
import shutil
import subprocess

import pytest

from test_sanitize_cpu import CSRC, HERE, ROOT, SAN_ENV, _run

pytestmark = pytest.mark.skipif(not os.path.exists("/opt/rocm/bin/hipcc"), reason="needs hipcc")

GLU, DX, DW, LIN = range(4)


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    """Calls (lines) -> for each the list of its launches, split into words."""
    at = tmp_path_factory.mktemp("plan")
    inc = ["-I", os.path.join(ROOT, "include"), "-I", CSRC]
    flags = ["-O1", "-g", "-std=c++17", "-fPIC", "-x", "hip", *inc]
    obj, drv, exe = (str(at / n) for n in ("dense.o", "driver.o", "plan"))
    _run(["/opt/rocm/bin/hipcc", *flags, "--offload-arch=gfx950", "-Xclang", "-target-feature", "-Xclang",
          "-packed-fp32-ops", "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
          "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer",
          "-c", os.path.join(CSRC, "dense.cpp"), "-o", obj], at)
    _run(["/opt/rocm/llvm/bin/clang++", *flags, "--cuda-host-only", "-fsanitize=address,undefined",
          "-fno-omit-frame-pointer", "-c", os.path.join(HERE, "dense_plan_driver.cpp"), "-o", drv], at)
    _run([shutil.which("g++"), "-fsanitize=address,undefined", obj, drv, "-L/opt/rocm/lib", "-lamdhip64",
          "-Wl,-rpath,/opt/rocm/lib", "-o", exe], at)

    def run(calls):
        r = subprocess.run([exe], input="\n".join(calls) + "\n", capture_output=True, text=True, env=SAN_ENV)
        assert r.returncode == 0, r.stdout[-500:] + r.stderr
        out = [[w.split() for w in line.split(";")] for line in r.stdout.splitlines()]
        assert len(out) == len(calls)
        return out

    return run


def test_the_stacks_length_has_no_part(plans):
    # adapters that no token names change neither tile nor split, hence no bits
    for T in (1, 64, 65, 116, 198, 333, 1024, 2048, 3900, 7168, 16384):
        for K, N in ((2048, 4096), (840, 1984), (8200, 264)):
            for r in (8, 32, 256):
                for w in (0, 1):
                    calls = [f"lora {T} {K} {N} {n} {r} {w} 0" for n in (1, 2, 8, 64, 512, 4096, 65536)]
                    got = plans(calls)
                    assert got[0][0][0] != "error" and all(p == got[0] for p in got), calls
