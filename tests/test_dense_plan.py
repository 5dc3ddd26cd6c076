"""The launches that the dense operators plan, on the CPU: their host code, built
with host-only sanitizers against recorders in place of the kernel launchers.
Every call of every test here also has the planner, its workspaces and its
partial tiles checked (tests/sanitize/dense_plan_driver.cpp)."""
import math
import os
import random
import shutil
import subprocess

import pytest

import test_gpu_dense_edges as E
import test_gpu_glu as G
import test_gpu_lora as L
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


def test_a_long_stack_has_no_part(plans):
    # from 64 adapters on, more of them that no token names change neither tile nor
    # split, hence no bits
    for T in (1, 64, 65, 116, 198, 333, 1024, 2048, 3900, 7168, 16384):
        for K, N in ((2048, 4096), (840, 1984), (8200, 264)):
            for r in (8, 32, 256):
                for w in (0, 1):
                    calls = [f"lora {T} {K} {N} {n} {r} {w} 0" for n in (64, 65, 512, 4096, 65536)]
                    got = plans(calls)
                    assert got[0][0][0] != "error" and all(p == got[0] for p in got), calls


# Every variant that a plan can choose (a sweep of 60000 calls finds no other), and
# the stages of 64 k that the GPU tests have to run it with: more than its ring
# holds, or than its wavefronts take at a time ("finish": splits).
VARIANTS = {
    **{(m, v): n for m in (GLU, DX, DW, LIN) for v, n in (
        ("256", 5), ("128 alone", 5), ("128 shared", 5), ("64 x 8", 9), ("64 x 4", 5), ("finish", 2),
        ("finish, over 8", 9))},
    **{("grads", bm, order): 5 for bm in (64, 128) for order in ("dw first", "dx first")},
    **{(GLU, v): 0 for v in (16, 32, 64, "64 wide")}, **{(LIN, v): 0 for v in ("fused", 16, 32, 64)},
    **{("shrink", *v): 0 for v in ((1, 8), (1, 4), (8, 8), (16, 8), (16, 4))},
}


def variants(call, launches):
    """(kernel, stages of 64 k) of a call's launches, as the launchers choose
    them (launch_any, launch_skinny, shrink)."""
    out = []
    for w in launches:
        v = [int(x) for x in w[1:]]
        if w[0] == "dense":
            mode, bm, mt, nt, splits, stages = v
            if bm == 256:
                out.append(((mode, "256"), stages))
            elif bm == 128:
                out.append(((mode, "128 alone" if mt * nt <= 256 else "128 shared"), stages))
            else:
                out.append(((mode, "64 x 8" if mt * nt * splits <= 256 else "64 x 4"), -(-stages // splits)))
                if splits > 1:
                    out.append(((mode, "finish" if splits <= 8 else "finish, over 8"), splits))
        elif w[0] == "grads":
            out.append((("grads", v[3], "dw first" if v[6] else "dx first"), min(v[2], v[5])))
        elif w[0] == "skinny":
            mode, T, fused = v
            cols = int(call.split()[3])
            wide = mode == GLU and 32 < T and cols >= 8 * 255 + 1
            out.append(((mode, "fused" if fused else 16 if T <= 16 else 32 if T <= 32 else "64 wide" if wide else 64), 0))
        elif w[0] == "shrink":
            T, rank, K = v
            rpad = -(-rank // 32) * 32
            if T * rank * K * 2 <= 192 << 20 and T * (rpad // 16) <= 2048:
                out.append((("shrink", 1, 8 if T * (rpad // 16) <= 512 else 4), 0))
            else:
                tpf = 8 if -(-T // 16) * (rpad // 32) <= 96 else 16
                out.append((("shrink", tpf, 8 if -(-T // tpf) * (rpad // 32) <= 256 else 4), 0))
    return out


def test_the_gpu_tests_run_every_variant(plans):
    # a change of the plan's constants must not take a variant out of them
    calls = [f"{op} {T} {H} {I} 1 1" for T, H, I in G.SHAPES + E.GRADIENTS for op in ("glu", "bwd")]
    calls += [f"lora {T} {K} {N} {n} {r} {w} 0" for T, K, N, n, r in L.SHAPES + E.PROJECTIONS for w in (0, 1)]
    most = {}
    for call, launches in zip(calls, plans(calls)):
        for v, stages in variants(call, launches):
            most[v] = max(most.get(v, 0), stages)
    assert set(most) == set(VARIANTS)
    assert all(most[v] >= n for v, n in VARIANTS.items()), {v: (most[v], n) for v, n in VARIANTS.items() if most[v] < n}


def test_plans_of_any_size(plans):
    # the recorders' checks (tiles and splits cover the result once, partial tiles
    # inside the advertised workspace) over the whole range, odd sizes among them
    rng = random.Random(7)

    def size(low, high, step):
        v = math.exp(rng.uniform(math.log(low), math.log(high)))
        return max(step, round(v / step) * step)

    calls = []
    for _ in range(20000):
        T, a, b = size(1, 200000, 1), size(8, 65536, 8), size(8, 65536, 8)
        want = rng.choice(("1 1", "1 0", "0 1"))
        calls.append(rng.choice((f"glu {T} {a} {b}", f"bwd {T} {a} {b} {want}",
                                 f"lora {T} {a} {b} {size(1, 65536, 1)} {size(8, 256, 8)} {rng.randrange(2)} {rng.randrange(2)}")))
    calls += [f"bwd 0 {a} {b} 1 1" for a, b in ((8, 8), (4096, 2048), (65536, 8))]
    got = plans(calls)
    refused = [c for c, p in zip(calls, got) if p[0][0] == "error"]
    assert len(refused) < len(calls) // 2   # beyond 2 GiB
    seen = {v for c, p in zip(calls, got) if c not in refused for v, _ in variants(c, p)}
    assert seen <= set(VARIANTS) and len(seen) >= len(VARIANTS) - 5, set(VARIANTS) - seen


def test_an_ordinary_call_beside_a_long_stack(plans):
    # a prompt of one request takes the large tiles, however many are loaded
    for call, bm in (("7168 2048 4096", 256), ("1024 2048 4096", 128), ("1024 4096 4096", 128)):
        T, K, N = call.split()
        for n in (8, 64, 512, 3000, 65536):
            (p,) = plans([f"lora {T} {K} {N} {n} 32 1 0"])
            assert p[1][:3] == ["dense", str(LIN), str(bm)], (call, n, p)
