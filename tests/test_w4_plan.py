"""The launches that the 4-bit products plan, on the CPU: every call of every test
here also has what the kernels and the workspace rely on checked
(tests/sanitize/w4_plan_driver.cpp)."""
import math
import os
import random
import shutil
import subprocess

import pytest

import test_gpu_w4 as W
import test_gpu_w4_tiles as X
from test_sanitize_cpu import CSRC, HERE, SAN_ENV, _run


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    """Calls (rows, K, N, experts, group, zeros, pair) -> for each the list of its
    launches: rows, columns, wavefronts, columns' tiles a block, rows of tiles, blocks."""
    at = tmp_path_factory.mktemp("plan")
    exe = str(at / "plan")
    _run([shutil.which("g++"), "-O1", "-g", "-std=c++17", "-Wall", "-Werror", "-fsanitize=address,undefined",
          "-fno-sanitize-recover=all", "-I", CSRC, os.path.join(HERE, "w4_plan_driver.cpp"), "-o", exe], at)

    def run(calls):
        r = subprocess.run([exe], input="".join(" ".join(str(int(v)) for v in c) + "\n" for c in calls),
                           capture_output=True, text=True, env=SAN_ENV)
        assert r.returncode == 0, (r.stdout[-200:], r.stderr)
        out = [[tuple(map(int, w.split())) for w in line.split(";")] for line in r.stdout.splitlines()]
        assert len(out) == len(calls)
        return out

    return run


# Every kernel that a plan can choose (a sweep of 400000 calls finds all of them and no
# other): pair, group, rows and columns of a tile, and of narrow tiles the
# wavefronts, of wide ones whether there are zeros.
NARROW = {False: ((4, 16), (4, 32), (16, 16), (16, 32), (32, 32)), True: ((4, 16), (16, 16), (32, 16))}
WIDE = {False: ((64, 128), (128, 256)), True: ((64, 64), (128, 128))}
KERNELS = {(glu, group, *tile, waves) for glu in (False, True) for group in (32, 64, 128) for tile in NARROW[glu]
           for waves in (4, 8)}
KERNELS |= {(glu, group, *tile, zeros) for glu in (False, True) for group in (32, 64, 128) for tile in WIDE[glu]
            for zeros in ("zeros", "none")}


def kernels(call, launches):
    """(kernel, whether it runs longer than its ring holds) of a call's launches."""
    T, K, N, E, group, zeros, glu = call
    out = []
    for rows, cols, waves, tiles, _, _ in launches:
        if rows < 64:   # a wavefront's shares of 256 k, two slots
            out.append(((bool(glu), group, rows, cols, waves), -(-K // (256 * waves)) * tiles > 2))
        else:           # stages of 128 k, three slots, one more than whole rounds
            out.append(((bool(glu), group, rows, cols, "zeros" if zeros else "none"), K > 3 * 128))
    return out


def _calls():
    """The calls of the GPU tests."""
    out = [(*s, z, False) for s in W.SHAPES for z in (True, False)] + [(*s, True, True) for s in W.SHAPES]
    for s in W.VARIANTS:
        out += [(*s, True, False), (*s, True, True)] + ([(*s, False, False)] if s[3] > 1 else [])
    out += [(*s, z, glu) for s in W.EIGHTS + X.TILES + X.LISTS for z in (False, True) for glu in (False, True)]
    out += [(T, K, N, E, group, K // group % 2 == 0, glu) for T, N, E in X.TAILS for group in (32, 64, 128)
            for K in X.tails(group) for glu in (False, True)]
    return out


def test_the_gpu_tests_run_every_kernel(plans):
    # a change of the estimates' constants must not take a kernel out of them
    calls = _calls()
    seen, long = set(), set()
    for call, launches in zip(calls, plans(calls)):
        for k, more in kernels(call, launches):
            seen.add(k)
            if more:
                long.add(k)
    assert seen == KERNELS, (KERNELS - seen, seen - KERNELS)
    assert long == KERNELS, KERNELS - long


def test_the_gpu_tests_run_partial_tiles_of_128_rows(plans):
    # with at most 64 rows left the upper wavefronts load and prepare alone: in every
    # such kernel, also in the steady part of the ring
    calls = [c for c in _calls() if c[3] == 1 and 0 < c[0] % 128 <= 64 and c[1] > 3 * 128]
    seen = {k for c, p in zip(calls, plans(calls)) for k, _ in kernels(c, p) if k[2] == 128}
    assert seen == {k for k in KERNELS if k[2] == 128}


def test_the_gpu_tests_run_both_wide_tiles_at_every_end_of_k(plans):
    for T, N, E in X.TAILS:
        for group in (32, 64, 128):
            for glu in (False, True):
                calls = [(T, K, N, E, group, K // group % 2 == 0, glu) for K in X.tails(group)]
                # (short K may take another tile: from one round of the ring on)
                rows = {p[0][0] for c, p in zip(calls, plans(calls)) if c[1] >= 384}
                assert rows <= {32, 64, 128} and len(rows & {64, 128}) == 1, (T, group, glu, rows)
    both = [plans([(T, 1024, 2056, 3, 128, True, glu) for T, _, _ in X.TAILS]) for glu in (False, True)]
    assert [{p[0][0] for p in b} for b in both] == [{64, 128}] * 2


def test_the_gpu_tests_run_every_pair_of_lists(plans):
    # the others' tile, the crowded experts' (a sweep of 600000 calls finds no other)
    want = {(glu, a, b) for glu in (False, True) for a in NARROW[glu] + WIDE[glu] for b in NARROW[glu] + WIDE[glu]
            if a[0] < b[0]} - {(False, (4, 16), b) for b in ((32, 32), *WIDE[False])}
    calls = [c for c in _calls() if c[3] > 1 and c[0] >= 128]
    seen = {(bool(c[6]), p[0][:2], p[1][:2]) for c, p in zip(calls, plans(calls)) if len(p) == 2}
    assert seen == want, (want - seen, seen - want)


def test_plans_of_any_size(plans):
    rng = random.Random(3)

    def size(low, high, step):
        v = math.exp(rng.uniform(math.log(low), math.log(high)))
        return max(step, round(v / step) * step)

    calls = []
    while len(calls) < 40000:
        group = rng.choice((32, 64, 128))
        K, N, T = min(65536, size(group, 65536, group)), size(8, 65536, 8), size(1, 1 << 25, 1)
        if K * N // 2 >= 1 << 31 or T * max(K, N) * 2 >= 1 << 31:   # (refused before a plan)
            continue
        E = rng.choice((1, 1, 1024, size(2, 1024, 1)))
        calls.append((T, K, N, E, group, rng.random() < 0.5, rng.random() < 0.5))
    # the ends of the ranges
    calls += [((1 << 31) // (2 * max(K, N)) - 1, K, N, E, 32, True, glu) for K in (32, 65536) for N in (8, 65528)
              for E in (1, 2, 1024) for glu in (False, True) if K * N // 2 < 1 << 31]
    seen = {k for c, p in zip(calls, plans(calls)) for k, _ in kernels(c, p)}
    assert seen <= KERNELS and len(seen) >= len(KERNELS) - 4, KERNELS - seen
