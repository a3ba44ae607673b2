"""The entry tables of the grouped-row attention kernels stay inside what the host
sizes them for, whatever the row offsets hold: a host program on the kernels' own
arithmetic over random offsets, in order and out of order (no GPU needed)."""
import os
import random
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    exe = str(tmp_path_factory.mktemp("tables") / "group_tables_host")
    subprocess.run([cxx, "-O1", "-std=c++17", "-o", exe, os.path.join(HERE, "group_tables_host.cpp")], check=True)

    def run(cases):
        text = "\n".join(" ".join(map(str, [c[x] for x in FIELDS] + c["offsets"] + c["lens"] + c["own"])) for c in cases)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split("\n")
        return [[int(x) for x in line.split()] for line in out if line]
    return run


FIELDS = ("H", "Hkv", "R", "ncol", "chunk_w", "chunk_n", "a_rows", "shared", "n_rows", "n_groups", "max0", "max1")


def case(rng, offsets, n_rows, H=32, Hkv=32, R=2048, shared=False, max0=512, max1=256, full=False):
    n = len(offsets) - 1
    length = (lambda top: top) if full else (lambda top: rng.randint(0, top))
    unit = max(16, 128 // Hkv)
    return dict(H=H, Hkv=Hkv, R=R, ncol=128, chunk_w=256, chunk_n=2 * unit, a_rows=max(1, min(64 // H, 16 * Hkv // H)),
                shared=int(shared), n_rows=n_rows, n_groups=n, max0=max0, max1=max1, offsets=list(offsets),
                lens=[length(max0) for _ in range(n)], own=[length(max(max0, max1)) for _ in range(n_rows if shared else 0)])


def check(c, got):
    rows, ordered, k_cost, v_units, v_tiles, a_blocks, a_tiles, k_most, u_most, v_most, a_most = got
    assert ordered and rows <= c["n_rows"], c["offsets"][:20]
    assert k_cost <= k_most and v_units <= u_most and v_tiles <= v_most and a_tiles <= a_most, c["offsets"][:20]
    assert a_blocks <= a_most * (max(c["max0"], c["max1"]) // 64 + 1)


def test_offsets_that_go_up_and_down(model):
    rng = random.Random(3)
    cases = [case(rng, [0, 64] * 32 + [64], 64, full=True),                   # every other group has all rows
             case(rng, [0, 256] * 32, 256, H=64, Hkv=8, full=True, shared=True),
             case(rng, [0, 8] * 500, 8, full=True),                           # more groups than rows
             case(rng, [0, 4096] * 2048, 4096, R=4096, max0=16384, full=True),   # sums past 32 bits, were all rows taken
             case(rng, [-7, 5, -1, 1 << 30, 3, -(1 << 31), 9], 9)]
    out = model(cases)
    for c, got in zip(cases, out):
        check(c, got)
    # a group keeps its rows however the offsets behind it fall
    assert [x[0] for x in out] == [64, 256, 8, 4096, 9]


def test_random_offsets(model):
    rng = random.Random(4)
    cases = []
    for _ in range(400):
        n_rows, n = rng.randint(1, 300), rng.randint(1, 60)
        H = 1 << rng.randint(0, 6)
        Hkv = 1 << rng.randint(0, H.bit_length() - 1)
        pick = rng.choice([lambda: rng.randint(0, n_rows), lambda: rng.choice([0, n_rows]),
                           lambda: rng.randint(-2 * n_rows, 3 * n_rows), lambda: rng.randint(-(1 << 31), (1 << 31) - 1)])
        off = [pick() for _ in range(n + 1)]
        if rng.random() < 0.3:
            off.sort()
        cases.append(case(rng, off, n_rows, H, Hkv, 64 * rng.randint(1, 64), rng.random() < 0.5, rng.randint(0, 3000),
                          rng.randint(0, 3000), rng.random() < 0.3))
    for c, got in zip(cases, model(cases)):
        check(c, got)


def test_offsets_in_order_give_the_rows_between_them(model):
    rng = random.Random(5)
    cases = []
    for _ in range(100):
        n_rows = rng.randint(1, 200)
        off = sorted([0] + [rng.randint(0, n_rows) for _ in range(rng.randint(1, 20))])
        cases.append(case(rng, off, n_rows))
    for c, got in zip(cases, model(cases)):
        check(c, got)
        assert got[0] == c["offsets"][-1]
