"""Which kernels the 8-bit floating-point products go to, on the CPU: the real planner
with launchers that write down what they are given (tests/sanitize/f8_kinds.cpp)."""
import os
import random
import shutil
import subprocess

import pytest

from f8_tile_cases import CASES, PLACED

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "newton_schulz_04_amd", "csrc")
ROCM = "/opt/rocm"


@pytest.fixture(scope="module")
def kinds(tmp_path_factory):
    """kinds(lists) of (dtype, products (m, n, k, fp32 scales, squares, offset, ld)):
    for each list its workspace and its products' [(kind, pieces)]."""
    gxx = shutil.which("g++")
    if not gxx or not os.path.exists(os.path.join(ROCM, "include", "hip", "hip_runtime.h")):
        pytest.skip("g++ or the HIP headers are missing")
    exe = str(tmp_path_factory.mktemp("f8_kinds") / "f8_kinds")
    subprocess.run([gxx, "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include", f"-I{ROOT}/include",
                    f"-I{CSRC}", os.path.join(CSRC, "ns_f8_api.cpp"), os.path.join(HERE, "sanitize", "f8_kinds.cpp"),
                    "-o", exe, f"-L{ROCM}/lib", f"-Wl,-rpath,{ROCM}/lib", "-lamdhip64"], check=True)

    def run(lists):
        text = "".join(f"{'bf16 fp32'.split().index(dtype)} {len(ps)}\n" +
                       "".join(" ".join(str(int(v)) for v in p) + "\n" for p in ps) for dtype, ps in lists)
        r = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=300,
                           env=dict(os.environ, HIP_VISIBLE_DEVICES=""))
        assert r.returncode == 0, r.stderr
        out = []
        for line in r.stdout.splitlines():
            need, *rest = line.split()
            out.append((int(need), list(zip(rest[::2], map(int, rest[1::2])))))
        assert len(out) == len(lists)
        return out
    return run


def test_the_gpu_tests_reach_every_kind_of_tile(kinds):
    got = kinds([(dtype, [(m, n, k, any_, sq, 0, n) for m, n, k, any_, sq, _ in ps]) for _, dtype, ps in CASES])
    seen = set()
    for (name, dtype, ps), (need, each) in zip(CASES, got):
        for (m, n, k, any_, sq, want), (kind, pieces) in zip(ps, each):
            assert kind == {"cut": "small"}.get(want, want), (name, dtype, m, n, k)
            assert (pieces > 1) == (want == "cut"), (name, dtype, m, n, k)
            seen.add((want, dtype, bool(any_)))
    assert {("big", "bf16", False), ("big", "fp32", False), ("mid", "bf16", False), ("mid", "fp32", True),
            ("small", "bf16", True), ("small", "fp32", False), ("cut", "bf16", False), ("cut", "fp32", False)} <= seen


def test_cuts_and_workspaces_depend_on_sizes_alone(kinds):
    """Wherever the output lies and at whatever pitch: the same workspace, the same pieces
    (which is what the bits depend on), large tiles only where it goes four at a time."""
    rng = random.Random(1)
    sizes = [(dtype, [(m, n, k, False, True)]) for m, n, k, dtype in PLACED]
    for _ in range(1500):
        one = lambda: (rng.randint(1, 5000), 4 * rng.randint(1, 1300), round(2 ** rng.uniform(4, 17)),   # noqa: E731
                       rng.random() < 0.2, rng.random() < 0.5)
        sizes.append((rng.choice(["bf16", "fp32"]), [one() for _ in range(rng.choice([1, 1, 2, 5]))]))
    lists, elt = [], {"bf16": 2, "fp32": 4}
    for dtype, ps in sizes:
        for place in range(3):   # aligned, one value further, at an odd pitch
            lists.append((dtype, [(*p, elt[dtype] * (place == 1), p[1] + (place == 2)) for p in ps]))
    got = kinds(lists)
    turned = set()
    for i, (dtype, ps) in enumerate(sizes):
        (need, each), *others = got[3 * i:3 * i + 3]
        for other, kind in others:
            assert other == need and [n for _, n in kind] == [n for _, n in each], (dtype, ps)
            assert all(k != "big" for k, _ in kind), (dtype, ps)
            turned |= {(dtype, a, b) for (a, _), (b, _) in zip(each, kind) if a != b}
    assert {("bf16", "big", "mid"), ("bf16", "big", "small"), ("fp32", "big", "small")} <= turned
    for i in range(len(PLACED)):
        assert got[3 * i] == (0, [("big", 1)])


def test_products_of_a_list_take_no_kind_that_is_not_theirs(kinds):
    """Lists of mixed scale types and lengths: mid tiles of bf16 outputs go to one-byte
    scales, those of fp32 outputs to fp32 scales, and what stands beside a product of the
    other type does not change its kind."""
    rng = random.Random(2)
    lists = []
    for _ in range(3000):
        one = lambda any_: (rng.randint(33, 4000), rng.randint(30, 5000), round(2 ** rng.uniform(4, 15)),   # noqa: E731
                            any_, rng.random() < 0.5)
        ps = [one(rng.random() < 0.5) for _ in range(rng.choice([1, 2, 5, 40]))]
        lists.append((rng.choice(["bf16", "fp32"]), [(*p, 0, p[1]) for p in ps]))
    got = kinds(lists + [(dtype, [p for p in ps if p[3] == any_]) for any_ in (0, 1) for dtype, ps in lists])
    for i, (dtype, ps) in enumerate(lists):
        each = got[i][1]
        assert {k for k, _ in each} <= {"few", "small", "mid", "big"}
        for any_ in (0, 1):
            alone = got[len(lists) * (1 + any_) + i][1]
            mine = [e for p, e in zip(ps, each) if p[3] == any_]
            assert [k for k, _ in mine] == [k for k, _ in alone], (dtype, ps)
