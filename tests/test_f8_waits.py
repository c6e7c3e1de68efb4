"""The counted waits of the 8-bit floating-point tile kernels, in the machine code of
the built library.

A wavefront waits before a barrier with `s_waitcnt vmcnt(N)`, which leaves in flight the
N vector-memory operations issued last: the loads to LDS of the slots after the one that
is read next, N or a multiple of a slot's count. That holds as long as every way from one
such wait to the next issues the loads of exactly one slot (none between the wait before
the loop and a first step that has a third slot in flight already); other operations
between them only make a wait longer. This disassembles the library and follows every
path back from each wait.
"""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "newton_schulz_04_amd", "libns.so")
OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
# loads of a slot by a wavefront: rows of A and of B / (8 rows a load x wavefronts)
SHAPES = {"k_f8_big": (16, 2), "Li128ELi2E": (8, 2), "Li128ELi3E": (6, 3)}   # loads, slots of the ring


def functions(tmp_path):
    lib = shutil.copy(LIB, tmp_path)
    subprocess.run([OBJDUMP, "--offloading", lib], check=True, capture_output=True, cwd=tmp_path)
    for part in sorted(os.listdir(tmp_path)):
        if "gfx950" not in part:
            continue
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", part], check=True, capture_output=True, text=True,
                              cwd=tmp_path).stdout
        for name, body in re.findall(r"^[0-9a-f]+ <(\S*k_f8_(?:big|tiles)\S*)>:\n(.*?)(?=^\S|\Z)", text, re.M | re.S):
            yield name, re.findall(r"^\t(.*?)\s*// ([0-9A-F]+):", body, re.M), body


def graph(name, lines, body):
    """Each instruction's kind (D a load to LDS, an int the N of a counted wait, None) and
    where control may come from."""
    at = {int(addr, 16): k for k, (_, addr) in enumerate(lines)}
    start = int(lines[0][1], 16)
    kinds, comes = [None] * len(lines), [[k - 1] if k else [] for k in range(len(lines))]
    targets = dict(re.findall(r"// ([0-9A-F]+):.*?<%s(?:\+0x([0-9a-f]+))?>" % re.escape(name), body))
    for k, (text, addr) in enumerate(lines):
        op = text.split()[0]
        if op == "s_barrier":
            back = k - 1
            if lines[back][0] == "s_waitcnt lgkmcnt(0)":
                back -= 1
            wait = re.fullmatch(r"s_waitcnt vmcnt\((\d+)\)", lines[back][0])
            if wait:
                kinds[k] = int(wait.group(1))
        elif op.startswith("buffer_load") and text.endswith(" lds"):
            kinds[k] = "D"
        if op in ("s_branch", "s_endpgm") and k + 1 < len(lines):
            comes[k + 1].remove(k)
        if op.startswith(("s_cbranch", "s_branch")):
            comes[at[start + int(targets[addr] or "0", 16)]].append(k)
    return kinds, comes


def ways(kinds, comes, at, most):
    """(the wait before, or None for the start; loads to LDS on the way) of every path back."""
    found, met, todo = set(), set(), [(k, 0) for k in comes[at]]
    while todo:
        k, n = todo.pop()
        if (k, n) in met or n > most:
            continue
        met.add((k, n))
        if isinstance(kinds[k], int):
            found.add((k, n))
            continue
        n += kinds[k] == "D"
        if k == 0:
            found.add((None, n))
        todo += [(c, n) for c in comes[k]]
    return found


@pytest.mark.skipif(not os.path.exists(LIB), reason="the library is not built")
@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no disassembler")
def test_waits_leave_only_later_slots_in_flight(tmp_path):
    seen = 0
    for name, lines, body in functions(tmp_path):
        loads, ring = next(v for key, v in SHAPES.items() if key in name)
        kinds, comes = graph(name, lines, body)
        waits = [k for k, v in enumerate(kinds) if isinstance(v, int)]
        first = [k for k in waits if any(w is None for w, _ in ways(kinds, comes, k, 64))]
        assert len(first) == 1 and len(waits) >= ring, name
        for k in waits:
            back = ways(kinds, comes, k, 64)
            if k in first:
                # all slots of the ring issued, the first one whole
                assert back == {(None, ring * loads)} and kinds[k] == (ring - 1) * loads, (name, back)
                continue
            assert kinds[k] == loads, (name, kinds[k])
            for wait, n in back:
                # (a ring of three is full when its first step waits)
                want = 0 if ring == 3 and wait in first else loads
                assert n == want, (name, k, wait, n)
            seen += 1
    assert seen >= 100, "the tile kernels were not found"
