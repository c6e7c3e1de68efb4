"""The tile kernels' counted waits, in the machine code of the built library.

A wavefront of a tile kernel waits before each barrier with `s_waitcnt
vmcnt(N)`, N vector-memory operations left in flight: those that the source
issues after the last load of the slot that is read next. Should the compiler
drop or reorder a load, N would count an older one, and a slot could be read
before it has arrived, which no run shows reliably. This disassembles the
library and follows every path of the loops backwards from each such wait.

In the code between two waits ("step") stand: the second part of a slot's loads
to LDS (`late` of them, issued behind the wait), then the first part of the next
slot's, and loads to registers. Behind the wait of step s the slot s + 1 is
read, whose last loads are the late ones of step s - 2 (rings of four slots) or
s - 1 (three). Small matmul tiles issue the two parts the other way round, so
that a slot's loads end with a step: those of slot s + 1 end RING - 2 steps back.
"""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "newton_schulz_04_amd", "libns.so")
OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
VM = re.compile(r"(buffer|global|flat|scratch)_(load|store|atomic)")


class Code:
    """A function's instructions: for each its kind (D a load to LDS, V other
    vector memory, an int the N of a counted wait, None), and the instructions
    that control may come from."""

    def __init__(self, name, lines, body):
        at = {addr: k for k, (_, addr) in enumerate(lines)}
        start = lines[0][1]
        self.kinds, self.comes = [], [[k - 1] if k else [] for k in range(len(lines))]
        for k, (text, addr) in enumerate(lines):
            op = text.split()[0]
            wait = re.fullmatch(r"s_waitcnt vmcnt\((\d+)\)", lines[k - 2][0]) if k > 1 and op == "s_barrier" else None
            if wait and lines[k - 1][0] == "s_waitcnt lgkmcnt(0)":
                self.kinds.append(int(wait.group(1)))
            elif VM.match(op):
                self.kinds.append("D" if text.endswith(" lds") else "V")
            else:
                self.kinds.append(None)
            if op in ("s_branch", "s_endpgm") and k + 1 < len(lines):
                self.comes[k + 1].remove(k)
            if op.startswith(("s_cbranch", "s_branch")):
                to = re.search(r"// %012X:.*?<%s(?:\+0x([0-9a-f]+))?>" % (addr, re.escape(name)), body)
                self.comes[at[start + int(to.group(1) or "0", 16)]].append(k)


def functions(tmp_path):
    lib = shutil.copy(LIB, tmp_path)
    subprocess.run([OBJDUMP, "--offloading", lib], check=True, capture_output=True, cwd=tmp_path)
    for part in sorted(os.listdir(tmp_path)):
        if "gfx950" not in part:
            continue
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", part], check=True, capture_output=True, text=True,
                              cwd=tmp_path).stdout
        for name, body in re.findall(r"^[0-9a-f]+ <(\S*k_q8_(?:big|mid)\S*)>:\n(.*?)(?=^\S|\Z)", text, re.M | re.S):
            lines = re.findall(r"^\t(.*?)\s*// ([0-9A-F]+):", body, re.M)
            yield name, [(t, int(a, 16)) for t, a in lines], body


def paths(code, at, first, steps):
    """All ways back from instruction `at` over at most `steps` steps: the
    steps' strings of D and V in program order, the oldest first, and whether
    they begin with the wait before the first step, whose N is `first`."""
    found, todo, met = set(), [(k, ("",)) for k in code.comes[at]], set()
    while todo:
        k, done = todo.pop()
        # (a loop on the way, such as one over outputs, is not a step)
        if (k, done) in met or len(done[0]) > 64:
            continue
        met.add((k, done))
        kind = code.kinds[k]
        if isinstance(kind, int):
            if kind == first or len(done) == steps:
                found.add((done, kind == first))
                continue
            done = ("",) + done
        elif kind:
            done = (kind + done[0],) + done[1:]
        todo += [(j, done) for j in code.comes[k]]
    return found


# (N before the first step: (N of a step, late loads, loads of a slot)): large
# matmul tiles and their halves, large gradient tiles (both), small ones. N may
# be less by the loads to registers in the steps behind a loop, which make none.
LARGE = {8: (12, 4, 8), 6: (9, 3, 6)}
LARGE_GRAD = {4: ((12, 10), 2, 0)}
SMALL_GRAD = {2: ((3, 1), 1, 0)}
SMALL = {10: (8, 0, 4), 6: (4, 0, 4)}


def test_every_wait_covers_the_slot_read_next(tmp_path):
    if not os.path.exists(OBJDUMP) or not os.path.exists(LIB):
        pytest.skip("the library or llvm-objdump is missing")
    kernels, waits, firsts = 0, 0, 0
    for name, lines, body in functions(tmp_path):
        kernels += 1
        large = "k_q8_big" in name
        matmul = re.search(r"k_q8_\w{3}ILi(\d)", name).group(1) == "0"
        back = 2 if large or "Li4EEEvNS" in name else 1   # (the ring's size is the last argument)
        forms = (LARGE if large else SMALL) if matmul else LARGE_GRAD if large else SMALL_GRAD
        code = Code(name, lines, body)
        for at, n in enumerate(code.kinds):
            if not isinstance(n, int):
                continue
            if n in forms:
                # the last slots' loads go last: whatever else is in flight, no
                # more of them than these
                firsts += 1
                continue
            fit = [(f, late, slot) for f, (ns, late, slot) in forms.items() if n in (ns if isinstance(ns, tuple) else (ns,))]
            assert len(fit) == 1, (name, at, n)
            first, late, slot = fit[0]
            ways = paths(code, at, first, back)
            assert ways, (name, at, n)
            for steps, begins in ways:
                if matmul and not large:
                    # a step ends with a slot's loads; of those in flight behind
                    # the first wait the slots that the steps since read are done
                    left = len("".join(steps)) + (max(0, first - len(steps) * slot) if begins else 0)
                elif len(steps) < back:
                    continue   # read from the first slots, which have arrived
                else:
                    # the oldest step's late loads, if it is not the first step
                    places = [k for k, c in enumerate(steps[0]) if c == "D"]
                    skip = 0 if begins else places[late - 1] + 1
                    left = len(steps[0][skip:] + "".join(steps[1:]))
                assert left >= n, (name, at, n, steps, begins)
                waits += 1
    assert kernels >= 12 and waits >= 60 and firsts >= 12, (kernels, waits, firsts)


def listing(steps, n):
    """A loop of `steps`, a string of D and V each behind a wait for n."""
    text = {"D": "buffer_load_dwordx4 v1, s[0:3], 0 offen lds", "V": "buffer_load_dword v2, v1, s[0:3], 0 offen"}
    lines = []
    for step in steps:
        lines += [f"s_waitcnt vmcnt({n})", "s_waitcnt lgkmcnt(0)", "s_barrier"] + [text[c] for c in step]
    lines += ["s_cbranch_scc1 7", "s_endpgm"]
    body = "".join(f"\t{t}   // {8 * k:012X}:" + (" 0 <f+0x0>\n" if "cbranch" in t else " 0\n")
                   for k, t in enumerate(lines))
    return body


@pytest.mark.parametrize("steps,back,ways", [
    (["DDV"] * 4, 2, {("DDV", "DDV")}), (["DDV", "VDD", "DDV", "DDV"], 1, {("DDV",), ("VDD",)}),
    (["DD", "DDV"], 2, {("DD", "DDV"), ("DDV", "DD")})])
def test_the_ways_back(steps, back, ways):
    body = listing(steps, 3)
    lines = [(t, int(a, 16)) for t, a in re.findall(r"^\t(.*?)\s*// ([0-9A-F]+):", body, re.M)]
    code = Code("f", lines, body)
    assert [k for k in code.kinds if isinstance(k, int)] == [3] * len(steps)
    got = set()
    for at, kind in enumerate(code.kinds):
        if isinstance(kind, int):
            got |= {way for way, begins in paths(code, at, None, back)}
    assert got == ways
