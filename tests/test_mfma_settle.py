"""What the grouped products' inline asm leaves to its kernels, read off the assembly built from
gmm.hip (CPU only, no GPU).  The persistent kernel multiplies in asm, so the compiler inserts no wait
states between a matrix product and the first use of its accumulators: in every such kernel the settle
names all the accumulators, and no other instruction touches one between its product and the settle.
The DMAs set m0, a register that a clobber list cannot name (it is reserved: the compiler keeps no
value in it, and sets it right before an instruction of its own that reads it): no code outside the asm
uses it at all."""
import os
import re
import subprocess

import pytest

from nvfp4_block_scaled_mxfp8_amd.build import CSRC, HIPCC_FLAGS, hipcc


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    """The lines of gmm.hip's device code."""
    out = str(tmp_path_factory.mktemp("asm") / "gmm.s")
    flags = [f for f in HIPCC_FLAGS if f not in ("-fPIC", "-shared")]
    r = subprocess.run([hipcc()] + flags + ["--cuda-device-only", "-S", os.path.join(CSRC, "gmm.hip"), "-o", out],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    return open(out).read().splitlines(keepends=True)


@pytest.fixture(scope="module")
def kernels(assembly):
    """{kernel name: its lines} of the stream kernels."""
    found, name = {}, None
    for line in assembly:
        m = re.match(r"(_Z\S*gmm_stream_kernel\S*):", line)
        if m:
            name = m.group(1)
            found[name] = []
        elif line.startswith(".Lfunc_end"):
            name = None
        elif name:
            found[name].append(line)
    assert len(found) == 10, sorted(found)          # two types, forward, dgrad and three kinds of wgrad
    return found


def _regs(text):
    """Vector registers that an instruction's operands name."""
    r = set()
    for a, b in re.findall(r"\bv\[(\d+):(\d+)\]", text):
        r.update(range(int(a), int(b) + 1))
    r.update(int(a) for a in re.findall(r"\bv(\d+)\b", text))
    return r


def _blocks(lines):
    """Basic blocks: {label: (instructions as (text, in inline asm), successors)}, the entry's label ""."""
    blocks, order, in_asm = {"": []}, [""], False
    for line in lines:
        if "#ASMSTART" in line or "#ASMEND" in line:
            in_asm = "#ASMSTART" in line
            continue
        m = re.match(r"(\.LBB\S+):", line)
        if m:
            order.append(m.group(1))
            blocks[order[-1]] = []
            continue
        code = line.strip() if "; settled" in line else line.split(";")[0].strip()
        if code and not code.startswith(".") and not code.endswith(":"):
            blocks[order[-1]].append((code, in_asm))
            if not in_asm and re.match(r"s_c?branch|s_endpgm", code):
                order.append(order[-1] + "+")          # what follows the branch
                blocks[order[-1]] = []
    flow = {}
    for at, label in enumerate(order):
        last = blocks[label][-1][0] if blocks[label] and not blocks[label][-1][1] else ""
        to = [last.split()[-1]] if re.match(r"s_c?branch", last) else []
        if not re.match(r"s_branch|s_endpgm", last) and at + 1 < len(order):
            to.append(order[at + 1])
        flow[label] = (blocks[label], to)
    return flow


def test_accumulators_are_settled_before_they_are_read(kernels):
    for name, lines in kernels.items():
        flow = _blocks(lines)
        settles = [c for code, _ in flow.values() for c, _ in code if "; settled" in c]
        assert len(settles) == 1 and len(_regs(settles[0].split("; settled")[1])) == 128, (name, settles)
        before, todo = {label: set() for label in flow}, set(flow)
        while todo:                                     # registers that a product may still be writing
            label = todo.pop()
            code, to = flow[label]
            hot = set(before[label])
            for c, in_asm in code:
                if "; settled" in c:
                    assert hot <= _regs(c.split("; settled")[1]), (name, "accumulators that the settle leaves out", sorted(hot))
                    hot = set()
                elif in_asm and c.startswith("v_mfma"):
                    hot |= _regs(c.split(",")[0])
                elif hot:
                    assert not (_regs(c) & hot), (name, "touched before it is settled", c)
            for t in to:
                if not hot <= before[t]:
                    before[t] |= hot
                    todo.add(t)


def test_no_other_code_uses_m0(assembly):
    in_asm, set_by_asm = False, 0
    for line in assembly:
        if "#ASMSTART" in line or "#ASMEND" in line:
            in_asm = "#ASMSTART" in line
            continue
        code = line.split(";")[0].strip()
        if re.search(r"\bm0\b", code) and not code.startswith("."):
            assert in_asm and code.startswith("s_mov_b32 m0,"), code
            set_by_asm += 1
    assert set_by_asm > 100
