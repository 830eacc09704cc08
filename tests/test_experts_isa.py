"""The waits that the experts' kernels owe the hardware, read from the assembly
that the compiler makes of them (CPU; needs hipcc, no GPU).

gfx950 does not hold a vector memory instruction back until a scalar register
that a vector instruction wrote (v_readfirstlane, v_readlane, a compare) has
its new value: five wait states have to lie between them.  It neither holds a
load into LDS back for a fresh M0: one wait state.  The compiler places them
for its own instructions and not for those inside inline assembly, so every
load into LDS is followed back through the control flow here.  An instruction
is one wait state, s_nop n is n + 1.
"""
import os
import re
import shutil
import subprocess

import pytest

from combine_layout_amd import build

VMEM_SGPR, LDS_M0 = 5, 1
BRANCH = re.compile(r"s_(branch|cbranch_\w+)$")


def registers(operand):
    """The scalar registers of one operand."""
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    if m:
        return {f"s{i}" for i in range(int(m[1]), int(m[2]) + 1)}
    if re.fullmatch(r"s\d+|m0", operand):
        return {operand}
    m = re.fullmatch(r"vcc(_lo|_hi)?", operand)
    return {"vcc"} if m else set()


def parse(text):
    """Functions of an assembly text: name -> blocks [(label, instructions)],
    an instruction being (mnemonic, operands, line)."""
    out, name, blocks = {}, None, None
    for at, raw in enumerate(text.split("\n"), 1):
        line = raw.split(";")[0].strip()
        m = re.fullmatch(r"(_Z\w+|k_\w+):", line)
        if m:
            name, blocks = m[1], [("", [])]
            out[name] = blocks
        elif name is None or not line:
            continue
        elif re.fullmatch(r"\.L\w+:", line):
            if line.startswith(".Lfunc_end"):
                name = None
            else:
                blocks.append((line[:-1], []))
        elif not line.startswith("."):
            op, _, rest = line.partition(" ")
            blocks[-1][1].append((op, [o.strip() for o in rest.split(",")], at))
            if BRANCH.match(op) or op == "s_endpgm":
                blocks.append((f"behind {at}", []))
    return out


def written(op, operands):
    """Scalar registers that a vector instruction writes."""
    if not op.startswith("v_"):
        return set()
    regs = registers(operands[0])
    if "_co_" in op or "div_scale" in op:
        regs |= registers(operands[1])
    return regs


def faults(blocks):
    """(line, instruction, register, wait states) of every load into LDS that
    comes too soon after a write of a register that it reads, and the loads."""
    index = {label: i for i, (label, _) in enumerate(blocks)}
    # per block: register -> wait states since a vector instruction wrote it (a scalar one, of M0)
    entry = [None] * len(blocks)
    entry[0] = {}
    todo, found, loads = [0], set(), set()
    while todo:
        i = todo.pop()
        age, targets, falls = dict(entry[i]), [], True
        for op, operands, line in blocks[i][1]:
            if op.startswith("buffer_load") and operands[-1].split()[-1] == "lds":
                loads.add(line)
                for reg in set().union(*(registers(w) for o in operands for w in o.split())):
                    if age.get(reg, VMEM_SGPR) < VMEM_SGPR:
                        found.add((line, op, reg, age[reg]))
                if age.get("m0", LDS_M0) < LDS_M0:
                    found.add((line, op, "m0", age["m0"]))
            step = int(operands[0], 0) + 1 if op == "s_nop" else 1
            age = {r: n + step for r, n in age.items() if n + step < VMEM_SGPR}
            for reg in written(op, operands):
                age[reg] = 0
            if op.startswith("s_") and operands and op not in ("s_nop", "s_waitcnt"):
                for reg in registers(operands[0]) - ({"vcc"} if op.startswith(("s_cmp", "s_bitcmp")) else set()):
                    age.pop(reg, None)      # now a scalar instruction's, which the hardware waits for
                    if reg == "m0":
                        age[reg] = 0
            if BRANCH.match(op):
                targets.append(index[operands[0]])
                falls = op != "s_branch"
            elif op == "s_endpgm":
                falls = False
        if falls and i + 1 < len(blocks):
            targets.append(i + 1)
        for t in targets:
            if entry[t] is None:
                new = age
            else:
                new = dict(entry[t])
                for reg, n in age.items():
                    new[reg] = min(n, new.get(reg, VMEM_SGPR))
            if new != entry[t]:
                entry[t] = new
                todo.append(t)
    return sorted(found), loads


def left_at_barriers(blocks):
    """The most LDS operations (scalar loads counted with them, as the hardware
    does) that a wavefront can still have under way at each barrier: line -> number."""
    index = {label: i for i, (label, _) in enumerate(blocks)}
    entry, todo, left = [None] * len(blocks), [0], {}
    entry[0] = 0
    while todo:
        i = todo.pop()
        n, targets, falls = entry[i], [], True
        for op, operands, line in blocks[i][1]:
            if op.startswith(("ds_", "s_load", "s_buffer_load")):
                n = min(n + 1, 15)
            elif op == "s_waitcnt":
                m = re.search(r"lgkmcnt\((\d+)\)", " ".join(operands))
                n = min(n, int(m[1])) if m else n
            elif op == "s_barrier":
                left[line] = max(left.get(line, 0), n)
            if BRANCH.match(op):
                targets.append(index[operands[0]])
                falls = op != "s_branch"
            elif op == "s_endpgm":
                falls = False
        if falls and i + 1 < len(blocks):
            targets.append(i + 1)
        for t in targets:
            if entry[t] is None or n > entry[t]:
                entry[t] = n
                todo.append(t)
    return left


GOOD = """
k_a:
\ts_cbranch_scc1 .LBB0_2
\tv_readfirstlane_b32 s4, v0
\ts_mov_b32 m0, s9
\ts_nop 3
\tbuffer_load_dwordx4 v1, s[4:7], s8 offen lds
.LBB0_2:
\ts_endpgm
.Lfunc_end0:
"""


def test_the_reader_finds_planted_faults():
    """The walk over the control flow itself, on a few lines."""
    def count(text):
        found, loads = faults(parse(text)["k_a"])
        assert len(loads) == 1
        return found
    assert count(GOOD) == []
    short = count(GOOD.replace("s_nop 3", "s_nop 2"))
    assert [(f[2], f[3]) for f in short] == [("s4", 4)]
    assert [(f[2], f[3]) for f in count(GOOD.replace("v_readfirstlane_b32 s4", "v_readlane_b32 s8"))] == []
    assert count(GOOD.replace("s_mov_b32 m0, s9\n\ts_nop 3", "s_nop 5\n\ts_mov_b32 m0, s9"))[0][2] == "m0"
    # a write in the block before, past the branch
    over = GOOD.replace("\ts_cbranch", "\tv_cmp_eq_u32 s[6:7], v0, v1\n\ts_cbranch").replace(
        "\tv_readfirstlane_b32 s4, v0\n", "").replace("s_nop 3", "s_nop 1")
    assert {(f[2], f[3]) for f in count(over)} == {("s6", 4), ("s7", 4)}


WAITED = """
k_b:
.LBB1_1:
\ts_barrier
\tds_read_b128 v[0:3], v4
\tds_read_b128 v[4:7], v8
\ts_waitcnt vmcnt(3) lgkmcnt(0)
\ts_cbranch_scc1 .LBB1_1
\ts_endpgm
"""


def test_the_reader_counts_what_is_left_at_a_barrier():
    assert left_at_barriers(parse(WAITED)["k_b"]) == {4: 0}
    assert left_at_barriers(parse(WAITED.replace("lgkmcnt(0)", "lgkmcnt(1)"))["k_b"]) == {4: 1}
    assert left_at_barriers(parse(WAITED.replace(" lgkmcnt(0)", ""))["k_b"]) == {4: 15}


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    hipcc = shutil.which(build.HIPCC)
    if not hipcc:
        pytest.skip("hipcc not installed")
    out = str(tmp_path_factory.mktemp("isa") / "experts.s")
    subprocess.check_call([hipcc, *[f for f in build.HIP_FLAGS if f != "-shared"], "-S", "--cuda-device-only",
                           os.path.join(build.CSRC, "afd_experts.hip"), "-o", out], stderr=subprocess.DEVNULL)
    with open(out) as f:
        return parse(f.read())


def test_loads_into_lds_wait_for_their_registers(kernels):
    seen, bad = 0, []
    for name, blocks in kernels.items():
        found, loads = faults(blocks)
        seen += len(loads)
        bad += [f"{name} line {line}: {op} reads {reg} after {n} wait states" for line, op, reg, n in found]
        if "k_product_many" in name:
            assert loads, f"{name}: no loads found"
    assert seen > 100
    assert not bad, f"{len(bad)} of {seen} loads:\n" + "\n".join(bad[:20])


def test_lds_reads_are_over_at_barriers(kernels):
    """A stage is loaded anew behind the barrier after its last read; the barrier is
    written in assembly, where the compiler adds no wait of its own."""
    seen = 0
    for name, blocks in kernels.items():
        left = left_at_barriers(blocks)
        seen += len(left)
        assert not any(left.values()), f"{name}: {left}"
    assert seen > 50
