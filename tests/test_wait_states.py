"""The built library's code (CPU: it is read, not run): wait states behind its
matrix instructions, and spilled registers. The hardware does not hold back an instruction that
uses the result of an MFMA too early; the compiler has to put enough
instructions or s_nop between the two on every path, and it has been seen not
to where a conditional block follows the MFMA at once. So the paths are walked
here: from every MFMA, through both sides of every branch, to the first use of
its result by anything but the accumulator input of a later MFMA (which is
interlocked)."""
import os
import re
import shutil
import subprocess

import pytest

import gated_delta_rule_74_amd as gdn

OBJDUMP, READOBJ = ("/opt/rocm/llvm/bin/" + t for t in ("llvm-objdump", "llvm-readobj"))
REG = re.compile(r"\b([va])\[(\d+):(\d+)\]|\b([va])(\d+)\b")


def needed(op):
    """Wait states between an MFMA and a use of its result: passes + 2 for fp32
    operands (16x16x4: 8 passes), passes + 4 for bf16 (16x16x16 and 16x16x32: 4 passes)."""
    return 8 + 2 if op.endswith("x4_f32") else 4 + 4


def regs(*operands):
    out = set()
    for o in operands:
        for m in REG.finditer(o):
            if m.group(1):
                out.update((m.group(1), i) for i in range(int(m.group(2)), int(m.group(3)) + 1))
            else:
                out.add((m.group(4), int(m.group(5))))
    return out


def kernels(listing):
    """{name: [(mnemonic, operands, address, branch target or None)]} of an llvm-objdump listing."""
    out, name, base = {}, None, 0
    for line in listing.splitlines():
        m = re.match(r"([0-9a-f]+) <(\S+)>:", line)
        if m:
            base, name = int(m.group(1), 16), m.group(2)
            out[name] = []
            continue
        m = re.match(r"\t(\S+)\s*(.*?)\s*// ([0-9A-F]+):.*?(?:<(\S+?)(?:\+0x([0-9a-f]+))?>)?$", line)
        if name and m:
            target = None if m.group(4) is None else base + int(m.group(5) or "0", 16)
            out[name].append((m.group(1), m.group(2).split(", "), int(m.group(3), 16), target))
    return out


def effects(op, args):
    """Registers an instruction reads (the accumulator input of an MFMA left out) and writes."""
    if op.startswith("v_mfma"):
        return regs(*args[1:3]), regs(args[0])
    if op.startswith(("ds_write", "global_store", "scratch_store", "flat_store", "buffer_store")):
        return regs(*args), set()
    if not op.startswith(("v_", "ds_", "global_", "scratch_", "flat_", "buffer_")):
        return set(), set()
    if "swap" in op:
        return regs(*args), regs(*args[:2])
    return regs(*args[1:]), regs(args[0])


def early_uses(code):
    """(MFMA, use, wait states) of every use that comes too early on some path."""
    at, found = {c[2]: i for i, c in enumerate(code)}, []
    for i, (op, args, _, _) in enumerate(code):
        if not op.startswith("v_mfma"):
            continue
        want, paths, seen = needed(op), [(i + 1, 0, frozenset(regs(args[0])))], set()
        while paths:
            j, waited, live = paths.pop()
            if j >= len(code) or waited >= want or not live or (j, waited, live) in seen:
                continue
            seen.add((j, waited, live))
            o, a, _, target = code[j]
            reads, writes = effects(o, a)
            # (a vector instruction's write of the register is as early as its read; an MFMA's is in order)
            if reads & live or (writes & live and not o.startswith("v_mfma")):
                found.append((op + " " + ", ".join(args), o + " " + ", ".join(a), waited))
                continue
            live, waited = live - writes, waited + (int(a[0]) + 1 if o == "s_nop" else 1)
            if o == "s_endpgm":
                continue
            if o.startswith(("s_cbranch", "s_branch")):
                paths.append((at[target], waited, live))
            if o != "s_branch":
                paths.append((j + 1, waited, live))
    return found


LINES = """0000000000001000 <kernel>:
\tv_mfma_f32_16x16x32_bf16 v[0:3], v[4:7], v[8:11], 0 // 000000001000: D3B50000 02021104
\ts_cbranch_scc1 3 // 000000001008: BF850003 <kernel+0x14>
{filler}
\tv_add_f32_e32 v20, v1, v21 // 000000001014: 02282B01
\ts_endpgm // 000000001018: BF810000
"""


def test_the_walk_finds_an_early_use_behind_a_branch():
    """A use behind a skipped block that hides it from a reader of straight lines; none behind a longer one."""
    quick = LINES.format(filler="\ts_nop 7 // 00000000100C: BF800007")
    (mfma, use, waited), = early_uses(kernels(quick)["kernel"])
    assert mfma.startswith("v_mfma") and use.startswith("v_add") and waited == 1
    slow = quick.replace("s_cbranch_scc1 3", "s_nop 7").replace(" <kernel+0x14>", "")
    assert not early_uses(kernels(slow)["kernel"])
    acc = quick.replace("v_add_f32_e32 v20, v1, v21", "v_mfma_f32_16x16x32_bf16 v[0:3], v[30:33], v[34:37], v[0:3]")
    assert not early_uses(kernels(acc)["kernel"])


def code_objects(tmp_path):
    """The library's gfx950 code objects, one per source."""
    gdn.lib()  # (raises if it has not been built)
    shutil.copy(gdn.LIB_PATH, tmp_path / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=tmp_path, check=True, capture_output=True)
    return sorted(tmp_path.glob("lib.so.*gfx950*"))


@pytest.mark.skipif(not os.path.exists(READOBJ), reason="no llvm-readobj")
def test_attention_backward_keeps_its_registers(tmp_path):
    """What the key-gradient kernels spill stays where two waves per SIMD were measured to be worth it."""
    spilled = {}
    for f in code_objects(tmp_path):
        notes = subprocess.run([READOBJ, "--notes", str(f)], check=True, capture_output=True, text=True).stdout
        spilled.update(re.findall(r"\.name: +(\S*mla_bwd_k_kernel\S*)\n\s+\.private_segment_fixed_size: (\d+)", notes))
    assert len(spilled) > 20
    assert max(int(n) for n in spilled.values()) <= 160, spilled


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump")
def test_no_mfma_result_is_used_too_early(tmp_path):
    products, bad = 0, []
    for f in code_objects(tmp_path):
        listing = subprocess.run([OBJDUMP, "-d", "--mcpu=gfx950", str(f)], check=True, capture_output=True,
                                 text=True).stdout
        for name, code in kernels(listing).items():
            products += sum(c[0].startswith("v_mfma") for c in code)
            bad += [(name,) + x for x in early_uses(code)]
    assert products > 1000  # (the listing was understood)
    assert not bad, f"{len(bad)} uses, first: {bad[0]}; kernels {sorted({b[0] for b in bad})}"
