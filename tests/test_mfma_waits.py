"""The wait states behind matrix instructions, read from the disassembly of the built library.

A matrix instruction's result may be read or overwritten by another kind of instruction only some
wait states after its issue: the hardware does not check, and an early reader gets the accumulator
without that instruction's share.  The compiler inserts the wait states; a build of an 8-bit integer
product once had none on the path out of its loop.  Here every path behind every matrix
instruction of the 8-bit integer kernels is followed until they have passed."""
import os
import re
import shutil
import struct
import subprocess

import pytest

import precision_quantized_linear_amd as qpl

OBJDUMP = next((p for p in ("/opt/rocm/llvm/bin/llvm-objdump", shutil.which("llvm-objdump") or "") if os.path.exists(p)),
               None)
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"
# wait states behind the instruction: passes + 4 (one pass is four cycles)
WAITS = {"v_mfma_i32_16x16x64_i8": 8, "v_mfma_i32_32x32x32_i8": 12}
ISSUE = 4   # at least what a matrix instruction occupies the unit for: four passes


def registers(text):
    """Names of the vector registers in an operand list: v[4:7], a12, ..."""
    out = set()
    for kind, lo, hi in re.findall(r"\b([va])\[(\d+):(\d+)\]", text):
        out |= {f"{kind}{i}" for i in range(int(lo), int(hi) + 1)}
    out |= {k + n for k, n in re.findall(r"\b([va])(\d+)\b", text)}
    return out


def early_reads(ins):
    """(instruction, reader) pairs that stand too close, along every path.  ins: [(address, text,
    branch target or None)] in order of address."""
    at = {a: i for i, (a, _, _) in enumerate(ins)}
    bad = []
    for i, (_, text, _) in enumerate(ins):
        op = text.split()[0]
        if not op.startswith("v_mfma"):
            continue
        need, dst = WAITS[op], registers(text.split(",")[0])
        seen, todo = {}, [(i + 1, 0)]
        while todo:
            j, waited = todo.pop()
            if waited >= need or j >= len(ins) or seen.get(j, need) <= waited:
                continue
            seen[j] = waited
            _, t, target = ins[j]
            o, _, args = t.partition(" ")
            if o == "s_endpgm":
                continue
            if target is not None:
                todo.append((at[target], waited + 1))
                if o == "s_branch":
                    continue
            if o.startswith("v_mfma"):
                todo.append((j + 1, waited + ISSUE))     # accumulation into the same registers is interlocked
                continue
            if not o.startswith("s_") and registers(args) & dst:
                bad.append((text, t))
                continue
            todo.append((j + 1, waited + (1 + int(args, 0) if o == "s_nop" else 1)))
    return bad


def code_objects(path):
    """The gfx950 code objects that a library carries, as bytes."""
    data = open(path, "rb").read()
    out, pos = [], data.find(MAGIC)
    while pos >= 0:
        p = pos + len(MAGIC)
        (n,) = struct.unpack_from("<Q", data, p)
        p += 8
        for _ in range(n):
            off, size, ln = struct.unpack_from("<QQQ", data, p)
            name = data[p + 24:p + 24 + ln]
            p += 24 + ln
            if b"gfx950" in name and size:
                out.append(data[pos + off:pos + off + size])
        pos = data.find(MAGIC, pos + 1)
    return out


def kernels(objects, match="k_int8_"):
    """{symbol: [(address, text, branch target or None)]} of the kernels whose name holds `match`."""
    out = {}
    for obj in objects:
        if match.encode() not in obj:
            continue
        r = subprocess.run([OBJDUMP, "-d", "-"], input=obj, capture_output=True)
        if r.returncode != 0:
            raise RuntimeError(r.stderr.decode())
        cur = None
        for line in r.stdout.decode().splitlines():
            m = re.match(r"^([0-9a-f]+) <(\S+)>:$", line)
            if m:
                cur, start = (out.setdefault(m.group(2), []) if match in m.group(2) else None), int(m.group(1), 16)
                continue
            m = re.match(r"^\t(.+?)\s*// ([0-9A-F]+): [0-9A-F ]+(?:<\S+?(?:\+0x([0-9a-f]+))?>)?$", line)
            if cur is None or not m:
                continue
            text, addr = m.group(1), int(m.group(2), 16)
            branch = text.startswith(("s_branch", "s_cbranch"))
            cur.append((addr, text, start + int(m.group(3) or "0", 16) if branch else None))
    return out


def listing(text):
    """[(address, text, target)] of a listing with labels, one address per instruction."""
    lines = [l.strip() for l in text.strip().splitlines()]
    labels, ins = {}, []
    for l in lines:
        if l.endswith(":"):
            labels[l[:-1]] = len(ins)
        else:
            ins.append(l)
    return [(i, l, labels[l.split()[1]] if l.startswith(("s_branch", "s_cbranch")) else None) for i, l in enumerate(ins)]


LOOP = """
top:
  v_mfma_i32_16x16x64_i8 v[4:7], v[8:11], v[12:15], v[4:7]
  s_cbranch_scc1 top
  {behind}
  ds_write_b128 v20, v[4:7]
  s_endpgm
"""


@pytest.mark.parametrize("behind,found", [("s_mov_b32 s0, s1", 1), ("s_nop 5", 1), ("s_nop 7", 0), ("s_nop 15", 0),
                                          ("v_add_u32_e32 v5, v5, v5", 1), ("v_mov_b32_e32 v21, v22", 1)])
def test_the_scan_finds_early_readers(behind, found):
    assert len(early_reads(listing(LOOP.format(behind=behind)))) == found


def test_the_scan_follows_branches():
    far = """
  v_mfma_i32_32x32x32_i8 a[0:15], v[8:11], v[12:15], a[0:15]
  s_cbranch_scc0 out
  s_nop 15
  s_endpgm
out:
  s_nop 3
  v_accvgpr_read_b32 v0, a15
  s_endpgm
"""
    assert len(early_reads(listing(far))) == 1
    assert not early_reads(listing(far.replace("s_nop 3", "s_nop 11")))


@pytest.mark.skipif(OBJDUMP is None, reason="no llvm-objdump")
def test_no_reader_stands_too_close():
    found = kernels(code_objects(qpl.LIB_PATH))
    count = {n: sum(t.startswith("v_mfma") for _, t, _ in ins) for n, ins in found.items()}
    assert sum(c > 0 for c in count.values()) >= 40 and all(len(ins) > 50 for ins in found.values())
    assert all(op in WAITS for ins in found.values() for _, t, _ in ins for op in [t.split()[0]] if "mfma" in op)
    bad = {n: early_reads(ins)[:3] for n, ins in found.items() if early_reads(ins)}
    assert not bad
