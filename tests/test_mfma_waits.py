"""The waits between matrix instructions and the instructions that read or overwrite
their results, on every path through the built kernels.

The hardware does not hold a vector instruction back until a matrix result is
written: the compiler counts wait states and puts s_nop between them.  It has been
seen to count along one of two paths only, where a branch follows the matrix
instruction and both ways read its result: the kernel then took old values on the
other.  This follows each path in the disassembly of the library's own kernels."""
import os
import re
import struct
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "dsa_lightning_indexer_03_amd", "libdsaidx.so")
OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"

# wait states until a result may be touched, by the instruction's passes (4, 8, 8 with 8-bit operands)
WAITS = {"16x16x32": 8, "32x32x16": 12, "16x16x128": 12}
READERS = ("v_", "ds_", "global_", "buffer_", "flat_", "scratch_")


def registers(text):
    out = set()
    for lo, hi, one in re.findall(r"\bv\[(\d+):(\d+)\]|\bv(\d+)\b", text):
        out.update([int(one)] if one else range(int(lo), int(hi) + 1))
    return out


def kernels(path):
    """{name: [(address, mnemonic, operands, branch target or None)]} of a code object."""
    dump = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", path], capture_output=True, text=True, check=True).stdout
    return parse(dump)


def parse(dump):
    found, rows, start = {}, None, 0
    for line in dump.splitlines():
        head = re.match(r"^([0-9a-f]+) <(.*)>:$", line)
        if head:
            rows, start = found.setdefault(head.group(2), []), int(head.group(1), 16)
            continue
        row = re.match(r"^\s+(\S+)\s*(.*?)\s*// ([0-9A-F]+):(.*)$", line)
        if row and rows is not None:
            to = re.search(r"<.*?(?:\+0x([0-9a-f]+))?>", row.group(4))
            rows.append((int(row.group(3), 16), row.group(1), row.group(2),
                         start + int(to.group(1) or "0", 16) if to else None))
    return found


def too_early(rows):
    """(matrix instructions, [(one, the instruction that touches its result, states between them)])."""
    where = {address: i for i, (address, *_) in enumerate(rows)}
    touched = [registers(ops) for _, _, ops, _ in rows]
    bad, count = [], 0
    for i, (_, name, ops, _) in enumerate(rows):
        if not name.startswith("v_mfma"):
            continue
        count += 1
        need = WAITS[re.search(r"\d+x\d+x\d+", name).group()]
        result = registers(ops.split(",")[0])
        seen, paths = {}, [(i + 1, 0)]
        while paths:
            j, states = paths.pop()
            while j < len(rows) and states < need and seen.get(j, need) > states:
                seen[j] = states
                _, other, text, to = rows[j]
                if other.startswith("v_mfma"):
                    args = [registers(x) for x in re.findall(r"v\[\d+:\d+\]|v\d+|[^,\s]+", text)]
                    if (args[1] | args[2]) & result:
                        bad.append((f"{name} {ops}", f"{other} {text}", states))
                        break
                    if args[0] & result:   # (accumulated on, or written over by another: interlocked)
                        break
                elif other.startswith(READERS) and touched[j] & result:
                    bad.append((f"{name} {ops}", f"{other} {text}", states))
                    break
                states += int(text, 0) + 1 if other == "s_nop" else 1
                if other in ("s_endpgm", "s_setpc_b64"):
                    break
                if other == "s_branch":
                    j = where[to]
                    continue
                if other.startswith("s_cbranch"):
                    paths.append((where[to], states))
                j += 1
    return count, bad


SAMPLE = """
0000000000000100 <f>:
	v_mfma_f32_16x16x32_bf16 v[4:7], v[8:11], v[12:15], v[4:7]  // 000000000100: D3B50004 04120908
	s_cbranch_scc1 {skip}                                      // 000000000108: BF850001 <f+0x{to}>
	s_nop 7                                                    // 00000000010C: BF800007
	v_mul_f32_e32 v1, v2, v7                                   // 000000000110: 0A020F02
	s_endpgm                                                   // 000000000114: BF810000
"""


def test_the_walk():
    """A branch past the wait is found; one that goes past the reader too is not."""
    count, bad = too_early(parse(SAMPLE.format(skip=1, to="10"))["f"])
    assert count == 1 and [x[2] for x in bad] == [1] and "v_mul_f32" in bad[0][1]
    assert too_early(parse(SAMPLE.format(skip=2, to="14"))["f"]) == (1, [])


def test_no_result_is_touched_early(tmp_path):
    if not os.path.exists(LIB):
        pytest.skip("libdsaidx.so not built")
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    with open(LIB, "rb") as f:
        data = f.read()
    magic, total, wrong = b"__CLANG_OFFLOAD_BUNDLE__", 0, []
    at = data.find(magic)
    while at >= 0:
        entry = at + 32
        for _ in range(struct.unpack_from("<Q", data, at + 24)[0]):
            offset, size, length = struct.unpack_from("<QQQ", data, entry)
            target = data[entry + 24:entry + 24 + length]
            entry += 24 + length
            if b"gfx950" in target and size:
                path = str(tmp_path / "object")
                with open(path, "wb") as f:
                    f.write(data[at + offset:at + offset + size])
                for name, rows in kernels(path).items():
                    count, bad = too_early(rows)
                    total += count
                    wrong += [(name, *x) for x in bad]
        at = data.find(magic, at + 24)
    assert total > 5000 and not wrong, f"{len(wrong)} of {total}: {wrong[:3]}"
