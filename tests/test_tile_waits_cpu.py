"""The counted waits of the tile kernels, in the code that the compiler made of them.

Before a step of the tile kernel's loop a wave waits until at most n of its memory operations are
outstanding, n being what the step before issued; operations retire in order, so the copies to LDS and the
loads of the steps before that have landed.  That holds as long as the step before really issued n: were
loads joined, moved or dropped, the wait would be too short and LDS would be read early.  Here the built
library is disassembled, and for every barrier behind such a wait the fewest memory operations on any way
to it from the barrier before (or from the kernel's start) are counted."""
import os
import re
import struct
import subprocess
from collections import deque

import pytest

import block_quantized_matmul_gguf_amd as qmm

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
MEMORY = re.compile(r"(global|buffer|flat|scratch)_(load|store|atomic)")


def code_objects(path):
    """The gfx950 code objects of a library's offload bundles."""
    data, magic, at = open(path, "rb").read(), b"__CLANG_OFFLOAD_BUNDLE__", 0
    while (at := data.find(magic, at)) >= 0:
        count, = struct.unpack_from("<Q", data, at + len(magic))
        p = at + len(magic) + 8
        for _ in range(count):
            offset, size, length = struct.unpack_from("<QQQ", data, p)
            if b"gfx950" in data[p + 24:p + 24 + length] and size:
                yield data[at + offset:at + offset + size]
            p += 24 + length
        at += len(magic)


def kernels(path):
    """{name: [(address, text)]} of the tile kernels in a code object's disassembly."""
    out, name = {}, None
    text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", path], check=True, capture_output=True, text=True).stdout
    for line in text.splitlines():
        head = re.match(r"[0-9a-f]+ <(.*)>:$", line)
        if head:
            name = head.group(1)
            continue
        part = re.match(r"\s+(\S.*?)\s*// ([0-9A-F]+):(.*)$", line)
        if part and name and "moe_tile" in name:
            out.setdefault(name, []).append((int(part.group(2), 16), part.group(1), part.group(3)))
    return out


def successors(code):
    """For each instruction the indices of those that may follow it."""
    at, first = {a: i for i, (a, _, _) in enumerate(code)}, code[0][0]
    follow = []
    for i, (_, text, note) in enumerate(code):
        op = text.split()[0]
        if op == "s_endpgm":
            follow.append([])
            continue
        assert not op.startswith(("s_setpc", "s_swappc", "s_call")), text
        to = []
        if op.startswith(("s_branch", "s_cbranch")):
            plus = re.search(r"<[^>+]*(?:\+0x([0-9a-f]+))?>", note)
            to.append(at[first + int(plus.group(1) or "0", 16)])
        if op != "s_branch":
            to.append(i + 1)
        follow.append([j for j in to if j < len(code)])
    return follow


def waits(code):
    """(wait's count, fewest memory operations since the last barrier or the start) at each counted wait."""
    before = [[] for _ in code]
    for i, to in enumerate(successors(code)):
        for j in to:
            before[j].append(i)
    found = []
    for b, (_, text, _) in enumerate(code):
        if text.split()[0] != "s_barrier":
            continue
        i = b - 1
        while i > 0 and not re.match(r"s_waitcnt.*vmcnt|s_barrier|s_c?branch", code[i][1]):
            assert not MEMORY.match(code[i][1]), code[i]  # nothing is issued between the wait and its barrier
            i -= 1
        count = re.match(r"s_waitcnt.*vmcnt\((\d+)\)", code[i][1])
        count = int(count.group(1)) if count else 0
        if count == 0:
            continue  # no wait for memory, or one for all of it
        # shortest ways backwards, whose steps cost 0 or 1
        best, queue, fewest = {}, deque((k, 0) for k in before[i]), None
        while queue and fewest is None:
            j, cost = queue.popleft()
            if best.get(j, 1 << 30) <= cost:
                continue
            best[j] = cost
            if j == 0 or code[j][1].split()[0] == "s_barrier":
                fewest = cost
            elif MEMORY.match(code[j][1]):
                queue.extend((k, cost + 1) for k in before[j])
            else:
                queue.extendleft((k, cost) for k in before[j])
        found.append((count, fewest))
    return found


def test_counted_waits_are_never_too_short(tmp_path):
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    qmm.lib()
    seen = {}
    for n, obj in enumerate(code_objects(qmm.LIB_PATH)):
        if b"moe_tile" not in obj:
            continue
        path = tmp_path / f"{n}.elf"
        path.write_bytes(obj)
        for name, code in kernels(str(path)).items():
            seen[name] = waits(code)
    assert len(seen) >= 33  # five formats with five kernels each, four kinds of 4-bit groups with two
    for name, found in seen.items():
        # two bodies (f32) or three, two steps a loop; where a step's weights have to be there as well the
        # compiler adds a wait for everything
        assert len(found) >= (2 if "ELi2EL" in name else 3), (name, found)
        for count, fewest in found:
            assert fewest is not None and fewest >= count, (name, found)


def test_a_wait_that_is_too_short_is_seen():
    """The count itself, on a loop of its own making: five loads a turn, one way round without the last."""
    def listing(n):
        lines = ["s_mov_b32 s0, 4"] + ["global_load_dword v1, v[2:3], off"] * 8
        lines += ["s_waitcnt vmcnt(%d)" % n, "s_waitcnt lgkmcnt(0)", "s_barrier"] + ["global_load_dword v1, v[2:3], off"] * 4
        lines += ["s_cbranch_scc0 1", "global_load_lds_dwordx4 v[2:3], off", "s_cbranch_scc1 65500", "s_endpgm"]
        code = [(256 + 4 * i, t, "") for i, t in enumerate(lines)]
        skip, back = 9 + 3 + 4, len(lines) - 2
        code[skip] = (code[skip][0], lines[skip], f"  <k+0x{4 * back:x}>")
        code[back] = (code[back][0], lines[back], f"  <k+0x{4 * 9:x}>")
        return code
    assert waits(listing(4)) == [(4, 4)]
    assert waits(listing(5)) == [(5, 4)]
