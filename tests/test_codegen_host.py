"""CPU test of the built kernels' instructions: the loads that go straight to LDS
are written as inline assembly, so the wait states in front of them are the
sources' to keep (CDNA3 and CDNA4 instruction set references, "Manually inserted
wait states"):

  * one between a scalar write of M0 and the load that takes its LDS address
    from there;
  * five between a vector instruction's write of a scalar register and the load
    that reads it as its descriptor or offset.

Every instruction takes one wait state, s_nop N takes N + 1.  All ways through
the code that end in such a load are walked backwards, branches included.
"""
import os
import re
import struct
import subprocess

import pytest

import linear_cross_entropy_gemm_amd as L

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
LIB = os.path.join(os.path.dirname(L.__file__), "libflce.so")

_LINE = re.compile(r"^\t(\S+)\s*(.*?)\s*// ([0-9A-F]+):(?: [0-9A-F]{8})+(?: <(\S+)\+0x([0-9a-f]+)>)?")


def code_objects(path):
    """The gfx950 code objects that the library carries, one per source."""
    data, out, i = open(path, "rb").read(), [], 0
    magic = b"__CLANG_OFFLOAD_BUNDLE__"
    while (i := data.find(magic, i)) >= 0:
        p = i + 32
        for _ in range(struct.unpack_from("<Q", data, i + 24)[0]):
            off, size, n = struct.unpack_from("<QQQ", data, p)
            if b"gfx950" in data[p + 24:p + 24 + n] and size:
                out.append(data[i + off:i + off + size])
            p += 24 + n
        i += len(magic)
    return out


def _scalars(operand):
    m = re.fullmatch(r"s(\d+)|s\[(\d+):(\d+)\]", operand)
    if not m:
        return set()
    return {int(m[1])} if m[1] else set(range(int(m[2]), int(m[3]) + 1))


def early_loads(listing):
    """(number of loads to LDS, those that come too early) in a disassembly."""
    ins, symbols = [], {}
    for line in listing:
        if m := re.match(r"^([0-9a-f]+) <(.*)>:", line):
            symbols[m[2]] = int(m[1], 16)
            ins.append(None)
        elif m := _LINE.match(line):
            ins.append((int(m[3], 16), m[1], [x.strip() for x in m[2].split(",")], m[4], m[5]))
    where = {x[0]: i for i, x in enumerate(ins) if x}
    jumps = {}
    for i, x in enumerate(ins):
        if x and x[1].startswith(("s_branch", "s_cbranch")):
            jumps.setdefault(where[symbols[x[3]] + int(x[4], 16)], []).append(i)
    loads, early = 0, set()
    for i, x in enumerate(ins):
        if not x or not x[1].startswith("buffer_load") or x[2][-1].split()[-1] != "lds":
            continue
        loads += 1
        read = _scalars(x[2][1]) | _scalars(x[2][2].split()[0])
        ways, seen = [(i, 0)], set()
        while ways:
            at = ways.pop()
            j, waited = at
            if at in seen or waited >= 5:
                continue
            seen.add(at)
            before = list(jumps.get(j, ()))
            if j and ins[j - 1] and ins[j - 1][1] not in ("s_branch", "s_endpgm"):
                before.append(j - 1)
            for k in before:
                _, op, args, _, _ = ins[k]
                if waited < 1 and args[0] == "m0":
                    early.add((hex(x[0]), op, "m0"))
                if op.startswith("v_") and (args[0] == "m0" or _scalars(args[0]) & read):
                    early.add((hex(x[0]), op, args[0]))
                ways.append((k, waited + (int(args[0], 0) + 1 if op == "s_nop" else 1)))
    return loads, sorted(early)


def _listing(*code):
    out = ["0000000000001000 <kernel>:"]
    for i, c in enumerate(code):
        out.append(f"\t{c}  // {0x1000 + 4 * i:012X}: 00000000" + (" <kernel+0x8>" if "branch" in c else ""))
    return out


@pytest.mark.parametrize("code, early", [
    (("s_mov_b32 m0, s1", "buffer_load_dwordx4 v0, s[4:7], 0 offen lds"), 1),
    (("s_mov_b32 m0, s1", "s_nop 0", "buffer_load_dwordx4 v0, s[4:7], 0 offen lds"), 0),
    (("v_readfirstlane_b32 s6, v1", "s_nop 3", "buffer_load_dword v0, s[4:7], s9 offen lds"), 1),
    (("v_readfirstlane_b32 s6, v1", "s_nop 4", "buffer_load_dword v0, s[4:7], s9 offen lds"), 0),
    (("v_readfirstlane_b32 s9, v1", "s_nop 0", "buffer_load_dword v0, s[4:7], s9 offen lds"), 1),
    (("v_readfirstlane_b32 s8, v1", "s_nop 0", "buffer_load_dword v0, s[4:7], s9 offen lds"), 0),
    # the way through the branch (to the load) is too short
    (("v_mov_b32 v2, v3", "s_nop 4", "buffer_load_dword v0, s[4:7], 0 offen lds", "v_readlane_b32 s5, v1, 0",
      "s_cbranch_scc1 65533"), 1),
    (("s_mov_b32 m0, s1", "buffer_load_dwordx4 v0, s[4:7], 0 offen"), 0),   # not a load to LDS
])
def test_the_walk_finds_what_comes_too_early(code, early):
    assert len(early_loads(_listing(*code))[1]) == early


def test_loads_to_lds_wait_for_their_scalar_operands(tmp_path):
    if not os.path.exists(OBJDUMP):
        pytest.skip("the disassembler of the ROCm toolchain is needed")
    objects = code_objects(LIB)
    assert objects
    loads, early = 0, []
    for i, o in enumerate(objects):
        f = tmp_path / f"{i}.o"
        f.write_bytes(o)
        text = subprocess.run([OBJDUMP, "-d", str(f)], capture_output=True, text=True, check=True).stdout
        n, e = early_loads(text.splitlines())
        loads += n
        early += e
    assert loads > 500   # the products of the head and those of the 4-bit projection
    assert not early, (len(early), early[:8])
