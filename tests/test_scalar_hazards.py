"""The built kernels on the CPU: a scalar register that a vector instruction wrote is read by a memory instruction only
five wait states later, which CDNA asks for and the hardware does not check.  The compiler counts them for its own
instructions and does not look into inline assembly."""
import os
import re
import shutil
import struct
import subprocess

import pytest

OBJDUMP = shutil.which("llvm-objdump") or "/opt/rocm/llvm/bin/llvm-objdump"
NEEDED = 5
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"
LINE = re.compile(r"^\s+(\S+)\s*(.*?)\s*// ([0-9A-F]{12}):.*?(?:<(\S+)\+0x([0-9a-f]+)>)?$")
HEAD = re.compile(r"^([0-9a-f]{16}) <(\S+)>:$")
SGPR = re.compile(r"\bs(?:\[(\d+):(\d+)\]|(\d+)\b)")
MEMORY = ("buffer_", "tbuffer_", "global_", "flat_", "scratch_")


def code_objects(data):
    """The gfx950 code objects of a library's bundles."""
    at = data.find(MAGIC)
    while at >= 0:
        n, = struct.unpack_from("<Q", data, at + 24)
        p = at + 32
        for _ in range(n):
            offset, size, length = struct.unpack_from("<QQQ", data, p)
            if size and b"gfx950" in data[p + 24:p + 24 + length]:
                yield data[at + offset:at + offset + size]
            p += 24 + length
        at = data.find(MAGIC, at + 24)


def registers(text):
    out = set()
    for lo, hi, one in SGPR.findall(text):
        out.update(range(int(lo), int(hi) + 1) if lo else (int(one),))
    return out


def instructions(listing):
    """{kernel: [(address, mnemonic, operands, branch target or None)]}."""
    out, base, now = {}, {}, None
    for line in listing.splitlines():
        m = HEAD.match(line)
        if m:
            now = out.setdefault(m.group(2), [])
            base[m.group(2)] = int(m.group(1), 16)
            continue
        m = LINE.match(line)
        if m and now is not None:
            name, ops, at, symbol, offset = m.groups()
            target = None
            if name.startswith(("s_branch", "s_cbranch")):
                assert symbol, line
                target = base[symbol] + int(offset, 16)
            now.append((int(at, 16), name, ops, target))
    return out


def late_writes(code):
    """(address, register, wait states) of the reads that come too early, over all ways through a kernel."""
    at = {a: i for i, (a, *_) in enumerate(code)}
    young = [None] * len(code)    # register -> wait states since its write, where fewer than NEEDED
    work, found = [(0, {})], set()
    while work:
        i, state = work.pop()
        while i < len(code):
            if young[i] is not None:
                if all(young[i].get(r, NEEDED) <= n for r, n in state.items()):
                    break
                state = {r: min(young[i].get(r, NEEDED), state.get(r, NEEDED)) for r in {*young[i], *state}}
            young[i] = dict(state)
            address, name, ops, target = code[i]
            if name.startswith(MEMORY):
                found.update((address, r, state[r]) for r in registers(ops) & state.keys())
            passed = int(ops.split()[0], 0) + 1 if name == "s_nop" else 1
            state = {r: n + passed for r, n in state.items() if n + passed < NEEDED}
            if name.startswith("v_"):
                parts = re.split(r",\s*", ops)
                for r in registers(parts[0]) | (registers(parts[1]) if "_co_" in name or "div_scale" in name else set()):
                    state[r] = 0
            elif name.startswith("s_") and not name.startswith(("s_cmp", "s_bitcmp", "s_set", "s_waitcnt", "s_nop", "s_cbranch", "s_branch")):
                for r in registers(ops.split(",")[0]):
                    state.pop(r, None)
            if target is not None:
                work.append((at[target], dict(state)))
                if name == "s_branch":
                    break
            if name == "s_endpgm":
                break
            i += 1
    return sorted(found)


def test_the_walk_finds_early_reads():
    text = """0000000000000000 <k>:
	v_readfirstlane_b32 s6, v0                                 // 000000000000: 7E0C0500
	s_mov_b32 m0, s4                                           // 000000000004: BEFC0004
	s_nop 0                                                    // 000000000008: BF800000
	buffer_load_dwordx4 v2, s[4:7], 0 offen lds                // 00000000000C: E05D1000 80010002
	s_nop 1                                                    // 000000000014: BF800001
	buffer_load_dwordx4 v2, s[4:7], 0 offen lds                // 000000000018: E05D1000 80010002
	v_readfirstlane_b32 s9, v0                                 // 000000000020: 7E120500
	s_cbranch_scc1 65531                                       // 000000000024: BF85FFFB <k+0x14>
	buffer_load_dwordx4 v2, s[8:11], 0 offen lds               // 000000000028: E05D1000 80020002
	s_mov_b32 s9, 0                                            // 000000000030: BE890080
	buffer_load_dwordx4 v2, s[8:11], 0 offen lds               // 000000000034: E05D1000 80020002
	s_endpgm                                                   // 00000000003C: BF810000
"""
    assert late_writes(instructions(text)["k"]) == [(0x0C, 6, 2), (0x28, 9, 1)]


def test_memory_instructions_read_settled_scalars(tmp_path):
    from int8_ivf_ann_amd import svt
    if not os.path.exists(svt.LIB_PATH):
        from int8_ivf_ann_amd import build
        build.build()
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    with open(svt.LIB_PATH, "rb") as f:
        objects = list(code_objects(f.read()))
    assert len(objects) >= 10
    direct, early = 0, {}
    for i, code in enumerate(objects):
        path = tmp_path / f"{i}.co"
        path.write_bytes(code)
        text = subprocess.run([OBJDUMP, "-d", "--mcpu=gfx950", str(path)], capture_output=True, text=True, check=True).stdout
        for kernel, body in instructions(text).items():
            direct += sum(name.startswith("buffer_load") and ops.endswith("lds") for _, name, ops, _ in body)
            found = late_writes(body)
            if found:
                early[kernel] = [(hex(a), f"s{r}", n) for a, r, n in found]
    assert direct > 100   # the hand-written loads are among them
    assert not early, early
