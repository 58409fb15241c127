"""Wait states between a vector instruction that writes a scalar register and
the vector memory instruction that reads it, in the code built for gfx950.

The hardware needs five between the two (an instruction is one, s_nop n is
n + 1) and does not wait by itself.  The compiler inserts them for the
instructions it knows; the asynchronous loads into LDS are inline assembly,
where nothing but the assembly itself sees to them.  A load that comes too
early may read half of an address as it was before."""
import re
import struct
import subprocess

import pytest

NEEDED = 5
OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def code_objects():
    """The device code in the library, one ELF per source file."""
    from routed_expert_int4_amd import build
    try:
        data = open(build.LIB, "rb").read()
    except FileNotFoundError:
        data = open(build.build(), "rb").read()
    for found in re.finditer(MAGIC, data):
        at = found.start()
        count, = struct.unpack_from("<Q", data, at + len(MAGIC))
        entry = at + len(MAGIC) + 8
        for _ in range(count):
            offset, size, name = struct.unpack_from("<QQQ", data, entry)
            target = data[entry + 24:entry + 24 + name]
            entry += 24 + name
            if b"gfx950" in target and size:
                yield data[at + offset:at + offset + size]


def registers(operand):
    """Numbers of the scalar registers an operand names (vcc: its name)."""
    operand = operand.strip()
    if m := re.fullmatch(r"-?\|?s\[(\d+):(\d+)\]\|?", operand):
        return set(range(int(m[1]), int(m[2]) + 1))
    if m := re.fullmatch(r"-?\|?s(\d+)\|?", operand):
        return {int(m[1])}
    return {"vcc"} if operand.startswith("vcc") else set()


def too_early(listing):
    """(kernel, instruction, wait states) of each vector memory instruction that
    reads a scalar register too soon after its write, along the code as it lies."""
    kernel, written, clock = "", {}, 0
    for line in listing:
        if m := re.match(r"[0-9a-f]+ <(.*)>:", line):
            kernel, written, clock = m[1], {}, 0
            continue
        text = line.split("//")[0].strip()
        if not text or text.endswith(":"):
            continue
        name, _, rest = text.partition(" ")
        operands = [o for o in re.split(r",\s*|\s+", rest.strip()) if o]
        if name.startswith(("global_", "buffer_", "scratch_", "flat_")):
            for o in operands:
                for r in registers(o):
                    if r in written and clock - written[r] < NEEDED:
                        yield kernel, text, clock - written[r]
        clock += 1 + (int(operands[0], 0) if name == "s_nop" else 0)
        if name.startswith("v_"):
            for o in operands[:2 if re.match(r"v_(add|sub|subrev|addc|subb|subbrev)_co_|v_div_scale|v_mad_[iu]64", name) else 1]:
                for r in registers(o):
                    written[r] = clock
        elif name.startswith("s_") and not name.startswith(("s_nop", "s_waitcnt", "s_barrier", "s_cmp", "s_cbranch", "s_branch")) and operands:
            for r in registers(operands[0]):
                written.pop(r, None)  # the scalar unit's writes are waited for
        if name in ("s_branch", "s_endpgm", "s_setpc_b64"):
            written = {}


def test_the_scan_itself():
    listing = ["0000 <k>:", "\tv_readlane_b32 s4, v1, s2 // 00", "\tv_readfirstlane_b32 s5, v1", "\ts_mov_b32 m0, s9", "\ts_nop 0",
               "\tglobal_load_lds_dwordx4 v0, s[4:5]"]
    assert [w for _, _, w in too_early(listing)] == [3, 2]
    listing[4] = "\ts_nop 3"
    assert not list(too_early(listing))
    listing[3:5] = ["\ts_mov_b32 s5, s9", "\ts_mov_b32 s4, s9"]
    assert not list(too_early(listing))


def test_bases_of_loads_have_their_wait_states(tmp_path):
    found, loads = [], 0
    for i, code in enumerate(code_objects()):
        path = tmp_path / f"{i}.co"
        path.write_bytes(code)
        res = subprocess.run([OBJDUMP, "-d", "--mcpu=gfx950", "--no-show-raw-insn", str(path)], capture_output=True, text=True)
        if res.returncode != 0:
            pytest.fail(res.stderr)
        found += too_early(res.stdout.splitlines())
        loads += res.stdout.count("global_load_lds_")
    assert loads > 100, "the asynchronous loads are not in the listing"
    assert not found, f"{len(found)}: " + "; ".join(f"{k}: {t} after {w}" for k, t, w in found[:10])
