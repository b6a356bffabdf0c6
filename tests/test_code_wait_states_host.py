"""The built library's code (no GPU): a vector memory instruction reads a scalar
register at the earliest five wait states after a vector instruction wrote it,
and one that loads to LDS reads m0 at the earliest one after a scalar one did.
The compiler keeps this in its own code and does not look into inline assembly,
and the hardware does not wait."""
import os
import re
import shutil
import struct
import subprocess

import pytest

from padding_free_pair_amd import _native

MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"
NEEDED = 5
M0 = -1  # among the numbers of the scalar registers
WRITES = re.compile(r"^v_(readfirstlane|readlane)_b32 (s\d+|m0)\b|^v_cmp\w* (s\[(\d+):(\d+)\])|"
                    r"^v_\w+_co_u32\w* v\d+, (s\[(\d+):(\d+)\])")
READS = re.compile(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b")


def _objdump():
    for cand in ("/opt/rocm/llvm/bin/llvm-objdump", shutil.which("llvm-objdump")):
        if cand and os.path.exists(cand):
            return cand
    pytest.skip("needs llvm-objdump")


def device_objects(path):
    """The gfx950 code objects within a library built by hipcc."""
    data = open(path, "rb").read()
    at = data.find(MAGIC)
    while at >= 0:
        pos = at + len(MAGIC)
        (n,) = struct.unpack_from("<Q", data, pos)
        pos += 8
        for _ in range(n):
            off, size, length = struct.unpack_from("<QQQ", data, pos)
            triple = data[pos + 24:pos + 24 + length].decode()
            pos += 24 + length
            if "gfx950" in triple and size:
                yield data[at + off:at + off + size]
        at = data.find(MAGIC, at + 1)


def too_early(lines):
    """(kernel, wait states, instruction) of each read that comes too early, in the
    order of the listing."""
    kernel, written = "", {}  # register -> wait states since its write
    for line in lines:
        head = re.match(r"^[0-9a-f]+ <(\S+)>:$", line)
        if head:
            if not head.group(1).startswith("L"):
                kernel, written = head.group(1), {}
            continue
        text = line.split("//")[0].strip()
        if not text or text.endswith(":"):
            continue
        if text.startswith(("global_", "buffer_", "scratch_", "flat_")):
            read = {M0} if "_lds_" in text or text.endswith(" lds") else set()
            for m in READS.finditer(text):
                lo = int(m.group(1) or m.group(3))
                read.update(range(lo, int(m.group(2) or lo) + 1))
            for r in sorted(read):
                if written.get(r, NEEDED) < NEEDED:
                    yield kernel, written[r], text
        states = int(text.split()[1], 0) + 1 if text.startswith("s_nop") else 1
        written = {r: n + states for r, n in written.items() if n + states < NEEDED}
        if re.match(r"s_\w+ m0,", text):
            written[M0] = NEEDED - 1
        m = WRITES.match(text)
        if m:
            if m.group(2):
                written[M0 if m.group(2) == "m0" else int(m.group(2)[1:])] = 0
            else:
                lo, hi = (m.group(4), m.group(5)) if m.group(3) else (m.group(7), m.group(8))
                written.update({r: 0 for r in range(int(lo), int(hi) + 1)})


def test_listing_reader():
    """The reader itself: four wait states are too few, five are enough, and a
    scalar write in between is not a vector one."""
    code = ["0000 <k>:", "\tv_readfirstlane_b32 s4, v1", "\ts_mov_b32 m0, s9", "\ts_nop 2",
            "\tglobal_load_lds_dwordx4 v2, s[4:5]"]
    assert [(n, s) for _, n, s in too_early(code)] == [(4, code[-1].strip())]
    assert not list(too_early(code[:3] + ["\ts_nop 3"] + code[4:]))
    assert not list(too_early(["\ts_mov_b32 s4, s8"] + code[2:]))
    assert len(list(too_early(["\ts_mov_b32 m0, s9", code[-1]]))) == 1
    assert len(list(too_early(["\tv_readfirstlane_b32 m0, v1", "\ts_nop 2", code[-1]]))) == 1


def test_scalar_addresses_are_written_in_time(tmp_path):
    if not os.path.exists(_native.LIB_PATH):
        from padding_free_pair_amd import build
        build.build(verbose=False)
    dump, found, objects, ends = _objdump(), [], 0, 0
    for data in device_objects(_native.LIB_PATH):
        objects += 1
        f = tmp_path / f"{objects}.co"
        f.write_bytes(data)
        out = subprocess.run([dump, "-d", "--no-show-raw-insn", str(f)], capture_output=True,
                             text=True, check=True).stdout
        ends += out.count("s_endpgm")
        found += list(too_early(out.splitlines()))
    assert ends > 0  # a listing of kernels
    assert not found, (len(found), found[:5])
