"""The order of loads in the built tile kernels of products with group-scaled 4-bit weights, read
from this library's own code.

Those kernels wait for a stage's rows in LDS by the number of loads issued after them, which
holds only if loads are issued stage by stage, each stage's all of the same number. That is a
matter of the compiler's schedule as well as of the source, so the built code is checked."""
import os
import re
import struct
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "dense_sparse_bit_amd", "libmq.so")
TOOLS = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin")
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def _device_code(path, tmp_path):
    """The gfx950 code objects of a library: its fat binary is one bundle for each source."""
    fat = tmp_path / "fat"
    subprocess.run([os.path.join(TOOLS, "llvm-objcopy"), f"--dump-section=.hip_fatbin={fat}", path, str(tmp_path / "copy")], check=True)
    data = fat.read_bytes()
    for m in re.finditer(MAGIC, data):
        at = m.start() + len(MAGIC)
        count, = struct.unpack_from("<Q", data, at)
        at += 8
        for _ in range(count):
            offset, size, n = struct.unpack_from("<QQQ", data, at)
            name = data[at + 24:at + 24 + n].decode()
            at += 24 + n
            if "gfx950" in name and size:
                yield data[m.start() + offset:m.start() + offset + size]


def _segments(text):
    """{kernel: [loads between two barriers]}: L a load to LDS, W one to registers."""
    kernels, at = {}, None
    for line in text.splitlines():
        m = re.match(r"^[0-9a-f]+ <(\S*k_w4_wide\S*)>:", line)
        if m:
            at = kernels.setdefault(m.group(1), [""])
        elif re.match(r"^[0-9a-f]+ <", line) and not re.match(r"^[0-9a-f]+ <(L|\.L)", line):
            at = None
        elif at is not None:
            op = line.split("//")[0].split()
            if op and op[0].startswith("buffer_load"):
                at[-1] += "L" if "lds" in op else "W"
            elif op and op[0] == "s_barrier":
                at.append("")
    return kernels


def test_loads_are_issued_stage_by_stage(tmp_path):
    if not os.path.exists(os.path.join(TOOLS, "llvm-objdump")):
        pytest.skip("no disassembler")
    found = {}
    for i, code in enumerate(_device_code(LIB, tmp_path)):
        if b"k_w4_wide" not in code:
            continue
        path = tmp_path / f"code{i}"
        path.write_bytes(code)
        r = subprocess.run([os.path.join(TOOLS, "llvm-objdump"), "-d", "--no-show-raw-insn", str(path)], check=True, capture_output=True, text=True)
        found.update(_segments(r.stdout))
    # the tiles that products take, and no others: 128 x 256 and 64 x 256 not with groups of 32
    tiles = {(groups, rt, ct) for groups in (1, 2, 4) for rt, ct in ((1, 1), (2, 1), (2, 2), (3, 2), (4, 2)) if groups < 4 or rt % 2 or ct == 1}
    built = [tuple(map(int, re.search(r"Li(\d)ELi(\d)ELi(\d)E+v", kernel).groups())) for kernel in found]
    assert sorted(built) == sorted(2 * list(tiles))
    for kernel, segments in found.items():
        deep = max(len(re.findall("L+W+", s)) for s in segments)
        for s in segments:
            # equal stages, whole ones; after the last stage's, rows alone
            assert re.fullmatch(r"(L+W+)\1*|L*", s), (kernel, s)
        # two or three stages ahead where tiles are small
        rt, ct = map(int, re.search(r"Li(\d)ELi(\d)E+v", kernel).groups())
        assert deep == (3 if rt * ct == 1 else 2 if rt == 2 else 1), (kernel, deep)


@pytest.mark.parametrize("text,right", [("LLWWLLWW", True), ("LLWW", True), ("LL", True), ("", True), ("LLWWWLLW", False), ("WLLWLLWW", False),
                                        ("LLWWLWW", False)])
def test_the_rule_itself(text, right):
    assert bool(re.fullmatch(r"(L+W+)\1*|L*", text)) == right
