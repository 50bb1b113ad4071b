"""The compiled kernels of the language-model operators: what the source leaves
to the compiler (CPU: the device assembly that the build's own flags give).

s_barrier does not wait for LDS accesses that a wave still has in flight, and
the compiler may sink what consumes a read below the barrier.  Behind a barrier
other waves write the same LDS, so no wave may reach one with an access out:
every path from a ds_ instruction to an s_barrier has to pass an s_waitcnt that
covers it."""
import importlib.util
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def build_module():
    spec = importlib.util.spec_from_file_location("qg_build", os.path.join(ROOT, "quantized_gemm_qg_amd", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def kernels(text):
    """(name, lines) of every function of a device assembly."""
    name, lines = None, []
    for line in text.splitlines():
        line = line.split(";")[0].strip()
        if re.match(r"\w+:$", line):
            name, lines = line[:-1], []
        elif line.startswith(".Lfunc_end"):
            if name:
                yield name, lines
            name = None
        elif line:
            lines.append(line)


def blocks_of(lines):
    """Basic blocks and their successors."""
    blocks, labels = [[]], {}
    for line in lines:
        m = re.match(r"(\.L\w+):", line)
        if m:
            blocks.append([])
            labels[m.group(1)] = len(blocks) - 1
        elif not line.startswith("."):
            blocks[-1].append(line)
            if re.match(r"s_(c?branch|endpgm)", line):
                blocks.append([])
    follow = []
    for i, b in enumerate(blocks):
        last = b[-1] if b else ""
        m = re.match(r"s_(c?)branch\w*\s+(\S+)", last)
        to = [labels[m.group(2)]] if m else []
        if not last.startswith("s_endpgm") and not (m and not m.group(1)) and i + 1 < len(blocks):
            to.append(i + 1)
        follow.append(to)
    return blocks, follow


def lds_accesses_out_at_barriers(lines):
    """The most LDS accesses in flight at each s_barrier, over all paths (LDS
    answers in order, so lgkmcnt(n) leaves at most n)."""
    blocks, follow = blocks_of(lines)
    entry, work, out = {0: 0}, [0], {}
    while work:
        i = work.pop()
        n = entry[i]
        for j, line in enumerate(blocks[i]):
            if line.startswith("ds_"):
                n = min(n + 1, 64)
            elif line.startswith("s_waitcnt"):
                m = re.search(r"lgkmcnt\((\d+)\)", line)
                if m:
                    n = min(n, int(m.group(1)))
            elif line.startswith("s_barrier"):
                out[i, j] = max(out.get((i, j), 0), n)
        for to in follow[i]:
            if n > entry.get(to, -1):
                entry[to] = n
                work.append(to)
    return list(out.values())


def test_the_count_follows_every_path():
    straight = ["ds_read_b128 v[0:3], v9", "ds_read_b128 v[4:7], v9", "s_waitcnt lgkmcnt(1)", "s_barrier", "s_endpgm"]
    assert lds_accesses_out_at_barriers(straight) == [1]
    waited = straight[:2] + ["s_waitcnt vmcnt(3) lgkmcnt(0)"] + straight[3:]
    assert lds_accesses_out_at_barriers(waited) == [0]
    one_way = ["s_cbranch_scc1 .LBB0_2", "ds_write_b32 v1, v2", ".LBB0_2:", "s_barrier", "s_endpgm"]
    assert lds_accesses_out_at_barriers(one_way) == [1]
    loop = [".LBB0_1:", "s_barrier", "ds_read_b32 v1, v2", "s_cbranch_scc1 .LBB0_1", "s_endpgm"]
    assert lds_accesses_out_at_barriers(loop)[0] > 0


@pytest.fixture(scope="module", params=["qg_ffn.hip", "qg_int8.hip", "qg_logprobs.hip"])
def compiled(request, tmp_path_factory):
    """Device assembly of one source, and what the compiler said."""
    b, asm = build_module(), tmp_path_factory.mktemp("asm") / "device.s"
    r = subprocess.run([b.hipcc(), "-S", "--cuda-device-only", *b._flags(), *b.EXTRA.get(request.param, []), "-x", "hip",
                        os.path.join(b.CSRC, request.param), "-o", str(asm)], check=True, capture_output=True, text=True)
    return asm.read_text(), r.stderr


def test_no_barrier_is_reached_with_lds_accesses_out(compiled):
    found = {name: lds_accesses_out_at_barriers(lines) for name, lines in kernels(compiled[0])}
    assert sum(map(len, found.values())) > 0
    assert {name: n for name, n in found.items() if any(n)} == {}


def test_only_the_written_out_copies_use_m0(compiled):
    """Where there are any: they change m0 behind the compiler's back (a clobber
    of a reserved register does not make it save it)."""
    written_out, uses = False, {True: [], False: []}
    for line in compiled[0].splitlines():
        if "#ASMSTART" in line or "#ASMEND" in line:
            written_out = "#ASMSTART" in line
        elif re.search(r"\bm0\b", line.split(";")[0]):
            uses[written_out].append(line)
    assert not uses[True] or uses[False] == []


def test_the_device_code_compiles_without_warnings(compiled):
    assert compiled[1] == ""
