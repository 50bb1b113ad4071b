"""The compiled kernels of the norm, the adapters and the head's cross entropy: what
the source leaves to the compiler (CPU: the device assembly that the build's own
flags give; how it is read: test_device_assembly.py)."""
import os
import re
import subprocess

import pytest

from test_device_assembly import build_module, kernels, lds_accesses_out_at_barriers


@pytest.fixture(scope="module", params=["qg_norm.hip", "qg_lora.hip", "qg_xent.hip"])
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
    written_out, uses = False, {True: [], False: []}
    for line in compiled[0].splitlines():
        if "#ASMSTART" in line or "#ASMEND" in line:
            written_out = "#ASMSTART" in line
        elif re.search(r"\bm0\b", line.split(";")[0]):
            uses[written_out].append(line)
    assert not uses[True] or uses[False] == []


def test_the_device_code_compiles_without_warnings(compiled):
    assert compiled[1] == ""


def test_the_products_have_no_lds_but_their_ring(compiled):
    """How many workgroups of a shape a CU holds is counted from the LDS that the launch asks for."""
    fixed = dict(re.findall(r"\.amdhsa_kernel (\S+)\n\s*\.amdhsa_group_segment_fixed_size (\d+)", compiled[0]))
    assert fixed
    assert {name: n for name, n in fixed.items() if "mm_kernel" in name and n != "0"} == {}
