"""What the built kernels keep of their registers in memory.  Read from the code objects' own notes, on the CPU."""
import os
import re
import struct
import subprocess

import pytest

from lossless_draft_verification_online_amd.build import LIBRARY, is_stale

LLVM = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin")


def code_objects():
    """The gfx950 parts of the offload bundles in libsdv.so."""
    data = open(LIBRARY, "rb").read()
    magic = b"__CLANG_OFFLOAD_BUNDLE__"
    for m in re.finditer(magic, data):
        at = m.start() + len(magic)
        n, = struct.unpack_from("<Q", data, at)
        at += 8
        for _ in range(n):
            off, size, name = struct.unpack_from("<QQQ", data, at)
            what = data[at + 24:at + 24 + name].decode()
            at += 24 + name
            if what.endswith("gfx950") and size:
                yield data[m.start() + off:m.start() + off + size]


@pytest.fixture(scope="module")
def spilled(tmp_path_factory):
    """Vector registers that a kernel keeps in memory, by its name, for those that do."""
    if is_stale():
        pytest.fail(f"{LIBRARY} is missing or older than its sources; run __graft_entry__.build()")
    out, kernels = {}, 0
    for k, code in enumerate(code_objects()):
        at = tmp_path_factory.mktemp("code") / f"{k}.o"
        at.write_bytes(code)
        notes = subprocess.run([os.path.join(LLVM, "llvm-readelf"), "--notes", str(at)], capture_output=True, text=True, check=True)
        for m in re.finditer(r"\.name: +(_Z\S+)\n(?:.*\n)*?.*\.vgpr_spill_count: (\d+)", notes.stdout):
            kernels += 1
            if int(m[2]):
                out[m[1]] = int(m[2])
    assert kernels > 100
    names = subprocess.run(["c++filt", *out], capture_output=True, text=True, check=True).stdout.split("\n")
    return {re.sub(r"\(.*", "", n).removeprefix("void ").replace("sdv::", ""): v for n, v in zip(names, out.values())}


# Sums and operands of 256 values pass the 256 registers of two waves per SIMD, rotations beside their binary64 path the 64
# of eight.  Times follow these numbers: attention over a bf16 cache by units of 256 values took 1492 us with 28 of them in
# memory and 1807 with 32.
HELD = {
    "attend_impl::attend_rows<128, false>": 1,
    "attend_impl::attend_units<Bf16, 256, 1, 4, false, false>": 47,
    "attend_impl::attend_units<Bf16, 256, 1, 4, true, false>": 28,
    "attend_impl::attend_units<Bf16, 256, 2, 4, false, false>": 41,
    "attend_impl::attend_units<Bf16, 256, 2, 4, true, false>": 38,
    "attend_impl::attend_units<F32, 256, 1, 4, false, false>": 6,
    "attend_impl::attend_units<F32, 256, 1, 4, true, false>": 7,
    "attend_impl::attend_ranges<Bf16, 256, 1, false>": 55,
    "attend_impl::attend_ranges<Bf16, 256, 2, false>": 68,
    "attend_impl::attend_ranges<F32, 128, 1, false>": 5,
    "attend_impl::attend_ranges<F32, 256, 1, false>": 25,
    "attend_impl::attend_ranges<Bf16, 256, 1, true>": 27,
    "cache8_impl::append8<Bf16, false>": 4,
    "cache8_impl::append8<F32, false>": 10,
}


def test_registers_in_memory(spilled):
    assert not {name: (n, HELD.get(name, 0)) for name, n in spilled.items() if n > HELD.get(name, 0)}
