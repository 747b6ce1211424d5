"""Wait states around the loads straight to LDS (on the CPU, no GPU needed).

The compiler keeps the distances that the hardware asks for between its own
instructions, but does not see the ones inside an asm string.  The kernels with
such loads are compiled to assembly and checked here:

* a load that goes to LDS reads M0; after a scalar write of M0 it needs one wait
  state in between, or it may go to the address of the load before it;
* a memory instruction that reads a scalar register written by a vector
  instruction needs five.
"""
import concurrent.futures as cf
import os
import re
import shutil
import subprocess

import pytest

from muon_step_03_amd import build

HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
# the sources that include lds_tiles.h
SOURCES = [s for s in build.SOURCES
           if "lds_tiles.h" in open(os.path.join(build.CSRC, s)).read()]


def scalars(operand):
    """The scalar registers that an operand names: {36, 37} of s[36:37]."""
    m = re.fullmatch(r"s(\d+)|s\[(\d+):(\d+)\]", operand)
    if not m:
        return set()
    return {int(m[1])} if m[1] else set(range(int(m[2]), int(m[3]) + 1))


def faults(listing):
    """(loads straight to LDS, too short distances) of an assembly listing."""
    loads, found = 0, []
    since_m0 = 9        # wait states since M0 was written
    valu = {}           # scalar register -> wait states since a vector write
    for n, line in enumerate(listing.splitlines(), 1):
        line = line.split(";")[0].strip()
        if not line or line.startswith(".") or line.endswith(":"):
            continue
        name, _, rest = line.partition(" ")
        ops = [o.strip() for o in rest.replace("\t", " ").split(",")]
        if name.startswith("global_load_lds") or (name.startswith("buffer_load") and rest.endswith(" lds")):
            loads += 1
            if since_m0 < 1:
                found.append((n, "M0", line))
            read = set().union(*(scalars(o.split(" ")[0]) for o in ops))
            if any(valu.get(s, 9) < 5 for s in read):
                found.append((n, "scalar", line))
        states = int(ops[0], 0) + 1 if name == "s_nop" else 1
        since_m0 += states
        valu = {s: d + states for s, d in valu.items() if d + states < 5}
        if name.startswith("s_") and ops[0] == "m0":
            since_m0 = 0
        if name.startswith("v_"):
            wrote = scalars(ops[0])
            if "_co_" in name or name.startswith(("v_div_scale", "v_mad_u64", "v_mad_i64")):
                wrote |= scalars(ops[1])      # the carry, or the flag
            valu.update((s, 0) for s in wrote)
    return loads, found


def test_the_check_itself():
    assert faults("\ts_mov_b32 m0, s3\n\tglobal_load_lds_dword v1, s[4:5]") == (
        1, [(2, "M0", "global_load_lds_dword v1, s[4:5]")])
    assert faults("s_mov_b32 m0, s3\ns_nop 0\nglobal_load_lds_dword v1, s[4:5]") == (1, [])
    assert faults("s_mov_b32 m0, s3\nv_mov_b32_e32 v2, v3\nglobal_load_lds_dword v1, s[4:5]") == (1, [])
    late = "v_readfirstlane_b32 s5, v0\ns_mov_b32 m0, s3\ns_nop %d\nglobal_load_lds_dword v1, s[4:5]"
    assert [len(faults(late % n)[1]) for n in (2, 3)] == [1, 0]


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
@pytest.mark.timeout(600)
def test_distances_in_the_built_kernels():
    def listing(src):
        r = subprocess.run([HIPCC, *build.HIPCC_FLAGS, "--cuda-device-only", "-S",
                            os.path.join(build.CSRC, src), "-o", "-"], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-3000:]
        return r.stdout

    assert set(SOURCES) >= {"k_weight_grad.hip", "k_ns_bf16.hip"}
    with cf.ThreadPoolExecutor(max_workers=4) as ex:
        listings = list(ex.map(listing, SOURCES))
    for src, text in zip(SOURCES, listings):
        loads, found = faults(text)
        assert loads > 0, src
        assert not found, (src, len(found), found[:3])
