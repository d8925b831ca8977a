"""Direct-to-LDS loads take their LDS address from M0 and are inline asm here,
so the compiler's hazard recognizer does not protect them: an instruction of
the scalar unit that writes M0 needs one wait state before such a load, one of
the vector unit five (as before any vector memory instruction that reads the
scalar register), or the load may go to an earlier load's address.  This
compiles every source with the library's own flags and checks every such load
(host only; needs hipcc)."""
import concurrent.futures
import os
import re
import shutil
import subprocess

import pytest

from state_space_sequence_02_amd.build import FLAGS, HIPCC, sources


def _to_lds(line):
    return "_load_lds_" in line or (line.startswith("buffer_load") and line.split()[-1] == "lds")


def _m0_hazards(asm):
    """(load, writer of M0, wait states between) for every direct-to-LDS load that comes too soon
    behind it.  Every instruction is one wait state, s_nop n has n + 1."""
    ins = []
    for line in asm.splitlines():
        line = re.split(r";|//", line)[0].strip()
        if line and not line.endswith(":") and not line.startswith("."):
            ins.append(line)
    out = []
    for k, line in enumerate(ins):
        if not _to_lds(line):
            continue
        waits = 0
        for p in reversed(ins[max(0, k - 5):k]):
            if waits >= 5:
                break
            op, _, rest = p.partition(" ")
            if op == "s_nop":
                waits += int(rest, 0) + 1
                continue
            if rest.split(",")[0].strip() == "m0" and waits < (5 if op.startswith("v_") else 1):
                out.append((line, p, waits))
            waits += 1
    return out


def test_scan_finds_planted_cases():
    mov, add, lane = "s_mov_b32 m0, s4\n", "s_add_i32 m0, s4, 0x400\n", "v_readfirstlane_b32 m0, v1\n"
    off, base = "global_load_lds_dwordx4 v[2:3], off\n", "global_load_lds_dword v2, s[6:7]\n"
    buffer = "buffer_load_dwordx4 v2, s[8:11], 0 offen lds\n"
    for load in (off, base, buffer):
        for write in (mov, add, lane):
            assert len(_m0_hazards(write + load)) == 1
            assert len(_m0_hazards(write + load + load)) == (2 if write == lane else 1)
        for write in (mov, add):
            for one in ("s_nop 0\n", "v_add_u32_e32 v2, v3, v4\n", "\t;;#ASMSTART\n\ts_nop 0\n"):
                assert not _m0_hazards(write + one + load)
            assert len(_m0_hazards(write + "\t;;#ASMSTART\n" + load)) == 1
            assert len(_m0_hazards(write + ".LBB0_1:\n" + load)) == 1
        assert len(_m0_hazards(lane + "s_nop 3\n" + load)) == 1
        assert not _m0_hazards(lane + "s_nop 4\n" + load)
    # other loads do not read M0
    assert not _m0_hazards(mov + "global_load_dwordx4 v[4:7], v[2:3], off\n")
    assert not _m0_hazards(mov + "buffer_load_dwordx4 v[4:7], v2, s[8:11], 0 offen\n")


def _asm(source):
    got = subprocess.run([HIPCC, *FLAGS, "--cuda-device-only", "-S", source, "-o", "-"], check=True,
                         capture_output=True, text=True)
    return got.stdout


@pytest.mark.skipif(shutil.which(HIPCC) is None and not os.path.exists(HIPCC),
                    reason="hipcc not available")
def test_loads_to_lds_wait_for_m0():
    loads, bad = 0, {}
    with concurrent.futures.ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
        for source, asm in zip(sources(), pool.map(_asm, sources())):
            loads += sum(_to_lds(line.strip()) for line in asm.splitlines())
            found = _m0_hazards(asm)
            if found:
                bad[os.path.basename(source)] = (len(found), found[:2])
    assert loads > 1000
    assert not bad, bad
