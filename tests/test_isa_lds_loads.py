"""Wait states before the loads into LDS that the kernels issue from inline asm (CPU; compiles the kernels to
gfx950 assembly with hipcc).

A load into LDS takes its LDS address from M0, and a scalar write of M0 needs one wait state (another instruction, or
s_nop) before it; a vector instruction that writes a scalar register needs five before a vector memory instruction
reads that register as its base.  The compiler keeps both distances for its own instructions and cannot for those of
inline asm, so the generated code is checked."""
import concurrent.futures as cf
import glob
import os
import re
import subprocess

import pytest

from tests.test_isa_mfma_exec import CSRC, HIPCC, _device_asm

LOAD = re.compile(r"(global|buffer|scratch)_load_lds_")


def _wait_states(ins):
    m = re.match(r"s_nop\s+(\d+)", ins)
    return int(m.group(1)) + 1 if m else 1


def _scalars(operand):
    """Scalar registers an operand names: s7 -> {7}, s[4:5] -> {4, 5}."""
    m = re.fullmatch(r"s\[(\d+):(\d+)\]|s(\d+)", operand)
    if not m:
        return set()
    return {int(m.group(3))} if m.group(3) else set(range(int(m.group(1)), int(m.group(2)) + 1))


def short_waits(asm_text):
    """(loads into LDS, those too close to a write of M0 or to a vector write of their base) of an assembly text.
    Code is read in its written order; a jump between a write and a load counts as the one instruction that it is."""
    loads, bad, before = 0, [], []
    for ln in asm_text.splitlines():
        t = ln.split(";")[0].strip()
        if re.match(r"^_Z\S+:", t):
            before = []
        if not t or t.endswith(":") or t.startswith("."):
            continue
        ops = [o.strip() for o in t.partition(" ")[2].split(",")]
        if LOAD.match(t):
            loads += 1
            base = set().union(*(_scalars(o.split()[0]) for o in ops if o))
            states = 0
            for p, pops in reversed(before):
                writes_m0 = p.startswith("s_") and pops and pops[0] == "m0"
                writes_base = p.startswith("v_") and pops and _scalars(pops[0]) & base
                if (writes_m0 and states < 1) or (writes_base and states < 5):
                    bad.append((p, t))
                states += _wait_states(p)
                if states >= 5:
                    break
        before = (before + [(t, ops)])[-8:]
    return loads, bad


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs hipcc")
def test_loads_into_lds_wait_for_their_address(tmp_path):
    srcs = [os.path.join(CSRC, f) for f in ("gemm_tiled.hip", "gemm_w4.hip", "gemm_w4_tiled.hip")]
    others = set(glob.glob(os.path.join(CSRC, "*.hip"))) - set(srcs)
    assert not any("load_lds_" in open(f).read() for f in others)  # every file that issues such loads is listed
    with cf.ThreadPoolExecutor(max_workers=len(srcs)) as ex:
        outs = list(ex.map(lambda s: _device_asm(s, str(tmp_path)), srcs))
    for s, o in zip(srcs, outs):
        loads, bad = short_waits(open(o).read())
        assert loads > 10, s
        assert not bad, f"{os.path.basename(s)}: {len(bad)} of {loads} loads, e.g. {bad[0]}"


def test_check_flags_a_missing_wait():
    k = lambda *ins: "\n".join(("_ZN3r9k1kEv:",) + ins)
    load = "global_load_lds_dwordx4 v1, s[2:3]"
    assert short_waits(k("s_mov_b32 m0, s4", "\t;;#ASMSTART", load))[1] == [("s_mov_b32 m0, s4", load)]
    assert short_waits(k("s_mov_b32 m0, s4", "s_nop 0", load)) == (1, [])
    assert short_waits(k("s_mov_b32 m0, s4", "v_add_u32_e32 v0, v0, v1", load)) == (1, [])
    assert short_waits(k("v_readfirstlane_b32 s3, v0", "s_nop 3", load))[1]
    assert short_waits(k("v_readfirstlane_b32 s3, v0", "s_nop 4", load)) == (1, [])
    assert short_waits(k("v_readfirstlane_b32 s4, v0", load)) == (1, [])
    assert short_waits(k("s_add_i32 m0, s4, 16", ".LBB0_1:", "global_load_lds_dword v[0:1], off"))[1]
