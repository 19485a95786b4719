"""The build's check of the backward dx kernel's compiled code (CPU only)."""
import os

import pytest

from int4_weight_only_linear_amd import build as B

DX_NAME = "_ZN5w4a1612_GLOBAL__N_19dx_kernelILi1ELi2EEEvNS0_8DxParamsENS_8LoraTermE"


def _dx_listing(ops):
    return "\n".join([f"0000000000001000 <{DX_NAME}>:"] + [f"\t{op} v0, v1   // 000000001000: 00000000" for op in ops]
                     + ["0000000000002000 <_ZN5other>:"])


def test_dx_waits_in_this_build():
    obj = os.path.join(B.BUILD, "w4a16_dx.hip.o")
    if not os.path.exists(obj):
        pytest.skip("not built")
    # two steps a loop turn, three tile heights, two types
    assert B.check_dx_waits(obj) >= 12


def test_dx_wait_check_catches_a_wrong_order():
    words = ["global_load_dword"] * 8 + ["global_load_dwordx4"] * 4
    stop = ["s_waitcnt vmcnt(12) lgkmcnt(0)", "s_barrier"]
    dy = ["global_load_lds_dwordx4"] * 4
    good = words + stop + dy + words + stop + dy + ["s_cbranch_scc1 65000"]
    assert B.dx_waits_in(_dx_listing(good)) == 2
    for bad in (words + stop + words + dy + stop,                       # dy after the words
                words + stop + dy + words[1:] + stop,                   # a dropped load
                words + stop + dy + words + ["global_load_dword"] + stop,  # one more
                words + ["s_waitcnt vmcnt(11) lgkmcnt(0)", "s_barrier"],   # another count
                words + stop + dy + words + stop + dy + ["global_load_dword", "s_cbranch_scc1 65000"]):  # hoisted over the end
        with pytest.raises(RuntimeError):
            B.dx_waits_in(_dx_listing(bad))
    # a full wait is always fine
    assert B.dx_waits_in(_dx_listing(dy + ["s_waitcnt vmcnt(0) lgkmcnt(0)", "s_barrier"])) == 0
