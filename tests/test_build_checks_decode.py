"""The compiled decode kernels (CPU only): adapters live in instances of
their own, and every kernel the host code launches by name is in the device
code (a name that the two passes of the compiler spell differently, such as one
with an unnamed type in it, aborts at its first launch)."""
import json
import os
import re
import subprocess

import pytest

from int4_weight_only_linear_amd import build as B


def test_plain_instances_carry_no_adapter():
    path = os.path.join(B.BUILD, "w4a16_gemv.hip.o.resources.json")
    if not os.path.exists(path):
        pytest.skip("not built")
    with open(path) as f:
        res = json.load(f)
    mode = re.compile(r"gemv_one_kernelILi\dELi\d+ELb\dELi\dELi\dELb\dELi(\d)E")
    kinds = {}
    for name, r in res.items():
        m = mode.search(name)
        lora = "LoraParams" in name or (m is not None and m.group(1) in "34")
        kinds.setdefault((m.group(1) if m else "small", lora), []).append(r["TotalSGPRs"])
        assert r["VGPRs Spill"] == 0, name
    # a plain instance needs 32 scalar registers, a K split 44 (with the
    # adapters' argument in it 68 and more)
    assert max(kinds["0", False]) <= 40 and max(kinds["2", False]) <= 52
    assert set(kinds) == {("0", False), ("1", False), ("2", False), ("3", True), ("4", True), ("small", False), ("small", True)}


@pytest.mark.parametrize("src", [s for s in B.SOURCES if s.endswith(".hip")])
def test_host_and_device_names_agree(src, tmp_path):
    obj = os.path.join(B.BUILD, src + ".o")
    if not os.path.exists(obj):
        pytest.skip("not built")
    fat = tmp_path / "fatbin"
    subprocess.run([B._llvm_tool("llvm-objcopy"), f"--dump-section=.hip_fatbin={fat}", obj, str(tmp_path / "o")], check=True)
    device = fat.read_bytes()
    with open(obj, "rb") as f:
        host = f.read().replace(device, b"")
    launched = {n for n in re.findall(rb"\0(_ZN5w4a16[\w$.]*kernel[\w$.]*)(?=\0)", host) if b"__device_stub" not in n}
    built = set(re.findall(rb"(_ZN5w4a16[\w$.]*kernel[\w$.]*)\.kd", device))
    assert launched and launched <= built, sorted(launched - built)[:3]
