"""What the written-out waits of the training kernels rely on, read from the built
library's kernel descriptors: no vector register is spilled and no scratch memory is
used, whose loads and stores the waits do not count (no GPU needed)."""
import os
import re
import shutil
import subprocess

import pytest

from sparse_moe_routed_amd import _abi

LLVM = "/opt/rocm/llvm/bin"
pytestmark = pytest.mark.skipif(
    not os.path.exists(_abi.LIB_PATH) or not os.path.exists(os.path.join(LLVM, "llvm-readelf")),
    reason="needs libmoe.so (run __graft_entry__.build()) and ROCm's llvm tools")

# kernels whose loads into LDS are waited for by count
COUNTED = ("k_gate_up_save", "k_dh", "k_dx", "k_dx_dw", "k_dw", "k_dw_wide")


def kernels(tmp_path):
    """[(name, {descriptor entry: value})] of the library's GPU code."""
    lib = shutil.copy(_abi.LIB_PATH, tmp_path / "lib.so")
    subprocess.run([f"{LLVM}/llvm-objdump", "--offloading", lib], check=True, capture_output=True, cwd=tmp_path)
    out = []
    for f in sorted(tmp_path.iterdir()):
        if "gfx950" not in f.name:
            continue
        notes = subprocess.run([f"{LLVM}/llvm-readelf", "--notes", str(f)], check=True, capture_output=True,
                               text=True).stdout
        # one list item per kernel
        for item in re.split(r"\n  - ", notes)[1:]:
            d = dict(re.findall(r"^ *\.(\w+): +(\S+)$", item, re.M))
            if "symbol" in d:
                out.append((d["symbol"].strip("'"), d))
    return out


def test_no_spills_where_loads_are_counted(tmp_path):
    found = {n: 0 for n in COUNTED}
    for symbol, d in kernels(tmp_path):
        name = re.match(r"_ZN3moe(\d+)", symbol)
        name = symbol[name.end():name.end() + int(name[1])] if name else symbol
        if name not in found:
            continue
        found[name] += 1
        assert d["vgpr_spill_count"] == "0" and d["private_segment_fixed_size"] == "0", (symbol, d)
    assert all(found.values()), found
