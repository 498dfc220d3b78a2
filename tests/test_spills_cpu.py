"""The compiler's own report of the attention's kernels: none keeps registers in
scratch memory (a wave that waits for nothing but itself pays for each)."""
import os
import re
import subprocess

import pytest

from rank_adapter_gemm_token_amd import build

pytestmark = pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="no compiler")


def report(src):
    """Of each kernel of a source: what -Rpass-analysis=kernel-resource-usage names."""
    r = subprocess.run([build.HIPCC, *build.CXXFLAGS, *build.DEVICE_FLAGS, "--cuda-device-only", "-x", "hip", "-c",
                        os.path.join(build.CSRC, src), "-o", os.devnull, "-Rpass-analysis=kernel-resource-usage"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    kernels = {}
    for line in r.stderr.splitlines():
        m = re.search(r"remark: (?:\S+:\d+:\d+: )?\s*(\S.*?): (\S+) \[-Rpass", line)
        if m and m.group(1) == "Function Name":
            name = m.group(2)
            kernels[name] = {}
        elif m:
            kernels[name][m.group(1)] = m.group(2)
    return kernels


def test_attention_keeps_no_registers_in_scratch():
    kernels = report("attend.hip")
    assert sum("k_attendI" in k for k in kernels) == 8
    spilled = {k: (v["VGPRs Spill"], v["ScratchSize [bytes/lane]"]) for k, v in kernels.items()
               if v["VGPRs Spill"] != "0" or v["ScratchSize [bytes/lane]"] != "0"}
    assert not spilled


def test_cache_writes_keep_what_they_need_in_registers():
    """Eight waves a SIMD (64 registers), none of them saved and fetched back."""
    kernels = {k: v for k, v in report("kv_cache.hip").items() if "k_kv_write" in k}
    assert len(kernels) == 4
    for k, v in kernels.items():
        assert v["SGPRs Spill"] == v["VGPRs Spill"] == v["ScratchSize [bytes/lane]"] == "0", (k, v)
        assert int(v["VGPRs"]) <= 64, (k, v)
