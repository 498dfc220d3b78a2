"""A tree's missing list of parents: refused after the batch's counts, before any
list is read."""
import subprocess
import sys

import pytest

from test_host_cpu import ROOT, SANITIZE, _native_check

# Lists at addresses that cannot be read, and no plan that has room for them.
UNREAD = """
import ctypes
from rank_adapter_gemm_token_amd import lora
b = lora.lora_attend_batch(1 << 30, 0, 8, 8, 8, 8, 8, None, None, None)
lib = lora.raw_lib()
assert lib.lora_attend_plan_set_tree(None, None, ctypes.byref(b), None, None) == lora.LORA_EINVAL
assert lib.lora_attend_plan_set_tree(None, None, None, None, None) == lora.LORA_EINVAL
print("ok")
"""


@pytest.mark.parametrize("flags", [[], SANITIZE], ids=["plain", "asan_ubsan"])
def test_counts_are_checked_before_the_lists_are_read(tmp_path, flags):
    _native_check(tmp_path, "attend_parent_check", "attend_plan.cpp", flags)


def test_no_plan_no_list_is_read():
    r = subprocess.run([sys.executable, "-c", UNREAD], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr
