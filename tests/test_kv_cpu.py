"""The quantised cache, the attention over it and the draft verification, as
far as no GPU is needed: arguments refused before the device is touched, the
binding's own checks, and the attention planner (compiled on its own)."""
import ctypes
import os
import subprocess

import pytest
import torch

from rank_adapter_gemm_token_amd import lora
from test_host_cpu import SANITIZE, _native_check

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EINVAL, OK = lora.LORA_EINVAL, lora.LORA_OK


@pytest.mark.parametrize("flags", [[], SANITIZE], ids=["plain", "asan_ubsan"])
def test_attend_planner(tmp_path, flags):
    _native_check(tmp_path, "attend_plan_check", "attend_plan.cpp", flags)


def test_kv_create_refuses():
    lib, h = lora.raw_lib(), ctypes.c_void_p(1)
    for args in [(0, 16, 1, 128, 1), (1, 8, 1, 128, 1), (1, 24, 1, 128, 1), (1, 2048, 1, 128, 1), (1, 16, 0, 128, 1),
                 (1, 16, 257, 128, 1), (1, 16, 1, 96, 1), (1, 16, 1, 128, 0), (1, 16, 1, 128, 7),
                 (1 << 27, 16, 1, 128, 1)]:
        assert lib.lora_kv_create(*args, ctypes.byref(h)) == EINVAL, args
        assert not h.value
    assert lib.lora_kv_create(1, 16, 1, 128, 1, None) == EINVAL


def test_null_handles():
    lib = lora.raw_lib()
    n = ctypes.c_uint64()
    f = ctypes.c_float(1.0)
    assert lib.lora_kv_destroy(None) == OK
    assert lib.lora_kv_write(None, None, 0, None, 0, None, 1, None) == EINVAL
    assert lib.lora_kv_read(None, None, 1, None, None, None) == EINVAL
    assert lib.lora_kv_poll_errors(None, ctypes.byref(n)) == EINVAL
    assert lib.lora_attend_plan_destroy(None) == OK
    b = lora.lora_attend_batch()
    assert lib.lora_attend_plan_set(None, None, ctypes.byref(b), None) == EINVAL
    assert lib.lora_attend(None, None, None, 0, f, None, None, None) == EINVAL
    assert lib.lora_verifier_destroy(None) == OK
    assert lib.lora_verify(None, None, None, 0, 8, None, None, None, 1, 1, None, None, None) == EINVAL


def test_plan_and_verifier_create_refuse():
    lib, h = lora.raw_lib(), ctypes.c_void_p(1)
    good = [4, 1, 8, 16, 8, 2, 128]
    for at, bad in [(0, 0), (0, 65537), (1, -1), (1, 65537), (2, 0), (2, 65537), (3, -1), (3, (1 << 26) + 1),
                    (4, 7), (4, 1), (4, 66), (5, 0), (5, 257), (6, 80)]:
        args = list(good)
        args[at] = bad
        assert lib.lora_attend_plan_create(*args, ctypes.byref(h)) == EINVAL, args
        assert not h.value
    assert lib.lora_attend_plan_create(*good, None) == EINVAL
    for n in (0, -1, 65536):
        assert lib.lora_verifier_create(n, ctypes.byref(h)) == EINVAL
    assert lib.lora_verifier_create(1, None) == EINVAL


def test_batch_struct_layout_matches_header(tmp_path):
    fields = [n for n, _ in lora.lora_attend_batch._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(
        ['#include <stdio.h>', '#include <stddef.h>', '#include "lora.h"', 'int main(void){',
         'printf("%zu\\n", sizeof(lora_attend_batch));'] +
        ['printf("%%zu\\n", offsetof(lora_attend_batch, %s));' % f for f in fields] + ['return 0;}']))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(lora.lora_attend_batch)] + [getattr(lora.lora_attend_batch, f).offset for f in fields]


def test_limits_match_header():
    text = open(os.path.join(ROOT, "include", "lora.h")).read()
    for name in ("LORA_KV_MAX_HEADS", "LORA_KV_MAX_PAGE", "LORA_ATTEND_MAX_TOKENS", "LORA_ATTEND_MAX_PAGES",
                 "LORA_VERIFY_MAX_SEQS", "LORA_VERIFY_MAX_VOCAB", "LORA_VERIFY_MAX_DRAFTS"):
        value = text.split("#define " + name)[1].split("/*")[0].split("\n")[0].strip()
        assert eval(value) == getattr(lora, name), name


def test_binding_refuses_host_and_misshaped_tensors():
    """Checked before the library is called, so a handle that names nothing will do."""
    lora._kvs[-1] = (2, 64, torch.float16)
    lora._attend_plans[-1] = [4, 64, 3]
    try:
        k, s = torch.zeros(3, 2, 64, dtype=torch.float16), torch.zeros(3, dtype=torch.int32)
        with pytest.raises(ValueError, match="device"):
            lora.lora_kv_write(-1, k, k, s, 3)
        with pytest.raises(ValueError, match="device"):
            lora.lora_kv_read(-1, s, 3, k, k)
        with pytest.raises(ValueError, match="device"):
            lora.lora_attend(-1, -1, torch.zeros(3, 4, 64, dtype=torch.float16), 1.0, k)
        i = torch.zeros(2, dtype=torch.int32)
        with pytest.raises(ValueError, match="kv_len"):
            lora.lora_attend_plan_set(-1, -1, i, i.long(), i, i, torch.zeros(3, dtype=torch.int32))
        with pytest.raises(ValueError, match="pages"):
            lora.lora_attend_plan_set(-1, -1, i, i, i, i, torch.tensor([0, 2, 5], dtype=torch.int32))
        with pytest.raises(ValueError, match="prefix_page0"):
            lora.lora_attend_plan_set(-1, -1, i, i, i, i, torch.tensor([0, 1, 2], dtype=torch.int32), i, i,
                                      torch.tensor([0, 1], dtype=torch.int32))
    finally:
        del lora._kvs[-1], lora._attend_plans[-1]
