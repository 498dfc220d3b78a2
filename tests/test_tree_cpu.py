"""Attention plans of drafted trees, as far as no GPU is needed: the planner
(compiled on its own), refusals, and the binding's own checks."""
import ctypes

import pytest
import torch

from rank_adapter_gemm_token_amd import lora
from test_host_cpu import SANITIZE, _native_check


@pytest.mark.parametrize("flags", [[], SANITIZE], ids=["plain", "asan_ubsan"])
def test_tree_planner(tmp_path, flags):
    _native_check(tmp_path, "attend_tree_check", "attend_plan.cpp", flags)


def test_null_handles():
    b = lora.lora_attend_batch()
    assert lora.raw_lib().lora_attend_plan_set_tree(None, None, ctypes.byref(b), None, None) == lora.LORA_EINVAL
    assert lora.raw_lib().lora_verify_tree(None, None, 0, 8, None, None, None, None, 1, 1, None, None, None,
                                           None) == lora.LORA_EINVAL


def test_binding_refuses():
    i = torch.zeros(2, dtype=torch.int32)
    lora._attend_plans[None] = [4, 64, 0]
    try:
        args = dict(q_len=i + 2, kv_len=i + 2, group=i - 1, pages=i[:0], page0=torch.zeros(3, dtype=torch.int32))
        for bad in (None, torch.zeros(3, dtype=torch.int32), torch.zeros(4), torch.zeros(8, dtype=torch.int32)[::2]):
            with pytest.raises(ValueError, match="parent"):
                lora.lora_attend_plan_set_tree(None, None, bad, **args, stream=0)
        with pytest.raises(lora.LoraError):  # long enough: the library's turn, which knows no such plan
            lora.lora_attend_plan_set_tree(None, None, torch.zeros(4, dtype=torch.int32), **args, stream=0)
    finally:
        del lora._attend_plans[None]
