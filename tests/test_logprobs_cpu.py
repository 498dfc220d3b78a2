"""The log probabilities, as far as no GPU is needed: arguments refused before
the device is touched and the binding's own checks."""
import ctypes
import os

import pytest
import torch

from rank_adapter_gemm_token_amd import lora

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_create_refuses():
    lib, h = lora.raw_lib(), ctypes.c_void_p(1)
    for n in (0, -1, (1 << 20) + 1):
        assert lib.lora_scorer_create(n, ctypes.byref(h)) == lora.LORA_EINVAL
        assert not h.value
    assert lib.lora_scorer_create(1, None) == lora.LORA_EINVAL
    assert lib.lora_scorer_destroy(None) == lora.LORA_OK
    assert lib.lora_logprobs(None, None, 8, 0, 8, None, 1.0, 0, 1, None, None, None, None, None) == lora.LORA_EINVAL


def test_limits_match_header():
    text = open(os.path.join(ROOT, "include", "lora.h")).read()
    for name in ("LORA_SCORE_MAX_ROWS", "LORA_SCORE_MAX_TOP"):
        value = text.split("#define " + name)[1].split("/*")[0].split("\n")[0].strip()
        assert eval(value) == getattr(lora, name), name


def test_binding_refuses():
    z = torch.zeros(3, 8)
    for bad in (z, z[0], z.long()):
        with pytest.raises(ValueError, match="logits"):
            lora.lora_logprobs(None, bad, None, stream=0)
