"""Positions of several axes: a tensor whose axes do not lie n_tokens apart is
refused before the device is touched."""
import pytest
import torch

from rank_adapter_gemm_token_amd import lora


@pytest.fixture
def handles():
    """A cache and tables of the binding's that the library does not know."""
    lora._kvs[-1] = (2, 64, torch.float16)
    lora._ropes[-1], lora._ropes[-3] = 1, 3
    yield
    del lora._kvs[-1], lora._ropes[-1], lora._ropes[-3]


def call(rope, positions, n=4):
    k, s = torch.zeros(n, 2, 64, dtype=torch.float16), torch.zeros(n, dtype=torch.int32)
    lora.lora_kv_append(-1, rope, k, k, s, positions, n, stream=0)


@pytest.mark.parametrize("shape", [(3, 5), (3, 64), (4, 3), (12, 1), (1, 12), (2, 3, 2)])
def test_another_pitch_is_refused(handles, shape):
    with pytest.raises(ValueError, match="positions: expected \\[3, 4\\]"):
        call(-3, torch.zeros(shape, dtype=torch.int32))


@pytest.mark.parametrize("rope,shape", [(-3, (3, 4)), (-3, (4, 4)), (-3, (12,)), (-3, (64,)), (-1, (4,)), (-1, (1, 64)),
                                        (-1, (64, 1)), (-1, (9,))])
def test_these_are_not(handles, rope, shape):
    """Refused for being on the host alone: keys are looked at next."""
    with pytest.raises(ValueError, match="k: expected a device tensor"):
        call(rope, torch.zeros(shape, dtype=torch.int32))


def test_no_tokens_no_positions(handles):
    with pytest.raises(ValueError, match="k: expected a device tensor"):
        call(-3, torch.zeros((3, 64), dtype=torch.int32), n=0)
