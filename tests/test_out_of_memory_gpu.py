"""A handle that does not fit the device is refused, and that is all: the next
call on another one is not told of it."""
import pytest
import torch

from rank_adapter_gemm_token_amd import lora

pytestmark = pytest.mark.gpu


def too_large():
    """More than a device holds, many times over: nothing is allocated."""
    return [
        lambda: lora.lora_kv_create((1 << 27) - 1, 16, 256, 128, torch.float16),
        lambda: lora.lora_attend_plan_create(1, 0, 65536, 1, 8192, 256, 128),
        lambda: lora.lora_pool_create(1 << 24, 64, 64, 1024, 16, torch.float16),
    ]


@pytest.mark.parametrize("which", range(3))
def test_the_next_call_is_none_the_wiser(which):
    kv = lora.lora_kv_create(4, 16, 2, 64, torch.float16)
    k, s = torch.ones((3, 2, 64), dtype=torch.float16, device="cuda"), torch.tensor([5, 6, 9], dtype=torch.int32).cuda()
    try:
        with pytest.raises(lora.LoraError) as e:
            too_large()[which]()
        assert e.value.status == lora.LORA_ENOMEM
        lora.lora_kv_write(kv, k, k, s, 3)
        assert not torch.isnan(torch.ones(5, device="cuda")).any()  # nor torch's
        a, b = torch.empty_like(k), torch.empty_like(k)
        lora.lora_kv_read(kv, s, 3, a, b)
        assert torch.equal(a, k) and torch.equal(b, k)
    finally:
        lora.lora_kv_destroy(kv)
