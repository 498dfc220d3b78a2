"""Draft verification with bounds of rows whose difference passes 32 bits."""
import pytest
import torch

from rank_adapter_gemm_token_amd import lora

pytestmark = pytest.mark.gpu

TOP = 2 ** 31 - 1


@pytest.mark.parametrize("row0", [[0, TOP, -TOP - 1], [0, TOP, -TOP + 10], [TOP, -TOP - 1, 4], [0, 2, -TOP - 1]])
def test_bounds_far_apart_are_not_followed(row0):
    """(-2^31) - (2^31 - 1) is 1 in 32 bits: a sequence without drafts, at row
    2^31 - 1, if the difference were asked alone."""
    i = dict(dtype=torch.int32, device="cuda")
    v = lora.lora_verifier_create(2)
    p, q, u = torch.ones((4, 8), device="cuda"), torch.ones((2, 8), device="cuda"), torch.full((4,), 0.5, device="cuda")
    tokens, accepted = torch.full((4,), -7, **i), torch.full((2,), -7, **i)
    lora.lora_verify(v, p, q, torch.zeros(2, **i), torch.tensor(row0, **i), u, 2, 4, tokens, accepted)
    good = [b <= row0[b] < row0[b + 1] <= 4 - (1 - b) for b in range(2)]
    assert [a >= 0 for a in accepted.tolist()] == good
    assert all(t == -7 for t in tokens.tolist()[2 if good[0] else 0:])
    torch.cuda.synchronize()
    lora.lora_verifier_destroy(v)
