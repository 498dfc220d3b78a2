"""Draft verification where a running sum's rounding decides."""
import pytest
import torch

from rank_adapter_gemm_token_amd import lora

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("drafts", [0, 1])
@pytest.mark.parametrize("unit", [8, 512, 32768])
def test_a_place_without_weight_is_not_drawn(unit, drafts, dtype):
    """Weights t, t, 1/2, nothing, ..., 1/2 with t = 2^-54, a unit apart (a
    lane's, a segment's, a part's entries), and u times the whole = 1/2.  Added
    in one order t + t + 1/2 is above 1/2, in another it is 1/2, so the place
    after it may be the first whose running sum passes.  It has no weight: the
    token is one of the two of 1/2, by which order does not matter."""
    t, V = 2.0 ** -54, 32 * unit
    p = torch.zeros((1 + drafts, V))
    # The first row refuses its draft, and nothing of q is among the weights.
    p[:, [0, unit]], p[:, [2 * unit, 10 * unit]] = t, 0.5
    q = torch.zeros((drafts, V))
    q[:, 5 * unit] = 1.0
    i = dict(dtype=torch.int32, device="cuda")
    v = lora.lora_verifier_create(1)
    tokens, accepted = torch.full((1 + drafts,), -7, **i), torch.full((1,), -7, **i)
    u = torch.full((1 + drafts,), 0.5, device="cuda")
    lora.lora_verify(v, p.to(dtype).cuda(), q.to(dtype).cuda(), torch.full((drafts,), 5 * unit, **i),
                     torch.tensor([0, 1 + drafts], **i), u, 1, 1 + drafts, tokens, accepted)
    assert accepted.tolist() == [0]
    assert tokens[0].item() in (2 * unit, 10 * unit), tokens.tolist()
    assert tokens[1:].tolist() == [-1] * drafts
    torch.cuda.synchronize()
    lora.lora_verifier_destroy(v)
