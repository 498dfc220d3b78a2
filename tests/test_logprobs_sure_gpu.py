"""Rows with one logit far above the others, at many magnitudes: no log
probability is above 0 and no entropy below, whatever rounds."""
import pytest
import torch

from rank_adapter_gemm_token_amd import lora
from test_logprobs_gpu import DT, Scorer, buffers, check

pytestmark = pytest.mark.gpu


def sure(n, vocab, dtype, gap, seed):
    """Row r's largest logit is anywhere in 2^-4 .. 2^6 of either sign, the others
    `gap` and up to 3 more below it."""
    g = torch.Generator().manual_seed(seed)
    most = torch.exp2(torch.rand((n, 1), generator=g) * 10 - 4) * torch.where(torch.rand((n, 1), generator=g) < 0.3, -1.0, 1.0)
    z = (most - gap - 3 * torch.rand((n, vocab), generator=g)).to(DT[dtype])
    at = torch.randint(0, vocab, (n, 1), generator=g)
    z.scatter_(1, at, most.to(DT[dtype]))
    return z.cuda(), at[:, 0].to(torch.int32)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,vocab", [(200, 17), (200, 2500), (120, 9000), (600, 10000), (3, 70000)])
@pytest.mark.parametrize("scale", [0.3, 0.8, 1.0, 1.0 / 0.7, 5.0])
@pytest.mark.parametrize("gap", [400.0, 40.0, 18.0])
def test_signs(dtype, n, vocab, scale, gap):
    z, at = sure(n, vocab, dtype, gap, vocab + n)
    got = buffers(n, 3)
    with Scorer(n) as s:
        lora.lora_logprobs(s, z, at.cuda(), scale, *got)
        lp, h, ids, tlp = got
        assert (lp <= 0).all() and (h >= 0).all() and (tlp <= 0).all()
        assert not torch.signbit(h).any()
        assert torch.equal(ids[:, 0].cpu(), at)
        check(z, at, scale, 3, got, range(0, n, max(1, n // 6)))
