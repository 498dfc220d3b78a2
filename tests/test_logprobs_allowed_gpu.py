"""Rows of which a mask of -inf leaves one range of neighbouring tokens, or fewer
tokens than alternatives are asked for: what a grammar allows."""
import pytest
import torch

from rank_adapter_gemm_token_amd import lora
from test_logprobs_gpu import Scorer, buffers, check, logits

pytestmark = pytest.mark.gpu


def allowed(n, vocab, dtype, kind):
    z = logits(n, vocab, dtype, n + vocab).contiguous()
    keep = torch.zeros((n, vocab), dtype=torch.bool, device="cuda")
    for r in range(n):
        first = (r * 7919) % (vocab - 4000)
        if kind == "range":        # neighbours: few groups of lanes hold any
            keep[r, first:first + 200 + r % 3] = True
        elif kind == "long":       # more than a list holds, in half of the groups at most
            keep[r, first:first + 3000] = True
        elif kind == "few":        # fewer than the alternatives
            keep[r, first:first + 17 * (r % 4 + 1):17] = True
        else:                      # one, and at the row's end
            keep[r, vocab - 1] = True
    return z.masked_fill_(~keep, float("-inf")), keep


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind", ["range", "long", "few", "one"])
@pytest.mark.parametrize("n,vocab", [(2, 131072), (64, 131072), (300, 33000), (600, 20000), (5, 7000)])
def test_allowed(dtype, kind, n, vocab):
    z, keep = allowed(n, vocab, dtype, kind)
    t = keep.int().argmax(1).to(torch.int32)
    rows = sorted({0, 1, n // 2, n - 1})
    with Scorer(n) as s:
        for top in (1, 20, 32):
            got = buffers(n, top)
            lora.lora_logprobs(s, z, t.cuda(), 1.0, *got)
            check(z, t.cpu(), 1.0, top, got, rows)
            # Nothing forbidden stands before something allowed.
            some = keep.sum(1).clamp(max=top)
            good = keep.gather(1, got[2].long())
            assert torch.equal(good.sum(1), some)
            assert torch.equal(good, torch.arange(top, device="cuda") < some[:, None])
