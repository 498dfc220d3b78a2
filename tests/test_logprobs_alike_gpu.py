"""A token has one log probability, bit for bit: as the given token and as an
alternative, at every place, however many alternatives are asked for."""
import pytest
import torch

from rank_adapter_gemm_token_amd import lora
from test_logprobs_gpu import Scorer, buffers, logits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,vocab", [(150, 300), (40, 8000), (20, 9000), (600, 20000), (3, 131072)])
def test_given_and_alternative(dtype, n, vocab):
    z = logits(n, vocab, dtype, vocab)
    with Scorer(n) as s:
        lp, h, ids, tlp = buffers(n, 32)
        lora.lora_logprobs(s, z, None, 0.9, None, h, ids, tlp)
        for k in range(32):
            lora.lora_logprobs(s, z, ids[:, k].contiguous(), 0.9, lp, None, ids, tlp)
            assert torch.equal(lp, tlp[:, k]), k
        for top in (0, 1, 5, 17):
            one, hh, i, t = buffers(n, top)
            lora.lora_logprobs(s, z, ids[:, 31].contiguous(), 0.9, one, hh, i, t)
            assert torch.equal(one, lp) and torch.equal(hh, h) and torch.equal(t, tlp[:, :top]), top
