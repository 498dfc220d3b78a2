"""Attention of prompts, whole and in chunks, of batches in another order, and
of batches that have nothing new."""
import numpy as np
import pytest
import torch

from rank_adapter_gemm_token_amd import lora
from test_attend_gpu import DT, Step

pytestmark = pytest.mark.gpu


def some(T, n, seed=0):
    """The first and last tokens, those about the borders of 32 and 64, others."""
    at = {0, 1, T - 1, T - 2, 31, 32, 33, 63, 64, 65, T // 2}
    return {t for t in at | {int(x) for x in np.random.default_rng(seed).integers(0, T, n)} if 0 <= t < T}


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 2, 64), (8, 1, 128), (3, 3, 128), (32, 1, 64)])
def test_a_whole_prompt(dtype, heads, kv_heads, dim):
    """A thousand new tokens see up to themselves, and no stale row past them."""
    with Step([1000], [1000], [-1], [], heads, kv_heads, dim, 16, dtype) as s:
        s.check(*s.run(), tokens=some(1000, 40))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_prompts_in_chunks_on_prefixes(dtype):
    """Chunks of two prompts in the middle, of one from its start, beside single
    tokens; prefixes that end inside a page and a tile."""
    q, kv = [512, 300, 1, 700, 5], [1536, 300, 800, 1111, 5]
    with Step(q, kv, [0, 1, 0, -1, 1], [777, 1000], 8, 2, 128, 64, dtype) as s:
        s.check(*s.run(), tokens=some(sum(q), 60))


def test_as_many_new_tokens_as_a_plan_takes():
    """65536 of them, in prompts of 512 on one prefix."""
    B, n = 128, 512
    with Step([n] * B, [n] * B, [0] * B, [130], 2, 1, 64, 64, "bf16") as s:
        assert s.T == lora.LORA_ATTEND_MAX_TOKENS
        s.check(*s.run(), tokens=some(s.T, 60))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_sequences_in_any_order_give_the_same_bits(dtype):
    """64 sequences of one group, with full blocks of query rows in any order:
    each one's output and lse do not depend on its neighbours or its place."""
    B, rng = 64, np.random.default_rng(4)
    kv = [int(x) for x in rng.integers(1, 400, B)]
    with Step([1] * B, kv, [0] * B, [640], 8, 8, 128, 16, dtype) as s:
        s.q = s.q.contiguous()
        out, lse = s.run()
        s.check(out, lse, tokens=some(B, 4))
        first = (s.q, s.kv_len, s.pages)
        for seed in range(3):
            at = [int(x) for x in np.random.default_rng(seed).permutation(B)]
            i = torch.tensor(at, device="cuda")
            s.q, s.kv_len, s.pages = first[0][i], [first[1][x] for x in at], [first[2][x] for x in at]
            o, l = s.run()
            assert torch.equal(o, out[i]) and torch.equal(l, lse[i])


def test_nothing_new_writes_nothing():
    """No sequences, and sequences without new tokens: out and lse stay."""
    with Step([0, 0], [20, 0], [0, -1], [33], 4, 2, 64, 16, "f16", room=4) as s:
        q = torch.ones((3, 4, 64), dtype=DT["f16"], device="cuda")
        none = torch.zeros(0, dtype=torch.int32)
        for set_plan in (s.set_plan, lambda: lora.lora_attend_plan_set(s.plan, s.kv, none, none, none, none, none)):
            set_plan()
            out, lse = torch.full_like(q, 7.0), torch.full((3, 4), 7.0, device="cuda")
            lora.lora_attend(s.kv, s.plan, q, 1.0, out, lse)
            torch.cuda.synchronize()
            assert (out == 7).all() and (lse == 7).all() and (q == 1).all()
