"""The serving step of examples/draft_step.py: the routed products, the cache,
the attention and the verification together."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "draft_step.py")


def example():
    spec = importlib.util.spec_from_file_location("draft_step", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_steps_make_tokens():
    torch.manual_seed(1)
    s = example().Server(drafts=4)
    before = list(s.kv_len)
    for _ in range(5):
        kept = s.step()
        assert all(1 <= len(k) <= 5 and all(0 <= t < s.vocab for t in k) for k in kept)
        assert [len(k) for k in kept] == [a - b for a, b in zip(s.kv_len, before)]
        assert [k[-1] for k in kept] == s.last
        before = list(s.kv_len)
    s.close()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_drafted_tokens_see_what_single_ones_see(dtype):
    """Probabilities after four new tokens at once and after one at a time: the
    same keys are seen, so they agree to the 16-bit rounding of the layers'
    products (2e-2, the products' own tolerance)."""
    m = example()
    s = m.Server(drafts=3, dtype=dtype)
    g = torch.Generator().manual_seed(2)
    tokens = torch.randint(s.vocab, (len(s.last), 4), generator=g).tolist()
    together = s.probabilities(tokens).view(len(s.last), 4, -1).clone()
    for j in range(4):
        alone = s.probabilities([[t[j]] for t in tokens])
        s.kv_len = [n + 1 for n in s.kv_len]
        err = (together[:, j] - alone).abs().amax(1) / alone.amax(1)
        assert err.max() <= 2e-2, (j, err.max())
    s.close()


def test_a_draft_equal_to_the_target_is_kept():
    """u q(d) < p(d) for every u below 1 where q = p: all drafts are kept."""
    m = example()
    s = m.Server(drafts=3)
    torch.manual_seed(3)
    tokens = [[t] for t in s.last]
    rows = []
    for _ in range(3):  # draft with the target itself, one token at a time
        p = s.probabilities([[t[-1]] for t in tokens])
        s.kv_len = [n + 1 for n in s.kv_len]
        rows.append(p)
        for t, new in zip(tokens, torch.multinomial(p, 1)[:, 0].tolist()):
            t.append(new)
    last = s.probabilities([[t[-1]] for t in tokens])
    S = len(tokens)
    p = torch.stack(rows + [last], 1).flatten(0, 1).contiguous()
    q = torch.stack(rows, 1).flatten(0, 1).contiguous()
    out, acc = torch.empty(4 * S, dtype=torch.int32, device="cuda"), torch.empty(S, dtype=torch.int32, device="cuda")
    m.lora.lora_verify(s.verifier, p, q, m.i32([x for t in tokens for x in t[1:]], "cuda"),
                       m.i32([4 * i for i in range(S + 1)], "cuda"), torch.rand(4 * S, device="cuda"), S, 4 * S, out, acc)
    assert acc.tolist() == [3] * S
    assert out.view(S, 4)[:, :3].tolist() == [t[1:] for t in tokens]
    s.close()
