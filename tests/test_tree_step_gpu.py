"""The serving step of examples/tree_step.py: the routed products, appended and
turned keys, the attention of drafted trees, the walk and the log probabilities
together."""
import importlib.util
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

EXAMPLES = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples")


def example():
    sys.path.insert(0, EXAMPLES)
    try:
        spec = importlib.util.spec_from_file_location("tree_step", os.path.join(EXAMPLES, "tree_step.py"))
        m = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(m)
    finally:
        sys.path.remove(EXAMPLES)
    return m


def close_to(a, b):
    """Logits after the same tokens.  Each way rounds to 16 bits some twelve times
    one after the other (norm, products, attention, residual of two layers, norm,
    head), each off by at most 2^-8 (bf16) of the row's size: sqrt(12) 2^-8 = 1.4e-2
    for roundings that have nothing to do with each other, and sqrt(2) of that
    between two such ways, 2e-2 of the row's largest logit.  (Probabilities would
    be off by exp of as much of a logit: a logit of 5 by its own rounding alone,
    2^-8 of it each way, moves its probability by 4e-2.)"""
    a, b = a.float(), b.float()
    return ((a - b).abs().amax(1) / b.abs().amax(1)).max().item() <= 2e-2


def test_steps_make_tokens():
    torch.manual_seed(1)
    m = example()
    s = m.Server()
    before = list(s.kv_len)
    for _ in range(5):
        kept, scores = s.step()
        assert all(1 <= len(k) <= 5 and all(0 <= t < s.vocab for t in k) for k in kept)
        assert [len(k) for k in kept] == [a - b for a, b in zip(s.kv_len, before)] == [len(x) for x in scores]
        assert all(x <= 0 for y in scores for x in y)
        before = list(s.kv_len)
    s.close()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_a_node_sees_what_its_path_sees(dtype):
    """Each path of the tree as a chain of its own: the same logits."""
    m = example()
    s = m.Server(dtype=dtype)
    g = torch.Generator().manual_seed(2)
    S, n = len(s.last), len(m.PARENT)
    tokens = torch.randint(s.vocab, (S, n), generator=g).tolist()
    tree = s.logits(tokens, [m.PARENT] * S).view(S, n, -1).clone()
    for leaf in (4, 5, 6):
        path, j = [], leaf
        while j >= 0:
            path.insert(0, j)
            j = m.PARENT[j]
        chain = s.logits([[t[i] for i in path] for t in tokens]).view(S, len(path), -1)
        for at, i in enumerate(path):
            assert close_to(tree[:, i], chain[:, at]), (leaf, i)
    s.close()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_kept_paths_continue_as_their_tokens_would(dtype):
    """After a path through the tree is kept and moved to the front, the next
    token's logits are those after the same tokens given one at a time."""
    m = example()
    a, b = m.Server(dtype=dtype), m.Server(dtype=dtype)
    g = torch.Generator().manual_seed(3)
    S, n = len(a.last), len(m.PARENT)
    tokens = torch.randint(a.vocab, (S, n), generator=g).tolist()
    paths = [[[0, 2, 5], [0, 1, 4], [0], [0, 1, 3, 6]][s % 4] for s in range(S)]
    a.logits(tokens, [m.PARENT] * S)
    a.keep(paths)
    a.kv_len = [c + len(p) for c, p in zip(a.kv_len, paths)]
    for step in range(4):
        # Sequences whose path has ended write a token that the next one is put in the place of.
        b.logits([[t[p[min(step, len(p) - 1)]]] for t, p in zip(tokens, paths)])
        b.kv_len = [c + (step < len(p)) for c, p in zip(b.kv_len, paths)]
    assert a.kv_len == b.kv_len
    last = torch.randint(a.vocab, (S, 1), generator=g).tolist()
    assert close_to(a.logits(last), b.logits(last))
    a.close()
    b.close()


def test_the_scores_are_the_tokens_probabilities():
    """Whatever is drawn, its score is its row's."""
    m = example()
    torch.manual_seed(4)
    s = m.Server()
    S, n = len(s.last), len(m.PARENT)
    trees = s.draft()
    z = s.logits(trees, [m.PARENT] * S).view(S, n, -1).float().clone()
    kept, scores = s.step(torch.rand(S * n, device="cuda"))
    for b in range(S):
        node = 0
        for t, x in zip(kept[b], scores[b]):
            # Both are fp32 sums over 1024 entries of the same logits.
            assert abs(torch.log_softmax(z[b, node].double(), -1)[t].item() - x) <= 1e-5
            node = next((j for j in range(n) if m.PARENT[j] == node and trees[b][j] == t), None)
    s.close()
