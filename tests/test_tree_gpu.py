"""Attention of drafted trees over the quantised cache against the 64-bit form,
token by token: shapes and sizes of trees, types, head layouts, lengths from
none to long, shared prefixes, ragged batches, split and unsplit work, poisoned
nodes, chains, graphs replayed over plans of both kinds.  The tolerance is
kv_reference's, derived there."""
import gc

import numpy as np
import pytest
import torch

import tree_reference as tree
from rank_adapter_gemm_token_amd import lora
from test_attend_gpu import DT, Step

pytestmark = pytest.mark.gpu


def parents(kind, n, rng):
    if kind == "chain":
        return [j - 1 for j in range(n)]
    if kind == "star":       # all siblings below the first
        return [-1] + [0] * (n - 1)
    if kind == "roots":      # each follows the context alone
        return [-1] * n
    if kind == "binary":
        return [(j + 1) // 2 - 1 for j in range(n)]
    if kind == "combs":      # two long branches, their nodes in turn
        return [-1, 0, 0][:n] + [j - 2 for j in range(3, n)]
    if kind == "forest":
        return [int(rng.integers(-1, j)) if j else -1 for j in range(n)]
    return [int(rng.integers(max(0, j - 5), j)) if j else -1 for j in range(n)]  # "near"


KINDS = ["chain", "star", "roots", "binary", "combs", "forest", "near"]


class TreeStep(Step):
    def __init__(self, kinds, *args, **kw):
        super().__init__(*args, **kw)
        rng = np.random.default_rng(kw.get("seed", 0) + 99)
        self.trees = [parents(k, n, rng) for k, n in zip(kinds, self.q_len)]

    def parent(self):
        return torch.tensor([p for t in self.trees for p in t], dtype=torch.int32)

    def set_plan(self, stream=None):
        lora.lora_attend_plan_set_tree(self.plan, self.kv, self.parent(), **self.lists(), stream=stream)

    def seen(self, s, j):
        before = self.kv_len[s] - self.q_len[s]
        last = super().seen(s, self.q_len[s] - 1)          # the prefix and all of the sequence's own
        first = len(last) - max(0, self.kv_len[s])
        own = [before + i for i in tree.sees(self.trees[s], j)]
        return last[:first + max(0, before)] + [last[first + i] for i in own if i >= 0]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 8, 128), (14, 2, 64), (32, 1, 128), (12, 4, 128)])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,before", [(1, 0), (2, 63), (7, 64), (16, 1), (33, 500), (65, 40), (130, 0)])
def test_one_tree(dtype, heads, kv_heads, dim, kind, n, before):
    with TreeStep([kind], [n], [n + before], [-1], [], heads, kv_heads, dim, 16, dtype, seed=n) as s:
        s.check(*s.run())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,dim,page", [(8, 8, 128, 64), (8, 2, 128, 16), (6, 2, 64, 32)])
@pytest.mark.parametrize("prefix", [[1], [64], [300, 0, 77], [2049, 130]])
def test_batches_with_prefixes(dtype, heads, kv_heads, dim, page, prefix):
    rng = np.random.default_rng(len(prefix) + prefix[0])
    B = 23
    q_len = [int(x) for x in rng.integers(0, 20, B)]
    kv_len = [int(n + x) for n, x in zip(q_len, rng.integers(0, 150, B))]
    kv_len[3] = q_len[3] // 2   # its first new tokens have no key
    kv_len[4] = 0
    group = [int(x) for x in rng.integers(-1, len(prefix), B)]
    group[4] = -1
    kinds = [KINDS[int(x)] for x in rng.integers(0, len(KINDS), B)]
    with TreeStep(kinds, q_len, kv_len, group, prefix, heads, kv_heads, dim, page, dtype, seed=B) as s:
        s.check(*s.run())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("kind", ["near", "binary", "forest"])
def test_long_contexts_and_large_trees(dtype, kind):
    """Spans split over workgroups; trees over several tiles and pages."""
    with TreeStep([kind] * 2, [40, 700], [5040, 1400], [-1, 0], [900], 8, 2, 128, 64, dtype, seed=4) as s:
        out, lse = s.run()
        s.check(out, lse, set(range(40)) | set(range(40, 740, 23)))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_hidden_nodes_do_not_count_whatever_they_hold(dtype):
    """A poisoned node reaches itself and what is below it; a key far above the
    others in a sibling moves nothing."""
    q_len, kv_len = [16, 16], [90, 16]
    with TreeStep(["binary", "star"], q_len, kv_len, [-1, -1], [], 8, 2, 64, 16, dtype, seed=8) as s:
        node = [[s.pages[b][i // 16] * 16 + i % 16 for i in range(kv_len[b] - 16, kv_len[b])] for b in range(2)]
        s.k_in[node[0][4], 0, 3] = float("nan")
        s.v_in[node[0][6], 1, 5] = float("inf")
        s.k_in[node[1][7]] *= 1000.0
        s.k_in[node[1][9], 1, 0] = float("-inf")
        s.write()
        out, lse = s.run()
        s.check(out, lse)
        assert out[:16].isnan().any(-1).any(-1).tolist() == [j in (4, 9, 10, 6, 13, 14) for j in range(16)]
        assert out[16:].isnan().any(-1).any(-1).tolist() == [j == 9 for j in range(16)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_a_chain_is_a_chain(dtype):
    q_len, kv_len, group = [5, 1, 17, 0, 3], [300, 1, 17, 9, 2], [0, -1, 0, 0, -1]
    with TreeStep(["chain"] * 5, q_len, kv_len, group, [130], 8, 2, 128, 16, dtype) as s:
        out, lse = s.run()
        s.check(out, lse)
        Step.set_plan(s)
        again, lse2 = s.run(plan=False)
        assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("captured", ["tree", "chain", "none"])
def test_graphs_are_replayed_over_plans_of_both_kinds(captured):
    """One graph, captured with a plan of one kind, replayed after others."""
    q_len, kv_len = [9, 14, 3], [200, 30, 3]
    stream = torch.cuda.Stream()
    with TreeStep(["near", "binary", "star"], q_len, kv_len, [0, -1, 0], [70], 8, 2, 128, 16, "bf16") as s:
        out = torch.empty((s.T, 8, 128), dtype=s.dtype, device="cuda")
        lse = torch.empty((s.T, 8), device="cuda")
        e = torch.zeros(0, dtype=torch.int32)
        if captured == "tree":
            s.set_plan()
        elif captured == "chain":
            Step.set_plan(s)
        else:
            lora.lora_attend_plan_set_tree(s.plan, s.kv, e, e, e, e, e, e)
        torch.cuda.synchronize()
        gc.collect()
        gc.disable()
        try:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                lora.lora_attend(s.kv, s.plan, s.q, s.scale, out, lse, stream=torch.cuda.current_stream())
        finally:
            gc.enable()
        rng = np.random.default_rng(5)
        for i in range(4):
            s.trees = [parents(KINDS[(i + b) % len(KINDS)], n, rng) for b, n in enumerate(q_len)]
            s.set_plan()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            s.check(out, lse)
            eager, elsa = s.run()
            if captured != "none":  # launched as the eager call is
                assert torch.equal(out, eager) and torch.equal(lse, elsa)
            s.check(eager, elsa)
        # A chain's plan.
        s.trees = [parents("chain", n, rng) for n in q_len]
        Step.set_plan(s)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        s.check(out, lse)
        # A refused tree: NaN for the tokens of the plan before.
        bad = s.parent()
        bad[3] = 3
        with pytest.raises(lora.LoraError):
            lora.lora_attend_plan_set_tree(s.plan, s.kv, bad, **s.lists())
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert out.isnan().all() and lse.isnan().all()
        s.set_plan()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        s.check(out, lse)


def test_refusals():
    with TreeStep(["near"], [6], [20], [-1], [], 4, 2, 64, 16, "f16") as s:
        good = s.parent()
        out, lse = s.run()
        for at, bad in [(0, 0), (0, -2), (3, 3), (3, 4), (5, 1 << 30), (2, -(1 << 31))]:
            p = good.clone()
            p[at] = bad
            with pytest.raises(lora.LoraError) as e:
                lora.lora_attend_plan_set_tree(s.plan, s.kv, p, **s.lists())
            assert e.value.status == lora.LORA_EINVAL
            with pytest.raises(lora.LoraError):  # the plan is empty
                lora.lora_attend(s.kv, s.plan, s.q, s.scale, out, lse)
        lists = {k: v for k, v in s.lists().items()}
        b = lora._batch(**lists)
        import ctypes
        assert lora.raw_lib().lora_attend_plan_set_tree(s.plan, s.kv, ctypes.byref(b), None, None) == lora.LORA_EINVAL
        again, _ = s.run()
        assert torch.equal(out, again)
