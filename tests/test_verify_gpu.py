"""Draft verification against the 64-bit form: every token equal."""
import numpy as np
import pytest
import torch

import kv_reference as ref
from rank_adapter_gemm_token_amd import lora

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def call(p, q, draft, row0, u, verifier=None):
    B, T = len(row0) - 1, p.shape[0]
    v = lora.lora_verifier_create(B) if verifier is None else verifier
    i = dict(dtype=torch.int32, device="cuda")
    tokens, accepted = torch.full((T,), -7, **i), torch.full((B,), -7, **i)
    lora.lora_verify(v, p, q, torch.tensor(draft, **i), torch.tensor(row0, **i),
                     torch.tensor(u, dtype=torch.float32, device="cuda"), B, T, tokens, accepted)
    got = tokens.tolist(), accepted.tolist()
    if verifier is None:
        lora.lora_verifier_destroy(v)
    return got


def same(p, q, draft, row0, u, **kw):
    got = call(p, q, draft, row0, u, **kw)
    want = ref.verify(p.double().cpu().numpy(), q.double().cpu().numpy(), draft, row0,
                      np.asarray(u, dtype=np.float32).astype(np.float64))
    assert got[1] == want[1]
    assert got[0] == want[0]
    return got


def batch(n_drafts, V, dtype, seed, noise=0.7, sharp=2.0):
    g = torch.Generator().manual_seed(seed)
    n = np.asarray(n_drafts)
    T, D = int((n + 1).sum()), int(n.sum())
    row0 = [0] + [int(x) for x in np.cumsum(n + 1)]
    z = torch.randn((T, V), generator=g) * sharp
    rows = [row0[b] + i for b in range(len(n)) for i in range(n[b])]
    zq = z[rows] + noise * torch.randn((D, V), generator=g)
    p, q = torch.softmax(z, -1), torch.softmax(zq, -1)
    draft = [int(x) for x in torch.multinomial(q, 1, generator=g)] if D else []
    u = torch.rand((T,), generator=g).tolist()
    return p.to(DT[dtype]).cuda(), q.to(DT[dtype]).cuda(), draft, row0, u


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 7, 64, 1000, 2047, 2048, 2049, 4097, 32000, 50257, 140001])
def test_ragged_batches(dtype, V):
    kept = []
    for seed in range(3):
        rng = np.random.default_rng(seed)
        n = [int(x) for x in rng.integers(0, 8, 9)]
        kept += same(*batch(n, V, dtype, seed * 100 + V))[1]
    assert max(kept) > 0


def test_longest_drafts_and_one_sequence():
    same(*batch([63], 500, "f32", 1, noise=0.05))
    same(*batch([63, 0, 1], 500, "f32", 2, noise=0.0))  # all kept: the last token from p alone
    same(*batch([0], 40000, "f32", 3))
    same(*batch([1] * 300, 333, "f32", 4))


@pytest.mark.parametrize("V", [32767, 32768, 32769, 65536, 99999, 1 << 21])
@pytest.mark.parametrize("B", [1, 40, 300])
def test_rows_of_several_parts(V, B):
    """Rows of one and of many parts, by one workgroup and by several; few
    probabilities that are not 0, so that whole parts have none."""
    if B * V > 1 << 23:
        B = max(1, (1 << 23) // V)
    g = torch.Generator().manual_seed(V + B)
    n = [i % 2 for i in range(B)]
    row0 = [0] + [int(x) for x in np.cumsum(np.array(n) + 1)]
    p, q = torch.zeros(row0[-1], V), torch.zeros(sum(n), V)
    for x in (p, q):
        at = torch.randint(0, V, (len(x), 5), generator=g)
        x.scatter_(1, at, torch.rand(at.shape, generator=g))
    draft = [int(x) for x in q.argmax(1)]
    u = torch.rand(row0[-1], generator=g).tolist()
    u[0] = 1 - 2.0 ** -24
    same(p.cuda(), q.cuda(), draft, row0, u)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_borders(dtype):
    """u at both ends; p and q equal, far apart, with zeros; ties of the
    acceptance, which refuse; weights exactly summing to the aim."""
    V = 8
    p = torch.tensor([[0, .25, .25, 0, .5, 0, 0, 0]] * 4, dtype=DT[dtype], device="cuda")
    q = torch.tensor([[0, .5, .25, .25, 0, 0, 0, 0]] * 2, dtype=DT[dtype], device="cuda")
    row0 = [0, 2, 4]
    for u in (0.0, 0.25, 0.5, 0.75, 1 - 2.0 ** -24):
        for w in (0.0, 0.25, 0.5, 1 - 2.0 ** -24):
            for d in range(V):
                same(p, q, [d, 7 - d], row0, [u, w, w, u])
    # 0.5 q = p exactly: not below, refused; then index 4 has all that is left.
    assert call(p, q, [1, 1], row0, [0.5, 0.0, 0.5, 0.0]) == ([4, -1, 4, -1], [0, 0])
    # p = q: kept for any u; refused only where both are 0, and then drawn from p.
    assert call(p, p[:2].contiguous(), [0, 2], row0, [0.0, 0.0, 0.9, 0.99]) == ([1, -1, 2, 4], [0, 1])


def test_what_has_no_answer_says_so():
    V = 5000
    p, q, draft, row0, u = batch([2, 2, 2, 2, 2, 2], V, "f32", 7)
    u = [0.0] * len(u)
    draft[2] = V            # sequence 1: outside the vocabulary
    draft[5] = -1           # sequence 2
    p[row0[3]:row0[4]] = float("nan")   # the rows of an invalid token
    p[row0[4] + 2] = 0.0    # nothing to draw from after two kept
    p[row0[5] + 2, 77] = float("inf")
    tokens, accepted = same(p, q, draft, row0, u)
    assert accepted == [2, -1, -1, -1, -1, -1]
    assert tokens[row0[1]:] == [-1] * 15


def test_nan_and_negative_entries_weigh_nothing():
    V = 3000
    p, q, draft, row0, u = batch([3, 1], V, "f32", 9)
    p[:, 100:200] = float("nan")
    p[:, 200:300] = -1.0
    q[:, 250:400] = float("nan")
    same(p, q, draft, row0, u)


def test_lists_that_do_not_ascend_are_not_followed():
    p, q, draft, _, u = batch([1, 1, 1], 100, "f32", 11)
    for row0, ok in (([0, 2, 2, 6], [1, 0, 1]), ([0, 2, 1, 6], [1, 0, 0]), ([0, 2, 4, 7], [1, 1, 0]),
                     ([-1, 2, 4, 6], [0, 1, 1]), ([0, 6, 4, 6], [0, 0, 1]), ([1 << 30, 2, 4, -5], [0, 1, 0])):
        _, accepted = call(p, q, draft, row0, u)
        assert [a >= 0 for a in accepted] == [bool(x) for x in ok], (row0, accepted)


def test_a_verifier_again_and_again():
    """Its counters are back at rest after every call, of any size."""
    v = lora.lora_verifier_create(40)
    try:
        for i, (n, V) in enumerate([([3] * 40, 9000), ([1], 100), ([2, 0] * 10, 70000), ([3] * 40, 9000)]):
            same(*batch(n, V, "bf16", 50 + i), verifier=v)
    finally:
        lora.lora_verifier_destroy(v)


def test_graph_replays_match_eager_calls():
    v = lora.lora_verifier_create(5)
    i = dict(dtype=torch.int32, device="cuda")
    n = [2, 0, 4, 1, 3]
    p, q, draft, row0, u = batch(n, 20000, "f32", 1)
    dd, rr, uu = torch.tensor(draft, **i), torch.tensor(row0, **i), torch.tensor(u, device="cuda")
    tokens, accepted = torch.empty(len(u), **i), torch.empty(5, **i)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st), torch.cuda.graph(graph, stream=st):
        lora.lora_verify(v, p, q, dd, rr, uu, 5, len(u), tokens, accepted)
    for seed in range(4):
        p2, q2, draft, row0, u = batch(n, 20000, "f32", 20 + seed)
        p.copy_(p2), q.copy_(q2), dd.copy_(torch.tensor(draft, **i)), uu.copy_(torch.tensor(u))
        graph.replay()
        torch.cuda.synchronize()
        got = tokens.tolist(), accepted.tolist()
        assert got == same(p, q, draft, row0, u, verifier=v)
    torch.cuda.synchronize()
    lora.lora_verifier_destroy(v)


def test_refusals():
    import ctypes
    lib = lora.raw_lib()
    v = lora.lora_verifier_create(2)
    p, q, draft, row0, u = batch([1, 1], 64, "f32", 1)
    i = dict(dtype=torch.int32, device="cuda")
    d, r, x = torch.tensor(draft, **i), torch.tensor(row0, **i), torch.tensor(u, device="cuda")
    t, a = torch.empty(4, **i), torch.empty(2, **i)
    good = [v, p.data_ptr(), q.data_ptr(), 0, 64, d.data_ptr(), r.data_ptr(), x.data_ptr(), 2, 4, t.data_ptr(),
            a.data_ptr(), None]
    assert lib.lora_verify(*good) == lora.LORA_OK
    for at, bad in [(1, None), (2, None), (3, 5), (4, 0), (4, (1 << 21) + 1), (5, None), (6, None), (7, None), (8, -1),
                    (9, -1), (10, None), (11, None), (1, p.data_ptr() + 2), (6, r.data_ptr() + 1)]:
        args = list(good)
        args[at] = bad
        assert lib.lora_verify(*args) == lora.LORA_EINVAL, at
    args = list(good)
    args[8] = 3
    assert lib.lora_verify(*args) == lora.LORA_ETOKENS
    args[8] = 0
    assert lib.lora_verify(*args) == lora.LORA_OK
    with pytest.raises(ValueError):
        lora.lora_verify(v, p, q.half(), d, r, x, 2, 4, t, a)
    with pytest.raises(ValueError):
        lora.lora_verify(v, p, q, d, r, x.double(), 2, 4, t, a)
    torch.cuda.synchronize()
    lora.lora_verifier_destroy(v)
