"""The walk down drafted trees against the 64-bit form: every token and node
equal.  Types, vocabularies, shapes and sizes of trees, ragged batches, rows
without weight, lists of parents and rows that are none, siblings that hold the
same token, borders of a running sum, the distribution of what comes out,
graphs."""
import gc

import numpy as np
import pytest
import torch

import tree_reference as ref
from rank_adapter_gemm_token_amd import lora
from test_tree_gpu import KINDS, parents

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
I = dict(dtype=torch.int32, device="cuda")


def call(p, draft, parent, row0, u, verifier=None, n_rows=None):
    B, T = len(row0) - 1, p.shape[0] if n_rows is None else n_rows
    v = lora.lora_verifier_create(B) if verifier is None else verifier
    tokens, path, accepted = (torch.full((n,), -7, **I) for n in (T, T, B))
    lora.lora_verify_tree(v, p, torch.tensor(draft, **I), torch.tensor(parent, **I), torch.tensor(row0, **I),
                          torch.tensor(u, dtype=torch.float32, device="cuda"), B, T, tokens, path, accepted)
    got = tokens.tolist(), path.tolist(), accepted.tolist()
    if verifier is None:
        lora.lora_verifier_destroy(v)
    return got


def same(p, draft, parent, row0, u, **kw):
    got = call(p, draft, parent, row0, u, **kw)
    want = ref.verify_tree(p.double().cpu().numpy(), draft, parent, row0, np.asarray(u, dtype=np.float32).astype(np.float64))
    assert got[2] == want[2]
    assert got[1] == want[1]
    assert got[0] == want[0]
    return got


def batch(kinds, sizes, V, dtype, seed, sharp=6.0):
    """Trees whose nodes hold their parent's likeliest next tokens."""
    g, rng = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
    row0 = [0] + [int(x) for x in np.cumsum(sizes)]
    z = torch.randn((row0[-1], V), generator=g) * sharp
    best = torch.topk(z + 0.3 * torch.randn(z.shape, generator=g), min(V, 8), 1).indices
    parent, draft = [], []
    for k, n, r0 in zip(kinds, sizes, row0):
        tree, seen = parents(k, n, rng), {}
        for j, up in enumerate(tree):
            seen[up] = seen.get(up, -1) + 1
            draft.append(int(best[r0 + max(up, 0), seen[up] % best.shape[1]]))
        parent += tree
    p = torch.softmax(z, -1).to(DT[dtype])
    return p.cuda(), draft, parent, row0, torch.rand((row0[-1],), generator=g).tolist()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 7, 300, 2049, 32000, 32769, 140001])
def test_ragged_batches(dtype, V):
    kept = []
    for seed in range(3):
        rng = np.random.default_rng(seed + V)
        sizes = [int(x) for x in rng.integers(1, 30 if V < 10000 else 9, 9)]
        kinds = [KINDS[int(x)] for x in rng.integers(0, len(KINDS), 9)]
        kept += same(*batch(kinds, sizes, V, dtype, seed * 100 + V))[2]
    assert max(kept) > 0


@pytest.mark.parametrize("n", [1, 64, 1024, 1025, 2500])
@pytest.mark.parametrize("kind", ["chain", "near", "star", "forest"])
def test_large_trees(kind, n):
    """More nodes than threads; a chain that is kept as a whole."""
    p, draft, parent, row0, u = batch([kind, kind], [n, 3], 40, "f32", n, sharp=2.0)
    same(p, draft, parent, row0, u)
    if kind == "chain":
        draft[1:n] = ref.verify_tree(p.double().cpu().numpy(), [0] * (n + 3), [-1] * (n + 3), list(range(n + 4)),
                                     np.asarray(u, dtype=np.float32).astype(np.float64))[0][:n - 1]
        assert same(p, draft, parent, row0, u)[2][0] == n - 1


def test_many_sequences():
    sizes = [1 + i % 7 for i in range(700)]
    got = same(*batch(["near"] * 700, sizes, 500, "bf16", 2))
    assert 0 < sum(got[2]) < sum(sizes)


def test_rows_without_weight():
    """No answer where the walk comes by such a row; others do not count."""
    p, draft, parent, row0, u = batch(["star"] * 6, [4] * 6, 50, "f32", 3)
    p[row0[0]] = 0.0                    # the root's
    p[row0[1]] = -1.0
    p[row0[2], 7] = float("nan")        # counts as nothing
    p[row0[3], 9] = float("inf")
    for r in range(1, 4):               # sure to come to node 2, whose row has nothing
        p[row0[4] + r] = 0.0 if r == 2 else 1.0
        p[row0[5] + r] = 0.0 if r != 2 else 1.0
    for b in (4, 5):
        p[row0[b]] = 0.0
        p[row0[b], draft[row0[b] + 2]] = 1.0
    got = same(p, draft, parent, row0, u)
    assert got[2][:2] == [-1, -1] and got[2][2] >= 0 and got[2][3] == -1 and got[2][4] == -1 and got[2][5] == 1


def test_siblings_and_odd_parents():
    """The first of two siblings that hold a token; nodes that point at
    themselves, past the end or ahead are never come to."""
    V = 16
    p = torch.zeros((10, V), device="cuda")
    p[:, 3] = 1.0
    draft = [3] * 10
    parent = [0, 1, 5, 0, 0, 4, 99, -1, 3, 8]   # 0 -> 3 -> 8 -> 9
    assert call(p, draft, parent, [0, 10], [0.5] * 10) == ([3] * 4 + [-1] * 6, [0, 3, 8, 9] + [-1] * 6, [3])
    same(p, draft, parent, [0, 10], [0.5] * 10)


@pytest.mark.parametrize("row0", [[0, 0, 4], [0, 3, 2], [-1, 2, 4], [0, 2, 5], [1, 1, 4], [3, 2, 1], [0, 4, 4],
                                  [0, 1 << 30, 4], [0, 2, -(1 << 31)]])
def test_bounds_that_are_none(row0):
    """Nothing is read or written outside; a sequence with good bounds has its
    answer where no other's reach into it."""
    p, draft, parent, _, u = batch(["chain"] * 2, [2, 2], 64, "f32", 1)
    v = lora.lora_verifier_create(2)
    tokens, path, accepted = call(p, draft, parent, row0, u, verifier=v)
    good = [b <= row0[b] < row0[b + 1] <= 4 - (1 - b) for b in range(2)]
    assert [a >= 0 for a in accepted] == good
    covered = {r for b in range(2) if good[b] for r in range(row0[b], row0[b + 1])}
    assert all((tokens[r] == -7) == (r not in covered) for r in range(4))
    assert call(p, draft, parent, [0, 2, 4], u, verifier=v) == call(p, draft, parent, [0, 2, 4], u)  # the next call is whole
    lora.lora_verifier_destroy(v)


def test_bounds_that_overlap():
    """Sequences that share rows write over each other's answers, which are then
    none in particular; ones whose own bounds are none have -1, ones that share
    nothing their answer, and the next call is whole."""
    p, draft, parent, row0, u = batch(["near"] * 4, [3, 3, 3, 3], 64, "f32", 1)
    v = lora.lora_verifier_create(4)
    for bad in ([0, 5, 3, 8, 12], [0, 8, 1, 10, 12], [0, 9, 2, 11, 4]):
        accepted = call(p, draft, parent, bad, u, verifier=v)[2]
        fits = [b <= bad[b] < bad[b + 1] <= 12 - (3 - b) for b in range(4)]
        assert all(-1 <= a < 12 for a in accepted) and all(a == -1 for a, f in zip(accepted, fits) if not f)
        if fits[3]:  # nobody else's rows reach into the last one's
            assert accepted[3] == ref.verify_tree(p.double().cpu().numpy()[bad[3]:], draft[bad[3]:], parent[bad[3]:],
                                                  [0, 12 - bad[3]], [np.float64(np.float32(x)) for x in u[bad[3]:]])[2][0]
        assert call(p, draft, parent, row0, u, verifier=v) == same(p, draft, parent, row0, u)
    lora.lora_verifier_destroy(v)


@pytest.mark.parametrize("bad", [[0, 1000, 2, 1002, 1010], [0, 700, 1, 2, 1010], [0, 1001, 3, 1003, 1010]])
def test_large_trees_that_overlap(bad):
    """The same of trees past 512 nodes, whose lists lie in memory that
    sequences with the same rows share: the walks end inside their trees."""
    p, draft, parent, row0, u = batch(["near"] * 4, [400, 400, 200, 10], 16, "f32", 3)
    v = lora.lora_verifier_create(4)
    tokens, path, accepted = call(p, draft, parent, bad, u, verifier=v)
    fits = [b <= bad[b] < bad[b + 1] <= 1010 - (3 - b) for b in range(4)]
    assert all((a == -1) if not f else (-1 <= a < bad[b + 1] - bad[b]) for b, (a, f) in enumerate(zip(accepted, fits)))
    assert all(-1 <= t < 16 or t == -7 for t in tokens) and all(-1 <= n < 1010 or n == -7 for n in path)
    assert call(p, draft, parent, row0, u, verifier=v) == same(p, draft, parent, row0, u)  # the next call is whole
    lora.lora_verifier_destroy(v)


@pytest.mark.parametrize("unit", [8, 512, 32768])
def test_a_place_without_weight_is_not_drawn(unit):
    """As for lora_verify: weights whose order of adding decides about 1/2."""
    t, V = 2.0 ** -54, 32 * unit
    p = torch.zeros((2, V))
    p[:, [0, unit]], p[:, [2 * unit, 10 * unit]] = t, 0.5
    tokens, path, accepted = call(p.cuda(), [0, 5 * unit], [-1, 0], [0, 2], [0.5, 0.5])
    assert accepted == [0] and tokens[0] in (2 * unit, 10 * unit) and tokens[1] == -1 and path == [0, -1]


def test_the_tokens_are_the_target_s():
    """Over many draws the first token has the root's distribution and the
    second its parent's, whatever the tree holds (5 standard deviations of each
    share)."""
    n, V = 40000, 5
    root, below = torch.tensor([0.4, 0.1, 0.25, 0.05, 0.2]), torch.tensor([0.1, 0.2, 0.3, 0.15, 0.25])
    p = torch.stack([root, below, below]).repeat(n, 1).cuda()
    u = torch.rand(3 * n, generator=torch.Generator().manual_seed(4)).tolist()
    tokens, path, accepted = call(p, [0, 2, 0] * n, [-1, 0, 0] * n, list(range(0, 3 * n + 1, 3)), u)
    first, second = torch.tensor(tokens[::3]), torch.tensor(tokens[1::3])
    kept = torch.tensor(accepted) == 1
    assert torch.equal(kept, (first == 0) | (first == 2))
    for got, want in ((first, root), (second[kept], below)):
        share = torch.bincount(got.long(), minlength=V) / len(got)
        assert ((share - want).abs() <= 5 * (want * (1 - want) / len(got)).sqrt()).all()


def test_refusals():
    lib = lora.raw_lib()
    p, i, u = torch.ones((4, 8), device="cuda"), torch.zeros(8, **I), torch.zeros(4, device="cuda")
    v = lora.lora_verifier_create(2)
    row0, out = torch.tensor([0, 2, 4], **I), torch.zeros((3, 8), **I)
    good = dict(v=v, p=p.data_ptr(), dtype=0, vocab=8, draft=i.data_ptr(), parent=i.data_ptr(), row0=row0.data_ptr(),
                u=u.data_ptr(), seqs=2, rows=4, tokens=out[0].data_ptr(), path=out[1].data_ptr(), acc=out[2].data_ptr(),
                stream=None)

    def check(**change):
        return lib.lora_verify_tree(*{**good, **change}.values())
    assert check() == lora.LORA_OK
    assert check(seqs=0, row0=None) == lora.LORA_OK
    assert check(seqs=3) == lora.LORA_ETOKENS
    for change in (dict(v=None), dict(seqs=-1), dict(rows=-1), dict(vocab=0), dict(vocab=(1 << 21) + 1), dict(dtype=5),
                   dict(p=None), dict(draft=None), dict(parent=None), dict(row0=None), dict(u=None), dict(tokens=None),
                   dict(path=None), dict(acc=None), dict(p=good["p"] + 2), dict(parent=good["parent"] + 1),
                   dict(path=good["path"] + 2)):
        assert check(**change) == lora.LORA_EINVAL, change
    with pytest.raises(ValueError, match="parent"):
        lora.lora_verify_tree(v, p, i, i[:3], row0, u, 2, 4, out[0], out[1], out[2])
    # No rows: every sequence's bounds are none.
    assert check(rows=0, p=None, draft=None, parent=None, u=None, tokens=None, path=None) == lora.LORA_OK
    assert out[2, :2].tolist() == [-1, -1]
    lora.lora_verifier_destroy(v)


@pytest.mark.parametrize("V,sizes", [(500, [9, 1, 30]), (70000, [5, 2])])
def test_captured_and_replayed(V, sizes):
    stream = torch.cuda.Stream()
    v = lora.lora_verifier_create(len(sizes))
    p, draft, parent, row0, u = batch(["near"] * len(sizes), sizes, V, "f32", 1)
    T, B = row0[-1], len(sizes)
    dev = [torch.tensor(x, **I) for x in (draft, parent, row0)] + [torch.tensor(u, device="cuda")]
    out = [torch.full((n,), -7, **I) for n in (T, T, B)]
    torch.cuda.synchronize()
    gc.collect()
    gc.disable()
    try:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            lora.lora_verify_tree(v, p, *dev, B, T, *out, stream=torch.cuda.current_stream())
    finally:
        gc.enable()
    for i in range(4):
        new = batch([KINDS[i]] * B, sizes, V, "f32", 20 + i)
        p.copy_(new[0])
        for x, y in zip(dev, new[1:]):
            x.copy_(torch.tensor(y, dtype=x.dtype))
        graph.replay()
        torch.cuda.synchronize()
        assert tuple(x.tolist() for x in out) == same(*new)
    lora.lora_verifier_destroy(v)


def test_two_at_once():
    """Two verifiers on two streams, several calls each way in flight."""
    some = [batch(["near"] * 3, [9, 1, 30], 70000, "bf16", 11), batch(["binary"] * 2, [16, 5], 140001, "f32", 12)]
    streams = [torch.cuda.Stream() for _ in some]
    vs = [lora.lora_verifier_create(3) for _ in some]
    on = [(torch.tensor(d, **I), torch.tensor(up, **I), torch.tensor(r, **I), torch.tensor(u, dtype=torch.float32, device="cuda"))
          for _, d, up, r, u in some]
    out = [[tuple(torch.full((n,), -7, **I) for n in (r[-1], r[-1], len(r) - 1)) for _ in range(8)] for _, _, _, r, _ in some]
    torch.cuda.synchronize()
    for i in range(8):
        for k, (p, _, _, r, _) in enumerate(some):
            lora.lora_verify_tree(vs[k], p, *on[k], len(r) - 1, r[-1], *out[k][i], stream=streams[k])
    torch.cuda.synchronize()
    for k, (p, d, up, r, u) in enumerate(some):
        want = same(p, d, up, r, u)
        assert all(tuple(x.tolist() for x in o) == want for o in out[k])
        lora.lora_verifier_destroy(vs[k])
