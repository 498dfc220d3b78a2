"""Log probabilities, entropies and alternatives against the 64-bit form: types,
vocabularies from one entry to several parts, rows at any stride and alignment,
many and few rows, equal logits, masks of -inf and of the type's lowest value,
rows that are no distribution, scales, results not asked for, graphs."""
import gc

import numpy as np
import pytest
import torch

import tree_reference as ref
from rank_adapter_gemm_token_amd import lora

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


class Scorer:
    def __init__(self, rows):
        self.h = lora.lora_scorer_create(rows)

    def __enter__(self):
        return self.h

    def __exit__(self, *a):
        torch.cuda.synchronize()
        lora.lora_scorer_destroy(self.h)


def buffers(n, top):
    return (torch.full((n,), 7.0, device="cuda"), torch.full((n,), 7.0, device="cuda"),
            torch.full((n, top), 7, dtype=torch.int32, device="cuda"), torch.full((n, top), 7.0, device="cuda"))


def check(z, tokens, scale, top, got, rows=None):
    """c (z - M) is rounded three times (c itself, the difference, and the part
    of M c that fp32 does not hold): 3 * 2^-24 of its own size, or of the 1 that
    the last may be.  A term 2^y is off by ln 2 of that and by the exponential's
    2^-22; a sum of terms of one sign by 2^-24 for each of the additions on a
    term's way, 120 at most (32 of a batch, those of batches, lanes, waves and
    workgroups).  In l that is relative, in the logarithm
    absolute.  s is a sum of such terms times y, whose sizes add up to at most
    |log p| times p: the entropy's own terms; what e^y has lost is multiplied by
    y once more.  The result is rounded once."""
    lp, h, ids, tlp = (x.cpu().double().numpy() for x in got)
    zz, e = z.double().cpu().numpy(), 2.0 ** -24
    for r in range(len(zz)) if rows is None else rows:
        t = -1 if tokens is None else int(tokens[r])
        want = ref.logprobs(zz[r], t, scale, top)
        if np.isnan(want[1]):
            assert np.isnan(lp[r]) and np.isnan(h[r]) and (ids[r] == -1).all() and np.isnan(tlp[r]).all(), r
            continue
        assert ids[r].tolist() == want[2], (r, ids[r], want[2])
        y = scale * (zz[r].max() - zz[r])
        p = np.exp(-y)
        p, y = p / p.sum(), np.where(np.isfinite(y), y, 0.0)
        ey = 3 * e * y + 4 * e                         # of one y (absolute)
        el = (p * ey).sum() + 120 * e                  # of l (relative), of log l (absolute)
        for have, log_p in [(lp[r], want[0])] + list(zip(tlp[r], want[3])):
            if np.isnan(log_p) or np.isinf(log_p):
                assert have == log_p or (np.isnan(have) and np.isnan(log_p)), (r, have, log_p)
            else:
                assert abs(have - log_p) <= el + 4 * e * abs(log_p) + e, (r, have, log_p, el)
        assert abs(h[r] - want[1]) <= el + (p * (ey + 124 * e) * (1 + y)).sum() + 4 * e * want[1] + e, (r, h[r], want[1])


def logits(n, vocab, dtype, seed, pad=0, at=0, spread=4.0):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn((n, vocab), generator=g) * spread * torch.rand((n, 1), generator=g)
    wide = torch.full((n * (vocab + pad) + at,), float("nan"), dtype=DT[dtype], device="cuda")
    out = wide[at:].view(n, vocab + pad)[:, :vocab]
    out.copy_(z)
    return out


def tokens_for(n, vocab, seed):
    t = np.random.default_rng(seed).integers(0, vocab, n)
    if n > 2:
        t[1], t[2] = -1, vocab
    return torch.tensor(t, dtype=torch.int32)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 9, 31, 33, 300, 511, 2048, 8191, 8192, 8193, 32000, 32767, 32769, 50257])
@pytest.mark.parametrize("n,pad,at", [(1, 0, 0), (5, 3, 1), (9, 64, 8)])
def test_rows(dtype, vocab, n, pad, at):
    z, t = logits(n, vocab, dtype, vocab + n, pad, at), tokens_for(n, vocab, n)
    with Scorer(16) as s:
        for top in (0, 1, 5, 32):
            if top > vocab:
                continue
            got = buffers(n, top)
            lora.lora_logprobs(s, z, t.cuda(), 1.0, *got)
            check(z, t, 1.0, top, got)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,vocab", [(3, 131072), (2, 400001), (1, 1 << 21), (100, 131072), (257, 70000), (300, 9000)])
def test_large_vocabularies(dtype, n, vocab):
    """Parts of a row in several workgroups, and one after the other in one."""
    z, t = logits(n, vocab, dtype, n), tokens_for(n, vocab, n)
    rows = sorted(set(range(0, n, max(1, n // 5))) | {n - 1})
    with Scorer(n) as s:
        for top in (3, 32):
            got = buffers(n, top)
            lora.lora_logprobs(s, z, t.cuda(), 0.7, *got)
            check(z, t, 0.7, top, got, rows)
            again = buffers(n, top)
            lora.lora_logprobs(s, z, t.cuda(), 0.7, *again)
            for x, y in zip(got, again):
                assert torch.equal(x.nan_to_num(0.5), y.nan_to_num(0.5))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("vocab", [40, 3001, 40000, 131072])
def test_equal_logits(dtype, vocab):
    """Ties go to the lowest index: all equal, few levels, runs of the largest,
    zeros of both signs, ascending and descending rows."""
    z = torch.zeros((8, vocab), dtype=DT[dtype], device="cuda")
    g = torch.Generator().manual_seed(1)
    z[1] = torch.randint(0, 4, (vocab,), generator=g).to(z)
    z[2, vocab // 2:] = 3.0
    z[3, ::2] = -0.0
    z[4] = torch.linspace(-9, 9, vocab).to(z)
    z[5] = torch.linspace(9, -9, vocab).to(z)
    z[6] = -2.5
    z[7] = torch.randn(vocab, generator=g).mul(2).round().to(z)
    t = tokens_for(8, vocab, 3)
    with Scorer(8) as s:
        for top in (1, 17, 32):
            got = buffers(8, top)
            lora.lora_logprobs(s, z, t.cuda(), 1.0, *got)
            check(z, t, 1.0, top, got)


@pytest.mark.parametrize("n,vocab,threads", [(2, 131072, 1024), (600, 20000, 256)])
def test_many_above_the_first_bound(n, vocab, threads):
    """Where only 31 of the 64 groups of lanes hold anything high, and ascending,
    the 32nd alternative's first bound leaves nearly half of the row, and every
    next one the rest but for a few hundred."""
    i = torch.arange(vocab, device="cuda")
    group = (i // 512 % (threads // 64) * 64 + i // 8 % 64) // (threads // 64)
    z = torch.where(group < 31, i.float() / vocab, -10.0 - i.float() / vocab).expand(n, vocab).contiguous()
    t = tokens_for(n, vocab, n)
    with Scorer(n) as s:
        got = buffers(n, 32)
        lora.lora_logprobs(s, z, t.cuda(), 1.0, *got)
        check(z[:3], t[:3], 1.0, 32, [x[:3] for x in got])
        assert all((x[3:] == x[3:4]).all() for x in got[1:])  # entropy and alternatives: rows are alike


def test_two_at_once():
    """Two scorers on two streams, several calls each way in flight."""
    rows = [logits(3, 131072, "f32", 5), logits(4, 140001, "bf16", 6)]
    t = [tokens_for(len(z), z.shape[1], 9) for z in rows]
    on = [x.cuda() for x in t]
    got = [[buffers(len(z), 7) for _ in range(8)] for z in rows]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in rows]
    with Scorer(4) as a, Scorer(4) as b:
        for i in range(8):
            for k, s in enumerate((a, b)):
                lora.lora_logprobs(s, rows[k], on[k], 1.0, *got[k][i], stream=streams[k])
        torch.cuda.synchronize()
    for k, z in enumerate(rows):
        check(z, t[k], 1.0, 7, got[k][0])
        for other in got[k][1:]:
            assert all(torch.equal(x.nan_to_num(3.0), y.nan_to_num(3.0)) for x, y in zip(got[k][0], other))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("vocab", [64, 5000, 66000])
def test_masks(dtype, vocab):
    """-inf nearly everywhere, everywhere but once, in whole parts; the type's
    lowest value as a mask, nearly everywhere and everywhere."""
    z = logits(9, vocab, dtype, 2).contiguous()
    low = torch.finfo(DT[dtype]).min
    z[0, 7:] = float("-inf")
    z[1] = float("-inf")
    z[1, vocab - 1] = 3.0
    z[2, :vocab // 2] = float("-inf")
    z[3, ::3] = float("-inf")
    z[4, 10:] = low
    z[5] = low
    z[6, :vocab - 3] = low
    z[7, 1:] = float("-inf")
    t = torch.tensor([3, vocab - 1, 0, 3, 2, 4, vocab - 1, 0, 5], dtype=torch.int32)
    with Scorer(9) as s:
        for top in (1, 20):
            got = buffers(9, top)
            lora.lora_logprobs(s, z, t.cuda(), 1.0, *got)
            check(z, t, 1.0, top, got)
            assert got[0][1] == 0 and got[1][1] == 0 and got[0][7] == 0


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("vocab", [64, 5000, 66000])
def test_rows_that_are_no_distribution(dtype, vocab):
    z = logits(7, vocab, dtype, 2).contiguous()
    z[1, 3] = float("nan")
    z[2, vocab - 1] = float("inf")
    z[3] = float("-inf")
    z[4] = float("nan")
    z[5, 1], z[5, 2] = float("inf"), float("-inf")
    t = torch.zeros(7, dtype=torch.int32)
    with Scorer(7) as s:
        got = buffers(7, 4)
        lora.lora_logprobs(s, z, t.cuda(), 1.0, *got)
        check(z, t, 1.0, 4, got)
        assert got[0].isnan().tolist() == [False, True, True, True, True, True, False]


@pytest.mark.parametrize("scale", [2.0 ** -64, 0.01, 1.0, 3.7, 1000.0, 2.0 ** 64])
@pytest.mark.parametrize("shift", [0.0, 300.0, -40000.0])
def test_scales(scale, shift):
    z = (logits(4, 9000, "f32", 3) + shift).contiguous()
    t = tokens_for(4, 9000, 1)
    with Scorer(4) as s:
        got = buffers(4, 6)
        lora.lora_logprobs(s, z, t.cuda(), scale, *got)
        check(z, t, scale, 6, got)


def test_results_not_asked_for():
    z, t = logits(5, 3000, "bf16", 1), tokens_for(5, 3000, 1).cuda()
    with Scorer(5) as s:
        all_ = buffers(5, 3)
        lora.lora_logprobs(s, z, t, 1.0, *all_)
        lp, h, ids, tlp = buffers(5, 3)
        lora.lora_logprobs(s, z, t, 1.0, logprob=lp)
        lora.lora_logprobs(s, z, None, 1.0, entropy=h)
        lora.lora_logprobs(s, z, None, 1.0, top_ids=ids, top_logprobs=tlp)
        for x, y in zip(all_, (lp, h, ids, tlp)):
            assert torch.equal(x.nan_to_num(0.5), y.nan_to_num(0.5))
        lora.lora_logprobs(s, z, None, 1.0, logprob=lp)
        assert lp.isnan().all()
        lora.lora_logprobs(s, z[:0], None, 1.0)


def test_refusals():
    lib = lora.raw_lib()
    z, lp, h, ids, tlp = torch.zeros((4, 64), device="cuda"), *buffers(4, 3)
    t = torch.zeros(4, dtype=torch.int32, device="cuda")
    with Scorer(4) as s:
        good = dict(s=s, z=z.data_ptr(), stride=64, dtype=0, vocab=64, t=t.data_ptr(), scale=1.0, top=3, n=4,
                    lp=lp.data_ptr(), h=h.data_ptr(), ids=ids.data_ptr(), tlp=tlp.data_ptr(), stream=None)

        def call(**change):
            return lib.lora_logprobs(*{**good, **change}.values())
        assert call() == lora.LORA_OK
        assert call(n=0, z=None) == lora.LORA_OK
        assert call(top=0, ids=None, tlp=None) == lora.LORA_OK
        assert call(n=5) == lora.LORA_ETOKENS
        for change in (dict(n=-1), dict(z=None), dict(z=good["z"] + 2), dict(stride=63), dict(dtype=3), dict(vocab=0),
                       dict(vocab=(1 << 21) + 1, stride=1 << 22), dict(scale=0.0), dict(scale=-1.0),
                       dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=1e-20), dict(top=-1), dict(top=33),
                       dict(vocab=2, top=3), dict(ids=None), dict(tlp=None), dict(t=good["t"] + 2), dict(lp=good["lp"] + 1)):
            assert call(**change) == lora.LORA_EINVAL, change
        for bad in (dict(logits=z.T), dict(top_ids=ids), dict(top_ids=ids[:2], top_logprobs=tlp),
                    dict(tokens=t[:3]), dict(logprob=lp.double())):
            with pytest.raises(ValueError):
                lora.lora_logprobs(s, **{**dict(logits=z, tokens=t, logprob=lp), **bad})


@pytest.mark.parametrize("n,vocab", [(3, 131072), (40, 5000)])
def test_captured_and_replayed(n, vocab):
    stream = torch.cuda.Stream()
    z, t = logits(n, vocab, "bf16", 1).contiguous(), tokens_for(n, vocab, 1).cuda()
    with Scorer(n) as s:
        got = buffers(n, 8)
        torch.cuda.synchronize()
        gc.collect()
        gc.disable()
        try:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                lora.lora_logprobs(s, z, t, 1.0, *got, stream=torch.cuda.current_stream())
        finally:
            gc.enable()
        for i in range(4):
            z.copy_(logits(n, vocab, "bf16", 10 + i))
            graph.replay()
            torch.cuda.synchronize()
            eager = buffers(n, 8)
            lora.lora_logprobs(s, z, t, 1.0, *eager)
            for x, y in zip(got, eager):
                assert torch.equal(x.nan_to_num(0.5), y.nan_to_num(0.5))
            check(z, t.cpu(), 1.0, 8, got, [0, n - 1])
