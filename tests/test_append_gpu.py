"""Appended keys: turned by their positions and held as lora_kv_write holds the
turned key, bit for bit; queries turned beside them.  Over types, head layouts,
parts of a head, both pairings, one and several axes, runs of slots that fill
blocks and that do not, strides, padding, bad slots and positions, rows that
are not finite, captured calls."""
import gc

import numpy as np
import pytest
import torch

import kv_reference as ref
import tree_reference as tree
from rank_adapter_gemm_token_amd import lora
from test_kv_gpu import DT, Cache, rows, slot_list

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Rope:
    def __init__(self, n_positions, rot, axes=1, pairs=False, scale=1.0, base=10000.0):
        n = rot // 2
        self.n_positions, self.axes, self.pairs, self.scale = n_positions, axes, pairs, scale
        self.freq = base ** (-np.arange(n) / n)
        self.axis = [(i * 7) % axes for i in range(n)] if axes % 2 else [i * axes // n for i in range(n)]
        self.h = lora.lora_rope_create(n_positions, torch.from_numpy(self.freq), axis=torch.tensor(self.axis, dtype=torch.int32),
                                       n_axes=axes, pairs=pairs, scale=scale)

    def turned(self, x, positions):
        return tree.turned(x, np.asarray(positions).reshape(self.axes, -1), self.freq, self.axis, self.pairs, self.scale)

    def __enter__(self):
        return self

    def __exit__(self, *a):
        lora.lora_rope_destroy(self.h)


def append(c, rope, k, v, slots, positions, q=None, q_out=None, stream=None):
    """The call, and what the cache should hold after it."""
    T = len(slots)
    positions = np.asarray(positions).reshape(rope.axes, T)
    lora.lora_kv_append(c.h, rope.h, k, v, i32(slots), i32(positions), T, q=q, q_out=q_out, stream=stream)
    at = [i for i, x in enumerate(slots) if 0 <= x < c.n]
    bad = ((positions < 0) | (positions >= rope.n_positions)).any(0)
    kk, _ = rope.turned(k.double().cpu().numpy(), np.where(bad, 0, positions))
    kk[bad] = np.nan
    kk, vv = ref.held_pair(kk[at], v.double().cpu().numpy()[at])
    c.k[[slots[i] for i in at]] = kk
    c.v[[slots[i] for i in at]] = vv


def check_queries(rope, q, q_out, positions):
    """fp32: cosine and sine are off by half a step (2^-24), so is the product
    that the other is added to and the sum; then one rounding to 16 bits."""
    want, mass = rope.turned(q.double().cpu().numpy(), positions)
    half, tiny = torch.finfo(q.dtype).eps / 2, torch.finfo(q.dtype).tiny
    tol = half * np.abs(want) + 2 * half * tiny + 4 * 2.0 ** -24 * mass
    turns = np.zeros(q.shape[2], dtype=bool)
    turns[:2 * len(rope.freq)] = True
    tol[:, :, ~turns] = 0.0
    got = q_out.double().cpu().numpy()
    assert (np.abs(got - want) <= tol).all(), np.max(np.abs(got - want) - tol)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("kv_heads,heads,dim,page,rot,axes,pairs", [
    (1, 1, 128, 16, 128, 1, False), (3, 6, 64, 64, 64, 1, False), (8, 9, 128, 32, 128, 3, False),
    (2, 14, 64, 16, 16, 2, False), (1, 5, 128, 64, 48, 1, False), (2, 2, 128, 16, 96, 4, False),
    (1, 4, 128, 16, 128, 1, True), (3, 3, 64, 32, 48, 3, True), (2, 7, 128, 16, 64, 2, True)])
@pytest.mark.parametrize("kind", ["run", "off", "scattered", "pages", "padded", "holes", "halves"])
@pytest.mark.parametrize("T", [1, 17, 50])
def test_appended_rows_read_back(dtype, kv_heads, heads, dim, page, rot, axes, pairs, kind, T):
    rng = np.random.default_rng(T * 7 + heads)
    n_pages = -(-(2 * T + 60) // page) + 2
    with Cache(n_pages, page, kv_heads, dim, dtype) as c, Rope(5000, rot, axes, pairs) as rope:
        slots = slot_list(kind, T, c.n, page, rng)
        # Every slot holds something first: an append must leave the others alone.
        every = list(range(c.n))
        c.write(rows(c.n, kv_heads, dim, dtype, 1), rows(c.n, kv_heads, dim, dtype, 2), every)
        qkv = torch.cat([rows(T, n, dim, dtype, s, 2.0) for n, s in ((heads, 3), (kv_heads, 4), (kv_heads, 5))], 1)
        q, k, v = qkv.split([heads, kv_heads, kv_heads], 1)
        positions = rng.integers(0, 5000, (axes, T))
        q_out = torch.full((T + 1, heads, dim), 7.0, dtype=DT[dtype], device="cuda")
        append(c, rope, k, v, slots, positions, q, q_out)
        c.check(every)
        check_queries(rope, q, q_out[:T], positions)
        assert (q_out[T] == 7.0).all()
        # In place, within the projection's output; keys and values stay.
        before = qkv.clone()
        append(c, rope, k, v, slots, positions, q, q)
        assert torch.equal(q, q_out[:T]) and torch.equal(before[:, heads:], qkv[:, heads:])
        append(c, rope, k, v, slots, positions)
        c.check(every)
        assert lora.lora_kv_poll_errors(c.h) == 0


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_many_tokens_of_several_heads_a_workgroup(dtype, pairs):
    T, heads, kv_heads = 4200, 33, 9
    rng = np.random.default_rng(5)
    with Cache(300, 16, kv_heads, 64, dtype) as c, Rope(100, 64, 1, pairs) as rope:
        slots = list(range(20, 20 + T))
        slots[7::50] = [-1] * len(slots[7::50])
        k, v, q = (rows(T, n, 64, dtype, s) for n, s in ((kv_heads, 1), (kv_heads, 2), (heads, 3)))
        positions = rng.integers(0, 100, (1, T))
        q_out = torch.empty_like(q)
        append(c, rope, k, v, slots, positions, q, q_out)
        c.check(list(range(c.n)))
        check_queries(rope, q, q_out, positions)


@pytest.mark.parametrize("pairs", [False, True])
def test_far_positions(pairs):
    """Angles of a million turns, in a table of which one row is used."""
    n = 1 << 20
    with Cache(2, 16, 1, 64, "bf16") as c, Rope(n, 64, 1, pairs) as rope:
        k, v, q = (rows(4, h, 64, "bf16", s) for h, s in ((1, 1), (1, 2), (3, 3)))
        q_out = torch.empty_like(q)
        positions = [n - 1, n - 2, 0, n // 2 + 1]
        append(c, rope, k, v, [3, 4, 5, 30], positions, q, q_out)
        c.check(list(range(c.n)))
        check_queries(rope, q, q_out, positions)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_position_zero_is_a_write(dtype):
    T = 40
    k, v = rows(T, 2, 128, dtype, 1, 3.0), rows(T, 2, 128, dtype, 2, 3.0)
    with Cache(4, 16, 2, 128, dtype) as a, Cache(4, 16, 2, 128, dtype) as b, Rope(8, 128) as rope:
        a.write(k, v, list(range(T)))
        append(b, rope, k, v, list(range(T)), [0] * T, k, torch.empty_like(k))
        for x, y in zip(a.read(list(range(64))), b.read(list(range(64)))):
            assert torch.equal(x, y)


def test_scaled_angles():
    with Cache(2, 16, 2, 64, "f16") as c, Rope(64, 32, 1, False, scale=1.375) as rope:
        k, v, q = (rows(9, h, 64, "f16", s) for h, s in ((2, 1), (2, 2), (4, 3)))
        q_out = torch.empty_like(q)
        append(c, rope, k, v, list(range(9)), list(range(50, 59)), q, q_out)
        c.check(list(range(c.n)))
        check_queries(rope, q, q_out, list(range(50, 59)))


@pytest.mark.parametrize("slot0", [0, 3])
def test_bad_positions_and_slots(slot0):
    """Slots 16 in order from a block's start, and not: both ways of writing."""
    T, axes = 20, 2
    with Cache(3, 16, 2, 64, "bf16") as c, Rope(100, 32, axes) as rope:
        every = list(range(c.n))
        c.write(rows(c.n, 2, 64, "bf16", 1), rows(c.n, 2, 64, "bf16", 2), every)
        slots = list(range(slot0, slot0 + T))
        positions = np.stack([np.arange(T), 99 - np.arange(T)])
        positions[0, 2], positions[1, 5], positions[0, 9], positions[1, 9] = -1, 100, 1 << 30, -(1 << 31)
        slots[7], slots[11] = 48, -5          # outside the cache
        slots[13], positions[0, 13] = -1, -1  # padding: not counted
        slots[14] = -1                        # padding with a position: its queries turn
        k, v, q = (rows(T, h, 64, "bf16", s) for h, s in ((2, 3), (2, 4), (3, 5)))
        q_out = torch.empty_like(q)
        append(c, rope, k, v, slots, positions, q, q_out)
        c.check(every)
        bad = [2, 5, 9, 13]
        assert q_out[bad].isnan().all()
        good = [i for i in range(T) if i not in bad]
        check_queries(rope, q[good], q_out[good], positions[:, good])
        assert lora.lora_kv_poll_errors(c.h) == 5
        assert lora.lora_kv_poll_errors(c.h) == 0


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_extreme_rows(dtype, pairs):
    """Rows that are not finite are poisoned, and only they; bf16's largest
    values turn into infinity where the sum passes fp32; zeros and the
    smallest values are held as lora_kv_write would hold them."""
    T, big = 24, torch.finfo(DT[dtype]).max
    with Cache(3, 16, 1, 128, dtype) as c, Rope(64, 64, 1, pairs) as rope:
        k, v = rows(T, 1, 128, dtype, 1), rows(T, 1, 128, dtype, 2)
        k[1, 0, 5], k[2, 0, 100], v[4, 0, 3] = float("nan"), float("inf"), float("-inf")
        k[6], v[6], k[8] = 0.0, 0.0, -0.0
        k[9], k[10] = torch.finfo(DT[dtype]).tiny, torch.finfo(DT[dtype]).smallest_normal / 8
        k[11, 0, ::2] = big          # at 45 degrees a pair of the largest grows by sqrt(2)
        k[12] = big
        k[13, 0, 7] = big
        append(c, rope, k, v, list(range(T)), [i * 2 for i in range(T)])
        y, _ = rope.turned(k.double().cpu().numpy(), [i * 2 for i in range(T)])
        with np.errstate(invalid="ignore"):
            over = np.abs(y[:, 0]).max(-1) >= 2.0 ** 128 - 2.0 ** 103  # rounds to infinity in fp32
        c.k[:T][over], c.v[:T][over] = np.nan, np.nan
        assert np.isnan(c.k[[1, 2, 4]]).all() and np.isnan(c.v[[1, 2, 4]]).all() and not np.isnan(c.k[[0, 3, 5]]).any()
        c.check(list(range(c.n)))


def test_infinite_queries_stay_in_their_pair():
    with Cache(1, 16, 1, 64, "f16") as c, Rope(64, 32) as rope:
        k, q = rows(2, 1, 64, "f16", 1), rows(2, 2, 64, "f16", 2)
        q[0, 1, 3], q[1, 0, 40] = float("inf"), float("-inf")
        out = torch.empty_like(q)
        append(c, rope, k, k, [0, 1], [5, 6], q, out)
        odd = ~out.isfinite()
        want = torch.zeros_like(odd)
        want[0, 1, 3] = want[0, 1, 19] = want[1, 0, 40] = True
        assert torch.equal(odd, want) and out[1, 0, 40] == float("-inf")


def test_refusals():
    lib, P = lora.raw_lib(), lambda t: t.data_ptr()
    with Cache(2, 16, 2, 64, "f16") as c, Rope(64, 64) as rope, Rope(64, 128) as wide:
        k, q = rows(4, 2, 64, "f16", 1), rows(4, 3, 64, "f16", 2)
        s, p = i32([0, 1, 2, 3]), i32([0, 1, 2, 3])
        good = dict(kv=c.h, rope=rope.h, k=P(k), ks=128, v=P(k), vs=128, slots=P(s), positions=P(p), n=4, q=P(q), qs=192,
                    heads=3, out=P(q), os=192, stream=None)

        def call(**change):
            return lib.lora_kv_append(*{**good, **change}.values())
        assert call() == lora.LORA_OK
        assert call(n=0, k=None, positions=None, q=None) == lora.LORA_OK
        assert call(q=None, qs=-1, heads=-1, out=None, os=0) == lora.LORA_OK
        for change in (dict(kv=None), dict(rope=None), dict(n=-1), dict(k=None), dict(v=None), dict(slots=None),
                       dict(positions=None), dict(positions=P(p) + 2), dict(ks=120), dict(vs=132), dict(k=P(k) + 8),
                       dict(out=None), dict(heads=0), dict(heads=1 << 20), dict(qs=184), dict(os=196), dict(q=P(q) + 2),
                       dict(out=P(q) + 4), dict(os=200), dict(heads=4)):
            assert call(**change) == lora.LORA_EINVAL, change
        assert call(rope=wide.h) == lora.LORA_EMISMATCH
        with pytest.raises(ValueError, match="q_out"):
            lora.lora_kv_append(c.h, rope.h, k, k, s, p, 4, q=q)
        with pytest.raises(ValueError, match="positions"):
            lora.lora_kv_append(c.h, rope.h, k, k, s, p[:3], 4)
        with pytest.raises(ValueError, match="q_out"):
            lora.lora_kv_append(c.h, rope.h, k, k, s, p, 4, q=q, q_out=k)
        torch.cuda.synchronize()


def test_captured_and_replayed():
    """A captured append reads slots and positions as a replay finds them."""
    T = 21
    stream = torch.cuda.Stream()
    with Cache(6, 16, 2, 128, "bf16") as c, Rope(500, 128) as rope:
        k, v, q = (rows(T, h, 128, "bf16", s) for h, s in ((2, 1), (2, 2), (4, 3)))
        slots, positions, out = i32(range(T)), i32([range(T)]), torch.empty_like(q)
        torch.cuda.synchronize()
        gc.collect()
        gc.disable()  # nothing may be freed while the stream is captured
        try:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                lora.lora_kv_append(c.h, rope.h, k, v, slots, positions, T, q=q, q_out=out,
                                    stream=torch.cuda.current_stream())
        finally:
            gc.enable()
        for i in range(4):
            new, at = [(i * 17 + j * 5) % 96 for j in range(T)], [[100 * i + j for j in range(T)]]
            slots.copy_(i32(new))
            positions.copy_(i32(at))
            for x, seed in ((k, 10 + i), (v, 20 + i), (q, 30 + i)):
                x.copy_(rows(T, x.shape[1], 128, "bf16", seed))
            graph.replay()
            torch.cuda.synchronize()
            got = out.clone()
            eager = torch.empty_like(out)
            append(c, rope, k, v, new, at, q, eager)  # the same rows again: what the cache should hold
            assert torch.equal(got, eager)
            check_queries(rope, q, got, at)
            c.check(list(range(c.n)))
