"""Attention over the quantised cache against the 64-bit form, token by token:
types, head layouts, lengths from none to long, shared prefixes, ragged new
tokens, split and unsplit work, scales of every size, poisoned and unwritten
rows, strides, streams and graphs.  The tolerance is kv_reference's, derived
there."""
import numpy as np
import pytest
import torch

import kv_reference as ref
from rank_adapter_gemm_token_amd import lora

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


class Step:
    """A cache with every row written, and a batch on it."""

    def __init__(self, q_len, kv_len, group, prefix, heads, kv_heads, dim, page, dtype, seed=0, kscale=1.0,
                 vscale=1.0, qscale=1.0, spread=0.7, room=0):
        rng = np.random.default_rng(seed)
        self.q_len, self.kv_len, self.group, self.prefix = q_len, kv_len, group, prefix
        self.heads, self.kv_heads, self.dim, self.page, self.dtype = heads, kv_heads, dim, page, DT[dtype]
        own = [-(-n // page) for n in kv_len]
        pre = [-(-n // page) for n in prefix]
        total = sum(own) + sum(pre)
        self.n_pages = total + 2
        table = [int(x) for x in rng.permutation(self.n_pages)]
        self.pages = [[table.pop() for _ in range(n)] for n in own]
        self.prefix_pages = [[table.pop() for _ in range(n)] for n in pre]
        self.kv = lora.lora_kv_create(self.n_pages, page, kv_heads, dim, self.dtype)
        n = self.n_pages * page
        g = torch.Generator().manual_seed(seed)

        def rows(scale):
            x = torch.randn((n, kv_heads, dim), generator=g) * scale
            return (x * torch.exp(spread * torch.randn((n, kv_heads, 1), generator=g))).to(self.dtype)
        self.k_in, self.v_in = rows(kscale), rows(vscale)
        self.T = sum(q_len)
        # Queries as a part of a wider row.
        wide = torch.randn((max(1, self.T), heads * dim + 64), generator=g) * qscale
        self.q = wide.to(self.dtype).cuda()[:self.T, :heads * dim].unflatten(1, (heads, dim))
        self.scale = dim ** -0.5
        self.write()
        self.plan = lora.lora_attend_plan_create(max(1, len(q_len)) + room, len(prefix) + room,
                                                 max(1, self.T) + room, total + room, heads, kv_heads, dim)

    def write(self, slots=None):
        n = self.n_pages * self.page
        s = torch.arange(n, dtype=torch.int32) if slots is None else torch.tensor(slots, dtype=torch.int32)
        k, v = (x.cuda()[s.long().cuda()].contiguous() for x in (self.k_in, self.v_in))
        lora.lora_kv_write(self.kv, k, v, s.cuda(), s.numel())
        self.k, self.v = ref.held_pair(self.k_in.double().numpy(), self.v_in.double().numpy())

    def lists(self):
        def csr(rows):
            first = np.concatenate([[0], np.cumsum([len(r) for r in rows])])
            return [x for r in rows for x in r], first
        p, p0 = csr(self.pages)
        pp, pp0 = csr(self.prefix_pages)
        d = dict(q_len=self.q_len, kv_len=self.kv_len, group=self.group, pages=p, page0=p0, prefix_len=self.prefix,
                 prefix_pages=pp, prefix_page0=pp0)
        return {k: torch.tensor(np.array(v, dtype=np.int32)) for k, v in d.items()}

    def set_plan(self, stream=None):
        lora.lora_attend_plan_set(self.plan, self.kv, **self.lists(), stream=stream)

    def run(self, lse=True, plan=True):
        if plan:
            self.set_plan()
        out = torch.full((self.T, self.heads, self.dim), 7.0, dtype=self.dtype, device="cuda")
        l = torch.full((self.T, self.heads), 7.0, device="cuda") if lse else None
        lora.lora_attend(self.kv, self.plan, self.q, self.scale, out, l)
        return out, l

    def seen(self, s, j):
        """Slots of the keys that new token j of sequence s sees."""
        at = []
        if self.group[s] >= 0:
            g = self.group[s]
            at += [self.prefix_pages[g][i // self.page] * self.page + i % self.page for i in range(self.prefix[g])]
        n = max(0, self.kv_len[s] - self.q_len[s] + j + 1)
        return at + [self.pages[s][i // self.page] * self.page + i % self.page for i in range(n)]

    def check(self, out, lse, tokens=None):
        q = self.q.double().cpu().numpy()
        got, gl = out.double().cpu().numpy(), None if lse is None else lse.double().cpu().numpy()
        t = 0
        for s, n in enumerate(self.q_len):
            for j in range(n):
                if tokens is None or t in tokens:
                    self._check_token(t, self.seen(s, j), q, got, gl)
                t += 1

    def _check_token(self, t, at, q, got, gl):
        k, v = self.k[at], self.v[at]
        poisoned = np.isnan(k).any((0, 2)) if len(at) else np.zeros(self.kv_heads, bool)
        bad = np.repeat(poisoned, self.heads // self.kv_heads)
        want, wl, absv, top, mass = ref.attend(q[t], (np.nan_to_num(k), np.nan_to_num(v)), self.scale)
        assert np.isnan(got[t][bad]).all()
        tol, ltol = ref.attend_tolerance(want, absv, top, mass, len(at), self.dim, self.dtype)
        err = np.abs(got[t] - want)
        assert (err <= tol)[~bad].all(), "token %d: %.3g times its tolerance" % (t, np.nanmax((err / tol)[~bad]))
        if gl is None:
            return
        assert np.isnan(gl[t][bad]).all()
        if len(at) == 0:
            assert (gl[t] == -np.inf).all() and (got[t] == 0).all()
        else:
            assert (np.abs(gl[t] - wl) <= ltol)[~bad].all(), (t, gl[t], wl)

    def __enter__(self):
        return self

    def __exit__(self, *a):
        torch.cuda.synchronize()
        lora.lora_attend_plan_destroy(self.plan)
        lora.lora_kv_destroy(self.kv)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,dim", [(1, 1, 128), (8, 8, 128), (8, 2, 64), (14, 2, 64), (32, 1, 128),
                                                (12, 4, 128), (40, 2, 64)])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 200, 1111])
def test_one_sequence(dtype, heads, kv_heads, dim, n):
    with Step([1], [n], [-1], [], heads, kv_heads, dim, 16, dtype, seed=n) as s:
        s.check(*s.run())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,dim,page", [(8, 8, 128, 64), (8, 2, 128, 16), (6, 2, 64, 32)])
@pytest.mark.parametrize("prefix", [[1], [64], [500], [300, 0, 77], [2049, 130]])
def test_shared_prefixes(dtype, heads, kv_heads, dim, page, prefix):
    rng = np.random.default_rng(len(prefix) + prefix[0])
    B = 21
    group = [int(x) for x in rng.integers(-1, len(prefix), B)]
    q_len = [int(x) for x in rng.integers(0, 4, B)]
    kv_len = [int(x) for x in rng.integers(4, 150, B)]
    with Step(q_len, kv_len, group, prefix, heads, kv_heads, dim, page, dtype, seed=prefix[0]) as s:
        s.check(*s.run())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_many_rows_of_one_prefix(dtype):
    """Blocks of query rows that end inside a sequence's tokens, and many of them."""
    B = 70
    with Step([3] * B, [3 + i % 5 for i in range(B)], [0] * B, [777], 4, 2, 64, 16, dtype) as s:
        s.check(*s.run())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
def test_workgroups_of_items_of_different_sizes(dtype, dim):
    """So many short sequences that each is one wave's work, with query rows for
    one and for two blocks side by side in a workgroup."""
    rng = np.random.default_rng(dim)
    B = 90
    q_len = [int(x) for x in rng.integers(1, 9, B)]
    kv_len = [int(x) for x in rng.integers(8, 200, B)]
    with Step(q_len, kv_len, [-1] * B, [], 128, 32, dim, 16, dtype) as s:
        s.check(*s.run(), tokens=set(range(0, sum(q_len), 3)))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_rows_that_see_nothing(dtype):
    """No keys at all; new tokens before a sequence's first key; an empty
    prefix; sequences with nothing new."""
    with Step([2, 3, 1, 0, 4, 1, 2], [0, 1, 0, 9, 2, 1, 0], [-1, -1, 0, 1, 1, 0, 1], [0, 40], 6, 2, 64, 16,
              dtype) as s:
        out, lse = s.run()
        s.check(out, lse)
        assert (lse == -torch.inf).sum() == (2 + 2 + 1) * 6


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_a_prompt_in_one_call(dtype):
    """As many new tokens as keys: causal over several tiles and row blocks."""
    with Step([150, 70], [150, 201], [-1, 0], [65], 4, 2, 128, 16, dtype) as s:
        s.check(*s.run())


@pytest.mark.parametrize("dtype,kscale,vscale,qscale", [("f16", 1e-3, 1e-3, 100.0), ("f16", 300.0, 2000.0, 0.02),
                                                        ("bf16", 1e-12, 1e-15, 1e12), ("bf16", 1e10, 1e20, 1e-9),
                                                        ("f16", 8.0, 1.0, 8.0), ("bf16", 1.0, 1.0, 0.0)])
def test_sizes_of_values(dtype, kscale, vscale, qscale):
    with Step([1, 2, 1], [333, 80, 700], [0, 0, -1], [260], 4, 2, 64, 16, dtype, kscale=kscale, vscale=vscale,
              qscale=qscale, spread=1.5) as s:
        s.check(*s.run())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_values_of_very_different_size(dtype):
    """Value rows from 2^-12 to 2^12 and rows of zeros side by side."""
    with Step([1, 1], [500, 90], [0, 0], [129], 4, 2, 64, 16, dtype) as s:
        e = torch.randint(-12, 13, (s.v_in.shape[0], s.kv_heads, 1), generator=torch.Generator().manual_seed(1))
        s.v_in = (s.v_in.float() * torch.exp2(e.float())).to(s.dtype)
        s.v_in[::3] = 0
        s.k_in[::5] = 0
        s.write()
        s.check(*s.run())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_a_poisoned_row_is_seen_by_its_readers_alone(dtype):
    """NaN and infinity in keys and values: of a head, for the tokens that see
    them; not in the rest of a page past a length, nor after a causal limit."""
    with Step([3, 3, 1], [40, 70, 30], [0, 1, -1], [50, 64], 4, 2, 64, 16, dtype) as s:
        def at(pages, i):
            return pages[i // 16] * 16 + i % 16
        s.k_in[at(s.pages[0], 38), 0, 3] = float("nan")       # the second of three new tokens, head 0
        s.v_in[at(s.pages[1], 69), 1, 7] = float("inf")       # the last of three new tokens, head 1
        s.v_in[at(s.prefix_pages[1], 10), 0, 0] = float("-inf")  # everyone of group 1, head 0
        for i in range(50, 64):                               # past a prefix's length
            s.v_in[at(s.prefix_pages[0], i)] = float("nan")
        for i in range(30, 32):                               # past a sequence's length
            s.k_in[at(s.pages[2], i)] = float("inf")
        s.write()
        out, lse = s.run()
        s.check(out, lse)
        nan = out.isnan().all(-1).cpu()
        assert nan.sum() == 2 * 2 + 1 * 2 + 3 * 2


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_queries_that_are_not_finite_are_alone(dtype):
    """A NaN or infinite query spoils its own row's output and no other's."""
    with Step([1, 3, 1], [40, 70, 30], [0, 0, -1], [300], 8, 2, 64, 16, dtype) as s:
        s.q = s.q.contiguous()
        clean, lse = s.run()
        s.check(clean, lse)
        s.q[2, 5] = float("nan")
        s.q[4, 0, 3] = float("inf")
        out, l = s.run()
        bad = torch.zeros(s.T, s.heads, dtype=torch.bool, device="cuda")
        bad[2, 5] = bad[4, 0] = True
        assert out[bad].isnan().all() and l[bad].isnan().all()
        assert torch.equal(out[~bad], clean[~bad]) and torch.equal(l[~bad], lse[~bad])


def test_nothing_to_do():
    """No sequences, and sequences with nothing new: nothing is written."""
    with Step([0, 0], [20, 0], [0, -1], [33], 4, 2, 64, 16, "f16", room=4) as s:
        out, lse = s.run()
        assert out.numel() == 0
        i = torch.zeros(0, dtype=torch.int32)
        lora.lora_attend_plan_set(s.plan, s.kv, i, i, i, i, i)
        kept = torch.full((2, 4, 64), 7.0, dtype=torch.float16, device="cuda")
        lora.lora_attend(s.kv, s.plan, kept, 1.0, torch.empty_like(kept))
        assert (kept == 7).all()


def test_pages_past_32_bit_bytes():
    """A cache of over 4 GiB of keys and of values, a sequence whose pages lie
    at its ends and around 2^31 and 2^32 bytes."""
    heads, dim, page = 32, 128, 64
    per = page * heads * dim
    n_pages = (1 << 32) // per + 40
    kv = lora.lora_kv_create(n_pages, page, heads, dim, torch.bfloat16)
    plan = lora.lora_attend_plan_create(1, 1, 1, 16, heads, heads, dim)
    try:
        pages = [0, (1 << 31) // per - 1, (1 << 31) // per, (1 << 32) // per - 1, (1 << 32) // per, n_pages - 1]
        prefix = [(1 << 32) // per + 7, 5]
        g = torch.Generator().manual_seed(1)
        n = (len(pages) + len(prefix)) * page
        k, v = (torch.randn((n, heads, dim), generator=g).bfloat16() for _ in range(2))
        slots = [p * page + i for p in prefix + pages for i in range(page)]
        lora.lora_kv_write(kv, k.cuda(), v.cuda(), torch.tensor(slots, dtype=torch.int32, device="cuda"), n)

        def i32(x):
            return torch.tensor(x, dtype=torch.int32)
        lora.lora_attend_plan_set(plan, kv, i32([1]), i32([len(pages) * page]), i32([0]), i32(pages),
                                  i32([0, len(pages)]), i32([2 * page]), i32(prefix), i32([0, 2]))
        q = torch.randn((1, heads, dim), generator=g).bfloat16()
        out, lse = torch.empty_like(q, device="cuda"), torch.empty((1, heads), device="cuda")
        lora.lora_attend(kv, plan, q.cuda(), dim ** -0.5, out, lse)
        kk, vv = ref.held_pair(k.double().numpy(), v.double().numpy())
        want, wl, absv, top, mass = ref.attend(q[0].double().numpy(), (kk, vv), dim ** -0.5)
        tol, ltol = ref.attend_tolerance(want, absv, top, mass, n, dim, torch.bfloat16)
        assert (np.abs(out[0].double().cpu().numpy() - want) <= tol).all()
        assert (np.abs(lse[0].double().cpu().numpy() - wl) <= ltol).all()
    finally:
        torch.cuda.synchronize()
        lora.lora_attend_plan_destroy(plan)
        lora.lora_kv_destroy(kv)


def test_rows_never_written_are_zeros():
    with Step([1, 1], [100, 40], [-1, 0], [33], 2, 1, 64, 16, "f16") as s:
        lora.lora_kv_destroy(s.kv)
        s.kv = lora.lora_kv_create(s.n_pages, s.page, s.kv_heads, s.dim, s.dtype)
        n = s.n_pages * s.page
        some = [i for i in range(n) if i % 3]
        s.k_in[::3] = 0
        s.v_in[::3] = 0
        s.write(some)
        s.check(*s.run())


def test_equal_batches_in_any_order_give_equal_bits():
    """Which sequences share a batch changes no bit where the split does not
    change, and calling again changes none at all."""
    with Step([1] * 40, [100 + i for i in range(40)], [i % 2 for i in range(40)], [640, 1000], 8, 8, 128, 16,
              "bf16") as s:
        a, la = s.run()
        for _ in range(3):
            b, lb = s.run()
            assert torch.equal(a, b) and torch.equal(la, lb)


def test_without_lse_and_scale():
    with Step([2, 1], [90, 300], [-1, -1], [], 4, 4, 64, 16, "f16") as s:
        for scale in (0.0, -0.3, 1.0):
            s.scale = scale
            s.check(*s.run(lse=False))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_long_rows(dtype):
    n = 40000
    with Step([1, 1], [n, 33], [0, 0], [9000], 2, 1, 128, 64, dtype, qscale=2.0) as s:
        s.check(*s.run())


def test_large_batch_spot_checked():
    """Sizes of a served batch: some of its tokens against the 64-bit form."""
    rng = np.random.default_rng(5)
    B = 200
    group = [int(x) for x in rng.integers(0, 3, B)]
    kv = [int(x) for x in rng.integers(1, 300, B)]
    with Step([1] * B, kv, group, [2000, 100, 3333], 32, 32, 128, 64, "bf16") as s:
        out, lse = s.run()
        assert not out.isnan().any()
        s.check(out, lse, tokens=set(int(x) for x in rng.integers(0, B, 12)))


def test_another_stream_and_plans_in_a_row():
    """Plans and attention on a stream of their own, with the next plan made
    while the last attention may still run."""
    st = torch.cuda.Stream()
    with Step([1, 2, 1], [100, 300, 50], [0, 0, -1], [500], 4, 2, 64, 16, "f16", room=8) as s:
        lists = []
        for i in range(6):
            kv = [100 - i, 300 - 40 * i, 50]
            lists.append(kv)
        outs = []
        torch.cuda.synchronize()
        for kv in lists:
            s.kv_len = kv
            s.set_plan(stream=st)
            out = torch.empty((s.T, s.heads, s.dim), dtype=s.dtype, device="cuda")
            lse = torch.empty((s.T, s.heads), device="cuda")
            lora.lora_attend(s.kv, s.plan, s.q, s.scale, out, lse, stream=st)
            outs.append((out, lse))
        st.synchronize()
        for kv, (out, lse) in zip(lists, outs):
            s.kv_len = kv
            s.check(out, lse)


def test_a_graph_follows_the_plan():
    """Captured once, replayed after plans of fewer and of more work."""
    with Step([1, 2, 1], [100, 300, 50], [0, 0, -1], [500], 4, 2, 64, 16, "f16", room=8) as s:
        s.kv_len, short = [1, 2, 0], [100, 300, 50]
        s.prefix, long = [0], [500]
        s.set_plan()
        out = torch.empty((s.T, s.heads, s.dim), dtype=s.dtype, device="cuda")
        lse = torch.empty((s.T, s.heads), device="cuda")
        st = torch.cuda.Stream()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(st), torch.cuda.graph(graph, stream=st):
            lora.lora_attend(s.kv, s.plan, s.q, s.scale, out, lse)
            with pytest.raises(lora.LoraError):  # a plan is not captured
                s.set_plan()
        for kv, prefix in ((short, long), ([1, 2, 0], [0]), ([60, 299, 1], [499]), (short, long)):
            s.kv_len, s.prefix = kv, prefix
            s.set_plan()
            torch.cuda.synchronize()
            out.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            s.check(out, lse)
            eager, el = s.run()
            assert torch.equal(eager, out) and torch.equal(el, lse)


def test_a_graph_of_two_launches_follows_the_plan():
    """As above where the partial results are joined by a second launch."""
    rng = np.random.default_rng(3)
    B = 60
    kv = [int(x) for x in rng.integers(100, 400, B)]
    with Step([1] * B, kv, [i % 3 - 1 for i in range(B)], [300, 600], 32, 32, 64, 16, "bf16", room=8) as s:
        s.set_plan()
        out = torch.empty((s.T, s.heads, s.dim), dtype=s.dtype, device="cuda")
        lse = torch.empty((s.T, s.heads), device="cuda")
        st = torch.cuda.Stream()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(st), torch.cuda.graph(graph, stream=st):
            lora.lora_attend(s.kv, s.plan, s.q, s.scale, out, lse)
        for k in (kv, [1] * B, [min(n, 120) for n in kv], kv):
            s.kv_len = k
            s.set_plan()
            torch.cuda.synchronize()
            out.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            s.check(out, lse, tokens={0, 1, 2, 17, 59})
            eager, el = s.run()
            assert torch.equal(eager, out) and torch.equal(el, lse)


def test_refusals():
    lib = lora.raw_lib()
    with Step([1, 1], [20, 40], [-1, 0], [33], 4, 2, 64, 16, "f16") as s:
        out = torch.empty((2, 4, 64), dtype=torch.float16, device="cuda")
        q, o = s.q.data_ptr(), out.data_ptr()
        import ctypes
        f = ctypes.c_float
        assert lib.lora_attend(s.kv, s.plan, q, 320, f(1), o, None, None) == lora.LORA_EINVAL  # no plan yet
        s.set_plan()
        assert lib.lora_attend(s.kv, s.plan, q, 320, f(1), o, None, None) == lora.LORA_OK
        for args in [(None, 320, f(1), o), (q, 320, f(1), None), (q, 255, f(1), o), (q, 252, f(1), o),
                     (q + 2, 320, f(1), o), (q, 320, f(float("nan")), o), (q, 320, f(float("inf")), o),
                     (q, 320, f(1), q)]:
            assert lib.lora_attend(s.kv, s.plan, *args, None, None) == lora.LORA_EINVAL, args
        other = lora.lora_kv_create(s.n_pages + 1, 16, 2, 64, torch.float16)
        wide = lora.lora_kv_create(s.n_pages, 16, 2, 128, torch.float16)
        try:
            for kv in (other, wide):
                assert lib.lora_attend(kv, s.plan, q, 320, f(1), o, None, None) == lora.LORA_EMISMATCH
            good, s.kv = s.kv, wide
            with pytest.raises(lora.LoraError) as e:
                s.set_plan()
            assert e.value.status == lora.LORA_EMISMATCH
            s.kv = good
        finally:
            lora.lora_kv_destroy(other)
            lora.lora_kv_destroy(wide)
        page = s.pages[1][0]
        s.pages[1][0] = s.n_pages  # a page the cache has not
        with pytest.raises(lora.LoraError) as e:
            s.set_plan()
        assert e.value.status == lora.LORA_EINVAL
        # A refused plan leaves none.
        assert lib.lora_attend(s.kv, s.plan, q, 320, f(1), o, None, None) == lora.LORA_EINVAL
        s.pages[1][0] = page
        s.check(*s.run())
