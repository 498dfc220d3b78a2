"""The operators of one serving step with drafted tokens, as they are measured:

  cache   new keys and values quantised into the paged 8-bit cache as they are
          written, and rows of the cache read back;
  attend  attention of a batch's new tokens over that cache, where sequences of
          one tenant share a long prefix that is computed once for all of them;
  verify  drafted tokens accepted or replaced against the target's
          probabilities, from given random numbers.

`own` false: the plain forms, elementary torch operations in 32 bits (64 where
a border decides).  `own` true: the calls a user's program makes of
rank_adapter_gemm_token_amd.lora.
"""
import numpy as np
import torch

own = False

DTYPE = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- the cases --

def _cache(name, tokens, heads, dim, page, dtype, run):
    """tokens: new tokens a call; run: they come in runs of so many neighbours
    (1: one new token for each sequence, as in decode)."""
    return {"name": name, "op": "cache", "tokens": tokens, "heads": heads, "dim": dim, "page": page,
            "dtype": dtype, "run": run}


def _attend(name, seqs, new, heads, kv_heads, dim, page, groups, prefix, own_len, ragged, dtype):
    """new: new tokens a sequence (ragged: 0 .. new); own_len: a sequence's own
    tokens, the new ones among them (ragged: from `new` to own_len); prefix:
    tokens of a group's prefix (ragged: half to all of it); groups 0: none."""
    return {"name": name, "op": "attend", "seqs": seqs, "new": new, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "page": page, "groups": groups, "prefix": prefix, "own_len": own_len, "ragged": ragged,
            "dtype": dtype}


def _verify(name, seqs, drafts, vocab, ragged, dtype):
    return {"name": name, "op": "verify", "seqs": seqs, "drafts": drafts, "vocab": vocab, "ragged": ragged,
            "dtype": dtype}


def listed():
    return [
        # One sequence's next token, few key/value heads: latency alone.
        _cache("cache_one_token", 1, 8, 128, 64, "bf16", 1),
        # A decode step of 64 sequences of a 4096-wide model: one row each, far apart.
        _cache("cache_decode_64", 64, 32, 128, 16, "f16", 1),
        # Prefill of eight 512-token chunks: long runs, bandwidth.
        _cache("cache_prefill_4096", 4096, 32, 128, 64, "bf16", 512),
        # One sequence alone, no prefix, 4096-wide: latency and the split of a long row.
        _attend("attend_single", 1, 1, 32, 32, 128, 64, 0, 0, 2001, False, "f16"),
        # 64 decoding tokens of six tenants, each tenant's system prompt shared.
        _attend("attend_decode_64", 64, 1, 32, 32, 128, 64, 6, 2048, 512, True, "f16"),
        # Four drafted tokens and the last accepted one a sequence, grouped heads, a long shared document.
        _attend("attend_drafted_64", 64, 5, 32, 8, 128, 16, 4, 8192, 1024, True, "bf16"),
        # One prefix for the whole batch, as long as it gets here: the largest call.
        _attend("attend_prefix_256", 256, 1, 32, 32, 128, 64, 1, 16384, 256, True, "bf16"),
        # Odd everything: seven heads to a key head, short ragged lengths, sequences with nothing new.
        _attend("attend_odd", 19, 3, 14, 2, 64, 16, 3, 301, 133, True, "bf16"),
        # One sequence, four drafts, a 32000-token vocabulary: latency.
        _verify("verify_one", 1, 4, 32000, False, "f32"),
        # 64 sequences with up to seven drafts each.
        _verify("verify_64", 64, 7, 32000, True, "f32"),
        # A large batch over a large vocabulary, probabilities kept in 16 bits.
        _verify("verify_256", 256, 4, 131072, False, "bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number of lo .. hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["cache", "attend", "attend", "verify"])
    if op == "cache":
        run = rng.choice([1, 1, 7, 64, 333, 512])
        c = _cache("", _log(rng, 1, 4096), rng.choice([1, 2, 4, 8, 12, 32, 40]), rng.choice([64, 128]),
                   rng.choice([16, 32, 64, 128]), rng.choice(["f16", "bf16"]), run)
    elif op == "attend":
        most = _cost(listed()[6])
        while True:
            kv = rng.choice([1, 2, 4, 8, 8, 32])
            per = rng.choice([1, 1, 2, 4, 5, 7, 8]) if kv < 32 else 1
            groups = rng.choice([0, 1, 1, 2, 4, 7])
            new = rng.choice([1, 1, 2, 3, 5, 8])
            c = _attend("", _log(rng, 1, 256), new, kv * per, kv, rng.choice([64, 128]), rng.choice([16, 32, 64]),
                        groups, _log(rng, 1, 16384) if groups else 0, _log(rng, new, 4096), rng.random() < 0.7,
                        rng.choice(["f16", "bf16"]))
            if _cost(c) <= most:
                break
    else:
        c = _verify("", _log(rng, 1, 256), rng.randint(1, 8), _log(rng, 300, 131072), rng.random() < 0.5,
                    rng.choice(["f32", "f16", "bf16"]))
    del c["name"]
    return c


def _cost(c):
    w = work(c)
    return w["bytes"] / 8e12 + w["flops"] / 2.5e15


def work(case):
    c = case
    if c["op"] == "cache":
        # Keys and values read once in 16 bits, held once in 8 bits with a
        # scale, and the rows read back written once in 16 bits.
        rows = c["tokens"] * c["heads"] * 2
        back = (c["tokens"] + _old_rows(c)) * c["heads"] * 2
        d = c["dim"]
        return {"bytes": rows * (2 * d + d + 1) + back * (d + 1 + 2 * d) + 4 * (2 * c["tokens"] + _old_rows(c)),
                "flops": rows * d * 3 + back * d}
    if c["op"] == "attend":
        # The mean lengths of what prepare() makes.
        f = 0.75 if c["ragged"] else 1.0
        new = c["seqs"] * c["new"] * (0.5 if c["ragged"] and c["new"] > 1 else 1.0)
        pre = c["prefix"] * f
        mean = (c["new"] + c["own_len"]) / 2 if c["ragged"] else c["own_len"]
        tokens = c["groups"] * pre + c["seqs"] * mean
        row = c["kv_heads"] * (c["dim"] + 1) * 2
        return {"bytes": int(tokens * row + new * c["heads"] * (4 * c["dim"] + 4)),
                "flops": int(4 * c["dim"] * c["heads"] * new * ((pre if c["groups"] else 0) + mean))}
    # One row of the target's and one of the draft's probabilities a sequence.
    e = 4 if c["dtype"] == "f32" else 2
    return {"bytes": c["seqs"] * (2 * c["vocab"] * e + (c["drafts"] + 1) * 16), "flops": c["seqs"] * c["vocab"] * 3}


def _old_rows(c):
    return c["tokens"] // 4 + 3


# --------------------------------------------------------------- the inputs --

class _Handle:
    """A handle of the library, destroyed with the state that holds it."""

    def __init__(self, destroy, handle):
        self.destroy, self.h = destroy, handle

    def __del__(self):
        self.destroy(self.h)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    return {"cache": _prepare_cache, "attend": _prepare_attend, "verify": _prepare_verify}[case["op"]](case, g, rng)


def _counts(case, most, rng):
    """0 .. most for each sequence, once at least `most`.  Their sum, and with
    it the outputs' shape, goes by the case; who has how many, by the seed."""
    n = np.random.default_rng([case["seqs"], most]).integers(0, most + 1, case["seqs"])
    n[0] = most
    return rng.permutation(n)


def _rows(n, heads, dim, dtype, g):
    """Keys or values: a spread of sizes from token to token, and a few
    channels several times larger than the others."""
    x = torch.randn((n, heads, dim), device="cuda", generator=g)
    x *= torch.exp(0.5 * torch.randn((n, 1, 1), device="cuda", generator=g))
    x *= torch.where(torch.rand((1, heads, dim), device="cuda", generator=g) < 0.03, 6.0, 1.0)
    return x.to(dtype)


def _empty_cache(n_slots, heads, dim):
    """The plain cache: elements and one scale a row and head, for keys and for
    values; one more row takes what is written nowhere."""
    def part():
        return {"e": torch.zeros((n_slots + 1, heads, dim), device="cuda", dtype=torch.uint8),
                "s": torch.ones((n_slots + 1, heads), device="cuda")}
    return {"k": part(), "v": part(), "n_slots": n_slots}


def _fill(st, c, n_slots, slots, k, v):
    """The cache as it stands before the call, in the form the call reads."""
    if own:
        from rank_adapter_gemm_token_amd import lora
        st["kv"] = _Handle(lora.lora_kv_destroy, lora.lora_kv_create(
            n_slots // c["page"], c["page"], st["heads"], c["dim"], DTYPE[c["dtype"]]))
        lora.lora_kv_write(st["kv"].h, k, v, slots, slots.numel())
    else:
        st["plain"] = _empty_cache(n_slots, st["heads"], c["dim"])
        _write(st["plain"], k, v, slots)


def _prepare_cache(c, g, rng):
    T, page, run, dt = c["tokens"], c["page"], c["run"], DTYPE[c["dtype"]]
    old = _old_rows(c)
    runs = -(-T // run)
    pages_each = -(-run // page) + 1
    n_pages = runs * pages_each + -(-old // page) + 2
    table = rng.permutation(n_pages)
    slots = []
    for i in range(runs):  # each run starts somewhere in a page of its own and goes on in further ones
        at = int(rng.integers(0, page)) + np.arange(min(run, T - i * run))
        own_pages = table[i * pages_each:(i + 1) * pages_each]
        slots.append(own_pages[at // page] * page + at % page)
    slots = np.concatenate(slots)
    if T > 8:  # a padded batch: some tokens go nowhere
        slots[rng.integers(0, T, max(1, T // 50))] = -1
    at = np.arange(old)
    old_slots = table[runs * pages_each + at // page] * page + at % page
    back = np.concatenate([slots[slots >= 0], old_slots])
    back = np.concatenate([back, back[:T + old - len(back)]])
    st = {"case": c, "heads": c["heads"], "k": _rows(T, c["heads"], c["dim"], dt, g),
          "v": _rows(T, c["heads"], c["dim"], dt, g),
          "slots": torch.from_numpy(slots.astype(np.int32)).cuda(),
          "back": torch.from_numpy(back.astype(np.int32)).cuda()}
    o = torch.from_numpy(old_slots.astype(np.int32)).cuda()
    st["old"] = (o, _rows(old, c["heads"], c["dim"], dt, g), _rows(old, c["heads"], c["dim"], dt, g))
    _fill(st, c, n_pages * page, *st["old"])
    return st


def _prepare_attend(c, g, rng):
    B, G, page, dt = c["seqs"], c["groups"], c["page"], DTYPE[c["dtype"]]
    if c["ragged"]:
        q_len = _counts(c, c["new"], rng) if c["new"] > 1 else np.ones(B, dtype=np.int64)
        kv_len = rng.integers(c["new"], c["own_len"] + 1, B)
        prefix_len = rng.integers((c["prefix"] + 1) // 2, c["prefix"] + 1, G)
    else:
        q_len, kv_len, prefix_len = np.full(B, c["new"]), np.full(B, c["own_len"]), np.full(G, c["prefix"])
    group = rng.integers(0, G, B) if G else np.full(B, -1)
    if G and B > 8:  # a sequence or two of no group
        group[rng.integers(0, B, B // 16)] = -1
    own_pages, pre_pages = -(-kv_len // page), -(-prefix_len // page)
    total = int(own_pages.sum() + pre_pages.sum())
    n_pages = total + 3
    table = rng.permutation(n_pages)[:total].astype(np.int32)
    n_pre = int(pre_pages.sum())

    def first(n):
        return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    host = {"q_len": q_len, "kv_len": kv_len, "group": group, "pages": table[n_pre:], "page0": first(own_pages),
            "prefix_len": prefix_len, "prefix_pages": table[:n_pre], "prefix_page0": first(pre_pages)}
    host = {k: torch.from_numpy(np.ascontiguousarray(v, dtype=np.int32)) for k, v in host.items()}
    st = {"case": c, "heads": c["kv_heads"], "host": host, "scale": c["dim"] ** -0.5}
    T = int(q_len.sum())
    # The queries are a part of the fused projection's output.
    qkv = torch.randn((T, (c["heads"] + 2 * c["kv_heads"]) * c["dim"]), device="cuda", generator=g).to(dt)
    st["q"] = qkv[:, :c["heads"] * c["dim"]].unflatten(1, (c["heads"], c["dim"]))
    # Every page's rows are written, the ones past a length too.
    n_slots = n_pages * page
    step = max(1, (1 << 27) // (c["kv_heads"] * c["dim"]))
    slots = torch.arange(n_slots, device="cuda", dtype=torch.int32)
    k = torch.cat([_rows(min(step, n_slots - i), c["kv_heads"], c["dim"], dt, g) for i in range(0, n_slots, step)])
    v = torch.cat([_rows(min(step, n_slots - i), c["kv_heads"], c["dim"], dt, g) for i in range(0, n_slots, step)])
    _fill(st, c, n_slots, slots, k, v)
    if own:
        from rank_adapter_gemm_token_amd import lora
        st["plan"] = _Handle(lora.lora_attend_plan_destroy, lora.lora_attend_plan_create(
            B, G, T, total, c["heads"], c["kv_heads"], c["dim"]))
        lora.lora_attend_plan_set(st["plan"].h, st["kv"].h, **host)
    else:
        st["dev"] = _padded(host, page, T)
    return st


def _padded(host, page, T):
    """The batch's lists as rectangles on the device: what a program of batched
    products keeps for a step.  -1: nothing there."""
    q_len, group = host["q_len"].numpy(), host["group"].numpy()
    q0 = np.concatenate([[0], np.cumsum(q_len)])
    B, G = len(q_len), len(host["prefix_len"])

    def rect(rows):
        w = max([len(r) for r in rows] + [1])
        return torch.tensor([list(r) + [-1] * (w - len(r)) for r in rows], device="cuda", dtype=torch.int64)

    def pages(p, p0):
        return rect([p[p0[i]:p0[i + 1]].tolist() for i in range(len(p0) - 1)])
    d = {"T": T, "q_len": host["q_len"].cuda().long(), "kv_len": host["kv_len"].cuda().long(),
         "own_rows": rect([range(q0[b], q0[b + 1]) for b in range(B)]),
         "own_pages": pages(host["pages"], host["page0"])}
    if G:
        d["prefix_len"] = host["prefix_len"].cuda().long()
        d["prefix_pages"] = pages(host["prefix_pages"], host["prefix_page0"])
        d["prefix_rows"] = rect([[t for b in range(B) if group[b] == i for t in range(q0[b], q0[b + 1])]
                                 for i in range(G)])
    return d


def _prepare_verify(c, g, rng):
    B, V, dt = c["seqs"], c["vocab"], DTYPE[c["dtype"]]
    n = _counts(c, c["drafts"], rng) if c["ragged"] else np.full(B, c["drafts"])
    T, D = int((n + 1).sum()), int(n.sum())
    row0 = np.concatenate([[0], np.cumsum(n + 1)]).astype(np.int32)
    seq_of = np.repeat(np.arange(B), n)
    drafted = torch.from_numpy(np.arange(D) + seq_of).cuda()  # the target row of each drafted token
    z = 3.0 * torch.randn((T, V), device="cuda", generator=g)
    p = torch.softmax(z, -1).to(dt)
    z = z[drafted] + 0.7 * torch.randn((D, V), device="cuda", generator=g)
    q = torch.softmax(z, -1)
    draft = torch.multinomial(q, 1, generator=g).view(-1).to(torch.int32)
    return {"case": c, "p": p, "q": q.to(dt), "draft": draft, "row0": torch.from_numpy(row0).cuda(),
            "u": torch.rand((T,), device="cuda", generator=g),
            "tokens": torch.empty((T,), device="cuda", dtype=torch.int32),
            "accepted": torch.empty((B,), device="cuda", dtype=torch.int32), **_verifier(B)}


def _verifier(B):
    if own:
        from rank_adapter_gemm_token_amd import lora
        return {"verifier": _Handle(lora.lora_verifier_destroy, lora.lora_verifier_create(B))}
    return {}


# ------------------------------------------------------------------ the run --

def run(state):
    return {"cache": _run_cache, "attend": _run_attend, "verify": _run_verify}[state["case"]["op"]](state)


def _run_cache(st):
    k, v, back = st["k"], st["v"], st["back"]
    if own:
        from rank_adapter_gemm_token_amd import lora
        k_out = torch.empty((back.numel(), *k.shape[1:]), device="cuda", dtype=k.dtype)
        v_out = torch.empty_like(k_out)
        lora.lora_kv_write(st["kv"].h, k, v, st["slots"], k.shape[0])
        lora.lora_kv_read(st["kv"].h, back, back.numel(), k_out, v_out)
        return k_out, v_out
    _write(st["plain"], k, v, st["slots"])
    return tuple(_held(st["plain"][x], back).to(k.dtype) for x in "kv")


def _run_attend(st):
    q = st["q"]
    if own:
        from rank_adapter_gemm_token_amd import lora
        out = torch.empty(q.shape, device="cuda", dtype=q.dtype)
        lse = torch.empty(q.shape[:2], device="cuda", dtype=torch.float32)
        lora.lora_attend(st["kv"].h, st["plan"].h, q, st["scale"], out, lse)
        return out, lse
    return _attend_plain(st)


def _run_verify(st):
    B, T = st["case"]["seqs"], st["p"].shape[0]
    if own:
        from rank_adapter_gemm_token_amd import lora
        lora.lora_verify(st["verifier"].h, st["p"], st["q"], st["draft"], st["row0"], st["u"], B, T, st["tokens"],
                         st["accepted"])
        return st["tokens"], st["accepted"]
    return _verify_plain(st)


# ---------------------------------------------------------- the plain forms --

def _write(cache, k, v, slots):
    """Row x of a head is held as e * 2^s: the least whole s >= -64 with
    |x| <= 448 * 2^s, and e = x / 2^s rounded to e4m3, ties to even."""
    at = torch.where(slots < 0, cache["n_slots"], slots).long()
    for part, x in ((cache["k"], k), (cache["v"], v)):
        x = x.float()
        amax = x.abs().amax(-1)
        m, e = torch.frexp(amax)
        s = torch.where(m <= 0.875, e - 9, e - 8)
        s = torch.where(amax == 0, -64, s).clamp(min=-64).float()
        part["e"][at] = (x * torch.exp2(-s)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        part["s"][at] = torch.exp2(s)


def _held(part, slots):
    slots = slots.long()
    return part["e"][slots].view(torch.float8_e4m3fn).float() * part["s"][slots][..., None]


def _block(st, q, rows, pages, length, limit):
    """Unnormalised attention of the query rows `rows` [n, r] (-1: none) over
    the tokens of `pages` [n, p]; limit [n, r]: how many of them a row sees.
    Returns (largest score, sum, weighted values) for [n, kv_heads, r, per]."""
    c = st["case"]
    page, kv, per = c["page"], c["kv_heads"], c["heads"] // c["kv_heads"]
    slots = (pages.clamp(min=0)[:, :, None] * page + torch.arange(page, device="cuda")).flatten(1)
    slots = slots[:, :max(1, length)]
    n, r, L = rows.shape[0], rows.shape[1], slots.shape[1]
    k = _held(st["plain"]["k"], slots).permute(0, 2, 3, 1)  # [n, kv, dim, L]
    v = _held(st["plain"]["v"], slots).permute(0, 2, 1, 3)  # [n, kv, L, dim]
    x = q[rows.clamp(min=0)].float().view(n, r, kv, per, -1).permute(0, 2, 1, 3, 4).reshape(n * kv, r * per, -1)
    s = torch.bmm(x, k.reshape(n * kv, -1, L)) * st["scale"]
    seen = torch.arange(L, device="cuda") < limit[:, :, None]  # [n, r, L]
    s = s.view(n, kv, r, per, L).masked_fill(~seen[:, None, :, None, :], -torch.inf)
    m = s.amax(-1)
    p = torch.exp(s - torch.where(m == -torch.inf, 0.0, m)[..., None])
    o = torch.bmm(p.view(n * kv, r * per, L), v.reshape(n * kv, L, -1)).view(n, kv, r, per, -1)
    return m, p.sum(-1), o


def _attend_plain(st):
    q, d, h = st["q"], st["dev"], st["host"]
    T, H, dim = q.shape
    parts = []

    def add(rows, m, s, o):
        """[n, kv, r, per] to [T, heads], -inf and 0 where a token is in no row."""
        at = torch.where(rows < 0, T, rows).flatten()
        full = [torch.full((T + 1, H), -torch.inf, device="cuda"), torch.zeros((T + 1, H), device="cuda"),
                torch.zeros((T + 1, H, dim), device="cuda")]
        full[0][at] = m.transpose(1, 2).reshape(-1, H)
        full[1][at] = s.transpose(1, 2).reshape(-1, H)
        full[2][at] = o.transpose(1, 2).reshape(-1, H, dim)
        parts.append([f[:T] for f in full])
    if h["prefix_len"].numel():
        rows = d["prefix_rows"]
        limit = d["prefix_len"][:, None].expand(rows.shape)
        add(rows, *_block(st, q, rows, d["prefix_pages"], int(h["prefix_len"].max()), limit))
    rows = d["own_rows"]
    # New token j of n sees the sequence's own tokens up to itself.
    limit = (d["kv_len"] - d["q_len"])[:, None] + 1 + torch.arange(rows.shape[1], device="cuda")
    add(rows, *_block(st, q, rows, d["own_pages"], int(h["kv_len"].max()), limit))
    m = torch.stack([p[0] for p in parts]).amax(0)
    w = [torch.exp(p[0] - torch.where(m == -torch.inf, 0.0, m)) for p in parts]
    s = sum(f * p[1] for f, p in zip(w, parts))
    o = sum(f[..., None] * p[2] for f, p in zip(w, parts))
    out = torch.where(s[..., None] > 0, o / s[..., None], 0.0)
    return out.to(q.dtype), m + torch.log(s)


def _verify_plain(st):
    """Drafted token d at a row is kept while u q(d) < p(d); at the first that
    is not, the token is drawn from max(0, p - q), after the last from p: the
    first index at which the running sum passes u times the whole."""
    p, q, u, row0 = st["p"], st["q"], st["u"].double(), st["row0"].long()
    B, T = row0.numel() - 1, p.shape[0]
    n = row0[1:] - row0[:-1] - 1
    j = torch.arange(int(st["case"]["drafts"]) + 1, device="cuda")
    row = row0[:-1, None] + j                                   # the target's rows, [B, drafts + 1]
    drow = (row - torch.arange(B, device="cuda")[:, None]).clamp(max=max(0, q.shape[0] - 1))
    d = st["draft"].long()[drow] if q.shape[0] else torch.zeros_like(drow)
    r = row.clamp(max=T - 1)
    keep = u[r] * (q[drow, d].double() if q.shape[0] else 0.0) < p[r, d].double()
    keep &= j < n[:, None]
    a = keep.long().cumprod(1).sum(1)                           # how many are kept
    at = row0[:-1] + a
    w = p[at].double()
    if q.shape[0]:
        less = q[(at - torch.arange(B, device="cuda")).clamp(max=q.shape[0] - 1)].double()
        rest = (w - less).clamp(min=0)
        w = torch.where(((a < n) & (rest.sum(1) > 0))[:, None], rest, w)
    c = w.cumsum(1)
    new = (c <= u[at, None] * c[:, -1:]).sum(1)
    tokens = torch.full((T + 1,), -1, device="cuda", dtype=torch.int32)
    tokens[torch.where(keep.long().cumprod(1) > 0, row, T)] = d.int()
    tokens[at] = new.int()
    return tokens[:T], a.int()


# -------------------------------------------------------------- in 64 bits --

def exact(case, seed):
    st = prepare(case, seed)
    return {"cache": _exact_cache, "attend": _exact_attend, "verify": _exact_verify}[case["op"]](st)


def _e4m3(x):
    """The nearest of e4m3's values to float64 x, |x| <= 448, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _exact_rows(x):
    """What a cache row stands for, by its definition."""
    x = x.double()
    need = (x.abs().amax(-1, keepdim=True) / 448).clamp(min=2.0 ** -64)
    s = torch.exp2(torch.ceil(torch.log2(need)))
    return _e4m3(x / s) * s


def _exact_cache(st):
    held = {}
    for name, new, old in (("k", st["k"], st["old"][1]), ("v", st["v"], st["old"][2])):
        vals = torch.cat([_exact_rows(new), _exact_rows(old)])
        where = {int(s): i for i, s in enumerate(st["slots"].tolist()) if s >= 0}
        where.update({int(s): i + new.shape[0] for i, s in enumerate(st["old"][0].tolist())})
        held[name] = vals[[where[int(s)] for s in st["back"].tolist()]]
    return held["k"], held["v"]


def _exact_attend(st):
    c, h = st["case"], {k: v.tolist() for k, v in st["host"].items()}
    q = st["q"].double()
    H, per, page = c["heads"], c["heads"] // c["kv_heads"], c["page"]
    out = torch.zeros(q.shape, device="cuda", dtype=torch.float64)
    lse = torch.full(q.shape[:2], -torch.inf, device="cuda", dtype=torch.float64)

    def tokens(pages, n, part):
        at = torch.tensor([pages[i // page] * page + i % page for i in range(n)], device="cuda", dtype=torch.long)
        x = st["plain"][part]["e"][at].view(torch.float8_e4m3fn).double() * st["plain"][part]["s"][at][..., None].double()
        return x.transpose(0, 1)  # [kv, n, dim]
    pre = [[tokens(h["prefix_pages"][h["prefix_page0"][g]:h["prefix_page0"][g + 1]], h["prefix_len"][g], x)
            for x in "kv"] for g in range(len(h["prefix_len"]))]
    t = 0
    for b in range(c["seqs"]):
        mine = h["pages"][h["page0"][b]:h["page0"][b + 1]]
        if h["q_len"][b] == 0:
            continue
        k, v = (tokens(mine, h["kv_len"][b], x) for x in "kv")
        P = 0
        if h["group"][b] >= 0:
            pk, pv = pre[h["group"][b]]
            P = pk.shape[1]
            k, v = torch.cat([pk, k], 1), torch.cat([pv, v], 1)
        for j in range(h["q_len"][b]):
            n = P + max(0, h["kv_len"][b] - h["q_len"][b] + j + 1)
            if n:
                x = q[t].view(H // per, per, -1)
                s = torch.matmul(x, k[:, :n].transpose(1, 2).contiguous()) * st["scale"]
                lse[t] = torch.logsumexp(s, -1).flatten()
                out[t] = torch.matmul(torch.softmax(s, -1), v[:, :n].contiguous()).flatten(0, 1)
            t += 1
    return out, lse


def _exact_verify(st):
    row0, draft, u = st["row0"].tolist(), st["draft"].tolist(), st["u"].double().tolist()
    tokens, kept = [-1] * row0[-1], []
    for b in range(len(row0) - 1):
        at, a, n = row0[b], 0, row0[b + 1] - row0[b] - 1
        while a < n:
            d = draft[at + a - b]
            if not u[at + a] * float(st["q"][at + a - b, d]) < float(st["p"][at + a, d]):
                break
            tokens[at + a] = d
            a += 1
        w = st["p"][at + a].double().cpu().numpy()
        if a < n:
            rest = np.maximum(w - st["q"][at + a - b].double().cpu().numpy(), 0.0)
            w = rest if rest.sum() > 0 else w
        c = np.cumsum(w)
        tokens[at + a] = int(np.searchsorted(c, u[at + a] * c[-1], side="right"))
        kept.append(a)
    return (torch.tensor(tokens, dtype=torch.int32), torch.tensor(kept, dtype=torch.int32))
