"""Serving steps with drafted tokens, on random weights: several tenants, each
with an adapter on every projection and a system prompt that all of its
sequences share.

    python examples/draft_step.py [--steps 8] [--drafts 3]

One step runs, for the last accepted and the drafted tokens of every sequence,
    per layer:  lora_apply_routed (q, k and v in one product), lora_kv_write
                of its key and value parts, lora_attend over the tenant's
                prefix and the sequence's own tokens, lora_apply_routed (o)
    at the end: the head (base only), softmax, lora_verify.
The routing plan and the attention plan are made once a step and used by every
layer.  The prompt of a tenant is prefilled once, with the same calls.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from rank_adapter_gemm_token_amd import lora  # noqa: E402


def i32(x, device="cpu"):
    return torch.tensor(x, dtype=torch.int32, device=device)


class Projection:
    """A base weight with its pool of adapters."""

    def __init__(self, d_in, d_out, tenants, rank, max_tokens, dtype, g):
        def rand(*shape, scale):
            return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()
        self.W = rand(d_out, d_in, scale=d_in ** -0.5)
        self.d_out = d_out
        self.pool = lora.lora_pool_create(d_in, d_out, rank, max(1, tenants), max_tokens, dtype)
        for t in range(tenants):
            lora.lora_set_tenant_quota(self.pool, t, 1 << 40)
            lora.lora_register(self.pool, t, t, rand(rank, d_in, scale=d_in ** -0.5), rand(d_out, rank, scale=0.1),
                               rank, 2.0 * rank)

    def __call__(self, x, plan):
        y = torch.empty((x.shape[0], self.d_out), dtype=x.dtype, device="cuda")
        lora.lora_apply_routed(self.pool, plan, x, self.W, y)
        return y

    def close(self):
        lora.lora_pool_destroy(self.pool)


class Server:
    """The model, its caches and its sequences."""

    def __init__(self, tenants=3, seqs=12, layers=2, heads=8, kv_heads=2, dim=64, vocab=1024, prompt=150, room=128,
                 drafts=3, page=16, dtype=torch.bfloat16, seed=0):
        self.g = torch.Generator().manual_seed(seed)
        self.heads, self.kv_heads, self.dim, self.vocab, self.page, self.dtype = heads, kv_heads, dim, vocab, page, dtype
        self.hidden, self.drafts = heads * dim, drafts
        self.max_tokens = max(prompt, seqs * (drafts + 1))
        args = dict(tenants=tenants, rank=16, max_tokens=self.max_tokens, dtype=dtype, g=self.g)
        self.layers = [(Projection(self.hidden, (heads + 2 * kv_heads) * dim, **args),
                        Projection(self.hidden, self.hidden, **args)) for _ in range(layers)]
        self.embed = torch.randn((vocab, self.hidden), generator=self.g).to(dtype).cuda()
        self.head = Projection(self.hidden, vocab, 0, 16, self.max_tokens, dtype, self.g)
        # The draft: a table of next-token probabilities.
        self.bigram = torch.softmax(1.5 * torch.randn((vocab, vocab), generator=self.g), -1).cuda()

        prompt_pages, own_pages = -(-prompt // page), -(-room // page)
        n_pages = tenants * prompt_pages + seqs * own_pages
        table = torch.randperm(n_pages, generator=self.g).tolist()
        self.prompt_len = [prompt - 7 * t for t in range(tenants)]
        self.prompt_pages = [[table.pop() for _ in range(prompt_pages)] for _ in range(tenants)]
        self.tenant = [s % tenants for s in range(seqs)]
        self.pages = [[table.pop() for _ in range(own_pages)] for _ in range(seqs)]
        self.kv_len = [0] * seqs                     # own tokens held
        self.last = torch.randint(vocab, (seqs,), generator=self.g).tolist()  # accepted, not yet held
        self.room = own_pages * page

        self.caches = [lora.lora_kv_create(n_pages, page, kv_heads, dim, dtype) for _ in range(layers)]
        self.routing = lora.lora_plan_create(self.max_tokens, tenants)
        self.head_routing = lora.lora_plan_create(self.max_tokens, 1)
        self.attention = lora.lora_attend_plan_create(seqs, tenants, self.max_tokens, n_pages, heads, kv_heads, dim)
        self.verifier = lora.lora_verifier_create(seqs)
        for t in range(tenants):
            self.prefill(t)

    def slots(self, pages, first, n):
        return [pages[i // self.page] * self.page + i % self.page for i in range(first, first + n)]

    def forward(self, tokens, tenant, slots, batch):
        """Probabilities [tokens, vocab] after each of the step's tokens."""
        T = len(tokens)
        slots = i32(slots, "cuda")
        lora.lora_plan_route(self.routing, self.layers[0][0].pool, i32(tenant, "cuda"), T)
        lora.lora_attend_plan_set(self.attention, self.caches[0], **batch)
        h, kv, d = self.heads, self.kv_heads, self.dim
        x = self.embed[torch.tensor(tokens, device="cuda")]
        for (qkv, out), cache in zip(self.layers, self.caches):
            y = qkv(torch.nn.functional.rms_norm(x, (self.hidden,)), self.routing).unflatten(1, (h + 2 * kv, d))
            lora.lora_kv_write(cache, y[:, h:h + kv], y[:, h + kv:], slots, T)
            a = torch.empty((T, h, d), dtype=self.dtype, device="cuda")
            lora.lora_attend(cache, self.attention, y[:, :h], d ** -0.5, a)
            x = x + out(a.flatten(1), self.routing)
        base = torch.full((T,), lora.LORA_BASE_ONLY, dtype=torch.int32, device="cuda")
        lora.lora_plan_route(self.head_routing, self.head.pool, base, T)
        z = self.head(torch.nn.functional.rms_norm(x, (self.hidden,)), self.head_routing)
        return torch.softmax(z.float(), -1)

    def prefill(self, t):
        """A tenant's prompt: one sequence of new tokens only, into the pages
        that its sequences will name as their prefix."""
        n = self.prompt_len[t]
        tokens = torch.randint(self.vocab, (n,), generator=self.g).tolist()
        self.forward(tokens, [t] * n, self.slots(self.prompt_pages[t], 0, n),
                     dict(q_len=i32([n]), kv_len=i32([n]), group=i32([-1]), pages=i32(self.prompt_pages[t]),
                          page0=i32([0, len(self.prompt_pages[t])])))

    def batch(self, new):
        def flat(lists):
            first = [0]
            for x in lists:
                first.append(first[-1] + len(x))
            return i32([v for x in lists for v in x]), i32(first)
        pages, page0 = flat(self.pages)
        prefix_pages, prefix_page0 = flat(self.prompt_pages)
        return dict(q_len=i32(new), kv_len=i32([c + n for c, n in zip(self.kv_len, new)]), group=i32(self.tenant),
                    pages=pages, page0=page0, prefix_len=i32(self.prompt_len), prefix_pages=prefix_pages,
                    prefix_page0=prefix_page0)

    def draft(self):
        """Drafted tokens a sequence, and their distributions [drafts of all, vocab]."""
        at = torch.tensor(self.last, device="cuda")
        tokens, q = [], []
        for _ in range(self.drafts):
            q.append(self.bigram[at])
            at = torch.multinomial(q[-1], 1)[:, 0]
            tokens.append(at)
        return torch.stack(tokens, 1).tolist(), torch.stack(q, 1).flatten(0, 1).contiguous()

    def probabilities(self, tokens):
        """Of each sequence's new tokens (the last accepted one first); their
        keys and values are in the cache afterwards."""
        new = [len(x) for x in tokens]
        slots = [s for i, n in enumerate(new) for s in self.slots(self.pages[i], self.kv_len[i], n)]
        tenant = [t for t, n in zip(self.tenant, new) for _ in range(n)]
        return self.forward([t for x in tokens for t in x], tenant, slots, self.batch(new))

    def step(self):
        """Draft, run the target once, verify; returns the tokens kept a sequence."""
        drafted, q = self.draft()
        p = self.probabilities([[last] + d for last, d in zip(self.last, drafted)])
        S, n = len(self.last), self.drafts
        row0 = i32([s * (n + 1) for s in range(S + 1)], "cuda")
        tokens = torch.empty(S * (n + 1), dtype=torch.int32, device="cuda")
        accepted = torch.empty(S, dtype=torch.int32, device="cuda")
        lora.lora_verify(self.verifier, p, q, i32([t for d in drafted for t in d], "cuda"), row0,
                         torch.rand(S * (n + 1), device="cuda"), S, S * (n + 1), tokens, accepted)
        tokens, accepted = tokens.view(S, n + 1).tolist(), accepted.tolist()
        kept = []
        for s, k in enumerate(accepted):
            if k < 0:
                raise RuntimeError("sequence %d: nothing to draw from" % s)
            # The keys of refused tokens are past the new length: nobody sees
            # them, and the next step writes over them.
            self.kv_len[s] += k + 1
            self.last[s] = tokens[s][k]
            kept.append(tokens[s][:k + 1])
        return kept

    def full(self):
        return max(self.kv_len) + self.drafts + 1 > self.room

    def close(self):
        for h in self.caches:
            lora.lora_kv_destroy(h)
        lora.lora_plan_destroy(self.routing)
        lora.lora_plan_destroy(self.head_routing)
        lora.lora_attend_plan_destroy(self.attention)
        lora.lora_verifier_destroy(self.verifier)
        for qkv, out in self.layers:
            qkv.close()
            out.close()
        self.head.close()


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--drafts", type=int, default=3)
    args = ap.parse_args()
    torch.manual_seed(0)
    server = Server(drafts=args.drafts)
    for i in range(args.steps):
        if server.full():
            break
        kept = server.step()
        print("step %d: %d tokens for %d sequences" % (i, sum(len(k) for k in kept), len(kept)), flush=True)
    server.close()


if __name__ == "__main__":
    main()
