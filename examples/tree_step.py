"""Serving steps whose drafted tokens form a tree, on random weights: several
tenants, each with an adapter on every projection and a system prompt that all
of its sequences share.

    python examples/tree_step.py [--steps 8]

One step runs, for the last accepted token of every sequence and the tree of
drafts below it,
    per layer:  lora_apply_routed (q, k and v in one product), lora_kv_append
                (keys turned by their depth's position as they are written, the
                queries in place), lora_attend over the tenant's prefix, the
                sequence's own tokens and each node's ancestors,
                lora_apply_routed (o)
    at the end: the head (base only), softmax, lora_verify_tree, lora_logprobs
                of the tokens that came out; the kept path's keys and values
                move to the front (lora_kv_read, lora_kv_write).
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from draft_step import Server as DraftServer, i32, lora  # noqa: E402

# The tree of drafts: of each node the one it follows, and which of its
# parent's likeliest next tokens it holds.
PARENT = [-1, 0, 0, 1, 1, 2, 3]
CHOICE = [0, 0, 1, 0, 1, 0, 0]


def depths(parent):
    d = []
    for p in parent:
        d.append(0 if p < 0 else d[p] + 1)
    return d


class Server(DraftServer):
    """The model of draft_step.py with positions, and trees in place of chains."""

    def __init__(self, **args):
        self.positions = None  # of the step's tokens
        self.parent = None     # the step's trees; None: chains
        dim, prompt, room = args.get("dim", 64), args.get("prompt", 150), args.get("room", 128)
        n = dim // 2
        self.rope = lora.lora_rope_create(prompt + room + 64, 10000.0 ** (-torch.arange(n, dtype=torch.float64) / n))
        super().__init__(drafts=len(PARENT) - 1, **args)
        self.scorer = lora.lora_scorer_create(self.max_tokens)

    def forward(self, tokens, tenant, slots, batch):
        """Logits [tokens, vocab] after each of the step's tokens."""
        T = len(tokens)
        positions = list(range(T)) if self.positions is None else self.positions  # none: a prompt from its start
        slots, positions = i32(slots, "cuda"), i32(positions, "cuda")
        lora.lora_plan_route(self.routing, self.layers[0][0].pool, i32(tenant, "cuda"), T)
        if self.parent is None:
            lora.lora_attend_plan_set(self.attention, self.caches[0], **batch)
        else:
            lora.lora_attend_plan_set_tree(self.attention, self.caches[0], i32(self.parent), **batch)
        h, kv, d = self.heads, self.kv_heads, self.dim
        x = self.embed[torch.tensor(tokens, device="cuda")]
        for (qkv, out), cache in zip(self.layers, self.caches):
            y = qkv(torch.nn.functional.rms_norm(x, (self.hidden,)), self.routing).unflatten(1, (h + 2 * kv, d))
            q = y[:, :h]
            lora.lora_kv_append(cache, self.rope, y[:, h:h + kv], y[:, h + kv:], slots, positions, T, q=q, q_out=q)
            a = torch.empty((T, h, d), dtype=self.dtype, device="cuda")
            lora.lora_attend(cache, self.attention, q, d ** -0.5, a)
            x = x + out(a.flatten(1), self.routing)
        base = torch.full((T,), lora.LORA_BASE_ONLY, dtype=torch.int32, device="cuda")
        lora.lora_plan_route(self.head_routing, self.head.pool, base, T)
        return self.head(torch.nn.functional.rms_norm(x, (self.hidden,)), self.head_routing)

    def logits(self, tokens, parents=None):
        """Of each sequence's new tokens (the last accepted one first), whose
        trees `parents` are (None: chains); their keys and values are in the
        cache afterwards, in the tokens' order."""
        new = [len(x) for x in tokens]
        trees = [list(range(-1, n - 1)) for n in new] if parents is None else parents
        self.parent = None if parents is None else [p for t in trees for p in t]
        self.positions = [self.prompt_len[t] + n + d for t, n, tree in zip(self.tenant, self.kv_len, trees)
                          for d in depths(tree)]
        slots = [s for i, n in enumerate(new) for s in self.slots(self.pages[i], self.kv_len[i], n)]
        tenant = [t for t, n in zip(self.tenant, new) for _ in range(n)]
        return self.forward([t for x in tokens for t in x], tenant, slots, self.batch(new))

    def draft(self):
        """The nodes' tokens, a sequence: each its parent's likeliest ones by the draft."""
        best = torch.topk(self.bigram, max(CHOICE) + 1, 1).indices.tolist()
        trees = []
        for last in self.last:
            tree = [last]
            for p, c in zip(PARENT[1:], CHOICE[1:]):
                tree.append(best[tree[p]][c])
            trees.append(tree)
        return trees

    def keep(self, paths):
        """Moves the keys and values of each sequence's path to its front."""
        moves = [(a, b) for s, path in enumerate(paths)
                 for a, b in zip([self.slots(self.pages[s], self.kv_len[s], max(path) + 1)[n] for n in path],
                                 self.slots(self.pages[s], self.kv_len[s], len(path))) if a != b]
        if moves:
            old, new = (i32(list(x), "cuda") for x in zip(*moves))
            k = torch.empty((len(moves), self.kv_heads, self.dim), dtype=self.dtype, device="cuda")
            v = torch.empty_like(k)
            for cache in self.caches:
                lora.lora_kv_read(cache, old, len(moves), k, v)
                lora.lora_kv_write(cache, k, v, new, len(moves))

    def step(self, u=None):
        """Draft, run the target once, walk down; returns the tokens kept a
        sequence, and their log probabilities."""
        trees = self.draft()
        S, n = len(trees), len(PARENT)
        z = self.logits(trees, [PARENT] * S)
        tokens, path, accepted = (torch.empty(m, dtype=torch.int32, device="cuda") for m in (S * n, S * n, S))
        u = torch.rand(S * n, device="cuda") if u is None else u
        lora.lora_verify_tree(self.verifier, torch.softmax(z.float(), -1), i32([t for x in trees for t in x], "cuda"),
                              i32(PARENT * S, "cuda"), i32([s * n for s in range(S + 1)], "cuda"), u, S, S * n, tokens,
                              path, accepted)
        # The rows that the tokens were drawn from, row by row of the answer.
        rows = torch.arange(S, device="cuda").repeat_interleave(n) * n + path.clamp(min=0)
        logprob, entropy = torch.empty(S * n, device="cuda"), torch.empty(S * n, device="cuda")
        top = torch.empty((S * n, 3), dtype=torch.int32, device="cuda"), torch.empty((S * n, 3), device="cuda")
        lora.lora_logprobs(self.scorer, z[rows], tokens, 1.0, logprob, entropy, *top)
        tokens, path, logprob = (x.view(S, n).tolist() for x in (tokens, path, logprob))
        kept, scores, paths = [], [], []
        for s, k in enumerate(accepted.tolist()):
            if k < 0:
                raise RuntimeError("sequence %d: nothing to draw from" % s)
            paths.append(path[s][:k + 1])
            kept.append(tokens[s][:k + 1])
            scores.append(logprob[s][:k + 1])
        self.keep(paths)
        for s, t in enumerate(kept):
            self.kv_len[s] += len(t)
            self.last[s] = t[-1]
        return kept, scores

    def full(self):
        return max(self.kv_len) + len(PARENT) > self.room

    def close(self):
        super().close()
        lora.lora_rope_destroy(self.rope)
        lora.lora_scorer_destroy(self.scorer)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=8)
    args = ap.parse_args()
    torch.manual_seed(0)
    server = Server()
    for i in range(args.steps):
        if server.full():
            break
        kept, scores = server.step()
        print("step %d: %d tokens for %d sequences, mean log probability %.3f"
              % (i, sum(len(k) for k in kept), len(kept), sum(map(sum, scores)) / sum(map(len, scores))), flush=True)
    server.close()


if __name__ == "__main__":
    main()
