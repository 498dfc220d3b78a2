"""Plain 64-bit forms of the turned keys and queries, of which new tokens a
drafted tree's token sees, of log probabilities and of the walk down a drafted
tree, written from their definitions (include/lora.h), on the CPU.  Shares no
code with the library."""
import math

import numpy as np


def pair_of(i, n, pairs):
    """The two elements of pair i of n."""
    return (2 * i, 2 * i + 1) if pairs else (i, i + n)


def turned(x, positions, freq, axis, pairs, scale=1.0):
    """x [T, heads, dim] float64, positions [axes, T]; also the sum of the
    magnitudes that each element is made of."""
    y, mass, n = x.copy(), np.abs(x), len(freq)
    for i in range(n):
        a, b = pair_of(i, n, pairs)
        angle = positions[axis[i]].astype(np.float64) * freq[i]
        c, s = (np.cos(angle) * scale)[:, None], (np.sin(angle) * scale)[:, None]
        with np.errstate(invalid="ignore"):
            y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
            y[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
        mass[:, :, a] = np.abs(x[:, :, a] * c) + np.abs(x[:, :, b] * s)
        mass[:, :, b] = np.abs(x[:, :, b] * c) + np.abs(x[:, :, a] * s)
    return y, mass


def sees(parent, j):
    """The nodes that node j of a tree sees: itself and those above it."""
    out = []
    while j >= 0:
        out.append(j)
        j = parent[j]
    return sorted(out)


def logprobs(z, token, scale, k):
    """One row of logits, float64: log probability of `token` (NaN outside the
    vocabulary), entropy, the k likeliest and their log probabilities.  A row
    that holds NaN or +inf, or nothing above -inf, is no distribution."""
    if np.isnan(z).any() or not math.isfinite(z.max()):
        return math.nan, math.nan, [-1] * k, [math.nan] * k
    y = (z - z.max()) * scale  # before the sum: far from 0 a logarithm would be lost beside the logit
    e = np.exp(y)
    lp = y - math.log(math.fsum(e))
    some = e > 0
    entropy = -math.fsum(np.exp(lp[some]) * lp[some])
    ids = np.argsort(-z, kind="stable")[:k].tolist()  # the lower index first among equals
    return (lp[token] if 0 <= token < len(z) else math.nan), entropy, ids, [lp[i] for i in ids]


def draw(w, u):
    """The first index with weight at which the running sum passes u times the
    whole (the last with weight, if rounding keeps it below); None: no weight,
    or no finite sum."""
    w = np.where(w > 0, w, 0.0)
    total = math.fsum(w) if np.isfinite(w).all() else math.inf
    if not 0 < total < math.inf:
        return None
    c = np.cumsum(w)
    passed = np.nonzero((c > float(u) * c[-1]) & (w > 0))[0]
    return int(passed[0]) if len(passed) else int(np.nonzero(w > 0)[0][-1])


def verify_tree(p, draft, parent, row0, u):
    """p [rows, V] float64.  Returns tokens, path, accepted."""
    tokens, path, accepted = [-1] * len(p), [-1] * len(p), []
    for b in range(len(row0) - 1):
        r0, n = row0[b], row0[b + 1] - row0[b]
        out, nodes, node = [], [], 0
        while node is not None:
            token = draw(p[r0 + node], u[r0 + node])
            if token is None:
                out = None
                break
            out.append(token)
            nodes.append(node)
            node = next((j for j in range(node + 1, n) if parent[r0 + j] == node and draft[r0 + j] == token), None)
        if out is None:
            accepted.append(-1)
            continue
        tokens[r0:r0 + len(out)], path[r0:r0 + len(out)] = out, nodes
        accepted.append(len(out) - 1)
    return tokens, path, accepted
