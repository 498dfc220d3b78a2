"""Plain 64-bit forms of the quantised cache, the attention over it and the
draft verification, written from their definitions (include/lora.h), on the
CPU, a token at a time.  Shares no code with the library."""
import math

import numpy as np
import torch


def e4m3(x):
    """Nearest e4m3 value to float64 x (|x| <= 448), ties to even."""
    mag = np.abs(x)
    _, e = np.frexp(np.maximum(mag, 2.0 ** -6))
    step = np.exp2(e - 4.0)
    return np.round(x / step) * step  # numpy rounds halves to even


def held(x):
    """x [..., dim] float64: what the cache holds for these rows (NaN rows where
    a value is not finite; poisoning by the partner row is the caller's)."""
    amax = np.max(np.where(np.isfinite(x), np.abs(x), 0.0), axis=-1, keepdims=True)
    s = np.full(amax.shape, -64.0)
    some = amax > 0
    s[some] = np.maximum(-64.0, np.ceil(np.log2(amax[some] / 448.0)))
    # log2 rounds: settle the border itself.
    s = np.where((amax > 448.0 * np.exp2(s)), s + 1, s)
    s = np.where((s > -64) & (amax <= 448.0 * np.exp2(s - 1)), s - 1, s)
    ok = np.isfinite(x).all(-1, keepdims=True)
    out = e4m3(np.where(ok, x, 0.0) / np.exp2(s)) * np.exp2(s)
    return np.where(ok, out, np.nan)


def held_pair(k, v):
    """Keys and values as held: a row that is not finite poisons its partner."""
    k, v = held(k), held(v)
    bad = np.isnan(k).any(-1, keepdims=True) | np.isnan(v).any(-1, keepdims=True)
    return np.where(bad, np.nan, k), np.where(bad, np.nan, v)


def rounded(x, dtype):
    """float64 numpy to dtype, rounded once (torch rounds float64 through
    float32 for none of these types' values: the held values have 4 bits)."""
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype)


def attend(q, rows, scale):
    """q [H, D]; rows: (k, v) float64 [n, kv_heads, D] of the keys the token
    sees.  Returns out [H, D], lse [H] and what the tolerance needs: the
    weights' sum of |v|, the largest weight times |v|, the scores' error scale."""
    H, D = q.shape
    k, v = rows
    n, kv, _ = k.shape
    if n == 0:
        z = np.zeros((H, D))
        return z, np.full(H, -np.inf), z, np.zeros(H), np.zeros(H)
    per = H // kv
    kh, vh = np.repeat(k.transpose(1, 0, 2), per, 0), np.repeat(v.transpose(1, 0, 2), per, 0)  # [H, n, D]
    s = np.einsum("hd,hnd->hn", q, kh) * scale
    mass = np.max(np.einsum("hd,hnd->hn", np.abs(q), np.abs(kh)), -1) * abs(scale)
    m = s.max(-1, keepdims=True)
    p = np.exp(s - m)
    total = p.sum(-1, keepdims=True)
    p = p / total
    out = np.einsum("hn,hnd->hd", p, vh)
    absv = np.einsum("hn,hnd->hd", p, np.abs(vh))
    top = np.max(p * np.abs(vh).max(-1), -1)
    return out, (m + np.log(total))[:, 0], absv, top, mass


def attend_tolerance(ref, absv, top, mass, n, dim, dtype):
    """Bounds of |out - ref| [H, D] and |lse - ref| [H].

    A score is a sum of dim exact products in fp32: off by (dim + 3) 2^-24 of
    the sum of their magnitudes, and by 2^-22 of itself for the change of base
    and the subtraction (the exponents added are below 2^7).  Weights move by
    twice that (numerator and sum), are rounded to fp16 (half a step, 2^-11;
    below fp16's normal range half of 2^-24, against a largest weight of at
    least 1, times elements up to 448 that stand for up to twice the row's
    largest), and the output is rounded once."""
    ds = (dim + 3) * 2.0 ** -24 * mass + 2.0 ** -22 * (mass + 128.0)
    half = torch.finfo(dtype).eps / 2
    sub = torch.finfo(dtype).tiny * half * 2  # below the type's normal range steps are absolute
    out = (half * np.abs(ref) + sub + (2.0 ** -11 + 2 * ds[:, None] + 2.0 ** -20) * absv
           + (2.0 ** -24 * n * top)[:, None])
    return out, ds + 2.0 ** -20


def verify(p, q, draft, row0, u):
    """p [rows, V], q [rows - seqs, V] float64.  Returns tokens, accepted."""
    V = p.shape[1]
    tokens, accepted = [-1] * len(p), []
    for b in range(len(row0) - 1):
        r0, n, k = row0[b], row0[b + 1] - row0[b] - 1, 0
        ds = [int(draft[r0 - b + i]) for i in range(n)]
        if any(d < 0 or d >= V for d in ds):
            accepted.append(-1)
            continue
        while k < n and float(u[r0 + k]) * q[r0 - b + k, ds[k]] < p[r0 + k, ds[k]]:
            k += 1
        w = np.where(p[r0 + k] > 0, p[r0 + k], 0.0)
        if k < n:
            with np.errstate(invalid="ignore"):
                rest = p[r0 + k] - q[r0 - b + k]
            rest = np.where(rest > 0, rest, 0.0)
            if rest.sum() > 0:
                w = rest
        total = math.fsum(w) if np.isfinite(w).all() else math.inf
        if not (0 < total < math.inf):
            accepted.append(-1)
            continue
        c = np.cumsum(w)
        passed = np.nonzero((c > float(u[r0 + k]) * c[-1]) & (w > 0))[0]
        token = int(passed[0]) if len(passed) else int(np.nonzero(w > 0)[0][-1])
        tokens[r0:r0 + k + 1] = ds[:k] + [token]
        accepted.append(k)
    return tokens, accepted
