"""Plain 64-bit forms of the group-rollout operators, written from their
definitions, for the GPU tests."""

import math

import numpy as np
import torch


def page_tables(lens, new, free, page, table, n_slots):
    """numpy in, (table, slots, cu, used) out; every length valid."""
    table = table.copy()
    used, slots, cu = 0, [], [0]
    for i, (n, a) in enumerate(zip(lens.tolist(), new.tolist())):
        for j in range(-(-n // page), -(-(n + a) // page)):
            if j < table.shape[1]:
                table[i, j] = free[used] if used < len(free) else -1
                used += 1
        for pos in range(n, n + a):
            j = pos // page
            pg = table[i, j] if j < table.shape[1] else -1
            slots.append(int(pg) * page + pos % page if pg >= 0 else -1)
        cu.append(cu[-1] + a)
    slots = (slots + [-1] * n_slots)[:n_slots]
    return table, np.array(slots, np.int64), np.array(cu, np.int64), used


def attention(q, k, v, scale):
    """q [D], k, v [n, D] in float64 -> out, lse, sum p |v|, bound on a score's error."""
    if len(k) == 0:
        return torch.zeros_like(q), -math.inf, torch.zeros_like(q), 0.0
    s = (k @ q) * scale
    lse = torch.logsumexp(s, 0)
    p = torch.exp(s - lse)
    # D products and sums in fp32, the scale and the exponent's rounding
    delta = (q.numel() + 4) * 2.0 ** -24 * float(((k.abs() @ q.abs()) * abs(scale)).max())
    return p @ v, float(lse), p @ v.abs(), delta


def filter_row(z, tau, k, p, min_p, u):
    """One row (float64 numpy): (token, log mu, kept indices in index order)."""
    V = len(z)
    if tau == 0:
        tau, k = 1.0, 1
    order = np.argsort(-z, kind="stable")
    x = (z[order] - z[order[0]]) / tau
    w = np.exp(x)
    n = min(k if k > 0 else V, V, int((x > -np.inf).sum()))
    if p < 1:
        head = w[:n]
        before = np.concatenate([[0.0], np.cumsum(head)[:-1]])
        n = max(1, int((before < p * head.sum()).sum()))
    if min_p > 0:
        n = min(n, int((x >= math.log(min_p)).sum()))
    kept = np.sort(order[:n])
    mine = np.exp((z[kept] - z[order[0]]) / tau)
    cum = np.cumsum(mine)
    # u = 0: the first kept token, whose probability is positive even where
    # float64 has it as 0
    token = kept[int((cum <= u * cum[-1]).sum()) if u > 0 else 0]
    return int(token), (z[token] - z[order[0]]) / tau - math.log(cum[-1]), kept


def pack(kept_rows, V):
    """[T] index arrays -> [T, ceil(V/32)] int32 words."""
    bits = np.zeros((len(kept_rows), (V + 31) // 32 * 32), np.uint8)
    for r, kept in enumerate(kept_rows):
        bits[r, kept] = 1
    return np.packbits(bits, axis=1, bitorder="little").view(np.int32).reshape(len(kept_rows), -1)


def keep_logprob(z, tau, token, kept, g):
    """One row (float64 torch): (log p, lse, dz)."""
    x = torch.where(kept, z / tau, -math.inf)
    lse = torch.logsumexp(x, 0)
    p = torch.exp(x - lse)
    one = torch.zeros_like(z)
    one[token] = 1
    return float(x[token] - lse), float(lse), (g / tau) * (one - p)
