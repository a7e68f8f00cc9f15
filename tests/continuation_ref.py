"""64-bit plain implementations of the norm, of attention over drafted trees and of beam search, on the CPU, and the
error bounds that the tests hold the kernels to (roundings counted as in decode_ref)."""
import numpy as np
import torch

import decode_ref as ref
from decode_ref import U32

HALF_STEP = {torch.float32: U32, torch.bfloat16: ref.UBF16}

# The sum of a row's squares: a lane adds at most 32 values in a row, then 5 halvings and at most 32 warps.  All terms
# have one sign, so each rounding costs at most U32 of the sum; the root halves that, and four roundings follow.
NORM = (32 + 5 + 32) / 2 * U32 + 5 * U32


def norm(s, weight, eps):
    """s [rows, cols] fp64 (what is normalised), weight [cols] or None -> y in fp64."""
    r = 1.0 / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    return s * r * (1.0 if weight is None else weight)


def norm_grad(s, weight, dy, dsum, eps):
    """-> dx, dweight, and bounds on their errors before dx is rounded."""
    rows, cols = s.shape
    w = np.ones(cols) if weight is None else weight
    r = 1.0 / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    u, g = s * r, dy * w
    dot = (g * u).mean(-1, keepdims=True)
    add = 0.0 if dsum is None else dsum
    dx = r * (g - u * dot) + add
    # the dot product: as many roundings as the squares, of terms of both signs; u and r as the norm's
    e_dot = (2 * NORM + (32 + 5 + 32) * U32) * np.abs(g * u).mean(-1, keepdims=True)
    e_dx = r * ((NORM + 4 * U32) * (np.abs(g) + 2 * np.abs(u * dot)) + np.abs(u) * e_dot) + 2 * U32 * np.abs(add)
    size = np.abs(dy * u).sum(0)
    # a block adds its rows in a row, the blocks' sums are added by 32 warps: never more roundings than rows and 64
    return dx, (dy * u).sum(0), e_dx + 1e-38, (NORM + U32 * (rows + 64)) * size + 1e-38


def seen_by(mask, draft, ctx, window, i):
    """The cached positions that drafted token i of a sequence sees, in order (ctx may be below 0: then the first
    drafted tokens have no place)."""
    path = [j for j in range(draft) if (j <= i if mask is None else mask >> j & 1) and ctx + j >= 0]
    if window:
        path = path[-window:] if len(path) > window else path
        first = max(0, ctx - (window - len(path)))
    else:
        first = 0
    return list(range(first, max(ctx, 0))) + [ctx + j for j in path]


def tree_row(q, k, v, keys, scale):
    """One row and head: q [D], k, v [n, D] fp64 -> as decode_ref.attention over the keys it sees."""
    return ref.attention(q, k[keys], v[keys], scale)


def beam_totals(x, scores):
    """x [seqs * beams, V] fp64, scores [seqs, beams] fp64 -> totals [seqs, beams * V] (-inf: no candidate)."""
    B, W = scores.shape
    with np.errstate(all="ignore"):
        m = x.max(-1, keepdims=True)
        lp = x - m - np.log(np.exp(x - m).sum(-1, keepdims=True))
        lp = np.where(np.isnan(lp), -np.inf, lp)
        lp[np.isnan(x).any(-1) | (m[:, 0] == np.inf)] = -np.inf
        t = lp.reshape(B, W, -1) + scores[:, :, None]
    return np.where(np.isnan(t), -np.inf, t).reshape(B, -1)


def beam_best(totals, n):
    """-> (flat indices [n] or fewer, in order) of one sequence: larger totals first, then lower indices."""
    order = np.lexsort((np.arange(len(totals)), -totals))[:n]
    return [int(i) for i in order if totals[i] > -np.inf]


def beam_eps(V, total):
    """The sum of a row's exponentials as decode_ref has it, and the total's one rounding to fp32."""
    return ref.logprob_eps(V) + U32 * np.abs(total)


def reorder(table, parents, seq_len, page, W):
    """Page tables after a selection: lists -> (new table, copies [(from page, to page, rows)])."""
    new, copies = [list(r) for r in table], []
    for b, n in enumerate(seq_len):
        full, rest = divmod(n, page)
        spare = [w for w in range(W) if w not in parents[b]]
        seen = set()
        for w, p in enumerate(parents[b]):
            p = p if 0 <= p < W else -1
            row = b * W + w
            if p >= 0:
                new[row][:full] = table[b * W + p][:full]
            if p >= 0 and p not in seen:
                home = p
            else:
                home = spare.pop(0)
            seen.add(p)
            if rest:
                new[row][full] = table[b * W + home][full]
                if p >= 0 and home != p:
                    copies.append((table[b * W + p][full], table[b * W + home][full], rest))
    return new, copies
