"""64-bit plain implementations of the decoding step's operators, on the CPU, and
the error bounds that the tests hold the kernels to.

Bounds count roundings: u32 = 2^-24 for fp32, half a step of the output's type
(bf16: 2^-8) relative to the value, and for e4m3 codes 2^-4 relative plus half a
subnormal step.  `sum` terms use the worst case of n roundings in a row.
"""
import math

import numpy as np
import torch

U32, UBF16, UE4M3 = 2.0 ** -24, 2.0 ** -8, 2.0 ** -4


def f64(t):
    return t.detach().cpu().double().numpy()


def e4m3_value(codes, exp):
    """uint8 codes [..., D] and exponent bytes [...] -> fp64 values."""
    c = codes.detach().cpu().contiguous().view(torch.float8_e4m3fn).double().numpy()
    return np.ldexp(c, exp.detach().cpu().numpy().astype(np.int64)[..., None] - 127)


def e4m3_cache(x):
    """fp32 values [..., D] -> (codes, exponent bytes): the smallest exponent with max|x| <= 448 * 2^e."""
    amax = x.abs().amax(-1)
    f, e = torch.frexp(amax)
    e = torch.where(f <= 0.875, e - 9, e - 8)
    e = torch.where(amax == 0, torch.zeros_like(e), e).clamp(min=-126)
    return torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)


# ---------------------------------------------------------------- append

def rotate(x, pos, inv_freq, interleaved):
    """x [T, H, D] fp64, pos [T], inv_freq [R/2] -> (rotated, magnitude of each value's pair)."""
    x, r = x.copy(), 2 * len(inv_freq)
    mag = np.abs(x)
    if r:
        th = np.asarray(pos, np.float64)[:, None, None] * np.asarray(inv_freq, np.float64)
        a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., : r // 2], x[..., r // 2: r])
        u, w, m = a * np.cos(th) - b * np.sin(th), a * np.sin(th) + b * np.cos(th), np.hypot(a, b)
        if interleaved:
            x[..., 0:r:2], x[..., 1:r:2], mag[..., 0:r:2], mag[..., 1:r:2] = u, w, m, m
        else:
            x[..., : r // 2], x[..., r // 2: r], mag[..., : r // 2], mag[..., r // 2: r] = u, w, m, m
    return x, mag


# cos and sin within 2 steps (2^-23 each) of an angle held to 2^-31 of a turn, one product and one fused
# multiply-add: below 2^-20 of the pair's magnitude in all
ROT = 2.0 ** -20


def rotate_bound(want, mag):
    return UBF16 * np.abs(want) + ROT * mag + 1e-38


# ---------------------------------------------------------------- attention

def attention(q, k, v, scale):
    """One head: q [D], k, v [n, D] fp64 -> (out [D], lse, bound on |out error|, bound on |lse error|)."""
    n, D = k.shape
    if n == 0:
        return np.zeros(D), -math.inf, np.zeros(D), 0.0
    s = scale * (k @ q)
    m = s.max()
    p = np.exp(s - m)
    l = p.sum()
    p /= l
    out = p @ v
    # a score: D products summed in fp32 and the product with the scale; in the exponent also the rounding of
    # the score itself and of its difference with the maximum
    ds = float((U32 * (D + 4) * abs(scale) * (np.abs(k) @ np.abs(q)) + 4 * U32 * (np.abs(s) + abs(m))).max())
    # a weight: its exponential (2^-21), its two-part rounding (2^-16); the sums over n keys and their rescaling
    dw = 2 * ds + 2.0 ** -21 + 2.0 ** -16 + 2 * (n + 64) * U32
    eo = UBF16 * np.abs(out) + dw * (np.abs(v).T @ p) + 1e-38
    lse = m + math.log(l)
    return out, lse, eo, dw + 4 * U32 * (abs(lse) + abs(m))


# ---------------------------------------------------------------- log probabilities

def logprobs(x, token, top):
    """x [rows, V] fp64 -> dict as the binding's, fp64 (a row of -inf: lse -inf, entropy 0, logprobs -inf)."""
    rows, V = x.shape
    out = dict(lse=np.empty(rows), entropy=np.empty(rows), logprob=np.zeros(rows),
               top_ids=np.full((rows, top), -1, np.int64), top_logprobs=np.full((rows, top), -np.inf))
    with np.errstate(all="ignore"):
        for r in range(rows):
            m = x[r].max()
            if m == -np.inf:
                lse, H, log_l = -np.inf, 0.0, 0.0
            elif not np.isfinite(m):
                lse = H = log_l = math.nan
            else:
                z = x[r] - m
                e = np.exp(z)
                log_l = math.log(e.sum())
                lse, H = m + log_l, log_l - float(np.sum(np.where(e > 0, e * z, 0.0))) / e.sum()
            out["lse"][r], out["entropy"][r] = lse, H
            # from the row's maximum: exact where lse itself swallows ln l
            lp = (lambda v: -np.inf if v == -np.inf and not math.isnan(lse) else v - m - log_l)
            if token is not None and 0 <= token[r] < V:
                out["logprob"][r] = lp(x[r, token[r]])
            key = np.where(np.isnan(x[r]), -np.inf, x[r])
            order = np.lexsort((np.arange(V), np.isnan(x[r]), -key))[:top]
            out["top_ids"][r, : len(order)] = order
            out["top_logprobs"][r, : len(order)] = [lp(x[r, i]) for i in order]
    return out


def logprob_eps(V):
    """Relative error of sum e^(x - m): exponentials (2^-21), their arguments (|z| 2^-23 with p-weighted |z| < 16),
    V / 64 roundings in a row."""
    return 2.0 ** -21 + 16 * 2.0 ** -23 + (V / 64 + 64) * U32


def lse_bound(lse, V):
    return logprob_eps(V) + 4 * U32 * np.abs(lse)


def entropy_bound(H, V):
    return 4 * logprob_eps(V) * (1 + np.abs(H))


def grad(x, token, lse, H, g, h):
    """Gradient of sum g logprob + h entropy in fp64 from the given lse and H, and the sum of its terms' sizes."""
    z = x - lse[:, None]
    p = np.exp(z)
    pz = np.where(p > 0, p * (z + H[:, None]), 0.0)
    hit = np.zeros_like(x)
    has = (token >= 0) & (token < x.shape[1])
    hit[np.nonzero(has)[0], token[has]] = 1.0
    g = np.where(has, g, 0.0)[:, None]
    size = np.abs(g) * (hit + p) + np.abs(h)[:, None] * np.where(p > 0, p * (np.abs(z) + np.abs(H[:, None])), 0.0)
    # each term: the exponential (2^-21), its argument's rounding (|z| 2^-23) and four more roundings
    err = size * (2.0 ** -21 + np.where(p > 0, np.abs(z), 0.0) * 2.0 ** -23 + 4 * U32)
    return g * (hit - p) - h[:, None] * pz, err
