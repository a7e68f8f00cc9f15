"""The operators around the MoE layer in a decoding step, as cases to measure.

Three families, each computed in a plain form (elementary torch operations, fp32
or fp64) and, with ``own`` set, by the library's kernels:

* ``append``     rotate q and k by their positions and write k, v into a paged cache
* ``attention``  one new token per sequence over that cache
* ``logprobs``   log probability of a given token per row of logits, entropy, top
  alternatives; ``logprobs_grad`` is its gradient with respect to the logits

A cache holds bf16, or e4m3 codes with one power-of-two exponent per (token, head)
row: the row's values are code * 2^(exponent byte - 127), with the smallest exponent
that brings the row's largest magnitude to at most 448.
"""
import math

import torch

own = False
DEVICE = "cuda"
THETA = 10000.0


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a small decode batch's write: latency is all of it
        dict(name="append decode 8", op="append", tokens=8, seqs=8, heads=32, kv_heads=8, dim=128, rot=128, page=16,
             e4m3=False, interleaved=False, head_major=True, far=30000),
        # a mixed prefill batch of five prompts with 32 heads over 8, as beside d_model 4096
        dict(name="append prefill 16k", op="append", tokens=16384, seqs=5, heads=32, kv_heads=8, dim=128, rot=128,
             page=64, e4m3=False, interleaved=False, head_major=True, far=4000),
        # an 8-bit cache with a partly rotated, interleaved layout, odd token count, far positions
        dict(name="append e4m3 12001", op="append", tokens=12001, seqs=7, heads=16, kv_heads=2, dim=64, rot=32, page=32,
             e4m3=True, interleaved=True, head_major=False, far=900000),
        # one short chat turn: a single sequence, nothing to hide latency behind
        dict(name="attention 1 x 777", op="attention", seqs=1, longest=777, shortest=777, heads=32, kv_heads=8, dim=128,
             page=16, e4m3=False, window=0, head_major=True),
        # a serving batch of ragged lengths beside the 64-token decode workload
        dict(name="attention 64 x 8k ragged", op="attention", seqs=64, longest=8192, shortest=64, heads=32, kv_heads=8,
             dim=128, page=16, e4m3=False, window=0, head_major=True),
        # one long document: the cache's length is the only parallelism
        dict(name="attention 1 x 131072", op="attention", seqs=1, longest=131072, shortest=131072, heads=32, kv_heads=8,
             dim=128, page=64, e4m3=False, window=0, head_major=False),
        # a large batch on an 8-bit cache, 8 query heads per key head
        dict(name="attention 256 x 4k e4m3", op="attention", seqs=256, longest=4096, shortest=1, heads=64, kv_heads=8,
             dim=128, page=32, e4m3=True, window=0, head_major=True),
        # one shared key head for 16 query heads, a sliding window over long caches, some sequences empty
        dict(name="attention 33 window", op="attention", seqs=33, longest=16000, shortest=0, heads=16, kv_heads=1,
             dim=64, page=16, e4m3=False, window=4096, head_major=False),
        # what a decoding step returns beside its tokens
        dict(name="logprobs 4 x 32000", op="logprobs", rows=4, vocab=32000, f32=False, top=20, masked=0.0),
        # scoring prompts from fp32 logits
        dict(name="logprobs 4096 x 131072", op="logprobs", rows=4096, vocab=131072, f32=True, top=5, masked=0.0),
        # an odd vocabulary (rows not 16-byte aligned), part of it banned, all twenty alternatives
        dict(name="logprobs 2047 x 50257", op="logprobs", rows=2047, vocab=50257, f32=False, top=20, masked=0.3),
        # the training side of the same rows: policy and entropy gradients
        dict(name="logprobs grad 4096 x 50257", op="logprobs_grad", rows=4096, vocab=50257, f32=False, top=0,
             masked=0.0),
        ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "logprobs", "logprobs_grad"])
    if op == "append":
        dim = rng.choice([64, 128, 256])
        kv_heads = rng.choice([1, 2, 3, 4, 8])
        heads = kv_heads * rng.choice([1, 2, 4, 5, 8])
        tokens = _log(rng, 1, 2 ** 27 // (dim * (heads + 2 * kv_heads)))
        return dict(op=op, tokens=tokens, seqs=min(tokens, _log(rng, 1, 64)), heads=heads, kv_heads=kv_heads, dim=dim,
                    rot=dim if rng.random() < 0.6 else 16 * rng.randint(1, dim // 16), page=rng.choice([8, 16, 24, 64, 128]),
                    e4m3=rng.random() < 0.5, interleaved=rng.random() < 0.5, head_major=rng.random() < 0.5,
                    far=_log(rng, 1, 1000000))
    if op == "attention":
        dim = rng.choice([64, 128, 128, 256])
        kv_heads = rng.choice([1, 2, 4, 8])
        heads = kv_heads * rng.choice([1, 2, 4, 6, 8, 16])
        seqs = _log(rng, 1, 256)
        longest = _log(rng, 1, min(131072, 2 ** 29 // (seqs * kv_heads * dim)))
        return dict(op=op, seqs=seqs, longest=longest, shortest=rng.choice([0, 1, longest]), heads=heads,
                    kv_heads=kv_heads, dim=dim, page=rng.choice([8, 16, 24, 64, 128]), e4m3=rng.random() < 0.5,
                    window=_log(rng, 1, longest) if rng.random() < 0.25 else 0, head_major=rng.random() < 0.5)
    vocab = _log(rng, 1000, 200000)
    f32 = rng.random() < 0.5
    return dict(op=op, rows=_log(rng, 1, 2 ** 28 // vocab), vocab=vocab, f32=f32,
                top=rng.choice([0, 1, 5, 20, 32]) if op == "logprobs" else 0, masked=rng.choice([0.0, 0.0, 0.9]))


# ---------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device=DEVICE).manual_seed(seed)


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device=DEVICE, dtype=torch.float32).to(dtype)


def _lengths(case, seed):
    """Host lengths of the sequences: spread evenly over [shortest, longest], shuffled."""
    n, lo, hi = case["seqs"], case["shortest"], case["longest"]
    g = torch.Generator().manual_seed(seed + 1)
    u = (torch.arange(n, dtype=torch.float64) + torch.rand(n, generator=g, dtype=torch.float64)) / n
    lens = (lo + u * (hi - lo)).round().to(torch.int64)
    lens[-1] = hi
    return lens[torch.randperm(n, generator=g)]


def _page_table(lens, page, seed):
    """Pages of a pool in random order: (table [n, most] int32 with -1 past the last page, number of pages)."""
    need = (lens + page - 1) // page
    total = int(need.sum())
    order = torch.randperm(max(total, 1), generator=torch.Generator().manual_seed(seed + 2))
    most = max(1, int(need.max()))
    table = torch.full((len(lens), most), -1, dtype=torch.int32)
    used = torch.arange(most)[None] < need[:, None]
    table[used] = order[:total].to(torch.int32)
    return table.to(DEVICE), max(total, 1)


def _empty_cache(case, pages):
    """Key and value stores, [pages, page, kv_heads, dim] by shape; head-major ones keep a page's rows of one head together."""
    hk, d, page = case["kv_heads"], case["dim"], case["page"]

    def store(tail, dtype, fill):
        shape = (pages, hk, page, *tail) if case["head_major"] else (pages, page, hk, *tail)
        t = torch.full(shape, fill, dtype=dtype, device=DEVICE)
        return t.transpose(1, 2) if case["head_major"] else t

    if case["e4m3"]:
        return dict(k=store((d,), torch.uint8, 0), v=store((d,), torch.uint8, 0),
                    k_exp=store((), torch.uint8, 127), v_exp=store((), torch.uint8, 127))
    return dict(k=store((d,), torch.bfloat16, 0), v=store((d,), torch.bfloat16, 0), k_exp=None, v_exp=None)


def _kv_object(s):
    from token_level_top_gb300 import moe
    return moe.KVCache(s["k"], s["v"], s["k_exp"], s["v_exp"])


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "append":
        s = _prepare_append(case, seed, g)
    elif case["op"] == "attention":
        s = _prepare_attention(case, seed, g)
    else:
        s = _prepare_logprobs(case, seed, g)
    s["case"] = case
    return s


def _prepare_append(case, seed, g):
    T, hq, hk, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    n = case["seqs"]
    cpu = torch.Generator().manual_seed(seed + 3)
    # consecutive tokens of each sequence, after a history of up to `far` tokens
    each = torch.full((n,), T // n, dtype=torch.int64)
    each[: T % n] += 1
    start = torch.randint(0, case["far"], (n,), generator=cpu)
    seq = torch.repeat_interleave(torch.arange(n), each)
    within = torch.arange(T) - torch.repeat_interleave(torch.cumsum(each, 0) - each, each)
    # only the pages written now are resident in this pool: the table's other entries are -1
    first, last = start // case["page"], (start + each - 1) // case["page"]
    need = last - first + 1
    pages = int(((each + case["page"] - 2) // case["page"] + 1).sum())   # enough wherever the sequences start
    order = torch.randperm(pages, generator=cpu)[: int(need.sum())].to(torch.int32)
    table = torch.full((n, int(last.max()) + 1), -1, dtype=torch.int32)
    row = torch.repeat_interleave(torch.arange(n), need)
    col = torch.arange(int(need.sum())) - torch.repeat_interleave(torch.cumsum(need, 0) - need, need)
    table[row, torch.repeat_interleave(first, need) + col] = order
    inv_freq = THETA ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64) / case["rot"])
    qkv = _randn(g, T, (hq + 2 * hk) * d)   # one projection's output: q, k and v are views of it
    s = dict(q=qkv[:, : hq * d].view(T, hq, d), k_new=qkv[:, hq * d: (hq + hk) * d].view(T, hk, d),
             v_new=qkv[:, (hq + hk) * d:].view(T, hk, d), pos=(start[seq] + within).to(torch.int32).to(DEVICE),
             seq=seq.to(torch.int32).to(DEVICE), table=table.to(DEVICE), inv_freq=inv_freq.to(DEVICE),
             **_empty_cache(case, pages))
    if own:
        from token_level_top_gb300 import moe
        s.update(cache=_kv_object(s), phase=moe.rope_phase(inv_freq).to(DEVICE), status=moe.status_word(DEVICE))
    return s


def _prepare_attention(case, seed, g):
    lens = _lengths(case, seed)
    table, pages = _page_table(lens, case["page"], seed)
    s = _empty_cache(case, pages)
    for name in ("k", "v"):
        if case["e4m3"]:
            x = _randn(g, *s[name].shape, dtype=torch.float32)
            codes, exp = _to_e4m3(x)
            s[name].copy_(codes)
            s[name + "_exp"].copy_(exp)
        else:
            s[name].copy_(_randn(g, *s[name].shape))
    s.update(q=_randn(g, case["seqs"], case["heads"], case["dim"]) * 2.0, lens=lens.to(torch.int32).to(DEVICE),
             table=table, longest=int(lens.max()))
    if own:
        from token_level_top_gb300 import moe
        s.update(cache=_kv_object(s), ws=moe.attention_workspace(case["dim"], DEVICE))
    return s


def _prepare_logprobs(case, seed, g):
    n, v = case["rows"], case["vocab"]
    x = _randn(g, n, v, dtype=torch.float32) * 3.0
    # a few likely tokens per row, as a trained model's logits have them
    likely = torch.randint(0, v, (n, 8), generator=g, device=DEVICE)
    x.scatter_add_(1, likely, 10.0 * torch.rand(n, 8, generator=g, device=DEVICE))
    if case["masked"]:
        banned = torch.rand(v, generator=g, device=DEVICE) < case["masked"]
        x.masked_fill_(banned, -math.inf)
        x[:, 0] = 1.0
    x = x if case["f32"] else x.to(torch.bfloat16)
    token = likely[:, 0].to(torch.int32)
    token[::7] = torch.randint(0, v, (len(token[::7]),), generator=g, device=DEVICE).to(torch.int32)
    token[5::50] = -1   # rows that score no token (padding)
    s = dict(x=x, token=token)
    if case["op"] == "logprobs_grad":
        # what a training step keeps from the forward pass, and the gradients that reach it
        f = _logprobs_plain(x, token, 0)
        s.update(lse=f["lse"], entropy=f["entropy"], dlogprob=_randn(g, n, dtype=torch.float32),
                 dentropy=0.1 * _randn(g, n, dtype=torch.float32))
    if own:
        from token_level_top_gb300 import moe
        s["status"] = moe.status_word(DEVICE)
    return s


# ---------------------------------------------------------------- plain forms

def _to_e4m3(x):
    """fp32 rows -> (e4m3 codes uint8, exponent bytes uint8): the smallest exponent with max|x| <= 448 * 2^e."""
    amax = x.abs().amax(-1)
    f, e = torch.frexp(amax)
    e = torch.where(f <= 0.875, e - 9, e - 8)
    e = torch.where(amax == 0, torch.zeros_like(e), e).clamp(-126, 127)
    codes = torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, (e + 127).to(torch.uint8)


def _rotate(x, cos, sin, rot, interleaved):
    x = x.float()
    out = x.clone()
    c, s = cos[:, None, :], sin[:, None, :]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = a * c - b * s, a * s + b * c
    else:
        h = rot // 2
        a, b = x[..., :h], x[..., h:rot]
        out[..., :h], out[..., h:rot] = a * c - b * s, a * s + b * c
    return out


def _append_plain(s):
    case = s["case"]
    angle = s["pos"].double()[:, None] * s["inv_freq"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    q = _rotate(s["q"], cos, sin, case["rot"], case["interleaved"]).to(torch.bfloat16)
    k = _rotate(s["k_new"], cos, sin, case["rot"], case["interleaved"])
    v = s["v_new"].float()
    pos, page = s["pos"].long(), case["page"]
    p = s["table"][s["seq"].long(), pos // page].long()
    at = pos % page
    for name, x in (("k", k), ("v", v)):
        if case["e4m3"]:
            codes, exp = _to_e4m3(x)
            s[name][p, at] = codes
            s[name + "_exp"][p, at] = exp
        else:
            s[name][p, at] = x.to(torch.bfloat16)
    return q


def _cache_outputs(s):
    if s["case"]["e4m3"]:
        return dict(k=s["k"].view(torch.float8_e4m3fn), v=s["v"].view(torch.float8_e4m3fn), k_exp=s["k_exp"],
                    v_exp=s["v_exp"])
    return dict(k=s["k"], v=s["v"])


def _attention_plain(s):
    case = s["case"]
    B, hq, hk, d, page = case["seqs"], case["heads"], case["kv_heads"], case["dim"], case["page"]
    L = max(1, s["longest"])
    j = torch.arange(L, device=s["q"].device)
    lens = s["lens"].long()[:, None]
    live = j[None] < lens
    if case["window"]:
        live = live & (j[None] >= lens - case["window"])
    pages = s["table"].long().clamp_min(0)[:, j // page]
    at = (j % page)[None].expand_as(pages)

    def rows(name):
        x = s[name][pages, at]                                  # [B, L, hk, d]
        if case["e4m3"]:
            x = torch.ldexp(x.view(torch.float8_e4m3fn).float(), s[name + "_exp"][pages, at][..., None].int() - 127)
        return x.float()

    q = s["q"].float().view(B, hk, hq // hk, d)
    score = torch.matmul(q, rows("k").permute(0, 2, 3, 1)) * d ** -0.5   # [B, hk, g, L]
    score = score.masked_fill(~live[:, None, None], -math.inf)
    m = score.amax(-1, keepdim=True).clamp_min(-3e38)
    p = torch.exp(score - m)
    l = p.sum(-1, keepdim=True)
    out = torch.matmul(p, rows("v").transpose(1, 2)) / torch.where(l > 0, l, torch.ones_like(l))
    lse = (m + torch.log(l)).squeeze(-1)
    return dict(out=out.view(B, hq, d).to(torch.bfloat16), lse=lse.view(B, hq))


def _order_key(x):
    """int64 keys whose order is the values', ties to the lowest index (NaN is not expected here)."""
    b = torch.where(x == 0, torch.zeros_like(x), x).view(torch.int32).long()
    b = torch.where(b < 0, -(b & 0x7FFFFFFF), b)
    return b * 2 ** 32 - torch.arange(x.shape[-1], device=x.device)


def _logprobs_plain(x, token, top):
    x = x.float()
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    z = x - m
    e = torch.exp(z)
    l = e.sum(-1)
    lse = m.squeeze(-1) + torch.log(l)
    weighted = torch.where(e > 0, e * z, torch.zeros_like(e)).sum(-1)
    entropy = torch.where(l > 0, torch.log(l) - weighted / l, torch.zeros_like(l))
    given = torch.gather(x, 1, token.clamp_min(0).long()[:, None]).squeeze(1)
    logprob = torch.where(given == -math.inf, given, given - lse)
    out = dict(logprob=torch.where(token >= 0, logprob, torch.zeros_like(logprob)), entropy=entropy, lse=lse)
    if top:
        key = torch.topk(_order_key(x), min(top, x.shape[1]), dim=1).values
        ids = torch.remainder(-key, 2 ** 32)
        best = torch.gather(x, 1, ids)
        out["top_ids"] = ids.to(torch.int32)
        out["top_logprobs"] = torch.where(best == -math.inf, best, best - lse[:, None])
    return out


def _logprobs_grad_plain(s):
    z = s["x"].float() - s["lse"][:, None]
    p = torch.exp(z)
    weighted = torch.where(p > 0, p * (z + s["entropy"][:, None]), torch.zeros_like(p))
    g = torch.where(s["token"] >= 0, s["dlogprob"], torch.zeros_like(s["dlogprob"]))[:, None]
    dx = -g * p - s["dentropy"][:, None] * weighted
    dx.scatter_add_(1, s["token"].clamp_min(0).long()[:, None], g)
    return dx.to(s["x"].dtype)


def run(s):
    op = s["case"]["op"]
    if not own:
        if op == "append":
            q = _append_plain(s)
            return dict(q=q, **_cache_outputs(s))
        if op == "attention":
            return _attention_plain(s)
        if op == "logprobs":
            return _logprobs_plain(s["x"], s["token"], s["case"]["top"])
        return _logprobs_grad_plain(s)
    from token_level_top_gb300 import moe
    if op == "append":
        q = moe.kv_append(s["cache"], s["k_new"], s["v_new"], s["pos"], s["table"], q=s["q"], phase=s["phase"],
                          seq=s["seq"], interleaved=s["case"]["interleaved"], status=s["status"])
        return dict(q=q, **_cache_outputs(s))
    if op == "attention":
        out, lse = moe.paged_attention(s["cache"], s["ws"], s["q"], s["lens"], s["table"], window=s["case"]["window"],
                                       return_lse=True)
        return dict(out=out, lse=lse)
    if op == "logprobs":
        return moe.token_logprobs(s["x"], s["token"], top=s["case"]["top"], status=s["status"])
    return moe.token_logprobs_backward(s["x"], s["token"], s["lse"], s["entropy"], s["dlogprob"], s["dentropy"],
                                       status=s["status"])


# ---------------------------------------------------------------- floors

def work(case):
    if case["op"] == "append":
        T, hq, hk, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        elt = 1 + 1 / d if case["e4m3"] else 2
        return dict(bytes=T * d * (4 * hq + 4 * hk + 2 * hk * elt) + 12 * T, flops=3 * T * case["rot"] * (hq + hk))
    if case["op"] == "attention":
        lens = _lengths(case, 0)
        if case["window"]:
            lens = lens.clamp_max(case["window"])
        keys, hk, d = int(lens.sum()), case["kv_heads"], case["dim"]
        row = d + 1 if case["e4m3"] else 2 * d
        return dict(bytes=2 * keys * hk * row + case["seqs"] * case["heads"] * (4 * d + 4) + 4 * keys // case["page"],
                    flops=4 * keys * case["heads"] * d)
    elt = 4 if case["f32"] else 2
    n, v = case["rows"], case["vocab"]
    if case["op"] == "logprobs":
        return dict(bytes=n * (v * elt + 16 + 8 * case["top"]), flops=4 * n * v)
    return dict(bytes=n * (2 * v * elt + 20), flops=6 * n * v)


# ---------------------------------------------------------------- 64-bit values

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "attention":
        return _exact_attention(s)
    return _exact_logprobs(s)


def _exact_append(s):
    """Rotation as a complex product.  Stored rows are given before any rounding, in units of their row's scale."""
    case = s["case"]
    half = case["rot"] // 2
    turn = torch.polar(torch.ones_like(s["pos"][:, None] * s["inv_freq"]), s["pos"].double()[:, None] * s["inv_freq"])

    def rotated(x):
        x = x.double()
        head, rest = x[..., : case["rot"]], x[..., case["rot"]:]
        if case["interleaved"]:
            z = torch.view_as_complex(head.reshape(*head.shape[:-1], half, 2)) * turn[:, None]
            head = torch.view_as_real(z).reshape(head.shape)
        else:
            z = torch.complex(head[..., :half], head[..., half:]) * turn[:, None]
            head = torch.cat([z.real, z.imag], -1)
        return torch.cat([head, rest], -1)

    out = dict(q=rotated(s["q"]))
    pos, page = s["pos"].long(), case["page"]
    flat = s["table"][s["seq"].long(), pos // page].long() * page + pos % page
    for name, x in (("k", rotated(s["k_new"])), ("v", s["v_new"].double())):
        pages, hk, d = s[name].shape[0], case["kv_heads"], case["dim"]
        if case["e4m3"]:
            top = x.abs().amax(-1, keepdim=True)
            e = torch.ceil(torch.log2(torch.where(top > 0, top / 448.0, torch.ones_like(top))))
            x = x * torch.exp2(-e)
            out[name + "_exp"] = None
        stored = torch.zeros(pages * page, hk, d, dtype=torch.float64, device=x.device)
        stored[flat] = x
        out[name] = stored.view(pages, page, hk, d)
    return out


def _exact_attention(s):
    case = s["case"]
    hq, hk, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    lens = s["lens"].tolist()
    out = torch.zeros(case["seqs"], hq, d, dtype=torch.float64, device=s["q"].device)
    lse = torch.full((case["seqs"], hq), -math.inf, dtype=torch.float64, device=s["q"].device)
    for b, n in enumerate(lens):
        first = max(0, n - case["window"]) if case["window"] else 0
        if n == first:
            continue
        j = torch.arange(first, n, device=out.device)
        at = (s["table"][b].long()[j // page], j % page)

        def rows(name):
            x = s[name][at].permute(1, 0, 2)
            if not case["e4m3"]:
                return x.double()
            scale = torch.exp2(s[name + "_exp"][at].double() - 127.0).permute(1, 0)
            return x.view(torch.float8_e4m3fn).double() * scale[..., None]

        score = torch.einsum("hgd,hld->hgl", s["q"][b].double().view(hk, hq // hk, d), rows("k")) / math.sqrt(d)
        lse[b] = torch.logsumexp(score, -1).view(hq)
        out[b] = torch.einsum("hgl,hld->hgd", torch.softmax(score, -1), rows("v")).reshape(hq, d)
    return dict(out=out, lse=lse)


def _exact_logprobs(s):
    case, parts = s["case"], []
    step = max(1, 2 ** 27 // case["vocab"])
    for r in range(0, case["rows"], step):
        x, token = s["x"][r: r + step].double(), s["token"][r: r + step].long()
        logp = torch.log_softmax(x, -1)
        p = torch.exp(logp)
        entropy = torch.special.entr(p).sum(-1)
        chosen = torch.nn.functional.one_hot(token.clamp_min(0), case["vocab"]).bool() & (token >= 0)[:, None]
        if case["op"] == "logprobs_grad":
            g, h = s["dlogprob"][r: r + step].double()[:, None], s["dentropy"][r: r + step].double()[:, None]
            g = g * (token >= 0)[:, None]
            parts.append(g * (chosen.double() - p) + h * (torch.special.entr(p) - p * entropy[:, None]))
            continue
        d = dict(logprob=torch.where(chosen, logp, torch.zeros_like(logp)).sum(-1), entropy=entropy,
                 lse=torch.logsumexp(x, -1))
        if case["top"]:
            order = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, : case["top"]]
            d["top_ids"] = order.to(torch.int32)
            d["top_logprobs"] = torch.gather(logp, 1, order)
        parts.append(d)
    if case["op"] == "logprobs_grad":
        return torch.cat(parts)
    return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
