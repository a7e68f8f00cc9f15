"""Operators of a decoder layer around drafted and searched continuations, as cases to measure.

Five families, each computed in a plain form (elementary torch operations, fp32 or
fp64) and, with ``own`` set, by the library's kernels:

* ``norm``         a residual's addition, the root-mean-square norm of the sum, and its output in
  bf16 / fp32, in e4m3 codes with a scale per row, or both; ``norm_grad`` is its gradient
* ``append_axes``  keys and values into a paged cache at given slots, rotated by positions on
  several axes (time, height, width)
* ``tree``         attention of the drafted tokens of every sequence, a tree of up to 64 each, over
  the paged cache that holds them behind the sequence's context
* ``beam``         the best continuations over all beams and the vocabulary, and the beams' pages
  brought in line with the chosen parents

A cache holds bf16, or e4m3 codes with one power-of-two exponent per (token, head)
row: the row's values are code * 2^(exponent byte - 127).
"""
import math

import torch

own = False
DEVICE = "cuda"
THETA = 10000.0


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the norm before the experts of a 64-token decode batch, d_model 4096: latency is all of it; codes for e4m3 experts
        dict(name="norm decode 64 x 4096", op="norm", rows=64, cols=4096, f32=False, residual=True, y=True, e4m3=True, pad=0),
        # the same in a prefill of four batches of 4096 tokens, for experts that take bf16
        dict(name="norm prefill 16384 x 4096", op="norm", rows=16384, cols=4096, f32=False, residual=True, y=True, e4m3=False,
             pad=0),
        # its gradient in training: fp32 gradients from the experts' layer, bf16 rows, the residual's gradient added
        dict(name="norm grad 16384 x 4096", op="norm_grad", rows=16384, cols=4096, f32=False, dy32=True, residual=True, pad=0),
        # fp32 rows of an odd width inside wider ones, as a slice of an activation has them
        dict(name="norm grad 5001 x 1407", op="norm_grad", rows=5001, cols=1407, f32=True, dy32=True, residual=False, pad=2),
        # eight drafted trees of eight tokens: slots in a row, positions by depth
        dict(name="append axes drafts 64", op="append_axes", tokens=64, seqs=8, heads=32, kv_heads=8, dim=128, rot=128,
             page=16, e4m3=False, interleaved=False, head_major=True, axes=1, far=30000),
        # image patches of a few prompts: time, height and width, an 8-bit cache
        dict(name="append axes images 22k", op="append_axes", tokens=22000, seqs=6, heads=32, kv_heads=8, dim=128, rot=128,
             page=64, e4m3=True, interleaved=False, head_major=True, axes=3, far=4000),
        # one short chat turn with a small tree: nothing to hide latency behind
        dict(name="tree 1 x 777, 8 drafted", op="tree", seqs=1, longest=777, shortest=777, drafted=8, heads=32, kv_heads=8,
             dim=128, page=16, e4m3=False, window=0, head_major=True, masked=True),
        # a serving batch of ragged lengths beside the 64-token decode workload, 16 drafted tokens each
        dict(name="tree 64 x 8k, 16 drafted", op="tree", seqs=64, longest=8192, shortest=64, drafted=16, heads=32, kv_heads=8,
             dim=128, page=16, e4m3=False, window=0, head_major=True, masked=True),
        # a larger batch on an 8-bit cache, chains of up to eight drafted tokens, 8 query heads per key head
        dict(name="tree 128 x 4k e4m3, 8 drafted", op="tree", seqs=128, longest=4096, shortest=1, drafted=8, heads=64,
             kv_heads=8, dim=128, page=32, e4m3=True, window=0, head_major=True, masked=False),
        # long documents under a sliding window with the largest trees: arithmetic counts as well as the cache's bytes
        dict(name="tree 5 x 40k window, 61 drafted", op="tree", seqs=5, longest=40000, shortest=30000, drafted=61, heads=16,
             kv_heads=2, dim=64, page=64, e4m3=False, window=20000, head_major=False, masked=True),
        # one sentence with four beams
        dict(name="beam 1 x 4 x 32000", op="beam", seqs=1, beams=4, vocab=32000, f32=False, n=8, longest=300, kv_heads=8, dim=128,
             page=16, e4m3=False, finished=0.0, first=False),
        # a batch of 64 sentences with eight beams, twice as many candidates, some beams at their end
        dict(name="beam 64 x 8 x 131072", op="beam", seqs=64, beams=8, vocab=131072, f32=True, n=16, longest=400, kv_heads=8,
             dim=128, page=64, e4m3=False, finished=0.05, first=False),
        ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "append_axes", "tree", "tree", "tree", "beam", "beam"])
    if op in ("norm", "norm_grad"):
        cols = _log(rng, 16, 16384)
        case = dict(op=op, rows=_log(rng, 1, 2 ** 26 // cols), cols=cols if rng.random() < 0.3 else max(16, cols // 8 * 8),
                    f32=rng.random() < 0.4, residual=rng.random() < 0.7, pad=rng.choice([0, 0, 0, 8, 3]))
        if op == "norm":
            case["e4m3"] = rng.random() < 0.5
            case["y"] = not case["e4m3"] or rng.random() < 0.5
        else:
            case["dy32"] = case["f32"] or rng.random() < 0.5
        return case
    dim = rng.choice([64, 128, 128, 256])
    if op == "append_axes":
        kv_heads = rng.choice([1, 2, 3, 4, 8])
        heads = kv_heads * rng.choice([1, 2, 4, 5, 8])
        tokens = _log(rng, 1, 2 ** 27 // (dim * (heads + 2 * kv_heads)))
        return dict(op=op, tokens=tokens, seqs=min(tokens, _log(rng, 1, 64)), heads=heads, kv_heads=kv_heads, dim=dim,
                    rot=dim if rng.random() < 0.6 else 16 * rng.randint(1, dim // 16), page=rng.choice([8, 16, 24, 64, 128]),
                    e4m3=rng.random() < 0.5, interleaved=rng.random() < 0.5, head_major=rng.random() < 0.5,
                    axes=rng.randint(1, 4), far=_log(rng, 1, 1000000))
    kv_heads = rng.choice([1, 2, 4, 8])
    if op == "tree":
        heads = kv_heads * rng.choice([1, 2, 4, 5, 8, 16])
        seqs, drafted = _log(rng, 1, 256), _log(rng, 1, 64)
        longest = _log(rng, 1, min(131072, 2 ** 28 // (seqs * kv_heads * dim), 2 ** 28 // (seqs * heads * drafted)))
        return dict(op=op, seqs=seqs, longest=longest, shortest=rng.choice([0, 1, longest]), drafted=drafted, heads=heads,
                    kv_heads=kv_heads, dim=dim, page=rng.choice([8, 16, 24, 64, 128]), e4m3=rng.random() < 0.5,
                    window=_log(rng, 1, longest) if rng.random() < 0.25 else 0, head_major=rng.random() < 0.5,
                    masked=rng.random() < 0.7)
    vocab, beams = _log(rng, 1000, 200000), rng.choice([1, 2, 3, 4, 5, 8, 16])
    return dict(op=op, seqs=_log(rng, 1, max(1, min(128, 2 ** 26 // (vocab * beams)))), beams=beams, vocab=vocab,
                f32=rng.random() < 0.5, n=rng.choice([beams, 2 * beams, 2 * beams]), longest=_log(rng, 1, 600),
                kv_heads=kv_heads, dim=dim, page=rng.choice([8, 16, 24, 64]), e4m3=rng.random() < 0.5,
                finished=rng.choice([0.0, 0.1, 0.3]), first=rng.random() < 0.2)


# ---------------------------------------------------------------- inputs

def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device=DEVICE, dtype=torch.float32).to(dtype)


def _cpu(seed):
    return torch.Generator().manual_seed(seed)


def _spread(n, lo, hi, seed):
    """n host numbers spread evenly over [lo, hi], shuffled; hi is among them."""
    g = _cpu(seed)
    u = (torch.arange(n, dtype=torch.float64) + torch.rand(n, generator=g, dtype=torch.float64)) / n
    out = (lo + u * (hi - lo)).round().to(torch.int64)
    out[-1] = hi
    return out[torch.randperm(n, generator=g)]


def _page_table(lens, page, seed):
    """Pages of a pool in random order: (table [n, most] int32 with -1 past the last page, number of pages)."""
    need = (lens + page - 1) // page
    total = max(int(need.sum()), 1)
    order = torch.randperm(total, generator=_cpu(seed + 2))
    most = max(1, int(need.max()))
    table = torch.full((len(lens), most), -1, dtype=torch.int32)
    used = torch.arange(most)[None] < need[:, None]
    table[used] = order[: int(need.sum())].to(torch.int32)
    return table.to(DEVICE), total


def _empty_cache(case, pages):
    """Key and value stores, [pages, page, kv_heads, dim] by shape; head-major ones keep a page's rows of one head together."""
    hk, d, page, head_major = case["kv_heads"], case["dim"], case["page"], case.get("head_major", True)

    def store(tail, dtype, fill):
        shape = (pages, hk, page, *tail) if head_major else (pages, page, hk, *tail)
        t = torch.full(shape, fill, dtype=dtype, device=DEVICE)
        return t.transpose(1, 2) if head_major else t

    if case["e4m3"]:
        return dict(k=store((d,), torch.uint8, 0), v=store((d,), torch.uint8, 0),
                    k_exp=store((), torch.uint8, 127), v_exp=store((), torch.uint8, 127))
    return dict(k=store((d,), torch.bfloat16, 0), v=store((d,), torch.bfloat16, 0), k_exp=None, v_exp=None)


def _filled_cache(case, pages, g):
    s = _empty_cache(case, pages)
    for name in ("k", "v"):
        if case["e4m3"]:
            codes, exp = _to_e4m3(_randn(g, *s[name].shape, dtype=torch.float32))
            s[name].copy_(codes)
            s[name + "_exp"].copy_(exp)
        else:
            s[name].copy_(_randn(g, *s[name].shape))
    return s


def _kv_object(s):
    from token_level_top_gb300 import moe
    return moe.KVCache(s["k"], s["v"], s["k_exp"], s["v_exp"])


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    make = dict(norm=_prepare_norm, norm_grad=_prepare_norm, append_axes=_prepare_append, tree=_prepare_tree, beam=_prepare_beam)
    s = make[case["op"]](case, seed, g)
    s["case"] = case
    return s


def _prepare_norm(case, seed, g):
    n, d, dtype = case["rows"], case["cols"], torch.float32 if case["f32"] else torch.bfloat16

    def rows(dtype, scale=1.0):   # each `pad` values apart, as a slice of wider rows
        wide = _randn(g, n, d + case["pad"], dtype=torch.float32)
        wide[:, :d] *= scale
        return wide.to(dtype)[:, :d]

    # a residual stream has a few loud channels
    loud = torch.ones(d, device=DEVICE)
    loud[torch.randint(0, d, (max(1, d // 512),), generator=g, device=DEVICE)] = 20.0
    s = dict(x=rows(dtype, loud), weight=(1.0 + 0.1 * _randn(g, d, dtype=torch.float32)).to(dtype), eps=1e-6)
    if case["op"] == "norm":
        s["residual"] = rows(dtype, 2.0 * loud) if case["residual"] else None
    else:
        s["dy"] = rows(torch.float32 if case["dy32"] else dtype)
        s["dsum"] = rows(dtype) if case["residual"] else None
    if own:
        from token_level_top_gb300 import moe
        s["status"] = moe.status_word(DEVICE)
        if case["op"] == "norm_grad":
            s["ws"] = moe.norm_workspace(d, DEVICE)
    return s


def _prepare_append(case, seed, g):
    T, hq, hk, d, n = case["tokens"], case["heads"], case["kv_heads"], case["dim"], case["seqs"]
    cpu = _cpu(seed + 3)
    # consecutive slots of each sequence, after a history of up to `far` tokens
    each = torch.full((n,), T // n, dtype=torch.int64)
    each[: T % n] += 1
    start = torch.randint(0, case["far"], (n,), generator=cpu)
    seq = torch.repeat_interleave(torch.arange(n), each)
    within = torch.arange(T) - torch.repeat_interleave(torch.cumsum(each, 0) - each, each)
    slot = start[seq] + within
    # only the pages written now are resident in this pool: the table's other entries are -1
    first, last = start // case["page"], (start + each - 1) // case["page"]
    need = last - first + 1
    pages = int(((each + case["page"] - 2) // case["page"] + 1).sum())   # enough wherever the sequences start
    order = torch.randperm(pages, generator=cpu)[: int(need.sum())].to(torch.int32)
    table = torch.full((n, int(last.max()) + 1), -1, dtype=torch.int32)
    row = torch.repeat_interleave(torch.arange(n), need)
    col = torch.arange(int(need.sum())) - torch.repeat_interleave(torch.cumsum(need, 0) - need, need)
    table[row, torch.repeat_interleave(first, need) + col] = order
    # one axis: a tree's depths; more: patches in rows of 28 (time, height, width, and one more for layouts that have it)
    if case["axes"] == 1:
        rotary = (start[seq] + torch.minimum(within, within // 2 + 1))[None]
    else:
        rotary = torch.stack([start[seq] + within // 784, start[seq] + within // 28 % 28, start[seq] + within % 28,
                              within])[: case["axes"]]
    pairs = case["rot"] // 2
    axis = torch.randint(0, case["axes"], (pairs,), generator=cpu) if seed % 2 else torch.arange(pairs) * case["axes"] // pairs
    inv_freq = THETA ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64) / case["rot"])
    qkv = _randn(g, T, (hq + 2 * hk) * d)   # one projection's output: q, k and v are views of it
    s = dict(q=qkv[:, : hq * d].view(T, hq, d), k_new=qkv[:, hq * d: (hq + hk) * d].view(T, hk, d),
             v_new=qkv[:, (hq + hk) * d:].view(T, hk, d), slot=slot.to(torch.int32).to(DEVICE),
             seq=seq.to(torch.int32).to(DEVICE), table=table.to(DEVICE), inv_freq=inv_freq.to(DEVICE),
             rotary=rotary.to(torch.int32).to(DEVICE), axis=axis.to(torch.uint8).to(DEVICE), **_empty_cache(case, pages))
    if own:
        from token_level_top_gb300 import moe
        s.update(cache=_kv_object(s), phase=moe.rope_phase(inv_freq).to(DEVICE), status=moe.status_word(DEVICE))
    return s


def _tree_lengths(case, seed):
    """Host lengths of the contexts and numbers of drafted tokens (the same numbers whatever the seed, in another order)."""
    drafted = _spread(case["seqs"], (case["drafted"] + 1) // 2, case["drafted"], 4)
    return (_spread(case["seqs"], case["shortest"], case["longest"], seed + 1),
            drafted[torch.randperm(case["seqs"], generator=_cpu(seed + 4))])


def _prepare_tree(case, seed, g):
    context, drafted = _tree_lengths(case, seed)
    lens = context + drafted
    table, pages = _page_table(lens, case["page"], seed)
    s = _filled_cache(case, pages, g)
    T = int(drafted.sum())
    mask = None
    if case["masked"]:
        # bit j: the token sees drafted token j of its sequence, which is itself or one of its ancestors
        pick, bits = torch.rand(T, generator=_cpu(seed + 5)).tolist(), []
        for n in drafted.tolist():
            own_bits = []
            for i in range(n):
                parent = int(pick[len(bits) + i] * (min(i, 6) + 1)) - 1   # one of the last few, or the context itself
                own_bits.append((own_bits[i - 1 - parent] if parent >= 0 else 0) | 1 << i)
            bits += own_bits
        mask = torch.tensor([b - 2 ** 64 if b >= 2 ** 63 else b for b in bits], dtype=torch.int64).to(DEVICE)
    row_start = torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(drafted, 0)])
    s.update(q=_randn(g, T, case["heads"], case["dim"]) * 2.0, lens=lens.to(torch.int32).to(DEVICE), table=table, mask=mask,
             row_start=row_start.to(torch.int32).to(DEVICE), longest=int(lens.max()), most=int(drafted.max()))
    if own:
        from token_level_top_gb300 import moe
        s.update(cache=_kv_object(s), ws=moe.tree_attention_workspace(case["dim"], DEVICE))
    return s


def _prepare_beam(case, seed, g):
    B, W, V, page = case["seqs"], case["beams"], case["vocab"], case["page"]
    x = _randn(g, B * W, V, dtype=torch.float32) * 2.0
    # a few likely tokens per beam, as a trained model's logits have them
    likely = torch.randint(0, V, (B * W, 12), generator=g, device=DEVICE)
    x.scatter_add_(1, likely, 12.0 * torch.rand(B * W, 12, generator=g, device=DEVICE))
    done = torch.rand(B * W, generator=g, device=DEVICE) < case["finished"]   # beams at their end continue with token 2 alone
    x[done] = -math.inf
    x[done, 2] = 0.0
    scores = -3.0 * torch.rand(B, W, generator=g, device=DEVICE) - 5.0
    if case["first"]:   # a search begins with one beam alive
        scores[:, 1:] = -math.inf
    # full pages are common to a sentence's beams, the page that fills is each beam's own; one more column waits for later
    lens = _spread(B, (case["longest"] + 1) // 2, case["longest"], seed + 1)
    full, tail = lens // page, (lens % page > 0).long()
    most = int(full.max()) + 2
    order = torch.randperm(B * (case["longest"] // page + W), generator=_cpu(seed + 2)).to(torch.int32)   # the whole pool
    table, used = torch.full((B, W, most), -1, dtype=torch.int32), 0
    for b, (f, t) in enumerate(zip(full.tolist(), tail.tolist())):
        table[b, :, :f] = order[used: used + f]
        used += f
        if t:
            table[b, :, f] = order[used: used + W]
            used += W
    s = _filled_cache(case, len(order), g)
    s.update(x=x if case["f32"] else x.to(torch.bfloat16), scores=scores, lens=lens.to(torch.int32).to(DEVICE),
             table=table.view(B * W, most).to(DEVICE))
    if own:
        from token_level_top_gb300 import moe
        s.update(cache=_kv_object(s), ws=moe.beam_workspace(B * W, case["n"], DEVICE))
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


def _cache_outputs(s):
    if s["case"]["e4m3"]:
        return dict(k=s["k"].view(torch.float8_e4m3fn), v=s["v"].view(torch.float8_e4m3fn), k_exp=s["k_exp"],
                    v_exp=s["v_exp"])
    return dict(k=s["k"], v=s["v"])


def _norm_plain(s):
    case, out = s["case"], {}
    x = s["x"].float()
    if case["residual"]:   # the norm is that of the sum as it is stored
        out["sum"] = (x + s["residual"].float()).to(s["x"].dtype)
        x = out["sum"].float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * s["weight"].float()
    if case["y"]:
        out["y"] = y.to(s["x"].dtype)
    if case["e4m3"]:
        amax = y.abs().amax(-1)
        scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
        out["codes"], out["scales"] = (y / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn), scale
    return out


def _norm_grad_plain(s):
    x, dy = s["x"].float(), s["dy"].float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"])
    unit = x * r
    wdy = dy * s["weight"].float()
    dx = r * (wdy - unit * (wdy * unit).mean(-1, keepdim=True))
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return dict(dx=dx.to(s["x"].dtype), dweight=(dy * unit).sum(0))


def _append_plain(s):
    case = s["case"]
    rot, half = case["rot"], case["rot"] // 2
    angle = s["rotary"].double()[s["axis"].long()].T * s["inv_freq"]          # [T, rot / 2]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def rotated(x):
        x = x.float()
        out = x.clone()
        first, second = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, half), slice(half, rot))
        a, b = x[..., first], x[..., second]
        out[..., first], out[..., second] = a * cos - b * sin, a * sin + b * cos
        return out

    pos, page = s["slot"].long(), case["page"]
    p, at = s["table"][s["seq"].long(), pos // page].long(), pos % page
    for name, x in (("k", rotated(s["k_new"])), ("v", s["v_new"].float())):
        if case["e4m3"]:
            s[name][p, at], s[name + "_exp"][p, at] = _to_e4m3(x)
        else:
            s[name][p, at] = x.to(torch.bfloat16)
    return rotated(s["q"]).to(torch.bfloat16)


def _seen(s, j, count_dtype=torch.int64):
    """Which cached tokens j [L] each of the [B, most] padded drafted tokens sees: [B, most, L]; and which of those exist."""
    case = s["case"]
    start = s["row_start"].long()
    n = (start[1:] - start[:-1])[:, None]                                     # [B, 1]
    i = torch.arange(s["most"], device=j.device)
    exists = i[None] < n
    row = (start[:-1, None] + i[None]).clamp_max(s["q"].shape[0] - 1)
    bits = s["mask"][row] if s["mask"] is not None else (2 << i)[None].expand(row.shape) - 1   # (2 << 63 is 0: every bit)
    context = s["lens"].long()[:, None] - n
    draft = j[None] - context                                                 # [B, L]
    of_tree = (draft >= 0) & (draft < n)
    tree = (torch.bitwise_right_shift(bits[:, :, None], draft.clamp(0, 63)[:, None]) & 1).bool() & of_tree[:, None]
    before = draft < 0
    if case["window"]:
        # the last `window` tokens of the row's path: what it sees of the drafted ones, the context before them
        later = tree.flip(-1).cumsum(-1, dtype=count_dtype).flip(-1)          # drafted tokens of the path from j on
        tree = tree & (later <= case["window"])
        left = case["window"] - later[..., :1]
        return (before[:, None] & (j[None, None] >= context[..., None] - left)) | tree, exists, row
    return before[:, None] | tree, exists, row


def _tree_plain(s):
    case = s["case"]
    B, hq, hk, d, page, M = case["seqs"], case["heads"], case["kv_heads"], case["dim"], case["page"], s["most"]
    j = torch.arange(s["longest"], device=s["q"].device)
    seen, exists, row = _seen(s, j)
    pages = s["table"].long().clamp_min(0)[:, j // page]
    at = (j % page)[None].expand_as(pages)

    def rows(name):
        x = s[name][pages, at]                                                # [B, L, hk, d]
        if case["e4m3"]:
            x = torch.ldexp(x.view(torch.float8_e4m3fn).float(), s[name + "_exp"][pages, at][..., None].int() - 127)
        return x.float()

    q = s["q"].float()[row].view(B, M, hk, hq // hk, d).permute(0, 2, 1, 3, 4).reshape(B, hk, M * (hq // hk), d)
    score = torch.matmul(q, rows("k").permute(0, 2, 3, 1)) * d ** -0.5        # [B, hk, M g, L]
    score = score.view(B, hk, M, hq // hk, -1).masked_fill_(~seen[:, None, :, None], -math.inf)
    m = score.amax(-1, keepdim=True).clamp_min(-3e38)
    p = torch.exp(score - m)
    del score
    total = p.sum(-1, keepdim=True)
    lse = (m + torch.log(total)).squeeze(-1)                                  # [B, hk, M, g]
    out = torch.matmul(p.view(B, hk, M * (hq // hk), -1), rows("v").transpose(1, 2)).view(B, hk, M, hq // hk, d)
    out = out / torch.where(total > 0, total, torch.ones_like(total))
    return dict(out=out.permute(0, 2, 1, 3, 4)[exists].reshape(-1, hq, d).to(torch.bfloat16),
                lse=lse.permute(0, 2, 1, 3)[exists].reshape(-1, hq))


def _order_key(x):
    """int64 keys whose order is the values', ties to the lowest index (NaN is not expected here)."""
    b = torch.where(x == 0, torch.zeros_like(x), x).view(torch.int32).long()
    b = torch.where(b < 0, -(b & 0x7FFFFFFF), b)
    return b * 2 ** 32 - torch.arange(x.shape[-1], device=x.device)


def _beam_plain(s):
    case = s["case"]
    B, W, V, n = case["seqs"], case["beams"], case["vocab"], case["n"]
    x = s["x"].float()
    ids = torch.remainder(-torch.topk(_order_key(x), min(n, V), dim=1).values, 2 ** 32)   # of each beam, in order
    wide = x.double()
    m = wide.amax(-1, keepdim=True)
    lse = m + torch.log(torch.exp(wide - m).sum(-1, keepdim=True))
    total = (s["scores"].double().view(-1, 1) + (torch.gather(wide, 1, ids) - lse)).view(B, -1)
    best, at = torch.sort(total, dim=1, descending=True, stable=True)         # beams in order, so ties go to the lowest
    best, at = best[:, :n], at[:, :n]
    none = best == -math.inf
    parents = torch.where(none, -1, at // min(n, V))
    tokens = torch.where(none, -1, torch.gather(ids.view(B, -1), 1, at))
    return dict(scores=best.float(), parents=parents.to(torch.int32), tokens=tokens.to(torch.int32))


def _reorder_plain(s, parents):
    """A beam that is the first of its parent's children keeps the parent's filling page; the others take those of the
    beams without children, in order, and get a copy of the parent's."""
    case = s["case"]
    B, W, page = case["seqs"], case["beams"], case["page"]
    p = parents.long()
    old, lens = s["table"].view(B, W, -1).long(), s["lens"].long()
    beams = torch.arange(W, device=p.device)
    same = (p[:, :, None] == p[:, None, :]) & (p >= 0)[:, :, None]
    first = (p >= 0) & ~(same & (beams[None, None] < beams[None, :, None])).any(-1)
    childless = ~(p[:, None, :] == beams[None, :, None]).any(-1)
    nth = (~first).long().cumsum(1) - 1                                       # of the beams that need another page
    free = torch.sort((~childless).to(torch.int8), dim=1, stable=True).indices
    home = torch.where(first, p, torch.gather(free, 1, nth.clamp_min(0)))
    source = torch.where(p >= 0, p, beams[None])
    full, rest = lens // page, lens % page
    col = torch.arange(old.shape[2], device=p.device)[None, None]
    wide = (B, W, old.shape[2])
    shared = torch.gather(old, 1, source[..., None].expand(wide))
    kept = torch.gather(old, 1, home[..., None].expand(wide))
    new = torch.where(col < full[:, None, None], shared, torch.where((col == full[:, None, None]) & (rest > 0)[:, None, None], kept, old))
    copied = ~first & (p >= 0) & (rest > 0)[:, None]
    at = full.clamp_max(old.shape[2] - 1)[:, None, None].expand(B, W, 1)
    src, dst = torch.gather(shared, 2, at)[..., 0][copied], torch.gather(kept, 2, at)[..., 0][copied]
    rows = torch.arange(page, device=p.device)[None] < rest[:, None].expand(B, W)[copied][:, None]
    for name in ("k", "v", "k_exp", "v_exp"):
        if s[name] is not None:
            t = s[name]
            keep = rows.view(*rows.shape, *[1] * (t.dim() - 2))
            t[dst] = torch.where(keep, t[src], t[dst])
    return new.view(B * W, -1).to(torch.int32)


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        if op == "norm":
            return _norm_plain(s)
        if op == "norm_grad":
            return _norm_grad_plain(s)
        if op == "append_axes":
            q = _append_plain(s)
            return dict(q=q, **_cache_outputs(s))
        if op == "tree":
            return _tree_plain(s)
        out = _beam_plain(s)
        out["table"] = _reorder_plain(s, out["parents"][:, : case["beams"]])
        return dict(out, **_cache_outputs(s))
    from token_level_top_gb300 import moe
    if op == "norm":
        out = moe.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=s["eps"], y=case["y"], e4m3=case["e4m3"],
                           status=s["status"])
        if case["e4m3"]:
            out["codes"] = out["codes"].view(torch.float8_e4m3fn)
        return out
    if op == "norm_grad":
        dx, dweight = moe.rms_norm_backward(s["ws"], s["x"], s["weight"], s["dy"], dsum=s["dsum"], eps=s["eps"])
        return dict(dx=dx, dweight=dweight)
    if op == "append_axes":
        q = moe.kv_append(s["cache"], s["k_new"], s["v_new"], s["slot"], s["table"], q=s["q"], phase=s["phase"], seq=s["seq"],
                          interleaved=case["interleaved"], rotary=s["rotary"], axis=s["axis"], status=s["status"])
        return dict(q=q, **_cache_outputs(s))
    if op == "tree":
        out, lse = moe.tree_attention(s["cache"], s["ws"], s["q"], s["row_start"], s["lens"], s["table"], mask=s["mask"],
                                      window=case["window"], return_lse=True)
        return dict(out=out, lse=lse)
    out = moe.beam_select(s["ws"], s["x"], s["scores"], case["n"])
    out["table"] = moe.beam_reorder(s["cache"], out["parents"][:, : case["beams"]], s["lens"], s["table"], status=s["ws"])
    return dict(out, **_cache_outputs(s))


# ---------------------------------------------------------------- floors

def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad"):
        n, elt = case["rows"] * case["cols"], 4 if case["f32"] else 2
        if op == "norm":
            return dict(bytes=n * (elt * (1 + 2 * case["residual"] + case["y"]) + case["e4m3"]) + 4 * case["rows"] * case["e4m3"] +
                        case["cols"] * elt, flops=6 * n)
        return dict(bytes=n * (elt * (2 + case["residual"]) + (4 if case["dy32"] else elt)) + case["cols"] * (elt + 4),
                    flops=12 * n)
    hk, d = case["kv_heads"], case["dim"]
    row = d + 1 if case["e4m3"] else 2 * d   # bytes of a cached row
    if op == "append_axes":
        T, hq = case["tokens"], case["heads"]
        return dict(bytes=T * (d * (4 * hq + 4 * hk) + 2 * hk * row) + (12 + 4 * case["axes"]) * T,
                    flops=3 * T * case["rot"] * (hq + hk))
    if op == "tree":
        context, drafted = _tree_lengths(case, 0)
        if case["window"]:
            context = context.clamp_max(case["window"])
        keys, T = int((context + drafted).sum()), int(drafted.sum())
        pairs = int((context * drafted + drafted * (drafted + 1) // 2).sum())
        return dict(bytes=2 * keys * hk * row + T * case["heads"] * (4 * d + 4) + 8 * T + 4 * keys // case["page"],
                    flops=4 * pairs * case["heads"] * d)
    rows, V = case["seqs"] * case["beams"], case["vocab"]
    # the logits, the tables, and on average a third of the beams' filling pages copied, half full
    moved = rows * case["page"] // 6 * hk * row * 2 * 2
    return dict(bytes=rows * (V * (4 if case["f32"] else 2) + 4) + 12 * case["seqs"] * case["n"] +
                8 * rows * (case["longest"] // case["page"] + 2) + moved, flops=4 * rows * V)


# ---------------------------------------------------------------- 64-bit values

def exact(case, seed):
    s = prepare(case, seed)
    return dict(norm=_exact_norm, norm_grad=_exact_norm_grad, append_axes=_exact_append, tree=_exact_tree,
                beam=_exact_beam)[case["op"]](s)


def _exact_norm(s):
    """Codes are given before their rounding, in units of their row's scale."""
    case, out = s["case"], {}
    x = s["x"].double()
    if case["residual"]:
        x = x + s["residual"].double()
        out["sum"] = x
        x = x.to(s["x"].dtype).double()   # the norm is that of the sum as it is stored
    length = torch.linalg.vector_norm(x, dim=-1, keepdim=True) / math.sqrt(case["cols"])
    y = x / torch.hypot(length, torch.full_like(length, math.sqrt(s["eps"]))) * s["weight"].double()
    if case["y"]:
        out["y"] = y
    if case["e4m3"]:
        top = torch.linalg.vector_norm(y, ord=math.inf, dim=-1)
        out["scales"] = torch.where(top > 0, top / 448.0, torch.ones_like(top))
        out["codes"] = y / out["scales"][:, None]
    return out


def _exact_norm_grad(s):
    x, w, dy = s["x"].double(), s["weight"].double(), s["dy"].double()
    var = torch.einsum("rc,rc->r", x, x)[:, None] / x.shape[1] + s["eps"]
    dot = torch.einsum("rc,c,rc->r", dy, w, x)[:, None]
    dx = dy * w / torch.sqrt(var) - x * dot / (x.shape[1] * var * torch.sqrt(var))
    if s["dsum"] is not None:
        dx = dx + s["dsum"].double()
    return dict(dx=dx, dweight=torch.einsum("rc,rc->c", dy, x / torch.sqrt(var)))


def _exact_append(s):
    """Rotation as a complex product.  Stored rows are given before any rounding, in units of their row's scale."""
    case = s["case"]
    half = case["rot"] // 2
    where = torch.index_select(s["rotary"].double(), 0, s["axis"].int())       # [rot / 2, T]
    angle = where.T * s["inv_freq"]
    turn = torch.polar(torch.ones_like(angle), angle)

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
    pos, page = s["slot"].long(), case["page"]
    flat = s["table"][s["seq"].long(), pos // page].long() * page + pos % page
    for name, x in (("k", rotated(s["k_new"])), ("v", s["v_new"].double())):
        if case["e4m3"]:
            top = x.abs().amax(-1, keepdim=True)
            x = x * torch.exp2(-torch.ceil(torch.log2(torch.where(top > 0, top / 448.0, torch.ones_like(top)))))
            out[name + "_exp"] = None
        stored = torch.zeros(s[name].shape[0] * page, case["kv_heads"], case["dim"], dtype=torch.float64, device=x.device)
        stored[flat] = x
        out[name] = stored.view(-1, page, case["kv_heads"], case["dim"])
    return out


def _exact_tree(s):
    case = s["case"]
    hq, hk, d, page, g = case["heads"], case["kv_heads"], case["dim"], case["page"], case["heads"] // case["kv_heads"]
    start, lens = s["row_start"].tolist(), s["lens"].tolist()
    bits = s["mask"].tolist() if s["mask"] is not None else None
    out = torch.zeros(len(s["q"]), hq, d, dtype=torch.float64, device=s["q"].device)
    lse = torch.full((len(s["q"]), hq), -math.inf, dtype=torch.float64, device=s["q"].device)
    for b, total in enumerate(lens):
        n = start[b + 1] - start[b]
        if n == 0:
            continue
        context = total - n
        first = max(0, context - case["window"]) if case["window"] else 0
        j = torch.arange(first, total, device=out.device)
        at = (s["table"][b].long()[j // page], j % page)

        def rows(name):
            x = s[name][at].permute(1, 0, 2)
            if not case["e4m3"]:
                return x.double()
            return x.view(torch.float8_e4m3fn).double() * torch.exp2(s[name + "_exp"][at].double() - 127.0).T[..., None]

        # the path of each row, drafted tokens by number; of a window its last ones
        seen = torch.zeros(n, total - first, dtype=torch.bool)
        for i in range(n):
            path = [m for m in range(n) if (bits[start[b] + i] >> m & 1 if bits else m <= i)]
            if case["window"]:
                path = path[-case["window"]:]
                seen[i, max(0, context - (case["window"] - len(path))) - first: context - first] = True
            else:
                seen[i, : context - first] = True
            for m in path:
                seen[i, context + m - first] = True
        hide = torch.where(seen, 0.0, -math.inf).double().to(out.device)[None, :, None]
        q = s["q"][start[b]: start[b + 1]].double().view(n, hk, g, d)
        score = torch.einsum("nhgd,hld->hngl", q, rows("k")) / math.sqrt(d) + hide
        lse[start[b]: start[b + 1]] = torch.logsumexp(score, -1).transpose(0, 1).reshape(n, hq)
        weight = torch.nan_to_num(torch.softmax(score, -1))
        out[start[b]: start[b + 1]] = torch.einsum("hngl,hld->nhgd", weight, rows("v")).reshape(n, hq, d)
    return dict(out=out, lse=lse)


def _exact_beam(s):
    case = s["case"]
    B, W, V, n, page = case["seqs"], case["beams"], case["vocab"], case["n"], case["page"]
    scores, parents, tokens = [], [], []
    for b in range(B):
        total = (torch.log_softmax(s["x"][b * W: (b + 1) * W].double(), -1) + s["scores"][b].double()[:, None]).flatten()
        least = torch.topk(total, min(n, len(total))).values[-1]
        near = torch.nonzero(total >= least).flatten()                        # in order of their index
        order = near[torch.sort(total[near], descending=True, stable=True).indices[:n]].tolist()
        order = [i for i in order if total[i] > -math.inf]
        missing = [-1] * (n - len(order))
        scores.append([float(total[i]) for i in order] + [-math.inf] * len(missing))
        parents.append([i // V for i in order] + missing)
        tokens.append([i % V for i in order] + missing)
    # the pages, beam by beam on the host
    table, lens = s["table"].view(B, W, -1).tolist(), s["lens"].tolist()
    new = [[list(r) for r in t] for t in table]
    cache = {name: s[name].clone() for name in ("k", "v", "k_exp", "v_exp") if s[name] is not None}
    for b in range(B):
        full, rest = divmod(lens[b], page)
        spare = [w for w in range(W) if w not in parents[b][:W]]
        settled = set()
        for w, p in enumerate(parents[b][:W]):
            if p >= 0:
                new[b][w][:full] = table[b][p][:full]
            home = p if p >= 0 and p not in settled else spare.pop(0)
            settled.add(p)
            if rest:
                new[b][w][full] = table[b][home][full]
                if home != p and p >= 0:
                    for name, t in cache.items():
                        t[table[b][home][full], :rest] = s[name][table[b][p][full], :rest]
    dev = s["x"].device
    out = dict(scores=torch.tensor(scores, dtype=torch.float64, device=dev),
               parents=torch.tensor(parents, dtype=torch.int32, device=dev),
               tokens=torch.tensor(tokens, dtype=torch.int32, device=dev),
               table=torch.tensor(new, dtype=torch.int32, device=dev).view(B * W, -1))
    for name, t in cache.items():
        if not case["e4m3"]:
            t = t.double()
        elif name in ("k", "v"):
            t = t.view(torch.float8_e4m3fn).double()
        out[name] = t
    return out
