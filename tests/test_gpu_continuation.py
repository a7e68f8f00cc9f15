"""Trees of drafted tokens and beams through all operators that they take, and calls that the operators' own tests do not make:
exponents far apart, caches past 32-bit offsets, several streams and threads."""
import importlib.util
import os
import sys
import threading

import numpy as np
import pytest
import torch

import continuation_ref as cref
import decode_ref as ref
from token_level_top_gb300 import build, moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    moe.lib()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def _rows(cache, name, table_row, n):
    """The first n cached rows of a sequence: (bits as stored, fp64 values [n, kv, D])."""
    j = torch.arange(n)
    at = table_row.cpu().long()[j // cache.k.shape[1]].cuda(), (j % cache.k.shape[1]).cuda()
    held = getattr(cache, name)[at].cpu()
    exp = getattr(cache, name + "_exp")
    if exp is None:
        return held, ref.f64(held)
    e = exp[at].cpu()
    return torch.cat([held, e[..., None]], -1), ref.e4m3_value(held, e)


# ---------------------------------------------------------------- operators together

@pytest.mark.parametrize("e4m3,D,page", [(False, 64, 16), (True, 128, 8), (False, 128, 24)])
def test_tree_then_its_branch(e4m3, D, page):
    """Context and drafted tokens appended (rotated by depth), attention over the tree, one branch appended again: its rows are
    the drafted ones' to the last bit, and decoding attention of the branch's end gives the tree's row."""
    g = torch.Generator().manual_seed(D + page)
    ctx, heads, kv, n = [37, 0, 200], 8, 2, 7
    parent = [-1, 0, 0, 1, 3, 2, 4]
    depth = [0, 1, 1, 2, 3, 2, 4]
    branch = [0, 1, 3, 4, 6]
    mask = [0] * n
    for i, p in enumerate(parent):
        mask[i] = (mask[p] if p >= 0 else 0) | 1 << i
    most = -(-(max(ctx) + n) // page)
    cache = moe.KVCache.empty(3 * most, page, kv, D, e4m3=e4m3)
    table = torch.randperm(3 * most, generator=g).to(torch.int32).view(3, most).cuda()
    phase = moe.rope_phase([10000.0 ** (-2 * i / D) for i in range(D // 2)]).cuda()
    x = torch.randn(sum(ctx) + 3 * n, heads + 2 * kv, D, generator=g).to(torch.bfloat16).cuda()
    q, k, v = x[:, :heads], x[:, heads: heads + kv], x[:, heads + kv:]
    old = sum(ctx)
    status, ws = moe.status_word(), moe.tree_attention_workspace(D)
    moe.kv_append(cache, k[:old], v[:old], _i32([j for c in ctx for j in range(c)]), table, phase=phase,
                  seq=_i32([b for b, c in enumerate(ctx) for _ in range(c)]), status=status)
    turned = moe.kv_append(cache, k[old:], v[old:], _i32([c + i for c in ctx for i in range(n)]), table, q=q[old:], phase=phase,
                           seq=_i32([b for b in range(3) for _ in range(n)]), rotary=_i32([[c + d for c in ctx for d in depth]]), status=status)
    out, lse = moe.tree_attention(cache, ws, turned, _i32([0, n, 2 * n, 3 * n]), _i32([c + n for c in ctx]), table,
                                  mask=torch.tensor(mask * 3).cuda(), return_lse=True)
    drafted = []
    for b, c in enumerate(ctx):
        dense = [_rows(cache, name, table[b], c + n) for name in ("k", "v")]
        drafted.append([held for held, _ in dense])
        for i in range(n):
            for h in range(heads):
                o, s, eo, es = cref.tree_row(ref.f64(turned)[b * n + i, h], dense[0][1][:, h // 4], dense[1][1][:, h // 4],
                                             cref.seen_by(mask[i], n, c, 0, i), D ** -0.5)
                assert (np.abs(ref.f64(out)[b * n + i, h] - o) <= eo).all() and abs(float(lse[b * n + i, h]) - s) <= es
    kept = torch.tensor([old + b * n + i for b in range(3) for i in branch]).cuda()
    moe.kv_append(cache, k[kept], v[kept], _i32([c + j for c in ctx for j in range(5)]), table, phase=phase,
                  seq=_i32([b for b in range(3) for _ in branch]), status=status)
    ends = torch.tensor([b * n + branch[-1] for b in range(3)]).cuda()
    got = moe.paged_attention(cache, moe.attention_workspace(D), turned[ends], _i32([c + 5 for c in ctx]), table)
    for b, c in enumerate(ctx):
        dense = []
        for held, name in zip(drafted[b], ("k", "v")):
            now, values = _rows(cache, name, table[b], c + 5)
            dense.append(values)
            assert torch.equal(now[:c], held[:c]) and torch.equal(now[c:], held[[c + i for i in branch]])
        for h in range(heads):
            o, _, eo, _ = ref.attention(ref.f64(turned[ends])[b, h], dense[0][:, h // 4], dense[1][:, h // 4], D ** -0.5)
            assert (np.abs(ref.f64(got)[b, h] - o) <= eo).all() and (np.abs(ref.f64(out[ends])[b, h] - o) <= eo).all()
    assert moe.device_status(status) == 0 and moe.device_status(ws) == 0


@pytest.mark.parametrize("e4m3,page", [(False, 4), (True, 8)])
def test_beams_keep_their_histories(e4m3, page):
    """Select, reorder, append, again and again: each beam's cached rows are those of the tokens on its way."""
    g = torch.Generator().manual_seed(page)
    B, W, V, kv, D, steps = 3, 5, 200, 2, 64, 14
    most = -(-(steps + 6) // page)
    cache = moe.KVCache.empty(B * W * most, page, kv, D, e4m3=e4m3)
    table = torch.randperm(B * W * most, generator=g).to(torch.int32).view(B * W, most).cuda()
    first = [6, 1, 4]
    status, ws = moe.status_word(), moe.beam_workspace(B * W, W)
    rows = [[[] for _ in range(W)] for _ in range(B)]       # what was cached for each beam
    lens = [0] * B

    def append(k, v, pos):
        moe.kv_append(cache, k, v, pos, table, status=status)

    for i in range(max(first)):                             # the sequences' beginnings, ragged: the same for all beams
        x = torch.randn(B, 2, kv, D, generator=g).to(torch.bfloat16)
        y = x.repeat_interleave(W, 0).cuda()
        append(y[:, 0], y[:, 1], _i32([i if i < first[b] else -1 for b in range(B) for _ in range(W)]))
        for b in range(B):
            if i < first[b]:
                lens[b] += 1
                for w in range(W):
                    rows[b][w].append(x[b])
    scores = torch.full((B, W), -float("inf"))
    scores[:, 0] = 0.0
    scores = scores.cuda()
    for _ in range(steps):
        logits = (2 * torch.randn(B * W, V, generator=g)).cuda()
        best = moe.beam_select(ws, logits, scores, W)
        table = moe.beam_reorder(cache, best["parents"], _i32(lens), table, status=status)
        scores = best["scores"]
        x = torch.randn(B * W, 2, kv, D, generator=g).to(torch.bfloat16)
        append(x[:, 0].cuda(), x[:, 1].cuda(), _i32([lens[b] for b in range(B) for _ in range(W)]))
        parents = best["parents"].tolist()
        rows = [[rows[b][parents[b][w]] + [x[b * W + w]] for w in range(W)] for b in range(B)]
        lens = [n + 1 for n in lens]
    for b in range(B):
        for w in range(W):
            want = torch.stack(rows[b][w])
            for i, name in enumerate(("k", "v")):
                held, _ = _rows(cache, name, table[b * W + w], lens[b])
                if e4m3:
                    codes, exp = ref.e4m3_cache(want[:, i].float())
                    assert torch.equal(held, torch.cat([codes, exp[..., None]], -1))
                else:
                    assert torch.equal(held, want[:, i])
    assert moe.device_status(status) == 0 and moe.device_status(ws) == 0


def test_norm_around_the_experts_and_back():
    """h + MoE(norm(h + a)): the norm's gradient takes the layer's fp32 dh and what reaches the sum past the layer."""
    T, d, E, F, k = 96, 256, 4, 128, 2
    g = torch.Generator(device="cuda").manual_seed(3)

    def w(*shape, fan):
        return (torch.randn(*shape, generator=g, device="cuda") * fan ** -0.5).to(torch.bfloat16)

    cfg = moe.Config(T=T, d_model=d, E=E, k=k, d_ff=F, cf=float(E), flags=moe.FLAG_BACKWARD)
    ws, nws = moe.workspace(cfg), moe.norm_workspace(d)
    wr, w13, w2 = w(E, d, fan=d), moe.pack_w13(w(E, F, d, fan=d), w(E, F, d, fan=d)), w(E, d, F, fan=F)
    h, a, dout = w(T, d, fan=1), w(T, d, fan=1), w(T, d, fan=1)
    weight = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16)
    s = moe.rms_norm(h, weight, residual=a)
    out = moe.layer_forward(cfg, ws, s["y"], wr, w13, w2)
    assert torch.isfinite(out).all()
    grads = moe.layer_backward(cfg, ws, s["y"], wr, w13, w2, dout)
    ds, dw = moe.rms_norm_backward(nws, s["sum"], weight, grads["dh"], dsum=dout)
    want, want_w, e, e_w = cref.norm_grad(ref.f64(s["sum"]), ref.f64(weight), ref.f64(grads["dh"]), ref.f64(dout), 1e-6)
    assert (np.abs(ref.f64(ds) - want) <= e + ref.UBF16 * (np.abs(want) + e)).all()
    assert (np.abs(ref.f64(dw) - want_w) <= e_w).all()
    moe.check_device(ws)


# ---------------------------------------------------------------- e4m3 caches whose exponents lie apart

def _exponents(kind, shape, g):
    """(bytes of k, bytes of v, factor on q)"""
    def pick(lo, hi):
        return torch.randint(lo, hi + 1, shape, generator=g).to(torch.uint8)
    if kind == "near":            # of a tile within 14
        return pick(120, 126), pick(113, 127), 1.0
    if kind == "values":          # outputs of the largest rows, whatever their weights
        return pick(118, 124), pick(40, 215), 1.0
    if kind == "values by turns":   # one tile in two far apart
        v = pick(118, 126)
        v[:, 64:128] = pick(60, 190)[:, 64:128]
        return pick(118, 124), v, 1.0
    if kind == "keys":
        return pick(0, 122), pick(120, 130), 1.0
    if kind == "large keys":
        return pick(188, 194), pick(120, 130), 2.0 ** -70
    return pick(48, 56), pick(40, 215), 2.0 ** 70   # "small keys"


@pytest.mark.parametrize("kind", ["near", "values", "values by turns", "keys", "large keys", "small keys"])
@pytest.mark.parametrize("D,page,hm,zeros", [(64, 16, True, False), (128, 5, False, True), (256, 64, True, True), (128, 32, True, False)])
def test_exponents_apart(kind, D, page, hm, zeros):
    g = torch.Generator().manual_seed(D + page)
    ctx, n, kv, heads = 300, 9, 2, 6
    L = ctx + n
    pages = -(-L // page) + 1
    shape = (kv, pages * page)
    ke, ve, factor = _exponents(kind, shape, g)
    parts = []
    for exp in (ke, ve):
        codes = torch.randint(0, 127, (*shape, D), generator=g).to(torch.uint8) | (torch.randint(0, 2, (*shape, D), generator=g) << 7).to(torch.uint8)
        if zeros:                 # rows of zeros as the append stores them
            codes[:, 7::20], exp[:, 7::20] = 0, 127
        parts += [codes, exp]

    def held(t):                  # [kv, pages * page, ...] -> [pages, page, kv, ...]
        t = t.reshape(kv, pages, page, *t.shape[2:]).cuda()
        return t.transpose(0, 1).contiguous().transpose(1, 2) if hm else t.permute(1, 2, 0, *range(3, t.dim())).contiguous()

    cache = moe.KVCache(held(parts[0]), held(parts[2]), held(parts[1]), held(parts[3]))
    q = (torch.randn(n, heads, D, generator=g) * factor).to(torch.bfloat16).cuda()
    ws = moe.tree_attention_workspace(D)
    scale = D ** -0.5 / 64
    out, lse = moe.tree_attention(cache, ws, q, _i32([0, n]), _i32([L]), torch.arange(pages, dtype=torch.int32)[None].cuda(), scale=scale,
                                  return_lse=True)
    assert moe.device_status(ws) == 0
    k, v = [ref.e4m3_value(c[:, :L], e[:, :L]) for c, e in (parts[:2], parts[2:])]
    codes = np.abs(ref.e4m3_value(parts[2][:, :L], torch.full((kv, L), 127)))
    for i in range(n):
        for h in range(heads):
            kh, vh, x = k[h // 3], v[h // 3], ref.f64(q)[i, h]
            keys = np.arange(ctx + i + 1)
            o, s, eo, es = cref.tree_row(x, kh, vh, keys, scale)
            # q's values below 2^-10 of the row's largest are off by up to 2^-17 of it
            small = np.abs(x) < 2.0 ** -9 * np.abs(x).max()
            ds = scale * 2.0 ** -17 * np.abs(x).max() * np.abs(kh[keys][:, small]).sum(-1).max(initial=0.0)
            # weights times 2^(exponent of the value row) are held to 2^-31 of the largest such product
            z = scale * (kh[keys] @ x)
            p = np.exp(z - z.max())
            p /= p.sum()
            most = (p * np.ldexp(1.0, ve[h // 3, keys].numpy().astype(int) - 127)).max()
            lost = 2.0 ** -31 * most * codes[h // 3, keys].sum(0)
            eo = eo + 2 * ds * (np.abs(vh[keys]).T @ p) + lost
            assert (np.abs(ref.f64(out)[i, h] - o) <= eo).all(), (i, h)
            assert abs(float(lse[i, h]) - s) <= es + 2 * ds, (i, h)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_e4m3_pages_out_of_range(D):
    g = torch.Generator().manual_seed(D)
    page, L, n = 16, 150, 4
    shape = (12, page, 1, D)
    codes = [torch.randint(0, 127, shape, generator=g).to(torch.uint8) for _ in range(2)]
    exps = [torch.randint(118, 126, shape[:3], generator=g).to(torch.uint8) for _ in range(2)]
    cache = moe.KVCache(*[t.cuda() for t in codes + exps])
    table = torch.tensor([[3, 5, -1, 0, 1, 10 ** 7, 7, 8, 9, 2, 12]], dtype=torch.int32)
    q = (torch.randn(n, 4, D, generator=g)).to(torch.bfloat16).cuda()
    ws = moe.tree_attention_workspace(D)
    out, lse = moe.tree_attention(cache, ws, q, _i32([0, n]), _i32([L]), table.cuda(), scale=2.0 ** -9, return_lse=True)
    assert moe.device_status(ws) == 8
    keys = [j for j in range(L) if 0 <= table[0, j // page] < 12]
    dense = [ref.e4m3_value(c, e) for c, e in zip(codes, exps)]
    k, v = [np.stack([d[max(0, min(int(table[0, j // page]), 11)), j % page, 0] for j in range(L)]) for d in dense]
    for i in range(n):
        for h in range(4):
            x = ref.f64(q)[i, h]
            small = np.abs(x) < 2.0 ** -9 * np.abs(x).max()
            mine = [j for j in keys if j <= L - n + i]
            ds = 2.0 ** -9 * 2.0 ** -17 * np.abs(x).max() * np.abs(k[mine][:, small]).sum(-1).max(initial=0.0)
            o, s, eo, es = cref.tree_row(x, k, v, mine, 2.0 ** -9)
            z = 2.0 ** -9 * (k[mine] @ x)
            p = np.exp(z - z.max()) / np.exp(z - z.max()).sum()
            assert (np.abs(ref.f64(out)[i, h] - o) <= eo + 2 * ds * (np.abs(v[mine]).T @ p) + 2.0 ** -31 * np.abs(v[mine]).sum(0)).all()
            assert abs(float(lse[i, h]) - s) <= es + 2 * ds


# ---------------------------------------------------------------- offsets past 32 bits

@pytest.mark.parametrize("e4m3", [False, True])
def test_caches_past_32_bit_offsets(e4m3):
    """The last pages of stores of more than 2^32 bytes and 2^31 values: append, tree and reordering as in a small cache."""
    page, kv, D, n = 64, 2, 128, 5
    small = 16
    pages = (2 ** 32 if e4m3 else 2 ** 31) // (page * kv * D) * 5 // 4 + small
    g = torch.Generator().manual_seed(1)
    x = torch.randn(2 * 300, 4 + 2 * kv, D, generator=g).to(torch.bfloat16).cuda()
    phase = moe.rope_phase([10000.0 ** (-2 * i / D) for i in range(D // 2)]).cuda()
    got = []
    for total, first in ((small, 0), (pages, pages - small)):
        def store(*tail, dtype):
            return torch.empty((total, kv, page, *tail), dtype=dtype, device="cuda").transpose(1, 2)
        t = torch.uint8 if e4m3 else torch.bfloat16
        parts = [store(D, dtype=t) for _ in range(2)] + ([store(dtype=torch.uint8) for _ in range(2)] if e4m3 else [])
        for s in parts:
            s[first:] = 0
        cache = moe.KVCache(*parts)
        table = (torch.arange(10, dtype=torch.int32).view(2, 5) + first + 3).cuda()
        status, ws = moe.status_word(), moe.tree_attention_workspace(D)
        pos = torch.arange(300, dtype=torch.int32).repeat(2).cuda()
        q = moe.kv_append(cache, x[:, 4: 4 + kv], x[:, 4 + kv:], pos, table, q=x[:, :4], phase=phase, seq=_i32([0] * 300 + [1] * 300),
                          rotary=pos[None] // 2, status=status)
        rows = torch.cat([q[300 - n: 300], q[600 - n:]])
        out = moe.tree_attention(cache, ws, rows, _i32([0, n, 2 * n]), _i32([300, 300]), table)
        new = moe.beam_reorder(cache, _i32([[1, 1]]), _i32([300]), table, status=status)
        assert moe.device_status(status) == 0 and moe.device_status(ws) == 0
        got.append([out, new - first] + [s[first:].clone() for s in parts])
        del cache, parts, s
    assert all(torch.equal(a, b) for a, b in zip(*got))
    torch.cuda.empty_cache()


# ---------------------------------------------------------------- several callers

def test_threads_and_streams():
    """Norm, its gradient, selection, reordering and appends from four threads, each with a stream and workspaces of its own."""
    g = torch.Generator().manual_seed(2)
    B, W, V, page, kv, D, cols = 4, 4, 5000, 8, 2, 64, 1407

    def make(i):
        gi = torch.Generator().manual_seed(i)
        return dict(x=torch.randn(333, cols, generator=gi).cuda(), r=torch.randn(333, cols, generator=gi).cuda(), w=torch.randn(cols, generator=gi).cuda(),
                    logits=torch.randn(B * W, V, generator=gi).cuda(), scores=-torch.rand(B, W, generator=gi).cuda(),
                    kv=torch.randn(B * W * 21, 2 + 2 * kv, D, generator=gi).to(torch.bfloat16).cuda(),
                    table=torch.randperm(B * W * 3, generator=gi).to(torch.int32).view(B * W, 3).cuda())

    pos = torch.arange(21, dtype=torch.int32).repeat(B * W).cuda()
    seq = torch.arange(B * W, dtype=torch.int32).repeat_interleave(21).cuda()
    phase = moe.rope_phase([0.5 ** i for i in range(D // 2)]).cuda()
    lens = _i32([21] * B)

    def run(s):
        nws, bws = moe.norm_workspace(cols), moe.beam_workspace(B * W, W)
        cache = moe.KVCache.empty(B * W * 3, page, kv, D)
        n = moe.rms_norm(s["x"], s["w"], residual=s["r"], e4m3=True)
        dx, dw = moe.rms_norm_backward(nws, n["sum"], s["w"], s["r"])
        q = moe.kv_append(cache, s["kv"][:, 2: 2 + kv], s["kv"][:, 2 + kv:], pos, s["table"], q=s["kv"][:, :2], phase=phase, seq=seq, rotary=pos[None] // 3)
        best = moe.beam_select(bws, s["logits"], s["scores"], W)
        table = moe.beam_reorder(cache, best["parents"], lens, s["table"])
        return [*n.values(), dx, dw, q, *best.values(), table, cache.k, cache.v]

    sets = [make(i) for i in range(4)]
    want = [run(s) for s in sets]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(15):
                    got = run(sets[i])
                torch.cuda.current_stream().synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                wrong.append(i)
        except Exception as e:   # noqa: BLE001
            wrong.append((i, e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_two_graphs_take_turns_with_one_workspace():
    """Graphs captured on one workspace, replayed one after the other on one stream."""
    g = torch.Generator().manual_seed(4)
    cols = 2000
    x = [torch.randn(n, cols, generator=g).cuda() for n in (700, 45)]
    dy = [torch.randn(n, cols, generator=g).cuda() for n in (700, 45)]
    logits = [torch.randn(n, 9000, generator=g).cuda() for n in (24, 6)]
    scores = [torch.zeros(n, 3).cuda() for n in (8, 2)]
    nws, bws = moe.norm_workspace(cols), moe.beam_workspace(24, 6)
    w = torch.randn(cols, generator=g).cuda()

    def run(i):
        return [*moe.rms_norm_backward(nws, x[i], w, dy[i]), *moe.beam_select(bws, logits[i], scores[i], 6).values()]

    want = [[t.clone() for t in run(i)] for i in range(2)]
    graphs, got = [], []
    for i in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            got.append(run(i))
        graphs.append(gr)
    for _ in range(5):
        for i in (0, 1, 1, 0):
            for t in got[i]:
                t.zero_()
            graphs[i].replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(got[i], want[i]))


# ---------------------------------------------------------------- the example

def _example():
    folder = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples")
    for name in ("decode_step", "tree_and_beams"):
        spec = importlib.util.spec_from_file_location(name, os.path.join(folder, name + ".py"))
        m = sys.modules[name] = importlib.util.module_from_spec(spec)   # dataclasses look it up there
        spec.loader.exec_module(m)
    return m


def _dense_logits(model, texts):
    """Logits of each text's last token with attention in fp64 over the whole text."""
    rows = []
    for t in texts:
        q, k, v = model.qkv(model.embed[torch.tensor(t).cuda()])
        th = torch.arange(len(t)).double().cuda()[:, None, None] * torch.tensor(model.inv_freq, dtype=torch.float64).cuda()
        turned = []
        for x in (q, k):
            a, b = x.double().chunk(2, -1)
            turned.append(torch.cat([a * th.cos() - b * th.sin(), a * th.sin() + b * th.cos()], -1))
        rep = model.heads // model.kv_heads
        p = torch.softmax(torch.einsum("hd,nhd->hn", turned[0][-1], turned[1].repeat_interleave(rep, 1)) * model.head_dim ** -0.5, -1)
        rows.append(torch.einsum("hn,nhd->hd", p, v.double().repeat_interleave(rep, 1)))
    return model.rest(model.embed[torch.tensor([t[-1] for t in texts]).cuda()], torch.stack(rows).to(torch.bfloat16)).double()


@pytest.mark.parametrize("e4m3", [False, True])
def test_trees_and_beams_against_a_dense_decoder(e4m3, monkeypatch):
    ex = _example()
    routes, plain = [], moe.layer_forward

    def layer(*args):
        out, aux = plain(*args, aux=True)
        routes.append(aux)
        return out

    monkeypatch.setattr(moe, "layer_forward", layer)

    def agree(logits, want):
        # Rows whose experts are others: the choice is a step, taken either way where the k-th and the next router logit are no
        # further apart than twice what a logit differs by (each of the two may move by that, towards the other).
        mine, other = routes[-2], routes[-1]
        same = (mine["assign"].sort(-1)[0] == other["assign"].sort(-1)[0]).all(-1)
        top = mine["logits"].sort(-1, descending=True)[0]
        assert (same | (top[:, model.k - 1] - top[:, model.k] <= 2 * (mine["logits"] - other["logits"]).abs().amax(-1))).all()
        logits, want = logits.double()[same], want[same]
        assert float((logits - want).norm() / want.norm()) < bound

    model = ex.NormedDecoder()
    g = torch.Generator().manual_seed(5)
    prompts = [torch.randint(0, model.vocab, (n,), generator=g).tolist() for n in (1, 33, 16, 70)]
    # bf16 values through three norms, three projections and the experts (an e4m3 cache: 2^-4 of a value's own, averaged over
    # dimensions and keys), relative to logits of unit scale
    bound = 0.1 if e4m3 else 0.04
    s = ex.TreeSession(model, prompts, room=30, e4m3=e4m3)
    texts = [list(p) for p in prompts]
    for _ in range(3):
        trees = [[(int(torch.randint(-1, i, (1,), generator=g)) if i else -1, int(torch.randint(0, model.vocab, (1,), generator=g)))
                  for i in range(n)] for n in (4, 0, 7, 1)]
        ways = []
        for t, tree in zip(texts, trees):
            nodes = [t]
            for parent, token in tree:
                nodes.append(nodes[parent + 1] + [token])
            ways += nodes
        got = s.verify(trees)
        s.check()
        agree(s.logits, _dense_logits(model, ways))
        for t, new in zip(texts, got):
            t += new
        assert s.len.tolist() == [len(t) - 1 for t in texts] and s.token.tolist() == [t[-1] for t in texts]
    b = ex.BeamSession(model, prompts, beams=3, room=12, page=8, e4m3=e4m3)
    for i in range(7):
        ways = [p + (b.tokens[j, w].tolist() if i else []) for j, p in enumerate(prompts) for w in range(3)]
        b.step()
        b.check()
        agree(b.logits, _dense_logits(model, ways))
    assert torch.isfinite(b.scores).all() and (b.scores[:, :-1] >= b.scores[:, 1:]).all()


def test_example_runs(capsys):
    _example().main()
    assert "cache: e4m3" in capsys.readouterr().out
