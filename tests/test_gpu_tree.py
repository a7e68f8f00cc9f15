"""Attention of drafted tokens over the paged cache against a plain 64-bit implementation, through the binding."""
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


def _tree_masks(n, g, kind):
    """Masks (python ints) of n drafted tokens: a tree's paths, a chain, anything, or nothing."""
    if kind == "tree":
        out = []
        for i in range(n):
            p = int(torch.randint(-1, i, (1,), generator=g)) if i else -1
            out.append((out[p] if p >= 0 else 0) | 1 << i)
        return out
    if kind == "any":   # bits past the sequence's drafted tokens do not count
        return [int(torch.randint(-2 ** 63, 2 ** 63 - 1, (1,), generator=g)) & (2 ** 64 - 1) for _ in range(n)]
    if kind == "none":
        return [0] * n
    return [None] * n


def _signed(m):
    return m - 2 ** 64 if m >= 2 ** 63 else m


class Case:
    def __init__(self, ctx, drafted, heads, kv, D, page, e4m3, hm, kind="tree", seed=0, kscale=1.0, junk=True):
        g = torch.Generator().manual_seed(seed + heads + D + page + sum(drafted))
        self.lens = [c + n for c, n in zip(ctx, drafted)]
        self.ctx, self.drafted, self.heads, self.kv, self.D, self.page, self.e4m3 = ctx, drafted, heads, kv, D, page, e4m3
        need = [-(-n // page) for n in self.lens]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=g).tolist()
        self.table = torch.full((len(ctx), max(1, max(need)) + 1), -7, dtype=torch.int32)
        for b, n in enumerate(need):
            for j in range(n):
                self.table[b, j] = order.pop()
        self.dense, stores, exps = [], [], []
        for i in range(2):
            shape = (pages, kv, page, D) if hm else (pages, page, kv, D)
            st = torch.full(shape, 0x7F if e4m3 else float("nan"), dtype=torch.uint8 if e4m3 else torch.bfloat16)
            ex = torch.full(shape[:3], 255, dtype=torch.uint8)
            if hm:
                st, ex = st.transpose(1, 2), ex.transpose(1, 2)
            rows = []
            for b, n in enumerate(self.lens):
                x = torch.randn(n, kv, D, generator=g) * (kscale if i == 0 else 1.0)
                j = torch.arange(n)
                at = self.table[b].long()[j // page], j % page
                if e4m3:
                    codes, e = ref.e4m3_cache(x * torch.exp2(torch.randint(-3, 4, (n, kv, 1), generator=g).float()))
                    st[at], ex[at] = codes, e
                    rows.append(ref.e4m3_value(codes, e))
                else:
                    st[at] = x.to(torch.bfloat16)
                    rows.append(ref.f64(x.to(torch.bfloat16)))
            self.dense.append(rows)
            stores.append(torch.empty_strided(st.shape, st.stride(), dtype=st.dtype, device="cuda").copy_(st))
            exps.append(torch.empty_strided(ex.shape, ex.stride(), dtype=ex.dtype, device="cuda").copy_(ex))
        self.cache = moe.KVCache(*stores, *(exps if e4m3 else []))
        self.T = sum(drafted)
        self.q = torch.randn(max(self.T, 1), heads, D, generator=g).to(torch.bfloat16)[: self.T].cuda()
        self.masks = [m for n in drafted for m in _tree_masks(n, g, kind)]
        self.mask = None if kind == "chain" else torch.tensor([_signed(m) for m in self.masks], dtype=torch.int64).cuda()
        self.start = torch.tensor([0] + list(np.cumsum(drafted)), dtype=torch.int32).cuda()
        self.seq_len = torch.tensor(self.lens, dtype=torch.int32).cuda()
        self.table = self.table.cuda()

    def run(self, ws=None, **kw):
        ws = moe.tree_attention_workspace(self.D) if ws is None else ws
        return moe.tree_attention(self.cache, ws, kw.pop("q", self.q), kw.pop("row_start", self.start), kw.pop("seq_len", self.seq_len),
                                  kw.pop("table", self.table), mask=kw.pop("mask", self.mask), **kw)

    def check(self, out, lse, window=0, scale=None, rows=None, dead=()):
        """Every row (or those in `rows`) against the formula; `dead` (b, key) pairs are left out."""
        scale = self.D ** -0.5 if scale is None else scale
        q, out, lse = ref.f64(self.q), ref.f64(out), ref.f64(lse)
        t = 0
        for b, n in enumerate(self.drafted):
            gone = {k for s, k in dead if s == b}
            for i in range(n):
                if rows is None or t in rows:
                    keys = [k for k in cref.seen_by(self.masks[t], n, self.ctx[b], window, i) if k not in gone]
                    for h in range(self.heads):
                        hk = h // (self.heads // self.kv)
                        o, s, eo, es = cref.tree_row(q[t, h], self.dense[0][b][:, hk], self.dense[1][b][:, hk], keys, scale)
                        assert (np.abs(out[t, h] - o) <= eo).all(), (b, i, h, np.abs(out[t, h] - o).max())
                        assert lse[t, h] == s if not keys else abs(lse[t, h] - s) <= es, (b, i, h, lse[t, h], s)
                t += 1


CASES = [
    # contexts, drafted, heads, kv, D, page, e4m3, head_major, masks, window
    ([0], [1], 1, 1, 64, 16, False, True, "chain", 0),
    ([5], [1], 4, 1, 128, 16, False, True, "tree", 0),
    ([63, 64, 65, 0], [1, 2, 3, 4], 4, 2, 128, 16, False, False, "tree", 0),
    ([0, 100, 7], [64, 0, 64], 2, 1, 64, 8, False, True, "tree", 0),
    ([500], [64], 16, 2, 128, 16, False, True, "tree", 0),          # 512 rows a key head: four tiles
    ([130, 1], [33, 5], 5, 1, 256, 24, False, True, "any", 0),
    ([300, 20], [7, 9], 6, 2, 128, 7, False, False, "any", 0),
    ([257], [16], 8, 2, 256, 1, False, True, "chain", 0),
    ([900, 3, 0, 64], [12, 12, 1, 30], 12, 3, 64, 128, False, True, "tree", 40),
    ([900, 3, 0, 64], [12, 12, 1, 30], 4, 2, 128, 16, False, False, "chain", 5),
    ([100, 30], [60, 50], 2, 2, 64, 16, False, True, "any", 8),     # windows shorter than a row's path
    ([77, 10], [9, 1], 2, 1, 128, 24, False, True, "tree", 1),
    ([70, 0], [20, 10], 4, 1, 128, 16, False, True, "none", 0),     # rows without drafted tokens: the context, or nothing
    ([70, 0], [20, 10], 4, 1, 64, 16, True, True, "none", 30),
    ([0], [1], 1, 1, 64, 16, True, True, "chain", 0),
    ([129, 0, 31], [8, 64, 3], 8, 2, 128, 16, True, False, "tree", 0),
    ([400], [33], 40, 2, 64, 32, True, True, "any", 100),
    ([260, 5], [10, 2], 6, 3, 256, 8, True, True, "tree", 0),
    ([3000, 10], [16, 4], 4, 1, 128, 64, False, False, "tree", 0),  # an item over many blocks
    ([2500], [40], 16, 1, 256, 48, True, True, "tree", 1000),
    ([20, 0, 3, 150] * 60, [3, 1, 0, 2] * 60, 4, 2, 64, 16, False, True, "tree", 0),    # many short items in a block
    ([90, 0, 3, 150] * 50, [1, 2, 5, 0] * 50, 10, 2, 128, 16, True, True, "chain", 0),
    ([1000] * 40, [4] * 40, 8, 4, 128, 16, False, True, "tree", 0),
]


@pytest.mark.parametrize("ctx,drafted,heads,kv,D,page,e4m3,hm,kind,window", CASES)
def test_tree(ctx, drafted, heads, kv, D, page, e4m3, hm, kind, window):
    c = Case(ctx, drafted, heads, kv, D, page, e4m3, hm, kind)
    ws = moe.tree_attention_workspace(D)
    out, lse = c.run(ws, window=window, return_lse=True)
    assert moe.device_status(ws) == 0
    rows = None if c.T * heads < 3000 else set(range(0, c.T, 1 + c.T * heads // 3000))
    c.check(out, lse, window, rows=rows)
    # the same again on the same workspace, to the last bit
    out2, lse2 = c.run(ws, window=window, return_lse=True)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_one_token_is_the_decoding_attention():
    """A single drafted token that sees itself: what paged_attention computes, within both kernels' roundings."""
    c = Case([100, 0, 999], [1, 1, 1], 8, 2, 128, 16, False, True, "chain")
    out, lse = c.run(return_lse=True)
    want, wlse = moe.paged_attention(c.cache, moe.attention_workspace(128), c.q, c.seq_len, c.table, return_lse=True)
    assert torch.allclose(lse, wlse, atol=1e-5) and (out.float() - want.float()).abs().max() <= 2.0 ** -7 * want.float().abs().max()


@pytest.mark.parametrize("scale", [1.0, -0.7, 0.0])
def test_large_scores_and_scales(scale):
    c = Case([300, 20], [9, 5], 4, 2, 128, 16, False, True, "tree", kscale=20.0)
    out, lse = c.run(scale=scale, return_lse=True)
    c.check(out, lse, scale=scale)


@pytest.mark.parametrize("scale", [0.3, -0.7, 0.0])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_scales_over_an_e4m3_cache(scale, D):
    c = Case([300, 20], [9, 40], 4, 1, D, 16, True, True, "tree")
    out, lse = c.run(scale=scale, return_lse=True)
    c.check(out, lse, scale=scale)


@pytest.mark.parametrize("e4m3,D", [(True, 64), (True, 128), (False, 64), (True, 256), (False, 128)])
def test_few_and_many_rows_in_turn(e4m3, D):
    """Items of few rows and of many, long and short, one after the other in the same blocks."""
    n = 140
    ctx, drafted = [[0, 130, 700, 5, 64][i % 5] for i in range(n)], [[2, 40, 1, 64, 16, 0, 33][i % 7] for i in range(n)]
    c = Case(ctx, drafted, 8, 2, D, 16, e4m3, True, "tree")
    ws = moe.tree_attention_workspace(D)
    out, lse = c.run(ws, return_lse=True)
    assert moe.device_status(ws) == 0
    c.check(out, lse, rows=set(range(0, c.T, 13)))
    out2, lse2 = c.run(ws, return_lse=True)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_row_of_q_that_is_not_a_number(e4m3):
    c = Case([200, 90], [20, 3], 4, 2, 64, 16, e4m3, True, "tree")
    want, wlse = c.run(return_lse=True)
    q = c.q.clone()
    q[5, 1, 7], q[21, 3, 0] = float("nan"), float("nan")
    out, lse = c.run(q=q, return_lse=True)
    hit = torch.zeros(c.T, 4, dtype=torch.bool, device="cuda")
    hit[5, 1] = hit[21, 3] = True
    assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse[~hit], wlse[~hit])
    assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()


def test_scores_that_rise_and_fall():
    """The running maximum is raised many times, also late and by different rows."""
    c = Case([1500], [30], 8, 1, 64, 16, False, True, "tree")
    big = torch.linspace(0.1, 12.0, 1530, dtype=torch.float64).to(torch.bfloat16)
    for name, dense in (("k", c.dense[0]),):
        st = getattr(c.cache, name)
        j = torch.arange(1530)
        at = c.table[0].cpu().long()[j // 16].cuda(), (j % 16).cuda()
        st[at] = (st[at].float() * big.cuda().float()[:, None, None]).to(torch.bfloat16)
        dense[0] = ref.f64(st[at])
    out, lse = c.run(return_lse=True)
    c.check(out, lse)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("window", [0, 50])
def test_what_a_row_does_not_see_has_no_effect(e4m3, window):
    """NaN and infinities in the keys and values of drafted tokens and of context behind a window reach only the rows that
    see them; all other rows keep their bits."""
    c = Case([200, 90], [20, 13], 4, 2, 64, 16, e4m3, True, "tree")
    base, blse = c.run(window=window, return_lse=True)
    c.check(base, blse, window)
    spoiled = [(0, 203), (0, 215), (1, 93), (0, 160), (1, 60)] if window else [(0, 203), (0, 215), (1, 93)]
    for part in ("v", "k"):
        st = getattr(c.cache, part)
        keep = st.clone()
        for i, (b, key) in enumerate(spoiled):
            pg, at = int(c.table[b, key // 16]), key % 16
            st[pg, at, 0, 5 * i] = 0x7F if e4m3 else [float("nan"), float("inf"), -float("inf")][i % 3]
        out, lse = c.run(window=window, return_lse=True)
        st.copy_(keep)
        t, hit = 0, 0
        for b, n in enumerate(c.drafted):
            for i in range(n):
                keys = cref.seen_by(c.masks[t], n, c.ctx[b], window, i)
                marks = [k for s, k in spoiled if s == b and k in keys]
                for h in range(4):
                    clean = h // 2 == 1 or not marks
                    if clean:
                        assert torch.equal(out[t, h], base[t, h]) and torch.equal(lse[t, h], blse[t, h]), (part, b, i, h)
                    else:
                        hit += 1
                        if part == "v":
                            bad = [5 * s for s, (sb, k) in enumerate(spoiled) if sb == b and k in marks]
                            odd = ~torch.isfinite(out[t, h])
                            assert odd[bad].all() and int(odd.sum()) == len(set(bad))
                            assert torch.equal(lse[t, h], blse[t, h])
                t += 1
        assert hit > 0


def test_nan_that_every_row_sees():
    c = Case([200], [5], 2, 1, 64, 16, False, True, "tree")
    pg = int(c.table[0, 3])
    c.cache.v[pg, 2, 0, 7] = float("nan")
    out = c.run()
    assert torch.isnan(out[:, :, 7]).all() and torch.isfinite(out[:, :, :7]).all() and torch.isfinite(out[:, :, 8:]).all()
    c.cache.v[pg, 2, 0, 7] = 0.0
    c.cache.k[pg, 2, 0, 7] = float("nan")
    out, lse = c.run(return_lse=True)
    assert torch.isnan(out).all() and torch.isnan(lse).all()


def test_rows_of_no_sequence_are_left():
    c = Case([40, 9, 100], [3, 2, 4], 4, 2, 64, 16, False, True, "tree")
    want, wlse = c.run(return_lse=True)
    T = c.T + 7
    q = torch.full((T, 4, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    q[2: 2 + c.T] = c.q
    mask = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    mask[2: 2 + c.T] = c.mask
    out = torch.full((T, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    ws = moe.tree_attention_workspace(64)
    got = c.run(ws, q=q, mask=mask, row_start=c.start + 2, out=out)
    assert got is out and torch.equal(out[2: 2 + c.T], want)
    assert (out[:2] == 5).all() and (out[2 + c.T:] == 5).all() and moe.device_status(ws) == 0


def test_strided_q_and_out():
    c = Case([40, 9], [3, 12], 4, 2, 64, 16, False, False, "tree")
    want = c.run()
    big = torch.zeros(c.T, 6, 80, dtype=torch.bfloat16, device="cuda")
    big[:, 1:5, :64] = c.q
    hold = torch.full((c.T, 4, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    got = c.run(q=big[:, 1:5, :64], out=hold[:, :, :64])
    assert torch.equal(got, want) and (hold[:, :, 64:] == 5).all()
    swapped = c.q.transpose(0, 1).contiguous().transpose(0, 1)     # heads apart
    assert torch.equal(c.run(q=swapped), want)


def test_bad_lengths_rows_and_pages():
    c = Case([40, 40, 40], [6, 5, 4], 4, 1, 64, 16, False, True, "tree")
    ws = moe.tree_attention_workspace(64)
    # a page outside the cache: its keys are left out
    t2 = c.table.clone()
    t2[0, 1] = 10 ** 6
    out, lse = c.run(ws, table=t2, return_lse=True)
    assert moe.device_status(ws) == 8
    c.check(out, lse, dead=[(0, k) for k in range(16, 32)])
    # every page bad: nothing is seen
    out, lse = c.run(ws, table=torch.full_like(c.table, -1), return_lse=True)
    assert moe.device_status(ws) == 8
    assert (out == 0).all() and (lse == -float("inf")).all()
    # lengths: none, below 0, shorter than the drafted tokens, longer than the table
    out, lse = c.run(ws, seq_len=torch.tensor([0, -5, 44], dtype=torch.int32).cuda(), return_lse=True)
    assert moe.device_status(ws) == 8
    assert (out[:11] == 0).all() and (lse[:11] == -float("inf")).all()
    c.check(out, lse, rows=range(11, 15))
    out, lse = c.run(ws, seq_len=torch.tensor([46, 3, 44], dtype=torch.int32).cuda(), return_lse=True)
    assert moe.device_status(ws) == 8
    short = Case([40, 40, 40], [6, 5, 4], 4, 1, 64, 16, False, True, "tree")
    short.ctx = [40, -2, 40]
    short.check(out, lse)
    t3 = c.table[:, :2].contiguous()
    out = c.run(ws, table=t3, seq_len=torch.tensor([32, 32, 10 ** 9], dtype=torch.int32).cuda())
    assert moe.device_status(ws) == 8
    assert torch.equal(out, c.run(ws, table=t3, seq_len=torch.tensor([32, 32, 32], dtype=torch.int32).cuda()))
    assert moe.device_status(ws) == 0
    # rows: falling, past the end, too many for one sequence, negative
    hold = torch.full_like(c.q, 5.0)
    # (where they fall, row 5 is in two sequences)
    for start, fine in (([0, 6, 5, 15], range(5)), ([0, 6, 11, 16], range(11)), ([-1, 6, 11, 15], range(6, 15))):
        out, lse = c.run(ws, row_start=torch.tensor(start, dtype=torch.int32).cuda(), out=hold.clone(), return_lse=True)
        assert moe.device_status(ws) == 8
        c.check(out, lse, rows=fine)
    many = Case([10], [65], 1, 1, 64, 16, False, True, "chain")
    out = many.run(ws, out=torch.full_like(many.q, 5.0))
    assert moe.device_status(ws) == 8 and (out == 5).all()


def test_no_sequences_and_no_rows():
    c = Case([40], [6], 4, 1, 64, 16, False, True, "tree")
    ws = moe.tree_attention_workspace(64)
    z = torch.zeros(1, dtype=torch.int32).cuda()
    out = c.run(ws, row_start=z, seq_len=z[:0], table=c.table[:0], out=torch.full_like(c.q, 5.0))
    assert (out == 5).all()
    assert c.run(ws, q=c.q[:0], mask=None, row_start=torch.zeros(2, dtype=torch.int32).cuda()).shape == (0, 4, 64)
    out = c.run(ws, row_start=torch.zeros(2, dtype=torch.int32).cuda(), out=torch.full_like(c.q, 5.0))
    assert (out == 5).all() and moe.device_status(ws) == 0


def test_in_a_graph_follows_rows_lengths_and_masks():
    c = Case([500, 30, 900], [8, 8, 8], 8, 2, 128, 16, False, True, "tree")
    ws, other = moe.tree_attention_workspace(128), moe.tree_attention_workspace(128)
    out = torch.zeros_like(c.q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.run(ws, out=out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(ws, out=out)
    g = torch.Generator().manual_seed(9)
    for lens, start in (([508, 38, 908], [0, 8, 16, 24]), ([8, 20, 300], [0, 1, 9, 9]), ([333, 30, 128], [2, 8, 8, 24])):
        c.seq_len.copy_(torch.tensor(lens, dtype=torch.int32))
        c.start.copy_(torch.tensor(start, dtype=torch.int32))
        c.mask.copy_(torch.tensor([_signed(int(m)) for m in torch.randint(0, 256, (24,), generator=g)]))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, c.run(other, out=torch.zeros_like(out)))
    assert moe.device_status(ws) == 0


def test_two_streams_with_workspaces_of_their_own():
    a = Case([3000, 20], [16, 4], 8, 2, 128, 16, False, True, "tree")
    b = Case([50] * 100, [4] * 100, 8, 2, 128, 16, True, True, "tree")
    want = a.run(), b.run()
    torch.cuda.synchronize()
    streams, ws = [torch.cuda.Stream() for _ in range(2)], [moe.tree_attention_workspace(128) for _ in range(2)]
    got = [[], []]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, c in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i].append(c.run(ws[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i]) and moe.device_status(ws[i]) == 0


def test_binding_refusals():
    c = Case([40], [6], 4, 1, 64, 16, False, True, "tree")
    ws = moe.tree_attention_workspace(64)
    for kw in (dict(q=c.q.cpu()), dict(q=c.q.float()), dict(q=c.q[:, :, :32]), dict(row_start=c.start[:1]), dict(row_start=c.start.long()),
               dict(seq_len=c.seq_len.cpu()), dict(mask=c.mask[:5]), dict(mask=c.mask.int()), dict(table=c.table[0]),
               dict(window=-1), dict(out=c.q[:5])):
        with pytest.raises(ValueError):
            c.run(ws, **kw)
    with pytest.raises(moe.MoEError):
        c.run(ws[: ws.numel() // 2])
    with pytest.raises(moe.MoEError):
        moe.tree_attention_workspace(96)
    with pytest.raises(moe.MoEError):
        c.run(ws, scale=float("nan"))


@pytest.mark.parametrize("falls,ctx,e4m3", [(1, 3000, False), (1, 3000, True), (38, 300, False)])
def test_rows_that_fall_leave_other_sequences_theirs(falls, ctx, e4m3):
    """A row_start that falls and rises again, so that the sequences' rows add up to more than there are: what falls has no
    rows, and the last sequence, whose rows are its own, has all of them."""
    n = 2 * falls + 1
    drafted = [64, 0] * falls + [64, 64]
    c = Case([ctx] + [0] * (n - 1) + [ctx], drafted, 16, 1, 64, 16, e4m3, True, "tree")
    last = c.T - 64
    q, mask = (torch.cat([t[:64], t[last:]]) for t in (c.q, c.mask))
    start = torch.tensor([0, 64] * (falls + 1) + [128], dtype=torch.int32).cuda()
    assert len(start) == len(c.seq_len) + 1
    ws = moe.tree_attention_workspace(64)
    out, lse = c.run(ws, q=q, mask=mask, row_start=start, out=torch.full_like(q, 5.0), return_lse=True)
    assert moe.device_status(ws) == 8
    whole, wlse = torch.zeros_like(c.q), torch.zeros(c.T, 16, device="cuda")
    whole[last:], wlse[last:] = out[64:], lse[64:]
    c.check(whole, wlse, rows=range(last, c.T))
    # and a call that is as it should be finds the workspace as it should be
    want, got = c.run(return_lse=True), c.run(ws, return_lse=True)
    assert moe.device_status(ws) == 0 and all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("ctx,drafted", [([2000, 3, 700], [16, 16, 4]), ([300] * 3 + [0] * 2, [16, 0, 1, 2, 40]), ([90] * 90, [16] * 90)])
def test_the_workspace_held_another_batch(ctx, drafted):
    """What a workspace held says nothing: here the lists of items that a batch of one cut item everywhere would leave, whose
    rows and parts all are in range."""
    c = Case(ctx, drafted, 16, 2, 128, 16, False, True, "tree")
    want, wlse = c.run(return_lse=True)
    ws = moe.tree_attention_workspace(128)
    ws[256: 256 + 304 * 24].view(torch.int32).view(304, 6).copy_(torch.tensor([0, 0, 0, 128, 0, 0], dtype=torch.int32))
    out, lse = c.run(ws, return_lse=True)
    assert moe.device_status(ws) == 0 and torch.equal(out, want) and torch.equal(lse, wlse)


@pytest.mark.parametrize("ctx", [[40, 20], [3000, 500]])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_value_rows_of_the_lowest_exponents(D, ctx):
    """Exponent bytes from 1 to 6: outputs below 2^-110, in whole items and in parts, of rows once and twice in a tile."""
    c = Case(ctx, [9, 40], 4, 1, D, 16, True, True, "tree")
    exps = c.cache.v_exp
    exps.copy_((exps.int() - 118).clamp(1, 6))
    for b, n in enumerate(c.lens):
        j = torch.arange(n, device="cuda")
        at = c.table[b].long()[j // 16], j % 16
        c.dense[1][b] = ref.e4m3_value(c.cache.v[at], exps[at])
    ws = moe.tree_attention_workspace(D)
    out, lse = c.run(ws, return_lse=True)
    assert moe.device_status(ws) == 0 and float((out == 0).float().mean()) < 0.1
    c.check(out, lse, rows=range(0, c.T, 3))


@pytest.mark.parametrize("window", [0, 150])
@pytest.mark.parametrize("D,ctx,drafted,heads,kv", [
    (64, [200, 90], [20, 13], 4, 2), (128, [200, 90], [20, 13], 4, 2), (256, [300], [40], 8, 2), (64, [5000], [50], 8, 2), (128, [5000, 64], [16, 3], 8, 2),
    (64, [130], [1], 1, 1), (128, [63], [2], 2, 1)])
def test_infinite_values(D, ctx, drafted, heads, kv, window):
    """An infinity among the values that a row sees is its output, whatever its weight and wherever it lies; with the other
    one, or NaN, the output is NaN.  All else keeps its bits."""
    c = Case(ctx, drafted, heads, kv, D, 16, False, True, "tree")
    inf, nan = float("inf"), float("nan")

    def at(key):
        return int(c.table[0, key // 16]), key % 16, 0

    n = ctx[0]
    c.cache.k[at(n - 20)] *= 300.0     # a key that takes all the weight of a row, or has none
    base, blse = c.run(window=window, return_lse=True)
    odd = [(n // 2, 3, inf), (n - 40, 7, -inf), (n // 3, 11, inf), (n - 10, 11, -inf), (n, 13, inf), (n // 4, 17, inf), (n, 17, inf),
           (n - 33, 19, nan), (n - 34, 19, inf), (n - 20, 23, inf), (n - 21, 29, -inf), (1, 31, inf), (n - 5, 31, inf)]
    for key, col, v in odd:
        c.cache.v[at(key) + (col,)] = v
    ws = moe.tree_attention_workspace(D)
    out, lse = c.run(ws, window=window, return_lse=True)
    assert moe.device_status(ws) == 0 and torch.equal(lse, blse)
    want = base.clone()
    for t in range(drafted[0]):
        keys = set(cref.seen_by(c.masks[t], drafted[0], n, window, t))
        for col in {o[1] for o in odd}:
            seen = [v for key, j, v in odd if j == col and key in keys]
            if seen:
                want[t, : heads // kv, col] = sum(seen)
    assert torch.equal(torch.isnan(out), torch.isnan(want)) and torch.equal(out.nan_to_num(0.5, inf, -inf), want.nan_to_num(0.5, inf, -inf))


def test_no_score_above_minus_infinity():
    """Zeros and -inf, whatever the values are: of keys with an infinity, in whole items and in parts."""
    for n in (150, 4000):
        c = Case([n], [5], 2, 1, 64, 16, False, True, "tree")
        c.q[..., 4] = 1.0
        c.cache.k[..., 4] = -float("inf")
        c.cache.v[..., 9] = float("inf")
        c.cache.v[..., 11] = float("nan")
        out, lse = c.run(return_lse=True)
        assert (out == 0).all() and (lse == -float("inf")).all()
