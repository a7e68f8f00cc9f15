"""Beam search's selection and the reordering of the beams' pages against plain implementations, through the binding."""
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


def _check(got, x, scores, n):
    """Against the exact totals: each place has the place's total (within the bound), candidates are distinct and real."""
    B, W = scores.shape
    V = x.shape[1]
    totals = cref.beam_totals(ref.f64(x), ref.f64(scores))
    s, p, t = ref.f64(got["scores"]), got["parents"].cpu().numpy(), got["tokens"].cpu().numpy()
    for b in range(B):
        best = cref.beam_best(totals[b], n)
        k = len(best)
        assert (s[b, k:] == -np.inf).all() and (p[b, k:] == -1).all() and (t[b, k:] == -1).all()
        assert (p[b, :k] >= 0).all() and (p[b, :k] < W).all() and (t[b, :k] >= 0).all() and (t[b, :k] < V).all()
        flat = [int(p[b, i]) * V + int(t[b, i]) for i in range(k)]
        assert len(set(flat)) == k
        want = totals[b][best]
        eps = cref.beam_eps(V, want)
        assert (np.abs(s[b, :k] - totals[b][flat]) <= eps).all()
        assert (np.abs(totals[b][flat] - want) <= 2 * eps).all()
        # where no other candidate is that near, it is this very one
        order = np.sort(totals[b])[::-1]
        for i in range(k):
            near = (i > 0 and order[i - 1] - order[i] <= 2 * eps[i]) or (i + 1 < len(order) and order[i] - order[i + 1] <= 2 * eps[i])
            assert near or flat[i] == best[i], (b, i)


@pytest.mark.parametrize("B,W,V,n,dtype,pad", [
    (1, 1, 1, 1, torch.float32, 0), (1, 1, 5, 8, torch.float32, 0), (2, 3, 7, 20, torch.bfloat16, 0), (3, 4, 1000, 8, torch.float32, 1),
    (5, 5, 50257, 10, torch.bfloat16, 0), (1, 64, 300, 32, torch.float32, 0), (2, 33, 4001, 32, torch.bfloat16, 3), (40, 8, 32000, 16, torch.float32, 0),
    (200, 4, 2000, 8, torch.float32, 0), (1, 2, 131072, 4, torch.bfloat16, 0), (130, 8, 16000, 16, torch.bfloat16, 0)])
def test_select(B, W, V, n, dtype, pad):
    g = torch.Generator().manual_seed(B + W + V + n)
    x = (3 * torch.randn(B * W, V + pad, generator=g)).to(dtype).cuda()[:, :V]
    scores = (-20 * torch.rand(B, W, generator=g)).cuda()
    ws = moe.beam_workspace(B * W, n)
    got = moe.beam_select(ws, x, scores, n)
    assert moe.device_status(ws) == 0
    _check(got, x, scores, n)
    again = moe.beam_select(ws, x, scores, n)
    assert all(torch.equal(got[k], again[k]) for k in got)


def test_dead_finished_and_masked_beams():
    g = torch.Generator().manual_seed(1)
    B, W, V, n = 5, 4, 500, 8
    x = torch.randn(B * W, V, generator=g)
    scores = -5 * torch.rand(B, W, generator=g)
    scores[0, 1:] = -float("inf")           # a search begins
    scores[1] = -float("inf")               # nothing alive
    x[2 * W + 1] = -float("inf")            # finished: one token, no cost
    x[2 * W + 1, 2] = 0.0
    x[3 * W: 4 * W, 3:] = -float("inf")     # three tokens allowed for each of four beams
    x[4 * W] = -float("inf")                # a row of nothing
    x, scores = x.cuda(), scores.cuda()
    ws = moe.beam_workspace(B * W, n)
    got = moe.beam_select(ws, x, scores, n)
    assert moe.device_status(ws) == 0
    _check(got, x, scores, n)
    assert (got["parents"][0] == 0).all() and (got["parents"][1] == -1).all()
    i = (got["parents"][2] == 1).nonzero().flatten()
    assert len(i) == 1 and int(got["tokens"][2, i]) == 2 and abs(float(got["scores"][2, i] - scores[2, 1])) <= 1e-6
    assert 0 not in got["parents"][4].tolist()


@pytest.mark.parametrize("B,W,V,dtype,live", [
    (2, 8, 78130, torch.float32, 1), (1, 2, 131072, torch.float32, 5), (3, 4, 32000, torch.bfloat16, 1), (2, 3, 131072, torch.bfloat16, 7),
    (30, 8, 40000, torch.float32, 2), (200, 8, 20000, torch.float32, 3), (1300, 1, 3000, torch.bfloat16, 1)])
def test_rows_with_few_candidates(B, W, V, dtype, live):
    """Rows read by clusters, blocks and streams of blocks with fewer tokens than places: the rest is empty, whatever the
    workspace held before."""
    g = torch.Generator(device="cuda").manual_seed(V)
    n = 8
    ws = moe.beam_workspace(B * W, n)
    x = torch.randn(B * W, V, generator=g, device="cuda").to(dtype)
    scores = -torch.rand(B, W, generator=g, device="cuda")
    moe.beam_select(ws, x, scores, n)
    few = torch.rand(B * W, generator=g, device="cuda") < 0.6
    few[0] = True
    keep = torch.randint(0, V, (B * W, live), generator=g, device="cuda")
    kept = x.gather(1, keep)
    x[few] = -float("inf")
    x.scatter_(1, keep, kept)
    got = moe.beam_select(ws, x, scores, n)
    assert moe.device_status(ws) == 0
    some = slice(0, 6)
    _check({k: t[some] for k, t in got.items()}, x[: 6 * W], scores[some], n)
    if W == 1:
        rows = few.nonzero().flatten()
        assert ((got["tokens"][rows] >= 0).sum(1) <= live).all()


def test_ties():
    """Equal totals: the lower beam, then the larger logit, then the lower token."""
    V, W, n = 64, 3, 12
    x = torch.zeros(W, V)
    x[:, 10] = x[:, 50] = x[:, 7] = 2.0
    x = x.cuda()
    got = moe.beam_select(moe.beam_workspace(W, n), x, torch.zeros(1, W).cuda(), n)
    assert got["parents"][0].tolist() == [0] * 3 + [1] * 3 + [2] * 3 + [0] * 3
    assert got["tokens"][0].tolist() == [7, 10, 50] * 3 + [0, 1, 2]
    assert torch.equal(got["scores"][0, :9], got["scores"][0, :1].expand(9))


def test_totals_a_rounding_apart():
    """Beams whose totals differ by less than fp32 holds at their size are ranked by the difference."""
    V = 100
    x = torch.zeros(4, V)
    x[:, 5] = 3.0
    scores = torch.tensor([[-100.0, -100.0, -100.0, -100.0]])
    x[1, 5] = 3.0 + 2.0 ** -20
    x[2, 5] = 3.0 + 2.0 ** -19
    got = moe.beam_select(moe.beam_workspace(4, 4), x.cuda(), scores.cuda(), 4)
    assert got["parents"][0].tolist() == [2, 1, 0, 3] and (got["tokens"] == 5).all()


def test_values_that_are_not_numbers():
    g = torch.Generator().manual_seed(2)
    x = torch.randn(6, 300, generator=g)
    x[1, 7], x[3, 0] = float("nan"), float("inf")
    scores = -torch.rand(2, 3, generator=g)
    scores[1, 1] = float("nan")
    x, scores = x.cuda(), scores.cuda()
    ws = moe.beam_workspace(6, 5)
    got = moe.beam_select(ws, x, scores, 5)
    assert moe.device_status(ws) == 5
    assert set(got["parents"][0].tolist()) <= {0, 2} and set(got["parents"][1].tolist()) == {2}
    _check(got, x, scores, 5)
    x[1, 7] = x[3, 0] = 0.0
    moe.beam_select(ws, x, scores[:1].expand(2, 3).contiguous(), 5)
    assert moe.device_status(ws) == 0


def _cache(pages, page, kv, D, e4m3, hm, g):
    shape = (pages, kv, page, D) if hm else (pages, page, kv, D)
    if e4m3:
        parts = [torch.randint(0, 126, shape, generator=g).to(torch.uint8).cuda() for _ in range(2)]
        parts += [torch.randint(100, 140, shape[:3], generator=g).to(torch.uint8).cuda() for _ in range(2)]
    else:
        parts = [torch.randn(shape, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    return moe.KVCache(*[t.transpose(1, 2) if hm else t for t in parts])


def _state(cache):
    return [t.cpu().clone() for t in (cache.k, cache.v, cache.k_exp, cache.v_exp) if t is not None]


@pytest.mark.parametrize("B,W,lens,page,kv,D,e4m3,hm", [
    (1, 1, [5], 4, 1, 64, False, True), (2, 3, [0, 9], 4, 2, 64, False, False), (3, 4, [16, 17, 31], 16, 2, 128, False, True),
    (2, 8, [7, 48], 16, 3, 256, True, True), (4, 5, [100, 1, 24, 47], 24, 1, 128, True, False), (1, 64, [90], 64, 2, 64, False, True),
    (2, 40, [3, 130], 128, 8, 128, False, True), (60, 4, [13] * 60, 1, 2, 64, False, False), (2, 33, [200, 129], 128, 4, 64, True, True)])
def test_reorder(B, W, lens, page, kv, D, e4m3, hm):
    g = torch.Generator().manual_seed(B * 100 + W + page)
    most = max(lens) // page + 3
    table = torch.full((B * W, most), -9, dtype=torch.int64)
    order, used = torch.randperm(B * (W + 2) * most, generator=g), 0
    for b, n in enumerate(lens):
        full = n // page
        for j in range(full):
            table[b * W: (b + 1) * W, j] = order[used]
            used += 1
        for j in range(full, most):
            table[b * W: (b + 1) * W, j] = order[used: used + W]
            used += W
    cache = _cache(len(order), page, kv, D, e4m3, hm, g)
    parents = torch.randint(0, W, (B, W + 2), generator=g)
    if W > 2:
        parents[-1, 1] = -1
    held = _state(cache)
    want, copies = cref.reorder(table.tolist(), parents[:, :W].tolist(), lens, page, W)
    status = moe.status_word()
    hold = torch.full((B * W, most + 1), 77, dtype=torch.int32).cuda()
    got = moe.beam_reorder(cache, parents.to(torch.int32).cuda()[:, :W], torch.tensor(lens, dtype=torch.int32).cuda(),
                           table.to(torch.int32).cuda(), out=hold[:, :most], status=status)
    assert moe.device_status(status) == 0
    assert got.cpu().tolist() == want and (hold[:, most] == 77).all()
    for src, dst, rows in copies:
        for t in held:
            t[dst, :rows] = t[src, :rows]
    assert all(torch.equal(a, b) for a, b in zip(_state(cache), held))


def test_reorder_that_changes_nothing_moves_nothing():
    g = torch.Generator().manual_seed(0)
    cache = _cache(20, 16, 2, 64, False, True, g)
    table = torch.arange(16, dtype=torch.int32).view(8, 2).cuda()
    held = _state(cache)
    lens = torch.tensor([5, 21], dtype=torch.int32).cuda()
    same = torch.arange(4, dtype=torch.int32).expand(2, 4).contiguous().cuda()
    assert torch.equal(moe.beam_reorder(cache, same, lens, table), table)
    turned = torch.tensor([[1, 2, 3, 0], [3, 2, 1, 0]], dtype=torch.int32).cuda()
    got = moe.beam_reorder(cache, turned, lens, table)
    assert got[:, 0].tolist() == [2, 4, 6, 0, 14, 12, 10, 8]
    assert got[:4, 1].tolist() == [1, 3, 5, 7] and got[4:, 1].tolist() == [15, 13, 11, 9]
    assert all(torch.equal(a, b) for a, b in zip(_state(cache), held))


def test_reorder_bad_indices():
    g = torch.Generator().manual_seed(0)
    cache, status = _cache(20, 16, 2, 64, False, True, g), moe.status_word()
    table = torch.arange(16, dtype=torch.int32).view(8, 2)
    lens = torch.tensor([5, 21], dtype=torch.int32).cuda()
    held = _state(cache)
    parents = torch.tensor([[0, 0, 4, 10 ** 6], [0, 1, 2, 3]], dtype=torch.int32)
    got = moe.beam_reorder(cache, parents.cuda(), lens, table.cuda(), status=status)
    assert moe.device_status(status) == 8
    want, copies = cref.reorder(table.tolist(), parents.tolist(), [5, 21], 16, 4)
    assert got.cpu().tolist() == want and len(copies) == 1
    for src, dst, rows in copies:
        for t in held:
            t[dst, :rows] = t[src, :rows]
    assert all(torch.equal(a, b) for a, b in zip(_state(cache), held))
    # pages that are none: nothing is copied; lengths past either end
    bad = table.clone()
    bad[0, 0], bad[6, 1] = 20, -1
    moe.beam_reorder(cache, torch.tensor([[0, 0, 0, 0], [2, 2, 2, 2]], dtype=torch.int32).cuda(), lens, bad.cuda(), status=status)
    assert moe.device_status(status) == 8
    same = torch.arange(4, dtype=torch.int32).expand(2, 4).contiguous().cuda()
    got = moe.beam_reorder(cache, same.flip(1), torch.tensor([-4, 10 ** 9], dtype=torch.int32).cuda(), table.cuda(), status=status)
    assert moe.device_status(status) == 8
    assert torch.equal(got[:4].cpu(), table[:4]) and torch.equal(got[4:].cpu(), table[4:].flip(0))
    assert all(torch.equal(a, b) for a, b in zip(_state(cache), held))


def test_select_and_reorder_in_a_graph():
    g = torch.Generator().manual_seed(5)
    B, W, V, page = 3, 4, 1000, 8
    x = (2 * torch.randn(B * W, V, generator=g)).cuda()
    scores = -torch.rand(B, W, generator=g).cuda()
    table = torch.arange(B * W * 4, dtype=torch.int32).view(B * W, 4).cuda()
    lens = torch.tensor([5, 8, 17], dtype=torch.int32).cuda()
    cache, ws = _cache(B * W * 4, page, 2, 64, False, True, g), moe.beam_workspace(B * W, 2 * W)
    out = torch.zeros_like(table)

    def step():
        got = moe.beam_select(ws, x, scores, 2 * W)
        moe.beam_reorder(cache, got["parents"][:, :W], lens, table, out=out, status=ws)
        return got

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in range(3):
        x.copy_(2 * torch.randn(B * W, V, generator=torch.Generator().manual_seed(seed)))
        before = [t.clone() for t in (cache.k, cache.v)]
        graph.replay()
        torch.cuda.synchronize()
        after = [t.clone() for t in (cache.k, cache.v, out)] + [got[k].clone() for k in got]
        cache.k.copy_(before[0])
        cache.v.copy_(before[1])
        plain = step()
        for a, b in zip(after, [cache.k, cache.v, out] + [plain[k] for k in plain]):
            assert torch.equal(a, b)
    assert moe.device_status(ws) == 0


def test_binding_refusals():
    x, scores = torch.randn(6, 50).cuda(), torch.zeros(2, 3).cuda()
    ws = moe.beam_workspace(6, 4)
    for a in ((ws, x.half(), scores, 4), (ws, x.cpu(), scores, 4), (ws, x, scores.cpu(), 4), (ws, x[:5], scores, 4),
              (ws, x, torch.zeros(3, 2).cuda().t(), 4), (ws.cpu(), x, scores, 4)):
        with pytest.raises(ValueError):
            moe.beam_select(*a)
    for a in ((ws, x, scores, 0), (ws, x, scores, 33), (ws[:512], x, scores, 4), (ws, torch.randn(130, 9).cuda(), torch.zeros(2, 65).cuda(), 4)):
        with pytest.raises(moe.MoEError):
            moe.beam_select(*a)
    cache = moe.KVCache.empty(8, 16, 1, 64)
    table, lens = torch.arange(6, dtype=torch.int32).view(6, 1).cuda(), torch.ones(2, dtype=torch.int32).cuda()
    parents = torch.zeros(2, 3, dtype=torch.int32).cuda()
    for a in ((cache, parents.cpu(), lens, table), (cache, parents.long(), lens, table), (cache, parents, lens[:1], table),
              (cache, parents, lens, table[:5])):
        with pytest.raises(ValueError):
            moe.beam_reorder(*a)
    with pytest.raises(moe.MoEError):   # in place: a row would be made of rows already new
        moe.beam_reorder(cache, parents, lens, table, out=table)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,W,V,pad", [
    (3, 8, 777, 0), (2, 64, 130, 1), (1, 8, 50257, 0), (1, 3, 131071, 0), (40, 5, 50257, 0), (150, 8, 50257, 0), (300, 8, 1001, 3), (30, 8, 131072, 1),
    (2, 4, 3, 0), (20, 8, 4096, 5)])
def test_ties_of_equal_rows_wherever_they_start(B, W, V, pad, dtype):
    """Equal rows that start at different places of 16 bytes have equal totals, whichever kernel reads them."""
    g = torch.Generator(device="cuda").manual_seed(V + B)
    n = 16
    two = (3 * torch.randn(B, 2, V, generator=g, device="cuda")).to(dtype)
    x = torch.empty(B * W, V + pad, dtype=dtype, device="cuda")[:, :V]
    kind = torch.arange(W, device="cuda") % 3 // 2     # beams 0, 1, 3, 4, .. of one row, beams 2, 5, .. of another
    x.copy_(two[:, kind].reshape(B * W, V))
    ws = moe.beam_workspace(B * W, n)
    got = moe.beam_select(ws, x, torch.zeros(B, W, device="cuda"), n)
    assert moe.device_status(ws) == 0
    s, p, t = got["scores"].cpu(), got["parents"].cpu(), got["tokens"].cpu()
    kind = kind.cpu()
    for b in range(B):
        for i in range(n - 1):
            if p[b, i + 1] < 0:
                break
            if kind[p[b, i]] == kind[p[b, i + 1]] and (x[b * W + p[b, i], t[b, i]] == x[b * W + p[b, i + 1], t[b, i + 1]]):
                # the same value of the same row: the lower beam first, of one beam the lower token
                assert s[b, i] == s[b, i + 1] and (p[b, i], t[b, i]) < (p[b, i + 1], t[b, i + 1]), (b, i)
    # the first place is the first beam of its row
    assert all(int(p[b, 0]) in (0, 2) for b in range(B))
    some = slice(0, 4)
    _check({k: v[some] for k, v in got.items()}, x[: 4 * W], torch.zeros(min(B, 4), W), n)
