"""The decoding step's operators (cache append, attention over the paged cache, token log probabilities and their
gradient) against plain 64-bit implementations, through the binding."""
import numpy as np
import pytest
import torch

import decode_ref as ref
from token_level_top_gb300 import build, moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    moe.lib()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _table(lens, page, g, spare=3):
    """Random pages for sequences of these lengths: (table int32 [n, most], pages); unused entries are -7."""
    need = [-(-n // page) for n in lens]
    total = sum(need) + spare
    order = torch.randperm(total, generator=g).tolist()
    table = torch.full((len(lens), max(1, max(need)) + 1), -7, dtype=torch.int32)
    for b, n in enumerate(need):
        for j in range(n):
            table[b, j] = order.pop()
    return table, total


def _store(pages, page, heads, tail, dtype, fill, head_major):
    if head_major:
        return torch.full((pages, heads, page, *tail), fill, dtype=dtype).transpose(1, 2)
    return torch.full((pages, page, heads, *tail), fill, dtype=dtype)


def _to_cuda(t):
    """To the device with its strides kept."""
    out = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda")
    return out.copy_(t)


# ---------------------------------------------------------------- append

APPEND = [
    # T, heads, kv, D, rot, page, e4m3, interleaved, head_major, far
    (1, 4, 1, 128, 128, 16, False, False, True, 1),
    (1, 0, 1, 64, 64, 1, False, True, False, 100),
    (7, 8, 2, 128, 128, 16, False, False, True, 50),
    (33, 5, 5, 64, 32, 24, False, True, False, 900000),
    (130, 12, 3, 256, 256, 8, False, False, False, 1000),
    (65, 6, 2, 256, 48, 7, False, False, True, 60000),
    (40, 4, 4, 128, 0, 32, False, False, True, 10),
    (1, 4, 1, 128, 128, 16, True, False, True, 3),
    (50, 8, 2, 64, 64, 16, True, False, False, 4000),
    (77, 3, 1, 128, 112, 24, True, True, True, 131072),
    (19, 2, 2, 256, 256, 64, True, True, False, 7),
    (6000, 4, 2, 64, 64, 64, True, False, True, 5000),
    (5500, 4, 1, 128, 128, 16, False, False, True, 5000),
]


@pytest.mark.parametrize("T,heads,kv,D,rot,page,e4m3,inter,hm,far", APPEND)
def test_append(T, heads, kv, D, rot, page, e4m3, inter, hm, far):
    g = _gen(T * 7 + D + rot)
    n_seqs = 1 + T // 9
    seq = torch.sort(torch.randint(0, n_seqs, (T,), generator=g)).values
    start = torch.randint(0, far, (n_seqs,), generator=g)
    pos = torch.empty(T, dtype=torch.int64)
    count = [0] * n_seqs
    for t in range(T):
        s = int(seq[t])
        pos[t] = start[s] + count[s]
        count[s] += 1
    pad = torch.zeros(T, dtype=torch.bool)
    if T > 4:
        pad[::5] = True
    width = int(pos.max()) // page + 1
    phase_freq = [10000.0 ** (-2 * i / max(rot, 1)) for i in range(rot // 2)]
    pages_needed = sorted({(int(seq[t]), int(pos[t]) // page) for t in range(T)})
    total = len(pages_needed) + 3
    order = torch.randperm(total, generator=g).tolist()
    table = torch.full((n_seqs, width), -7, dtype=torch.int32)
    for (s, j), p in zip(pages_needed, order):
        table[s, j] = p
    qkv = torch.randn(T, (heads + 2 * kv) * D, generator=g).to(torch.bfloat16).cuda()
    q = qkv[:, : heads * D].view(T, heads, D) if heads else None
    k = qkv[:, heads * D: (heads + kv) * D].view(T, kv, D)
    v = qkv[:, (heads + kv) * D:].view(T, kv, D)
    fill = 0x55 if e4m3 else 9.0
    dtype = torch.uint8 if e4m3 else torch.bfloat16
    stores = [_to_cuda(_store(total, page, kv, (D,), dtype, fill, hm)) for _ in range(2)]
    exps = [_to_cuda(_store(total, page, kv, (), torch.uint8, 99, hm)) for _ in range(2)] if e4m3 else []
    cache = moe.KVCache(*stores, *exps)
    status = moe.status_word()
    pos_in = torch.where(pad, torch.full_like(pos, -1), pos).to(torch.int32).cuda()
    phase = moe.rope_phase(phase_freq).cuda() if rot else None
    got = moe.kv_append(cache, k, v, pos_in, table.cuda(), q=q, phase=phase, seq=seq.to(torch.int32).cuda(),
                        interleaved=inter, status=status)
    assert moe.device_status(status) == 0
    live = ~pad.numpy()
    p = pos.numpy()
    if heads:
        want, mag = ref.rotate(ref.f64(q), p, phase_freq, inter)
        err = np.abs(ref.f64(got) - want)
        assert (err[live] <= ref.rotate_bound(want, mag)[live]).all()
        assert (ref.f64(got)[~live] == 0).all()
    else:
        assert got is None
    written = torch.zeros(total, page, dtype=torch.bool)
    at_page = torch.tensor([int(table[seq[t], pos[t] // page]) for t in range(T)])
    at = pos % page
    written[at_page[live], at[live]] = True
    for i, x in enumerate((k, v)):
        want, mag = ref.rotate(ref.f64(x), p, phase_freq if i == 0 else [], inter)
        if e4m3:
            codes = stores[i].cpu()[at_page, at]
            exp = exps[i].cpu()[at_page, at]
            amax = np.abs(want).max(-1)
            e = np.ceil(np.log2(amax / 448.0))
            near = np.abs(np.log2(amax / 448.0) - np.round(np.log2(amax / 448.0))) < 1e-5
            assert (near | (exp.numpy().astype(int) - 127 == e))[live].all()
            val = ref.e4m3_value(codes, exp)
            half_sub = np.ldexp(2.0 ** -10, exp.numpy().astype(int) - 127)[..., None]
            bound = ref.UE4M3 * np.abs(want) + half_sub + ref.ROT * mag
            assert (np.abs(val - want) <= bound)[live].all()
            assert (exps[i].cpu()[~written] == 99).all()
        else:
            val = ref.f64(stores[i].cpu()[at_page, at])
            bound = ref.rotate_bound(want, mag) if i == 0 else 0.0
            assert (np.abs(val - want) <= bound)[live].all()
        assert (stores[i].cpu()[~written] == fill).all(), "a place outside the tokens' own was written"


@pytest.mark.parametrize("inter", [False, True])
def test_append_far_positions(inter):
    """Positions up to 2^31 - 1: one page of 2^24 positions per table entry, so the cache stays small in heads."""
    D, page = 64, 1 << 24
    pos = torch.tensor([0, 1, 2 ** 24 + 1, 2 ** 31 - 1, 1234567890, 2 ** 30, 777777777], dtype=torch.int64)
    T = len(pos)
    freq = [1.0, 0.5, 3.0, 1e-9, 2 * np.pi, np.pi / 2, 0.0, 1e-3] * 4
    qq = torch.randn(T, 3, D, generator=_gen(5)).to(torch.bfloat16).cuda()
    k = torch.randn(T, 1, D, generator=_gen(6)).to(torch.bfloat16).cuda()
    # the table knows no page of these sequences: nothing may be written, q is rotated all the same
    table = torch.full((T, 128), -1, dtype=torch.int32).cuda()
    cache = moe.KVCache.empty(1, 4, 1, D)
    status = moe.status_word()
    # a cache of its own page size for the address arithmetic: strides say where a page lies, its size only the index
    cache.c.page_size = page
    got = moe.kv_append(cache, k, k, pos.to(torch.int32).cuda(), table, q=qq, phase=moe.rope_phase(freq).cuda(),
                        interleaved=inter, status=status)
    assert moe.device_status(status) == 8
    # the angle in exact integers: frequencies as the library holds them, products modulo a turn
    ph = [int(x) & (2 ** 64 - 1) for x in moe.rope_phase(freq).tolist()]
    turns = np.array([[((p * f) % 2 ** 64) / 2 ** 64 for f in ph] for p in pos.tolist()])
    x = ref.f64(qq)
    want, mag = ref.rotate(x, np.ones(T), [1.0] * 32, inter)
    a, b = (x[..., 0::2], x[..., 1::2]) if inter else (x[..., :32], x[..., 32:])
    c, s = np.cos(2 * np.pi * turns)[:, None], np.sin(2 * np.pi * turns)[:, None]
    u, w = a * c - b * s, a * s + b * c
    if inter:
        want[..., 0::2], want[..., 1::2] = u, w
    else:
        want[..., :32], want[..., 32:] = u, w
    assert (np.abs(ref.f64(got) - want) <= ref.rotate_bound(want, mag)).all()
    assert (cache.k.cpu() == 0).all()


def test_append_in_place_and_bad_indices():
    g = _gen(3)
    T, D = 6, 128
    q = torch.randn(T, 2, D, generator=g).to(torch.bfloat16).cuda()
    k = torch.randn(T, 1, D, generator=g).to(torch.bfloat16).cuda()
    phase = moe.rope_phase([10000.0 ** (-2 * i / D) for i in range(D // 2)]).cuda()
    table = torch.tensor([[0, 1], [2, 5], [-1, 3]], dtype=torch.int32).cuda()   # 5 and -1 are no pages of four
    pos = torch.tensor([3, 4, 9, 6, 0, 5], dtype=torch.int32).cuda()            # 9: past the table
    seq = torch.tensor([0, 1, 1, 7, 2, 2], dtype=torch.int32).cuda()            # 7: no such sequence
    cache = moe.KVCache.empty(4, 4, 1, D)
    status = moe.status_word()
    want = moe.kv_append(cache, k, k, pos, table, q=q, phase=phase, seq=seq, status=status)
    assert moe.device_status(status) == 8
    held = cache.k.cpu()
    assert held[0, 3].abs().sum() > 0 and held[3, 1].abs().sum() > 0
    held[0, 3] = 0
    held[3, 1] = 0
    assert (held == 0).all()
    out = moe.kv_append(cache, k, k, pos, table, q=q, phase=phase, seq=seq, q_out=q)
    assert out is q and torch.equal(q, want)


def test_append_e4m3_special_rows():
    """All-zero rows, the largest and smallest magnitudes, and values that are not finite."""
    D = 64
    v = torch.zeros(6, 1, D)
    v[1] = 448.0
    v[2, 0, 0], v[2, 0, 1] = 3.3e38, 1.0
    v[3, 0, :4] = torch.tensor([1e-40, -3e-39, 9e-41, 0.0])
    v[4, 0, :4] = torch.tensor([float("nan"), float("inf"), -float("inf"), 2.0])
    v[5, 0, :2] = torch.tensor([449.9, -1.0])    # rounds to 450 in bf16: the next exponent
    v = v.to(torch.bfloat16).cuda()
    cache = moe.KVCache.empty(1, 8, 1, D, e4m3=True)
    pos = torch.arange(6, dtype=torch.int32).cuda()
    q = moe.kv_append(cache, v, v, pos, torch.zeros(1, 1, dtype=torch.int32).cuda(), q=v,
                      seq=torch.zeros(6, dtype=torch.int32).cuda())
    assert ((q == v) | (q.isnan() & v.isnan())).all(), "rows of q keep their infinities"
    exp = cache.v_exp.cpu()[0, :6, 0].tolist()
    val = ref.e4m3_value(cache.v.cpu()[0, :6, 0], cache.v_exp.cpu()[0, :6, 0])
    want = ref.f64(v[:, 0])
    assert exp[0] == 127 and exp[1] == 127 and exp[3] == 1 and exp[5] == 128
    fine = np.isfinite(want)
    half_sub = np.ldexp(2.0 ** -10, np.array(exp) - 127)[:, None]
    assert (np.abs(val - want)[fine] <= (ref.UE4M3 * np.abs(want) + half_sub)[fine]).all()
    assert np.isnan(val[~fine]).all() and (~fine).sum() == 3


# ---------------------------------------------------------------- attention

ATT = [
    # lens, heads, kv, D, page, e4m3, head_major, window
    ([1], 1, 1, 64, 16, False, True, 0),
    ([1, 0, 2], 4, 1, 128, 16, False, True, 0),
    ([17], 4, 4, 256, 8, False, False, 0),
    ([129, 128, 127, 0, 16, 15], 8, 2, 128, 16, False, True, 0),
    ([1000], 32, 8, 128, 16, False, True, 0),
    ([5000, 3], 16, 1, 64, 24, False, False, 0),
    ([700, 41], 24, 2, 128, 7, False, True, 0),         # 12 query heads per key head
    ([300], 40, 1, 128, 64, False, False, 0),           # 40 of them
    ([257, 513], 18, 1, 256, 1, False, True, 0),
    ([2000, 90, 91, 1], 8, 2, 64, 128, False, False, 90),
    ([600, 5], 4, 2, 128, 24, False, True, 1),
    ([1], 1, 1, 64, 16, True, True, 0),
    ([33, 0, 1], 4, 2, 64, 16, True, False, 0),
    ([1024, 77], 16, 2, 128, 32, True, True, 0),
    ([3001], 16, 1, 128, 24, True, False, 1000),
    ([250, 2], 6, 3, 256, 8, True, True, 0),
    ([40] * 400, 4, 2, 64, 16, False, True, 0),         # many short sequences
    ([20000] + [1] * 37, 8, 2, 128, 64, False, True, 0),   # one long one among short ones
    ([9000, 8000, 10001], 4, 1, 128, 16, False, True, 0),  # parts in groups, items that share a block
    ([3001] * 5, 2, 1, 64, 32, False, False, 0),
    ([7000, 9000], 20, 2, 64, 16, True, True, 8000),
    ([12345], 16, 2, 256, 48, False, True, 0),
    ([0, 1, 0, 0, 65, 2] * 90, 6, 3, 128, 16, False, True, 0),   # runs that begin or end between items
    ([300, 1, 129] * 70, 4, 2, 64, 16, True, False, 0),
    ([777], 4, 4, 256, 16, True, True, 0),
]


def _attention_case(lens, heads, kv, D, page, e4m3, hm, g, junk=float("nan"), kscale=1.0, vscale=1.0):
    table, pages = _table(lens, page, g)
    B = len(lens)
    q = torch.randn(B, heads, D, generator=g).to(torch.bfloat16)
    dense, stores, exps = [], [], []
    for i in range(2):
        # everything outside the live positions is junk
        st = _store(pages, page, kv, (D,), torch.uint8 if e4m3 else torch.bfloat16, 0x7F if e4m3 else junk, hm)
        ex = _store(pages, page, kv, (), torch.uint8, 255, hm)
        rows = []
        for b, n in enumerate(lens):
            x = torch.randn(n, kv, D, generator=g) * (kscale if i == 0 else vscale)
            j = torch.arange(n)
            pg, at = table[b].long()[j // page], j % page
            if e4m3:
                x = x * torch.exp2(torch.randint(-3, 4, (n, kv, 1), generator=g).float())
                codes, e = ref.e4m3_cache(x)
                st[pg, at], ex[pg, at] = codes, e
                rows.append(ref.e4m3_value(codes, e))
            else:
                x = x.to(torch.bfloat16)
                st[pg, at] = x
                rows.append(ref.f64(x))
        dense.append(rows)
        stores.append(_to_cuda(st))
        exps.append(_to_cuda(ex))
    return q.cuda(), table.cuda(), moe.KVCache(*stores, *(exps if e4m3 else [])), dense


def _check_attention(out, lse, q, dense, lens, kv, window, scale):
    heads = q.shape[1]
    q, out, lse = ref.f64(q), ref.f64(out), ref.f64(lse)
    for b, n in enumerate(lens):
        first = max(0, n - window) if window else 0
        for h in range(heads):
            hk = h // (heads // kv)
            o, s, eo, es = ref.attention(q[b, h], dense[0][b][first:, hk], dense[1][b][first:, hk], scale)
            assert (np.abs(out[b, h] - o) <= eo).all(), (b, h, np.abs(out[b, h] - o).max())
            assert (lse[b, h] == s) if n == first else abs(lse[b, h] - s) <= es, (b, h, lse[b, h], s)


@pytest.mark.parametrize("lens,heads,kv,D,page,e4m3,hm,window", ATT)
def test_attention(lens, heads, kv, D, page, e4m3, hm, window):
    g = _gen(len(lens) * 31 + heads + D + page)
    q, table, cache, dense = _attention_case(lens, heads, kv, D, page, e4m3, hm, g)
    ws = moe.attention_workspace(D)
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    out, lse = moe.paged_attention(cache, ws, q, n, table, window=window, return_lse=True)
    assert moe.device_status(ws) == 0
    _check_attention(out, lse, q, dense, lens, kv, window, D ** -0.5)
    # the same again on the same workspace, to the last bit
    out2, lse2 = moe.paged_attention(cache, ws, q, n, table, window=window, return_lse=True)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_attention_large_scores_and_scale():
    """Scores in the hundreds (one key takes all the weight), a negative and a zero scale."""
    lens = [300, 77]
    q, table, cache, dense = _attention_case(lens, 8, 2, 128, 16, False, True, _gen(11), kscale=30.0)
    ws = moe.attention_workspace(128)
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    for scale in (1.0, -0.7, 0.0):
        out, lse = moe.paged_attention(cache, ws, q, n, table, scale=scale, return_lse=True)
        _check_attention(out, lse, q, dense, lens, 2, 0, scale)


def test_attention_strided_q_out_and_lse_optional():
    lens = [100, 7, 0]
    q, table, cache, dense = _attention_case(lens, 4, 2, 64, 16, False, False, _gen(12))
    ws = moe.attention_workspace(64)
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    want = moe.paged_attention(cache, ws, q, n, table)
    big = torch.zeros(3, 6, 80, dtype=torch.bfloat16, device="cuda")
    big[:, 1:5, :64] = q
    hold = torch.full((3, 4, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    got = moe.paged_attention(cache, ws, big[:, 1:5, :64], n, table, out=hold[:, :, :64])
    assert torch.equal(got, want) and (hold[:, :, 64:] == 5).all()


def test_attention_rows_without_finite_scores():
    """Infinite and NaN keys among the live ones do what the formula says; other rows are untouched."""
    lens = [64, 64, 64]
    q, table, cache, dense = _attention_case(lens, 2, 1, 64, 16, False, True, _gen(13))
    ws = moe.attention_workspace(64)
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    base = moe.paged_attention(cache, ws, q, n, table)
    q2 = q.abs()
    t = table.cpu()
    base2 = moe.paged_attention(cache, ws, q2, n, table)
    cache.k[int(t[0, 1]), 3] = -float("inf")     # score -inf: no weight
    cache.k[int(t[1, 0]), 0, 0, 5] = float("nan")
    got, lse = moe.paged_attention(cache, ws, q2, n, table, return_lse=True)
    k = np.delete(dense[0][0], 19, 0), np.delete(dense[1][0], 19, 0)
    for h in range(2):
        o, s, eo, es = ref.attention(ref.f64(q2)[0, h], k[0][:, 0], k[1][:, 0], 0.125)
        assert (np.abs(ref.f64(got)[0, h] - o) <= eo).all() and abs(float(lse[0, h]) - s) <= es
    assert torch.isnan(got[1]).all() and torch.isnan(lse[1]).all()
    assert torch.equal(got[2], base2[2])
    assert torch.isfinite(base).all()


def test_attention_bad_lengths_and_pages():
    lens = [40, 40, 40]
    q, table, cache, dense = _attention_case(lens, 4, 1, 64, 16, False, True, _gen(14))
    ws = moe.attention_workspace(64)
    t = table[:, :3].contiguous()          # three pages each: 48 positions, the last 8 of them junk
    n = torch.tensor([40, -5, 40], dtype=torch.int32).cuda()
    out, lse = moe.paged_attention(cache, ws, q, n, t, return_lse=True)
    assert moe.device_status(ws) == 8
    assert (out[1] == 0).all() and torch.isinf(lse[1]).all()
    # a page outside the cache: its keys are left out
    t2 = t.clone()
    t2[0, 1] = 10 ** 6
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    out, lse = moe.paged_attention(cache, ws, q, n, t2, return_lse=True)
    assert moe.device_status(ws) == 8
    keep = [j for j in range(40) if not 16 <= j < 32]
    dense[0][0], dense[1][0] = dense[0][0][keep], dense[1][0][keep]
    _check_attention(out, lse, q, dense, [24, 40, 40], 1, 0, 0.125)
    # longer than the table: as long as the table
    n = torch.tensor([40, 40, 10 ** 9], dtype=torch.int32).cuda()
    t3 = t[:, :2].contiguous()
    out = moe.paged_attention(cache, ws, q, n.clamp(max=32), t3)
    got = moe.paged_attention(cache, ws, q, n, t3)
    assert moe.device_status(ws) == 8
    assert torch.equal(out, got)
    # every page bad: nothing is live there
    out, lse = moe.paged_attention(cache, ws, q, n.clamp(max=32), torch.full_like(t3, -1), return_lse=True)
    assert moe.device_status(ws) == 8
    assert (out == 0).all() and (lse == -float("inf")).all()


def test_attention_in_a_graph_follows_the_lengths():
    lens = [500, 30, 900]
    q, table, cache, dense = _attention_case(lens, 8, 2, 128, 16, False, True, _gen(15))
    ws = moe.attention_workspace(128)
    n = torch.tensor([500, 30, 900], dtype=torch.int32).cuda()
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        moe.paged_attention(cache, ws, q, n, table, out=out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.paged_attention(cache, ws, q, n, table, out=out)
    for now in ([500, 30, 900], [1, 0, 899], [333, 30, 128]):
        n.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, moe.paged_attention(cache, ws, q, n, table))


def test_append_then_attention():
    """Positions written by the append are read back by the attention: one step after a prompt, both cache types."""
    g = _gen(16)
    B, heads, kv, D, page = 3, 8, 2, 128, 16
    prompt = [20, 1, 47]
    freq = [10000.0 ** (-2 * i / D) for i in range(D // 2)]
    for e4m3 in (False, True):
        table, pages = _table([n + 1 for n in prompt], page, g)
        cache = moe.KVCache.empty(pages, page, kv, D, e4m3=e4m3)
        ws, phase = moe.attention_workspace(D), moe.rope_phase(freq).cuda()
        table = table.cuda()
        total = sum(prompt)
        k = torch.randn(total + B, kv, D, generator=g).to(torch.bfloat16).cuda()
        v = torch.randn(total + B, kv, D, generator=g).to(torch.bfloat16).cuda()
        q = torch.randn(B, heads, D, generator=g).to(torch.bfloat16).cuda()
        seq = torch.repeat_interleave(torch.arange(B), torch.tensor(prompt)).to(torch.int32)
        pos = torch.cat([torch.arange(n) for n in prompt]).to(torch.int32)
        moe.kv_append(cache, k[:total], v[:total], pos.cuda(), table, phase=phase, seq=seq.cuda(), status=ws)
        last = torch.tensor(prompt, dtype=torch.int32).cuda()
        qr = moe.kv_append(cache, k[total:], v[total:], last, table, q=q, phase=phase, status=ws)
        out, lse = moe.paged_attention(cache, ws, qr, last + 1, table, return_lse=True)
        assert moe.device_status(ws) == 0
        rows = [[], []]
        for b, n in enumerate(prompt):
            j = torch.arange(n + 1)
            at = table[b].cpu().long()[j // page], j % page
            for i, st in enumerate((cache.k, cache.v)):
                st = st.cpu()[at]
                rows[i].append(ref.e4m3_value(st, (cache.k_exp, cache.v_exp)[i].cpu()[at]) if e4m3 else ref.f64(st))
            mine = [t for t in range(total) if int(seq[t]) == b] + [total + b]
            want, mag = ref.rotate(ref.f64(k)[mine], np.arange(n + 1), freq, False)
            slack = ref.UE4M3 + 2.0 ** -12 if e4m3 else ref.UBF16
            assert (np.abs(rows[0][-1] - want) <= slack * np.abs(want).max(-1, keepdims=True) + ref.ROT * mag).all()
        _check_attention(out, lse, qr, rows, [n + 1 for n in prompt], kv, 0, D ** -0.5)


# ---------------------------------------------------------------- log probabilities

LOGP = [
    # rows, vocab, bf16, top, row padding
    (1, 1, False, 1, 0), (1, 2, True, 3, 0), (3, 7, True, 7, 1), (5, 33, False, 32, 3), (2, 1000, True, 20, 0),
    (9, 4097, False, 5, 0), (4, 32000, True, 20, 0), (300, 1003, True, 1, 5), (3, 50257, True, 20, 0),
    (2, 50257, False, 32, 2), (1, 200001, True, 20, 0), (1000, 300, False, 4, 0), (17, 65536, True, 0, 0),
    (900, 3001, True, 32, 1), (800, 10239, False, 20, 0), (770, 20487, True, 0, 0), (1, 20001, False, 20, 3),
    (170, 100003, True, 20, 0), (153, 49999, False, 32, 1), (160, 98310, True, 0, 0),
]


def _logits(rows, vocab, bf16, pad, seed):
    g = _gen(seed)
    dt = torch.bfloat16 if bf16 else torch.float32
    whole = (torch.randn(rows, vocab + pad, generator=g) * 4).to(dt).cuda()
    token = torch.randint(0, vocab, (rows,), generator=g).to(torch.int32)
    token[::4] = -1
    return whole[:, :vocab], token.cuda()


def _check_logprobs(got, x, token, top):
    V = x.shape[1]
    want = ref.logprobs(ref.f64(x), None if token is None else token.cpu().numpy(), top)
    for name in ("lse", "entropy", "logprob"):
        if name not in got:
            continue
        a, b = ref.f64(got[name]), want[name]
        assert (np.isnan(a) == np.isnan(b)).all() and (a[np.isinf(b)] == b[np.isinf(b)]).all(), name
        f = np.isfinite(b)
        eb = ref.entropy_bound(b, V) if name == "entropy" else ref.lse_bound(want["lse"], V) + 4 * ref.U32 * np.abs(b)
        assert (np.abs(a - b)[f] <= eb[f]).all(), (name, np.abs(a - b)[f].max())
    if top:
        assert np.array_equal(got["top_ids"].cpu().numpy(), want["top_ids"])
        a, b = ref.f64(got["top_logprobs"]), want["top_logprobs"]
        f = np.isfinite(b)
        assert (np.isnan(a) == np.isnan(b)).all() and (a[np.isinf(b)] == b[np.isinf(b)]).all()
        eb = ref.lse_bound(want["lse"], V)[:, None] + 4 * ref.U32 * np.abs(b)
        assert (np.abs(a - b)[f] <= eb[f]).all()
    return want


@pytest.mark.parametrize("rows,vocab,bf16,top,pad", LOGP)
def test_logprobs(rows, vocab, bf16, top, pad):
    x, token = _logits(rows, vocab, bf16, pad, rows + vocab)
    status = moe.status_word()
    got = moe.token_logprobs(x, token, top=top, status=status)
    assert moe.device_status(status) == 0
    _check_logprobs(got, x, token, top)
    again = moe.token_logprobs(x, token, top=top)
    assert all(torch.equal(got[k], again[k]) for k in got)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("vocab,times", [(515, 90), (40001, 65)])
def test_logprobs_odd_rows_in_a_large_batch(vocab, times, bf16):
    """Rows of every odd kind many times over (more rows than blocks fit).  Copies of a row differ in alignment, so
    their sums may differ in the last bits; their alternatives may not."""
    x, _ = _logits(12, vocab, bf16, 3, 5)
    x = x.clone()
    x[0], x[1, 1:] = -float("inf"), -float("inf")
    x[2] = torch.finfo(x.dtype).min
    x[3] = 1.5
    x[4, : vocab // 2] = float("nan")
    x[5] = float("nan")
    x[6, 7] = float("inf")
    x[7] = torch.sort(x[7].float()).values.to(x.dtype)
    x[8] = torch.sort(x[8].float(), descending=True).values.to(x.dtype)
    x[9, vocab - 1], x[9, 0] = 99.0, 98.0
    token = (torch.arange(12) * 41 % vocab).to(torch.int32).cuda()
    token[3] = vocab + 5
    one = moe.token_logprobs(x, token, top=20)
    many = moe.token_logprobs(x.repeat(times, 1), token.repeat(times), top=20)
    keep = token.clone()
    keep[3] = -1
    _check_logprobs(one, x, keep, 20)
    ids = many["top_ids"].view(times, 12, 20)
    assert (ids == one["top_ids"]).all()
    for copy in (0, 1, times // 2, times - 1):
        _check_logprobs({name: got[12 * copy: 12 * copy + 12] for name, got in many.items()}, x, keep, 20)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("vocab", [515, 40001])
def test_logprobs_masks_ties_and_orders(vocab, bf16):
    """Rows of one value, sorted rows, banned tokens (-inf and the type's lowest), rows with nothing left."""
    dt = torch.bfloat16 if bf16 else torch.float32
    low = torch.finfo(dt).min
    x = torch.zeros(10, vocab)
    x[1] = torch.arange(vocab) / vocab * 20
    x[2] = -x[1]
    x[3, :] = -float("inf")
    x[3, 400], x[3, 7] = 2.0, 1.0
    x[4, :] = low
    x[4, 500] = 3.0
    x[5, :] = -float("inf")
    x[6, :] = low
    x[7] = torch.randint(0, 3, (vocab,), generator=_gen(9)).float()
    x[8] = torch.where(torch.arange(vocab) % 2 == 0, torch.tensor(0.0), torch.tensor(-0.0))
    x[9] = torch.randn(vocab, generator=_gen(10)) * 1e4
    x = x.to(dt).cuda()
    token = torch.tensor([0, vocab - 1, 3, 8, 2, 1, 0, -1, 5, 77], dtype=torch.int32).cuda()
    status = moe.status_word()
    got = moe.token_logprobs(x, token, top=20, status=status)
    assert moe.device_status(status) == 0
    _check_logprobs(got, x, token, 20)


@pytest.mark.parametrize("bf16", [False, True])
def test_logprobs_nan_infinity_and_bad_tokens(bf16):
    vocab = 3001
    x, _ = _logits(4, vocab, bf16, 0, 1)
    x = x.clone()
    x[0, 100] = float("nan")
    x[1, 100] = float("inf")
    token = torch.tensor([3, 4, vocab, vocab - 1], dtype=torch.int32).cuda()
    status = moe.status_word()
    got = moe.token_logprobs(x, token, top=6, status=status)
    assert moe.device_status(status) in (5, 8)
    token2 = torch.tensor([3, 4, -1, vocab - 1], dtype=torch.int32).cuda()
    _check_logprobs(got, x, token2, 6)
    got = moe.token_logprobs(x[2:], token[2:], status=status)
    assert moe.device_status(status) == 8
    got = moe.token_logprobs(x[:1], status=status)
    assert moe.device_status(status) == 5 and "logprob" not in got
    assert moe.device_status(status) == 0


@pytest.mark.parametrize("bf16", [False, True])
def test_logprobs_rows_mostly_nan(bf16):
    """Fewer numbers than alternatives: the NaNs follow, lowest index first; numbers among them rank by value."""
    dt = torch.bfloat16 if bf16 else torch.float32
    x = torch.full((3, 9001), float("nan"))
    x[0, 4000], x[0, 17], x[0, 8999] = 1.0, -float("inf"), 2.0
    x[1, 9000] = 0.5
    got = moe.token_logprobs(x.to(dt).cuda(), top=5)
    want = ref.logprobs(x.numpy().astype(np.float64), None, 5)
    assert np.array_equal(got["top_ids"].cpu().numpy(), want["top_ids"])


@pytest.mark.parametrize("split_rows", [1, 700])
def test_logprobs_many_values_above_the_threshold(split_rows):
    """Rows laid out against the threshold: 1500 distinct large values within the reach of a few threads, which
    leaves the others' maxima far below them; and thousands of ties at the n-th place."""
    vocab = 60000
    g = _gen(31)
    x = torch.randn(2, vocab, generator=g)
    for piece in range(0, 400):                       # 16-byte pieces of one column of threads
        x[0, piece * 1024: piece * 1024 + 4] += 50.0 if piece * 1024 + 4 <= vocab else 0.0
    x[0, 1024 * 3: 1024 * 3 + 2000] += 40.0
    x[1] = torch.where(torch.rand(vocab, generator=g) < 0.5, torch.tensor(3.0), torch.tensor(2.0))
    x[1, 59000:59005] = 4.0
    x = x.repeat_interleave(split_rows, 0)[: 2 * split_rows].cuda()
    got = moe.token_logprobs(x, top=32)
    rows = [0, 2 * split_rows - 1]
    want = ref.logprobs(ref.f64(x[rows]), None, 32)
    assert np.array_equal(got["top_ids"][rows].cpu().numpy(), want["top_ids"])
    assert (got["top_ids"][:split_rows] == got["top_ids"][0]).all()


def test_logprobs_of_one_row_repeated():
    x, _ = _logits(1, 5003, True, 0, 2)
    token = torch.arange(50, dtype=torch.int32).cuda()
    got = moe.token_logprobs(x.expand(50, -1), token, top=3)
    _check_logprobs(got, x.expand(50, -1), token, 3)


GRAD = [(1, 1, False, 0), (3, 7, True, 1), (5, 1000, False, 0), (4, 1003, True, 5), (33, 4099, False, 3),
        (7, 32000, True, 0), (2, 50257, False, 0), (3, 50257, True, 0), (700, 129, True, 0),
        (9, 8203, True, 1), (40, 300, False, 0), (3, 4101, False, 2)]


@pytest.mark.parametrize("rows,vocab,bf16,pad", GRAD)
def test_logprobs_backward(rows, vocab, bf16, pad):
    x, token = _logits(rows, vocab, bf16, pad, rows * 3 + vocab)
    f = moe.token_logprobs(x, token)
    g = torch.randn(rows, generator=_gen(1)).cuda()
    h = torch.randn(rows, generator=_gen(2)).cuda()
    half = (2.0 ** -8 if bf16 else 2.0 ** -24)
    for gg, hh in ((g, h), (g, None), (None, h)):
        dx = moe.token_logprobs_backward(x, token, f["lse"], f["entropy"], gg, hh)
        z = np.zeros(rows)
        want, err = ref.grad(ref.f64(x), token.cpu().numpy(), ref.f64(f["lse"]), ref.f64(f["entropy"]),
                             z if gg is None else ref.f64(gg), z if hh is None else ref.f64(hh))
        assert (np.abs(ref.f64(dx) - want) <= half * np.abs(want) + err + 1e-38).all()
    # in place, and into rows with a stride of their own
    whole = torch.full((rows, vocab + 9), 4.0, dtype=x.dtype, device="cuda")
    want = moe.token_logprobs_backward(x, token, f["lse"], f["entropy"], g, h)
    moe.token_logprobs_backward(x, token, f["lse"], f["entropy"], g, h, out=whole[:, 1: vocab + 1])
    assert torch.equal(whole[:, 1: vocab + 1], want) and (whole[:, 0] == 4).all() and (whole[:, vocab + 1:] == 4).all()
    y = x.clone()
    moe.token_logprobs_backward(y, token, f["lse"], f["entropy"], g, h, out=y)
    assert torch.equal(y, want)


def test_logprobs_backward_against_differences():
    """Central differences of the 64-bit forward: step 1e-5 leaves 1e-10 of truncation and 1e-10 of rounding."""
    rows, vocab = 3, 40
    x, token = _logits(rows, vocab, False, 0, 77)
    f = moe.token_logprobs(x, token)
    g, h = torch.randn(rows, generator=_gen(3)).cuda(), torch.randn(rows, generator=_gen(4)).cuda()
    dx = ref.f64(moe.token_logprobs_backward(x, token, f["lse"], f["entropy"], g, h))
    xn, t = ref.f64(x), token.cpu().numpy()

    def loss(y):
        r = ref.logprobs(y, t, 0)
        return r["logprob"] * ref.f64(g) + r["entropy"] * ref.f64(h)

    for i in range(vocab):
        d = np.zeros_like(xn)
        d[:, i] = 1e-5
        diff = (loss(xn + d) - loss(xn - d)) / 2e-5
        assert (np.abs(dx[:, i] - diff) <= 1e-8 + 2.0 ** -18 * (np.abs(ref.f64(g)) + 20 * np.abs(ref.f64(h)))).all()


def test_logprobs_backward_masked_rows():
    """Banned tokens get no gradient, a row with nothing left gets none at all."""
    x = torch.full((3, 300), -float("inf"), device="cuda")
    x[0, 5], x[0, 9] = 1.0, 2.0
    x[1, :] = torch.finfo(torch.float32).min
    x[1, 7] = 0.0
    token = torch.tensor([5, 7, 3], dtype=torch.int32).cuda()
    f = moe.token_logprobs(x, token)
    one = torch.ones(3, device="cuda")
    dx = moe.token_logprobs_backward(x, token, f["lse"], f["entropy"], one, one)
    assert torch.isfinite(dx).all() and (dx[2] == 0).all() and (dx[1] == 0).all()
    keep = torch.zeros(300, dtype=torch.bool, device="cuda")
    keep[5] = keep[9] = True
    assert (dx[0, ~keep] == 0).all() and dx[0, 5] != 0


def test_calls_follow_the_current_stream():
    """Results made on a side stream, with inputs made there."""
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        x, token = _logits(50, 9001, True, 0, 21)
        got = moe.token_logprobs(x, token, top=4)
    s.synchronize()
    _check_logprobs(got, x, token, 4)
