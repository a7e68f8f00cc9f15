"""The attention's head blocks and head sizes that the other tests pass over, and calls on streams of their own: beside
each other, from threads, with a workspace each."""
import threading

import pytest
import torch

import decode_ref as ref
from test_gpu_decode import _attention_case, _check_attention, _check_logprobs, _gen, _logits
from token_level_top_gb300 import build, moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    moe.lib()


SHAPES = [  # lens, heads, kv, D, page, window: 5 to 8 query heads per key head, and the counts beside them
    ([1, 0, 17, 300], 5, 1, 64, 16, 0), ([700, 33], 12, 2, 64, 24, 0), ([129, 2000, 1], 14, 2, 64, 16, 100),
    ([5000, 40], 8, 1, 64, 64, 0), ([1, 64, 65], 10, 2, 128, 16, 0), ([260, 7], 6, 1, 128, 7, 0),
    ([3001, 0, 2], 16, 2, 128, 32, 0), ([9000], 7, 1, 128, 16, 5000), ([400, 31], 8, 1, 256, 16, 0), ([500], 5, 1, 256, 24, 77),
    ([600, 90], 9, 1, 64, 16, 0), ([600, 90], 9, 1, 128, 16, 0), ([350], 11, 1, 256, 16, 0),
    ([40, 3] * 150, 8, 1, 64, 16, 0), ([130, 3] * 100, 6, 1, 128, 16, 0),
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lens,heads,kv,D,page,window", SHAPES)
def test_attention_head_counts(lens, heads, kv, D, page, window, e4m3):
    g = _gen(sum(lens) + heads + D)
    q, table, cache, dense = _attention_case(lens, heads, kv, D, page, e4m3, page != 16, g)
    ws = moe.attention_workspace(D)
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    out, lse = moe.paged_attention(cache, ws, q, n, table, window=window, return_lse=True)
    assert moe.device_status(ws) == 0
    _check_attention(out, lse, q, dense, lens, kv, window, D ** -0.5)
    out2, lse2 = moe.paged_attention(cache, ws, q, n, table, window=window, return_lse=True)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def _step(seed, e4m3, stream):
    """One decoding step on `stream`: prompts appended, attended over, logits read.  Returns what is to be checked."""
    with torch.cuda.stream(stream):
        lens, heads, kv, D, page = [70, 300, 1], 8, 2, 128, 16
        g = _gen(seed)
        q, table, cache, dense = _attention_case(lens, heads, kv, D, page, e4m3, True, g)
        ws = moe.attention_workspace(D)
        n = torch.tensor(lens, dtype=torch.int32).cuda()
        # one more token each, on a page that the table has room for, its key and value known to the reference
        new = torch.randn(2, 3, kv, D, generator=g).to(torch.bfloat16)
        pos = n.clone()
        last = [(-(-m // page) * page - m) > 0 for m in lens]     # sequences whose last page has room
        moe.kv_append(cache, new[0].cuda(), new[1].cuda(), torch.where(torch.tensor(last).cuda(), pos, -1), table, status=ws)
        out, lse = moe.paged_attention(cache, ws, q, n + torch.tensor(last, dtype=torch.int32).cuda(), table, return_lse=True)
        x, token = _logits(20, 5003, not e4m3, 0, seed)
        read = moe.token_logprobs(x, token, top=4, status=ws)
    stream.synchronize()
    assert moe.device_status(ws) == 0
    for b, has in enumerate(last):
        if has:
            for i in range(2):
                row = ref.f64(new[i][b])
                if e4m3:
                    codes, e = ref.e4m3_cache(new[i][b].float())
                    row = ref.e4m3_value(codes, e)
                dense[i][b] = torch.cat([torch.from_numpy(dense[i][b]), torch.from_numpy(row)[None]]).numpy()
    return out, lse, q, dense, [m + int(h) for m, h in zip(lens, last)], kv, x, token, read


def _check_step(out, lse, q, dense, lens, kv, x, token, read):
    _check_attention(out, lse, q, dense, lens, kv, 0, 128 ** -0.5)
    _check_logprobs(read, x, token, 4)


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_step_on_a_side_stream(e4m3):
    _check_step(*_step(3, e4m3, torch.cuda.Stream()))


def test_steps_of_threads_beside_each_other():
    """Four threads, each with a stream, a cache and a workspace of its own, several steps long."""
    got, errors = {}, []

    def run(i):
        try:
            s = torch.cuda.Stream()
            got[i] = [_step(10 * i + j, (i + j) % 2 == 1, s) for j in range(4)]
        except Exception as e:   # noqa: BLE001  (shown by the main thread)
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for steps in got.values():
        for step in steps:
            _check_step(*step)


def test_two_workspaces_at_once():
    """Calls in flight on two streams over one cache: each workspace keeps its parts, the results are those of one call."""
    lens = [5000, 300, 0, 2000]
    q, table, cache, dense = _attention_case(lens, 16, 2, 64, 16, False, True, _gen(7))
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    ws = [moe.attention_workspace(64) for _ in range(2)]
    want = moe.paged_attention(cache, ws[0], q, n, table)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        for s, w in zip(streams, ws):
            with torch.cuda.stream(s):
                outs.append(moe.paged_attention(cache, w, q, n, table))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
