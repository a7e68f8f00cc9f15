"""The binding of the decoding step's operators refuses what their kernels could not read: memory of the host or too
little of it, tensors of another type, rank or length.  No call below reaches a kernel but the valid ones."""
import pytest
import torch

from token_level_top_gb300 import build, moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def s():
    build.build()
    d = dict(cache=moe.KVCache.empty(4, 16, 2, 64), ws=moe.attention_workspace(64), status=moe.status_word(),
             k=torch.randn(3, 2, 64, device="cuda").to(torch.bfloat16), q=torch.randn(3, 4, 64, device="cuda").to(torch.bfloat16),
             pos=torch.zeros(3, dtype=torch.int32, device="cuda"), n=torch.ones(3, dtype=torch.int32, device="cuda"),
             table=torch.arange(3, dtype=torch.int32, device="cuda")[:, None], x=torch.randn(5, 33, device="cuda"),
             token=torch.arange(5, dtype=torch.int32, device="cuda"), phase=moe.rope_phase([0.5] * 32).cuda())
    d.update(moe.token_logprobs(d["x"], d["token"]))
    return d


BAD_STATUS = [torch.zeros(64, dtype=torch.int32), lambda t: t[:0], lambda t: t.view(torch.uint8)[2:10], lambda t: t.view(torch.uint8)[:2],
              lambda t: t[:1].expand(64), lambda t: t[::2]]


@pytest.mark.parametrize("i", range(len(BAD_STATUS)))
def test_status_words(s, i):
    bad = BAD_STATUS[i] if isinstance(BAD_STATUS[i], torch.Tensor) else BAD_STATUS[i](s["status"])
    for call in (lambda: moe.kv_append(s["cache"], s["k"], s["k"], s["pos"], s["table"], status=bad),
                 lambda: moe.token_logprobs(s["x"], s["token"], status=bad),
                 lambda: moe.token_logprobs_backward(s["x"], s["token"], s["lse"], status=bad)):
        with pytest.raises(ValueError, match="status"):
            call()


def test_workspaces(s):
    def call(ws):
        return moe.paged_attention(s["cache"], ws, s["q"], s["n"], s["table"])
    n = s["ws"].numel()
    for bad in (torch.zeros(n, dtype=torch.uint8), torch.zeros(1, dtype=torch.uint8, device="cuda").expand(n),
                torch.zeros(2 * n, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError, match="ws"):
            call(bad)
    with pytest.raises(moe.MoEError, match="workspace"):
        call(s["ws"][: n // 2])
    assert call(s["ws"]).shape == s["q"].shape
    assert moe.device_status(s["ws"]) == 0


@pytest.mark.parametrize("name", ["k", "v", "pos", "table", "q", "phase", "seq", "q_out"])
def test_append_arguments_on_the_host(s, name):
    a = dict(k=s["k"], v=s["k"], pos=s["pos"], table=s["table"], q=s["q"], phase=s["phase"], seq=s["pos"], q_out=torch.empty_like(s["q"]))
    a[name] = a[name].cpu()
    with pytest.raises(ValueError, match="CUDA device"):
        moe.kv_append(s["cache"], a["k"], a["v"], a["pos"], a["table"], q=a["q"], phase=a["phase"], seq=a["seq"], q_out=a["q_out"])


@pytest.mark.parametrize("name", ["q", "n", "table", "out"])
def test_attention_arguments_on_the_host(s, name):
    a = dict(q=s["q"], n=s["n"], table=s["table"], out=torch.empty_like(s["q"]))
    a[name] = a[name].cpu()
    with pytest.raises(ValueError, match="CUDA device"):
        moe.paged_attention(s["cache"], s["ws"], a["q"], a["n"], a["table"], out=a["out"])


@pytest.mark.parametrize("name", ["x", "token", "lse", "entropy", "g", "h", "out"])
def test_logprob_arguments_on_the_host(s, name):
    a = dict(x=s["x"], token=s["token"], lse=s["lse"], entropy=s["entropy"], g=s["lse"], h=s["lse"], out=torch.empty_like(s["x"]))
    a[name] = a[name].cpu()
    with pytest.raises(ValueError, match="CUDA device"):
        moe.token_logprobs_backward(a["x"], a["token"], a["lse"], a["entropy"], a["g"], a["h"], out=a["out"])
    if name in ("x", "token"):
        with pytest.raises(ValueError, match="CUDA device"):
            moe.token_logprobs(a["x"], a["token"])


def test_caches_of_two_places(s):
    c = s["cache"]
    with pytest.raises(ValueError, match="CUDA device"):
        moe.KVCache(c.k, c.v.cpu())
    with pytest.raises(ValueError, match="CUDA device"):
        moe.KVCache(c.k.cpu(), c.v)
    e = moe.KVCache.empty(4, 16, 2, 64, e4m3=True)
    with pytest.raises(ValueError, match="device"):
        moe.KVCache(e.k, e.v, e.k_exp, e.v_exp.cpu())
