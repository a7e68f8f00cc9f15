"""examples/decode_step.py: the decoding operators and the MoE layer together, against a plain dense decoder."""
import importlib.util
import os
import sys

import pytest
import torch

from token_level_top_gb300 import build, moe

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_step.py")
    spec = importlib.util.spec_from_file_location("decode_step", path)
    m = sys.modules["decode_step"] = importlib.util.module_from_spec(spec)   # dataclasses look it up there
    spec.loader.exec_module(m)
    return m


def _rotated(x, pos, inv_freq):
    th = pos.double()[:, None, None] * torch.tensor(inv_freq, dtype=torch.float64, device=x.device)
    a, b = x.double().chunk(2, -1)
    return torch.cat([a * th.cos() - b * th.sin(), a * th.sin() + b * th.cos()], -1)


@pytest.mark.parametrize("e4m3", [False, True])
def test_steps_against_a_dense_decoder(e4m3):
    build.build()
    ex = _example()
    model = ex.Decoder()
    g = torch.Generator().manual_seed(3)
    prompts = [torch.randint(0, model.vocab, (n,), generator=g).tolist() for n in (1, 33, 16, 90, 2)]
    s = ex.Session(model, prompts, room=8, e4m3=e4m3)
    texts = [list(p) for p in prompts]
    for _ in range(4):
        before = [t[:] for t in texts]
        ids, lp, read, logits = s.step(top=4)
        s.check()
        # the same step densely: keys and values of the whole text from the same projections, in fp64
        rows = []
        for b, t in enumerate(before):
            q, k, v = model.qkv(model.embed[torch.tensor(t).cuda()])
            pos = torch.arange(len(t)).cuda()
            q, k, v = _rotated(q, pos, model.inv_freq)[-1], _rotated(k, pos, model.inv_freq), v.double()
            rep = model.heads // model.kv_heads
            p = torch.softmax(torch.einsum("hd,nhd->hn", q, k.repeat_interleave(rep, 1)) * model.head_dim ** -0.5, -1)
            rows.append(torch.einsum("hn,nhd->hd", p, v.repeat_interleave(rep, 1)).flatten())
        att = torch.stack(rows).to(torch.bfloat16)
        x = model.embed[torch.tensor([t[-1] for t in before]).cuda()]
        x = x + att @ model.w_o.T
        x = x + moe.layer_forward(s.cfg, s.layer_ws, x, model.w_router, model.w13, model.w2)
        want = (x @ model.head.T).double()
        # bf16 values carried through two projections, the experts and the head: a few roundings of 2^-8 (an e4m3
        # cache: 2^-4 of a value's own, averaged over the dimensions and keys) relative to logits of unit scale
        rel = float((logits.double() - want).norm() / want.norm())
        assert rel < (0.08 if e4m3 else 0.03), rel
        logp = torch.log_softmax(logits.double(), -1)
        assert torch.allclose(lp.double(), logp.gather(1, ids.long()[:, None])[:, 0], atol=1e-5)
        assert torch.equal(read["top_ids"][:, 0], ids)
        assert torch.allclose(read["entropy"].double(), -(logp.exp() * logp).sum(-1), atol=1e-4)
        for b, t in enumerate(texts):
            t.append(int(ids[b]))
    assert s.len.tolist() == [len(t) - 1 for t in texts]


def test_example_runs(capsys):
    build.build()
    _example().main()
    assert "cache: e4m3" in capsys.readouterr().out
