"""Decoding with one MoE decoder layer: paged cache, attention, experts, log probabilities.

A toy decoder (random weights; embedding, one layer of attention and MoE FFN with
residuals, output head) takes a batch of prompts of different lengths through
the library: the prompts' keys and values go into the cache in one call, then each
step appends the new token, attends over the cache, runs the MoE layer and reads
the next tokens, their log probabilities and the alternatives off the logits.

    python examples/decode_step.py            # needs the built library and a GPU
"""
from __future__ import annotations

import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from token_level_top_gb300 import moe  # noqa: E402


@dataclass
class Decoder:
    """Weights (bf16, on the device) and shapes."""
    d: int = 512
    heads: int = 8
    kv_heads: int = 2
    head_dim: int = 64
    experts: int = 8
    k: int = 2
    d_ff: int = 1024
    vocab: int = 1000
    seed: int = 0

    def __post_init__(self):
        g = torch.Generator(device="cuda").manual_seed(self.seed)

        def w(*shape, fan):
            return (torch.randn(*shape, generator=g, device="cuda") * fan ** -0.5).to(torch.bfloat16)

        d, hd = self.d, self.head_dim
        self.embed = w(self.vocab, d, fan=1)
        self.w_qkv = w((self.heads + 2 * self.kv_heads) * hd, d, fan=d)
        self.w_o = w(d, self.heads * hd, fan=self.heads * hd)
        self.w_router = w(self.experts, d, fan=d)
        self.w13 = moe.pack_w13(w(self.experts, self.d_ff, d, fan=d), w(self.experts, self.d_ff, d, fan=d))
        self.w2 = w(self.experts, d, self.d_ff, fan=self.d_ff)
        self.head = w(self.vocab, d, fan=d)
        self.inv_freq = [10000.0 ** (-2 * i / hd) for i in range(hd // 2)]

    def qkv(self, x):
        """q, k, v as views of one projection's output."""
        n, hq, hk, hd = x.shape[0], self.heads, self.kv_heads, self.head_dim
        y = x @ self.w_qkv.T
        return (y[:, : hq * hd].view(n, hq, hd), y[:, hq * hd: (hq + hk) * hd].view(n, hk, hd),
                y[:, (hq + hk) * hd:].view(n, hk, hd))


class Session:
    """A batch of sequences with its cache: pages are handed out in the order that sequences need them."""

    def __init__(self, model: Decoder, prompts, room: int, page: int = 16, e4m3: bool = False):
        self.m = model
        B = len(prompts)
        most = max(len(p) for p in prompts) + room
        per_seq = -(-most // page)
        self.cache = moe.KVCache.empty(B * per_seq, page, model.kv_heads, model.head_dim, e4m3=e4m3)
        order = torch.randperm(B * per_seq, generator=torch.Generator().manual_seed(1))
        self.table = order.to(torch.int32).view(B, per_seq).cuda()
        self.phase = moe.rope_phase(model.inv_freq).cuda()
        self.ws = moe.attention_workspace(model.head_dim)      # its first word also takes the other calls' status
        self.cfg = moe.Config(T=B, d_model=model.d, E=model.experts, k=model.k, d_ff=model.d_ff, cf=float(model.experts))
        self.layer_ws = moe.workspace(self.cfg)
        # the prompts but their last tokens, in one ragged call: only their keys and values are needed
        lens = [len(p) - 1 for p in prompts]
        if sum(lens):
            seq = torch.repeat_interleave(torch.arange(B), torch.tensor(lens)).to(torch.int32).cuda()
            pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32).cuda()
            ids = torch.tensor([t for p in prompts for t in p[:-1]]).cuda()
            _, k, v = model.qkv(model.embed[ids])
            moe.kv_append(self.cache, k, v, pos, self.table, phase=self.phase, seq=seq, status=self.ws)
        self.len = torch.tensor(lens, dtype=torch.int32).cuda()
        self.token = torch.tensor([p[-1] for p in prompts], dtype=torch.int32).cuda()

    def step(self, top: int = 5):
        """One new token per sequence: (next tokens, their log probabilities, alternatives as moe.token_logprobs)."""
        m = self.m
        x = m.embed[self.token.long()]
        q, k, v = m.qkv(x)
        q = moe.kv_append(self.cache, k, v, self.len, self.table, q=q, phase=self.phase, status=self.ws)
        self.len += 1
        att = moe.paged_attention(self.cache, self.ws, q, self.len, self.table)
        x = x + att.flatten(1) @ m.w_o.T
        x = x + moe.layer_forward(self.cfg, self.layer_ws, x, m.w_router, m.w13, m.w2)
        logits = x @ m.head.T
        ids = logits.float().argmax(-1).to(torch.int32)
        read = moe.token_logprobs(logits, ids, top=top, status=self.ws)
        self.token = ids
        return ids, read["logprob"], read, logits

    def check(self):
        """Raises if a kernel recorded an error (an index out of range, a NaN)."""
        moe.check_device(self.ws, "decoding")
        moe.check_device(self.layer_ws, "MoE layer")


def main():
    model = Decoder()
    g = torch.Generator().manual_seed(7)
    prompts = [torch.randint(0, model.vocab, (n,), generator=g).tolist() for n in (1, 5, 17, 40)]
    for e4m3 in (False, True):
        s = Session(model, prompts, room=12, e4m3=e4m3)
        print("cache:", "e4m3" if e4m3 else "bf16")
        for i in range(4):
            ids, lp, read, _ = s.step()
            print(f"  step {i}: tokens {ids.tolist()}  logprob {[round(v, 3) for v in lp.tolist()]}  "
                  f"second {read['top_ids'][:, 1].tolist()}  entropy {[round(v, 2) for v in read['entropy'].tolist()]}")
        s.check()


if __name__ == "__main__":
    main()
