"""Several continuations at a time with one MoE decoder layer: trees of drafted tokens, and beam search.

The toy decoder of decode_step.py, with a norm before attention, experts and output head.  ``verify`` takes a tree of
drafted tokens per sequence through the decoder in one pass (cached behind each other, rotated by their depths, each
attending to its ancestors), keeps the branch that greedy decoding would have taken and caches its tokens again at their
places.  ``search`` carries beams: their pages are shared up to the one that is filling, and follow the selection.

    python examples/tree_and_beams.py            # needs the built library and a GPU
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from decode_step import Decoder, Session, moe  # noqa: E402


class NormedDecoder(Decoder):
    def __post_init__(self):
        super().__post_init__()
        g = torch.Generator(device="cuda").manual_seed(self.seed + 1)
        self.norms = [(1 + 0.1 * torch.randn(self.d, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(3)]
        self.layers = {}

    def qkv(self, x):
        return super().qkv(moe.rms_norm(x, self.norms[0])["y"])

    def rest(self, x, att):
        """Logits from the embeddings and what attention made of them, any number of rows."""
        if len(x) not in self.layers:
            cfg = moe.Config(T=len(x), d_model=self.d, E=self.experts, k=self.k, d_ff=self.d_ff, cf=float(self.experts))
            self.layers[len(x)] = cfg, moe.workspace(cfg)
        cfg, ws = self.layers[len(x)]
        s = moe.rms_norm(att.flatten(1) @ self.w_o.T, self.norms[1], residual=x)
        y = moe.layer_forward(cfg, ws, s["y"], self.w_router, self.w13, self.w2)
        return moe.rms_norm(y, self.norms[2], residual=s["sum"])["y"] @ self.head.T


class TreeSession(Session):
    """A batch of sequences that goes on by trees.  `token` is each sequence's newest token, not cached yet."""

    def __init__(self, model, prompts, room: int, **kw):
        super().__init__(model, prompts, room, **kw)
        self.tree_ws = moe.tree_attention_workspace(model.head_dim)

    def verify(self, trees):
        """trees: per sequence a list of (parent, token) of drafted tokens, parents first; parent -1 is the sequence's newest
        token.  Returns the tokens that greedy decoding yields, one list a sequence: of the drafted ones those on its way,
        and one more."""
        m, nodes, masks, depths, places, seqs, starts = self.m, [], [], [], [], [], [0]
        lens = self.len.tolist()
        for b, (newest, tree) in enumerate(zip(self.token.tolist(), trees)):
            mask, depth = [1], [0]
            for i, (parent, _) in enumerate(tree):
                mask.append(mask[parent + 1] | 2 << i)
                depth.append(depth[parent + 1] + 1)
            nodes += [newest] + [t for _, t in tree]
            masks += [v - (1 << 64) if v >> 63 else v for v in mask]
            depths += [lens[b] + d for d in depth]
            places += [lens[b] + i for i in range(len(mask))]
            seqs += [b] * len(mask)
            starts.append(len(nodes))

        def i32(v):
            return torch.tensor(v, dtype=torch.int32).cuda()

        x = m.embed[torch.tensor(nodes).cuda()]
        q, k, v = m.qkv(x)
        q = moe.kv_append(self.cache, k, v, i32(places), self.table, q=q, phase=self.phase, seq=i32(seqs), rotary=i32([depths]), status=self.ws)
        att = moe.tree_attention(self.cache, self.tree_ws, q, i32(starts), self.len + i32([1 + len(t) for t in trees]), self.table,
                                 mask=torch.tensor(masks, dtype=torch.int64).cuda())
        self.logits = m.rest(x, att)
        best = self.logits.float().argmax(-1).tolist()
        out, kept, at, of = [], [], [], []
        for b, tree in enumerate(trees):
            way, node = [], -1
            while True:
                kept.append(starts[b] + node + 1)
                at.append(lens[b] + len(way))
                of.append(b)
                way.append(best[starts[b] + node + 1])
                node = next((i for i, (parent, token) in enumerate(tree) if parent == node and token == way[-1]), None)
                if node is None:
                    break
            out.append(way)
        # the branch's tokens to their places: their depths are their positions there
        rows = torch.tensor(kept).cuda()
        moe.kv_append(self.cache, k[rows], v[rows], i32(at), self.table, phase=self.phase, seq=i32(of), status=self.ws)
        self.len += i32([len(w) for w in out])
        self.token = i32([w[-1] for w in out])
        return out

    def check(self):
        super().check()
        moe.check_device(self.tree_ws, "attention over drafted trees")


class BeamSession:
    """Beam search from one prompt per sequence."""

    def __init__(self, model, prompts, beams: int, room: int, page: int = 16, e4m3: bool = False):
        self.m, self.beams, B = model, beams, len(prompts)
        self.s = Session(model, [p for p in prompts for _ in range(beams)], room, page=page, e4m3=e4m3)
        self.scores = torch.full((B, beams), -float("inf")).cuda()
        self.scores[:, 0] = 0.0                                   # at first all beams are the same: one counts
        self.ws = moe.beam_workspace(B * beams, beams)
        self.tokens = torch.empty(B, beams, 0, dtype=torch.int32).cuda()

    def step(self):
        s, m = self.s, self.m
        x = m.embed[s.token.long()]
        q, k, v = m.qkv(x)
        q = moe.kv_append(s.cache, k, v, s.len, s.table, q=q, phase=s.phase, status=s.ws)
        s.len += 1
        self.logits = m.rest(x, moe.paged_attention(s.cache, s.ws, q, s.len, s.table))
        best = moe.beam_select(self.ws, self.logits, self.scores, self.beams)
        s.table = moe.beam_reorder(s.cache, best["parents"], s.len[:: self.beams].contiguous(), s.table, status=s.ws)
        self.scores, s.token = best["scores"], best["tokens"].flatten()
        self.tokens = torch.cat([self.tokens.gather(1, best["parents"].long()[:, :, None].expand(-1, -1, self.tokens.shape[2])),
                                 best["tokens"][:, :, None]], 2)
        return best

    def check(self):
        moe.check_device(self.s.ws, "decoding")
        moe.check_device(self.ws, "beam selection")


def main():
    model = NormedDecoder()
    g = torch.Generator().manual_seed(7)
    prompts = [torch.randint(0, model.vocab, (n,), generator=g).tolist() for n in (1, 5, 17, 40)]
    for e4m3 in (False, True):
        print("cache:", "e4m3" if e4m3 else "bf16")
        plain = TreeSession(model, prompts, room=40, e4m3=e4m3)
        known = [sum(w, []) for w in zip(*[plain.verify([[]] * len(prompts)) for _ in range(4)])]
        s = TreeSession(model, prompts, room=40, e4m3=e4m3)
        # a wrong guess and a right one for the next token, the right one's successors behind it
        got = s.verify([[(-1, (w[0] + 1) % model.vocab), (-1, w[0]), (1, w[1]), (0, w[2]), (2, w[2])] for w in known])
        print("  from trees", got, "one at a time", known)
        s.check()
        beams = BeamSession(model, prompts, beams=3, room=16, e4m3=e4m3)
        for _ in range(6):
            beams.step()
        for b, p in enumerate(prompts):
            print(f"  after {len(p)} tokens: {beams.tokens[b, 0].tolist()} ({float(beams.scores[b, 0]):.3f}), then {beams.tokens[b, 1].tolist()}")
        beams.check()


if __name__ == "__main__":
    main()
