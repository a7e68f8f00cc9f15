"""The norm, the append on several axes, attention over drafted trees and beam search without a GPU: argument checks of
the C ABI, the packed structures, and the plain implementations that the GPU tests rely on.  No call here reaches a kernel."""
import ctypes
import math

import numpy as np
import pytest
import torch

import continuation_ref as cref
from token_level_top_gb300 import build, moe

FAKE = 0x7f0000000000  # never dereferenced: every case below is refused or has nothing to do
P, R = ctypes.c_void_p, ctypes.byref


@pytest.fixture(scope="module")
def L():
    build.build()
    return moe.lib()


def _with(cls, base, kw):
    return cls(**{**base, **kw})


CACHE = dict(k=FAKE, v=FAKE, k_exp=None, v_exp=None, type=0, n_pages=4, page_size=16, n_kv_heads=2, head_dim=128,
             page_stride=4096, token_stride=128, head_stride=2048)
BAD_CACHES = [(dict(k=None), 1), (dict(type=2), 1), (dict(n_pages=0), 1), (dict(type=1), 1), (dict(k_exp=FAKE), 1),
              (dict(head_dim=96), 2), (dict(n_kv_heads=5000), 2), (dict(page_stride=-4096), 2), (dict(token_stride=-8), 2),
              (dict(k=FAKE + 8), 3), (dict(token_stride=132), 3), (dict(head_stride=2049), 3)]


def test_append_axes_refusals(L):
    base = dict(T=3, n_seqs=3, max_pages=2, n_heads=4, rot_dim=128, flags=0, pos=FAKE, seq=None, page_table=FAKE,
                table_stride=2, phase=FAKE, q=FAKE, k=FAKE, v=FAKE, q_out=FAKE, q_token_stride=512, q_head_stride=128,
                k_token_stride=256, k_head_stride=128, v_token_stride=256, v_head_stride=128, q_out_token_stride=512,
                q_out_head_stride=128)
    turn = dict(n_axes=3, rotary=FAKE, axis_stride=3, axis=FAKE)

    def call(c={}, a={}, r={}):
        return L.moe_kv_append_axes(R(_with(moe.MoEKVCache, CACHE, c)), R(_with(moe.MoEAppend, base, a)),
                                    R(_with(moe.MoERotation, turn, r)), None, None)

    for kw, st in BAD_CACHES:
        assert call(c=kw) == st, kw
    for kw, st in [(dict(T=-1), 1), (dict(pos=None), 1), (dict(rot_dim=24), 2), (dict(k=FAKE + 2), 3), (dict(phase=None), 1),
                   (dict(rot_dim=0, phase=None), 1)]:
        assert call(a=kw) == st, kw
    for kw, st in [(dict(n_axes=0), 1), (dict(n_axes=-1), 1), (dict(n_axes=5), 2), (dict(rotary=None), 1), (dict(axis_stride=-1), 1)]:
        assert call(r=kw) == st, kw
    c, a = _with(moe.MoEKVCache, CACHE, {}), _with(moe.MoEAppend, base, {})
    assert L.moe_kv_append_axes(R(c), R(a), None, None, None) == 1
    assert L.moe_kv_append_axes(R(c), None, R(_with(moe.MoERotation, turn, {})), None, None) == 1
    assert call(a=dict(T=0)) == 0


def test_tree_refusals(L):
    n = L.moe_tree_attention_workspace_size(128)
    assert n > 0 and L.moe_tree_attention_workspace_size(64) > 0 and L.moe_tree_attention_workspace_size(256) > 0
    for d in (0, -1, 32, 96, 512):
        assert L.moe_tree_attention_workspace_size(d) == 0
    base = dict(B=3, T=9, n_heads=4, max_pages=2, window=0, scale=0.1, row_start=FAKE, seq_len=FAKE, mask=None, page_table=FAKE,
                table_stride=2, q=FAKE, out=FAKE, lse=None, q_token_stride=512, q_head_stride=128, out_token_stride=512,
                out_head_stride=128)

    def call(c={}, a={}, ws=FAKE, nb=n):
        return L.moe_tree_attention(R(_with(moe.MoEKVCache, CACHE, c)), R(_with(moe.MoETreeAttention, base, a)), P(ws), nb, None)

    for kw, st in BAD_CACHES:
        assert call(c=kw) == st, kw
    for kw, st in [(dict(B=-1), 1), (dict(T=-1), 1), (dict(n_heads=0), 1), (dict(n_heads=3), 1), (dict(max_pages=0), 1),
                   (dict(window=-1), 1), (dict(table_stride=-2), 1), (dict(scale=math.inf), 1), (dict(scale=math.nan), 1),
                   (dict(n_heads=2048), 2), (dict(row_start=None), 1), (dict(seq_len=None), 1), (dict(page_table=None), 1),
                   (dict(q=None), 1), (dict(out=None), 1), (dict(q=FAKE + 2), 3), (dict(out=FAKE + 8), 3),
                   (dict(q_token_stride=4), 3), (dict(out_head_stride=100), 3)]:
        assert call(a=kw) == st, kw
    assert call(ws=None) == 1 and call(ws=FAKE + 16) == 3 and call(nb=n - 1) == 4
    assert call(a=dict(B=0)) == 0 and call(a=dict(T=0)) == 0 and call(a=dict(B=0, max_pages=0)) == 0
    assert L.moe_tree_attention(None, R(_with(moe.MoETreeAttention, base, {})), P(FAKE), n, None) == 1
    assert L.moe_tree_attention(R(_with(moe.MoEKVCache, CACHE, {})), None, P(FAKE), n, None) == 1
    assert L.moe_tree_attention_workspace_init(None, n, None) == 1
    assert L.moe_tree_attention_workspace_init(P(FAKE + 4), n, None) == 3
    assert L.moe_tree_attention_workspace_init(P(FAKE), 16, None) == 4


def test_beam_refusals(L):
    n = L.moe_beam_workspace_size(6, 4)
    assert n > 0 and L.moe_beam_workspace_size(0, 4) > 0
    for rows, k in ((-1, 4), (2 ** 31, 4), (6, 0), (6, 33)):
        assert L.moe_beam_workspace_size(rows, k) == 0

    def call(seqs=2, beams=3, vocab=10, type=0, x=FAKE, stride=10, sc=FAKE, n_=4, os_=FAKE, pa=FAKE, to=FAKE, ws=FAKE, nb=n):
        return L.moe_beam_select(seqs, beams, vocab, type, P(x), stride, P(sc), n_, P(os_), P(pa), P(to), P(ws), nb, None)

    for kw, st in [(dict(seqs=-1), 1), (dict(beams=0), 1), (dict(vocab=0), 1), (dict(type=2), 1), (dict(stride=-1), 1), (dict(n_=0), 1),
                   (dict(n_=33), 2), (dict(beams=65), 2), (dict(seqs=2 ** 30), 2), (dict(x=None), 1), (dict(sc=None), 1),
                   (dict(os_=None), 1), (dict(pa=None), 1), (dict(to=None), 1), (dict(ws=None), 1), (dict(ws=FAKE + 8), 3),
                   (dict(nb=n - 1), 4), (dict(x=FAKE + 2), 3), (dict(type=1, x=FAKE + 1), 3)]:
        assert call(**kw) == st, kw
    assert call(seqs=0) == 0
    assert L.moe_beam_workspace_init(None, n, None) == 1
    assert L.moe_beam_workspace_init(P(FAKE + 4), n, None) == 3
    assert L.moe_beam_workspace_init(P(FAKE), 16, None) == 4

    base = dict(seqs=2, beams=3, max_pages=5, parents=FAKE, parent_stride=3, seq_len=FAKE, page_table=FAKE, table_stride=5,
                page_table_out=FAKE + 4096, table_out_stride=5)

    def move(c={}, a={}):
        return L.moe_beam_reorder(R(_with(moe.MoEKVCache, CACHE, c)), R(_with(moe.MoEBeamReorder, base, a)), None, None)

    for kw, st in BAD_CACHES:
        assert move(c=kw) == st, kw
    for kw, st in [(dict(seqs=-1), 1), (dict(beams=0), 1), (dict(max_pages=-1), 1), (dict(parent_stride=-1), 1), (dict(table_stride=-1), 1),
                   (dict(beams=65), 2), (dict(parents=None), 1), (dict(seq_len=None), 1), (dict(page_table=None), 1),
                   (dict(page_table_out=None), 1), (dict(table_out_stride=4), 1), (dict(page_table_out=FAKE), 1),
                   (dict(page_table_out=FAKE + 4 * 29), 1), (dict(page_table_out=FAKE - 4 * 29), 1)]:
        assert move(a=kw) == st, kw
    assert move(a=dict(seqs=0)) == 0 and move(a=dict(max_pages=0)) == 0


def test_norm_refusals(L):
    base = dict(rows=3, cols=64, type=1, weight_type=1, eps=1e-6, x=FAKE, residual=FAKE, weight=FAKE, sum=FAKE + 4096, y=FAKE + 8192,
                codes=FAKE, scales=FAKE, x_stride=64, residual_stride=64, sum_stride=64, y_stride=64, codes_stride=64)

    def call(**kw):
        return L.moe_rms_norm(R(_with(moe.MoERmsNorm, base, kw)), None, None)

    for kw, st in [(dict(rows=-1), 1), (dict(cols=0), 1), (dict(type=2), 1), (dict(weight_type=2), 1), (dict(eps=0.0), 1),
                   (dict(eps=-1.0), 1), (dict(eps=math.nan), 1), (dict(eps=math.inf), 1), (dict(eps=1e-31), 1), (dict(x=None), 1),
                   (dict(codes=None), 1), (dict(scales=None), 1), (dict(residual=None), 1), (dict(x_stride=-1), 1),
                   (dict(residual_stride=-1), 1), (dict(sum_stride=63), 1), (dict(y_stride=0), 1), (dict(codes_stride=63), 1),
                   (dict(sum=None, y=None, codes=None, scales=None), 1), (dict(cols=16385, sum_stride=20000, y_stride=20000, codes_stride=20000), 2),
                   (dict(rows=2 ** 31), 2), (dict(x=FAKE + 1), 3), (dict(type=0, x=FAKE + 2), 3), (dict(weight=FAKE + 1), 3),
                   (dict(scales=FAKE + 2), 3), (dict(y=FAKE, y_stride=80), 1), (dict(sum=FAKE, sum_stride=80), 1), (dict(y=FAKE + 4096), 1)]:
        assert call(**kw) == st, kw
    assert call(rows=0) == 0
    assert L.moe_rms_norm(None, None, None) == 1
    n = L.moe_rms_norm_workspace_size(64)
    assert n > 0 and L.moe_rms_norm_workspace_size(0) == 0 and L.moe_rms_norm_workspace_size(16385) == 0
    grad = dict(rows=3, cols=64, type=1, dy_type=0, weight_type=1, eps=1e-6, x=FAKE, weight=FAKE, dy=FAKE, dsum=FAKE, dx=FAKE + 4096,
                dweight=FAKE, x_stride=64, dy_stride=64, dsum_stride=64, dx_stride=64)

    def back(ws=FAKE, nb=n, **kw):
        return L.moe_rms_norm_backward(R(_with(moe.MoERmsNormGrad, grad, kw)), P(ws), nb, None)

    for kw, st in [(dict(rows=-1), 1), (dict(cols=0), 1), (dict(type=2), 1), (dict(dy_type=2), 1), (dict(eps=0.0), 1), (dict(x=None), 1),
                   (dict(dy=None), 1), (dict(dx=None), 1), (dict(ws=None), 1), (dict(ws=FAKE + 8), 3), (dict(nb=n - 1), 4),
                   (dict(type=0, dy_type=1), 2), (dict(cols=16385), 2), (dict(x_stride=-1), 1), (dict(dx_stride=63), 1), (dict(dsum=FAKE + 1), 3),
                   (dict(dx=FAKE), 1), (dict(dx=FAKE, dy=FAKE + 64, dx_stride=72), 1), (dict(dweight=FAKE + 2), 3)]:
        assert back(**kw) == st, kw
    assert back(rows=0, ws=None, dweight=None) == 0
    assert L.moe_rms_norm_backward(None, P(FAKE), n, None) == 1


def test_packed_structures_match_their_fields():
    for packed, cls in ((moe._ROTATION, moe.MoERotation), (moe._TREE, moe.MoETreeAttention), (moe._REORDER, moe.MoEBeamReorder),
                        (moe._NORM, moe.MoERmsNorm), (moe._NORM_GRAD, moe.MoERmsNormGrad)):
        v = [0.5 if t is ctypes.c_float else 3 + 7 * i for i, (_, t) in enumerate(cls._fields_)]
        assert packed.pack(*v) == bytes(cls(*v)), cls


def test_binding_refuses_the_host():
    x, i = torch.zeros(4, 16), torch.zeros(4, dtype=torch.int32)
    for call in (lambda: moe.rms_norm(x), lambda: moe.rms_norm_backward(x, x, None, x), lambda: moe.beam_select(x, x, x, 2),
                 lambda: moe.beam_reorder(None, i[None], i, i[None]),
                 lambda: moe.tree_attention(None, x, torch.zeros(4, 2, 64, dtype=torch.bfloat16), i, i, i[None])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for call in (lambda: moe.rms_norm(x.half()), lambda: moe.rms_norm_backward(x, x, None, x.half()),
                 lambda: moe.beam_select(x, x.half(), x, 2)):
        with pytest.raises(ValueError, match="float32 or bfloat16"):
            call()
    for call in (lambda: moe.norm_workspace(20000), lambda: moe.tree_attention_workspace(96), lambda: moe.beam_workspace(4, 40)):
        with pytest.raises(moe.MoEError):
            call()


def test_reference_norm_against_autograd():
    g = torch.Generator().manual_seed(0)
    s, w, dy = (torch.randn(*n, generator=g, dtype=torch.float64).requires_grad_() for n in ((5, 12), (12,), (5, 12)))
    y = s * torch.rsqrt((s * s).mean(-1, keepdim=True) + 1e-3) * w
    assert np.allclose(cref.norm(s.detach().numpy(), w.detach().numpy(), 1e-3), y.detach().numpy())
    (y * dy.detach()).sum().backward()
    dx, dw, _, _ = cref.norm_grad(s.detach().numpy(), w.detach().numpy(), dy.detach().numpy(), None, 1e-3)
    assert np.allclose(dx, s.grad.numpy()) and np.allclose(dw, w.grad.numpy())


def test_reference_paths_and_windows():
    assert cref.seen_by(None, 3, 2, 0, 1) == [0, 1, 2, 3]
    assert cref.seen_by(0b101, 3, 2, 0, 2) == [0, 1, 2, 4]
    assert cref.seen_by(0b101, 3, 5, 4, 2) == [3, 4, 5, 7]
    assert cref.seen_by(0b111, 3, 5, 2, 2) == [6, 7]
    assert cref.seen_by(0, 3, 0, 0, 2) == [] and cref.seen_by(0, 3, 4, 3, 0) == [1, 2, 3]
    assert cref.seen_by(0b111, 3, -2, 0, 2) == [0]


def test_reference_beams():
    x = np.log(np.array([[0.5, 0.25, 0.25], [0.9, 0.05, 0.05]]))
    t = cref.beam_totals(x, np.log(np.array([[0.5, 0.5]])))
    assert np.allclose(np.exp(t), [[0.25, 0.125, 0.125, 0.45, 0.025, 0.025]])
    assert cref.beam_best(t[0], 4) == [3, 0, 1, 2]
    assert cref.beam_best(cref.beam_totals(x, np.array([[-np.inf, -1.0]]))[0], 9) == [3, 4, 5]
    table = [[1, 2, 3], [1, 4, 5], [1, 6, 7]]
    new, copies = cref.reorder(table, [[1, 1, 0]], [6], 4, 3)
    assert new == [[1, 4, 3], [1, 6, 5], [1, 2, 7]] and copies == [(4, 6, 2)]
    new, copies = cref.reorder(table, [[2, 2, 2]], [4], 4, 3)
    assert new == table and not copies
