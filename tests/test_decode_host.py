"""The decoding step's operators without a GPU: argument checks of the C ABI, the rotation phases, and the plain
64-bit implementations the GPU tests rely on.  No call here reaches a kernel."""
import ctypes
import math

import numpy as np
import pytest
import torch

import decode_ref as ref
from token_level_top_gb300 import build, moe

FAKE = 0x7f0000000000  # never dereferenced: every case below is refused or has nothing to do
R = ctypes.byref


@pytest.fixture(scope="module")
def L():
    build.build()
    return moe.lib()


def _cache(**kw):
    d = dict(k=FAKE, v=FAKE, k_exp=None, v_exp=None, type=0, n_pages=4, page_size=16, n_kv_heads=2, head_dim=128,
             page_stride=4096, token_stride=128, head_stride=2048)
    d.update(kw)
    return moe.MoEKVCache(**d)


BAD_CACHES = [(dict(k=None), 1), (dict(v=None), 1), (dict(type=2), 1), (dict(n_pages=0), 1), (dict(page_size=0), 1),
              (dict(n_kv_heads=0), 1), (dict(type=1), 1), (dict(k_exp=FAKE), 1), (dict(type=1, k_exp=FAKE), 1),
              (dict(head_dim=96), 2), (dict(n_kv_heads=5000), 2), (dict(k=FAKE + 8), 3), (dict(v=FAKE + 2), 3),
              (dict(token_stride=132), 3), (dict(page_stride=4), 3), (dict(head_stride=2049), 3),
              (dict(type=1, k_exp=FAKE, v_exp=FAKE, token_stride=136), 3)]


def _append(**kw):
    d = dict(T=3, n_seqs=3, max_pages=2, n_heads=4, rot_dim=128, flags=0, pos=FAKE, seq=None, page_table=FAKE,
             table_stride=2, phase=FAKE, q=FAKE, k=FAKE, v=FAKE, q_out=FAKE, q_token_stride=512, q_head_stride=128,
             k_token_stride=256, k_head_stride=128, v_token_stride=256, v_head_stride=128, q_out_token_stride=512,
             q_out_head_stride=128)
    d.update(kw)
    return moe.MoEAppend(**d)


def test_append_refusals(L):
    for kw, st in BAD_CACHES:
        assert L.moe_kv_append(R(_cache(**kw)), R(_append()), None, None) == st, kw
    for kw, st in [(dict(T=-1), 1), (dict(n_seqs=0), 1), (dict(max_pages=0), 1), (dict(n_heads=-1), 1),
                   (dict(table_stride=-1), 1), (dict(flags=2), 1), (dict(pos=None), 1), (dict(page_table=None), 1),
                   (dict(k=None), 1), (dict(v=None), 1), (dict(phase=None), 1), (dict(q=None), 1), (dict(q_out=None), 1),
                   (dict(n_heads=0), 1), (dict(T=4), 1), (dict(rot_dim=24), 2), (dict(rot_dim=144), 2),
                   (dict(rot_dim=-16), 2), (dict(n_heads=1025), 2),
                   (dict(q_head_stride=2 ** 32), 2), (dict(v_head_stride=-2 ** 33), 2), (dict(q=FAKE + 8), 3), (dict(k=FAKE + 2), 3),
                   (dict(v=FAKE + 8), 3), (dict(q_out=FAKE + 4), 3), (dict(phase=FAKE + 8), 3),
                   (dict(k_token_stride=260), 3), (dict(q_head_stride=129), 3), (dict(q_out_token_stride=4), 3)]:
        assert L.moe_kv_append(R(_cache()), R(_append(**kw)), None, None) == st, kw
    assert L.moe_kv_append(R(_cache(head_stride=2 ** 31)), R(_append()), None, None) == 2
    assert L.moe_kv_append(None, R(_append()), None, None) == 1
    assert L.moe_kv_append(R(_cache()), None, None, None) == 1
    assert L.moe_kv_append(R(_cache()), R(_append(T=0)), None, None) == 0
    assert L.moe_kv_append(R(_cache()), R(_append(T=0, n_seqs=0, max_pages=0)), None, None) == 0


def test_attention_refusals(L):
    n = L.moe_paged_attention_workspace_size(128)
    assert n > 0 and n % 256 == 0
    assert L.moe_paged_attention_workspace_size(64) > 0 and L.moe_paged_attention_workspace_size(256) > 0
    for d in (0, -1, 32, 96, 512):
        assert L.moe_paged_attention_workspace_size(d) == 0
    P = ctypes.c_void_p

    def att(**kw):
        d = dict(B=3, n_heads=4, max_pages=2, window=0, scale=0.1, seq_len=FAKE, page_table=FAKE, table_stride=2, q=FAKE,
                 out=FAKE, lse=None, q_token_stride=512, q_head_stride=128, out_token_stride=512, out_head_stride=128)
        d.update(kw)
        return moe.MoEAttention(**d)

    def call(c, a, ws=FAKE, nb=n):
        return L.moe_paged_attention(R(c), R(a), P(ws), nb, None)

    for kw, st in BAD_CACHES:
        assert call(_cache(**kw), att()) == st, kw
    for kw, st in [(dict(B=-1), 1), (dict(n_heads=0), 1), (dict(n_heads=3), 1), (dict(max_pages=0), 1),
                   (dict(window=-1), 1), (dict(table_stride=-2), 1), (dict(scale=math.inf), 1),
                   (dict(scale=math.nan), 1), (dict(n_heads=2048), 2), (dict(seq_len=None), 1),
                   (dict(page_table=None), 1), (dict(q=None), 1), (dict(out=None), 1), (dict(q=FAKE + 2), 3),
                   (dict(out=FAKE + 8), 3), (dict(q_token_stride=4), 3), (dict(out_head_stride=100), 3)]:
        assert call(_cache(), att(**kw)) == st, kw
    for kw in (dict(page_stride=2 ** 31), dict(token_stride=2 ** 31), dict(page_stride=-8), dict(token_stride=-8)):
        assert call(_cache(**kw), att()) == 2, kw
    assert call(_cache(), att(), ws=None) == 1
    assert call(_cache(), att(), ws=FAKE + 16) == 3
    assert call(_cache(), att(), nb=n - 1) == 4
    assert call(_cache(), att(B=0)) == 0
    assert call(_cache(), att(B=0, max_pages=0)) == 0
    assert L.moe_paged_attention(None, R(att()), P(FAKE), n, None) == 1
    assert L.moe_paged_attention(R(_cache()), None, P(FAKE), n, None) == 1
    assert L.moe_paged_attention_workspace_init(None, n, None) == 1
    assert L.moe_paged_attention_workspace_init(P(FAKE + 4), n, None) == 3
    assert L.moe_paged_attention_workspace_init(P(FAKE), 16, None) == 4


def test_logprobs_refusals(L):
    P = ctypes.c_void_p

    def fwd(rows=2, vocab=10, type=0, x=FAKE, stride=10, token=FAKE, top=0, lp=FAKE, ids=None, tl=None):
        return L.moe_token_logprobs(rows, vocab, type, P(x), stride, P(token), top, P(lp), None, None, P(ids), P(tl),
                                    None, None)

    for kw, st in [(dict(rows=-1), 1), (dict(vocab=0), 1), (dict(type=2), 1), (dict(stride=-1), 1), (dict(top=-1), 1),
                   (dict(top=33), 2), (dict(rows=2 ** 31), 2), (dict(x=None), 1), (dict(token=None), 1),
                   (dict(top=2), 1), (dict(top=2, ids=FAKE), 1), (dict(x=FAKE + 2), 3), (dict(type=1, x=FAKE + 1), 3)]:
        assert fwd(**kw) == st, kw
    assert fwd(rows=0) == 0

    def bwd(rows=2, vocab=10, type=1, x=FAKE, stride=10, token=FAKE, lse=FAKE, H=FAKE, g=FAKE, h=FAKE, dx=FAKE, ds=10):
        return L.moe_token_logprobs_backward(rows, vocab, type, P(x), stride, P(token), P(lse), P(H), P(g), P(h), P(dx),
                                             ds, None, None)

    for kw, st in [(dict(rows=-1), 1), (dict(vocab=0), 1), (dict(type=5), 1), (dict(stride=-1), 1), (dict(ds=9), 1),
                   (dict(rows=2 ** 31), 2), (dict(x=None), 1), (dict(lse=None), 1), (dict(dx=None), 1), (dict(H=None), 1),
                   (dict(token=None), 1), (dict(x=FAKE + 1), 3), (dict(dx=FAKE + 3), 3), (dict(stride=12), 1)]:
        assert bwd(**kw) == st, kw
    assert bwd(rows=0) == 0


def test_binding_refusals():
    """The binding raises before the library is called (tensors of the wrong kind have no place to be checked later)."""
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        moe.KVCache(k, k)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        moe.token_logprobs(torch.zeros(2, 3, dtype=torch.float16))
    with pytest.raises(ValueError, match="logits"):
        moe.token_logprobs(torch.zeros(2, 3))
    with pytest.raises(ValueError, match="logits"):
        moe.token_logprobs_backward(torch.zeros(2, 3), None, None)
    with pytest.raises(moe.MoEError):
        moe.attention_workspace(96)
    with pytest.raises(moe.MoEError):
        moe.rope_phase([float("nan")])


def test_packed_structures_match_their_fields():
    """The binding packs a call's structure at once: the same bytes as the ctypes fields give."""
    a = _append(T=7, n_seqs=9, seq=FAKE + 64, flags=1, q_out_head_stride=77)
    v = [getattr(a, n) or 0 for n, _ in moe.MoEAppend._fields_]
    assert moe._APPEND.pack(*v) == bytes(a)
    t = moe.MoEAttention(3, 4, 5, 6, 0.25, FAKE, FAKE + 1, 8, FAKE + 2, FAKE + 3, FAKE + 4, 9, 10, 11, 12)
    v = [getattr(t, n) for n, _ in moe.MoEAttention._fields_]
    assert moe._ATTENTION.pack(*v) == bytes(t)


def test_status_strings(L):
    for code, text in moe.STATUS.items():
        assert L.moe_status_string(code).decode() == text


def test_rope_phase_against_exact_fractions():
    from fractions import Fraction
    freq = [1.0, 0.0, -0.25, 1e-12, 123.456, 10000.0 ** (-3 / 64), -1e-300, 2 * math.pi]
    got = [int(x) & (2 ** 64 - 1) for x in moe.rope_phase(freq).tolist()]
    two_pi = Fraction(628318530717958647692528676655900576, 10 ** 35)
    for f, g in zip(freq, got):
        want = Fraction(f) / two_pi % 1
        d = abs(Fraction(g, 2 ** 64) - want)
        # a division of doubles (2^-53 of the turns) by a rounded 2 pi (another 2^-53), and the cut to 2^-64
        assert min(d, 1 - d) <= abs(Fraction(f) / two_pi) * Fraction(1, 2 ** 51) + Fraction(2, 2 ** 64) + \
            (Fraction(1, 2 ** 53) if f < 0 else 0), f


def test_reference_attention_against_torch():
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(n, 16, generator=g, dtype=torch.float64) for n in (1, 50, 50))
    out, lse, _, _ = ref.attention(q[0].numpy(), k.numpy(), v.numpy(), 0.3)
    s = torch.softmax(0.3 * q @ k.T, -1) @ v
    assert np.allclose(out, s[0].numpy(), rtol=1e-12) and math.isclose(lse, torch.logsumexp(0.3 * q @ k.T, -1).item())


def test_reference_logprobs_and_gradient_against_autograd():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(4, 30, generator=g, dtype=torch.float64, requires_grad=True)
    token = torch.tensor([3, -1, 0, 29])
    logp = torch.log_softmax(x, -1)
    lp = torch.where(token >= 0, logp[torch.arange(4), token.clamp_min(0)], torch.zeros(4, dtype=torch.float64))
    H = -(logp.exp() * logp).sum(-1)
    r = ref.logprobs(x.detach().numpy(), token.numpy(), 5)
    assert np.allclose(r["logprob"], lp.detach().numpy()) and np.allclose(r["entropy"], H.detach().numpy())
    assert np.array_equal(r["top_ids"], torch.topk(x, 5).indices.numpy())
    gl, gh = torch.randn(4, generator=g, dtype=torch.float64), torch.randn(4, generator=g, dtype=torch.float64)
    ((lp * gl).sum() + (H * gh).sum()).backward()
    want, _ = ref.grad(x.detach().numpy(), token.numpy(), r["lse"], r["entropy"], gl.numpy(), gh.numpy())
    assert np.allclose(x.grad.numpy(), want, atol=1e-14)


def test_reference_e4m3_rows():
    x = torch.tensor([[448.0, 1.0], [449.0, 1.0], [0.0, 0.0], [1e-40, 0.0], [-0.4375, 0.1]])
    codes, exp = ref.e4m3_cache(x)
    assert exp.tolist() == [127, 128, 127, 1, 117]
    v = ref.e4m3_value(codes, exp)
    assert (np.abs(v - x.double().numpy()) <= ref.UE4M3 * np.abs(x.numpy()) + np.ldexp(2.0 ** -10, exp.numpy().astype(int) - 127)[:, None]).all()


def test_reference_rotation_is_a_complex_product():
    x = np.random.default_rng(0).standard_normal((3, 2, 16))
    pos, f = [0, 7, 1000], [1.0, 0.3, 0.01, 2.0]
    for inter in (False, True):
        got, _ = ref.rotate(x, pos, f, inter)
        a, b = (x[..., 0:8:2], x[..., 1:8:2]) if inter else (x[..., :4], x[..., 4:8])
        z = (a + 1j * b) * np.exp(1j * np.array(pos)[:, None, None] * np.array(f))
        u, w = (got[..., 0:8:2], got[..., 1:8:2]) if inter else (got[..., :4], got[..., 4:8])
        assert np.allclose(z.real, u) and np.allclose(z.imag, w) and np.array_equal(got[..., 8:], x[..., 8:])
