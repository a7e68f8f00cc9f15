"""Attention over e4m3 caches whose value rows differ widely in size: exponents at both ends of their range, mixed within
a sequence, and rows of zeros."""
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


def _codes(shape, g):
    """e4m3 codes of rows as the append leaves them: the largest magnitude in (224, 448]."""
    x = torch.randn(*shape, generator=g)
    x *= (225 + 223 * torch.rand(*shape[:-1], 1, generator=g)) / x.abs().amax(-1, keepdim=True)
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def _run(lens, heads, kv, D, page, exponents, zero, window=0, far=False, seed=0):
    """exponents(n) -> value exponents [n, kv]; zero(n) -> which value rows are zeros [n, kv] (their exponent is 0).  far:
    keys small enough for scores within some units.  Checks outputs and lse against fp64."""
    g = torch.Generator().manual_seed(seed + heads + D)
    total = sum(-(-n // page) for n in lens) + 2
    order = torch.randperm(total, generator=g).tolist()
    table = torch.full((len(lens), max(-(-n // page) for n in lens) + 1), -1, dtype=torch.int32)
    k, v = [torch.full((total, page, kv, D), 0x7F, dtype=torch.uint8) for _ in range(2)]   # NaN where nothing lives
    ke, ve = [torch.full((total, page, kv), 255, dtype=torch.uint8) for _ in range(2)]
    dense, codes = [], []
    for b, n in enumerate(lens):
        for j in range(-(-n // page)):
            table[b, j] = order.pop()
        at = table[b].long()[torch.arange(n) // page], torch.arange(n) % page
        kc, kx = _codes((n, kv, D), g), torch.full((n, kv), -8 if not far else -12)
        vc, vx, z = _codes((n, kv, D), g), exponents(n), zero(n)
        vc[z] = torch.where(torch.rand(vc[z].shape, generator=g) < 0.5, 0, 0x80).to(torch.uint8)   # zeros of both signs
        vx = torch.where(z, 0, vx)
        k[at], v[at] = kc, vc
        ke[at], ve[at] = (kx + 127).to(torch.uint8), (vx + 127).to(torch.uint8)
        dense.append((ref.e4m3_value(kc, kx + 127), ref.e4m3_value(vc, vx + 127)))
        codes.append((ref.f64(vc.view(torch.float8_e4m3fn)), vx.numpy()))
    q = torch.randn(len(lens), heads, D, generator=g).to(torch.bfloat16)
    cache, ws = moe.KVCache(k.cuda(), v.cuda(), ke.cuda(), ve.cuda()), moe.attention_workspace(D)
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    out, lse = moe.paged_attention(cache, ws, q.cuda(), n, table.cuda(), window=window, return_lse=True)
    assert moe.device_status(ws) == 0
    again = moe.paged_attention(cache, ws, q.cuda(), n, table.cuda(), window=window)
    assert torch.equal(out, again)
    out, lse, q = ref.f64(out), ref.f64(lse), ref.f64(q)
    for b, n in enumerate(lens):
        first = max(0, n - window) if window else 0
        for h in range(heads):
            hk = h // (heads // kv)
            kd, vd = dense[b][0][first:, hk], dense[b][1][first:, hk]
            o, s, eo, es = ref.attention(q[b, h], kd, vd, D ** -0.5)
            # weights are held in 16-bit parts down to 2^-31 of the largest weight times its row's scale
            p = np.exp(D ** -0.5 * (kd @ q[b, h]) - s)
            c, x = np.abs(codes[b][0][first:, hk]), codes[b][1][first:, hk]
            some = c.max(-1) > 0
            eo = eo + (2.0 ** -31 * (p * np.ldexp(1.0, x))[some].max() * c.sum(0) if some.any() else 0.0)
            assert abs(lse[b, h] - s) <= es, ("lse", b, h, lse[b, h], s)
            worst = np.abs(out[b, h] - o) - eo
            assert (worst <= 0).all(), ("out", b, h, out[b, h][worst.argmax()], o[worst.argmax()], eo[worst.argmax()])


def _none(kv):
    return lambda n: torch.zeros(n, kv, dtype=torch.bool)


def _cycle(kv, *e):
    return lambda n: torch.tensor(e).repeat(n // len(e) + 1)[:n, None].expand(n, kv).clone()


SHAPES = [  # lens, heads, kv, D, page: every head block and head size, whole items and split ones
    ([1, 17, 64, 300], 4, 1, 64, 16), ([300, 20], 8, 1, 64, 24), ([33, 500], 16, 1, 64, 16), ([700, 16], 8, 2, 128, 16),
    ([260], 7, 1, 128, 7), ([5000, 3], 12, 1, 128, 32), ([400, 31], 8, 1, 256, 16), ([9000], 2, 1, 128, 64),
]


@pytest.mark.parametrize("lens,heads,kv,D,page", SHAPES)
@pytest.mark.parametrize("e", [(-126,), (-122,), (-105,), (110,), (-60, 60), (60, -60), (-110, 110), (110, -110),
                               (0, -3, 5, -126), (-90,) * 16 + (40,) * 16, (-90,) * 200 + (40,) * 64])
def test_value_exponents(lens, heads, kv, D, page, e):
    _run(lens, heads, kv, D, page, _cycle(kv, *e), _none(kv), seed=len(e))


@pytest.mark.parametrize("lens,heads,kv,D,page", SHAPES)
@pytest.mark.parametrize("e", [-7, -20, -28, -30, -32, -40, -120])
def test_rows_of_zeros_among_small_ones(lens, heads, kv, D, page, e):
    """A row of zeros has exponent 0, as the append stores it, whatever its neighbours' are."""
    def zero(n):
        z = torch.zeros(n, kv, dtype=torch.bool)
        z[min(5, n - 1):: 64] = True
        return z

    _run(lens, heads, kv, D, page, _cycle(kv, e, e - 1), zero, seed=-e)
    _run(lens, heads, kv, D, page, _cycle(kv, e, e - 1), zero, window=70, far=True, seed=-e)


@pytest.mark.parametrize("lens,heads,kv,D,page", SHAPES)
def test_rows_of_zeros_alone(lens, heads, kv, D, page):
    _run(lens, heads, kv, D, page, _cycle(kv, 0), lambda n: torch.ones(n, kv, dtype=torch.bool))


def test_appended_rows_of_all_sizes():
    """Values from 1e-37 to 1e30 and rows of zeros through the append and back."""
    g = torch.Generator().manual_seed(8)
    n, kv, D, page, heads = 97, 2, 128, 16, 8
    for sizes in ((1e-37,), (1e-36, 0.0), (1e-9, 0.0, 1e-8), (1e-30, 1e30), (1.0, 0.0, 1e-3)):
        scale = torch.tensor(sizes).repeat(n)[:n, None, None]
        k = torch.randn(n, kv, D, generator=g).to(torch.bfloat16).cuda()
        v = (torch.randn(n, kv, D, generator=g) * scale).to(torch.bfloat16).cuda()
        table = torch.randperm(7, generator=g).to(torch.int32)[None].cuda()
        cache, ws = moe.KVCache.empty(7, page, kv, D, e4m3=True), moe.attention_workspace(D)
        moe.kv_append(cache, k, v, torch.arange(n, dtype=torch.int32).cuda(), table, status=ws,
                      seq=torch.zeros(n, dtype=torch.int32).cuda())
        q = torch.randn(1, heads, D, generator=g).to(torch.bfloat16).cuda()
        out, lse = moe.paged_attention(cache, ws, q, torch.tensor([n], dtype=torch.int32).cuda(), table, return_lse=True)
        assert moe.device_status(ws) == 0
        j = torch.arange(n)
        at = table[0].cpu().long()[j // page], j % page
        kd, vd = [ref.e4m3_value(st.cpu()[at], ex.cpu()[at]) for st, ex in ((cache.k, cache.k_exp), (cache.v, cache.v_exp))]
        for h in range(heads):
            hk = h // (heads // kv)
            o, s, eo, es = ref.attention(ref.f64(q)[0, h], kd[:, hk], vd[:, hk], D ** -0.5)
            p = np.exp(D ** -0.5 * (kd[:, hk] @ ref.f64(q)[0, h]) - s)
            eo = eo + 2.0 ** -31 * n * (p[:, None] * np.abs(vd[:, hk])).max() * 2
            assert abs(float(lse[0, h]) - s) <= es
            assert (np.abs(ref.f64(out)[0, h] - o) <= eo).all(), (sizes, h)
