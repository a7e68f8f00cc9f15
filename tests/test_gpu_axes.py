"""Cache append with positions of rotation apart from the places, on one to four axes."""
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


def _turned(x, turns, rot, inter):
    """x [T, H, D] fp64 turned by turns [T, rot / 2] -> (values, magnitude of each value's pair)."""
    want, mag = x.copy(), np.abs(x)
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., : rot // 2], x[..., rot // 2: rot])
    c, s = np.cos(2 * np.pi * turns)[:, None], np.sin(2 * np.pi * turns)[:, None]
    u, w, m = a * c - b * s, a * s + b * c, np.hypot(a, b)
    if inter:
        want[..., 0:rot:2], want[..., 1:rot:2], mag[..., 0:rot:2], mag[..., 1:rot:2] = u, w, m, m
    else:
        want[..., : rot // 2], want[..., rot // 2: rot], mag[..., : rot // 2], mag[..., rot // 2: rot] = u, w, m, m
    return want, mag


@pytest.mark.parametrize("T,heads,kv,D,rot,page,e4m3,inter,axes", [
    (1, 4, 1, 64, 64, 16, False, False, 1), (7, 2, 1, 64, 32, 4, True, True, 3), (40, 8, 2, 128, 128, 16, False, False, 3),
    (33, 6, 3, 128, 112, 24, True, False, 2), (65, 4, 2, 256, 256, 64, False, True, 4), (300, 0, 2, 128, 128, 16, True, False, 3),
    (6000, 4, 2, 64, 48, 128, False, False, 3)])
def test_append_axes(T, heads, kv, D, rot, page, e4m3, inter, axes):
    g = torch.Generator().manual_seed(T + D + axes)
    pages = -(-T // page) + 1
    table = torch.randperm(pages, generator=g).to(torch.int32)[None].cuda()
    x = [torch.randn(T, n, D, generator=g).to(torch.bfloat16).cuda() if n else None for n in (heads, kv, kv)]
    slot = torch.arange(T, dtype=torch.int32)
    slot[3::11] = -1                                            # padding
    far = torch.randint(-2 ** 31, 2 ** 31 - 1, (axes + 1, T), generator=g).to(torch.int32)
    far[:, 0] = torch.tensor([0, -1, 2 ** 31 - 1, -2 ** 31, 5][: axes + 1], dtype=torch.int32)
    rotary = far.cuda()[:axes]
    axis = torch.randint(0, axes, (rot // 2,), generator=g).to(torch.uint8)
    freq = [10000.0 ** (-2 * i / rot) for i in range(rot // 2)]
    phase = moe.rope_phase(freq)
    cache, status = moe.KVCache.empty(pages, page, kv, D, e4m3=e4m3), moe.status_word()
    seq = torch.zeros(T, dtype=torch.int32).cuda()
    got = moe.kv_append(cache, x[1], x[2], slot.cuda(), table, q=x[0], phase=phase.cuda(), seq=seq, interleaved=inter,
                        rotary=rotary, axis=axis.cuda(), status=status)
    assert moe.device_status(status) == 0
    # angles in exact integers, modulo a turn
    ph = [int(v) & (2 ** 64 - 1) for v in phase.tolist()]
    at = far.tolist()
    turns = np.array([[(at[int(axis[i])][t] * ph[i] % 2 ** 64) / 2 ** 64 for i in range(rot // 2)] for t in range(T)])
    live = (slot >= 0).numpy()
    if heads:
        want, mag = _turned(ref.f64(x[0]), turns, rot, inter)
        assert (np.abs(ref.f64(got) - want) <= ref.rotate_bound(want, mag))[live].all()
        assert (ref.f64(got)[~live] == 0).all()
    pos = slot.clamp_min(0).long()
    where = table.cpu()[0].long()[pos // page], pos % page
    for name, y in (("k", x[1]), ("v", x[2])):
        want, mag = _turned(ref.f64(y), turns, rot, inter) if name == "k" else (ref.f64(y), np.abs(ref.f64(y)))
        held = getattr(cache, name).cpu()[where]
        if e4m3:
            exp = getattr(cache, name + "_exp").cpu()[where]
            half = np.ldexp(2.0 ** -10, exp.numpy().astype(int) - 127)[..., None]
            ok = np.abs(ref.e4m3_value(held, exp) - want) <= ref.UE4M3 * np.abs(want) + half + ref.ROT * mag
        else:
            ok = np.abs(ref.f64(held) - want) <= ref.rotate_bound(want, mag)
        assert ok[live].all()
    # without the map every pair goes by the first axis; one axis equal to the places is the plain call
    one = moe.kv_append(cache, x[1], x[2], slot.cuda(), table, q=x[0], phase=phase.cuda(), seq=seq, interleaved=inter,
                        rotary=rotary)
    k1 = cache.k.clone()
    zero = moe.kv_append(cache, x[1], x[2], slot.cuda(), table, q=x[0], phase=phase.cuda(), seq=seq, interleaved=inter,
                         rotary=rotary, axis=torch.zeros(rot // 2, dtype=torch.uint8).cuda())
    assert torch.equal(k1, cache.k) and (not heads or torch.equal(one, zero))
    plain = moe.kv_append(cache, x[1], x[2], slot.cuda(), table, q=x[0], phase=phase.cuda(), seq=seq, interleaved=inter)
    k1 = cache.k.clone()
    same = moe.kv_append(cache, x[1], x[2], slot.cuda(), table, q=x[0], phase=phase.cuda(), seq=seq, interleaved=inter,
                         rotary=slot.cuda()[None])
    assert torch.equal(k1, cache.k) and (not heads or torch.equal(plain, same))


def test_an_axis_that_is_not_there():
    """It is recorded, and its pairs are not turned."""
    g = torch.Generator().manual_seed(0)
    q = torch.randn(5, 2, 64, generator=g).to(torch.bfloat16).cuda()
    k = torch.randn(5, 1, 64, generator=g).to(torch.bfloat16).cuda()
    cache, status = moe.KVCache.empty(1, 8, 1, 64), moe.status_word()
    pos = torch.arange(5, dtype=torch.int32).cuda()
    phase = moe.rope_phase([0.3] * 16).cuda()
    axis = torch.zeros(16, dtype=torch.uint8)
    axis[3], axis[7] = 1, 255
    got = moe.kv_append(cache, k, k, pos, torch.zeros(1, 1, dtype=torch.int32).cuda(), q=q, phase=phase,
                        seq=torch.zeros(5, dtype=torch.int32).cuda(), rotary=(pos + 9)[None], axis=axis.cuda(), status=status)
    assert moe.device_status(status) == 8
    for i in (3, 7):
        assert torch.equal(got[..., [i, i + 16]], q[..., [i, i + 16]])
    assert not torch.equal(got[..., 4], q[..., 4])
    assert torch.equal(got[..., 32:], q[..., 32:])


def test_refusals():
    g = torch.Generator().manual_seed(0)
    k = torch.randn(5, 1, 64, generator=g).to(torch.bfloat16).cuda()
    cache, pos = moe.KVCache.empty(1, 8, 1, 64), torch.arange(5, dtype=torch.int32).cuda()
    table, phase = torch.zeros(5, 1, dtype=torch.int32).cuda(), moe.rope_phase([0.3] * 16).cuda()
    axis = torch.zeros(16, dtype=torch.uint8).cuda()

    def call(**kw):
        return moe.kv_append(cache, k, k, pos, table, **{**dict(phase=phase, rotary=pos[None], axis=axis), **kw})

    call()
    for kw in (dict(rotary=pos), dict(rotary=pos[None, :4]), dict(rotary=pos[None].long()), dict(rotary=pos[None].cpu()),
               dict(axis=axis[:15]), dict(axis=axis.int()), dict(axis=axis.cpu()), dict(phase=None, axis=None),
               dict(rotary=None), dict(rotary=pos[None].expand(2, 5).t().contiguous().t())):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(moe.MoEError):
        call(rotary=pos[None].expand(5, 5))
    call(rotary=pos[None].expand(4, 5))
