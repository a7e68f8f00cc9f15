"""Log probabilities of rows whose values are far from the usual: finite masks of every size, rows around large
values.  Log probabilities are held to a bound that does not grow with the row's lse."""
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


def _check(got, x, token, top, where):
    """Against fp64.  A log probability is z - ln l, z = x - max: the relative error of l, and the roundings of z (two:
    its own and, in units of log2, that of log2 e), of the logarithm (two) and of the difference."""
    V, xs = x.shape[1], ref.f64(x)
    want = ref.logprobs(xs, token.cpu().numpy(), top)
    log_l = want["lse"] - xs.max(-1)
    with np.errstate(invalid="ignore"):
        # (lse swallows ln l where the maximum is large: -ln p of the maximum itself)
        log_l = np.where(np.isfinite(xs.max(-1)), -ref.logprobs(xs, xs.argmax(-1), 0)["logprob"], log_l)

    def near(a, b, bound, name):
        assert (np.isnan(a) == np.isnan(b)).all(), (name, where)
        far = np.isinf(b)
        assert (a[far] == b[far]).all(), (name, where)
        worst = np.where(far | np.isnan(b), 0.0, np.abs(np.where(far, 0, a) - np.where(far, 0, b)) - bound)
        at = np.unravel_index(worst.argmax(), worst.shape)
        assert worst[at] <= 0, (name, where, at, a[at], b[at])

    eps = ref.logprob_eps(V)
    with np.errstate(invalid="ignore"):
        def bound(lp, ll):
            return eps + 4 * ref.U32 * (np.abs(lp) + 2 * np.abs(ll))

        near(ref.f64(got["logprob"]), want["logprob"], bound(want["logprob"], log_l), "logprob")
        near(ref.f64(got["entropy"]), want["entropy"], ref.entropy_bound(want["entropy"], V), "entropy")
        near(ref.f64(got["lse"]), want["lse"], ref.lse_bound(want["lse"], V), "lse")
        if top:
            assert np.array_equal(got["top_ids"].cpu().numpy(), want["top_ids"]), where
            near(ref.f64(got["top_logprobs"]), want["top_logprobs"], bound(want["top_logprobs"], log_l[:, None]), "top")


def _low(dt):
    return torch.finfo(dt).min


MASKS = [-1e4, -1e9, -1e10, -1e12, -1e15, -1e20, -1e29, -1e30, -1e31, -1e32, -1e37, -1e38]
# rows are 4 layouts of 14 masks each; every launch's own: vocabulary, how often the rows come, alternatives
LAUNCHES = [(33, 1, 5), (515, 1, 20), (50257, 1, 20), (50257, 1, 0), (98317, 4, 5), (515, 15, 20), (3001, 15, 0),
            (40001, 15, 20)]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("vocab,times,top", LAUNCHES)
def test_finite_masks(vocab, times, top, bf16):
    """Masked by finite values of every size: nine in ten at random, the first half, all but the last, all."""
    dt = torch.bfloat16 if bf16 else torch.float32
    g = torch.Generator().manual_seed(vocab + top)
    masks = MASKS + [_low(dt) / 2, _low(dt)]
    rows, token = [], []
    for mask in masks:
        x = torch.randn(4, vocab, generator=g) * 3
        banned = torch.zeros(4, vocab, dtype=torch.bool)
        banned[0] = torch.rand(vocab, generator=g) < 0.9
        banned[1, : vocab // 2] = True
        banned[2, : vocab - 1] = True
        banned[3] = True
        rows.append(x.masked_fill(banned, mask))
        token += [int((~banned[0]).nonzero()[0]) if not banned[0].all() else 0, vocab - 2, vocab - 1, vocab // 3]
    x = torch.cat(rows).to(dt).cuda()
    token = torch.tensor(token, dtype=torch.int32).cuda()
    n = len(x)
    status = moe.status_word()
    got = moe.token_logprobs(x.repeat(times, 1), token.repeat(times), top=top, status=status)
    assert moe.device_status(status) == 0
    for copy in sorted({0, times - 1}):
        _check({k: v[n * copy: n * copy + n] for k, v in got.items()}, x, token, top, (copy, masks))


OFFSETS = [0.0, 100.7, 1000.3, -1000.3, 9999.7, 65000.5, -65000.5, 1e6, -1e6, 1.6e7, 2.0 ** 24, -2.0 ** 24, 3e7, 1e9, 1e12,
           -1e20, 1e30, -2e37, 1e38]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("vocab,times,top", LAUNCHES)
def test_rows_around_large_values(vocab, times, top, bf16):
    """Rows spread by some steps of the type around values of every size, in random and in ascending order (the maximum
    rises with every piece)."""
    dt = torch.bfloat16 if bf16 else torch.float32
    g = torch.Generator().manual_seed(vocab * 3 + top)
    step = torch.finfo(dt).eps
    x = torch.cat([c + torch.randn(1, vocab, generator=g, dtype=torch.float64) * max(1.0, abs(c) * step * 2) for c in OFFSETS])
    x = x.to(dt)
    x = torch.cat([x, torch.sort(x.float(), dim=1).values.to(dt)]).cuda()
    n, times = len(x), 1 if times == 1 else 2 * times
    token = torch.randint(0, vocab, (n,), generator=g).to(torch.int32).cuda()
    status = moe.status_word()
    got = moe.token_logprobs(x.repeat(times, 1), token.repeat(times), top=top, status=status)
    assert moe.device_status(status) == 0
    for copy in sorted({0, times - 1}):
        _check({k: v[n * copy: n * copy + n] for k, v in got.items()}, x, token, top, (copy, OFFSETS))
