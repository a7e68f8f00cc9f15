"""The root-mean-square norm, its e4m3 output and its gradient against 64-bit implementations, through the binding."""
import numpy as np
import pytest
import torch

import continuation_ref as cref
import decode_ref as ref
from token_level_top_gb300 import build, moe

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    moe.lib()


def _rows(g, n, d, dtype, pad=0, scale=1.0, at=0):
    """Rows inside wider ones, `at` values from their start, on the device."""
    return (torch.randn(n, d + pad, generator=g) * scale).to(dtype).cuda()[:, at: at + d]


CASES = [
    # rows, cols, type, weight type, residual, pad, at
    (1, 1, F32, F32, False, 0, 0), (3, 2, BF, BF, True, 0, 0), (5, 7, BF, F32, True, 3, 1), (2, 8, BF, BF, False, 8, 8),
    (9, 64, F32, BF, True, 0, 0), (17, 100, F32, F32, True, 0, 0), (1, 255, BF, BF, True, 0, 0), (33, 256, BF, None, True, 0, 0),
    (7, 257, F32, F32, False, 2, 1), (130, 512, BF, BF, True, 8, 0), (11, 1000, F32, F32, True, 8, 4), (20, 1023, BF, F32, False, 0, 0),
    (12, 1024, BF, BF, True, 0, 0), (6, 1025, F32, F32, True, 0, 0), (64, 2048, BF, BF, False, 16, 8), (5, 2049, F32, None, True, 0, 0),
    (700, 4096, BF, BF, True, 0, 0), (3, 4097, BF, BF, True, 0, 0), (4, 8192, BF, F32, True, 0, 0), (3, 8193, F32, F32, False, 0, 0),
    (2, 16384, BF, BF, True, 0, 0), (2, 16384, F32, BF, True, 0, 0), (3, 16383, F32, F32, True, 1, 0), (2, 16383, BF, BF, True, 1, 1),
    (5000, 24, BF, BF, True, 0, 0), (1300, 40, F32, F32, False, 0, 0),
]


def _check_codes(codes, scales, y, bound):
    """Codes and scale against the exact y [rows, cols] whose computed value is within `bound`."""
    top = np.abs(y).max(-1)
    sc = ref.f64(scales)
    want = np.where(top > 0, top / 448.0, 1.0)
    assert (np.abs(sc - want) <= (bound.max(-1) / 448.0 + 2 * ref.U32 * want)).all()
    v = ref.f64(codes.view(torch.float8_e4m3fn))
    q = y / sc[:, None]
    # half a step of the code (relative, and of the subnormals), and what the value before may be off
    assert (np.abs(v - q) <= ref.UE4M3 * np.abs(q) + 2.0 ** -10 + bound / sc[:, None] * 1.1 + 1e-30).all()


@pytest.mark.parametrize("rows,cols,dtype,wtype,residual,pad,at", CASES)
def test_norm(rows, cols, dtype, wtype, residual, pad, at):
    g = torch.Generator().manual_seed(rows * 3 + cols)
    x = _rows(g, rows, cols, dtype, pad, 3.0, at)
    r = _rows(g, rows, cols, dtype, pad, 2.0, at) if residual else None
    w = (1 + 0.2 * torch.randn(cols, generator=g)).to(wtype).cuda() if wtype else None
    keep = x.clone(), r.clone() if residual else None
    status = moe.status_word()
    got = moe.rms_norm(x, w, residual=r, eps=1e-5, e4m3=True, status=status)
    assert moe.device_status(status) == 0
    assert torch.equal(x, keep[0]) and (not residual or torch.equal(r, keep[1]))
    s = ref.f64(x)
    if residual:
        assert torch.equal(got["sum"], (x.float() + r.float()).to(dtype))
        s = ref.f64(got["sum"])
    else:
        assert "sum" not in got
    y = cref.norm(s, None if w is None else ref.f64(w), 1e-5)
    bound = cref.NORM * np.abs(y) + 1e-38
    assert (np.abs(ref.f64(got["y"]) - y) <= bound + cref.HALF_STEP[dtype] * np.abs(y)).all()
    _check_codes(got["codes"], got["scales"], y, bound)
    # one output at a time is the same, and so is in place
    alone = moe.rms_norm(x, w, residual=r, eps=1e-5, y=False, e4m3=True)
    assert "y" not in alone and torch.equal(alone["codes"], got["codes"]) and torch.equal(alone["scales"], got["scales"])
    if residual:
        x2, r2 = x.clone(), r.clone()
        again = moe.rms_norm(x2, w, residual=r2, eps=1e-5, out=x2, sum_out=r2)
        assert again["y"] is x2 and torch.equal(x2, got["y"]) and torch.equal(r2, got["sum"])
    else:
        x2 = x.clone()
        moe.rms_norm(x2, w, eps=1e-5, out=x2)
        assert torch.equal(x2, got["y"])


@pytest.mark.parametrize("rows,cols,dtype,wtype,residual,pad,at", CASES)
@pytest.mark.parametrize("dy32", [False, True])
def test_norm_gradient(rows, cols, dtype, wtype, residual, pad, at, dy32):
    g = torch.Generator().manual_seed(rows + 5 * cols)
    x = _rows(g, rows, cols, dtype, pad, 3.0, at)
    dy = _rows(g, rows, cols, F32 if dy32 else dtype, pad, 1.0, at)
    dsum = _rows(g, rows, cols, dtype, pad, 1.0, at) if residual else None
    w = (1 + 0.2 * torch.randn(cols, generator=g)).to(wtype).cuda() if wtype else None
    ws = moe.norm_workspace(cols)
    dx, dw = moe.rms_norm_backward(ws, x, w, dy, dsum=dsum, eps=1e-5)
    want, want_w, e, e_w = cref.norm_grad(ref.f64(x), None if w is None else ref.f64(w), ref.f64(dy),
                                          None if dsum is None else ref.f64(dsum), 1e-5)
    assert dx.dtype is dtype and dw.dtype is F32
    assert (np.abs(ref.f64(dx) - want) <= e + cref.HALF_STEP[dtype] * (np.abs(want) + e)).all()
    assert (np.abs(ref.f64(dw) - want_w) <= e_w).all()
    # the same bits again, without the weights' gradient, and in place
    dx2, dw2 = moe.rms_norm_backward(ws, x, w, dy, dsum=dsum, eps=1e-5)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    dx3, none = moe.rms_norm_backward(None, x, w, dy, dsum=dsum, eps=1e-5, weight_grad=False)
    assert none is None and torch.equal(dx, dx3)
    hold = x.clone()
    assert torch.equal(moe.rms_norm_backward(ws, hold, w, dy, dsum=dsum, eps=1e-5, out=hold)[0], dx)
    if residual:
        hold = dsum.clone()
        assert torch.equal(moe.rms_norm_backward(ws, x, w, dy, dsum=hold, eps=1e-5, out=hold)[0], dx)
    if dy.dtype is dtype:
        hold = dy.clone()
        assert torch.equal(moe.rms_norm_backward(ws, x, w, hold, dsum=dsum, eps=1e-5, out=hold)[0], dx)


@pytest.mark.parametrize("rows,cols,dtype,dy32", [
    (2500, 1501, torch.bfloat16, False), (1300, 1501, torch.bfloat16, True), (1900, 3001, torch.bfloat16, False), (1600, 1407, F32, True),
    (900, 3583, F32, True), (3001, 255, torch.bfloat16, False), (4000, 1023, torch.bfloat16, True), (700, 5001, torch.bfloat16, False)])
def test_gradient_of_many_odd_rows(rows, cols, dtype, dy32):
    """Several rows a block, taken value by value."""
    g = torch.Generator().manual_seed(rows + cols)
    x, dsum = (2 * torch.randn(rows, cols, generator=g)).to(dtype).cuda(), torch.randn(rows, cols, generator=g).to(dtype).cuda()
    dy = torch.randn(rows, cols, generator=g).to(F32 if dy32 else dtype).cuda()
    w = (1 + 0.2 * torch.randn(cols, generator=g)).cuda()
    dx, dw = moe.rms_norm_backward(moe.norm_workspace(cols), x, w, dy, dsum=dsum)
    want, want_w, e, e_w = cref.norm_grad(ref.f64(x), ref.f64(w), ref.f64(dy), ref.f64(dsum), 1e-6)
    assert (np.abs(ref.f64(dx) - want) <= e + cref.HALF_STEP[dtype] * (np.abs(want) + e)).all()
    assert (np.abs(ref.f64(dw) - want_w) <= e_w).all()
    y = moe.rms_norm(x, w, residual=dsum)
    s = ref.f64(y["sum"])
    assert (np.abs(ref.f64(y["y"]) - cref.norm(s, ref.f64(w), 1e-6)) <= (cref.HALF_STEP[dtype] * 1.01 + cref.NORM) * np.abs(cref.norm(s, ref.f64(w), 1e-6)) + 1e-38).all()


def test_gradient_against_differences():
    """The formula's gradient against differences of the 64-bit norm, so that the kernel is held to the function."""
    g = np.random.default_rng(0)
    s, w, dy = g.standard_normal((3, 10)), 1 + 0.1 * g.standard_normal(10), g.standard_normal((3, 10))
    dx, dw, _, _ = cref.norm_grad(s, w, dy, None, 1e-2)
    h = 1e-6

    def loss(s, w):
        return (cref.norm(s, w, 1e-2) * dy).sum()

    for i, j in ((0, 0), (1, 4), (2, 9)):
        d = np.zeros_like(s)
        d[i, j] = h
        assert abs((loss(s + d, w) - loss(s - d, w)) / (2 * h) - dx[i, j]) < 1e-8
        e = np.zeros(10)
        e[j] = h
        assert abs((loss(s, w + e) - loss(s, w - e)) / (2 * h) - dw[j]) < 1e-8
    got = moe.rms_norm_backward(moe.norm_workspace(10), torch.tensor(s, dtype=F32).cuda(), torch.tensor(w, dtype=F32).cuda(),
                                torch.tensor(dy, dtype=F32).cuda(), eps=1e-2)
    assert np.allclose(ref.f64(got[0]), dx, atol=1e-5) and np.allclose(ref.f64(got[1]), dw, atol=1e-5)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cols", [16, 130, 4096])
def test_values_at_the_ends_of_the_range(dtype, cols):
    """Rows of zeros, rows whose squares overflow fp32, tiny rows, NaN and infinities: each row for itself."""
    g = torch.Generator().manual_seed(cols)
    x = torch.randn(9, cols, generator=g)
    x[0] = 0.0
    x[1] *= 1e30
    x[2] = torch.sign(x[2]) * 3e38
    x[3] *= 1e-30
    x[4, 1] = float("nan")
    x[5, 0] = float("inf")
    x[6, -1] = -float("inf")
    x[7, 3] = 2e38
    x = x.to(dtype).cuda()
    status = moe.status_word()
    got = moe.rms_norm(x, eps=1e-6, e4m3=True, status=status)
    assert moe.device_status(status) == 5
    fine = [0, 1, 2, 3, 7, 8]
    y = cref.norm(ref.f64(x)[fine], None, 1e-6)
    bound = cref.NORM * np.abs(y) + 1e-38
    assert (np.abs(ref.f64(got["y"])[fine] - y) <= bound + cref.HALF_STEP[dtype] * np.abs(y)).all()
    _check_codes(got["codes"][fine], got["scales"][fine], y, bound)
    assert float(got["scales"][0]) == 1.0 and (got["codes"][0] == 0).all()
    for r in (4, 5, 6):
        assert torch.isnan(got["y"][r]).all() and torch.isnan(got["scales"][r])
        assert ((got["codes"][r] & 0x7F) == 0x7F).all()
    assert moe.device_status(status) == 0
    moe.rms_norm(x[fine], eps=1e-6, status=status)
    assert moe.device_status(status) == 0
    dy = torch.randn(9, cols, generator=g).to(dtype).cuda()
    dx, _ = moe.rms_norm_backward(None, x, None, dy, eps=1e-6, weight_grad=False)
    want, _, e, _ = cref.norm_grad(ref.f64(x)[fine], None, ref.f64(dy)[fine], None, 1e-6)
    got = ref.f64(dx)[fine]
    top = float(torch.finfo(dtype).max)
    inside = np.abs(want) < 0.99 * top
    assert (np.abs(got - want) <= e + cref.HALF_STEP[dtype] * (np.abs(want) + e) + 1e-37)[inside].all()
    assert torch.isnan(dx[[4, 5, 6]]).all()


def test_repeated_rows_and_no_rows():
    x = torch.randn(1, 96, generator=torch.Generator().manual_seed(1)).cuda()
    many = x.expand(50, 96)          # one row for all
    got = moe.rms_norm(many, residual=many, e4m3=True)
    one = moe.rms_norm(x, residual=x, e4m3=True)
    for k in got:
        assert torch.equal(got[k], one[k].expand_as(got[k]))
    dx, dw = moe.rms_norm_backward(moe.norm_workspace(96), many, None, many)
    d1, w1 = moe.rms_norm_backward(moe.norm_workspace(96), x, None, x)
    assert torch.equal(dx, d1.expand_as(dx)) and torch.allclose(dw, 50 * w1, rtol=1e-5)
    none = x[:0]
    assert moe.rms_norm(none, e4m3=True)["y"].shape == (0, 96)
    dx, dw = moe.rms_norm_backward(moe.norm_workspace(96), none, None, none)
    assert dx.shape == (0, 96) and (dw == 0).all()


def test_more_rows_than_a_grid_side():
    n = 70000 * 8 + 5
    x = torch.randn(n, 16, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").to(BF)
    y = moe.rms_norm(x)["y"]
    want = cref.norm(ref.f64(x[-1000:]), None, 1e-6)
    assert (np.abs(ref.f64(y[-1000:]) - want) <= (cref.NORM + ref.UBF16) * np.abs(want) + 1e-38).all()


def test_on_a_side_stream_and_in_a_graph():
    g = torch.Generator().manual_seed(4)
    x, r = _rows(g, 64, 512, BF), _rows(g, 64, 512, BF)
    w, ws = torch.ones(512, dtype=BF, device="cuda"), moe.norm_workspace(512)
    y, s = torch.empty_like(x), torch.empty_like(x)
    dx = torch.empty_like(x)

    def step():
        moe.rms_norm(x, w, residual=r, out=y, sum_out=s)
        return moe.rms_norm_backward(ws, s, w, y, out=dx)[1]

    want = [t.clone() for t in (step(), y, s, dx)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dw = step()
    x.add_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    replayed = [t.clone() for t in (dw, y, s, dx)]
    for a, b, c in zip(replayed, [t.clone() for t in (step(), y, s, dx)], want):
        assert torch.equal(a, b) and not torch.equal(a, c)


@pytest.mark.parametrize("dtype,dy32", [(BF, False), (BF, True), (F32, True)])
@pytest.mark.parametrize("cols", [100, 300, 520, 1000, 1001, 2000, 4096])
def test_a_row_keeps_its_bits_beside_any_neighbour(cols, dtype, dy32):
    """Rows of a block with rows whose squares overflow, or with NaN: every other row's outputs and gradient to the last bit."""
    g = torch.Generator().manual_seed(cols)
    x = torch.randn(23, cols, generator=g).to(dtype).cuda()
    dy = torch.randn(23, cols, generator=g).to(F32 if dy32 else dtype).cuda()
    w = (1 + 0.2 * torch.randn(cols, generator=g)).cuda()
    odd = x.clone()
    odd[5] *= 1e30
    odd[10, 3], odd[21, 0] = float("nan"), float("inf")
    keep = [r for r in range(23) if r not in (5, 10, 21)]
    want, got = (moe.rms_norm(t, w, e4m3=True) for t in (x, odd))
    for k in want:
        assert torch.equal(want[k][keep], got[k][keep]), k
    want, got = (moe.rms_norm_backward(None, t, w, dy, weight_grad=False)[0] for t in (x, odd))
    assert torch.equal(want[keep], got[keep])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cols,size,eps", [(16384, 2e18, 1e38), (1000, 1e19, 3e38), (16, 3e38, 3e38), (1, 1.8e19, 3.3e38), (4096, 1.0, 3e38)])
def test_eps_of_any_size(cols, size, eps, dtype):
    """An eps that counts beside squares whose sum overflows."""
    g = torch.Generator().manual_seed(cols)
    x = (size * (0.25 + 0.75 * torch.rand(5, cols, generator=g))).to(dtype).cuda()
    y = cref.norm(ref.f64(x), None, eps)
    got = moe.rms_norm(x, eps=eps)["y"]
    assert (np.abs(ref.f64(got) - y) <= (cref.NORM + cref.HALF_STEP[dtype]) * np.abs(y) + 1e-38).all()
    dy = torch.randn(5, cols, generator=g).to(dtype).cuda()
    dsum = torch.zeros(5, cols, dtype=dtype, device="cuda")
    dx, dw = moe.rms_norm_backward(moe.norm_workspace(cols), x, None, dy, dsum=dsum, eps=eps)
    want, want_w, e, e_w = cref.norm_grad(ref.f64(x), None, ref.f64(dy), None, eps)
    # (dx is below the smallest normal number of fp32, or near it: to a step of the subnormal ones of either type)
    assert (np.abs(ref.f64(dx) - want) <= e + cref.HALF_STEP[dtype] * (np.abs(want) + e) + (2.0 ** -134 if dtype is BF else 2.0 ** -148)).all()
    assert (np.abs(ref.f64(dw) - want_w) <= e_w).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cols", [260, 500, 520, 1000, 1001, 2000, 257])
def test_ends_of_the_range_where_rows_share_a_block(dtype, cols):
    """Two and four warps a row, vector rows and odd ones: the nine rows fill blocks of two or four and one in part."""
    test_values_at_the_ends_of_the_range(dtype, cols)


@pytest.mark.parametrize("rows,cols,dtype,dy32", [
    (9001, 520, BF, True), (8003, 1000, BF, False), (7001, 1000, BF, True), (4001, 2048, BF, True), (3501, 1600, BF, False), (12001, 256, BF, True),
    (9001, 260, F32, True), (8001, 512, F32, True), (5003, 1000, F32, True), (2003, 4096, F32, True), (1201, 8192, BF, True), (901, 5120, BF, False)])
def test_gradient_of_many_aligned_rows(rows, cols, dtype, dy32):
    """Several passes of the grid over vector rows: the sums' buffers in turn, and dw carried from row to row."""
    test_gradient_of_many_odd_rows(rows, cols, dtype, dy32)
