"""Layer norm, forward and backward, against its formulas in 64 bits (gpu).

Tolerances, in u = 2^-24 (half a step of fp32) and the output type's own half
step: a sum of n fp32 terms in a tree of depth d is off by at most d u times
the sum of the terms' magnitudes, and every other operation by u of its
result.  d is the longest chain of additions that any of the kernels uses for
the size: a thread's own terms, then a butterfly and the warps' sums."""
import pytest
import torch

from moe_expert_epilogue_b200 import ops

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# below the smallest normal number a rounding is off by half the spacing there
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
bf, hf, f32 = torch.bfloat16, torch.float16, torch.float32
KINDS = [(bf, bf), (bf, f32), (hf, hf), (hf, f32), (f32, f32)]
EPS = 1e-5


def _inputs(rows, hidden, dt, wdt, seed, dev, offset=0.0):
    g = torch.Generator(device=dev).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    return ((r(rows, hidden) * 1.5 + offset).to(dt), (1 + 0.2 * r(hidden)).to(wdt),
            (0.2 * r(hidden)).to(wdt), r(rows, hidden).to(dt))


def _row_depth(hidden):
    return -(-hidden // 32) + 32       # a warp alone may hold a row


def _close(got, want, tol, dt, what):
    got, tol = got.double(), tol + HALF[dt] * want.abs() + TINY[dt]
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:3], want[bad][:3], tol[bad][:3])


def _check_fwd(x, w, b, y, mean, rstd):
    d = _row_depth(x.shape[1]) * U
    x, w = x.double(), w.double()
    m = x.mean(1, keepdim=True)
    c = x - m
    var = c.square().mean(1, keepdim=True)
    rs = 1 / (var + EPS).sqrt()
    em = d * x.abs().mean(1, keepdim=True)                 # the mean's error
    _close(mean[:, None], m, em, f32, "mean")
    # var: the squares' sum, each square twice the error of (x - mean); the mean's own error
    # enters squared, as sum (x - mean) vanishes
    er = 0.5 * (d + 6 * U) + 0.5 * em.square() * rs.square() + 2 * U   # rstd's relative error
    _close(rstd[:, None], rs, er * rs, f32, "rstd")
    want = c * rs * w
    tol = want.abs() * (er + 4 * U) + (w * rs).abs() * (em + U * c.abs())
    if b is not None:
        want = want + b.double()
        tol = tol + U * want.abs()
    _close(y, want, tol, y.dtype, "y")


def _check_bwd(gy, x, w, mean, rstd, gx, gw, gb):
    rows, hidden = x.shape
    d = _row_depth(hidden) * U
    xh = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    a, g, rs = gy.double() * w.double(), gy.double(), rstd.double()[:, None]
    s1, s2 = a.mean(1, keepdim=True), (a * xh).mean(1, keepdim=True)
    want = rs * (a - s1 - xh * s2)
    e1 = (d + 2 * U) * a.abs().mean(1, keepdim=True)
    e2 = (d + 5 * U) * (a * xh).abs().mean(1, keepdim=True)
    tol = rs * (e1 + xh.abs() * e2 + 4 * U * (xh * s2).abs() + 4 * U * (a.abs() + s1.abs()))
    _close(gx, want, tol, gx.dtype, "grad_x")
    dr = (rows // 148 + 64) * U
    _close(gw, (g * xh).sum(0), (dr + 4 * U) * (g * xh).abs().sum(0), gw.dtype, "grad_weight")
    if gb is not None:
        _close(gb, g.sum(0), dr * g.abs().sum(0), gb.dtype, "grad_bias")


SIZES = [(1, 1), (2, 7), (3, 8), (5, 33), (37, 129), (300, 256), (17, 504), (150, 1001),
         (149, 1024), (64, 2048), (11, 2056), (300, 4096), (31, 4104), (100, 7168), (33, 8192),
         (9, 8200), (5, 12288), (7, 20001)]


@pytest.mark.parametrize("dt,wdt", KINDS)
@pytest.mark.parametrize("rows,hidden", SIZES)
def test_sizes(cuda_device, rows, hidden, dt, wdt):
    x, w, b, gy = _inputs(rows, hidden, dt, wdt, rows + hidden, cuda_device)
    y, mean, rstd = ops.layer_norm_fwd(x, w, b, EPS)
    assert y.dtype == dt and mean.dtype == rstd.dtype == f32
    _check_fwd(x, w, b, y, mean, rstd)
    gx, gw, gb = ops.layer_norm_bwd(gy, x, w, mean, rstd)
    assert gx.dtype == dt and gw.dtype == gb.dtype == wdt
    _check_bwd(gy, x, w, mean, rstd, gx, gw, gb)


@pytest.mark.parametrize("dt,wdt", [(bf, f32), (f32, f32)])
@pytest.mark.parametrize("rows,hidden", [(1000, 256), (700, 1001), (2500, 2048), (1200, 7168)])
def test_many_rows(cuda_device, rows, hidden, dt, wdt):
    """Several rows for every row group."""
    x, w, _, gy = _inputs(rows, hidden, dt, wdt, 5, cuda_device)
    y, mean, rstd = ops.layer_norm_fwd(x, w, None, EPS)
    _check_fwd(x, w, None, y, mean, rstd)
    gx, gw, gb = ops.layer_norm_bwd(gy, x, w, mean, rstd, has_bias=False)
    assert gb is None
    _check_bwd(gy, x, w, mean, rstd, gx, gw, None)


@pytest.mark.parametrize("dt", [bf, hf, f32])
@pytest.mark.parametrize("hidden", [64, 1000, 4096])
@pytest.mark.parametrize("offset,pad", [(0, 8), (1, 3), (8, 0), (4, 5)])
def test_strides_and_alignment(cuda_device, dt, hidden, offset, pad):
    """Rows inside wider buffers, from any element; what lies between them stays as it was."""
    rows = 21
    x, w, b, gy = _inputs(rows, hidden, dt, dt, 3, cuda_device)

    def inside(t, fill):
        buf = torch.full((offset + rows * (hidden + pad),), fill, dtype=dt, device=cuda_device)
        v = buf[offset:].view(rows, hidden + pad)[:, :hidden]
        if t is not None:
            v.copy_(t)
        return buf, v

    xs, gs = inside(x, 7.0)[1], inside(gy, 7.0)[1]
    wb = torch.empty(hidden + 1, dtype=dt, device=cuda_device)
    ws = wb[1:] if offset else wb[:-1]
    ws.copy_(w)
    ybuf, ys = inside(None, 3.0)
    _, mean, rstd = ops.layer_norm_fwd(xs, ws, b, EPS, out=ys)
    _check_fwd(x, w, b, ys, mean, rstd)
    gbuf, gxs = inside(None, 3.0)
    _, gw, gb = ops.layer_norm_bwd(gs, xs, ws, mean, rstd, grad_x=gxs)
    _check_bwd(gy, x, w, mean, rstd, gxs, gw, gb)
    for buf in (ybuf, gbuf):
        assert (buf[:offset] == 3.0).all()
        if pad:
            assert (buf[offset:].view(rows, hidden + pad)[:, hidden:] == 3.0).all()


@pytest.mark.parametrize("hidden", [40, 1001, 4096, 9000])
def test_far_mean_constant_rows_and_non_finite_rows(cuda_device, hidden):
    """A mean far from 0, rows of one value, and a row with NaN or infinity that leaves the
    other rows alone."""
    x, w, b, gy = _inputs(12, hidden, f32, f32, 9, cuda_device, offset=1000.0)
    x[3] = 2.5
    x[4] = 0.0
    y, mean, rstd = ops.layer_norm_fwd(x, w, b, EPS)
    _check_fwd(x, w, b, y, mean, rstd)
    gx, gw, gb = ops.layer_norm_bwd(gy, x, w, mean, rstd)
    _check_bwd(gy, x, w, mean, rstd, gx, gw, gb)
    x2 = x.clone()
    x2[5, hidden // 2] = float("nan")
    x2[7, 0] = float("inf")
    y2, _, _ = ops.layer_norm_fwd(x2, w, b, EPS)
    keep = [i for i in range(12) if i not in (5, 7)]
    assert torch.equal(y2[keep], y[keep])
    assert y2[5].isnan().all() and y2[7].isnan().all()


@pytest.mark.parametrize("rows,hidden,dt", [(300, 1024, bf), (5, 4096, bf), (77, 1001, f32)])
def test_rows_do_not_depend_on_the_batch(cuda_device, rows, hidden, dt):
    x, w, b, gy = _inputs(rows, hidden, dt, f32, 11, cuda_device)
    y, mean, rstd = ops.layer_norm_fwd(x, w, b, EPS)
    gx, gw, _ = ops.layer_norm_bwd(gy, x, w, mean, rstd)
    for _ in range(3):
        assert torch.equal(ops.layer_norm_bwd(gy, x, w, mean, rstd)[1], gw)
    for n in (1, rows // 2):
        yn, mn, rn = ops.layer_norm_fwd(x[:n], w, b, EPS)
        assert torch.equal(yn, y[:n]) and torch.equal(mn, mean[:n]) and torch.equal(rn, rstd[:n])
        assert torch.equal(ops.layer_norm_bwd(gy[:n], x[:n], w, mn, rn)[0], gx[:n])


@pytest.mark.parametrize("hidden", [24, 1001])
def test_backward_against_differences(cuda_device, hidden):
    """The gradients of sum(gy * y) against central differences of the 64-bit definition."""
    x, w, b, gy = _inputs(3, hidden, f32, f32, 13, cuda_device)
    _, mean, rstd = ops.layer_norm_fwd(x, w, b, EPS)
    gx, gw, gb = ops.layer_norm_bwd(gy, x, w, mean, rstd)

    def loss(x, w, b):
        m = x.mean(1, keepdim=True)
        v = (x - m).square().mean(1, keepdim=True)
        return (gy.double() * ((x - m) / (v + EPS).sqrt() * w + b)).sum()

    args = [x.double(), w.double(), b.double()]
    step = 1e-5
    for k, grad in enumerate((gx, gw, gb)):
        for i in range(0, grad.numel(), max(1, grad.numel() // 7)):
            up, down = [a.clone() for a in args], [a.clone() for a in args]
            up[k].view(-1)[i] += step
            down[k].view(-1)[i] -= step
            num = float(loss(*up) - loss(*down)) / (2 * step)
            # 64-bit differences: step^2 of the third derivative and 1e-16 / step of a loss of
            # order sqrt(3 hidden); fp32 gradients: 2e-6 of a value of order 1
            assert abs(num - float(grad.view(-1)[i])) <= 2e-5 * (1 + abs(num))


def test_no_rows_no_columns(cuda_device):
    x = torch.empty(0, 64, device=cuda_device)
    w = torch.ones(64, device=cuda_device)
    y, mean, rstd = ops.layer_norm_fwd(x, w, w)
    assert y.shape == (0, 64) and mean.numel() == 0
    gw = torch.full((64,), 5.0, device=cuda_device)
    gx, gw, gb = ops.layer_norm_bwd(x, x, w, mean, rstd, grad_weight=gw)
    assert gx.shape == (0, 64) and (gw == 0).all() and (gb == 0).all()
    e = torch.empty(3, 0, device=cuda_device)
    assert ops.layer_norm_fwd(e, w[:0])[0].shape == (3, 0)


def test_one_row_of_any_stride(cuda_device):
    """A single row has no second row: its stride does not count."""
    x, w, b, _ = _inputs(1, 128, bf, bf, 1, cuda_device)
    want = ops.layer_norm_fwd(x, w, b)[0]
    assert torch.equal(ops.layer_norm_fwd(x[0].as_strided((1, 128), (0, 1)), w, b)[0], want)


def test_other_stream_and_graph(cuda_device):
    x, w, b, gy = _inputs(257, 2048, bf, f32, 15, cuda_device)
    y, mean, rstd = ops.layer_norm_fwd(x, w, b)
    want = [y, *ops.layer_norm_bwd(gy, x, w, mean, rstd)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for handle in (s, s.cuda_stream):
        y2, m2, r2 = ops.layer_norm_fwd(x, w, b, stream=handle)
        got = [y2, *ops.layer_norm_bwd(gy, x, w, m2, r2, stream=handle)]
        s.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y3, m3, r3 = ops.layer_norm_fwd(x, w, b)
        got = [y3, *ops.layer_norm_bwd(gy, x, w, m3, r3)]
    for _ in range(2):
        for t in got:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_offsets_past_32_bits(cuda_device):
    """Rows that start beyond 2^32 elements of a wide buffer."""
    ld = (1 << 31) // 3 // 64 * 64
    buf = torch.zeros(7 * ld, dtype=bf, device=cuda_device)
    xs = buf.view(7, ld)[:, :1000]
    x, w, b, gy = _inputs(7, 1000, bf, bf, 17, cuda_device)
    xs.copy_(x)
    y, mean, rstd = ops.layer_norm_fwd(xs, w, b)
    assert torch.equal(y, ops.layer_norm_fwd(x, w, b)[0])
    _check_fwd(x, w, b, y, mean, rstd)
    out = buf.view(7, ld)[:, 2000:3000]
    ops.layer_norm_bwd(gy, xs, w, mean, rstd, grad_x=out)
    assert torch.equal(out, ops.layer_norm_bwd(gy, x, w, mean, rstd)[0])


# rows, hidden, teams of a CTA, the stalled team and its row that is withheld
@pytest.mark.parametrize("rows,hidden,teams,team,k", [(9000, 1024, 16, 37, 1), (1500, 7168, 2, 5, 3),
                                                      (1500, 4104, 2, 0, 0)])
def test_backward_bounded_wait_runs_out(cuda_device, rows, hidden, teams, team, k):
    """A row whose copies never come: its team gives up after 2e7 cycles (10 ms), the device's
    error word says so, every other team's rows and that team's rows before are as ever, and so
    is the next ordinary call."""
    from moe_expert_epilogue_b200 import _abi
    x, w, _, gy = _inputs(rows, hidden, bf, f32, 19, cuda_device)
    _, mean, rstd = ops.layer_norm_fwd(x, w)
    want = ops.layer_norm_bwd(gy, x, w, mean, rstd, has_bias=False)
    ws = torch.empty(ops.layer_norm_bwd_workspace(rows, hidden), dtype=torch.uint8,
                     device=cuda_device)
    gx, gw = torch.zeros_like(x), torch.zeros_like(w)
    step = min(148, -(-rows // teams)) * teams
    stall = team + k * step
    assert _abi.moe_device_errors(clear=True) == 0
    _abi.moe_test_layer_norm_bwd_stalled(gy, x, w, mean, rstd, gx, gw, ws, ws.numel(), rows, hidden,
                                         stall, 20_000_000)
    torch.cuda.synchronize()
    assert _abi.moe_device_errors(clear=True) == _abi.MOE_DEVERR_TIMEOUT
    r = torch.arange(rows, device=cuda_device)
    whole = (r % step != team) | (r < stall)
    assert int(whole.sum()) < rows and torch.equal(gx[whole], want[0][whole])
    again = ops.layer_norm_bwd(gy, x, w, mean, rstd, has_bias=False, workspace=ws)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
    assert _abi.moe_device_errors(clear=True) == 0
