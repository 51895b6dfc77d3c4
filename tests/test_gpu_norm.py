"""Layer norm and its gradients on the GPU, through the public object, against the formulas in 64 bits.

Tolerances.  u is fp32's unit roundoff, U a type's (half the step beside 1).  A sum over a row of D values is taken
by lanes (at most 32 in a row, or D / 512 where no team of warps holds the row), a warp (5 levels) and up to 16
warps: it is off by at most c u times the sum of magnitudes with c = max(32, D / 512) + 32."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no CUDA device", allow_module_level=True)

from allreduce_ddp_assign_gb300 import lm
from test_gpu_lm import BF16, DEV, F16, F32, TINY, U, assert_guard, gen, guarded, randn, within

u = 2.0 ** -24
EPS = 1e-5


def terms(D):
    return max(32, D // 512 + 1) + 32


def rows64(s, eps):
    x = s.double()
    mean = x.mean(dim=1, keepdim=True)
    d = x - mean
    var = d.square().mean(dim=1, keepdim=True)
    return x, mean, d, var, (var + eps).rsqrt()


def check_forward(s, w, b, eps, y, stats, dt):
    D = s.shape[1]
    x, mean, d, var, rstd = rows64(s, eps)
    c = terms(D) * u
    off = c * x.abs().mean(dim=1, keepdim=True) + u * mean.abs()          # of the mean
    # squares around a mean that is off by `off`: their mean grows by off^2; rounding of each deviation and square
    rel = 0.5 * (c + 6 * u + off.square() / (var + eps)) + 4 * u          # of rstd
    # (a variance far below eps: the deviations' own roundings count against eps)
    rel = rel + 0.5 * (2 * u * d.abs().amax(dim=1, keepdim=True)).square() / (var + eps)
    within(stats[0][:, None], mean, off, "mean")
    within(stats[1][:, None], rstd, rel * rstd, "rstd")
    W, B = w.double(), torch.zeros_like(w, dtype=torch.float64) if b is None else b.double()
    want = d * rstd * W + B
    tol = W.abs() * rstd * (off + u * d.abs()) * (1 + rel) + (d * rstd * W).abs() * (rel + 3 * u) + 2 * u * want.abs()
    within(y, want, tol * (1 + U[dt]) + want.abs() * U[dt] + TINY[dt], "out")


#: rows, columns, row stride, elements before the first row: teams of 1, 2, 4, 8 and 16 warps, in vectors and
#: in single elements, lanes with no, some and all of their share, and rows that no team holds
SHAPES = [
    (1, 1, 1, 0), (3, 2, 2, 0), (5, 7, 9, 1), (33, 64, 64, 0), (17, 100, 104, 0), (700, 768, 768, 0), (9, 768, 776, 8),
    (9, 768, 769, 0), (37, 1001, 1001, 0), (64, 1024, 1024, 0), (21, 1032, 1032, 0), (10, 1600, 1600, 0),
    (11, 2048, 2048, 1), (5, 2056, 2056, 0), (7, 4096, 4096, 0), (3, 5000, 5000, 0), (3, 5001, 5003, 0),
    (4, 8192, 8200, 0), (2, 9000, 9000, 0), (2, 16384, 16384, 0), (2, 16383, 16383, 0), (2, 16392, 16392, 0), (3, 40001, 40001, 3),
    (2500, 40, 40, 0), (2500, 33, 33, 0),
]


@pytest.mark.parametrize("T,D,stride,off", SHAPES)
@pytest.mark.parametrize("dt,wdt", [(F32, F32), (BF16, BF16), (F16, F16), (BF16, F32), (F16, F32)])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("bias", [False, True])
def test_forward(T, D, stride, off, dt, wdt, residual, bias):
    g = gen(1)
    x = guarded(T, D, stride, dt, off)[1]
    x.copy_(randn(g, T, D) * (torch.rand(T, 1, generator=g, device=DEV) * 3 + 0.1) + randn(g, D))
    w, b = randn(g, D + 1, dtype=wdt)[off % 2:D + off % 2], randn(g, D, dtype=wdt) if bias else None
    buf, out = guarded(T, D, stride, dt, off)
    r = sbuf = sout = None
    s = x
    if residual:
        r = guarded(T, D, stride, dt, off)[1]
        r.copy_(randn(g, T, D))
        sbuf, sout = guarded(T, D, stride, dt, off)
        s = (x.float() + r.float()).to(dt)
    y, got, stats = lm.LayerNorm(D, dt, eps=EPS).forward(x, w, b, residual=r, out=out, sum_out=sout)
    assert y is out and torch.equal(got, s)
    check_forward(s, w, b, EPS, y, stats, dt)
    assert_guard(buf, out)
    if residual:
        assert got is sout
        assert_guard(sbuf, sout)


def grads64(s, dy, w, stats, ds):
    """The formulas with the statistics as they are given, and bounds of what precedes the results' own rounding."""
    x, g0, W = s.double(), dy.double(), w.double()
    mean, rstd = stats[0].double()[:, None], stats[1].double()[:, None]
    n = (x - mean) * rstd
    g = g0 * W
    m1, m2 = g.mean(dim=1, keepdim=True), (g * n).mean(dim=1, keepdim=True)
    dx = rstd * (g - m1 - n * m2)
    c = terms(s.shape[1]) * u
    off1, off2 = c * g.abs().mean(dim=1, keepdim=True), (c + 5 * u) * (g * n).abs().mean(dim=1, keepdim=True)
    tol = rstd * (off1 + n.abs() * off2 + 6 * u * (g.abs() + m1.abs() + (n * m2).abs()))
    if ds is not None:
        dx = dx + ds.double()
        tol = tol + u * (dx.abs() + ds.double().abs())
    return dx, tol, (g0 * n), g0


def check_backward(s, dy, w, stats, ds, gx, gw, gb, base, dt):
    T, D = s.shape
    dx, tol, pw, pb = grads64(s, dy, w, stats, ds)
    within(gx, dx, tol * (1 + U[dt]) + dx.abs() * U[dt] + TINY[dt], "grad_x")
    # a column: the rows of a thread one after another, a CTA's teams, 32 threads over the CTAs, those
    ctas = min(152, max(1, 2 ** 23 // D))
    c = (T / ctas + 64) * u
    for name, got, part, k in (("grad_weight", gw, pw, 0), ("grad_bias", gb, pb, 1)):
        if got is None:
            continue
        before = torch.zeros(D, dtype=torch.float64, device=DEV) if base is None else base[k].double()
        want = part.sum(dim=0) + before
        t = (c + 4 * u) * part.abs().sum(dim=0) + u * (want.abs() + before.abs())
        within(got, want, t * (1 + U[got.dtype]) + want.abs() * U[got.dtype] + TINY[got.dtype], name)


@pytest.mark.parametrize("T,D,stride,off", SHAPES)
@pytest.mark.parametrize("dt,wdt,gdt", [(F32, F32, F32), (BF16, BF16, BF16), (F16, F16, F16), (BF16, F32, F32), (F16, F16, F32), (BF16, F32, BF16)])
@pytest.mark.parametrize("grad_sum", [False, True])
@pytest.mark.parametrize("accumulate", [False, True])
def test_backward(T, D, stride, off, dt, wdt, gdt, grad_sum, accumulate):
    g = gen(2)
    s, dy = guarded(T, D, stride, dt, off)[1], guarded(T, D, stride, dt, off)[1]
    s.copy_(randn(g, T, D) * 2 + 0.5)
    dy.copy_(randn(g, T, D))
    ds = None
    if grad_sum:
        ds = guarded(T, D, stride, dt, off)[1]
        ds.copy_(randn(g, T, D))
    w = randn(g, D + 1, dtype=wdt)[off % 2:D + off % 2]
    _, mean, _, _, rstd = rows64(s, EPS)
    stats = torch.cat([mean, rstd], dim=1).t().float().contiguous()
    buf, gx = guarded(T, D, stride, dt, off)
    wbuf, gw = guarded(1, D, D, gdt, 3)
    bbuf, gb = guarded(1, D, D, gdt, 2)
    base = None
    if accumulate:
        base = [randn(g, D, dtype=gdt) for _ in range(2)]
        gw[0].copy_(base[0]), gb[0].copy_(base[1])
    f = lm.LayerNorm(D, dt, eps=EPS)
    res = f.backward(dy, s, w, stats, grad_sum=ds, grad_x=gx, grad_weight=gw[0], grad_bias=gb[0], accumulate=accumulate)
    assert res[0] is gx
    check_backward(s, dy, w, stats, ds, gx, gw[0], gb[0], base, dt)
    for bf, view in ((buf, gx), (wbuf, gw), (bbuf, gb)):
        assert_guard(bf, view)
    # equal calls give equal bits, what is not wanted is not needed, and made outputs are as passed ones
    if not accumulate:
        again = f.backward(dy, s, w, stats, grad_sum=ds)
        assert torch.equal(again[0], gx)
        if gdt == wdt:
            assert torch.equal(again[1], gw[0]) and torch.equal(again[2], gb[0])
        only = f.backward(dy, s, w, stats, grad_sum=ds, need_weight=False, need_bias=False)
        assert torch.equal(only[0], gx) and only[1:] == (None, None)
        one = f.backward(dy, s, w, stats, grad_sum=ds, grad_bias=gb[0], need_weight=False)
        assert one[1] is None and torch.equal(one[2], res[2])


@pytest.mark.parametrize("dt", [F32, BF16, F16])
@pytest.mark.parametrize("T,D", [(40, 768), (5, 20000), (9, 1001)])
def test_in_place(dt, T, D):
    """Outputs that are inputs: the residual stream updated in place, gradients written over what they came from."""
    g = gen(3)
    x, r, dy = (randn(g, T, D, dtype=dt) for _ in range(3))
    w, b = randn(g, D, dtype=dt), randn(g, D, dtype=dt)
    f = lm.LayerNorm(D, dt)
    y, s, stats = f.forward(x, w, b, residual=r)
    for out, total in (("x", "r"), ("r", "x"), ("x", None), (None, "x")):
        t = {"x": x.clone(), "r": r.clone(), None: None}
        y2, s2, st2 = f.forward(t["x"], w, b, residual=t["r"], out=t[out], sum_out=t[total])
        assert torch.equal(y, y2) and torch.equal(s, s2) and torch.equal(stats, st2)
        assert out is None or y2 is t[out]
    plain = f.forward(x, w, b)[0]
    xc = x.clone()
    assert torch.equal(f.forward(xc, w, b, out=xc)[0], plain)
    want = f.backward(dy, s, w, stats, grad_sum=r)
    for over in range(3):
        a = [dy.clone(), s.clone(), r.clone()]
        got = f.backward(a[0], a[1], w, stats, grad_sum=a[2], grad_x=a[over])
        assert all(torch.equal(p, q) for p, q in zip(want, got))


def test_no_rows():
    f = lm.LayerNorm(24, F32)
    none = torch.empty(0, 24, device=DEV)
    w = torch.ones(24, device=DEV)
    y, s, stats = f.forward(none, w, w, residual=none)
    assert y.shape == s.shape == (0, 24) and stats.shape == (2, 0)
    gx, gw, gb = f.backward(none, none, w, stats, grad_sum=none)
    assert gx.shape == (0, 24) and bool((gw == 0).all()) and bool((gb == 0).all())
    gw.fill_(3), gb.fill_(4)
    f.backward(none, none, w, stats, grad_weight=gw, grad_bias=gb, accumulate=True)
    assert bool((gw == 3).all()) and bool((gb == 4).all())


@pytest.mark.parametrize("dt", [F32, BF16, F16])
@pytest.mark.parametrize("D", [1, 40, 768, 777, 5000, 20000])
def test_rows_of_equal_values_and_rows_that_are_not_finite(dt, D):
    """Equal values: rstd = 1 / sqrt(eps) and the bias (a power of two at these widths' sums is exact only for
    some, so the deviations are at most the mean's error); NaN and infinity stay in their rows."""
    x = randn(gen(4), 6, D, dtype=dt)
    x[1], x[3, D // 2], x[4, D - 1] = 2.0, math.nan, math.inf
    w, b = torch.full((D,), 0.5, device=DEV, dtype=dt), torch.full((D,), 3.0, device=DEV, dtype=dt)
    f = lm.LayerNorm(D, dt, eps=1.0)
    y, _, stats = f.forward(x, w, b)
    # the mean of equal values is off by c u 2, and so is each deviation
    off = 2 * terms(D) * u
    assert bool(((y[1].double() - 3).abs() <= off + 3 * U[dt]).all())
    assert abs(float(stats[1, 1]) - 1) <= off ** 2 + 4 * u
    assert bool(y[3].isnan().all()) and bool(y[4].isnan().all())
    assert bool(y[[0, 1, 2, 5]].isfinite().all())
    gx, gw, gb = f.backward(torch.ones_like(x), x, w, stats)
    assert bool(gx[3].isnan().all()) and bool(gx[4].isnan().all()) and bool(gx[[0, 1, 2, 5]].isfinite().all())
    assert bool(gw.isnan().all()) and bool((gb == 6).all())


def test_gradients_against_differences():
    """sum(c y + c2 s) along a direction: the gradients against a central difference of the formula in 64 bits.

    With a step of 1e-5 the difference is off by 1e-10 of the third derivative and by 1e-16 / 1e-5 of the sum's terms:
    1e-8 of the sum of magnitudes covers both.  The gradients are off by what check_backward allows, along the
    direction; the statistics that they are computed with are fp32's, off by c u, which moves a gradient by as much
    of its terms (three of them)."""
    g = gen(5)
    T, D, h = 7, 96, 1e-5
    x, r, c, c2, dirx = (randn(g, T, D) for _ in range(5))
    w, b, dirw, dirb = (randn(g, D) for _ in range(4))
    f = lm.LayerNorm(D, F32)
    _, s, stats = f.forward(x, w, b, residual=r)
    gx, gw, gb = f.backward(c, s, w, stats, grad_sum=c2)

    def loss(k):
        t = s.double() + k * dirx.double()
        d = t - t.mean(dim=1, keepdim=True)
        n = d / (d.square().mean(dim=1, keepdim=True) + f.eps).sqrt()
        y = n * (w.double() + k * dirw.double()) + b.double() + k * dirb.double()
        return y * c.double() + t * c2.double()

    difference = float((loss(h) - loss(-h)).sum()) / (2 * h)
    along = [(gx.double() * dirx), (gw.double() * dirw), (gb.double() * dirb)]
    dx, tol, pw, pb = grads64(s, c, w, stats, c2)
    few = (terms(D) + 70) * u
    allowed = float(((tol + (1 + 3 * terms(D)) * u * (dx.abs() + c2.abs())) * dirx.abs()).sum())
    allowed += few * float((pw.abs().sum(dim=0) * dirw.abs() + pb.abs().sum(dim=0) * dirb.abs()).sum())
    allowed += 1e-8 * float(loss(0).abs().sum())
    assert abs(sum(float(a.sum()) for a in along) - difference) <= allowed


def test_offsets_beyond_32_bits():
    """More than 2^32 bytes and 2^31 elements: the last rows are as they are alone."""
    T, D = 1_100_000, 2048
    x = torch.empty(T, D, dtype=BF16, device=DEV)
    x[:] = randn(gen(6), 1, D, dtype=BF16)
    x[-3:] = randn(gen(7), 3, D, dtype=BF16)
    w, b = randn(gen(8), D, dtype=BF16), randn(gen(9), D, dtype=BF16)
    f = lm.LayerNorm(D, BF16)
    y, _, stats = f.forward(x, w, b)
    tail = x[-3:].clone()
    ty, _, ts = f.forward(tail, w, b)
    assert torch.equal(y[-3:], ty) and torch.equal(stats[:, -3:], ts)
    gx = f.backward(x, x, w, stats, grad_x=y, need_weight=False, need_bias=False)[0]
    assert torch.equal(gx[-3:], f.backward(tail, tail, w, ts)[0])


def test_another_stream_and_a_graph():
    g = gen(10)
    T, D = 300, 768
    x, r, dy = (randn(g, T, D, dtype=BF16) for _ in range(3))
    w, b = randn(g, D, dtype=BF16), randn(g, D, dtype=BF16)
    f = lm.LayerNorm(D, BF16)

    def calls(**on):
        y, s, stats = f.forward(x, w, b, residual=r, **on)
        return (y, s, stats) + f.backward(dy, s, w, stats, grad_sum=r, **on)

    want = [t.clone() for t in calls()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = calls(stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    graphs = []
    for _ in range(2):   # two graphs, each with scratch memory of its own
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            graphs.append((graph, calls()))
    x.mul_(2), r.mul_(2)
    want = [t.clone() for t in calls()]
    for _ in range(3):
        for graph, _ in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for _, got in graphs:
        assert all(torch.equal(p, q) for p, q in zip(want, got))


@pytest.mark.parametrize("T,D,stride,off", [(30011, 72, 72, 0), (30011, 33, 33, 1), (20011, 768, 768, 0), (9001, 1001, 1001, 0),
                                            (6007, 2056, 2056, 0), (3001, 2051, 2052, 3), (2503, 5001, 5001, 0), (2503, 8200, 8200, 0),
                                            (1201, 16384, 16384, 0)])
@pytest.mark.parametrize("dt,wdt", [(F32, F32), (BF16, F32), (F16, F16)])
@pytest.mark.parametrize("both", [False, True])
def test_many_rows(T, D, stride, off, dt, wdt, both):
    """Rows enough for every team to go around its ring in shared memory several times; in place as well."""
    g = gen(20)
    x, r, dy = (guarded(T, D, stride, dt, off)[1] for _ in range(3))
    for t in (x, r, dy):
        t.copy_(randn(g, T, D))
    w, b = randn(g, D, dtype=wdt), randn(g, D, dtype=wdt)
    f = lm.LayerNorm(D, dt, eps=EPS)
    y, s, stats = f.forward(x, w, b, residual=r if both else None)
    assert torch.equal(s, (x.float() + r.float()).to(dt) if both else x)
    check_forward(s, w, b, EPS, y, stats, dt)
    gx, gw, gb = f.backward(dy, s, w, stats, grad_sum=r if both else None)
    check_backward(s, dy, w, stats, r if both else None, gx, gw, gb, None, dt)
    buf, over = guarded(T, D, stride, dt, off)
    over.copy_(dy)
    again = f.backward(over, s, w, stats, grad_sum=r if both else None, grad_x=over)
    assert all(torch.equal(p, q) for p, q in zip(again, (gx, gw, gb)))
    assert_guard(buf, over)
    if both:
        again = f.forward(x, w, b, residual=r, sum_out=x, out=r)
        assert all(torch.equal(p, q) for p, q in zip(again, (y, s, stats)))


@pytest.mark.parametrize("T,D,stride,off", [(1300, 8201, 8201, 0), (700, 16391, 16392, 3), (700, 16392, 16392, 0), (1300, 12288, 12288, 0),
                                            (300, 65537, 65537, 1)])
@pytest.mark.parametrize("dt,wdt", [(F32, F32), (BF16, BF16), (F16, F32)])
@pytest.mark.parametrize("both", [False, True])
def test_many_rows_that_no_team_holds(T, D, stride, off, dt, wdt, both):
    """Several rows a CTA where a whole CTA goes over a row in passes (more rows than 4 an SM; 65537 columns, whose sums
    take a row of the workspace each, have 127 CTAs in the backward pass); 12288 columns of fp32 with a residual among
    them, and fp32 rows that stay in registers."""
    g = gen(21)
    x, r, dy = (guarded(T, D, stride, dt, off)[1] for _ in range(3))
    for t in (x, r, dy):
        t.copy_(randn(g, T, D))
    w, b = randn(g, D, dtype=wdt), randn(g, D, dtype=wdt)
    f = lm.LayerNorm(D, dt, eps=EPS)
    y, s, stats = f.forward(x, w, b, residual=r if both else None)
    assert torch.equal(s, (x.float() + r.float()).to(dt) if both else x)
    check_forward(s, w, b, EPS, y, stats, dt)
    gx, gw, gb = f.backward(dy, s, w, stats, grad_sum=r if both else None)
    check_backward(s, dy, w, stats, r if both else None, gx, gw, gb, None, dt)
    # onto what is there, and over an input
    base = [randn(g, D) for _ in range(2)]
    gw, gb = (t.clone() for t in base)
    buf, over = guarded(T, D, stride, dt, off)
    over.copy_(dy)
    f.backward(over, s, w, stats, grad_sum=r if both else None, grad_x=over, grad_weight=gw, grad_bias=gb, accumulate=True)
    assert torch.equal(over, gx)
    check_backward(s, dy, w, stats, r if both else None, over, gw, gb, base, dt)
    assert_guard(buf, over)
    if both:
        again = f.forward(x, w, b, residual=r, sum_out=x, out=r)
        assert all(torch.equal(p, q) for p, q in zip(again, (y, s, stats)))
