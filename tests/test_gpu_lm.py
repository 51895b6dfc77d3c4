"""Gradient clipping, the token embedding and the vocabulary loss on the GPU,
through the public objects, against the formulas in 64 bits.

Tolerances.  u is the unit roundoff of a type (fp32 2^-24, bf16 2^-8, fp16 2^-11: half the step beside 1)
and a result that is rounded once to its type may be off by u |result| (fp16: plus
half its smallest number, 2^-25).  What comes before the rounding is bounded below
at each test."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no CUDA device", allow_module_level=True)

import allreduce_ddp_assign_gb300 as D
from allreduce_ddp_assign_gb300 import lm

DEV = torch.device("cuda:0")
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
U = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}
TINY = {F32: 2.0 ** -149, BF16: 2.0 ** -133, F16: 2.0 ** -25}


@pytest.fixture(autouse=True)
def clean_status():
    D.ddp_lm_status(reset=True)
    yield
    torch.cuda.synchronize()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def guarded(rows, cols, stride, dtype, off=0, fill=-7.75):
    """A [rows, cols] view with row stride `stride`, `off` elements into a buffer of `fill`."""
    buf = torch.full((off + max(rows, 1) * stride + 64,), fill, dtype=dtype, device=DEV)
    return buf, buf[off:off + max(rows, 1) * stride].view(max(rows, 1), stride)[:rows, :cols]


def assert_guard(buf, view, fill=-7.75):
    """Nothing outside the view was written."""
    mask = torch.ones_like(buf, dtype=torch.bool)
    off = (view.data_ptr() - buf.data_ptr()) // buf.element_size() if view.numel() else 0
    if view.numel():
        idx = off + torch.arange(view.shape[0], device=DEV)[:, None] * view.stride(0) + \
            torch.arange(view.shape[1], device=DEV)[None, :]
        mask[idx.reshape(-1)] = False
    assert bool((buf[mask] == fill).all())


def within(got, want, tol, what=""):
    got = got.double()
    bad = (got - want).abs() > tol
    if bool(bad.any()):
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; first at {i}: got {float(got[i])!r} "
                             f"want {float(want[i])!r} tolerance {float(tol[i] if tol.dim() else tol)!r}")


# ---------------------------------------------------------------------------
# clipping
# ---------------------------------------------------------------------------
# At most 64 squares are summed in fp32 at a time (relative error 64 u of the sum, half of it after the square
# root); everything after that is in fp64 and rounded to fp32 once.
NORM_REL = 32 * 2.0 ** -24 + 2 * 2.0 ** -24

SIZES = {
    "one": [1],
    "few": [5, 0, 3, 1],
    "mixed": [4097, 1, 0, 63, 64, 65, 100003, 7],
    "many": [17 + (k * 37) % 300 for k in range(391)],
    "long": [1 << 22, 12345, (1 << 20) + 1],
}


def make_grads(seed, sizes, dtypes, scale=1.0, shift=0):
    """Tensors packed tight from `shift` elements into one buffer for each type, as a bucket packs them."""
    g = gen(seed)
    out = []
    flats = {}
    for dt in set(dtypes):
        n = sum(s for s, d in zip(sizes, dtypes) if d == dt)
        flats[dt] = [randn(g, n + shift, dtype=dt, scale=scale), shift]
    for s, dt in zip(sizes, dtypes):
        flat, at = flats[dt]
        out.append(flat[at:at + s])
        flats[dt][1] += s
    return out


def norm64(grads, inf):
    parts = [t.double() for t in grads if t is not None and t.numel()]
    if not parts:
        return 0.0
    if inf:
        return float(torch.stack([p.abs().max() for p in parts]).max())
    return math.sqrt(sum(float(p.square().sum()) for p in parts))


@pytest.mark.parametrize("inf", [False, True])
@pytest.mark.parametrize("name", list(SIZES))
@pytest.mark.parametrize("kinds", [(F32,), (BF16,), (F16,), (F32, BF16, F16)])
@pytest.mark.parametrize("shift", [0, 1])
def test_clip_out_of_place(name, kinds, inf, shift):
    sizes = SIZES[name]
    dts = [kinds[k % len(kinds)] for k in range(len(sizes))]
    grads = make_grads(1, sizes, dts, 0.37, shift)
    outs = [torch.full_like(t, 9.0) for t in grads]
    ref = norm64(grads, inf)
    c = lm.GradClipper(grads, out=outs, norm_type=math.inf if inf else 2)
    for max_norm in (0.5 * ref, 0.0, 10 * ref + 1):
        got = c.clip(max_norm)
        assert abs(float(got) - ref) <= (2.0 ** -24 if inf else NORM_REL) * ref
        coef = min(1.0, max_norm / (ref + 1e-6))
        for t, o, dt in zip(grads, outs, dts):
            want = t.double() * coef
            # the factor: the norm's error, its sum, the quotient and its rounding, all in fp32
            within(o, want, want.abs() * (U[dt] + NORM_REL + 4 * 2.0 ** -24) + TINY[dt], name)
        assert abs(float(c.norm()) - ref) <= (2.0 ** -24 if inf else NORM_REL) * ref


@pytest.mark.parametrize("dt", [F32, BF16, F16])
def test_clip_in_place_and_untouched_when_small(dt):
    grads = make_grads(2, SIZES["mixed"], [dt] * 8)
    before = [t.clone() for t in grads]
    c = lm.GradClipper(grads)
    ref = norm64(grads, False)
    n = c.clip(2 * ref)
    assert abs(float(n) - ref) <= NORM_REL * ref
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    c.clip(0.25 * ref)
    for a, b in zip(grads, before):
        want = b.double() * (0.25 * ref / (ref + 1e-6))
        within(a, want, want.abs() * (U[dt] + NORM_REL + 4 * 2.0 ** -24) + TINY[dt])


def test_clip_without_gradients():
    c = lm.GradClipper([None, torch.empty(0, device=DEV), None])
    assert float(c.norm()) == 0.0 and float(c.clip(1.0)) == 0.0
    assert float(lm.GradClipper([]).clip(1.0)) == 0.0
    g = make_grads(3, [100, 200], [F32, F32])
    c = lm.GradClipper([None, g[0], None, g[1]])
    assert abs(float(c.norm()) - norm64(g, False)) <= NORM_REL * norm64(g, False)


@pytest.mark.parametrize("scale", [1e30, 1e-30, 3e-44])
def test_norm_where_squares_leave_fp32(scale):
    x = (torch.rand(5001, generator=gen(4), device=DEV) + 0.5) * scale
    small = torch.full((100,), 1e-3 * scale, device=DEV)
    ref = norm64([x, small], False)
    got = float(lm.GradClipper([x, small]).norm())
    assert abs(got - ref) <= NORM_REL * ref + 2.0 ** -149
    mixed = torch.cat([x, torch.ones(10, device=DEV)])
    ref = norm64([mixed], False)
    assert abs(float(lm.GradClipper([mixed]).norm()) - ref) <= NORM_REL * ref


@pytest.mark.parametrize("dt", [F32, BF16, F16])
@pytest.mark.parametrize("at", [0, 77, 4999])
def test_norm_of_infinities_and_nans(dt, at):
    for inf in (False, True):
        x = torch.ones(5000, device=DEV, dtype=dt)
        out = torch.empty_like(x)
        c = lm.GradClipper([x], out=[out], norm_type=math.inf if inf else 2)
        x[at] = -math.inf
        assert float(c.clip(1.0)) == math.inf
        assert bool(out[at].isnan()) and int((out == 0).sum()) == 4999
        x[at] = math.nan
        assert math.isnan(float(c.clip(1.0))) and bool(out.isnan().all())


def test_clip_is_the_same_every_time_and_on_another_stream():
    grads = make_grads(5, SIZES["long"], [F32] * 3)
    outs = [torch.empty_like(t) for t in grads]
    c = lm.GradClipper(grads, out=outs)
    a, first = float(c.clip(1.0)), [o.clone() for o in outs]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        b = c.clip(1.0, stream=s)
        s.synchronize()
        assert float(b) == a and all(torch.equal(x, y) for x, y in zip(first, outs))


# ---------------------------------------------------------------------------
# embedding
# ---------------------------------------------------------------------------
EMBED = [  # tokens, vocab, dim, stride, offset
    (1, 1, 1, 1, 0), (1, 50257, 768, 768, 0), (7, 10, 5, 9, 1), (33, 100, 64, 64, 0), (129, 1000, 100, 104, 0),
    (1000, 5003, 257, 257, 3), (4099, 30522, 128, 136, 8), (20000, 300, 40, 40, 0),
]


@pytest.mark.parametrize("T,V,dim,stride,off", EMBED)
@pytest.mark.parametrize("dt", [F32, BF16, F16])
@pytest.mark.parametrize("idt", [torch.int32, torch.int64])
def test_embedding_forward(T, V, dim, stride, off, dt, idt):
    g = gen(10)
    w = guarded(V, dim, stride, dt, off)[1]
    w.copy_(randn(g, V, dim, dtype=dt))
    ids = torch.randint(0, V, (T,), generator=g, device=DEV).to(idt)
    buf, out = guarded(T, dim, stride, dt, off)
    lm.TokenEmbedding(V, dim, dt, scale=math.sqrt(dim)).forward(w, ids, out=out)
    want = w[ids.long()].double() * np.float32(math.sqrt(dim)).astype(np.float64)
    within(out, want, want.abs() * U[dt] + TINY[dt])
    assert_guard(buf, out)
    assert D.ddp_lm_status() == 0


def test_embedding_ids_out_of_range():
    w = randn(gen(11), 10, 16)
    ids = torch.tensor([3, 10, -1, 0, 1 << 40], device=DEV)
    e = lm.TokenEmbedding(10, 16, F32)
    out = e.forward(w, ids)
    assert torch.equal(out[0], w[3]) and torch.equal(out[3], w[0]) and bool((out[[1, 2, 4]] == 0).all())
    assert D.ddp_lm_status(reset=True) == 2
    go = randn(gen(12), 5, 16)
    gw = e.backward(go, ids)
    want = torch.zeros_like(w)
    want[3], want[0] = go[0], go[3]
    assert torch.equal(gw, want)
    assert D.ddp_lm_status(reset=True) == 2 and D.ddp_lm_status() == 0


def embed_grad64(go, ids, V, scale, pad):
    """(gradient, sum of magnitudes) in 64 bits."""
    keep = (ids >= 0) & (ids < V) & (ids != pad)
    g = go.double()[keep] * scale
    z = torch.zeros(V, go.shape[1], dtype=torch.float64, device=DEV)
    return z.index_add(0, ids[keep].long(), g), z.index_add(0, ids[keep].long(), g.abs())


@pytest.mark.parametrize("T,V,dim,stride,off", EMBED)
@pytest.mark.parametrize("dt,wdt", [(F32, F32), (BF16, BF16), (F16, F16), (BF16, F32), (F16, F32)])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("ids_kind", ["uniform", "one", "skewed", "padded"])
def test_embedding_backward(T, V, dim, stride, off, dt, wdt, accumulate, ids_kind):
    g = gen(20)
    ids = torch.randint(0, V, (T,), generator=g, device=DEV)
    pad = None
    if ids_kind == "one":
        ids[:] = V // 2
    elif ids_kind == "skewed":
        ids = torch.where(torch.rand(T, generator=g, device=DEV) < 0.6, ids % max(1, V // 50), ids)
    elif ids_kind == "padded":
        pad = V // 3
        ids[T // 2:] = pad
    go = guarded(T, dim, stride, dt, off)[1]
    go.copy_(randn(g, T, dim, dtype=dt))
    buf, gw = guarded(V, dim, stride, wdt, off)
    base = randn(g, V, dim, dtype=wdt) if accumulate else torch.zeros(V, dim, dtype=wdt, device=DEV)
    if accumulate:
        gw.copy_(base)
    scale = 1.5
    e = lm.TokenEmbedding(V, dim, dt, scale=scale, padding_idx=pad)
    e.backward(go, ids, grad_weight=gw, accumulate=accumulate)
    s, mag = embed_grad64(go, ids, V, scale, -1 if pad is None else pad)
    want = s + base.double()
    # fp32 sums of n terms in some order, the scale, the addition to what was there
    n = torch.bincount(ids, minlength=V).double()[:, None]
    tol = (n + 2) * 2.0 ** -24 * (mag + base.double().abs()) + want.abs() * U[wdt] + TINY[wdt]
    within(gw, want, torch.where(mag > 0, tol, torch.zeros_like(tol)), ids_kind)
    assert_guard(buf, gw)
    again = gw.clone()
    if accumulate:
        gw.copy_(base)
    e.backward(go, ids.to(torch.int32), grad_weight=gw, accumulate=accumulate)
    assert torch.equal(again, gw)


def test_embedding_without_tokens():
    e = lm.TokenEmbedding(50, 24, F32, padding_idx=0)
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    assert e.forward(randn(gen(1), 50, 24), none).shape == (0, 24)
    assert bool((e.backward(torch.empty(0, 24, device=DEV), none) == 0).all())
    gw = torch.ones(50, 24, device=DEV)
    e.backward(torch.empty(0, 24, device=DEV), none, grad_weight=gw, accumulate=True)
    assert bool((gw == 1).all())
    # nothing but padding
    assert bool((e.backward(torch.ones(9, 24, device=DEV), torch.zeros(9, dtype=torch.int64, device=DEV)) == 0).all())


def test_embedding_masked_rows_may_hold_anything():
    go = randn(gen(2), 64, 40)
    ids = torch.arange(64, device=DEV) % 8
    go[ids == 3] = math.nan
    go[0] = math.inf
    gw = lm.TokenEmbedding(10, 40, F32, padding_idx=3).backward(go, ids)
    assert bool((gw[3] == 0).all()) and bool((gw[0] == math.inf).all()) and bool(gw[[1, 2, 4, 5, 6, 7]].isfinite().all())


def test_embedding_gradient_against_differences():
    """<dY, forward(W)> is linear in W: its difference along E is <dW, E>.  Small integers keep every sum exact."""
    g = gen(30)
    V, dim, T = 37, 24, 200
    W = torch.randint(-4, 5, (V, dim), generator=g, device=DEV).float()
    E = torch.randint(-2, 3, (V, dim), generator=g, device=DEV).float()
    dY = torch.randint(-3, 4, (T, dim), generator=g, device=DEV).float()
    ids = torch.randint(0, V, (T,), generator=g, device=DEV)
    e = lm.TokenEmbedding(V, dim, F32, scale=0.5)
    up, down = [(e.forward(W + s * E, ids).double() * dY).sum() for s in (1, -1)]
    assert float((up - down) / 2) == float((e.backward(dY, ids).double() * E).sum())


def test_embedding_offsets_beyond_32_bits():
    """A table of more than 2^32 bytes and 2^31 elements: the last rows."""
    V, dim = 1_100_000, 2048
    w = torch.empty(V, dim, dtype=BF16, device=DEV)
    w[-5:] = randn(gen(31), 5, dim, dtype=BF16)
    w[0] = 1.0
    ids = torch.tensor([V - 1, 0, V - 5, V - 1], device=DEV)
    e = lm.TokenEmbedding(V, dim, BF16)
    out = e.forward(w, ids)
    assert torch.equal(out, w[ids])
    gw = e.backward(out, ids, grad_weight=w)
    assert torch.equal(gw[V - 5], out[2]) and bool((gw[0] == 1).all()) and int(gw[1:V - 5].count_nonzero()) == 0
    assert torch.equal(gw[V - 1], (out[0].float() * 2).to(BF16))


# ---------------------------------------------------------------------------
# vocabulary loss
# ---------------------------------------------------------------------------
LOSS = [  # tokens, vocab, dim, ignored share, aligned
    (1, 1, 1, 0.0, True), (1, 50257, 768, 0.0, True), (3, 7, 5, 0.0, True), (17, 256, 64, 0.0, True),
    (130, 1000, 72, 0.3, True), (257, 513, 257, 0.1, True), (300, 2049, 128, 0.9, True), (200, 700, 100, 0.2, False),
    (1000, 3001, 192, 0.0, True), (2, 5000, 200, 0.0, True), (2, 300, 77, 0.5, False), (64, 20000, 320, 0.5, True), (520, 4096, 520, 0.15, True),
]


def loss_case(seed, T, V, dim, ignored, dt, aligned=True, sharp=4.0):
    g = gen(seed)
    hoff, hs = (0, dim) if aligned else (3, dim + 5)
    h = guarded(T, dim, hs, dt, hoff, 0.0)[1]
    w = guarded(V, dim, hs, dt, hoff, 0.0)[1]
    h.copy_(randn(g, T, dim, dtype=dt))
    w.copy_(randn(g, V, dim, dtype=dt, scale=sharp / math.sqrt(dim)))
    y = torch.randint(0, V, (T,), generator=g, device=DEV)
    drop = torch.rand(T, generator=g, device=DEV) < ignored
    y[drop] = -100
    return h, w, y, ~drop


def loss64(h, w, y, valid, gl=None):
    """Everything in 64 bits, and bounds of what 32-bit sums may be off.

    z: D products, exact in fp32, summed in fp32 in some order, each step cutting off at most a unit in the last
    place: |dz| <= D 2^-23 sum|h||w|.  The exponent's argument is rounded twice (2^-22 |z - max|), exp and log
    are off by 4 u, the sums over a tile's 256 words and over the tiles by (256 + tiles) u."""
    H, W = h.double()[valid], w.double()
    yy = y[valid]
    z = H @ W.t()
    dz = (h.shape[1] + 2) * 2.0 ** -23 * (H.abs() @ W.abs().t())
    top = z.max(1, keepdim=True).values
    lse = (z - top).exp().sum(1, keepdim=True).log() + top
    loss = (lse - z.gather(1, yy[:, None]))[:, 0]
    V = w.shape[0]
    dlse = dz.max(1).values + 2.0 ** -22 * (z - top).abs().max(1).values + (264 + V / 256) * 2.0 ** -24 \
        + 4 * 2.0 ** -24 * (lse[:, 0].abs() + top[:, 0].abs())
    res = dict(loss=loss, lse=lse[:, 0], dlse=dlse,
               dloss=dlse + dz.gather(1, yy[:, None])[:, 0] + 2.0 ** -23 * (loss.abs() + z.abs().max(1).values))
    if gl is not None:
        p = (z - lse).exp()
        one = torch.nn.functional.one_hot(yy, V).double()
        g = (p - one) * gl.double()[valid][:, None]
        dp = p * (dz + dlse[:, None] + 2.0 ** -22 * (z - lse).abs() + 8 * 2.0 ** -24)
        res.update(g=g, dg=dp * gl.double()[valid].abs()[:, None], H=H, W=W)
    return res


@pytest.mark.parametrize("T,V,dim,ignored,aligned", LOSS)
@pytest.mark.parametrize("dt", [BF16, F16])
def test_loss_forward(T, V, dim, ignored, aligned, dt):
    h, w, y, valid = loss_case(40, T, V, dim, ignored, dt, aligned)
    loss, lse = lm.VocabLoss(V, dim, dt).forward(h, w, y)
    r = loss64(h, w, y, valid)
    within(lse[valid], r["lse"], r["dlse"], "lse")
    within(loss[valid], r["loss"], r["dloss"], "loss")
    assert bool((loss[~valid] == 0).all()) and bool((lse[~valid] == 0).all())
    again = lm.VocabLoss(V, dim, dt).forward(h, w, y.to(torch.int32))
    assert torch.equal(again[0], loss) and torch.equal(again[1], lse)
    assert D.ddp_lm_status() == 0


def check_grads(h, w, y, valid, gl, gh, gw, base, dt):
    r = loss64(h, w, y, valid, gl)
    K = max(h.shape[0], w.shape[0])
    # G: the softmax's error, one rounding to 16 bits after a division by max|gl| (a rounding of fp32 there and one
    # at the product with it), fp16: below 2^-14 / 2^14 an absolute step; then fp32 sums, a rounding to the type
    gmax = float(gl[valid].abs().max()) if bool(valid.any()) else 0.0
    eg = r["dg"] + (U[dt] + 4 * 2.0 ** -24 + (K + 2) * 2.0 ** -23) * r["g"].abs() + \
        (2.0 ** -39 * gmax if dt == F16 else 2.0 ** -133)
    if gh is not None:
        want = r["g"] @ r["W"]
        within(gh[valid], want, eg @ r["W"].abs() + want.abs() * U[dt] + TINY[dt], "grad_hidden")
        assert bool((gh[~valid] == 0).all())
    if gw is not None:
        s = r["g"].t() @ r["H"]
        want = s + base.double()
        tol = eg.t() @ r["H"].abs() + want.abs() * U[gw.dtype] + 2.0 ** -24 * (s.abs() + base.double().abs()) + TINY[gw.dtype]
        within(gw, want, tol, "grad_weight")


@pytest.mark.parametrize("T,V,dim,ignored,aligned", LOSS)
@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("piece", [0, 256])
def test_loss_backward(T, V, dim, ignored, aligned, dt, piece):
    h, w, y, valid = loss_case(41, T, V, dim, ignored, dt, aligned)
    f = lm.VocabLoss(V, dim, dt, piece=piece)
    _, lse = f.forward(h, w, y)
    gl = torch.rand(T, generator=gen(42), device=DEV) - 0.3
    stride, off = (dim, 0) if aligned else (dim + 3, 1)
    b1, gh = guarded(T, dim, stride, dt, off)
    b2, gw = guarded(V, dim, stride, dt, off)
    f.backward(h, w, y, lse, gl, grad_hidden=gh, grad_weight=gw)
    check_grads(h, w, y, valid, gl, gh, gw, torch.zeros_like(gw), dt)
    assert_guard(b1, gh)
    assert_guard(b2, gw)
    gh2, gw2 = f.backward(h, w, y, lse, gl)
    assert torch.equal(gh, gh2) and torch.equal(gw, gw2)


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("T,ignored", [(100, 0.0), (600, 0.8), (2, 0.0)])
def test_loss_backward_in_long_pieces(dt, T, ignored):
    """Few rows and long pieces: the hidden states' gradient is split along each piece and summed over the pieces."""
    V, dim = 9001, 264
    h, w, y, valid = loss_case(60, T, V, dim, ignored, dt)
    f = lm.VocabLoss(V, dim, dt, piece=4096)
    _, lse = f.forward(h, w, y)
    gl = torch.rand(T, generator=gen(61), device=DEV)
    gh, gw = f.backward(h, w, y, lse, gl)
    check_grads(h, w, y, valid, gl, gh, gw, torch.zeros_like(gw), dt)


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("wide", [False, True])
def test_loss_backward_accumulates(dt, wide):
    T, V, dim = 200, 1500, 136
    h, w, y, valid = loss_case(43, T, V, dim, 0.2, dt)
    f = lm.VocabLoss(V, dim, dt, piece=512)
    _, lse = f.forward(h, w, y)
    gl = torch.full((1,), 1.0 / T, device=DEV)
    base = randn(gen(44), V, dim, dtype=F32 if wide else dt, scale=1e-2)
    buf, gw = guarded(V, dim, dim + 8, base.dtype, 8)
    gw.copy_(base)
    gh, _ = f.backward(h, w, y, lse, gl, grad_weight=gw, accumulate=True)
    check_grads(h, w, y, valid, gl.expand(T), gh, gw, base, dt)
    assert_guard(buf, gw)
    only_h = f.backward(h, w, y, lse, gl, need_weight=False)
    assert torch.equal(only_h[0], gh) and only_h[1] is None
    only_w = f.backward(h, w, y, lse, gl, need_hidden=False)
    check_grads(h, w, y, valid, gl.expand(T), None, only_w[1], torch.zeros_like(only_w[1]), dt)


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("size", [0.0, 1e-6, 1e-3, 65536.0])
def test_loss_backward_scales(dt, size):
    """Any size of grad_loss, and tokens whose gradients differ by far."""
    T, V, dim = 70, 900, 64
    h, w, y, valid = loss_case(45, T, V, dim, 0.1, dt)
    f = lm.VocabLoss(V, dim, dt)
    _, lse = f.forward(h, w, y)
    gl = torch.rand(T, generator=gen(46), device=DEV) * size
    gl[::7] *= 1e-3
    gl[5] = 0.0
    gw = torch.empty(V, dim, dtype=F32, device=DEV)
    gh, _ = f.backward(h, w, y, lse, gl, grad_weight=gw)
    if size < 1000 or dt == BF16:
        check_grads(h, w, y, valid, gl, gh, gw, torch.zeros_like(gw), dt)
    else:
        check_grads(h, w, y, valid, gl, None, gw, torch.zeros_like(gw), dt)


@pytest.mark.parametrize("dt", [BF16, F16])
def test_loss_ignores_what_ignored_tokens_hold(dt):
    T, V, dim = 150, 600, 96
    h, w, y, valid = loss_case(47, T, V, dim, 0.4, dt)
    gl = torch.rand(T, generator=gen(48), device=DEV)
    f = lm.VocabLoss(V, dim, dt)
    loss, lse = f.forward(h, w, y)
    a = f.backward(h, w, y, lse, gl)
    h2, gl2 = h.clone(), gl.clone()
    h2[~valid] = math.nan
    gl2[~valid] = math.inf
    loss2, lse2 = f.forward(h2, w, y)
    b = f.backward(h2, w, y, lse2, gl2)
    assert torch.equal(loss, loss2) and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dt", [BF16, F16])
def test_loss_without_targets(dt):
    T, V, dim = 40, 300, 64
    h, w, y, _ = loss_case(49, T, V, dim, 0.0, dt)
    y[:] = -100
    f = lm.VocabLoss(V, dim, dt)
    loss, lse = f.forward(h, w, y)
    assert bool((loss == 0).all()) and bool((lse == 0).all())
    gh, gw = f.backward(h, w, y, lse, torch.ones(T, device=DEV))
    assert bool((gh == 0).all()) and bool((gw == 0).all())
    # no tokens at all
    e = torch.empty(0, dim, dtype=dt, device=DEV)
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    loss, lse = f.forward(e, w, none)
    assert loss.numel() == 0
    gh, gw = f.backward(e, w, none, lse, torch.ones(1, device=DEV))
    assert gh.shape == (0, dim) and bool((gw == 0).all())


def test_loss_targets_out_of_range():
    T, V, dim = 40, 300, 64
    h, w, y, valid = loss_case(50, T, V, dim, 0.0, BF16)
    f = lm.VocabLoss(V, dim, BF16)
    y[3], y[20], y[39] = V, -7, 1 << 40
    bad = torch.zeros(T, dtype=torch.bool, device=DEV)
    bad[[3, 20, 39]] = True
    loss, lse = f.forward(h, w, y)
    assert D.ddp_lm_status(reset=True) == 2
    assert bool((loss[bad] == 0).all()) and bool((loss[~bad] > 0).all())
    gh, _ = f.backward(h, w, y, lse, torch.ones(1, device=DEV))
    assert bool((gh[bad] == 0).all()) and D.ddp_lm_status(reset=True) == 2


@pytest.mark.parametrize("dt", [BF16, F16])
def test_loss_of_large_and_infinite_logits(dt):
    V, dim = 1000, 64
    w = torch.zeros(V, dim, dtype=dt, device=DEV)
    w[:, 0] = torch.arange(V, device=DEV).to(dt) * 8
    h = torch.zeros(3, dim, dtype=dt, device=DEV)
    h[0, 0], h[1, 0], h[2, 0] = 16.0, -16.0, 0.0
    y = torch.tensor([V - 1, 0, 5], device=DEV)
    loss, lse = lm.VocabLoss(V, dim, dt).forward(h, w, y)
    z = h.double() @ w.double().t()
    want = torch.logsumexp(z, 1)
    within(lse, want, want.abs() * 2.0 ** -20 + 2.0 ** -18)
    h[1, 0] = math.inf     # an infinite logit: NaN for that token, nothing for the others
    l2, _ = lm.VocabLoss(V, dim, dt).forward(h, w, y)
    assert bool(l2[1].isnan()) and torch.equal(l2[[0, 2]], loss[[0, 2]])


@pytest.mark.parametrize("dt", [BF16, F16])
def test_loss_gradient_against_differences(dt):
    """(L(h + e d) - L(h - e d)) / 2e against <dH, d>, and the same for the weight.

    Along d the logits move at rates of at most A, so the third derivative of a token's loss is below (2A)^3 and
    the quotient is off by e^2/6 (2A)^3, plus the losses' own errors over e, plus the gradients'."""
    T, V, dim, e = 24, 200, 32, 2.0 ** -4
    g = gen(51)
    # multiples of 2^-4 below 8: inputs and moved inputs are exact in both types
    h = (torch.randint(-31, 32, (T, dim), generator=g, device=DEV) / 16.0).to(dt)
    w = (torch.randint(-7, 8, (V, dim), generator=g, device=DEV) / 16.0).to(dt)
    # one coordinate of each row moves, so that the rates stay small
    dh = torch.nn.functional.one_hot(torch.randint(0, dim, (T,), generator=g, device=DEV), dim).to(dt)
    dw = torch.nn.functional.one_hot(torch.randint(0, dim, (V,), generator=g, device=DEV), dim).to(dt)
    y = torch.randint(0, V, (T,), generator=g, device=DEV)
    f = lm.VocabLoss(V, dim, dt)
    _, lse = f.forward(h, w, y)
    gl = torch.ones(T, device=DEV)
    gh, gw = f.backward(h, w, y, lse, gl)
    valid = torch.ones(T, dtype=torch.bool, device=DEV)
    r = loss64(h, w, y, valid, gl)
    eg = r["dg"] + (U[dt] + 400 * 2.0 ** -23) * r["g"].abs() + 2.0 ** -39
    for move, grad, direction, rate, tol in (
            (lambda s: f.forward(h + s * e * dh, w, y)[0], gh, dh, dh.double() @ w.double().t(),
             ((eg @ r["W"].abs() + (r["g"] @ r["W"]).abs() * U[dt]) * dh.double().abs()).sum()),
            (lambda s: f.forward(h, w + s * e * dw, y)[0], gw, dw, h.double() @ dw.double().t(),
             ((eg.t() @ r["H"].abs() + (r["g"].t() @ r["H"]).abs() * U[dt]) * dw.double().abs()).sum())):
        q = (move(1).double() - move(-1).double()).sum() / (2 * e)
        A = rate.abs().max(1).values
        err = (e * e / 6 * (2 * A) ** 3).sum() + 2 * r["dloss"].sum() / e + tol
        assert abs(float(q - (grad.double() * direction.double()).sum())) <= float(err)
        assert float(err) < 0.5 * float(A.sum())   # the bound says something


def test_loss_on_another_stream():
    T, V, dim = 300, 2000, 128
    h, w, y, _ = loss_case(52, T, V, dim, 0.1, BF16)
    f = lm.VocabLoss(V, dim, BF16)
    loss, lse = f.forward(h, w, y)
    gl = torch.ones(1, device=DEV)
    want = f.backward(h, w, y, lse, gl)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    l2, e2 = f.forward(h, w, y, stream=s)
    got = f.backward(h, w, y, e2, gl, stream=s)
    s.synchronize()
    assert torch.equal(loss, l2) and torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_loss_many_calls_in_a_row():
    """Calls of mixed tiles (few rows: the hidden states' gradient is split along the vocabulary) without a pause:
    no wait may run out, and every call gives the same bits."""
    T, V, dim = 864, 20000, 1086
    h, w, y, _ = loss_case(70, T, V, dim, 0.0, BF16)
    f = lm.VocabLoss(V, dim, BF16)
    loss, lse = f.forward(h, w, y)
    gl = torch.full((1,), 1.0 / T, device=DEV)
    gh, gw = f.backward(h, w, y, lse, gl)
    for _ in range(300):
        l2, e2 = f.forward(h, w, y)
        gh2, gw2 = f.backward(h, w, y, e2, gl)
    torch.cuda.synchronize()
    assert D.ddp_lm_status() == 0
    assert torch.equal(loss, l2) and torch.equal(gh, gh2) and torch.equal(gw, gw2)
