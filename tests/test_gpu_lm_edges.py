"""Clipping, embedding and vocabulary loss where memory, streams, ranges of values and
paths are out of the ordinary: what a dropped object's memory may become, losses whose
weights differ by many orders of magnitude, shapes that take the rarer branches.

Tolerances are derived as in test_gpu_lm.py (u: a type's unit roundoff), from which the
helpers come."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no CUDA device", allow_module_level=True)

import allreduce_ddp_assign_gb300 as D
from allreduce_ddp_assign_gb300 import lm
from allreduce_ddp_assign_gb300.session import BucketReducer
from test_gpu_lm import (BF16, DEV, F16, F32, NORM_REL, TINY, U, check_grads, embed_grad64, gen, loss64, loss_case, norm64,
                         randn, within)


@pytest.fixture(autouse=True)
def clean_status():
    D.ddp_lm_status(reset=True)
    yield
    torch.cuda.synchronize()


def busy_stream():
    """A stream with about half a second of waiting queued on it, after the current stream's work."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(1_000_000_000)
    return s


def addresses_given_out(like, copies=17):
    """Where the allocator puts new tensors of these sizes (nothing is written to them)."""
    kept = [torch.empty_like(t) for t in like for _ in range(copies)]
    return {t.data_ptr() for t in kept}


# ---------------------------------------------------------------------------
# memory in use on another stream
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("call", ["norm", "clip"])
def test_a_dropped_clipper_keeps_its_memory_until_the_stream_is_done(call):
    g = [randn(gen(k), 3001 + k) for k in range(5)]
    ref = norm64(g, False)
    out = [torch.empty_like(t) for t in g]
    c = lm.GradClipper(g, out=out)
    held = [c._tables] + g + out
    places, sizes = {t.data_ptr() for t in held}, [torch.empty_like(t, device="meta") for t in held]
    # first uses and memory for the tensors below may wait for the GPU: they come before, for one copy
    # less, so that the check has to take a block that was not free before
    c.norm(), c.clip(1.0), addresses_given_out([torch.empty_like(t, device=DEV) for t in sizes], 16)
    s = busy_stream()
    got = c.clip(0.5 * ref, stream=s) if call == "clip" else c.norm(stream=s)
    del c, g, out, held
    new = addresses_given_out([torch.empty_like(t, device=DEV) for t in sizes])
    waiting = not s.query()
    assert not places & new
    assert waiting   # else the check says nothing
    s.synchronize()
    assert abs(float(got) - ref) <= NORM_REL * ref


def test_a_clipper_holds_its_tensors_whatever_becomes_of_the_lists():
    g = [randn(gen(9), 5000), None, randn(gen(10), 70)]
    out = [torch.empty_like(t) if t is not None else None for t in g]
    ref = norm64(g, False)
    places = {t.data_ptr() for t in g + out if t is not None}
    sizes = [torch.empty_like(t) for t in g if t is not None]
    c = lm.GradClipper(g, out=out)
    g.clear()
    out[:] = [None] * 3
    assert not places & addresses_given_out(sizes)
    assert abs(float(c.clip(1.0)) - ref) <= NORM_REL * ref


def test_tensors_passed_to_another_stream_may_be_dropped():
    V, dim, T = 500, 72, 1100
    held = dict(weight=randn(gen(1), V, dim, dtype=BF16), hidden=randn(gen(2), T, dim, dtype=BF16),
                ids=torch.randint(0, V, (T,), generator=gen(3), device=DEV), lse=None,
                gl=torch.rand(T, generator=gen(4), device=DEV))
    e, f = lm.TokenEmbedding(V, dim, BF16), lm.VocabLoss(V, dim, BF16)

    def calls(h, **on):
        x = e.forward(h["weight"], h["ids"], **on)
        gw = e.backward(h["hidden"], h["ids"], **on)
        loss, lse = f.forward(h["hidden"], h["weight"], h["ids"], **on)
        gh, gw2 = f.backward(h["hidden"], h["weight"], h["ids"], h["lse"], h["gl"], **on)
        return x, gw, loss, lse, gh, gw2

    held["lse"] = f.forward(held["hidden"], held["weight"], held["ids"])[1].clone()
    want = calls(held)
    places, sizes = {t.data_ptr() for t in held.values()}, [torch.empty_like(t) for t in held.values()]
    addresses_given_out(sizes, 16)
    with torch.cuda.stream(warm := torch.cuda.Stream()):   # its scratch memory and outputs
        warm.wait_stream(torch.cuda.default_stream())
        calls(held)
        warm.synchronize()
    with torch.cuda.stream(warm):
        torch.cuda._sleep(1_000_000_000)
    got = calls(held, stream=warm)
    held.clear()
    new = addresses_given_out(sizes)
    waiting = not warm.query()
    assert not places & new
    assert waiting   # else the check says nothing
    warm.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


# ---------------------------------------------------------------------------
# losses whose weights differ by many orders of magnitude
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("T,piece,largest", [(90, 0, 1.0), (90, 512, 65536.0), (700, 0, 1024.0)])
def test_loss_gradients_of_tokens_with_very_different_weights(dt, aligned, T, piece, largest):
    """Every token's row of grad_hidden is right beside its own grad_loss, however small that is beside the others'.

    G' = (p - onehot) r 2^14 in fp16, r the token's grad_loss over the largest, or between 2^-10 and 2^-9 where that is
    smaller: off by one rounding (u) or half of the smallest step, 2^-25 / (r 2^14), at most 2^-29 of the token's own
    grad_loss where r was moved and 2^-39 of the largest elsewhere.  Where r was moved by 2^k the weight's gradient
    takes the hidden state times 2^-k: off by half of the smallest step, 2^-25 2^k."""
    V, dim = 3000, 64
    h, w, y, valid = loss_case(80, T, V, dim, 0.1, dt, aligned)
    size = 10.0 ** -(2.25 * (torch.arange(T, device=DEV) % 5).double())   # 1 to 1e-9
    gl = ((torch.rand(T, generator=gen(81), device=DEV).double() + 0.25) * size * largest).float()
    f = lm.VocabLoss(V, dim, dt, piece=piece)
    _, lse = f.forward(h, w, y)
    gw = torch.empty(V, dim, dtype=F32, device=DEV)
    gh, _ = f.backward(h, w, y, lse, gl, grad_weight=gw)
    r = loss64(h, w, y, valid, gl)
    g, gv = r["g"], gl.double()[valid][:, None]
    gmax = float(gv.max())
    K = max(T, V)
    eg = r["dg"] + (U[dt] + 4 * 2.0 ** -24 + (K + 2) * 2.0 ** -23) * g.abs()
    moved = gv / gmax < 2.0 ** -10
    back = torch.zeros_like(gv)
    if dt == F16:
        eg = eg + torch.where(moved, gv * 2.0 ** -29, torch.full_like(gv, gmax * 2.0 ** -39))
        k = -10 - torch.floor(torch.log2(gv / gmax))
        back = torch.where(moved, 2.0 ** (k - 25), back)
    else:
        eg = eg + 2.0 ** -133
    want = g @ r["W"]
    tol = eg @ r["W"].abs() + want.abs() * (U[dt] + 2.0 ** -23) + TINY[dt]
    got, top = gh[valid].double(), (65504.0 if dt == F16 else 3e38)
    fits = want.abs() + tol < top
    within(got[fits], want[fits], tol[fits], "grad_hidden")
    over = want.abs() - tol > 65520.0 if dt == F16 else ~fits
    assert bool((got[over].abs() == float("inf")).all())
    want = g.t() @ r["H"]
    tol = eg.t() @ r["H"].abs() + (g.abs().t() @ back.expand(-1, dim)) + want.abs() * 2.0 ** -23
    within(gw, want, tol, "grad_weight")
    # the rows of small weights are more than their target's term: the check above sees what the others add
    if dt == F16 and largest > 1:
        one = -gv * r["W"][y[valid]]
        small = (gv / gmax < 1e-5)[:, 0]
        e = (got - one).norm(dim=1)[small] / one.norm(dim=1)[small]
        assert float(e.median()) > 0.05


# ---------------------------------------------------------------------------
# gradients added straight into a reducer's main_grad
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("before", [5, 64])   # elements of the parameter before the table, as buckets pack them
def test_table_gradients_go_straight_into_main_grad(before):
    """Two replicas of a tied table: both gradients are added into fp32 views of main_grad, two micro-steps each, the
    reducer averages what is there (the table has no gradient tensor of its own) and the clip scales it.

    A gradient is off by what check_grads allows for each contribution; the average adds two roundings in fp32, the
    clip the norm's and the factor's."""
    W, V, dim, T = 2, 1009, 72, 300
    other = [torch.full((before,), 0.25 + w, device=DEV) for w in range(W)]
    r = BucketReducer([before, V * dim], None, W, D.DDP_ALLREDUCE, D.DDP_ORDER_REVERSE, 25 << 20, 1 << 20, 1,
                      [[other[w], None] for w in range(W)], coalesce=True)
    views = [r.view(1, w).view(V, dim) for w in range(W)]
    e, f = lm.TokenEmbedding(V, dim, BF16, scale=3.0), lm.VocabLoss(V, dim, BF16)
    table = randn(gen(90), V, dim, dtype=BF16, scale=0.3)
    gl = torch.full((1,), 1.0 / T, device=DEV)
    want, tol = torch.zeros(W, V, dim, dtype=torch.float64, device=DEV), torch.zeros(W, V, dim, dtype=torch.float64, device=DEV)
    r.main_grad.zero_()
    for w in range(W):
        for micro in range(2):
            ids = torch.randint(0, V, (T,), generator=gen(91 + 2 * w + micro), device=DEV)
            y = (ids * 7 + 3) % V
            h = e.forward(table, ids)
            _, lse = f.forward(h, table, y)
            dh, _ = f.backward(h, table, y, lse, gl, grad_weight=views[w], accumulate=True)
            e.backward(dh, ids, grad_weight=views[w], accumulate=True)
            q = loss64(h, table, y, torch.ones(T, dtype=torch.bool, device=DEV), gl.expand(T))
            eg = q["dg"] + (U[BF16] + 4 * 2.0 ** -24 + (max(T, V) + 2) * 2.0 ** -23) * q["g"].abs() + 2.0 ** -133
            s, mag = embed_grad64(dh, ids, V, 3.0, -1)
            want[w] += q["g"].t() @ q["H"] + s
            n = torch.bincount(ids, minlength=V).double()[:, None]
            # (four additions to what is there, each rounded)
            tol[w] += eg.t() @ q["H"].abs() + (n + 2) * 2.0 ** -24 * mag + 2.0 ** -22 * (q["g"].abs().t() @ q["H"].abs() + mag)
    local = [v.clone() for v in views]
    for w in range(W):
        within(local[w], want[w], tol[w], f"replica {w}")
    r.step(accumulate=True)
    mean = local[0] * 0.5 + local[1] * 0.5
    for w in range(W):
        assert torch.equal(views[w], mean)
        assert torch.equal(r.view(0, w), other[0] * 0.5 + other[1] * 0.5)
    ref = norm64([r.view(0, 0), mean], False)
    kept = mean.clone()
    norms = [lm.GradClipper.of_reducer(r, w).clip(0.5 * ref) for w in range(W)]
    for w in range(W):
        assert abs(float(norms[w]) - ref) <= NORM_REL * ref
        scaled = kept.double() * (0.5 * ref / (ref + 1e-6))
        within(views[w], scaled, scaled.abs() * (NORM_REL + 5 * 2.0 ** -24) + TINY[F32], "clipped")
    assert torch.equal(views[0], views[1])
    assert D.ddp_lm_status() == 0
    r.close()


# ---------------------------------------------------------------------------
# paths that only certain sizes take
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("T,V,dim", [
    (8300, 17003, 72),    # more than 32 row tiles, and two pieces of the vocabulary of the library's own choice
    (200, 700, 8456),     # more than 32 tiles along the width
])
def test_loss_of_many_tiles(T, V, dim, dt):
    h, w, y, valid = loss_case(100, T, V, dim, 0.05, dt)
    f = lm.VocabLoss(V, dim, dt)
    loss, lse = f.forward(h, w, y)
    r = loss64(h, w, y, valid)
    within(lse[valid], r["lse"], r["dlse"], "lse")
    within(loss[valid], r["loss"], r["dloss"], "loss")
    del r
    gl = torch.rand(T, generator=gen(101), device=DEV)
    gh, gw = f.backward(h, w, y, lse, gl)
    check_grads(h, w, y, valid, gl, gh, gw, torch.zeros_like(gw), dt)
    assert D.ddp_lm_status() == 0


@pytest.mark.parametrize("T,V,dim", [
    (5003, 300007, 12),    # more than 128 sorting CTAs
    (100003, 200003, 6),   # the same, and more tokens than their places have room for in shared memory
    (120001, 30522, 8),    # more tokens than room, 128 CTAs
])
@pytest.mark.parametrize("idt", [torch.int32, torch.int64])
@pytest.mark.parametrize("skip", [0, 1])   # ids that start off the 16-byte (8-byte) boundary
@pytest.mark.parametrize("accumulate", [False, True])
def test_embedding_gradient_of_long_lists_and_large_tables(T, V, dim, idt, skip, accumulate):
    g = gen(110)
    ids = torch.randint(0, V, (T + skip,), generator=g, device=DEV)
    ids = torch.where(torch.rand(T + skip, generator=g, device=DEV) < 0.3, ids % 50, ids)
    ids[T // 3:T // 3 + 400] = 7   # the padding id
    ids[11], ids[T // 2] = -3, V   # left out, and reported
    ids = ids.to(idt)[skip:]
    go = randn(g, T, dim)
    base = randn(g, V, dim) if accumulate else torch.zeros(V, dim, device=DEV)
    e = lm.TokenEmbedding(V, dim, F32, scale=1.5, padding_idx=7)
    gw = e.backward(go, ids, grad_weight=base.clone(), accumulate=accumulate)
    s, mag = embed_grad64(go, ids, V, 1.5, 7)
    n = torch.bincount(ids[(ids >= 0) & (ids < V)].long(), minlength=V).double()[:, None]
    tol = (n + 2) * 2.0 ** -24 * (mag + base.double().abs()) + TINY[F32]
    within(gw, s + base.double(), torch.where(mag > 0, tol, torch.zeros_like(tol)))
    assert torch.equal(gw, e.backward(go, ids.clone(), grad_weight=base.clone(), accumulate=accumulate))
    assert D.ddp_lm_status(reset=True) == 2


@pytest.mark.parametrize("idt", [torch.int32, torch.int64])
def test_targets_off_a_boundary(idt):
    T, V, dim = 300, 900, 64
    h, w, y, valid = loss_case(120, T, V, dim, 0.2, BF16)
    f = lm.VocabLoss(V, dim, BF16)
    off = torch.cat([y[:1], y]).to(idt)[1:]
    loss, lse = f.forward(h, w, y)
    gl = torch.rand(T + 1, generator=gen(121), device=DEV)[1:]
    a, b = f.backward(h, w, y, lse, gl), f.backward(h, w, off, lse, gl)
    assert all(torch.equal(p, q) for p, q in zip(f.forward(h, w, off) + b, (loss, lse) + a))


@pytest.mark.parametrize("T,V,dim,ignored,dt", [
    (864, 20000, 1086, 0.0, BF16), (2000, 9000, 512, 0.7, F16), (300, 30000, 128, 0.0, BF16), (8192, 3000, 64, 0.0, F16),
])
def test_each_of_many_calls_gives_the_same_bits(T, V, dim, ignored, dt):
    """Calls without a pause between them, every one compared with the first; no wait runs out."""
    h, w, y, _ = loss_case(130, T, V, dim, ignored, dt)
    f = lm.VocabLoss(V, dim, dt)
    loss, lse = f.forward(h, w, y)
    gl = torch.full((1,), 1.0 / T, device=DEV)
    gh, gw = f.backward(h, w, y, lse, gl)
    assert bool(torch.isfinite(loss).all()) and bool(torch.isfinite(gw).all())
    differ = torch.zeros((), dtype=torch.int64, device=DEV)
    for _ in range(300):
        l2, e2 = f.forward(h, w, y)
        gh2, gw2 = f.backward(h, w, y, e2, gl)
        differ += (l2 != loss).any() | (e2 != lse).any() | (gh2 != gh).any() | (gw2 != gw).any()
    assert int(differ) == 0
    assert D.ddp_lm_status() == 0
