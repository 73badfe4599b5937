"""GPU tests of rld_moe_dispatch, rld_moe_combine and their gradients against the
definitions in 64 bits, and of a whole MoE training step.

Bounds, derived (u = 2^-24; a result in fp32 is off by u of its value, one in BF16 by
h = 2^-8).  A dispatch copies: no error.  A sum over k choices and `add` is k fused
or single products and k + 1 additions, each off by u of a partial sum, all of them
at most S = sum |w row| + |add|: (2 k + 1) u S, then the result's rounding.  A row of
combine's gradient is one fp32 product and the result's rounding.  A weight's
gradient adds `width` products in some order: at most 2 width u sum |row dout|.
"""
import numpy as np
import pytest
import torch

import routed_lora_delta_amd as R
import workloads as W
from gpu_util import GroupedRun, require_gpu, say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
OUT = {True: 2.0 ** -24, False: 2.0 ** -8}
TINY = 2.0 ** -133  # half a BF16 subnormal's step


def dtype(f32):
    return torch.float32 if f32 else torch.bfloat16


class Routing:
    """Random choices of distinct experts, sorted as the router does; a share of the
    tokens routes nowhere, and a share of the other choices is missing as well."""

    def __init__(self, seed, T, k, experts=64, masked=0.1, missing=0.0):
        self.dev, self.T, self.k, self.n = require_gpu(), T, k, T * k
        rng = np.random.default_rng(seed)
        choice = np.argsort(rng.random((T, max(experts, k))), axis=1)[:, :k]
        choice[rng.random(T) < masked] = -1
        choice[rng.random((T, k)) < missing] = -1
        flat = choice.ravel()
        has = np.nonzero(flat >= 0)[0]
        order = has[np.argsort(flat[has], kind="stable")]
        self.routed = len(order)
        srows = np.full(self.n, -1)
        srows[:len(order)] = order
        places = np.full(self.n, -1)
        places[order] = np.arange(len(order))
        self.indices_h, self.srows_h, self.places_h = choice, srows, places
        self.indices, self.srows, self.places = (self.i32(v) for v in (choice, srows, places))
        self.rng = rng

    def i32(self, v):
        return torch.from_numpy(np.ascontiguousarray(v, np.int32)).to(self.dev)

    def rows_of(self, flat):
        """[T, k] row of each choice, -1 for none."""
        p = np.where(self.indices_h.ravel() >= 0, np.arange(self.n), -1) if flat else \
            self.places_h
        return torch.from_numpy(p.reshape(self.T, self.k)).to(self.dev)

    def randn(self, shape, f32, scale=1.0):
        g = torch.Generator(device=self.dev)
        g.manual_seed(int(self.rng.integers(1 << 30)))
        return (torch.randn(shape, generator=g, device=self.dev) * scale).to(dtype(f32))

    def tables(self, flat):
        return (None, None) if flat else (self.srows, self.places)


def spoiled(shape, f32, dev):
    """A buffer whose every element is the same odd value."""
    return torch.full(shape, 77.25, device=dev, dtype=dtype(f32))


def check_dispatch(r, width, f32, pad):
    x = r.randn((r.T, width + pad), f32)
    rows, places = spoiled((r.n, width + pad), f32, r.dev), torch.full((r.n + 1,), -7,
                                                                       dtype=torch.int32,
                                                                       device=r.dev)
    R.check(R.rld_moe_dispatch(x, f32, width + pad, r.T, r.k, width, r.srows, rows, width + pad,
                               places), "rld_moe_dispatch")
    want = spoiled((r.n, width + pad), f32, r.dev)
    token = torch.from_numpy(r.srows_h[:r.routed] // r.k).to(r.dev)
    want[:r.routed, :width] = x[token, :width]
    assert torch.equal(rows, want)  # the tail, and what lies behind width, as it was
    named = np.where(r.places_h >= 0, r.places_h, -7)
    assert np.array_equal(places.cpu().numpy(), np.append(named, -7))


def sum_of(rows, p, w, add, width):
    """(sum, sum of magnitudes) in 64 bits."""
    T, k = p.shape
    total = torch.zeros((T, width), dtype=torch.float64, device=rows.device)
    size = torch.zeros_like(total)
    for j in range(k):
        t = (p[:, j] >= 0).nonzero().flatten()
        v = rows[p[t, j], :width].double()
        if w is not None:
            v = v * w[t, j, None].double()
        total[t] += v
        size[t] += v.abs()
    if add is not None:
        total += add[:, :width].double()
        size += add[:, :width].double().abs()
    return total, size


def assert_sum(out, width, total, size, k, f32):
    err = (2 * k + 1) * U * size
    got = out[:, :width].double()
    assert bool(((got - total).abs() <= err + OUT[f32] * (total.abs() + err) + TINY).all())
    assert bool((out[:, width:] == 77.25).all())


def check_combine(r, width, f32, pad, flat, with_add, weighted=True):
    rows = r.randn((r.n, width + pad), f32)
    w = r.randn((r.T, r.k), True)
    add = r.randn((r.T, width + pad), f32) if with_add else None
    out = spoiled((r.T, width + pad), f32, r.dev)
    s, p = r.tables(flat)
    ld = width + pad
    if weighted:
        st = R.rld_moe_combine(rows, f32, ld, r.indices, s, p, w, r.T, r.k, width, add, ld, out,
                               ld)
    else:
        st = R.rld_moe_dispatch_grad(rows, f32, ld, s, p, r.T, r.k, width, add, ld, out, ld)
    R.check(st, "sum")
    total, size = sum_of(rows, r.rows_of(flat), w if weighted else None, add, width)
    assert_sum(out, width, total, size, r.k, f32)


def check_grad(r, width, f32, pad, flat, want_rows=True, want_w=True, in_place=False):
    ld = width + pad
    rows, dout = r.randn((r.n, ld), f32), r.randn((r.T, ld), f32)
    w = r.randn((r.T, r.k), True)
    kept = rows.clone()
    drows = rows if in_place else spoiled((r.n, ld), f32, r.dev)
    before = drows.clone()
    dw = torch.full((r.n + 1,), 77.25, device=r.dev)
    s, p = r.tables(flat)
    R.check(R.rld_moe_combine_grad(rows if want_w else None, f32, ld, r.indices, s, p,
                                   w if want_rows else None, dout, ld, r.T, r.k, width,
                                   drows if want_rows else None, ld, dw if want_w else None),
            "rld_moe_combine_grad")
    at = r.rows_of(flat)
    if want_rows:
        want = before.double()
        for j in range(r.k):
            t = (at[:, j] >= 0).nonzero().flatten()
            want[at[t, j], :width] = w[t, j, None].double() * dout[t, :width].double()
        err = U * want.abs()
        owned = torch.zeros(r.n, dtype=torch.bool, device=r.dev)
        owned[at[at >= 0]] = True
        off = (drows.double() - want).abs()
        assert bool((off <= (err + OUT[f32] * (want.abs() + err) + TINY) * owned[:, None]).all())
        assert torch.equal(drows[:, width:], before[:, width:])
    else:
        assert torch.equal(drows, before)
    if want_w:
        for j in range(r.k):
            t = at[:, j] >= 0
            prod = kept[at[:, j].clamp(min=0), :width].double() * dout[:, :width].double()
            want = torch.where(t, prod.sum(1), 0.0)
            err = torch.where(t, 2 * width * U * prod.abs().sum(1), 0.0) + U * want.abs()
            got = dw[:-1].view(r.T, r.k)[:, j].double()
            assert bool(((got - want).abs() <= err).all())
        assert float(dw[-1]) == 77.25
    else:
        assert bool((dw == 77.25).all())


# one token to more than a launch's worth of rows; every number of waves a token and of
# units a lane, whole and partial ones; choices below, at and above a batch of eight
SHAPES = [(1, 1, 8, 0), (1, 8, 2048, 0), (2, 32, 72, 8), (3, 5, 520, 8), (33, 8, 512, 0),
          (64, 2, 1000, 64), (129, 9, 1032, 0), (257, 4, 4104, 8), (333, 17, 64, 0),
          (70, 1, 2048, 8), (5, 3, 8200, 0), (67, 32, 128, 8), (301, 7, 200, 8),
          (95, 2, 256, 0), (1500, 8, 2048, 0)]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,k,width,pad", SHAPES)
def test_every_operator(T, k, width, pad, f32):
    say(f"case: move T={T} k={k} width={width} pad={pad} f32={f32}")
    r = Routing(T + k, T, k, missing=0.05)
    check_dispatch(r, width, f32, pad)
    check_combine(r, width, f32, pad, False, True)
    check_combine(r, width, f32, pad, False, False, weighted=False)
    check_combine(r, width, f32, pad, False, True, weighted=False)
    check_combine(r, width, f32, pad, True, False)
    check_grad(r, width, f32, pad, False)
    check_grad(r, width, f32, pad, True)


@pytest.mark.parametrize("T,k,width,pad,f32", [
    (2500, 8, 1024, 64, False), (2500, 8, 1024, 0, True), (1100, 32, 576, 0, False),
    (40000, 8, 64, 64, False), (9000, 32, 64, 0, False), (9000, 32, 32, 0, True),
    (20000, 8, 128, 0, True),
    (50000, 8, 200, 0, False),
    (5000, 8, 2056, 8, False), (3500, 11, 1000, 0, True)])
def test_dispatch_in_two_launches(T, k, width, pad, f32):
    """Rows of whole cache lines above 32 MB of reads saved, others above 128 MB."""
    say(f"case: dispatch in two launches T={T} k={k} width={width} pad={pad} f32={f32}")
    size = 4 if f32 else 2
    lines = width * size % 128 == 0 and pad * size % 128 == 0
    assert T * (k - 1) * width * size >= (32 if lines else 128) << 20
    check_dispatch(Routing(T, T, k, missing=0.05), width, f32, pad)


@pytest.mark.parametrize("masked,missing", [(1.0, 0.0), (0.0, 1.0), (0.0, 0.0), (0.5, 0.5)])
def test_tokens_that_route_nowhere(masked, missing):
    say(f"case: masked {masked} missing {missing}")
    for k in (3, 12):
        r = Routing(5, 70, k, masked=masked, missing=missing)
        check_dispatch(r, 264, False, 8)
        for flat in (False, True):
            check_combine(r, 264, False, 8, flat, True)
            check_combine(r, 264, True, 8, flat, False)
            check_grad(r, 264, False, 8, flat)


@pytest.mark.parametrize("want_rows,want_w", [(True, False), (False, True)])
@pytest.mark.parametrize("flat", [False, True])
def test_gradient_of_one_output(want_rows, want_w, flat):
    say("case: one gradient")
    check_grad(Routing(6, 45, 11, missing=0.1), 1000, False, 8, flat, want_rows, want_w)


@pytest.mark.parametrize("f32", [False, True])
def test_in_place(f32):
    """drows in rows' memory, and a sum in that of `add`."""
    say("case: in place")
    r = Routing(7, 200, 10, missing=0.05)
    check_grad(r, 2056, f32, 8, False, in_place=True)
    check_grad(r, 136, f32, 0, True, in_place=True)
    rows, w = r.randn((r.n, 2056), f32), r.randn((r.T, r.k), True)
    for weighted in (True, False):
        out = r.randn((r.T, 2064), f32)
        out[:, 2056:] = 77.25
        add = out.clone()
        if weighted:
            st = R.rld_moe_combine(rows, f32, 2056, None, r.srows, r.places, w, r.T, r.k, 2056,
                                   out, 2064, out, 2064)
        else:
            st = R.rld_moe_dispatch_grad(rows, f32, 2056, r.srows, r.places, r.T, r.k, 2056, out,
                                         2064, out, 2064)
        R.check(st, "sum in place")
        total, size = sum_of(rows, r.rows_of(False), w if weighted else None, add, 2056)
        assert_sum(out, 2056, total, size, r.k, f32)


def test_every_flat_row_without_indices():
    say("case: flat order, no indices")
    r = Routing(8, 37, 6, masked=0.0)
    check = R.rld_moe_combine
    rows, w = r.randn((r.n, 128), False), r.randn((r.T, r.k), True)
    out = spoiled((r.T, 128), False, r.dev)
    R.check(check(rows, False, 128, None, None, None, w, r.T, r.k, 128, None, 0, out, 128), "flat")
    total, size = sum_of(rows, r.rows_of(True), w, None, 128)
    assert_sum(out, 128, total, size, r.k, False)


def test_places_may_hold_anything_where_nothing_was_dispatched():
    """Choices that no sorted row names, as in a share of the experts: whatever their
    entries of places hold, rows of others among them, they find no row; rows that
    belong to nobody, NaN and infinite ones, do not count, nor do missing choices'
    NaN weights."""
    say("case: stale places")
    for trial in range(3):
        r = Routing(20 + trial, 150, 9, missing=0.3)
        r.srows_h[:r.routed // 2] = r.srows_h[r.routed - r.routed // 2:r.routed]
        r.srows_h[r.routed // 2:] = r.rng.choice([-1, -5, r.n, 2 ** 31 - 1, -2 ** 31],
                                                 r.n - r.routed // 2)
        has = np.nonzero((r.srows_h >= 0) & (r.srows_h < r.n))[0]
        stale = r.rng.integers(-3, r.n, r.n)
        stale[r.rng.random(r.n) < 0.2] = 2 ** 31 - 1
        stale[r.srows_h[has]] = has
        real = np.full(r.n, -1)
        real[r.srows_h[has]] = has
        r.places_h, r.srows, r.places = real, r.i32(r.srows_h), r.i32(stale)
        width = 520
        rows = r.randn((r.n, width), False)
        lost = np.setdiff1d(np.arange(r.n), has)
        rows[torch.from_numpy(lost).to(r.dev)] = torch.tensor(
            [np.nan, np.inf] * (width // 2), dtype=torch.bfloat16, device=r.dev)
        w = r.randn((r.T, r.k), True)
        w[r.rows_of(False) < 0] = np.nan
        dout = r.randn((r.T, width), False)
        out, drows = spoiled((r.T, width), False, r.dev), spoiled((r.n, width), False, r.dev)
        dw = torch.zeros((r.T, r.k), device=r.dev)
        R.check(R.rld_moe_combine(rows, False, width, r.indices, r.srows, r.places, w, r.T, r.k,
                                  width, None, 0, out, width), "combine")
        total, size = sum_of(rows, r.rows_of(False), w, None, width)
        assert_sum(out, width, total, size, r.k, False)
        R.check(R.rld_moe_combine_grad(rows, False, width, r.indices, r.srows, r.places, w, dout,
                                       width, r.T, r.k, width, drows, width, dw), "combine_grad")
        assert torch.isfinite(dw).all() and bool((dw[r.rows_of(False) < 0] == 0).all())
        assert bool((drows[torch.from_numpy(lost).to(r.dev)] == 77.25).all())
        # and a dispatch by these tables writes those rows and places alone
        rows2, places2 = spoiled((r.n, width), False, r.dev), r.places.clone()
        R.check(R.rld_moe_dispatch(dout, False, width, r.T, r.k, width, r.srows, rows2, width,
                                   places2), "dispatch")
        assert torch.equal(places2, r.places)
        assert bool((rows2[torch.from_numpy(lost).to(r.dev)] == 77.25).all())
        token = torch.from_numpy(r.srows_h[has] // r.k).to(r.dev)
        assert torch.equal(rows2[torch.from_numpy(has).to(r.dev)], dout[token])


def test_values_that_are_not_finite_reach_their_token_alone():
    say("case: infinities and NaN")
    r = Routing(9, 60, 4, masked=0.0)
    rows, w = r.randn((r.n, 64), False), r.randn((r.T, r.k), True).abs() + 0.5
    at = r.rows_of(False)
    rows[at[7, 1], 3], rows[at[9, 0], 5], rows[at[9, 2], 5] = np.inf, np.inf, -np.inf
    w[11, 3] = np.nan
    out, dout = spoiled((r.T, 64), False, r.dev), torch.ones((r.T, 64), device=r.dev).bfloat16()
    R.check(R.rld_moe_combine(rows, False, 64, None, r.srows, r.places, w, r.T, r.k, 64, None, 0,
                              out, 64), "combine")
    o = out.float().cpu().numpy()
    assert o[7, 3] == np.inf and np.isnan(o[9, 5]) and np.isnan(o[11]).all()
    o[7, 3] = o[9, 5] = o[11] = 0
    assert np.isfinite(o).all()
    drows, dw = spoiled((r.n, 64), False, r.dev), torch.zeros((r.T, r.k), device=r.dev)
    R.check(R.rld_moe_combine_grad(rows, False, 64, None, r.srows, r.places, w, dout, 64, r.T,
                                   r.k, 64, drows, 64, dw), "combine_grad")
    d, g = dw.cpu().numpy(), drows.float().cpu().numpy()
    assert d[7, 1] == np.inf and d[9, 0] == np.inf and d[9, 2] == -np.inf
    assert np.isinf(d).sum() == 3 and not np.isnan(d).any()
    assert np.isnan(g[int(at[11, 3])]).all() and np.isnan(g).sum() == 64


def test_a_token_alone_has_the_batch_bits():
    say("case: batch against one token")
    r = Routing(10, 90, 8, masked=0.1)
    width = 1544
    rows, w, dout = r.randn((r.n, width), False), r.randn((r.T, r.k), True), r.randn(
        (r.T, width), False)
    out, drows = spoiled((r.T, width), False, r.dev), spoiled((r.n, width), False, r.dev)
    dw = torch.zeros((r.T, r.k), device=r.dev)
    R.check(R.rld_moe_combine(rows, False, width, r.indices, None, None, w, r.T, r.k, width,
                              None, 0, out, width), "combine")
    R.check(R.rld_moe_combine_grad(rows, False, width, r.indices, None, None, w, dout, width, r.T,
                                   r.k, width, drows, width, dw), "combine_grad")
    for t in (0, 41, 89):
        sl = slice(t * r.k, (t + 1) * r.k)
        o, d, g = out[:1].clone(), spoiled((r.k, width), False, r.dev), dw[:1].clone()
        R.check(R.rld_moe_combine(rows[sl], False, width, r.indices[t], None, None, w[t], 1, r.k,
                                  width, None, 0, o, width), "combine")
        R.check(R.rld_moe_combine_grad(rows[sl], False, width, r.indices[t], None, None, w[t],
                                       dout[t], width, 1, r.k, width, d, width, g), "grad")
        assert torch.equal(o[0], out[t]) and torch.equal(d, drows[sl]) and torch.equal(g[0], dw[t])


def test_far_rows():
    """Rows past 4 GB and past 2^31 elements."""
    say("case: far rows")
    r = Routing(11, 70001, 8, masked=0.02)
    width = 4096
    assert r.n * width > 2 ** 31 and r.n * width * 2 > 2 ** 32
    x = r.randn((r.T, width), False)
    rows = spoiled((r.n, width), False, r.dev)
    places = torch.full((r.n,), -1, dtype=torch.int32, device=r.dev)
    R.check(R.rld_moe_dispatch(x, False, width, r.T, r.k, width, r.srows, rows, width, places),
            "dispatch")
    token = torch.from_numpy(r.srows_h[:r.routed] // r.k).to(r.dev)
    for lo in range(0, r.routed, 1 << 16):
        hi = min(r.routed, lo + (1 << 16))
        assert torch.equal(rows[lo:hi], x[token[lo:hi]])
    assert bool((rows[r.routed:] == 77.25).all())
    assert np.array_equal(places.cpu().numpy(), r.places_h)
    # powers of two as weights: sums of eight equal rows are exact
    w = torch.full((r.T, r.k), 0.25, device=r.dev)
    out, dw = torch.zeros_like(x), torch.zeros((r.T, r.k), device=r.dev)
    R.check(R.rld_moe_combine(rows, False, width, None, r.srows, places, w, r.T, r.k, width, None,
                              0, out, width), "combine")
    live = torch.from_numpy(r.indices_h[:, 0] >= 0).to(r.dev)
    assert torch.equal(out[live], x[live] * 2) and bool((out[~live] == 0).all())
    dout = torch.ones_like(x)
    R.check(R.rld_moe_combine_grad(rows, False, width, None, r.srows, places, w, dout, width, r.T,
                                   r.k, width, rows, width, dw), "combine_grad")
    want = torch.where(live, x.double().sum(1), 0.0)
    err = 2 * width * U * x.double().abs().sum(1)
    assert bool(((dw.double() - want[:, None]).abs() <= err[:, None]).all())
    assert bool((rows[:r.routed] == 0.25).all()) and bool((rows[r.routed:] == 77.25).all())


@pytest.mark.parametrize("T,k,width", [(90, 4, 136), (2500, 8, 1024), (40000, 8, 64)])
def test_flat_rows_named_twice(T, k, width):
    """Against the rule, in one launch and in two: each of the two rows holds the token
    or what it held, the one that places names holds the token, and the other finds
    nobody."""
    say(f"case: flat rows named twice T={T} k={k} width={width}")
    r = Routing(50 + k, T, k)
    twice = r.rng.choice(r.routed // 2, r.routed // 10, replace=False)
    r.srows_h[twice + r.routed // 2] = r.srows_h[twice]
    srows = r.i32(r.srows_h)
    x = r.randn((T, width), False)
    rows, places = spoiled((r.n, width), False, r.dev), torch.full_like(r.places, -1)
    R.check(R.rld_moe_dispatch(x, False, width, T, k, width, srows, rows, width, places), "twice")
    p, f = places.cpu().numpy(), r.srows_h
    named = np.unique(f[f >= 0])
    assert np.array_equal(f[p[named]], named) and (np.delete(p, named) == -1).all()
    token = torch.from_numpy(np.where(f >= 0, f // k, 0)).to(r.dev)
    same = (rows == x[token]).all(1).cpu().numpy()
    left = (rows == 77.25).all(1).cpu().numpy()
    assert same[p[named]].all() and (same | left)[f >= 0].all() and left[f < 0].all()
    w, dw = r.randn((T, k), True), torch.zeros((T, k), device=r.dev)
    out = spoiled((T, width), False, r.dev)
    R.check(R.rld_moe_combine(rows, False, width, None, srows, places, w, T, k, width, None, 0,
                              out, width), "combine")
    r.places_h = p
    total, size = sum_of(rows, r.rows_of(False), w, None, width)
    assert_sum(out, width, total, size, k, False)
    drows = spoiled((r.n, width), False, r.dev)
    R.check(R.rld_moe_combine_grad(rows, False, width, None, srows, places, w, x, width, T, k,
                                   width, drows, width, dw), "combine_grad")
    other = np.setdiff1d(np.nonzero(f >= 0)[0], p[named])
    assert len(other) and bool((drows[torch.from_numpy(other).to(r.dev)] == 77.25).all())


@pytest.mark.parametrize("T,k,width", [((1 << 24) + 5, 2, 8), ((1 << 22) + 3, 2, 136)])
def test_very_many_tokens(T, k, width):
    """Small whole numbers, so that every value is exact: a token's rows are its row of
    x, their sum with weights 1/2 and 2 is 5/2 of it."""
    say(f"case: {T} tokens of {k} rows of {width}")
    dev, n = require_gpu(), T * k
    srows = torch.randperm(n, device=dev, dtype=torch.int32)
    places = torch.zeros_like(srows)
    x = (torch.arange(T, device=dev)[:, None] % 61 + torch.arange(width, device=dev) % 7
         ).to(torch.bfloat16)
    rows = torch.zeros((n, width), dtype=torch.bfloat16, device=dev)
    R.check(R.rld_moe_dispatch(x, False, width, T, k, width, srows, rows, width, places),
            "dispatch")
    assert torch.equal(srows[places.long()], torch.arange(n, device=dev, dtype=torch.int32))
    assert torch.equal(rows, x[torch.div(srows.long(), k, rounding_mode="floor")])
    w = torch.tensor([0.5, 2.0], device=dev).repeat(T, 1)
    out, dw = torch.zeros_like(x), torch.zeros_like(w)
    R.check(R.rld_moe_combine(rows, False, width, None, srows, places, w, T, k, width, None, 0,
                              out, width), "combine")
    assert torch.equal(out, (x.float() * 2.5).to(torch.bfloat16))
    dout = torch.ones_like(x)
    R.check(R.rld_moe_combine_grad(rows, False, width, None, srows, places, w, dout, width, T, k,
                                   width, rows, width, dw), "combine_grad")
    assert torch.equal(dw, x.float().sum(1, keepdim=True).expand(T, k))
    assert torch.equal(rows[:, 0].float(), w.reshape(-1)[srows.long()])
    R.check(R.rld_moe_dispatch_grad(rows, False, width, srows, places, T, k, width, x, width, out,
                                    width), "dispatch_grad")
    assert torch.equal(out, (x.float() + 2.5).to(torch.bfloat16))


def test_gradient_against_differences():
    """out is linear in the rows and in the weights: central differences of the 64-bit
    combine agree to the rounding of the gradient itself."""
    say("case: differences")
    r = Routing(12, 9, 5, missing=0.1)
    width = 40
    rows, w = r.randn((r.n, width), True), r.randn((r.T, r.k), True)
    dout = r.randn((r.T, width), True)
    drows, dw = torch.zeros_like(rows), torch.zeros_like(w)
    R.check(R.rld_moe_combine_grad(rows, True, width, None, r.srows, r.places, w, dout, width,
                                   r.T, r.k, width, drows, width, dw), "combine_grad")
    at = r.rows_of(False)

    def value(rows, w):
        return float((sum_of(rows, at, w, None, width)[0] * dout.double()).sum())

    # the values are sums of some 2000 terms below 60: exact to 1e-10, over a step of 1/4
    for _ in range(12):
        t, j, c = (int(r.rng.integers(v)) for v in (r.T, r.k, width))
        up, down = w.clone().double(), w.clone().double()
        up[t, j] += 0.125
        down[t, j] -= 0.125
        diff = (value(rows, up) - value(rows, down)) * 4
        size = float((rows[at[t, j].clamp(min=0)].double() * dout[t].double()).abs().sum())
        assert abs(diff - float(dw[t, j])) <= 1e-9 + 2 * width * U * size
        p = int(r.rng.integers(r.n))
        up, down = rows.clone().double(), rows.clone().double()
        up[p, c] += 0.125
        down[p, c] -= 0.125
        diff = (value(up, w) - value(down, w)) * 4
        assert abs(diff - float(drows[p, c])) <= 1e-9 + 2 * U * abs(diff)


def test_same_bits_every_run_and_graph_replays():
    """The four calls in one captured graph, replayed with new routing, eager work and
    synchronizations between the replays; on a stream that is not the current one."""
    say("case: move graph")
    T, k, width = 1300, 8, 2048  # the dispatch's two launches
    r = Routing(13, T, k)
    x, dout, w = r.randn((T, width), False), r.randn((T, width), False), r.randn((T, k), True)
    rows, drows = (torch.zeros((r.n, width), dtype=torch.bfloat16, device=r.dev)
                   for _ in range(2))
    out, dx = torch.zeros_like(x), torch.zeros_like(x)
    places, dw = torch.zeros_like(r.places), torch.zeros_like(w)

    def step(st=None):
        R.check(R.rld_moe_dispatch(x, False, width, T, k, width, r.srows, rows, width, places,
                                   st), "dispatch")
        R.check(R.rld_moe_combine(rows, False, width, None, r.srows, places, w, T, k, width, x,
                                  width, out, width, st), "combine")
        R.check(R.rld_moe_combine_grad(rows, False, width, None, r.srows, places, w, dout, width,
                                       T, k, width, drows, width, dw, st), "combine_grad")
        R.check(R.rld_moe_dispatch_grad(drows, False, width, r.srows, places, T, k, width, dout,
                                        width, dx, width, st), "dispatch_grad")

    bufs = (rows, places, out, drows, dw, dx)
    step()
    torch.cuda.synchronize()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step(s)
    for trial in range(4):
        new = Routing(30 + trial, T, k, masked=0.2)
        r.srows.copy_(new.srows)
        for b in bufs:
            b.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        replayed = [b.clone() for b in bufs]
        total, size = sum_of(rows, new.rows_of(False), w, x, width)
        assert_sum(out, width, total, size, k, False)
        for side in (None, torch.cuda.Stream()):
            for b in bufs:
                b.zero_()
            torch.cuda.synchronize()
            step(side)
            torch.cuda.synchronize()
            for a, b in zip(replayed, bufs):
                assert torch.equal(a, b)


# ------------------------------------------------------ used together ----

def test_dispatched_rows_fold_like_gathered_ones():
    """The grouped fold of gate over rows that the dispatch laid out has the bits of
    the fold that gathers its rows itself."""
    say("case: dispatch -> grouped fold")
    dev = require_gpu()
    m = W.moe_grouped(num_tokens=200, top_k=4, num_experts=16, hidden=256, inter=128, max_loras=3,
                      n_adapted=12, ranks=(8, 16), max_rank=16, cap=300, projections=("gate",))
    p = m.projections[0]
    want = GroupedRun(m, p, dev)
    want.run()
    # row r of the workload is choice sorted_topk_pos[r] of token sorted_token_ids[r]
    srows = torch.from_numpy((m.sorted_token_ids * 4 + m.sorted_topk_pos).astype(np.int32)).to(dev)
    x = torch.from_numpy(np.ascontiguousarray(p.x, np.uint16).view(np.int16)).to(dev)
    rows = torch.zeros((m.te, 256), dtype=torch.int16, device=dev)
    places = torch.zeros(m.te, dtype=torch.int32, device=dev)
    R.check(R.rld_moe_dispatch(x, False, 256, 200, 4, 256, srows, rows, 256, places), "dispatch")
    own = GroupedRun(m, p, dev)
    xa = torch.zeros((m.te, 16), dtype=torch.int16, device=dev)
    wb = R.rld_moe_grouped_workspace_bytes(m.te, 256, 16, 3, 16)
    ws = torch.zeros(max(16, wb), dtype=torch.uint8, device=dev)
    R.check(R.rld_moe_grouped(own.route.route, rows, 256, False, 200, own.off, 16, own.stid,
                              own.rad, 0, m.te, own.base.ptr(), 128, xa, m.te, ws, wb),
            "grouped")
    torch.cuda.synchronize()
    assert np.array_equal(want.base.body(), own.base.body())
    assert not np.array_equal(own.base.body(), p.base.ravel())


def test_training_step_of_an_moe_layer():
    """Router, dispatch, the experts' products (PyTorch's, fp32), combine onto the
    residual, and back through all of them: every gradient against PyTorch's own of
    the definition in 64 bits.  fp32 throughout, so that one bound serves: each value
    passes fewer than 600 roundings on any path (two products of 64 and 96 terms, sums
    over 4 choices, a softmax of 16 whose error test_gpu_router.py derives, twice
    over), so 2000 u of the largest value of its tensor is more than they add up to."""
    say("case: MoE training step")
    dev = require_gpu()
    T, k, E, H, I = 75, 4, 16, 64, 96
    g = torch.Generator().manual_seed(3)
    x, wg = torch.randn((T, H), generator=g), torch.randn((E, H), generator=g) / 8
    w1, w2 = torch.randn((E, H, I), generator=g) / 8, torch.randn((E, I, H), generator=g) / 10
    dout = torch.randn((T, H), generator=g)
    mask = (torch.rand(T, generator=g) > 0.1).int()

    # 64 bits, on the CPU, by autograd
    leaves = [t.double().requires_grad_() for t in (x, wg, w1, w2)]
    X, WG, W1, W2 = leaves
    logits = X @ WG.T
    prob = torch.softmax(logits, 1)
    idx = torch.argsort(logits, dim=1, descending=True, stable=True)[:, :k]
    top = prob.gather(1, idx)
    wts = top / top.sum(1, keepdim=True) * mask[:, None]
    ys = torch.stack([torch.tanh(X @ W1[e]) @ W2[e] for e in range(E)], 1)
    ref = X + (wts[:, :, None] * ys.gather(1, idx[:, :, None].expand(T, k, H))).sum(1)
    live = mask.sum().double()
    counts = torch.bincount(idx[mask > 0].flatten(), minlength=E).double()
    loss = E / (k * live ** 2) * (counts * (prob * mask[:, None]).sum(0)).sum()
    (ref * dout.double()).sum().add(loss * 3).backward()

    # the library's step
    xd, doutd, md = x.to(dev), dout.to(dev), mask.to(dev)
    i32 = dict(dtype=torch.int32, device=dev)
    n = T * k
    ind, cnt, off = torch.zeros((T, k), **i32), torch.zeros(E + 1, **i32), torch.zeros(E + 1, **i32)
    stok, srows, places = (torch.zeros(n, **i32) for _ in range(3))
    w, ls = torch.zeros((T, k), device=dev), torch.zeros(1, device=dev)
    need = R.rld_moe_router_workspace_bytes(T, E, k)
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    lg = (xd @ wg.to(dev).T).contiguous()
    R.check(R.rld_moe_router(lg, True, E, md, T, E, k, True, ind, w, cnt, off, stok, srows, ls, ws,
                             need), "router")
    rows = torch.full((n, H), np.nan, device=dev)
    R.check(R.rld_moe_dispatch(xd, True, H, T, k, H, srows, rows, H, places), "dispatch")
    ends = off.cpu().tolist()
    ys_d, hid = torch.full((n, H), np.nan, device=dev), torch.zeros((n, I), device=dev)
    w1d, w2d = w1.to(dev), w2.to(dev)
    for e in range(E):
        sl = slice(ends[e], ends[e + 1])
        hid[sl] = torch.tanh(rows[sl] @ w1d[e])
        ys_d[sl] = hid[sl] @ w2d[e]
    out = torch.zeros((T, H), device=dev)
    R.check(R.rld_moe_combine(ys_d, True, H, ind, srows, places, w, T, k, H, xd, H, out, H),
            "combine")
    dys, dw = torch.full((n, H), np.nan, device=dev), torch.zeros((T, k), device=dev)
    R.check(R.rld_moe_combine_grad(ys_d, True, H, ind, srows, places, w, doutd, H, T, k, H, dys, H,
                                   dw), "combine_grad")
    dl, dlg = torch.full((1,), 3.0, device=dev), torch.zeros((T, E), device=dev)
    R.check(R.rld_moe_router_grad(lg, True, E, md, T, E, k, True, ind, cnt, dw, dl, dlg, E),
            "router_grad")
    drows = torch.full((n, H), np.nan, device=dev)
    dw1, dw2 = torch.zeros_like(w1d), torch.zeros_like(w2d)
    for e in range(E):
        sl = slice(ends[e], ends[e + 1])
        dh = (dys[sl] @ w2d[e].T) * (1 - hid[sl] ** 2)
        dw2[e], dw1[e] = hid[sl].T @ dys[sl], rows[sl].T @ dh
        drows[sl] = dh @ w1d[e].T
    dx = torch.zeros((T, H), device=dev)
    R.check(R.rld_moe_dispatch_grad(drows, True, H, srows, places, T, k, H, doutd + dlg @
                                    wg.to(dev), H, dx, H), "dispatch_grad")
    torch.cuda.synchronize()
    assert np.array_equal(ind.cpu().numpy()[mask.numpy() > 0], idx.numpy()[mask.numpy() > 0])
    for got, want in ((out, ref.detach()), (ls, loss.detach()[None]), (dx, X.grad),
                      (dlg.T @ xd, WG.grad), (dw1, W1.grad), (dw2, W2.grad)):
        assert float((got.cpu().double() - want).abs().max()) <= 2000 * U * float(want.abs().max())


# rows of fewer than 16 units and of 17 to 31, which lanes of a group do not fill, whole
# ones beside them; a wave's lanes with one unit and with two, the last round partly full;
# one wave a token and several
@pytest.mark.parametrize("k,width,f32", [
    (4, 64, False), (3, 104, False), (12, 24, False), (1, 8, False), (5, 128, False),
    (8, 200, False), (1, 136, False), (2, 256, False), (2, 1000, False), (1, 520, False),
    (2, 1544, False), (1, 8200, False), (1, 2048, False), (9, 1032, False), (8, 2048, False),
    (4, 40, True), (8, 104, True), (2, 200, True), (2, 1032, True), (4, 2056, True)])
@pytest.mark.parametrize("flat", [False, True])
def test_gradient_of_values_that_are_not_finite(k, width, f32, flat):
    """Infinities and NaN among the last 16 bytes of a token's dout, and of a row: an
    infinite weight's gradient with the sign of its product, NaN where NaN is, and the
    other tokens as ever."""
    say(f"case: dout not finite k={k} width={width} f32={f32} flat={flat}")
    T, n = 37, 4 if f32 else 8
    r = Routing(60 + k, T, k, masked=0.0)
    rows, dout, w = r.randn((r.n, width), f32), r.randn((T, width), f32), r.randn((T, k), True)
    rows = torch.where(rows.abs() < 0.01, 0.5, rows.float()).to(dtype(f32))
    w = torch.where(w.abs() < 0.01, 0.5, w)
    at = r.rows_of(flat)
    dout[5, width - 1], dout[6, width - n], dout[20, width - 3] = np.inf, -np.inf, np.nan
    rows[at[30, 0], width - 1], dout[30, width - 1] = np.inf, -2.0
    drows, dw = spoiled((r.n, width), f32, r.dev), torch.zeros((T, k), device=r.dev)
    s, p = r.tables(flat)
    R.check(R.rld_moe_combine_grad(rows, f32, width, None, s, p, w, dout, width, T, k, width,
                                   drows, width, dw), "combine_grad")
    for t, c, sign in ((5, width - 1, 1.0), (6, width - n, -1.0)):
        assert torch.equal(dw[t], sign * np.inf * torch.sign(rows[at[t], c].float())), t
        for j in range(k):
            assert float(drows[at[t, j], c]) == sign * np.inf * np.sign(float(w[t, j]))
    assert bool(torch.isnan(dw[20]).all()) and bool(torch.isnan(drows[at[20], width - 3]).all())
    assert float(dw[30, 0]) == -np.inf
    assert int((~torch.isfinite(drows)).sum()) == 3 * k
    rest = torch.ones((T, k), dtype=torch.bool, device=r.dev)
    rest[[5, 6, 20]], rest[30, 0] = False, False
    prod = rows[at.clamp(min=0)].double() * dout[:, None, :].double()
    err = 2 * width * U * prod.abs().sum(2) + U * prod.sum(2).abs()
    assert bool(((dw.double() - prod.sum(2)).abs() <= err)[rest].all())


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,k,width", [(90, 5, 136), (301, 8, 64), (70, 2, 1000), (33, 9, 2056),
                                       (2500, 8, 1024), (12000, 8, 1000)])
def test_every_operand_with_a_stride_of_its_own(T, k, width, f32):
    """Five strides that differ, in one launch of the dispatch and in two, in both orders."""
    say(f"case: own strides T={T} k={k} width={width} f32={f32}")
    r = Routing(80 + k, T, k, missing=0.05)
    sx, sr, so, sd, sa = (width + 8 * v for v in (3, 1, 5, 0, 2))
    x, add = r.randn((T, sx), f32), r.randn((T, sa), f32)
    rows, w = spoiled((r.n, sr), f32, r.dev), r.randn((T, k), True)
    places = torch.full((r.n,), -7, dtype=torch.int32, device=r.dev)
    R.check(R.rld_moe_dispatch(x, f32, sx, T, k, width, r.srows, rows, sr, places), "dispatch")
    want = spoiled((r.n, sr), f32, r.dev)
    token = torch.from_numpy(r.srows_h[:r.routed] // k).to(r.dev)
    want[:r.routed, :width] = x[token, :width]
    assert torch.equal(rows, want)
    assert np.array_equal(places.cpu().numpy(), np.where(r.places_h >= 0, r.places_h, -7))
    rows, dout = r.randn((r.n, sr), f32), r.randn((T, sd), f32)
    for flat in (False, True):
        at, (s, p) = r.rows_of(flat), r.tables(flat)
        out = spoiled((T, so), f32, r.dev)
        R.check(R.rld_moe_combine(rows, f32, sr, r.indices, s, p, w, T, k, width, add, sa, out,
                                  so), "combine")
        assert_sum(out, width, *sum_of(rows, at, w, add, width), k, f32)
        if not flat:
            out = spoiled((T, so), f32, r.dev)
            R.check(R.rld_moe_dispatch_grad(rows, f32, sr, s, p, T, k, width, add, sa, out, so),
                    "dispatch_grad")
            assert_sum(out, width, *sum_of(rows, at, None, add, width), k, f32)
        drows, dw = spoiled((r.n, so), f32, r.dev), torch.full((T, k), 77.25, device=r.dev)
        R.check(R.rld_moe_combine_grad(rows, f32, sr, r.indices, s, p, w, dout, sd, T, k, width,
                                       drows, so, dw), "combine_grad")
        want = spoiled((r.n, so), f32, r.dev).double()
        for j in range(k):
            t = (at[:, j] >= 0).nonzero().flatten()
            want[at[t, j], :width] = w[t, j, None].double() * dout[t, :width].double()
            prod = rows[at[t, j], :width].double() * dout[t, :width].double()
            got, val = dw[t, j].double(), prod.sum(1)
            err = 2 * width * U * prod.abs().sum(1) + U * val.abs()
            assert bool(((got - val).abs() <= err).all())
        assert bool((dw[at < 0] == 0).all())
        err = U * want.abs()
        off = (drows.double() - want).abs()
        assert bool((off <= err + OUT[f32] * (want.abs() + err) + TINY).all())
        assert bool((drows[want == 77.25] == 77.25).all())
