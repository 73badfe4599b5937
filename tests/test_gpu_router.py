"""GPU tests of rld_moe_router and rld_moe_router_grad against the definition in 64
bits, and of the router together with the projection and the MoE fold.

Bounds, derived (u = 2^-24, every operation rounds to nearest; expf is taken to
be within 2 units, 2^-22 relative).  exp(l - top): the difference l - top is
rounded (u |l - top| relative in the exponential).  The sum of E terms is off by
at most E u relative (all are positive); each quotient adds u.  So a probability
is off by at most (spread u + 2^-22 + E u + 2 u) relative, spread = the largest
|l - top| whose exponential is not below fp32's range (104); below it the
absolute error is under 2^-125.
"""
import numpy as np
import pytest
import torch

import oracle as O
import routed_lora_delta_amd as R
import workloads as W
from gpu_util import GroupedRun, require_gpu, say
from routed_lora_delta_amd.pool import DenseRoute

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TINY = 2.0 ** -125
INF = np.inf
LOWEST = {False: -3.3895313892515355e38, True: -3.4028234663852886e38}  # BF16, fp32


def rel_p(logits):
    """Relative error of a probability, from the spread that reaches the result."""
    fin = np.where(np.isfinite(logits), logits, np.nan)
    with np.errstate(all="ignore"):
        import warnings
        with warnings.catch_warnings():
            warnings.simplefilter("ignore")
            spread = np.nanmax(fin, 1) - np.nanmin(fin, 1)
    spread = np.where(np.isnan(spread), 0, np.minimum(spread, 104))[:, None]
    return spread * U + 2.0 ** -22 + logits.shape[1] * U + 3 * U


def reference(l, mask, k, norm):
    """The definition, token by token, on float64 logits."""
    T, E = l.shape
    idx = np.full((T, k), -1, np.int64)
    w = np.zeros((T, k))
    p = np.zeros((T, E))
    N, bad_any = 0, False
    for t in range(T):
        if mask is not None and mask[t] == 0:
            continue
        row = l[t]
        if np.isnan(row).any() or (row == INF).any():
            N, bad_any = N + 1, True
            w[t] = np.nan
            continue
        if (row == -INF).all():
            continue
        N += 1
        e = np.exp(row - row.max())
        p[t] = e / e.sum()
        order = sorted([i for i in range(E) if row[i] > -INF], key=lambda i: (-row[i], i))[:k]
        idx[t, :len(order)] = order
        w[t, :len(order)] = p[t, order]
        if norm:
            # over the chosen logits alone, so that nothing underflows
            q = np.exp(row[order] - row[order].max())
            w[t, :len(order)] = q / q.sum()
    flat = idx.ravel()
    counts = np.bincount(flat[flat >= 0], minlength=E)
    rows = np.array(sorted(np.nonzero(flat >= 0)[0], key=lambda r: (flat[r], r // k)), np.int64)
    srows = np.full(T * k, -1, np.int64)
    srows[:len(rows)] = rows
    stok = np.where(srows >= 0, srows // k, -1)
    loss = 0.0 if N == 0 else E / (k * N * N) * (counts * p.sum(0)).sum()
    if bad_any:
        loss = np.nan
    return dict(idx=idx, w=w, p=p, counts=np.append(counts, N), stok=stok, srows=srows, loss=loss,
                off=np.concatenate([[0], np.cumsum(counts)]))


def to_bits(v):
    return (np.ascontiguousarray(v, np.float32).view(np.uint32) >> 16).astype(np.uint16)


class Router:
    """One batch of logits on the device, in rows wider than the experts."""

    def __init__(self, l, f32, mask=None, pad=0):
        self.dev = require_gpu()
        self.T, self.E = l.shape
        self.f32, self.pad, self.ls = f32, pad, self.E + pad
        if not f32:
            l = (to_bits(l).astype(np.uint32) << 16).view(np.float32)
        self.l = np.ascontiguousarray(l, np.float32).astype(np.float64)
        full = np.full((self.T, self.ls), np.nan, np.float32)
        full[:, :self.E] = l
        self.ld = torch.from_numpy(full).to(self.dev)
        if not f32:
            self.ld = torch.from_numpy(to_bits(full).view(np.int16)).to(self.dev)
        self.mask = mask
        self.md = None if mask is None else torch.from_numpy(mask.astype(np.int32)).to(self.dev)

    def buffers(self, k):
        i32 = dict(dtype=torch.int32, device=self.dev)
        self.k = k
        self.idx = torch.full((self.T * k + 1,), 77, **i32)
        self.w = torch.full((self.T * k + 1,), 77.0, device=self.dev)
        self.cnt, self.off = torch.full((self.E + 2,), 77, **i32), torch.full((self.E + 2,), 77,
                                                                             **i32)
        self.stok, self.srows = (torch.full((self.T * k + 1,), 77, **i32) for _ in range(2))
        self.loss = torch.full((2,), 77.0, device=self.dev)
        self.need = R.rld_moe_router_workspace_bytes(self.T, self.E, k)
        self.ws = torch.full((self.need + 64,), 0xFF, dtype=torch.uint8, device=self.dev)

    def launch(self, norm, stream=None, tables=True):
        t = (lambda v: v) if tables else (lambda v: None)
        return R.rld_moe_router(self.ld, self.f32, self.ls, self.md, self.T, self.E, self.k, norm,
                                self.idx, self.w, t(self.cnt), t(self.off), t(self.stok),
                                t(self.srows), t(self.loss), self.ws, self.need, stream)

    def results(self):
        torch.cuda.synchronize()
        for t in (self.idx, self.w, self.cnt, self.off, self.stok, self.srows, self.loss):
            assert float(t[-1]) == 77.0, "a buffer was overrun"
        assert bool((self.ws[self.need:] == 0xFF).all()), "the workspace was overrun"
        n = lambda t: t[:-1].cpu().numpy()  # noqa: E731
        return dict(idx=n(self.idx).reshape(self.T, self.k), w=n(self.w).reshape(self.T, self.k),
                    counts=n(self.cnt), off=n(self.off), stok=n(self.stok), srows=n(self.srows),
                    loss=n(self.loss)[0])

    def check(self, k, norm):
        self.buffers(k)
        R.check(self.launch(norm), "rld_moe_router")
        got, want = self.results(), reference(self.l, self.mask, k, norm)
        for key in ("idx", "counts", "off", "stok", "srows"):
            assert np.array_equal(got[key], want[key]), key
        rp = rel_p(self.l)
        nan = np.isnan(want["w"])
        assert np.array_equal(np.isnan(got["w"]), nan)
        tol = (2 + k) * rp * np.abs(want["w"]) + TINY
        assert (np.abs(got["w"] - want["w"])[~nan] <= tol[~nan]).all()
        if np.isnan(want["loss"]):
            assert np.isnan(got["loss"])
        else:
            # sums over the tokens: at most T additions of positive terms
            assert abs(got["loss"] - want["loss"]) <= \
                (rp.max() + (self.T + 8) * U) * want["loss"] + 1e-30
        return got, want

    def grad(self, got, norm, dw, dloss, pad=0, in_place=False, stream=None):
        os_ = self.ls if in_place else self.E + pad
        dt = torch.float32 if self.f32 else torch.int16
        out = self.ld if in_place else torch.full((self.T, os_), 77, dtype=dt, device=self.dev)
        idx = torch.from_numpy(np.ascontiguousarray(got["idx"], np.int32)).to(self.dev)
        cnt = torch.from_numpy(np.ascontiguousarray(got["counts"], np.int32)).to(self.dev)
        self.keep = (idx, cnt, dw, dloss)
        R.check(R.rld_moe_router_grad(self.ld, self.f32, self.ls, self.md, self.T, self.E,
                                      got["idx"].shape[1], norm, idx, cnt, dw, dloss, out, os_,
                                      stream), "rld_moe_router_grad")
        torch.cuda.synchronize()
        h = out.cpu().numpy()
        if not in_place:
            assert (h[:, self.E:] == 77).all(), "the rest of a row was written"
        h = h[:, :self.E]
        return h.astype(np.float64) if self.f32 else \
            (h.view(np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)

    def check_grad(self, k, norm, with_w=True, with_loss=True, in_place=False):
        got, want = self.check(k, norm)
        rng = np.random.default_rng(5)
        dw = rng.standard_normal((self.T, k)).astype(np.float32)
        dl = np.float32(0.37 * self.T)
        d = self.grad(got, norm, torch.from_numpy(dw).to(self.dev) if with_w else None,
                      torch.tensor([dl], device=self.dev) if with_loss else None, pad=3,
                      in_place=in_place)
        ref, mag = gradient(self.l, want, dw if with_w else None, dl if with_loss else 0.0, k,
                            norm)
        bad = np.isnan(want["w"]).any(1)
        assert np.isnan(d[bad]).all() and np.isfinite(d[~bad]).all()
        rp = np.broadcast_to(rel_p(self.l) * (4 + k) + (self.E + 12) * U, d.shape)
        err = rp * mag + TINY * (1 + np.abs(mag))
        tol = err if self.f32 else err + 2.0 ** -8 * (np.abs(ref) + err)
        off = np.abs(d - ref)[~bad]
        assert (off <= tol[~bad]).all(), float((off - tol[~bad]).max())
        return d


def gradient(l, want, dw, dloss, k, norm):
    """(gradient, sum of its terms' magnitudes) to the logits, in 64 bits."""
    T, E = l.shape
    p, idx, N = want["p"], want["idx"], want["counts"][E]
    h = dloss * E * want["counts"][:E] / (k * float(max(N, 1)) ** 2)
    h = np.broadcast_to(h, (T, E)).copy()
    mh = np.abs(h)
    d, m = np.zeros((T, E)), np.zeros((T, E))
    if dw is not None:
        for t in range(T):
            on = idx[t] >= 0
            if not on.any():
                continue
            e, g = idx[t][on], dw[t][on].astype(np.float64)
            if norm:
                q = want["w"][t][on]
                d[t, e] += q * (g - (q * g).sum())
                m[t, e] += q * (np.abs(g) + (q * np.abs(g)).sum())
            else:
                h[t, e] += g
                mh[t, e] += np.abs(g)
    d += p * (h - (p * h).sum(1, keepdims=True))
    m += p * (mh + (p * mh).sum(1, keepdims=True))
    return d, m


def logits_of(rng, T, E, odd=True):
    l = rng.standard_normal((T, E)).astype(np.float32) * 2
    if odd and T >= 8:
        l[1] = -INF                       # nothing left
        l[2, : max(1, E - 2)] = -INF      # fewer experts than places
        l[3] = 0.5                        # all equal
        l[4] = np.round(l[4])             # ties
        l[5, ::2] = -0.0
        l[5, 1::2] = 0.0                  # zeros of both signs are equal
        l[6] *= 40                        # probabilities that underflow
    return l


SIZES = [(128, 128, 8), (129, 40, 3), (66000, 8, 2), (1, 1, 1), (1, 128, 8), (3, 5, 5), (8, 2, 1), (32, 128, 8), (63, 60, 4), (64, 64, 6),
         (65, 65, 3), (130, 8, 8), (200, 129, 32), (257, 256, 8), (70, 257, 10), (90, 512, 8),
         (77, 513, 2), (66, 1024, 32), (1000, 160, 6)]


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_router_and_gradient(T, E, k, f32, norm):
    say(f"case: router {T} {E} {k} f32={f32} norm={norm}")
    rng = np.random.default_rng(T * 7 + E)
    mask = (rng.random(T) < 0.8).astype(np.int32) if T % 2 else None
    Router(logits_of(rng, T, E), f32, mask, pad=E % 3).check_grad(k, norm)


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("k", [1, 2, 3, 4, 5, 7, 8, 9, 17])
@pytest.mark.parametrize("E", [64, 129, 512, 1000])
def test_every_width_of_the_choice(E, k, f32):
    """Choices of each count, among many equal logits and rows with few finite ones."""
    rng = np.random.default_rng(E + k)
    l = np.round(logits_of(rng, 67, E, odd=False))  # few values: ties
    l[5] = -INF
    l[5, E // 2: E // 2 + 3] = 1.0
    l[6] = 0.0
    l[7] = -0.0
    l[7, ::2] = 0.0
    Router(l, f32).check(k, True)


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T,E,k", [(1, 513, 1), (1, 1024, 32), (64, 1024, 32), (63, 1000, 9),
                                   (64, 400, 8)])
def test_one_block_of_many_experts(T, E, k, f32):
    """Batches of one launch at the widest tables, and their gradients."""
    say(f"case: router one block {T} {E} {k} f32={f32}")
    rng = np.random.default_rng(E + T)
    Router(logits_of(rng, T, E), f32).check_grad(k, True)


def test_gradient_in_place_bf16():
    rng = np.random.default_rng(18)
    l = logits_of(rng, 90, 257)
    a = Router(l, False, pad=3).check_grad(8, False)
    b = Router(l, False, pad=3).check_grad(8, False, in_place=True)
    assert np.array_equal(a, b)


def test_two_routers_at_once():
    """Two batches on two streams, each with its own tables and workspace: the tables
    of the same calls one after the other."""
    rng = np.random.default_rng(19)
    runs = [Router(logits_of(rng, 5000, 128), True), Router(logits_of(rng, 300, 64), False)]
    want = [r.check(k, True)[0] for r, k in zip(runs, (8, 4))]
    streams = [torch.cuda.Stream() for _ in runs]
    for r, k in zip(runs, (8, 4)):
        r.buffers(k)
    torch.cuda.synchronize()
    for _ in range(5):
        for r, s in zip(runs, streams):
            with torch.cuda.stream(s):
                R.check(r.launch(True), "rld_moe_router")
    for r, w in zip(runs, want):
        for key, got in r.results().items():
            assert np.array_equal(got, w[key]), key


@pytest.mark.parametrize("T", [64, 65, 128, 1025, 8192, 8193, 16385])
def test_batches_around_the_blocks_of_tokens(T):
    """Where the blocks become larger, or one more: the tables are those of the
    plain form, of a masked batch too."""
    rng = np.random.default_rng(T)
    mask = (rng.random(T) < 0.9).astype(np.int32)
    Router(logits_of(rng, T, 16), False, mask).check(2, False)


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "fp32"])
def test_lowest_values_and_large_ones(f32):
    """Masks of the type's lowest value are finite: such experts come last, with
    probability zero beside others and an even one among themselves."""
    rng = np.random.default_rng(3)
    l = logits_of(rng, 20, 40, odd=False)
    l[::2, 5:] = LOWEST[f32]
    l[1] = LOWEST[f32]
    l[3] = -LOWEST[f32]
    l[5, ::2] = -LOWEST[f32]
    r = Router(l, f32)
    for norm in (False, True):
        r.check_grad(8, norm)


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "fp32"])
def test_nan_and_inf_rows(f32):
    rng = np.random.default_rng(4)
    l = logits_of(rng, 70, 33)
    l[10, 3] = np.nan
    l[20] = np.nan
    l[30, 0] = INF
    l[40, :5] = INF
    l[41, 7] = np.nan
    mask = np.ones(70, np.int32)
    mask[41] = 0  # a masked token's NaN is not read into anything
    r = Router(l, f32, mask)
    r.check_grad(4, True)
    l[[10, 20, 30, 40]] = 0
    got, _ = Router(l, f32, mask).check(4, True)
    assert np.isfinite(got["loss"])


def test_nothing_routes():
    rng = np.random.default_rng(5)
    l = logits_of(rng, 100, 16)
    for r in (Router(l, True, np.zeros(100, np.int32)), Router(np.full((9, 16), -INF), False)):
        d = r.check_grad(4, False)
        assert (d == 0).all()


def test_no_tokens():
    r = Router(np.zeros((1, 16), np.float32), True)
    r.buffers(2)
    r.T = 0
    R.check(r.launch(True), "rld_moe_router")
    torch.cuda.synchronize()
    assert (r.cnt[:17] == 0).all() and (r.off[:17] == 0).all() and float(r.loss[0]) == 0
    assert int(r.idx[0]) == 77 and int(r.stok[0]) == 77


def test_tables_not_wanted():
    rng = np.random.default_rng(6)
    r = Router(logits_of(rng, 150, 64), False)
    got, _ = r.check(6, True)
    r.buffers(6)
    R.check(r.launch(True, tables=False), "rld_moe_router")
    torch.cuda.synchronize()
    assert np.array_equal(r.idx[:-1].cpu().numpy().reshape(150, 6), got["idx"])
    assert np.array_equal(r.w[:-1].cpu().numpy().reshape(150, 6), got["w"])
    assert (r.cnt == 77).all() and (r.stok == 77).all() and (r.loss == 77).all()


@pytest.mark.parametrize("with_w,with_loss", [(True, False), (False, True)])
@pytest.mark.parametrize("norm", [False, True])
def test_gradient_of_one_output(with_w, with_loss, norm):
    rng = np.random.default_rng(7)
    Router(logits_of(rng, 90, 128), True, pad=5).check_grad(8, norm, with_w, with_loss)


def test_gradient_in_place():
    rng = np.random.default_rng(8)
    l = logits_of(rng, 90, 60)
    a = Router(l, True, pad=4).check_grad(8, True)
    b = Router(l, True, pad=4).check_grad(8, True, in_place=True)
    assert np.array_equal(a, b)


def test_indices_out_of_range_are_not_read():
    """Chosen experts below 0 or past the last: no gradient through them."""
    rng = np.random.default_rng(9)
    r = Router(logits_of(rng, 40, 12, odd=False), True)
    got, want = r.check(3, False)
    wild, cut = got["idx"].copy(), want["idx"].copy()
    wild[::3, 1] = 12
    wild[1::3, 0] = 2 ** 31 - 1
    wild[2::3, 2] = -2 ** 31
    cut[(wild < 0) | (wild >= 12)] = -1
    dw = rng.standard_normal((40, 3)).astype(np.float32)
    d = r.grad(dict(got, idx=wild), False, torch.from_numpy(dw).to(r.dev), None)
    ref, mag = gradient(r.l, dict(want, idx=cut), dw, 0.0, 3, False)
    assert (np.abs(d - ref) <= (rel_p(r.l) * 7 + 24 * U) * mag + TINY).all()


@pytest.mark.parametrize("norm", [False, True])
def test_gradient_against_differences(norm):
    """Central differences in 64 bits of <dw, weights> + dloss * loss with the
    choice held: steps h, error h^2 of third derivatives (below 1 here) plus
    64-bit rounding over 2h."""
    rng = np.random.default_rng(10)
    T, E, k, h = 6, 9, 3, 1e-4
    r = Router(logits_of(rng, T, E, odd=False), True)
    got, want = r.check(k, norm)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    d = r.grad(got, norm, torch.from_numpy(dw).to(r.dev), torch.tensor([1.5], device=r.dev))

    def value(l):
        e = np.exp(l - l.max(1, keepdims=True))
        p = e / e.sum(1, keepdims=True)
        w = np.take_along_axis(p, want["idx"], 1)
        if norm:
            w = w / w.sum(1, keepdims=True)
        c = want["counts"][:E]
        return (dw * w).sum() + 1.5 * E / (k * T * T) * (c * p.sum(0)).sum()

    _, mag = gradient(r.l, want, dw, 1.5, k, norm)
    for t in range(T):
        for e in range(E):
            a, b = r.l.copy(), r.l.copy()
            a[t, e] += h
            b[t, e] -= h
            diff = (value(a) - value(b)) / (2 * h)
            assert abs(d[t, e] - diff) <= 16 * h * h + 1e-9 + 200 * U * mag[t, e]


def test_same_bits_every_run_and_graph_replays():
    """One captured graph of router and gradient, replayed with new logits and
    masks, eager work between the replays: the eager calls' bits each time."""
    say("case: router graph")
    rng = np.random.default_rng(11)
    T, E, k = 300, 128, 8
    dev = require_gpu()
    r = Router(logits_of(rng, T, E), False, np.ones(T, np.int32))
    r.buffers(k)
    dw = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).to(dev)
    dl = torch.ones(1, device=dev)
    out = torch.zeros((T, E), dtype=torch.int16, device=dev)

    def both(stream=None):
        R.check(r.launch(True, stream), "rld_moe_router")
        R.check(R.rld_moe_router_grad(r.ld, False, r.ls, r.md, T, E, k, True, r.idx, r.cnt, dw,
                                      dl, out, E, stream), "rld_moe_router_grad")

    both()
    torch.cuda.synchronize()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        both(s)
    for _ in range(4):
        r.ld.copy_(torch.from_numpy(to_bits(logits_of(rng, T, E)).view(np.int16)))
        r.md.copy_(torch.from_numpy((rng.random(T) < 0.7).astype(np.int32)))
        bufs = (r.idx, r.w, r.cnt, r.off, r.stok, r.srows, r.loss, out)
        g.replay()
        torch.cuda.synchronize()
        replayed = [b.clone() for b in bufs]
        for _ in range(2):
            for b in bufs[:-1]:
                b[:-1] = 5
            both()
            torch.cuda.synchronize()
            for a, b in zip(replayed, bufs):
                assert torch.equal(a, b)


@pytest.mark.parametrize("x", [0.5, 0.75, 1.25])
def test_loss_of_very_many_tokens(x):
    """2^22 equal tokens, one expert preferred by x: loss = E p.  An fp32 sum over the
    32768 blocks of tokens would drift by 70 to 100 units (each addition rounds the
    same way).  Bound: a probability's error, the at most 2 + 3 + 8 additions inside a
    block and the roundings of the sum and the loss."""
    say(f"case: router loss of very many tokens {x}")
    dev = require_gpu()
    T, E = 1 << 22, 8
    row = np.zeros((1, E), np.float32)
    row[0, 3] = x
    logits = torch.from_numpy(row).to(dev).repeat(T, 1)
    idx = torch.zeros((T, 1), dtype=torch.int32, device=dev)
    w, loss = torch.zeros((T, 1), device=dev), torch.zeros(1, device=dev)
    cnt = torch.zeros(E + 1, dtype=torch.int32, device=dev)
    need = R.rld_moe_router_workspace_bytes(T, E, 1)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=dev)
    R.check(R.rld_moe_router(logits, True, E, None, T, E, 1, False, idx, w, cnt, None, None, None,
                             loss, ws, need), "rld_moe_router")
    torch.cuda.synchronize()
    want = np.zeros(E + 1, np.int64)
    want[3] = want[E] = T
    assert np.array_equal(cnt.cpu().numpy(), want) and bool((idx == 3).all())
    p = np.exp(x) / (np.exp(x) + E - 1)
    tol = rel_p(row.astype(np.float64))[0, 0] + 15 * U
    assert abs(float(loss[0]) / (E * p) - 1) <= tol


# ------------------------------------------------------ used together ----

def test_router_tables_drive_the_grouped_fold():
    """The workload's logits through the router: its tables are the workload's own
    (host-made) ones, and the grouped fold of a window run on them has the same
    bits.  The sort order inside an expert is (token, position)."""
    say("case: router -> grouped fold")
    dev = require_gpu()
    m = W.moe_grouped(num_tokens=200, top_k=4, num_experts=16, hidden=256, inter=128, max_loras=3,
                      n_adapted=12, ranks=(8, 16), max_rank=16, cap=300, projections=("down",))
    rng = W.rng_for(4)
    l = rng.standard_normal((200, 16), dtype=np.float32)  # the workload's first draw
    r = Router(l, True)
    got, _ = r.check(4, True)
    assert np.array_equal(got["off"], m.expert_offsets)
    assert np.array_equal(got["stok"], m.sorted_token_ids)
    assert np.array_equal(got["srows"] % 4, m.sorted_topk_pos)
    p = m.projections[0]
    want = GroupedRun(m, p, dev)
    want.run()
    own = GroupedRun(m, p, dev)
    own.off, own.stid = r.off, r.stok
    own.run()
    assert np.array_equal(want.base.body(), own.base.body())
    assert not np.array_equal(own.base.body(), p.base.ravel())


def test_training_step_through_router_and_projection():
    """Logits by rld_proj (a router gate with adapters), routing and loss, and back
    through both gradients, in one captured graph: the logits' gradient against the
    definition, the adapters' and inputs' gradients against the formulas on the
    BF16 dlogits that the router handed over."""
    say("case: projection -> router -> gradients")
    dev = require_gpu()
    rng = np.random.default_rng(12)
    n, k_in, E, rank, slots, k = 130, 264, 64, 16, 3, 4
    adapters = [W.make_adapter(rng, s, rank, k_in, E, 16.0, False) for s in range(slots)]
    route = DenseRoute(adapters, slots, rank, k_in, E, dev)
    bits = lambda a: to_bits(a).view(np.int16)  # noqa: E731
    x = torch.from_numpy(bits(rng.standard_normal((n, k_in)))).to(dev)
    w = torch.from_numpy(bits(rng.standard_normal((E, k_in)) * 0.1)).to(dev)
    slot_h = rng.integers(-1, slots, n).astype(np.int32)
    slot = torch.from_numpy(slot_h).to(dev)
    logits = torch.zeros((n, E), dtype=torch.int16, device=dev)
    dlogits, dx = torch.zeros_like(logits), torch.zeros_like(x)
    da, db = (torch.zeros((slots, *s), device=dev) for s in ((rank, k_in), (E, rank)))
    at = torch.arange(slots, device=dev)
    dat, dbt = da.data_ptr() + at * (rank * k_in * 4), db.data_ptr() + at * (E * rank * 4)
    i32 = dict(dtype=torch.int32, device=dev)
    idx, cnt = torch.zeros((n, k), **i32), torch.zeros(E + 1, **i32)
    wts, loss = torch.zeros((n, k), device=dev), torch.zeros(1, device=dev)
    dw_h = rng.standard_normal((n, k)).astype(np.float32)
    dw, dl = torch.from_numpy(dw_h).to(dev), torch.full((1,), 2.0, device=dev)
    wb = max(R.rld_proj_workspace_bytes(n, k_in, E, rank, slots),
             R.rld_proj_grad_workspace_bytes(n, k_in, E, rank, slots),
             R.rld_moe_router_workspace_bytes(n, E, k))
    ws = torch.full((wb,), 0xFF, dtype=torch.uint8, device=dev)

    def step(st=None):
        R.check(R.rld_proj(route.route, w, k_in, x, k_in, slot, n, logits, E, ws, wb, st), "proj")
        R.check(R.rld_moe_router(logits, False, E, None, n, E, k, True, idx, wts, cnt, None, None,
                                 None, loss, ws, wb, st), "router")
        R.check(R.rld_moe_router_grad(logits, False, E, None, n, E, k, True, idx, cnt, dw, dl,
                                      dlogits, E, st), "router_grad")
        R.check(R.rld_proj_grad(route.route, w, k_in, x, k_in, dlogits, E, slot, n, dx, k_in, dat,
                                dbt, 0, ws, wb, st), "proj_grad")

    step()
    torch.cuda.synchronize()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step(s)
    val = lambda t: (t.cpu().numpy().view(np.uint16).astype(np.uint32) << 16).view(  # noqa: E731
        np.float32).astype(np.float64)
    eager = [t.clone() for t in (logits, idx, cnt, wts, loss, dlogits, dx, da, db)]
    for _ in range(3):
        for t in (logits, idx, cnt, wts, loss, dlogits, dx, da, db):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, (logits, idx, cnt, wts, loss, dlogits, dx, da, db)):
            assert torch.equal(a, b)
    want = reference(val(logits), None, k, True)
    assert np.array_equal(idx.cpu().numpy(), want["idx"])
    ref, mag = gradient(val(logits), want, dw_h, 2.0, k, True)
    err = (rel_p(val(logits)) * (4 + k) + (E + 12) * U) * mag
    got = val(dlogits)
    assert (np.abs(got - ref) <= err + 2.0 ** -8 * (np.abs(ref) + err)).all()
    for sl, ad in enumerate(adapters):
        rows = np.nonzero(slot_h == sl)[0]
        A = (ad.A.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
        B = (ad.B.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
        c = float(O.scale_for(16.0, rank, False))
        gl, u = c * got[rows] @ B, c * val(x)[rows] @ A.T
        gm, um = c * np.abs(got[rows]) @ np.abs(B), c * np.abs(val(x)[rows]) @ np.abs(A).T
        # both products' additions: 32 + 264/32 + 8 and 32 + 3 * 130 + 8, below 600
        for have, exact, m in ((da[sl], gl.T @ val(x)[rows], gm.T @ np.abs(val(x)[rows])),
                               (db[sl], got[rows].T @ u, np.abs(got[rows]).T @ um)):
            assert (np.abs(have.cpu().numpy() - exact) <= 600 * 2.0 ** -23 * m + 1e-30).all()
