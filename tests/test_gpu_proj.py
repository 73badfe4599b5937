"""GPU tests of rld_proj and rld_proj_grad against the formulas in 64 bits.

Bounds, derived (u = 2^-23: the matrix cores' inner additions are not specified
to round to nearest, and an addition that truncates is off by up to one unit):
  a product of depth D (fp32 additions on an element's longest chain) is off by
  at most gamma = D u / (1 - D u) times the sum of its terms' magnitudes;
  a low row enters a BF16 output as two BF16 parts (2^-8 relative each, so
  2^-16 of the value is left out) and an fp32 output as three (2^-24);
  a BF16 output is rounded once, by at most 2^-8 of what was rounded.
Depth: 32 for the terms of one matrix instruction, one addition per further
instruction, four waves' sums, the chunks' sums and the scale.
"""
import numpy as np
import pytest
import torch

import routed_lora_delta_amd as R
from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
NAN16 = 0x7FC1  # a quiet NaN: what must not be read, or not be written over


def gamma(d):
    return d * U / (1 - d * U)


def bf16_values(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def rand_bits(rng, shape, std):
    v = (rng.standard_normal(shape) * std).astype(np.float32)
    return (v.view(np.uint32) >> 16).astype(np.uint16)


def up(bits, dev):
    return torch.from_numpy(bits.view(np.int16)).to(dev)


class Case:
    """One projection: operands with NaN in every gap that a kernel must skip."""

    def __init__(self, n, k, m, r, slots, layout="mixed", xpad=0, wpad=0, opad=0, seed=0,
                 adapted=None):
        self.dev = require_gpu()
        self.n, self.k, self.m, self.r, self.slots = n, k, m, r, slots
        self.xs, self.ws, self.os = k + xpad, k + wpad, m + opad
        rng = np.random.default_rng(1000 + seed)
        self.rng = rng
        self.x = np.full((n, self.xs), NAN16, np.uint16)
        self.x[:, :k] = rand_bits(rng, (n, k), 1.0)
        self.w = np.full((m, self.ws), NAN16, np.uint16)
        self.w[:, :k] = rand_bits(rng, (m, k), k ** -0.5)
        self.dy = np.full((n, self.os), NAN16, np.uint16)
        self.dy[:, :m] = rand_bits(rng, (n, m), 1.0)
        # each slot's A and B with a NaN row behind it
        self.a = np.full((slots, r + 1, k), NAN16, np.uint16)
        self.a[:, :r] = rand_bits(rng, (slots, r, k), k ** -0.5)
        self.b = np.full((slots, m + 1, r), NAN16, np.uint16)
        self.b[:, :m] = rand_bits(rng, (slots, m, r), 0.3)
        self.scale = (rng.random(slots) + 0.5).astype(np.float32)
        self.adapted = np.ones(slots, bool) if adapted is None else np.asarray(adapted)
        if layout == "mixed":
            slot = rng.integers(-1, slots, size=n)
        elif layout == "runs":
            slot = np.sort(rng.integers(-1, slots, size=n))[::-1].copy()
        elif layout == "base":
            slot = np.full(n, -1)
        elif layout == "wild":  # ids that name no slot
            slot = rng.choice([-2**31, -7, -1, 0, slots - 1, slots, slots + 9, 2**31 - 1], size=n)
        self.slot = slot.astype(np.int32)
        d = self.dev
        self.xd, self.wd, self.dyd = up(self.x, d), up(self.w, d), up(self.dy, d)
        self.ad, self.bd = up(self.a, d), up(self.b, d)
        self.sd = torch.from_numpy(self.scale).to(d)
        self.slotd = torch.from_numpy(self.slot).to(d)
        on = torch.from_numpy(self.adapted).to(d)
        at = torch.arange(slots, device=d)
        self.at = torch.where(on, self.ad.data_ptr() + at * ((r + 1) * k * 2), 0)
        self.bt = torch.where(on, self.bd.data_ptr() + at * ((m + 1) * r * 2), 0)
        self.route = R.rld_route(self.at.data_ptr(), self.bt.data_ptr(), self.sd.data_ptr(),
                                 slots, k, m, r)

    def scratch(self, nbytes):
        # 0xFF bytes: NaN wherever a kernel read what it did not write; a guard behind
        t = torch.full((nbytes + 256,), 0xFF, dtype=torch.uint8, device=self.dev)
        return t

    def rows_of(self, s):
        return np.nonzero((self.slot == s) & self.adapted[s])[0]

    # ---- the formulas in 64 bits, with the sums of the terms' magnitudes ----
    def forward(self):
        x, w = bf16_values(self.x[:, :self.k]), bf16_values(self.w[:, :self.k])
        y, mag = x @ w.T, np.abs(x) @ np.abs(w).T
        low = np.zeros_like(y)
        for s in range(self.slots):
            i = self.rows_of(s)
            a, b = bf16_values(self.a[s, :self.r]), bf16_values(self.b[s, :self.m])
            c = float(self.scale[s])
            y[i] += c * (x[i] @ a.T) @ b.T
            low[i] = c * (np.abs(x[i]) @ np.abs(a).T) @ np.abs(b).T
        return y, mag, low

    def gradients(self):
        x, w = bf16_values(self.x[:, :self.k]), bf16_values(self.w[:, :self.k])
        dy = bf16_values(self.dy[:, :self.m])
        dx, mag = dy @ w, np.abs(dy) @ np.abs(w)
        low = np.zeros_like(dx)
        da, db = np.zeros((self.slots, self.r, self.k)), np.zeros((self.slots, self.m, self.r))
        mda, mdb = np.zeros_like(da), np.zeros_like(db)
        for s in range(self.slots):
            i = self.rows_of(s)
            a, b = bf16_values(self.a[s, :self.r]), bf16_values(self.b[s, :self.m])
            c = float(self.scale[s])
            g, gm = c * dy[i] @ b, c * np.abs(dy[i]) @ np.abs(b)
            u, um = c * x[i] @ a.T, c * np.abs(x[i]) @ np.abs(a).T
            dx[i] += g @ a
            low[i] = gm @ np.abs(a)
            da[s], mda[s] = g.T @ x[i], gm.T @ np.abs(x[i])
            db[s], mdb[s] = dy[i].T @ u, np.abs(dy[i]).T @ um
        return (dx, mag, low), (da, mda), (db, mdb)

    def depth(self, k):
        return 32 + -(-k // 32) + 4 + 24 * -(-k // 12288) + 2

    def check_rounded(self, got, want, mag, low, k, label):
        """got: BF16 values of a product of depth k plus the low part."""
        d = self.depth(k) + 2 * -(-self.r // 32) * 64
        err = gamma(d) * (mag + low) + (gamma(self.depth(k) + 32 + self.r) + 2.0 ** -16) * low
        tol = err + 2.0 ** -8 * (np.abs(want) + err)
        off = np.abs(got - want)
        bad = ~(off <= tol)
        assert not bad.any(), (f"{label}: {bad.sum()} of {bad.size} beyond the bound, first at "
                               f"{np.argwhere(bad)[0]}: got {got[bad][0]}, want {want[bad][0]}, "
                               f"bound {tol[bad][0]}")

    def check_grad(self, got, want, mag, k, rows, label):
        err = (gamma(self.depth(k)) + gamma(32 + 3 * rows + 8) + 2.0 ** -23) * mag
        bad = ~(np.abs(got - want) <= err + 2.0 ** -24 * np.abs(want))
        assert not bad.any(), (f"{label}: {bad.sum()} of {bad.size} beyond the bound, first at "
                               f"{np.argwhere(bad)[0]}: got {got[bad][0]}, want {want[bad][0]}")

    # ---- calls ----
    def out_rows(self, stride):
        return torch.full((self.n + 2, stride), NAN16, dtype=torch.int16, device=self.dev)

    def body(self, t, width, stride):
        """The written part; everything around it must be as it was."""
        h = t.cpu().numpy().view(np.uint16)
        assert (h[0] == NAN16).all() and (h[-1] == NAN16).all(), "a row outside was written"
        assert (h[1:-1, width:] == NAN16).all(), "the rest of a row was written"
        return h[1:-1, :width]

    def call_proj(self, out, ws, stream=None):
        need = R.rld_proj_workspace_bytes(self.n, self.k, self.m, self.r, self.slots)
        return R.rld_proj(self.route, self.wd, self.ws, self.xd, self.xs, self.slotd, self.n,
                          out.data_ptr() + 2 * self.os, self.os, ws, need, stream)

    def proj(self):
        need = R.rld_proj_workspace_bytes(self.n, self.k, self.m, self.r, self.slots)
        ws, out = self.scratch(need), self.out_rows(self.os)
        R.check(self.call_proj(out, ws), "rld_proj")
        torch.cuda.synchronize()
        assert bool((ws[need:] == 0xFF).all()), "the workspace was overrun"
        return self.body(out, self.m, self.os)

    def tables(self):
        s, r, k, m = self.slots, self.r, self.k, self.m
        self.dad = torch.full((s, r + 1, k), float("nan"), device=self.dev)
        self.dbd = torch.full((s, m + 1, r), float("nan"), device=self.dev)
        at = torch.arange(s, device=self.dev)
        self.dat = self.dad.data_ptr() + at * ((r + 1) * k * 4)
        self.dbt = self.dbd.data_ptr() + at * ((m + 1) * r * 4)

    def call_grad(self, dx, ws, accumulate=0, da=True, db=True, stream=None):
        need = R.rld_proj_grad_workspace_bytes(self.n, self.k, self.m, self.r, self.slots)
        return R.rld_proj_grad(self.route, self.wd, self.ws, self.xd, self.xs, self.dyd, self.os,
                               self.slotd, self.n,
                               None if dx is None else dx.data_ptr() + 2 * self.xs, self.xs,
                               self.dat if da else None, self.dbt if db else None, accumulate,
                               ws, need, stream)

    def grad(self):
        need = R.rld_proj_grad_workspace_bytes(self.n, self.k, self.m, self.r, self.slots)
        ws, dx = self.scratch(need), self.out_rows(self.xs)
        self.tables()
        R.check(self.call_grad(dx, ws), "rld_proj_grad")
        torch.cuda.synchronize()
        assert bool((ws[need:] == 0xFF).all()), "the workspace was overrun"
        return self.body(dx, self.k, self.xs), *self.slot_gradients()

    def slot_gradients(self):
        da, db = self.dad.cpu().numpy(), self.dbd.cpu().numpy()
        assert np.isnan(da[:, self.r]).all() and np.isnan(db[:, self.m]).all(), \
            "behind a slot's gradient was written"
        return da[:, :self.r].astype(np.float64), db[:, :self.m].astype(np.float64)

    def check_proj(self, got=None):
        got = self.proj() if got is None else got
        self.check_rounded(bf16_values(got), *self.forward(), self.k, "out")

    def check_grads(self):
        dx, da, db = self.grad()
        rx, ra, rb = self.gradients()
        self.check_rounded(bf16_values(dx), *rx, self.m, "dx")
        rows = max([len(self.rows_of(s)) for s in range(self.slots)] + [1])
        self.check_grad(da, *ra, self.m, rows, "dA")
        self.check_grad(db, *rb, self.k, rows, "dB")


SHAPES = [
    # n, k_in, n_out, rank, slots, layout, x pad, w pad, out pad
    (1, 8, 8, 8, 1, "mixed", 0, 0, 0),
    (1, 4096, 1024, 16, 16, "mixed", 0, 0, 0),
    (2, 64, 40, 16, 3, "mixed", 8, 8, 8),
    (5, 72, 264, 24, 2, "wild", 0, 16, 24),
    (16, 520, 136, 8, 40, "mixed", 8, 0, 0),
    (17, 2048, 768, 16, 4, "runs", 0, 0, 8),
    (63, 768, 2048, 128, 5, "mixed", 0, 8, 0),
    (64, 1032, 72, 40, 3, "runs", 16, 0, 16),
    (65, 200, 200, 64, 64, "mixed", 0, 0, 0),
    (100, 56, 1000, 16, 7, "base", 0, 0, 0),
    (129, 640, 328, 32, 2, "mixed", 0, 24, 8),
    (200, 1096, 520, 104, 9, "wild", 8, 8, 8),
    (257, 136, 4104, 16, 16, "runs", 0, 0, 0),
    (300, 4096, 264, 64, 32, "mixed", 0, 0, 64),
    (515, 312, 760, 128, 3, "runs", 8, 8, 0),
    (1030, 264, 136, 8, 200, "mixed", 0, 0, 0),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s[:6])))
def test_proj(shape):
    say(f"case: proj {shape}")
    Case(*shape, seed=SHAPES.index(shape)).check_proj()


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s[:6])))
def test_proj_grad(shape):
    say(f"case: proj_grad {shape}")
    Case(*shape, seed=SHAPES.index(shape)).check_grads()


@pytest.mark.parametrize("n,k,m,r", [(600, 4096, 1032, 16), (1237, 1024, 2056, 64)])
def test_proj_large(n, k, m, r):
    """Past every tile's edge, in both directions."""
    say(f"case: proj large {n} {k} {m} {r}")
    c = Case(n, k, m, r, 6, "runs", seed=77)
    c.check_proj()
    c.check_grads()


@pytest.mark.parametrize("n,k,m,r,slots,layout", [
    (2500, 200, 4360, 16, 3, "runs"),     # K of three steps and an eighth
    (2100, 72, 4872, 40, 40, "mixed"),    # one step and a tail, many slots a tile
    (2600, 328, 4104, 128, 2, "wild"),
    (4100, 64, 2568, 8, 5, "runs"),
])
def test_proj_many_tiles(n, k, m, r, slots, layout):
    """Grids of 256 x 256 tiles, forward and (k and m exchanged) backward."""
    say(f"case: proj many tiles {n} {k} {m} {r} {layout}")
    Case(n, k, m, r, slots, layout, 8, 16, 8, seed=21).check_proj()
    Case(n, m, k, r, slots, layout, 8, 16, 8, seed=22).check_grads()


def test_many_tiles_rows_apart():
    """A slot's NaN and infinities stay with its rows where a wave's tile holds
    rows of several slots."""
    say("case: proj many tiles, rows apart")
    c = Case(2304, 136, 4608, 16, 4, seed=23)
    out = c.proj()
    c.bd[1] = 0x7F80
    c.ad[1, 0] = NAN16
    out2 = c.proj()
    keep = c.slot != 1
    assert np.array_equal(out[keep], out2[keep]) and not np.array_equal(out, out2)


def test_unadapted_slots_are_base_rows():
    c = Case(70, 136, 200, 16, 4, adapted=[True, False, True, False], seed=3)
    c.check_proj()
    c.check_grads()
    assert (c.slot_gradients()[0][1] == 0).all() and (c.slot_gradients()[1][3] == 0).all()


def test_rows_do_not_reach_each_other():
    """Infinities and NaN in one row, in the adapters of one slot: the other rows'
    and slots' results keep their bits."""
    say("case: proj rows apart")
    c = Case(90, 328, 264, 24, 5, seed=4)
    out, (dx, da, db) = c.proj(), c.grad()
    victim = 2
    rows = np.nonzero(c.slot == victim)[0]
    assert 0 < len(rows) < 90
    c.ad[victim, 3, 7] = NAN16
    c.bd[victim, 1, 2] = NAN16
    c.xd[torch.from_numpy(rows).to(c.dev), 11] = 0x7F80
    c.dyd[torch.from_numpy(rows).to(c.dev), 5] = 0x7F80
    out2, (dx2, da2, db2) = c.proj(), c.grad()
    keep = np.nonzero(c.slot != victim)[0]
    other = [s for s in range(5) if s != victim]
    assert np.array_equal(out[keep], out2[keep]) and np.array_equal(dx[keep], dx2[keep])
    assert np.array_equal(da[other], da2[other]) and np.array_equal(db[other], db2[other])
    assert not np.isfinite(bf16_values(out2[rows])).all(1).any()


def test_same_bits_every_run():
    c = Case(333, 1096, 520, 40, 6, seed=5)
    out, g = c.proj(), c.grad()
    for _ in range(3):
        assert np.array_equal(out, c.proj())
        for a, b in zip(g, c.grad()):
            assert np.array_equal(a, b)


def test_grad_parts_not_wanted():
    """Every subset of dx, dA, dB, and single slots left out: the wanted parts keep
    their bits, the others stay as they were."""
    c = Case(140, 264, 136, 16, 3, seed=6)
    dx0, da0, db0 = c.grad()
    need = R.rld_proj_grad_workspace_bytes(c.n, c.k, c.m, c.r, c.slots)
    for want_dx in (True, False):
        for want_da in (True, False):
            for want_db in (True, False):
                if not (want_dx or want_da or want_db):
                    continue
                c.tables()
                dx = c.out_rows(c.xs)
                R.check(c.call_grad(dx if want_dx else None, c.scratch(need), 0, want_da, want_db),
                        "rld_proj_grad")
                torch.cuda.synchronize()
                h = dx.cpu().numpy().view(np.uint16)
                if want_dx:
                    assert np.array_equal(c.body(dx, c.k, c.xs), dx0)
                else:
                    assert (h == NAN16).all()
                da, db = c.slot_gradients()
                assert np.array_equal(da, da0) if want_da else np.isnan(da).all()
                assert np.array_equal(db, db0) if want_db else np.isnan(db).all()
    c.tables()
    c.dat[1] = 0
    c.dbt[2] = 0
    R.check(c.call_grad(None, c.scratch(need)), "rld_proj_grad")
    torch.cuda.synchronize()
    da, db = c.slot_gradients()
    assert np.isnan(da[1]).all() and np.isnan(db[2]).all()
    assert np.array_equal(da[[0, 2]], da0[[0, 2]]) and np.array_equal(db[:2], db0[:2])


def test_grad_accumulates():
    """accumulate: one fp32 addition to what was there, exactly."""
    c = Case(75, 200, 72, 24, 3, seed=7)
    _, da0, db0 = c.grad()
    need = R.rld_proj_grad_workspace_bytes(c.n, c.k, c.m, c.r, c.slots)
    c.tables()
    start_a = c.rng.standard_normal((c.slots, c.r, c.k)).astype(np.float32)
    start_b = c.rng.standard_normal((c.slots, c.m, c.r)).astype(np.float32)
    c.dad[:, :c.r] = torch.from_numpy(start_a).to(c.dev)
    c.dbd[:, :c.m] = torch.from_numpy(start_b).to(c.dev)
    R.check(c.call_grad(None, c.scratch(need), accumulate=1), "rld_proj_grad")
    torch.cuda.synchronize()
    da, db = c.slot_gradients()
    assert np.array_equal(da, (start_a + da0.astype(np.float32)).astype(np.float64))
    assert np.array_equal(db, (start_b + db0.astype(np.float32)).astype(np.float64))


@pytest.mark.parametrize("n,k,m,r,slots,adapted", [
    (1300, 264, 136, 16, 1, None),
    (2100, 136, 520, 64, 2, [False, True]),   # one slot left out, rows of no slot between
    (1100, 72, 40, 128, 1, None),
])
def test_grad_of_few_slots(n, k, m, r, slots, adapted):
    """Many rows a slot, so that their sums are made in pieces: the values, and the
    one addition where they accumulate; the same bits in both."""
    say(f"case: proj_grad few slots {n} {k} {m} {r}")
    c = Case(n, k, m, r, slots, "mixed", 8, 0, 8, seed=31, adapted=adapted)
    c.check_grads()
    _, da0, db0 = c.grad()
    need = R.rld_proj_grad_workspace_bytes(c.n, c.k, c.m, c.r, c.slots)
    c.tables()
    start_a = c.rng.standard_normal((c.slots, c.r, c.k)).astype(np.float32)
    start_b = c.rng.standard_normal((c.slots, c.m, c.r)).astype(np.float32)
    c.dad[:, :c.r] = torch.from_numpy(start_a).to(c.dev)
    c.dbd[:, :c.m] = torch.from_numpy(start_b).to(c.dev)
    scratch = c.scratch(need)
    R.check(c.call_grad(None, scratch, accumulate=1), "rld_proj_grad")
    torch.cuda.synchronize()
    assert (scratch[need:] == 0xFF).all()
    da, db = c.slot_gradients()
    assert np.array_equal(da, (start_a + da0.astype(np.float32)).astype(np.float64))
    assert np.array_equal(db, (start_b + db0.astype(np.float32)).astype(np.float64))


@pytest.mark.parametrize("accumulate", [0, 1])
def test_grad_of_no_rows(accumulate):
    c = Case(1, 72, 40, 8, 3, seed=8)
    c.n = 0
    c.tables()
    c.dad[:, :c.r] = 3.0
    c.dbd[:, :c.m] = 3.0
    need = R.rld_proj_grad_workspace_bytes(0, c.k, c.m, c.r, c.slots)
    R.check(R.rld_proj_grad(c.route, None, 0, None, 0, None, 0, None, 0, None, 0, c.dat, c.dbt,
                            accumulate, c.scratch(need), need), "rld_proj_grad")
    torch.cuda.synchronize()
    da, db = c.slot_gradients()
    want = 3.0 if accumulate else 0.0
    assert (da == want).all() and (db == want).all()


def test_gradients_against_differences():
    """<dA, D> and the like against central differences of sum(dy * y) in 64 bits
    (the formula is linear in each argument, so the differences are exact up to
    64-bit rounding; the bound is the gradients' own)."""
    c = Case(50, 136, 72, 16, 3, seed=9)
    dx, da, db = c.grad()
    (rx, mx, lx), (ra, ma), (rb, mb) = c.gradients()
    x = bf16_values(c.x[:, :c.k])
    w = bf16_values(c.w[:, :c.k])
    a, b = bf16_values(c.a[:, :c.r]), bf16_values(c.b[:, :c.m])
    dy = bf16_values(c.dy[:, :c.m])

    def total(x, a, b):
        y = x @ w.T
        for s in range(c.slots):
            i = c.rows_of(s)
            y[i] += float(c.scale[s]) * (x[i] @ a[s].T) @ b[s].T
        return (dy * y).sum()

    rng = np.random.default_rng(10)
    rows = max(len(c.rows_of(s)) for s in range(c.slots))
    h = 0.5
    for name, got, mag, move in (
            ("x", bf16_values(dx), mx + lx, lambda d: (total(x + h * d, a, b),
                                                       total(x - h * d, a, b))),
            ("A", da, ma, lambda d: (total(x, a + h * d, b), total(x, a - h * d, b))),
            ("B", db, mb, lambda d: (total(x, a, b + h * d), total(x, a, b - h * d)))):
        d = rng.standard_normal(got.shape)
        hi, lo = move(d)
        tol = ((gamma(600 + 3 * rows) + 2.0 ** -16) * mag * np.abs(d)).sum() + 1e-9 * abs(hi - lo)
        if name == "x":
            tol += (2.0 ** -8 * np.abs(got) * np.abs(d)).sum()
        assert abs((got * d).sum() - (hi - lo) / (2 * h)) <= tol, name


def test_graph_replays_with_new_routing():
    """Two captured graphs (projection; gradient) sharing one workspace, replayed in
    turn with new routing, with eager calls and host waits between the replays."""
    say("case: proj graphs")
    c = Case(96, 520, 264, 16, 6, seed=11)
    need = max(R.rld_proj_workspace_bytes(c.n, c.k, c.m, c.r, c.slots),
               R.rld_proj_grad_workspace_bytes(c.n, c.k, c.m, c.r, c.slots))
    ws, out, dx = c.scratch(need), c.out_rows(c.os), c.out_rows(c.xs)
    c.tables()
    R.check(c.call_proj(out, ws), "eager")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1, stream=s):
        R.check(c.call_proj(out, ws, s), "captured rld_proj")
    with torch.cuda.graph(g2, stream=s):
        R.check(c.call_grad(dx, ws, stream=s), "captured rld_proj_grad")
    rng = np.random.default_rng(12)
    dat, dbt, dad, dbd = c.dat, c.dbt, c.dad, c.dbd
    for _ in range(4):
        c.slot = rng.integers(-1, 6, size=c.n).astype(np.int32)
        c.slotd.copy_(torch.from_numpy(c.slot))
        dad[:, :c.r] = 9.0
        out[1:-1, :c.m] = NAN16
        g1.replay()
        g2.replay()
        g1.replay()
        torch.cuda.synchronize()
        got = c.body(out, c.m, c.os), c.body(dx, c.k, c.xs), dad.clone(), dbd.clone()
        want = c.proj(), *c.grad()
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
        assert np.array_equal(got[2].cpu().numpy()[:, :c.r], want[2])
        assert np.array_equal(got[3].cpu().numpy()[:, :c.m], want[3])
        c.dat, c.dbt, c.dad, c.dbd = dat, dbt, dad, dbd


def test_on_another_stream():
    c = Case(200, 264, 136, 16, 4, seed=13)
    want = c.proj()
    s = torch.cuda.Stream()
    ws, out = c.scratch(R.rld_proj_workspace_bytes(c.n, c.k, c.m, c.r, c.slots)), c.out_rows(c.os)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        R.check(c.call_proj(out, ws), "rld_proj")
    s.synchronize()
    assert np.array_equal(c.body(out, c.m, c.os), want)


def test_two_calls_at_once():
    """Gradients of two projections on two streams, each with its own workspace: the
    bits of the same calls one after the other."""
    cases = [Case(1300, 264, 392, 32, 2, seed=41), Case(150, 1032, 264, 64, 5, seed=42)]
    want = [c.grad() for c in cases]
    runs = []
    for c in cases:
        c.tables()
        need = R.rld_proj_grad_workspace_bytes(c.n, c.k, c.m, c.r, c.slots)
        runs.append((c, c.scratch(need), c.out_rows(c.xs), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for c, ws, dx, s in runs:
            with torch.cuda.stream(s):
                R.check(c.call_grad(dx, ws), "rld_proj_grad")
    torch.cuda.synchronize()
    for (c, ws, dx, s), (dx0, da0, db0) in zip(runs, want):
        da, db = c.slot_gradients()
        assert np.array_equal(c.body(dx, c.k, c.xs), dx0)
        assert np.array_equal(da, da0) and np.array_equal(db, db0)


def test_far_rows():
    """Rows whose byte offsets pass 32 bits: a row stride of 2^21 elements and rows
    that reach 4 GiB behind the start, as projection and as gradient."""
    say("case: proj far rows")
    dev = require_gpu()
    stride, n, k, m, r = 1 << 21, 1050, 64, 72, 8
    c = Case(n, k, m, r, 3, seed=14)
    far = torch.full((n * stride,), NAN16, dtype=torch.int16, device=dev).view(n, stride)
    assert far.numel() * 2 > 1 << 32
    far[:, :k] = c.xd
    want, grads = c.proj(), c.grad()
    c.xd, c.xs = far, stride
    out = c.out_rows(c.os)
    ws = c.scratch(R.rld_proj_workspace_bytes(n, k, m, r, 3))
    R.check(c.call_proj(out, ws), "rld_proj")
    torch.cuda.synchronize()
    assert np.array_equal(c.body(out, m, c.os), want)
    c.tables()
    need = R.rld_proj_grad_workspace_bytes(n, k, m, r, 3)
    R.check(c.call_grad(None, c.scratch(need)), "rld_proj_grad")
    torch.cuda.synchronize()
    for a, b in zip(c.slot_gradients(), grads[1:]):
        assert np.array_equal(a, b)


def test_far_rows_of_large_tiles():
    """Grids of large tiles over rows that 32-bit offsets do not reach in sorted
    order (they are then taken in their own order): the projection and dx with
    wide strides have the bits of the narrow ones' bounds, dA and dB too."""
    say("case: proj far rows, large tiles")
    n, k, m, r = 2060, 328, 4616, 16
    c = Case(n, k, m, r, 5, "mixed", seed=15)
    wide = 1 << 18
    assert n * wide * 2 > 1 << 30
    far = torch.full((n, wide), NAN16, dtype=torch.int16, device=c.dev)
    far[:, :k] = c.xd[:, :k]
    c.xd, c.xs = far, wide
    c.check_proj()
    c = Case(n, m, k, r, 5, "mixed", seed=16)  # dx [n, 4616] from dy [n, 328]
    far[:, :k] = c.dyd[:, :k]
    far[:, k:] = NAN16
    c.dyd, c.os = far, wide
    c.check_grads()


def smaller(bits, e):
    """The values times 2^-e (zero where that is below the normal range)."""
    return np.where((bits >> 7 & 0xFF) > e, bits - (e << 7), 0).astype(np.uint16)


@pytest.mark.parametrize("n,k,m,r", [
    (40, 72, 264, 16),       # finish adds up the chunks
    (700, 72, 2312, 128),    # low rows summed before finish
    (2304, 72, 4616, 16),    # large tiles
])
def test_low_rows_next_to_the_largest_number(n, k, m, r):
    """Low rows that are finite in fp32 and would round to an infinity in BF16 (1.998
    2^127: the largest BF16 is 1.9921875 2^127): the outputs that they give are
    ordinary numbers, forward and in dx and dA.  (dB's u would underflow: not made.)"""
    say(f"case: proj low rows next to the largest number {n} {k} {m} {r}")
    c = Case(n, k, m, r, 2, seed=51)
    rows = c.rows_of(1)
    c.scale[1] = 1.998
    c.x[rows, :k] = 0
    c.x[rows, 0] = 0x7F00  # 2^127
    c.w[:, 0] = 0
    c.a[1, :r, 0] = 0
    c.a[1, 0, 0] = 0x3F80  # 1
    c.b[1, :m] = smaller(c.b[1, :m], 100)
    c.sd.copy_(torch.from_numpy(c.scale))
    for t, v in ((c.xd, c.x), (c.wd, c.w), (c.ad, c.a), (c.bd, c.b)):
        t.copy_(up(v, c.dev))
    c.check_proj()
    c = Case(n, m, k, r, 2, seed=52)  # dx [n, m] from dy [n, k]
    rows = c.rows_of(1)
    c.scale[1] = 1.998
    c.dy[rows, :k] = 0
    c.dy[rows, 0] = 0x7F00
    c.w[0, :m] = 0
    c.b[1, 0] = 0
    c.b[1, 0, 0] = 0x3F80
    c.a[1, :r] = smaller(c.a[1, :r], 100)
    c.x[rows, :m] = smaller(c.x[rows, :m], 100)
    c.sd.copy_(torch.from_numpy(c.scale))
    for t, v in ((c.xd, c.x), (c.dyd, c.dy), (c.wd, c.w), (c.ad, c.a), (c.bd, c.b)):
        t.copy_(up(v, c.dev))
    c.tables()
    dx = c.out_rows(c.xs)
    need = R.rld_proj_grad_workspace_bytes(n, m, k, r, 2)
    R.check(c.call_grad(dx, c.scratch(need), db=False), "rld_proj_grad")
    torch.cuda.synchronize()
    rx, ra, _ = c.gradients()
    c.check_rounded(bf16_values(c.body(dx, m, c.xs)), *rx, k, "dx")
    c.check_grad(c.slot_gradients()[0], *ra, k, max(len(c.rows_of(s)) for s in range(2)), "dA")


@pytest.mark.parametrize("n,k,m,r", [(40, 72, 264, 16), (2304, 72, 4616, 16)])
def test_infinite_low_rows(n, k, m, r):
    """An infinity in x makes every value of a low row infinite: the outputs are the
    infinities and NaN of the formula, not NaN throughout."""
    say(f"case: proj infinite low rows {n} {k} {m} {r}")
    c = Case(n, k, m, r, 2, seed=53)
    rows = c.rows_of(1)
    c.x[rows, 0] = 0x7F80
    c.a[1, :r, 0] &= 0x7FFF
    c.b[1, :m // 2] &= 0x7FFF  # of one sign: no infinity meets its negative
    for t, v in ((c.xd, c.x), (c.ad, c.a), (c.bd, c.b)):
        t.copy_(up(v, c.dev))
    with np.errstate(invalid="ignore"):
        want = c.forward()
        got = bf16_values(c.proj())
    assert np.isposinf(want[0][rows]).any() and np.isnan(want[0][rows]).any()
    assert not np.isfinite(want[0][rows]).any()
    assert np.array_equal(got[rows], want[0][rows], equal_nan=True)
    rest = np.setdiff1d(np.arange(n), rows)
    c.check_rounded(got[rest], *(v[rest] for v in want), k, "out")


@pytest.mark.parametrize("n,k,m,r,slots,layout", [
    (2400, 128, 4104, 8, 2, "runs"),      # two steps
    (2500, 256, 4360, 16, 3, "runs"),     # four
    (2100, 264, 4872, 40, 6, "mixed"),    # four and an eighth
    (2600, 1024, 4104, 64, 4, "runs"),    # 16, the low rows in two chunks
    (2300, 1096, 4104, 128, 3, "mixed"),  # 17 and an eighth, three chunks
    (2304, 4096, 4104, 64, 4, "runs"),    # 64, eight chunks
    (4100, 40, 2568, 16, 3, "mixed"),     # no whole step
])
def test_many_tiles_of_every_depth(n, k, m, r, slots, layout):
    """Large tiles of even and odd numbers of steps with and without a tail, and of
    low rows that are summed from chunks before, in both directions."""
    say(f"case: proj many tiles of every depth {n} {k} {m} {r} {layout}")
    Case(n, k, m, r, slots, layout, 8, 16, 8, seed=61).check_proj()
    Case(n, m, k, r, slots, layout, 8, 16, 8, seed=62).check_grads()


def test_far_rows_of_large_tiles_in_chunks():
    """Rows in their own order (too far for 32-bit offsets), low rows of three chunks."""
    say("case: proj far rows, large tiles, chunks")
    n, k, m, r = 2060, 1032, 4616, 24
    wide = 1 << 18
    assert n * wide * 2 > 1 << 30
    c = Case(n, k, m, r, 5, "mixed", seed=63)
    far = torch.full((n, wide), NAN16, dtype=torch.int16, device=c.dev)
    far[:, :k] = c.xd[:, :k]
    c.xd, c.xs = far, wide
    c.check_proj()
    c = Case(n, m, k, r, 5, "mixed", seed=64)
    far[:, :k] = c.dyd[:, :k]
    far[:, k:] = NAN16
    c.dyd, c.os = far, wide
    c.check_grads()


@pytest.mark.parametrize("n,k,m,r,slots", [
    # sorted first, low rows summed before finish: ranks up to 32, 64, 128
    (1030, 4104, 1000, 24, 16), (1030, 4104, 1032, 64, 16), (700, 2056, 1032, 128, 24),
    # sorted first, finish adds up the chunks
    (1030, 4104, 520, 16, 16),
    # sorted beside the product, summed before finish: ranks up to 32, 128
    (1100, 1032, 2056, 32, 4), (900, 520, 2056, 128, 4),
])
@pytest.mark.parametrize("layout", ["mixed", "runs"])
def test_proj_of_many_slots_and_rows(n, k, m, r, slots, layout):
    """Every way that the low rows of a split product take."""
    say(f"case: proj of many slots and rows {n} {k} {m} {r} {slots} {layout}")
    Case(n, k, m, r, slots, layout, 8, 0, 8, seed=65).check_proj()
