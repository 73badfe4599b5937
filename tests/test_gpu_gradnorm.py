"""GPU tests of rld_grad_norm and rld_grad_clip against the definitions in 64 bits.

Bounds, derived (u = 2^-24; a result in fp32 is off by u of its value, one in BF16 by
h = 2^-8).  The squares of fp32 numbers are exact in 64 bits, and N additions there are
off by less than N 2^-53 of the sum, so of 2^27 elements the root is off by less than
2^-27 of its value before it is rounded: a norm is within 1.2 u.  A clipped value is
x limit / (norm + 1e-6): the norm as it was handed over, then a sum, a quotient and a
product, each off by u (1e-6 itself by less): 4 u, then the result's rounding.
"""
import math

import numpy as np
import pytest
import torch

import routed_lora_delta_amd as R
import workloads as W
from gpu_util import require_gpu, say
from routed_lora_delta_amd.pool import DenseRoute, GradList

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
OUT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
STEP = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134}  # half a subnormal's
GAP = 8  # elements between one gradient and the next, at least


class Grads:
    """Gradients of these (elements, group, BF16?) in two pools, each behind a gap that
    holds an odd value, and outputs in two more."""

    def __init__(self, spec, groups, seed=0, scale=1.0, in_place=False):
        self.dev, self.groups = require_gpu(), groups
        g = torch.Generator(device=self.dev)
        g.manual_seed(seed)
        at, size = {}, {False: GAP, True: GAP}
        for i, (n, _, b) in enumerate(spec):
            at[i] = size[bool(b)]
            size[bool(b)] += (n + GAP + 7) // 8 * 8
        self.pool = {b: torch.full((size[b],), 77.25, device=self.dev,
                                   dtype=torch.bfloat16 if b else torch.float32)
                     for b in (False, True)}
        self.span = [(bool(b), at[i], at[i] + n, group) for i, (n, group, b) in enumerate(spec)]
        for b, lo, hi, _ in self.span:
            self.pool[b][lo:hi] = (torch.randn(hi - lo, generator=g, device=self.dev) *
                                   scale).to(self.pool[b].dtype)
        self.in_place = in_place
        self.out = self.pool if in_place else {b: torch.full_like(t, 77.25)
                                               for b, t in self.pool.items()}
        size = {False: 4, True: 2}
        self.list = GradList(
            [(self.pool[b].data_ptr() + lo * size[b],
              0 if in_place else self.out[b].data_ptr() + lo * size[b], hi - lo, group, b)
             for b, lo, hi, group in self.span], groups, self.dev)
        self.need = R.rld_grad_norm_workspace_bytes(self.list.list)
        self.ws = torch.full((self.need + 16,), 0xFF, dtype=torch.uint8, device=self.dev)
        self.norms = torch.full((groups + 1,), 77.25, device=self.dev)
        self.squares = torch.full((groups + 1,), 77.25, dtype=torch.float64, device=self.dev)

    def tensors(self, group, pool=None):
        return [(pool or self.pool)[b][lo:hi] for b, lo, hi, g in self.span if g == group]

    def norm(self, squares=True, stream=None):
        R.check(R.rld_grad_norm(self.list.list, self.norms, self.squares if squares else None,
                                self.ws, self.need, stream), "rld_grad_norm")

    def check_norm(self):
        self.norm()
        want = [sum(float((t.double() ** 2).sum()) for t in self.tensors(g))
                for g in range(self.groups)]
        got, sq = self.norms.cpu().numpy().astype(np.float64), self.squares.cpu().numpy()
        assert got[-1] == 77.25 and sq[-1] == 77.25
        assert bool((self.ws[self.need:] == 0xFF).all())
        for g, w in enumerate(want):
            assert abs(sq[g] - w) <= 2.0 ** -26 * w, g
            if math.sqrt(w) > 3.5e38:  # fp32 ends at 2^128 - 2^104 < 3.41e38
                assert got[g] == math.inf
                continue
            assert abs(got[g] - math.sqrt(w)) <= 1.2 * U * math.sqrt(w) + 2.0 ** -150, g

    def clip(self, limits, stream=None):
        lim = torch.tensor(limits, dtype=torch.float32, device=self.dev)
        R.check(R.rld_grad_clip(self.list.list, self.norms, lim, stream), "rld_grad_clip")
        torch.cuda.synchronize()

    def check_clip(self, limits):
        before = {b: t.clone() for b, t in self.pool.items()}
        norms = self.norms.cpu().numpy().astype(np.float64)
        self.clip(limits)
        want_pool = before if self.in_place else {b: torch.full_like(t, 77.25)
                                                  for b, t in self.pool.items()}
        for b, lo, hi, g in self.span:
            limit = float(np.float32(limits[g]))
            clipped = 0 <= limit < math.inf and limit / (norms[g] + 1e-6) < 1
            x, y = before[b][lo:hi], self.out[b][lo:hi]
            if not clipped:
                near = 0 <= limit < math.inf and limit / (norms[g] + 1e-6) < 1 + 4 * U
                assert torch.equal(x, y) or near
            if clipped:
                want = x.double() * (limit / (norms[g] + 1e-6))
                err = 4 * U * want.abs()
                bound = err + OUT[x.dtype] * (want.abs() + err) + STEP[x.dtype]
                assert bool(((y.double() - want).abs() <= bound).all()), (b, lo, hi, g)
            want_pool[b][lo:hi] = y
        for b in (False, True):  # what lies between the gradients
            assert torch.equal(self.out[b], want_pool[b])
            if not self.in_place:
                assert torch.equal(self.pool[b], before[b])


# elements of one to several chunks (2048 fp32, 4096 BF16), and around each border
SIZES = [0, 1, 2, 3, 4, 5, 7, 8, 9, 15, 17, 255, 256, 257, 2040, 2044, 2047, 2048, 2049, 2052,
         4088, 4095, 4096, 4097, 4104, 8191, 8192, 8193, 20000, 131072, 131077]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("groups", [1, 3, 40])
def test_every_size_in_both_types(groups, in_place):
    say(f"case: gradients of every size, {groups} groups")
    rng = np.random.default_rng(groups)
    spec = [(n, int(rng.integers(groups)), b) for n in SIZES for b in (0, 1)]
    g = Grads(spec, groups, groups, in_place=in_place)
    g.check_norm()
    norms = g.norms.cpu().numpy()[:-1]
    pick = [0.3, 0.999, 1.0, 1.001, 2.0, 0.0, -1.0, math.nan, math.inf, 1e-30]
    g.check_clip([float(v) * pick[i % 10] for i, v in enumerate(norms)])


@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 255, 256, 257])
def test_few_chunks(n):
    """One wave a chunk, one gradient in one group after the other."""
    say(f"case: {n} chunks")
    g = Grads([(2048, i, 0) for i in range(n)], n, n)
    g.check_norm()
    g.check_clip([0.5 if i % 2 else 1e9 for i in range(n)])


def test_many_small_gradients_of_many_groups():
    say("case: 9000 small gradients")
    rng = np.random.default_rng(1)
    spec = [(int(rng.integers(1, 40)), int(rng.integers(1200)), int(rng.integers(2)))
            for _ in range(9000)]
    g = Grads(spec, 1200, 2)
    g.check_norm()
    g.check_clip([float(v) for v in rng.uniform(0.1, 20, 1200)])


def test_groups_without_gradients():
    say("case: empty groups")
    g = Grads([(5000, 2, 0), (0, 5, 1), (3, 7, 1)], 9)
    g.check_norm()
    assert np.array_equal(g.norms.cpu().numpy()[:-1] > 0, [i in (2, 7) for i in range(9)])
    g.check_clip([0.1] * 9)
    none = Grads([], 4)
    none.check_norm()
    none.check_clip([1.0] * 4)


def test_values_at_the_ends_of_the_range():
    """Squares beyond fp32's range either way, and subnormal gradients."""
    say("case: range")
    for scale in (1e30, 1e37, 1e-30, 1e-38, 3e-42):
        g = Grads([(10001, 0, 0), (9999, 1, 1)], 2, 3, scale)
        g.check_norm()
        # 10000 values of 1e37 have a norm of 1e39, past fp32's end; the others' fit.
        # BF16 rounds what is below 2^-134 = 4.6e-41, 15 times 3e-42, to zero
        assert float(g.norms[0]) > 0 and (float(g.norms[1]) > 0) == (scale != 3e-42)
        assert bool(torch.isfinite(g.norms).all()) == (scale != 1e37)
        n = float(g.norms[0])
        g.check_clip([0.5 * n, 0.5 * n])
    g = Grads([(4, 0, 0)], 1)
    g.pool[False][GAP:GAP + 4] = 3.4e38  # the norm itself is past fp32's range
    g.norm()
    assert float(g.norms[0]) == math.inf and math.isfinite(float(g.squares[0]))
    g.clip([1.0])
    assert bool((g.out[False][GAP:GAP + 4] == 0).all())


def test_not_finite_values_stay_in_their_group():
    say("case: NaN and infinities")
    g = Grads([(5000, 0, 0), (5000, 1, 1), (5000, 2, 0), (5000, 3, 1), (70, 4, 0)], 5, 4)
    first = [lo for _, lo, _, _ in g.span]
    g.pool[False][first[0] + 4999] = math.nan
    g.pool[True][first[1] + 17] = math.inf
    g.norm()
    n = g.norms.cpu().numpy()
    assert np.isnan(n[0]) and n[1] == np.inf and np.isfinite(n[2:5]).all()
    before = {b: t.clone() for b, t in g.pool.items()}
    g.clip([1.0, 1.0, 0.5, -1.0, math.nan])
    assert torch.isnan(g.out[False][first[0]:first[0] + 5000]).all()
    y = g.out[True][first[1]:first[1] + 5000]
    assert bool(torch.isnan(y[17])) and float(y.nan_to_num(nan=0.0).abs().sum()) == 0
    want = before[False][first[2]:first[2] + 5000].double() * (0.5 / (float(n[2]) + 1e-6))
    off = (g.out[False][first[2]:first[2] + 5000].double() - want).abs()
    assert bool((off <= 5 * U * want.abs()).all())
    assert torch.equal(g.out[True][first[3]:first[3] + 5000], before[True][first[3]:first[3] + 5000])
    assert torch.equal(g.out[False][first[4]:first[4] + 70], before[False][first[4]:first[4] + 70])
    # groups that are not clipped keep a NaN norm's gradients as they are
    g2 = Grads([(300, 0, 0)], 1, in_place=True)
    g2.pool[False][GAP + 5] = math.nan
    kept = g2.pool[False].clone()
    g2.norm()
    for limit in (-1.0, math.inf, math.nan):
        g2.clip([limit])
        assert torch.equal(g2.pool[False].view(torch.int32), kept.view(torch.int32))


def test_long_runs_of_chunks():
    """More than 64 chunks a wave (2.2 GB), the groups' borders inside runs, and
    gradients past 32 bits of bytes and elements of the pool."""
    say("case: long runs")
    big = 275_000_001
    spec = [(big, 1, 0), (7, 0, 0), (big, 0, 0), (100_000, 2, 0)]
    g = Grads(spec, 3, 5, in_place=True)
    assert g.list.list.num_chunks > 4096 * 64
    g.check_norm()
    n = g.norms.cpu().numpy()
    keep = {lo: g.pool[False][lo:hi].clone() for _, lo, hi, _ in g.span}
    g.clip([n[0] * 0.5, n[1] * 2.0, n[2] * 0.25])
    for (_, lo, hi, group), f in zip(g.span, (1.0, 0.5, 0.5, 0.25)):
        y = g.pool[False][lo:hi]
        limit = float(np.float32(n[group] * (0.5, 2.0, 0.25)[group]))
        want = f if f == 1.0 else limit / (float(n[group]) + 1e-6)
        for a in range(0, hi - lo, 1 << 26):
            x = keep[lo][a:a + (1 << 26)].double() * want
            assert bool(((y[a:a + (1 << 26)].double() - x).abs() <= 5 * U * x.abs()).all())


def test_same_bits_every_run_and_graph_replays():
    """One captured norm and clipping, replayed with new gradients and limits, eager
    work and synchronizations between."""
    say("case: gradient graph")
    rng = np.random.default_rng(7)
    spec = [(int(rng.integers(1, 60000)), int(rng.integers(5)), int(rng.integers(2)))
            for _ in range(300)]
    g = Grads(spec, 5, 8)
    lim = torch.ones(5, device=g.dev)

    def step(st=None):
        g.norm(stream=st)
        R.check(R.rld_grad_clip(g.list.list, g.norms, lim, st), "rld_grad_clip")

    step()
    torch.cuda.synchronize()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(s)
    for trial in range(4):
        for t in g.pool.values():
            t.copy_((torch.randn(t.shape, device=g.dev) * 10.0 ** (trial - 2)).to(t.dtype))
        lim.copy_(torch.from_numpy(rng.uniform(1, 500, 5).astype(np.float32)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        bufs = (g.norms, g.squares, g.out[False], g.out[True])
        replayed = [b.clone() for b in bufs]
        g.norms[:5], g.squares[:5] = 5, 5
        for flag, lo, hi, _ in g.span:
            g.out[flag][lo:hi] = 5
        step(torch.cuda.Stream())
        torch.cuda.synchronize()
        for b, a in zip(bufs, replayed):
            for flag, lo, hi, _ in g.span:
                if b is g.out[flag]:
                    assert torch.equal(a[lo:hi], b[lo:hi])
            if b is g.norms or b is g.squares:
                assert torch.equal(a, b)
        g.check_norm()
        g.check_clip(lim.cpu().tolist())


def test_two_lists_at_once():
    say("case: two lists on two streams")
    a, b = (Grads([(700_001, i % 3, i % 2) for i in range(9)], 3, 10 + j) for j in range(2))
    a.norm()
    b.norm()
    torch.cuda.synchronize()
    want = [t.clone() for t in (a.norms, a.squares, b.norms, b.squares)]
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        a.norms[:3], b.norms[:3] = 0, 0
        torch.cuda.synchronize()
        a.norm(stream=sa)
        b.norm(stream=sb)
        torch.cuda.synchronize()
        for x, y in zip(want, (a.norms, a.squares, b.norms, b.squares)):
            assert torch.equal(x, y)


def test_adapters_of_a_projection_clipped_by_their_own_norms():
    """dA_s and dB_s as rld_proj_grad leaves them, a group for each slot: each slot's
    norm and clipped gradients, and a slot without rows."""
    say("case: projection's gradients -> norm -> clip")
    dev = require_gpu()
    rng = np.random.default_rng(9)
    n, k_in, n_out, rank, slots = 130, 264, 136, 16, 4
    adapters = [W.make_adapter(rng, s, rank, k_in, n_out, 16.0, False) for s in range(slots)]
    route = DenseRoute(adapters, slots, rank, k_in, n_out, dev)
    x, dy = (torch.randn((n, c), device=dev).bfloat16() for c in (k_in, n_out))
    w = torch.randn((n_out, k_in), device=dev).bfloat16()
    slot = torch.from_numpy(rng.integers(-1, slots - 1, n).astype(np.int32)).to(dev)
    da, db = (torch.full((slots, *s), 5.0, device=dev) for s in ((rank, k_in), (n_out, rank)))
    at = torch.arange(slots, device=dev)
    wb = R.rld_proj_grad_workspace_bytes(n, k_in, n_out, rank, slots)
    ws = torch.empty(wb, dtype=torch.uint8, device=dev)
    g = GradList([(t.data_ptr() + s * t[0].numel() * 4, 0, t[0].numel(), s, 0)
                  for t in (da, db) for s in range(slots)], slots, dev)
    need = R.rld_grad_norm_workspace_bytes(g.list)
    assert need <= wb  # one scratch buffer serves both calls
    norms, limits = torch.zeros(slots, device=dev), torch.tensor([1e-3, 1e9, 50.0, 1.0], device=dev)
    R.check(R.rld_proj_grad(route.route, w, k_in, x, k_in, dy, n_out, slot, n, None, k_in,
                            da.data_ptr() + at * (rank * k_in * 4),
                            db.data_ptr() + at * (n_out * rank * 4), 0, ws, wb), "proj_grad")
    torch.cuda.synchronize()
    before = [t.clone() for t in (da, db)]
    R.check(R.rld_grad_norm(g.list, norms, None, ws, wb), "norm")
    R.check(R.rld_grad_clip(g.list, norms, limits), "clip")
    torch.cuda.synchronize()
    for s in range(slots):
        want = math.sqrt(sum(float((t[s].double() ** 2).sum()) for t in before))
        assert abs(float(norms[s]) - want) <= 1.2 * U * want
        f = min(1.0, float(limits[s]) / (float(norms[s]) + 1e-6))
        for t, b in zip((da, db), before):
            x64 = b[s].double() * f
            assert bool(((t[s].double() - x64).abs() <= 5 * U * x64.abs()).all())
    assert float(norms[3]) == 0.0 and float(norms[0]) > 1e-3
