"""rld_proj, rld_proj_grad, rld_moe_router and rld_moe_router_grad on the CPU: the
refusals, each before any launch, and the workspace sizes.  Every call here fails
validation or is an empty batch that launches nothing."""
import glob
import os
import re

import pytest

import routed_lora_delta_amd as R

FAKE = 0x7F0000001000  # 16-byte aligned, never dereferenced by validation


def _route(**kw):
    a = dict(a_table=FAKE, b_table=FAKE, scale_table=FAKE, max_loras=4, k_in=64, n_out=128,
             max_rank=16)
    a.update(kw)
    return R.rld_route(*[a[f] for f, _ in R.rld_route._fields_])


def _proj(route=None, **kw):
    a = dict(w=FAKE, ws=64, x=FAKE, xs=64, seq=FAKE, n=4, out=FAKE, os=128, wk=FAKE, wb=1 << 30)
    a.update(kw)
    return R.rld_proj(route or _route(), a["w"], a["ws"], a["x"], a["xs"], a["seq"], a["n"],
                      a["out"], a["os"], a["wk"], a["wb"], 0)


def _grad(route=None, **kw):
    a = dict(w=FAKE, ws=64, x=FAKE, xs=64, dy=FAKE, dys=128, seq=FAKE, n=4, dx=FAKE, dxs=64,
             da=FAKE, db=FAKE, acc=0, wk=FAKE, wb=1 << 30)
    a.update(kw)
    return R.rld_proj_grad(route or _route(), a["w"], a["ws"], a["x"], a["xs"], a["dy"],
                           a["dys"], a["seq"], a["n"], a["dx"], a["dxs"], a["da"], a["db"],
                           a["acc"], a["wk"], a["wb"], 0)


ROUTES = [
    (dict(a_table=None), R.RLD_EINVAL), (dict(b_table=None), R.RLD_EINVAL),
    (dict(scale_table=None), R.RLD_EINVAL), (dict(max_loras=0), R.RLD_EINVAL),
    (dict(k_in=0), R.RLD_EINVAL), (dict(n_out=0), R.RLD_EINVAL), (dict(max_rank=0), R.RLD_EINVAL),
    (dict(max_rank=136), R.RLD_EUNSUPPORTED), (dict(max_rank=12), R.RLD_EALIGN),
    (dict(k_in=60), R.RLD_EALIGN), (dict(n_out=100), R.RLD_EALIGN),
    (dict(max_loras=1 << 23), R.RLD_EUNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", ROUTES)
def test_route_refusals(kw, status):
    assert _proj(_route(**kw)) == status
    assert _grad(_route(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(w=None), R.RLD_EINVAL), (dict(x=None), R.RLD_EINVAL), (dict(seq=None), R.RLD_EINVAL),
    (dict(out=None), R.RLD_EINVAL), (dict(wk=None), R.RLD_EINVAL),
    (dict(ws=56), R.RLD_EINVAL), (dict(xs=56), R.RLD_EINVAL), (dict(os=120), R.RLD_EINVAL),
    (dict(ws=68), R.RLD_EALIGN), (dict(xs=68), R.RLD_EALIGN), (dict(os=132), R.RLD_EALIGN),
    (dict(w=FAKE + 8), R.RLD_EALIGN), (dict(x=FAKE + 2), R.RLD_EALIGN),
    (dict(out=FAKE + 8), R.RLD_EALIGN), (dict(wk=FAKE + 8), R.RLD_EALIGN),
    (dict(ws=(1 << 21) + 8), R.RLD_EUNSUPPORTED), (dict(xs=(1 << 21) + 8), R.RLD_EUNSUPPORTED),
    (dict(os=(1 << 21) + 8), R.RLD_EUNSUPPORTED),
    (dict(n=1 << 30), R.RLD_EUNSUPPORTED), (dict(wb=255), R.RLD_ENOSPACE),
])
def test_proj_refusals(kw, status):
    assert _proj(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(w=None), R.RLD_EINVAL), (dict(x=None), R.RLD_EINVAL), (dict(dy=None), R.RLD_EINVAL),
    (dict(seq=None), R.RLD_EINVAL), (dict(wk=None), R.RLD_EINVAL),
    (dict(dx=None, da=None, db=None), R.RLD_EINVAL),
    (dict(ws=56), R.RLD_EINVAL), (dict(xs=56), R.RLD_EINVAL), (dict(dys=120), R.RLD_EINVAL),
    (dict(dxs=56), R.RLD_EINVAL), (dict(ws=68), R.RLD_EALIGN), (dict(xs=68), R.RLD_EALIGN),
    (dict(dys=132), R.RLD_EALIGN), (dict(dxs=68), R.RLD_EALIGN), (dict(dy=FAKE + 8), R.RLD_EALIGN),
    (dict(dx=FAKE + 8), R.RLD_EALIGN), (dict(wk=FAKE + 4), R.RLD_EALIGN),
    (dict(da=FAKE + 4), R.RLD_EALIGN), (dict(db=FAKE + 4), R.RLD_EALIGN),
    (dict(dys=(1 << 21) + 8), R.RLD_EUNSUPPORTED), (dict(ws=(1 << 21) + 8), R.RLD_EUNSUPPORTED),
    (dict(dxs=(1 << 21) + 8), R.RLD_EUNSUPPORTED),
    (dict(n=1 << 30), R.RLD_EUNSUPPORTED), (dict(wb=512), R.RLD_ENOSPACE),
])
def test_proj_grad_refusals(kw, status):
    assert _grad(**kw) == status


def test_proj_empty_batch_is_a_no_op():
    assert _proj(n=0, x=None, seq=None, out=None, wk=None, wb=0) == R.RLD_OK
    # dx alone of no rows: nothing to launch
    assert _grad(n=0, x=None, dy=None, seq=None, da=None, db=None) == R.RLD_OK


def _router(**kw):
    a = dict(l=FAKE, f=0, ls=128, m=None, T=8, E=128, k=8, norm=1, i=FAKE, w=FAKE, c=FAKE,
             o=FAKE, t=FAKE, r=FAKE, loss=FAKE, wk=FAKE, wb=1 << 30)
    a.update(kw)
    return R.rld_moe_router(a["l"], a["f"], a["ls"], a["m"], a["T"], a["E"], a["k"], a["norm"],
                            a["i"], a["w"], a["c"], a["o"], a["t"], a["r"], a["loss"], a["wk"],
                            a["wb"], 0)


@pytest.mark.parametrize("kw,status", [
    (dict(l=None), R.RLD_EINVAL), (dict(ls=127), R.RLD_EINVAL), (dict(E=0), R.RLD_EINVAL),
    (dict(k=0), R.RLD_EINVAL), (dict(E=4, k=5), R.RLD_EINVAL), (dict(i=None), R.RLD_EINVAL),
    (dict(w=None), R.RLD_EINVAL), (dict(wk=None), R.RLD_EINVAL),
    (dict(E=1025, ls=1025), R.RLD_EUNSUPPORTED), (dict(k=33), R.RLD_EUNSUPPORTED),
    (dict(T=1 << 26), R.RLD_EUNSUPPORTED), (dict(l=FAKE + 1), R.RLD_EALIGN),
    (dict(l=FAKE + 2, f=1), R.RLD_EALIGN), (dict(i=FAKE + 2), R.RLD_EALIGN),
    (dict(w=FAKE + 1), R.RLD_EALIGN), (dict(m=FAKE + 2), R.RLD_EALIGN),
    (dict(c=FAKE + 2), R.RLD_EALIGN), (dict(o=FAKE + 2), R.RLD_EALIGN),
    (dict(t=FAKE + 2), R.RLD_EALIGN), (dict(r=FAKE + 2), R.RLD_EALIGN),
    (dict(loss=FAKE + 2), R.RLD_EALIGN), (dict(wk=FAKE + 8), R.RLD_EALIGN),
    (dict(wb=64), R.RLD_ENOSPACE),
])
def test_router_refusals(kw, status):
    assert _router(**kw) == status


def test_router_empty_batch_with_no_tables_is_a_no_op():
    assert _router(T=0, l=None, i=None, w=None, c=None, o=None, t=None, r=None, loss=None,
                   wk=None, wb=0) == R.RLD_OK


def _router_grad(**kw):
    a = dict(l=FAKE, f=0, ls=128, m=None, T=8, E=128, k=8, norm=1, i=FAKE, c=FAKE, dw=FAKE,
             dl=FAKE, o=FAKE, os=128)
    a.update(kw)
    return R.rld_moe_router_grad(a["l"], a["f"], a["ls"], a["m"], a["T"], a["E"], a["k"],
                                 a["norm"], a["i"], a["c"], a["dw"], a["dl"], a["o"], a["os"], 0)


@pytest.mark.parametrize("kw,status", [
    (dict(l=None), R.RLD_EINVAL), (dict(ls=127), R.RLD_EINVAL), (dict(os=127), R.RLD_EINVAL),
    (dict(o=None), R.RLD_EINVAL), (dict(dw=None, dl=None), R.RLD_EINVAL),
    (dict(i=None), R.RLD_EINVAL), (dict(c=None), R.RLD_EINVAL), (dict(k=0), R.RLD_EINVAL),
    (dict(E=4, k=5), R.RLD_EINVAL), (dict(E=1025, ls=1025), R.RLD_EUNSUPPORTED),
    (dict(k=33), R.RLD_EUNSUPPORTED), (dict(T=1 << 26), R.RLD_EUNSUPPORTED),
    (dict(l=FAKE + 1), R.RLD_EALIGN), (dict(o=FAKE + 2, f=1), R.RLD_EALIGN),
    (dict(m=FAKE + 2), R.RLD_EALIGN), (dict(i=FAKE + 2), R.RLD_EALIGN),
    (dict(c=FAKE + 2), R.RLD_EALIGN), (dict(dw=FAKE + 2), R.RLD_EALIGN),
    (dict(dl=FAKE + 2), R.RLD_EALIGN),
])
def test_router_grad_refusals(kw, status):
    assert _router_grad(**kw) == status


def test_router_grad_empty_batch_is_a_no_op():
    assert _router_grad(T=0, l=None, o=None) == R.RLD_OK


def test_workspace_sizes_grow_with_the_call():
    p = R.rld_proj_workspace_bytes
    assert p(0, 64, 64, 16, 4) == 0 and p(4, 64, 64, 16, 0) == 0 and p(4, 64, 0, 16, 4) == 0
    assert p(4, 64, 64, 16, 4) >= 4 * 16 * 4 + 4 * 64 * 4
    assert p(5, 4096, 64, 16, 4) > p(4, 4096, 64, 16, 4)
    g = R.rld_proj_grad_workspace_bytes
    assert g(4, 64, 128, 16, 0) == 0 and g(0, 64, 128, 16, 4) > 0
    assert g(5, 4096, 128, 16, 4) > g(4, 4096, 128, 16, 4)
    r = R.rld_moe_router_workspace_bytes
    assert r(0, 128, 8) == 0 and r(129, 128, 8) > r(128, 128, 8) > 0


def test_workspace_for_the_largest_call_does_for_every_smaller_one():
    for k, m, rank, slots in [(4096, 1024, 16, 16), (768, 2048, 64, 2), (64, 12288, 8, 1)]:
        for size in (R.rld_proj_workspace_bytes, R.rld_proj_grad_workspace_bytes):
            last = 0
            for n in [1, 2, 15, 16, 17, 32, 33, 63, 64, 65, 100, 128, 129, 256, 500, 512, 513, 1000,
                      1024, 1025, 2000, 2047, 2304, 2305, 4096, 8192, 20000, 1 << 17, 1 << 20]:
                now = size(n, k, m, rank, slots)
                assert now >= last, (size, n, k, m)
                last = now
    last = 0
    for t in [1, 64, 65, 128, 129, 8191, 8192, 8193, 16384, 16385, 32768, 32769, 65536]:
        now = R.rld_moe_router_workspace_bytes(t, 128, 8)
        assert now >= last, t
        last = now


@pytest.mark.parametrize("tokens", [(1 << 26) - 3, (1 << 26) - 1])
def test_router_refuses_tokens_whose_grid_would_pass_32_bits(tokens):
    """At 64 lanes a token, in blocks of 256, they are 2^32 threads."""
    assert _router_grad(T=tokens, E=512, ls=512, os=512) == R.RLD_EUNSUPPORTED
    assert _router(T=tokens, E=512, ls=512, k=2) == R.RLD_EUNSUPPORTED


def test_inline_assembly_declares_m0():
    """A statement that writes m0 says so: the compiler may hold a value there."""
    csrc = os.path.join(os.path.dirname(R.library_path()), "csrc")
    found = 0
    for path in glob.glob(os.path.join(csrc, "*.h*")):
        with open(path) as f:
            for stmt in re.findall(r"\basm\b[^;]*;", f.read()):
                if re.search(r"s_mov_b32 m0\b", stmt):
                    found += 1
                    assert '"m0"' in stmt.rsplit(":", 1)[1], (path, stmt)
    assert found


def test_sorts_of_minutes_are_refused():
    """The sort by slot reads n ids for each of max_loras slots."""
    wide = dict(k_in=64, n_out=64)
    many = _route(max_loras=1 << 20, **wide)
    assert _proj(many, n=1 << 18, os=64) == R.RLD_EUNSUPPORTED
    assert _grad(many, n=1 << 18, dys=64) == R.RLD_EUNSUPPORTED
    assert _proj(many, n=(1 << 18) - 1, os=64, wb=64) == R.RLD_ENOSPACE  # the next check
