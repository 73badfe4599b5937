"""The MoE token movement, the gradient norm and clipping on the CPU: refusals, each
before any launch, the packed list of gradients and the workspace size.  Every device
call here fails validation or launches nothing."""
import ctypes

import numpy as np
import pytest

import routed_lora_delta_amd as R

FAKE = 0x7F0000001000  # 16-byte aligned, never dereferenced by validation


def _dispatch(**kw):
    a = dict(x=FAKE, f=0, xs=64, T=4, k=2, h=64, sr=FAKE, rows=FAKE, rs=64, pl=FAKE)
    a.update(kw)
    return R.rld_moe_dispatch(a["x"], a["f"], a["xs"], a["T"], a["k"], a["h"], a["sr"],
                              a["rows"], a["rs"], a["pl"], 0)


def _dispatch_grad(**kw):
    a = dict(d=FAKE, f=0, ds=64, sr=FAKE, pl=FAKE, T=4, k=2, h=64, add=FAKE, adds=64, dx=FAKE,
             dxs=64)
    a.update(kw)
    return R.rld_moe_dispatch_grad(a["d"], a["f"], a["ds"], a["sr"], a["pl"], a["T"], a["k"],
                                   a["h"], a["add"], a["adds"], a["dx"], a["dxs"], 0)


def _combine(**kw):
    a = dict(rows=FAKE, f=0, rs=64, i=FAKE, sr=FAKE, pl=FAKE, w=FAKE, T=4, k=2, h=64, add=FAKE,
             adds=64, out=FAKE, os=64)
    a.update(kw)
    return R.rld_moe_combine(a["rows"], a["f"], a["rs"], a["i"], a["sr"], a["pl"], a["w"],
                             a["T"], a["k"], a["h"], a["add"], a["adds"], a["out"], a["os"], 0)


def _combine_grad(**kw):
    a = dict(rows=FAKE, f=0, rs=64, i=FAKE, sr=FAKE, pl=FAKE, w=FAKE, d=FAKE, ds=64, T=4, k=2,
             h=64, dr=FAKE, drs=64, dw=FAKE)
    a.update(kw)
    return R.rld_moe_combine_grad(a["rows"], a["f"], a["rs"], a["i"], a["sr"], a["pl"], a["w"],
                                  a["d"], a["ds"], a["T"], a["k"], a["h"], a["dr"], a["drs"],
                                  a["dw"], 0)


ALL = [_dispatch, _dispatch_grad, _combine, _combine_grad]
EINVAL, EALIGN, EUNSUPPORTED = R.RLD_EINVAL, R.RLD_EALIGN, R.RLD_EUNSUPPORTED


@pytest.mark.parametrize("call", ALL)
@pytest.mark.parametrize("kw,status", [
    (dict(k=0), EINVAL), (dict(h=0), EINVAL), (dict(k=33), EUNSUPPORTED), (dict(h=60), EALIGN),
    (dict(h=(1 << 21) + 8), EUNSUPPORTED), (dict(T=1 << 30), EUNSUPPORTED),
    (dict(T=1 << 26, k=32), EUNSUPPORTED), (dict(sr=FAKE + 2), EALIGN),
    (dict(pl=FAKE + 1), EALIGN), (dict(sr=None), EINVAL), (dict(pl=None), EINVAL),
])
def test_refusals_of_every_call(call, kw, status):
    assert call(**kw) == status


def test_grids_past_32_bits_are_refused():
    # 2^26 - 3 pieces of 1 KB, one wave each
    T = (1 << 26) - 3
    assert _dispatch(T=T, k=1) == EUNSUPPORTED
    assert _dispatch(T=T // 4 + 1, k=1, h=2048, xs=2048, rs=2048) == EUNSUPPORTED
    assert _dispatch(T=T // 8 + 1, k=1, f=1, h=2048, xs=2048, rs=2048) == EUNSUPPORTED
    assert _combine(T=T, k=1) == EUNSUPPORTED
    assert _dispatch_grad(T=T, k=1) == EUNSUPPORTED
    assert _combine_grad(T=T, k=1) == EUNSUPPORTED


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), EINVAL), (dict(rows=None), EINVAL), (dict(xs=56), EINVAL),
    (dict(rs=56), EINVAL), (dict(xs=68), EALIGN), (dict(rs=68), EALIGN),
    (dict(x=FAKE + 8), EALIGN), (dict(rows=FAKE + 8), EALIGN),
])
def test_dispatch_refusals(kw, status):
    assert _dispatch(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(d=None), EINVAL), (dict(dx=None), EINVAL), (dict(ds=56), EINVAL),
    (dict(adds=56), EINVAL), (dict(dxs=56), EINVAL), (dict(ds=68), EALIGN),
    (dict(adds=68), EALIGN), (dict(dxs=68), EALIGN), (dict(d=FAKE + 8), EALIGN),
    (dict(add=FAKE + 8), EALIGN), (dict(dx=FAKE + 4), EALIGN),
    (dict(sr=None, pl=None), EINVAL),
])
def test_dispatch_grad_refusals(kw, status):
    assert _dispatch_grad(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(rows=None), EINVAL), (dict(out=None), EINVAL), (dict(w=None), EINVAL),
    (dict(rs=56), EINVAL), (dict(adds=56), EINVAL), (dict(os=56), EINVAL),
    (dict(rs=68), EALIGN), (dict(adds=68), EALIGN), (dict(os=68), EALIGN),
    (dict(rows=FAKE + 8), EALIGN), (dict(add=FAKE + 8), EALIGN), (dict(out=FAKE + 2), EALIGN),
    (dict(w=FAKE + 2), EALIGN), (dict(i=FAKE + 2), EALIGN),
])
def test_combine_refusals(kw, status):
    assert _combine(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(rows=None), EINVAL), (dict(d=None), EINVAL), (dict(w=None), EINVAL),
    (dict(dr=None, dw=None), EINVAL), (dict(rs=56), EINVAL), (dict(ds=56), EINVAL),
    (dict(drs=56), EINVAL), (dict(rs=68), EALIGN), (dict(ds=68), EALIGN), (dict(drs=68), EALIGN),
    (dict(rows=FAKE + 8), EALIGN), (dict(d=FAKE + 8), EALIGN), (dict(dr=FAKE + 8), EALIGN),
    (dict(w=FAKE + 2), EALIGN), (dict(dw=FAKE + 2), EALIGN), (dict(i=FAKE + 2), EALIGN),
])
def test_combine_grad_refusals(kw, status):
    assert _combine_grad(**kw) == status


def test_no_tokens_is_a_no_op():
    assert _dispatch(T=0, x=None, sr=None, rows=None, pl=None) == R.RLD_OK
    assert _dispatch_grad(T=0, d=None, sr=None, pl=None, add=None, dx=None) == R.RLD_OK
    assert _combine(T=0, rows=None, i=None, sr=None, pl=None, w=None, add=None,
                    out=None) == R.RLD_OK
    assert _combine_grad(T=0, rows=None, i=None, sr=None, pl=None, w=None, d=None) == R.RLD_OK
    assert _combine_grad(T=0, dr=None, dw=None) == EINVAL


# ---------------------------------------------------------------- gradients ----

CHUNK = 8192  # bytes


def entries(rows):
    """rows: (addr, out_addr, count, group, bf16)."""
    return np.array(rows, np.dtype(R.rld_grad_entry))


def pack(rows, groups):
    e = entries(rows)
    n = ctypes.c_uint32(77)
    assert R.rld_grad_chunks(e, len(e), ctypes.byref(n)) == R.RLD_OK
    chunks = np.zeros(max(1, n.value), np.dtype(R.rld_grad_chunk))
    starts = np.full(groups + 1, 0xFFFFFFFF, np.uint32)
    assert R.rld_grad_pack(e, len(e), groups, chunks, n.value, starts) == R.RLD_OK
    return chunks[:n.value], starts


@pytest.mark.parametrize("groups", [1, 3, 7])
def test_pack_covers_each_gradient_once_and_sorts_by_group(groups):
    rng = np.random.default_rng(groups)
    rows, at = [], FAKE
    for i in range(40):
        bf16 = int(rng.integers(2))
        count = int(rng.choice([0, 1, 5, 2047, 2048, 2049, 4096, 4097, 100003]))
        out = at + (1 << 40) if i % 3 else 0
        rows.append((at, out, count, int(rng.integers(groups)), bf16))
        at += (count * 4 + 63) // 16 * 16
    chunks, starts = pack(rows, groups)
    want = []  # the definition: group by group, entry by entry, piece by piece
    for g in range(groups):
        assert starts[g] == len(want)
        for addr, out, count, group, bf16 in rows:
            size = 2 if bf16 else 4
            for done in range(0, count if group == g else 0, CHUNK // size):
                want.append((addr + done * size, (out or addr) + done * size,
                             min(CHUNK // size, count - done), g, bf16, 0))
    assert starts[groups] == len(want) == len(chunks)
    assert [tuple(int(v) for v in c) for c in chunks] == want


def test_pack_of_nothing():
    for rows in ([], [(0, 0, 0, 1, 0), (FAKE, 0, 0, 0, 1)]):
        chunks, starts = pack(rows, 2)
        assert len(chunks) == 0 and starts.tolist() == [0, 0, 0]


@pytest.mark.parametrize("row,groups,status", [
    ((FAKE, 0, 8, 2, 0), 2, EINVAL), ((0, 0, 8, 0, 0), 1, EINVAL),
    ((0, FAKE, 8, 0, 0), 1, EINVAL), ((FAKE + 8, 0, 8, 0, 0), 1, EALIGN),
    ((FAKE, FAKE + 4, 8, 0, 0), 1, EALIGN), ((FAKE, 0, 8, 0, 0), 0, EINVAL),
    ((FAKE, 0, 8, 0, 0), (1 << 20) + 1, EUNSUPPORTED),
    ((FAKE, 0, 1 << 42, 0, 0), 1, EUNSUPPORTED), ((FAKE, 0, (1 << 64) - 1, 0, 1), 1, EUNSUPPORTED),
])
def test_pack_refusals(row, groups, status):
    e = entries([row])
    chunks = np.zeros(4, np.dtype(R.rld_grad_chunk))
    starts = np.zeros(4, np.uint32)
    assert R.rld_grad_pack(e, 1, groups, chunks, 4, starts) == status


def test_pack_refuses_missing_and_short_arrays():
    e = entries([(FAKE, 0, 5000, 0, 0)])  # three chunks
    n = ctypes.c_uint32()
    chunks = np.zeros(3, np.dtype(R.rld_grad_chunk))
    starts = np.zeros(2, np.uint32)
    assert R.rld_grad_chunks(e, 1, None) == EINVAL
    assert R.rld_grad_chunks(None, 1, ctypes.byref(n)) == EINVAL
    assert R.rld_grad_pack(None, 1, 1, chunks, 3, starts) == EINVAL
    assert R.rld_grad_pack(e, 1, 1, None, 3, starts) == EINVAL
    assert R.rld_grad_pack(e, 1, 1, chunks, 3, None) == EINVAL
    assert R.rld_grad_pack(e, 1, 1, chunks, 2, starts) == R.RLD_ENOSPACE
    assert not chunks["addr"].any()
    assert R.rld_grad_pack(e, 1, 1, chunks, 3, starts) == R.RLD_OK


def _list(**kw):
    a = dict(chunks=FAKE, group_starts=FAKE, num_chunks=8, num_groups=2)
    a.update(kw)
    return R.rld_grad_list(*[a[f] for f, _ in R.rld_grad_list._fields_])


LISTS = [
    (dict(chunks=None), EINVAL), (dict(group_starts=None), EINVAL), (dict(num_groups=0), EINVAL),
    (dict(chunks=FAKE + 8), EALIGN), (dict(group_starts=FAKE + 2), EALIGN),
    (dict(num_groups=(1 << 20) + 1), EUNSUPPORTED), (dict(num_chunks=(1 << 30) + 1), EUNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", LISTS)
def test_list_refusals(kw, status):
    assert R.rld_grad_norm(_list(**kw), FAKE, None, FAKE, 1 << 30, 0) == status
    assert R.rld_grad_clip(_list(**kw), FAKE, FAKE, 0) == status
    assert R.rld_grad_norm_workspace_bytes(_list(**kw)) == 0


def test_norm_and_clip_refusals():
    l = _list()
    need = R.rld_grad_norm_workspace_bytes(l)
    assert need >= 8 * (8 + 2 - 1)
    assert R.rld_grad_norm(l, None, None, FAKE, need, 0) == EINVAL
    assert R.rld_grad_norm(l, FAKE, None, None, need, 0) == EINVAL
    assert R.rld_grad_norm(l, FAKE + 2, None, FAKE, need, 0) == EALIGN
    assert R.rld_grad_norm(l, FAKE, FAKE + 4, FAKE, need, 0) == EALIGN
    assert R.rld_grad_norm(l, FAKE, None, FAKE + 8, need, 0) == EALIGN
    assert R.rld_grad_norm(l, FAKE, None, FAKE, need - 1, 0) == R.RLD_ENOSPACE
    assert R.rld_grad_clip(l, None, FAKE, 0) == EINVAL
    assert R.rld_grad_clip(l, FAKE, None, 0) == EINVAL
    assert R.rld_grad_clip(l, FAKE + 1, FAKE, 0) == EALIGN
    assert R.rld_grad_clip(l, FAKE, FAKE + 2, 0) == EALIGN


def test_empty_lists_launch_nothing():
    none = R.rld_grad_list(None, None, 0, 0)
    assert R.rld_grad_norm(none, None, None, None, 0, 0) == R.RLD_OK
    assert R.rld_grad_clip(none, None, None, 0) == R.RLD_OK
    assert R.rld_grad_clip(_list(num_chunks=0, chunks=None), None, None, 0) == R.RLD_OK


def test_workspace_holds_a_sum_for_each_wave_and_group():
    last = 0
    for n in (0, 1, 2, 4095, 4096, 4097, 1 << 20):
        now = R.rld_grad_norm_workspace_bytes(_list(num_chunks=n, num_groups=5))
        assert now >= last and now % 16 == 0 and now >= 8 * (min(n, 4096) + 4)
        last = now
    assert R.rld_grad_norm_workspace_bytes(_list(num_groups=1 << 20)) >= 8 * ((1 << 20) + 7)
