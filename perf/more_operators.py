"""What is measured of the MoE token movement and of the adapters' gradient norm.

Six operators, each in its plain form (elementary torch operations, sums in 32
bits or more) and, where `own` is true, as calls of this library:

  dispatch       rows[p] = x[f / top_k] for f = sorted_rows[p], places[f] = p    rld_moe_dispatch
  dispatch_grad  dx[t] = add[t] + the sum of token t's rows of drows       rld_moe_dispatch_grad
  combine        out[t] = add[t] + sum_j w[t, j] * row of (t, j)                 rld_moe_combine
  combine_grad   drows of (t, j) = w[t, j] * dout[t], dw[t, j] = row . dout[t]
                                                                           rld_moe_combine_grad
  norm           the norm of each adapter slot's gradients                         rld_grad_norm
  clip           that, and every gradient times min(1, limit / (norm + 1e-6))
                                                                 rld_grad_norm, rld_grad_clip
"""
import math

import torch

own = False

DEV = "cuda"
ALIGN = 128  # elements: a gradient in its pool starts at a multiple, zeros lie behind it

# k_in x n_out of the adapted projections: a decoder layer's attention and FFN, an expert's FFN
ATTN = "4096x4096 4096x1024 4096x1024 4096x4096"
LAYER = ATTN + " 4096x12288 4096x12288 12288x4096"
EXPERT = "2048x768 2048x768 768x2048"


# ------------------------------------------------------------------- cases ----

def _move(name, op, tokens, experts, top_k, width, dtype="bf16", pad=0, add=False, flat=False):
    return {"name": name, "op": op, "tokens": tokens, "experts": experts, "top_k": top_k,
            "width": width, "dtype": dtype, "pad": pad, "add": add, "flat": flat}


def _grads(name, op, modules, layers, ranks, slots, dtype="fp32"):
    return {"name": name, "op": op, "modules": modules, "layers": layers, "ranks": ranks,
            "slots": slots, "dtype": dtype}


def listed():
    return [
        # the MoE decode batch on its way to the experts
        _move("dispatch decode 32", "dispatch", 32, 128, 8, 2048),
        # the MoE prefill batch
        _move("dispatch prefill 4096", "dispatch", 4096, 128, 8, 2048),
        # a short ragged training batch in full precision, added to what dx holds
        _move("dispatch grad short", "dispatch_grad", 333, 64, 4, 4096, "fp32", 8, True),
        # the MoE prefill batch in training
        _move("dispatch grad 4096", "dispatch_grad", 4096, 128, 8, 2048),
        # one request's next token: flat rows as the decode gather leaves them, onto the residual
        _move("combine one token", "combine", 1, 128, 8, 2048, add=True, flat=True),
        # a long packed prefill, rows wider than their content
        _move("combine long prefill", "combine", 32771, 128, 8, 2048, pad=64, add=True),
        # a short ragged training batch of few choices
        _move("combine grad short", "combine_grad", 1237, 60, 2, 1000),
        # a long training batch
        _move("combine grad long", "combine_grad", 16387, 128, 8, 2048),
        # one adapted projection of one adapter
        _grads("norm one projection", "norm", "4096x4096", 1, "16", 1),
        # four adapters of different ranks on every projection of a 36-layer model
        _grads("norm 36 layers", "norm", LAYER, 36, "16 8 16 32", 4),
        # adapters of 96 experts each, one MoE layer
        _grads("clip experts", "clip", EXPERT, 96, "32 16", 4),
        # sixteen adapters on the attention of 36 layers, gradients in BF16
        _grads("clip attention bf16", "clip", ATTN, 36, "16 8", 16, "bf16"),
    ]


MOST_ROWS = 32771 * 8 * 2048 * 2  # bytes of the largest listed rows
MOST_GRADS = 90_000_000           # elements, under the largest list's


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["dispatch", "dispatch_grad", "combine", "combine", "combine_grad", "norm",
                     "clip"])
    while op in ("norm", "clip"):
        if rng.random() < 0.5:
            modules = rng.choice([ATTN, LAYER, EXPERT, "4096x4096 4096x1024"])
        else:  # any sizes, odd ones too: the elements of a gradient need not be even in number
            modules = " ".join(f"{_log_int(rng, 33, 12288)}x{_log_int(rng, 33, 12288)}"
                               for _ in range(rng.choice([1, 2, 3, 5])))
        case = _grads("", op, modules, _log_int(rng, 1, 128),
                      " ".join(str(rng.choice([1, 3, 8, 13, 16, 32, 64]))
                               for _ in range(rng.choice([1, 2, 3]))),
                      _log_int(rng, 1, 32), rng.choice(["fp32", "fp32", "bf16"]))
        if sum(n for n, _ in _tensors(case)) <= MOST_GRADS:
            del case["name"]
            return case
    while True:
        experts = rng.choice([8, 60, 64, 128, 256])
        top_k = rng.choice([1, 2, 3, 4, 6, 8])
        width = rng.choice([2048, 4096, 768, _log_int(rng, 64, 8192, 8)])
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        tokens = _log_int(rng, 1, 32771)
        if tokens * top_k * width * (2 if dtype == "bf16" else 4) <= MOST_ROWS:
            break
    case = _move("", op, tokens, experts, top_k, width, dtype, rng.choice([0, 0, 8, 64]),
                 op in ("combine", "dispatch_grad") and rng.random() < 0.5,
                 op.startswith("combine") and rng.random() < 0.25)
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs ----

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _prepare_move(case, seed):
    g = _gen(seed)
    t, e, k, h, pad, op = (case[v] for v in ("tokens", "experts", "top_k", "width", "pad", "op"))
    st, dt, n = dict(case), _dtype(case), t * k
    i32 = {"dtype": torch.int32, "device": DEV}
    # the router's choice, some experts preferred; one token in ten is padding
    score = torch.randn((t, e), generator=g, device=DEV)
    score += 0.5 * torch.randn((1, e), generator=g, device=DEV)
    choice = score.topk(k, 1).indices
    choice[torch.randperm(t, generator=g, device=DEV)[:t // 10]] = -1
    st["indices"] = choice.to(torch.int32)
    w = torch.softmax(torch.randn((t, k), generator=g, device=DEV), 1)
    st["weights"] = torch.where(choice >= 0, w, 0.0)
    flat = torch.where(choice >= 0, choice, e).reshape(-1)
    order = torch.sort(flat, stable=True).indices
    routed = torch.arange(n, device=DEV) < (flat < e).sum()
    st["sorted_rows"] = torch.where(routed, order, -1).to(torch.int32)
    st["places"] = torch.full((n,), -1, **i32)
    if op != "dispatch":  # an earlier dispatch left them
        st["places"][order[routed]] = torch.arange(n, **i32)[routed]
    if op == "dispatch":
        st["x"] = _normal(g, (t, h + pad), dt)
    else:  # rows that no token owns hold what happens to be there
        st["rows"] = _normal(g, (n, h + pad), dt)
    if case["add"]:
        st["add_rows"] = _normal(g, (t, h + pad), dt)
    if op == "combine_grad":
        st["dout"] = _normal(g, (t, h + pad), dt)
        st["dweights"] = torch.zeros((t, k), device=DEV)
    st["out"] = torch.zeros((n if op in ("dispatch", "combine_grad") else t, h + pad), dtype=dt,
                            device=DEV)
    return st


def _tensors(case):
    """(elements, slot) of each gradient, module by module as a backward pass leaves them."""
    ranks = [int(r) for r in case["ranks"].split()]
    shapes = [tuple(int(v) for v in m.split("x")) for m in case["modules"].split()]
    return [(ranks[s % len(ranks)] * side, s)
            for _ in range(case["layers"]) for sides in shapes for side in sides
            for s in range(case["slots"])]


def _prepare_grads(case, seed):
    g = _gen(seed)
    st, dt, slots = dict(case), _dtype(case), case["slots"]
    tensors = _tensors(case)
    sizes = torch.tensor([n for n, _ in tensors])
    slot = torch.tensor([s for _, s in tensors])
    room = (sizes + ALIGN - 1) // ALIGN
    ends = room.cumsum(0)
    # one pool holds the gradients; block_slot names the slot of each of its blocks
    st["block_slot"] = torch.repeat_interleave(slot, room).to(DEV)
    pool = torch.randn((int(ends[-1]), ALIGN), generator=g, device=DEV)
    size = 10.0 ** (torch.rand(slots, generator=g, device=DEV) * 4 - 5)
    pool *= size[st["block_slot"]][:, None]
    left = sizes - (room - 1) * ALIGN  # elements of a gradient's last block
    pool[(ends - 1).to(DEV)] *= torch.arange(ALIGN, device=DEV)[None, :] < left.to(DEV)[:, None]
    st["pool"] = pool.to(dt)
    st["starts"], st["sizes"], st["slot"] = ((ends - room) * ALIGN).tolist(), sizes.tolist(), \
        slot.tolist()
    st["norms"] = torch.zeros(slots, device=DEV)
    if case["op"] == "clip":
        # limits about where the norms are: some slots are clipped, some are not
        count = torch.zeros(slots, dtype=torch.int64).index_add(0, slot, sizes).to(DEV)
        st["limits"] = size * count.sqrt() * (torch.rand(slots, generator=g, device=DEV) + 0.5)
        st["out"] = torch.zeros_like(st["pool"])
    if own:  # the device list of a step's gradients, made once as their addresses stay
        from routed_lora_delta_amd import rld_grad_norm_workspace_bytes
        from routed_lora_delta_amd.pool import GradList
        base, to, b = st["pool"].data_ptr(), st["out"].data_ptr() if "out" in st else 0, \
            st["pool"].element_size()
        st["list"] = GradList([(base + o * b, to + o * b if to else 0, n, s, dt == torch.bfloat16)
                               for o, n, s in zip(st["starts"], st["sizes"], st["slot"])],
                              slots, DEV)
        st["need"] = rld_grad_norm_workspace_bytes(st["list"].list)
        st["scratch"] = torch.empty(st["need"], dtype=torch.uint8, device=DEV)
    return st


def prepare(case, seed):
    return _prepare_grads(case, seed) if case["op"] in ("norm", "clip") else \
        _prepare_move(case, seed)


# -------------------------------------------------------------- plain forms ----

def _row_of(st):
    """[tokens, top_k]: the row of each choice, -1 where there is none."""
    t, k = st["tokens"], st["top_k"]
    if st["flat"]:
        mine = torch.arange(t * k, device=DEV).view(t, k)
        return torch.where(st["indices"] >= 0, mine, -1)
    return st["places"].view(t, k).long()


def _plain_dispatch(st):
    h, k, to = st["width"], st["top_k"], st["sorted_rows"].long()
    has = to >= 0
    token = torch.div(to.clamp(min=0), k, rounding_mode="floor")
    rows = torch.where(has[:, None], st["x"][:, :h][token], 0)
    # one place more takes what has none
    n = st["tokens"] * k
    places = torch.full((n + 1,), -1, dtype=torch.int32, device=DEV)
    places[torch.where(has, to, n)] = torch.arange(n, dtype=torch.int32, device=DEV)
    return {"rows": rows, "places": places[:n]}


def _plain_combine(st, weighted):
    h, p = st["width"], _row_of(st)
    rows = torch.where((p >= 0)[:, :, None], st["rows"][:, :h][p.clamp(min=0)].float(), 0.0)
    if weighted:
        rows = rows * st["weights"][:, :, None]
    out = rows.sum(1)
    if st["add"]:
        out = out + st["add_rows"][:, :h].float()
    return out.to(_dtype(st))


def _plain_combine_grad(st):
    h, k, p = st["width"], st["top_k"], _row_of(st)
    has, dout = p >= 0, st["dout"][:, :h].float()
    rows = st["rows"][:, :h][p.clamp(min=0)].float()
    dw = torch.where(has, (rows * dout[:, None, :]).sum(2), 0.0)
    if st["flat"]:
        back = torch.where(has.reshape(-1), torch.arange(has.numel(), device=DEV), -1)
    else:
        back = st["sorted_rows"].long()
    at = back.clamp(min=0)
    token = torch.div(at, k, rounding_mode="floor")
    d = st["weights"].reshape(-1)[at][:, None] * dout[token]
    return {"drows": torch.where((back >= 0)[:, None], d, 0.0).to(_dtype(st)), "dweights": dw}


def _plain_norm(st):
    squares = st["pool"].double().square().sum(1)
    mine = st["block_slot"][:, None] == torch.arange(st["slots"], device=DEV)[None, :]
    return torch.where(mine, squares[:, None], 0.0).sum(0).sqrt().float()


def _plain_clip(st):
    norms = _plain_norm(st)
    factor = torch.clamp(st["limits"] / (norms + 1e-6), max=1.0)
    out = st["pool"].float() * factor[st["block_slot"]][:, None]
    return {"norms": norms, "grads": out.to(_dtype(st))}


# --------------------------------------------------------------- own calls ----

def _own(st):
    import routed_lora_delta_amd as R
    op = st["op"]
    if op in ("norm", "clip"):
        R.check(R.rld_grad_norm(st["list"].list, st["norms"], None, st["scratch"], st["need"]),
                "rld_grad_norm")
        if op == "norm":
            return st["norms"]
        R.check(R.rld_grad_clip(st["list"].list, st["norms"], st["limits"]), "rld_grad_clip")
        return {"norms": st["norms"], "grads": st["out"]}
    t, k, h, f32, stride = st["tokens"], st["top_k"], st["width"], st["dtype"] == "fp32", \
        st["width"] + st["pad"]
    by, at = (None, None) if st["flat"] else (st["sorted_rows"], st["places"])
    if op == "dispatch":
        R.check(R.rld_moe_dispatch(st["x"], f32, stride, t, k, h, by, st["out"], stride, at),
                "rld_moe_dispatch")
        return {"rows": st["out"][:, :h], "places": st["places"]}
    if op == "dispatch_grad":
        R.check(R.rld_moe_dispatch_grad(st["rows"], f32, stride, by, at, t, k, h,
                                        st["add_rows"] if st["add"] else None, stride, st["out"],
                                        stride), "rld_moe_dispatch_grad")
        return st["out"][:, :h]
    if op == "combine":
        R.check(R.rld_moe_combine(st["rows"], f32, stride, st["indices"], by, at, st["weights"],
                                  t, k, h, st["add_rows"] if st["add"] else None, stride,
                                  st["out"], stride), "rld_moe_combine")
        return st["out"][:, :h]
    R.check(R.rld_moe_combine_grad(st["rows"], f32, stride, st["indices"], by, at, st["weights"],
                                   st["dout"], stride, t, k, h, st["out"], stride,
                                   st["dweights"]), "rld_moe_combine_grad")
    return {"drows": st["out"][:, :h], "dweights": st["dweights"]}


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op in ("combine", "dispatch_grad"):
        return _plain_combine(state, op == "combine")
    return {"dispatch": _plain_dispatch, "combine_grad": _plain_combine_grad, "norm": _plain_norm,
            "clip": _plain_clip}[op](state)


# ---------------------------------------------------------------- the work ----

def work(case):
    size, op = 2 if case["dtype"] == "bf16" else 4, case["op"]
    if op in ("norm", "clip"):
        n = sum(c for c, _ in _tensors(case))
        return {"bytes": n * size * (1 if op == "norm" else 2), "flops": n * (2 if op == "norm"
                                                                             else 3)}
    t, k, h = case["tokens"], case["top_k"], case["width"]
    live = t - t // 10
    row, tables = h * size, t * k * (4 if case["flat"] else 8)
    if op == "dispatch":
        return {"bytes": live * row * (1 + k) + tables, "flops": 0}
    if op == "combine_grad":
        return {"bytes": live * row * (1 + 2 * k) + tables + 8 * t * k, "flops": 3 * live * k * h}
    out = t * row * (2 if case["add"] else 1)
    if op == "combine":
        return {"bytes": live * row * k + out + tables + 4 * t * k, "flops": 2 * live * k * h}
    return {"bytes": live * row * k + out + tables, "flops": live * k * h}


# ----------------------------------------------------- the values in 64 bits ----

def _exact_sum(st, weighted):
    """Choice by choice: the rows that the tables name, found from indices and sorted_rows."""
    t, k, h = st["tokens"], st["top_k"], st["width"]
    out = st["add_rows"][:, :h].double() if st["add"] else \
        torch.zeros((t, h), dtype=torch.float64, device=DEV)
    for j in range(k):
        token = (st["indices"][:, j] >= 0).nonzero().flatten()
        row = _find(st, token, j)
        part = st["rows"][row][:, :h].double()
        out[token] += part * st["weights"][token, j].double()[:, None] if weighted else part
    return out


def _find(st, token, j):
    """The rows of choice j of these tokens."""
    mine = token * st["top_k"] + j
    if st["flat"]:
        return mine
    known, at = st["sorted_rows"].long().sort()
    return at[torch.searchsorted(known, mine)]


def _exact_combine_grad(st):
    t, k, h = st["tokens"], st["top_k"], st["width"]
    drows = torch.zeros((t * k, h), dtype=torch.float64, device=DEV)
    dw = torch.zeros((t, k), dtype=torch.float64, device=DEV)
    for j in range(k):
        token = (st["indices"][:, j] >= 0).nonzero().flatten()
        row = _find(st, token, j)
        d = st["dout"][token][:, :h].double()
        drows[row] = d * st["weights"][token, j].double()[:, None]
        dw[token, j] = (d * st["rows"][row][:, :h].double()).sum(1)
    return {"drows": drows, "dweights": dw}


def _exact_grads(st):
    flat = st["pool"].reshape(-1)
    squares = [0.0] * st["slots"]
    pieces = list(zip(st["starts"], st["sizes"], st["slot"]))
    for o, n, s in pieces:
        squares[s] = squares[s] + (flat[o:o + n].double() ** 2).sum()
    norms = torch.stack([torch.as_tensor(v, dtype=torch.float64, device=DEV)
                         for v in squares]).sqrt()
    if st["op"] == "norm":
        return norms
    factor = torch.clamp(st["limits"].double() / (norms + 1e-6), max=1.0)
    out = torch.zeros(flat.shape, dtype=torch.float64, device=DEV)
    for o, n, s in pieces:
        out[o:o + n] = flat[o:o + n].double() * factor[s]
    return {"norms": norms, "grads": out.view(st["pool"].shape)}


def _exact_dispatch(st):
    t, k, h = st["tokens"], st["top_k"], st["width"]
    rows = torch.zeros((t * k, h), dtype=torch.float64, device=DEV)
    for j in range(k):
        token = (st["indices"][:, j] >= 0).nonzero().flatten()
        rows[_find(st, token, j)] = st["x"][token][:, :h].double()
    return {"rows": rows, "places": None}


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op == "dispatch":
        return _exact_dispatch(st)
    if op in ("norm", "clip"):
        return _exact_grads(st)
    return _exact_combine_grad(st) if op == "combine_grad" else _exact_sum(st, op == "combine")
