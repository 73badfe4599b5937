"""What is measured of the projection with routed adapters and of the MoE router.

Four operators, each in its plain form (elementary torch operations in 32 bits)
and, where `own` is true, as a call of this library:

  proj         out_i = x_i W^T + scale_s (x_i A_s^T) B_s^T          rld_proj
  proj_grad    its gradient: dx, and dA_s, dB_s of every slot         rld_proj_grad
  router       top-k experts of each token, their weights, counts,
               the expert-sorted rows and the balance loss            rld_moe_router
  router_grad  the gradient of weights and balance loss to the logits rld_moe_router_grad
"""
import math

import torch

own = False

DEV = "cuda"
SCRATCH = 512 << 20  # a serving or training program keeps one scratch buffer for all its calls


# ------------------------------------------------------------------- cases ----

def _proj(name, op, n, k_in, n_out, rank, slots, layout, pad):
    return {"name": name, "op": op, "n": n, "k_in": k_in, "n_out": n_out, "rank": rank,
            "slots": slots, "layout": layout, "pad": pad}


def _route(name, op, tokens, experts, top_k, dtype, norm, disabled):
    return {"name": name, "op": op, "tokens": tokens, "experts": experts, "top_k": top_k,
            "dtype": dtype, "norm": norm, "disabled": disabled}


def listed():
    return [
        # a single request's next token through q or o: latency
        _proj("proj one token", "proj", 1, 4096, 4096, 16, 16, "mixed", 0),
        # the decode batch of the attention workload: 64 requests, each its own adapter
        _proj("proj decode 64", "proj", 64, 4096, 4096, 16, 16, "mixed", 0),
        # the decode batch of the FFN workload: 256 requests through gate or up
        _proj("proj decode 256 ffn", "proj", 256, 4096, 12288, 64, 32, "mixed", 0),
        # packed prompts of several requests through k or v, into an interleaved row
        _proj("proj ragged prompts", "proj", 1237, 4096, 1024, 16, 16, "runs", 64),
        # a prefill batch through gate or up
        _proj("proj prefill ffn", "proj", 4096, 4096, 12288, 64, 8, "runs", 0),
        # a short training micro-batch through k or v
        _proj("grad short batch", "proj_grad", 333, 4096, 1024, 16, 4, "runs", 0),
        # an expert-sized projection, examples of many adapters shuffled in one batch
        _proj("grad shuffled batch", "proj_grad", 2050, 2048, 768, 32, 16, "mixed", 8),
        # a training batch through the FFN's down projection
        _proj("grad ffn down", "proj_grad", 4096, 12288, 4096, 64, 4, "runs", 0),
        # the decode batch of the MoE workload
        _route("router decode 32", "router", 32, 128, 8, "bf16", True, 0),
        # a long packed prefill, two experts taken out of service
        _route("router prefill", "router", 32771, 128, 8, "fp32", True, 2),
        # the training batch of the MoE prefill workload
        _route("router grad 4096", "router_grad", 4096, 128, 8, "bf16", True, 0),
        # a long training batch, weights left as the softmax gave them
        _route("router grad long", "router_grad", 32771, 128, 8, "fp32", False, 0),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["proj", "proj", "proj_grad", "router", "router_grad"])
    if op.startswith("proj"):
        while True:
            if rng.random() < 0.5:  # this repository's projections
                k_in, n_out = rng.choice([(4096, 4096), (4096, 1024), (4096, 12288),
                                          (12288, 4096), (2048, 768), (768, 2048)])
            else:
                k_in, n_out = _log_int(rng, 64, 12288, 8), _log_int(rng, 64, 12288, 8)
            n = _log_int(rng, 1, 4096)
            rank, slots = rng.choice([8, 16, 24, 32, 64, 128]), rng.choice([1, 2, 4, 8, 16, 32])
            if n * k_in * n_out > 4096 * 4096 * 12288 // 2:
                continue
            # gradients of every slot are written: the largest would outweigh the products
            if op == "proj_grad" and slots * rank * (k_in + n_out) > 4 * 64 * 16384:
                continue
            return {"op": op, "n": n, "k_in": k_in, "n_out": n_out, "rank": rank, "slots": slots,
                    "layout": rng.choice(["runs", "mixed"]), "pad": rng.choice([0, 0, 8, 64])}
    experts = rng.choice([8, 60, 64, 128, 160, 256])
    return {"op": op, "tokens": _log_int(rng, 1, 32771 * 128 // max(128, experts)),
            "experts": experts, "top_k": rng.choice([1, 2, 4, 6, 8]),
            "dtype": rng.choice(["bf16", "fp32"]), "norm": rng.choice([True, False]),
            "disabled": rng.choice([0, 0, 0, 1, 3])}


# ------------------------------------------------------------------ inputs ----

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _slots_of(case, g):
    """Slot of each row: -1 is the base model.  "runs": the rows of a request lie
    together; "mixed": every row its own request."""
    n, slots = case["n"], case["slots"]
    if case["layout"] == "mixed":
        s = torch.randint(0, slots, (n,), generator=g, device=DEV)
        base = torch.rand(n, generator=g, device=DEV) < 0.1
        return torch.where(base, -1, s).to(torch.int32)
    runs = max(1, min(2 * slots, n // 32))
    cuts = torch.randint(0, n, (runs - 1,), generator=g, device=DEV).sort().values
    run = torch.searchsorted(cuts, torch.arange(n, device=DEV), right=True)
    s = torch.randint(0, slots, (runs,), generator=g, device=DEV)
    s = torch.where(torch.rand(runs, generator=g, device=DEV) < 0.1, -1, s)
    return s[run].to(torch.int32)


def _prepare_proj(case, seed):
    g = _gen(seed)
    n, k, m, r, s, pad = (case[v] for v in ("n", "k_in", "n_out", "rank", "slots", "pad"))
    st = dict(case)
    st["w"] = _normal(g, (m, k), 1.0 / math.sqrt(k))
    st["x_rows"] = _normal(g, (n, k + pad))
    st["x"] = st["x_rows"][:, :k]
    # true ranks below the padded one leave zero rows of A and zero columns of B
    ranks = torch.randint(max(1, r // 2), r + 1, (s,), generator=g, device=DEV)
    inside = torch.arange(r, device=DEV)[None, :] < ranks[:, None]
    a = (torch.rand((s, r, k), generator=g, device=DEV) * 2 - 1) / math.sqrt(k)
    b = torch.randn((s, m, r), generator=g, device=DEV) * 0.02
    st["a"] = (a * inside[:, :, None]).to(torch.bfloat16)
    st["b"] = (b * inside[:, None, :]).to(torch.bfloat16)
    st["scale"] = 16.0 / ranks.float()
    st["slot"] = _slots_of(case, g)
    # with eight slots or more the last one does not adapt this module
    st["adapted"] = torch.arange(s, device=DEV) < (s - 1 if s >= 8 else s)
    at = torch.arange(s, device=DEV)
    st["a_table"] = torch.where(st["adapted"], st["a"].data_ptr() + at * (r * k * 2), 0)
    st["b_table"] = torch.where(st["adapted"], st["b"].data_ptr() + at * (m * r * 2), 0)
    st["scratch"] = torch.empty(SCRATCH, dtype=torch.uint8, device=DEV)
    if case["op"] == "proj":
        st["out_rows"] = torch.zeros((n, m + pad), dtype=torch.bfloat16, device=DEV)
        return st
    st["dy_rows"] = _normal(g, (n, m + pad))
    st["dy"] = st["dy_rows"][:, :m]
    st["dx_rows"] = torch.zeros((n, k + pad), dtype=torch.bfloat16, device=DEV)
    st["da"] = torch.zeros((s, r, k), device=DEV)
    st["db"] = torch.zeros((s, m, r), device=DEV)
    st["da_table"] = st["da"].data_ptr() + at * (r * k * 4)
    st["db_table"] = st["db"].data_ptr() + at * (m * r * 4)
    return st


def _prepare_router(case, seed):
    g = _gen(seed)
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    st = dict(case)
    # some experts are preferred over others, as a trained router's are
    logits = torch.randn((t, e), generator=g, device=DEV)
    logits += 0.5 * torch.randn((1, e), generator=g, device=DEV)
    off = torch.randperm(e, generator=g, device=DEV)[:case["disabled"]]
    logits[:, off] = -math.inf
    st["logits"] = logits.to(dtype)
    # the batch is padded: about one token in ten is none
    st["mask"] = (torch.rand(t, generator=g, device=DEV) >= 0.1).to(torch.int32)
    i32 = {"dtype": torch.int32, "device": DEV}
    st["scratch"] = torch.empty(SCRATCH, dtype=torch.uint8, device=DEV)
    if case["op"] == "router":
        st["indices"] = torch.zeros((t, k), **i32)
        st["weights"] = torch.zeros((t, k), device=DEV)
        st["counts"] = torch.zeros(e + 1, **i32)
        st["offsets"] = torch.zeros(e + 1, **i32)
        st["tokens_sorted"] = torch.zeros(t * k, **i32)
        st["positions"] = torch.zeros(t * k, **i32)
        st["loss"] = torch.zeros(1, device=DEV)
        return st
    f = _plain_router(st)
    st["indices"], st["counts"] = f["indices"], f["counts"]
    st["dweights"] = torch.randn((t, k), generator=g, device=DEV) / t
    st["dloss"] = torch.rand(1, generator=g, device=DEV) + 0.5
    st["dlogits"] = torch.zeros((t, e), dtype=dtype, device=DEV)
    return st


def prepare(case, seed):
    return _prepare_proj(case, seed) if case["op"].startswith("proj") else \
        _prepare_router(case, seed)


# -------------------------------------------------------------- plain forms ----

def _own_columns(st, wide):
    """[n, slots, rank] of a product with every slot's matrix: the row's own slot kept."""
    s, r = st["slots"], st["rank"]
    mine = st["slot"][:, None] == torch.arange(s, device=DEV)[None, :]
    mine = mine & st["adapted"][None, :]
    kept = torch.where(mine[:, :, None], wide.view(-1, s, r), 0.0)
    return (kept * st["scale"][None, :, None]).reshape(-1, s * r)


def _plain_proj(st):
    x = st["x"].float()
    a = st["a"].float().reshape(-1, st["k_in"])
    b = st["b"].float().permute(0, 2, 1).reshape(-1, st["n_out"])
    y = x @ st["w"].float().T
    return (y + _own_columns(st, x @ a.T) @ b).to(torch.bfloat16)


def _plain_proj_grad(st):
    s, r, k, m = st["slots"], st["rank"], st["k_in"], st["n_out"]
    x, dy = st["x"].float(), st["dy"].float()
    a = st["a"].float().reshape(-1, k)
    b = st["b"].float().permute(0, 2, 1).reshape(-1, m)
    xa = _own_columns(st, x @ a.T)
    g = _own_columns(st, dy @ b.T)
    dx = (dy @ st["w"].float() + g @ a).to(torch.bfloat16)
    da = (g.T @ x).view(s, r, k)
    db = (xa.T @ dy).view(s, r, m).permute(0, 2, 1).contiguous()
    return {"dx": dx, "da": da, "db": db}


def _probabilities(st):
    l = st["logits"].float()
    live = (st["mask"] != 0) & (l.amax(1) > -math.inf)
    top = torch.where(live, l.amax(1), 0.0)
    e = torch.exp(l - top[:, None])
    p = torch.where(live[:, None], e / e.sum(1, keepdim=True), 0.0)
    return l, live, p


def _plain_router(st):
    t, e, k = st["tokens"], st["experts"], st["top_k"]
    l, live, p = _probabilities(st)
    order = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :k]
    chosen = live[:, None] & (l.gather(1, order) > -math.inf)
    indices = torch.where(chosen, order, -1)
    w = torch.where(chosen, p.gather(1, order), 0.0)
    if st["norm"]:
        w = w / torch.where(live, w.sum(1), 1.0)[:, None]
    flat = torch.where(chosen, order, e).reshape(-1)
    counts = torch.bincount(flat, minlength=e + 1)[:e]
    rows = torch.arange(t * k, device=DEV)
    by_expert = torch.sort(flat, stable=True).indices
    positions = torch.where(rows < counts.sum(), by_expert, -1)
    tokens = torch.div(positions, k, rounding_mode="floor")
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    n = live.sum()
    loss = (p.double().sum(0) * counts).sum() * (e / k) / torch.clamp(n, min=1).double() ** 2
    i32 = torch.int32
    return {"indices": indices.to(i32), "weights": w,
            "counts": torch.cat([counts, n[None]]).to(i32), "offsets": offsets.to(i32),
            "tokens": tokens.to(i32), "positions": positions.to(i32),
            "loss": loss.float()[None]}


def _plain_router_grad(st):
    e, k = st["experts"], st["top_k"]
    _, live, p = _probabilities(st)
    n = torch.clamp(st["counts"][e], min=1).double()
    g = (st["dloss"].double() * (e / k) / n ** 2 * st["counts"][:e]).float()[None, :]
    d = p * (g - (p * g).sum(1, keepdim=True))
    at = torch.clamp(st["indices"], min=0).long()
    chosen = st["indices"] >= 0
    w = torch.where(chosen, p.gather(1, at), 0.0)
    dw = torch.where(chosen, st["dweights"], 0.0)
    if st["norm"]:
        w = w / torch.where(live, w.sum(1), 1.0)[:, None]
        d = d.scatter_add(1, at, w * (dw - (w * dw).sum(1, keepdim=True)))
    else:
        d = d.scatter_add(1, at, w * dw) - p * (w * dw).sum(1, keepdim=True)
    return d.to(st["logits"].dtype)


# --------------------------------------------------------------- own calls ----

def _own(st):
    import routed_lora_delta_amd as R
    op = st["op"]
    if op.startswith("proj"):
        route = R.rld_route(st["a_table"].data_ptr(), st["b_table"].data_ptr(),
                            st["scale"].data_ptr(), st["slots"], st["k_in"], st["n_out"],
                            st["rank"])
        k, m, pad, n = st["k_in"], st["n_out"], st["pad"], st["n"]
    if op == "proj":
        R.check(R.rld_proj(route, st["w"], k, st["x_rows"], k + pad, st["slot"], n,
                           st["out_rows"], m + pad, st["scratch"], SCRATCH), "rld_proj")
        return st["out_rows"][:, :m]
    if op == "proj_grad":
        R.check(R.rld_proj_grad(route, st["w"], k, st["x_rows"], k + pad, st["dy_rows"], m + pad,
                                st["slot"], n, st["dx_rows"], k + pad, st["da_table"],
                                st["db_table"], False, st["scratch"], SCRATCH), "rld_proj_grad")
        return {"dx": st["dx_rows"][:, :k], "da": st["da"], "db": st["db"]}
    t, e, k = st["tokens"], st["experts"], st["top_k"]
    f32 = st["dtype"] == "fp32"
    if op == "router":
        R.check(R.rld_moe_router(st["logits"], f32, e, st["mask"], t, e, k, st["norm"],
                                 st["indices"], st["weights"], st["counts"], st["offsets"],
                                 st["tokens_sorted"], st["positions"], st["loss"],
                                 st["scratch"], SCRATCH), "rld_moe_router")
        return {"indices": st["indices"], "weights": st["weights"], "counts": st["counts"],
                "offsets": st["offsets"], "tokens": st["tokens_sorted"],
                "positions": st["positions"], "loss": st["loss"]}
    R.check(R.rld_moe_router_grad(st["logits"], f32, e, st["mask"], t, e, k, st["norm"],
                                  st["indices"], st["counts"], st["dweights"], st["dloss"],
                                  st["dlogits"], e), "rld_moe_router_grad")
    return st["dlogits"]


def run(state):
    if own:
        return _own(state)
    return {"proj": _plain_proj, "proj_grad": _plain_proj_grad, "router": _plain_router,
            "router_grad": _plain_router_grad}[state["op"]](state)


# ---------------------------------------------------------------- the work ----

def work(case):
    if case["op"].startswith("proj"):
        n, k, m, r = case["n"], case["k_in"], case["n_out"], case["rank"]
        used = min(case["slots"], n)
        adapters = used * r * (k + m) * 2
        if case["op"] == "proj":
            return {"bytes": 2 * (m * k + n * k + n * m) + adapters + 4 * n,
                    "flops": 2 * n * k * m + 2 * n * r * (k + m)}
        grads = case["slots"] * r * (k + m) * 4
        return {"bytes": 2 * (m * k + 2 * n * k + n * m) + adapters + grads + 4 * n,
                "flops": 2 * n * k * m + 6 * n * r * (k + m)}
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "router":
        return {"bytes": t * e * size + t * 4 + t * k * 16 + e * 8, "flops": 6 * t * e}
    return {"bytes": 2 * t * e * size + t * 4 + t * k * 8 + e * 4, "flops": 8 * t * e}


# ----------------------------------------------------- the values in 64 bits ----

def _exact_proj(st):
    x, w = st["x"].double(), st["w"].double()
    y = x @ w.T
    for s in range(st["slots"]):
        rows = (st["slot"] == s).nonzero().flatten()
        if rows.numel() and bool(st["adapted"][s]):
            low = x[rows] @ st["a"][s].double().T
            y[rows] += st["scale"][s].double() * (low @ st["b"][s].double().T)
    return y


def _exact_proj_grad(st):
    x, dy, w = st["x"].double(), st["dy"].double(), st["w"].double()
    dx, da, db = dy @ w, st["a"].double() * 0, st["b"].double() * 0
    for s in range(st["slots"]):
        rows = (st["slot"] == s).nonzero().flatten()
        if rows.numel() and bool(st["adapted"][s]):
            a, b, c = st["a"][s].double(), st["b"][s].double(), st["scale"][s].double()
            xs, ys = x[rows], dy[rows]
            dlow = c * (ys @ b)
            dx[rows] += dlow @ a
            da[s] = dlow.T @ xs
            db[s] = c * (ys.T @ (xs @ a.T))
    return {"dx": dx, "da": da, "db": db}


def _exact_router(st):
    l = st["logits"].double()
    t, e, k = st["tokens"], st["experts"], st["top_k"]
    live = (st["mask"] != 0) & ~(l == -math.inf).all(1)
    rows = live.nonzero().flatten()
    weights = torch.zeros((t, k), dtype=torch.float64, device=DEV)
    counts = torch.zeros(e, dtype=torch.float64, device=DEV)
    p = torch.softmax(l[rows], 1)
    left = p.clone()
    left[l[rows] == -math.inf] = -1.0
    for j in range(min(k, e)):
        best, at = left.max(1)
        ok = best >= 0
        # equal values: the lowest index
        at = (left == best[:, None]).to(torch.int8).argmax(1)
        weights[rows, j] = torch.where(ok, best, 0.0)
        counts += torch.bincount(at[ok], minlength=e)
        left[torch.arange(len(rows), device=DEV), at] = -1.0
    if st["norm"]:
        weights[rows] /= weights[rows].sum(1, keepdim=True)
    n = max(1, len(rows))
    loss = e * ((counts / (n * k)) * (p.sum(0) / n)).sum()
    return {"indices": None, "weights": weights, "counts": None, "offsets": None,
            "tokens": None, "positions": None, "loss": loss[None]}


def _exact_router_grad(st):
    l = st["logits"].double()
    e, k = st["experts"], st["top_k"]
    rows = ((st["mask"] != 0) & ~(l == -math.inf).all(1)).nonzero().flatten()
    d = torch.zeros_like(l)
    p = torch.softmax(l[rows], 1)
    n = max(1, len(rows))
    g = st["dloss"].double() * e * (st["counts"][:e].double() / (n * k)) / n
    g = g[None, :].repeat(len(rows), 1)
    index, dw = st["indices"][rows].long(), st["dweights"][rows].double()
    if not st["norm"]:
        for j in range(k):
            r = (index[:, j] >= 0).nonzero().flatten()
            g[r, index[r, j]] += dw[r, j]
    d[rows] = p * g - p * (p * g).sum(1, keepdim=True)
    if st["norm"]:
        picked = torch.zeros_like(p)
        dpicked = torch.zeros_like(p)
        for j in range(k):
            r = (index[:, j] >= 0).nonzero().flatten()
            picked[r, index[r, j]] = p[r, index[r, j]]
            dpicked[r, index[r, j]] = dw[r, j]
        q = picked / picked.sum(1, keepdim=True)
        d[rows] += q * dpicked - q * (q * dpicked).sum(1, keepdim=True)
    return d


def exact(case, seed):
    st = prepare(case, seed)
    return {"proj": _exact_proj, "proj_grad": _exact_proj_grad, "router": _exact_router,
            "router_grad": _exact_router_grad}[case["op"]](st)
