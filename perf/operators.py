"""Cases of the mixture-of-experts operators: routing, sorting slots by expert,
carrying token rows to their experts and back, with the gradients.

T tokens choose k of E experts each; slot s = t * k + j is choice j of token t.
The operators are

  route    top-k experts of each row of router logits, with their weights
  sort     slots sorted stably by expert: order, position (the inverse) and
           per-expert offsets
  dispatch rows[position[t, j]] = x[t], optionally times weights[t, j]
  combine  out[t] = sum over j of weights[t, j] * rows[position[t, j]]

and the gradients of route, dispatch and combine.
"""
import math

import numpy as np
import torch

own = False

_DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2}


def _case(name, op, T, k, E=0, H=0, dtype="bf16", mode="softmax", renorm=False, weighted=True, pad=0.0, shard=1):
    c = {"op": op, "T": T, "k": k, "E": E, "H": H, "dtype": dtype, "mode": mode, "renorm": renorm,
         "weighted": weighted, "pad": pad, "shard": shard}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # The router of one decoded token: pure latency.
        _case("route_token", "route", 1, 6, E=64, dtype="bf16"),
        # A prefill batch over many experts, sigmoid gates made to sum to one.
        _case("route_prefill", "route", 16384, 8, E=256, dtype="f32", mode="sigmoid", renorm=True),
        # Training step of a router with an odd expert count and a plain softmax.
        _case("route_grad", "route_bwd", 8191, 4, E=60, dtype="f32"),
        # A decode batch of 32 tokens: a few hundred slots.
        _case("sort_decode", "sort", 32, 8, E=128),
        # A long-context prefill: a million slots, a padded tail, half of the
        # experts on another rank.
        _case("sort_prefill", "sort", 131072, 8, E=256, pad=0.03, shard=2),
        # A decode batch's rows to their experts.
        _case("dispatch_decode", "dispatch", 24, 4, E=32, H=2880, weighted=False),
        # A training batch, odd row width in 16-bit floats, weights on the way in.
        _case("dispatch_odd", "dispatch", 8191, 2, E=8, H=1537, dtype="f16"),
        # The gradient of a padded training batch's dispatch.
        _case("dispatch_grad", "dispatch_bwd", 16384, 6, E=64, H=2048, weighted=False, pad=0.05),
        # One token's expert outputs joined: pure latency.
        _case("combine_token", "combine", 1, 8, E=256, H=7168),
        # A prefill batch joined: the largest forward.
        _case("combine_prefill", "combine", 16384, 8, E=128, H=4096),
        # The gradient of a joined training batch, with that of the weights.
        _case("combine_grad", "combine_bwd", 8192, 8, E=128, H=2048),
        # Full-precision training with an odd width and padded rows.
        _case("combine_grad_f32", "combine_bwd", 4093, 2, E=16, H=4099, dtype="f32", pad=0.1),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route_bwd", "sort", "dispatch", "dispatch_bwd", "combine", "combine_bwd"])
    E = _log(rng, 8, 512)
    k = min(E, rng.choice([1, 2, 3, 4, 6, 8, 8, 10]))
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    pad = rng.choice([0.0, 0.0, rng.uniform(0.0, 0.3)])
    if op in ("route", "route_bwd"):
        T = _log(rng, 1, 32768)
        T = max(1, min(T, (1 << 23) // E))
        return _case(None, op, T, k, E=E, dtype=dtype, mode=rng.choice(["softmax", "sigmoid"]),
                     renorm=rng.random() < 0.5)
    if op == "sort":
        return _case(None, op, _log(rng, 1, 131072 * 8 // k), k, E=E, pad=pad, shard=rng.choice([1, 1, 2, 4]))
    H = _log(rng, 128, 8192)
    if rng.random() < 0.6:
        H = (H + 63) // 64 * 64
    T = _log(rng, 1, 16384)
    T = max(1, min(T, (1 << 29) // (H * k * _BYTES[dtype])))
    return _case(None, op, T, k, E=E, H=H, dtype=dtype, weighted=rng.random() < 0.6, pad=pad)


def work(case):
    T, k, E, H, b = case["T"], case["k"], case["E"], case["H"], _BYTES[case["dtype"]]
    M = T * k
    op = case["op"]
    if op == "route":
        return {"bytes": T * E * b + M * 8, "flops": T * E * 4}
    if op == "route_bwd":
        return {"bytes": 2 * T * E * b + M * 8, "flops": T * E * 8}
    if op == "sort":
        return {"bytes": 4 * M + 8 * M + 4 * (_local(case) + 1), "flops": 0}
    used = _used_tokens(case)      # padded tokens' rows: nothing to read
    w = 4 * M if case["weighted"] else 0
    if op == "dispatch":
        return {"bytes": used * H * b + M * H * b + 4 * M + w, "flops": used * k * H}
    if op == "dispatch_bwd":
        extra = used * H * b + w if case["weighted"] else 0      # x read, the weights' gradient written
        return {"bytes": used * k * H * b + T * H * b + 4 * M + w + extra, "flops": 2 * used * k * H}
    if op == "combine":
        return {"bytes": used * k * H * b + T * H * b + 4 * M + w, "flops": 2 * used * k * H}
    extra = used * k * H * b + w if case["weighted"] else 0      # rows read, the weights' gradient written
    return {"bytes": used * H * b + M * H * b + 4 * M + w + extra, "flops": 3 * used * k * H}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _local(case):
    """Experts that this rank holds."""
    return max(1, case["E"] // case["shard"])


def _first(case):
    """The first of them: the last rank's share."""
    return case["E"] - _local(case)


def _used_tokens(case):
    return case["T"] - int(case["T"] * case["pad"])


def _logits(case, gen):
    """Router logits: some experts are liked by every token."""
    T, E = case["T"], case["E"]
    liking = torch.randn(E, generator=gen, device="cuda") * 0.7
    return (torch.randn(T, E, generator=gen, device="cuda") * 1.5 + liking).to(_DTYPES[case["dtype"]])


def _ids(case, gen):
    """Distinct experts of each token, popular ones more often; -1 in padding."""
    T, E, k = case["T"], case["E"], case["k"]
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    liking = torch.randn(E, generator=gen, device="cuda") * 0.5
    for a in range(0, T, 16384):
        b = min(T, a + 16384)
        score = torch.randn(b - a, E, generator=gen, device="cuda") + liking
        ids[a:b] = torch.topk(score, k, dim=1).indices.to(torch.int32)
    ids[_used_tokens(case):] = -1
    return ids


def _sorted_plain(ids, first, count):
    """order, position, offsets of slots sorted stably by expert."""
    flat = ids.reshape(-1).long() - first
    key = torch.where((flat >= 0) & (flat < count), flat, torch.full_like(flat, count))
    order = torch.argsort(key, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=order.device)
    position = torch.where(key < count, place, -1 - place).to(torch.int32).reshape(ids.shape)
    counts = torch.zeros(count + 1, dtype=torch.int64, device=ids.device)
    counts.index_add_(0, key, torch.ones_like(key))
    offsets = torch.zeros(count + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = torch.cumsum(counts[:count], 0).to(torch.int32)
    return order.to(torch.int32), position, offsets


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    T, k, H, op = case["T"], case["k"], case["H"], case["op"]
    dt = _DTYPES[case["dtype"]]
    st = {"case": case}
    if op in ("route", "route_bwd"):
        st["logits"] = _logits(case, gen)
        if op == "route_bwd":
            st["experts"] = _chosen(st["logits"], k)
            st["grad_weights"] = torch.randn(T, k, generator=gen, device="cuda")
        return st
    st["ids"] = _ids(case, gen)
    if op == "sort":
        return st
    # What follows the sort: every slot's place, and its weight.
    _, st["position"], _ = _sorted_plain(st["ids"], 0, case["E"])
    st["weights"] = None
    if case["weighted"]:
        w = torch.rand(T, k, generator=gen, device="cuda") + 0.05
        st["weights"] = w / w.sum(1, keepdim=True)
    if op in ("dispatch", "dispatch_bwd"):
        st["x"] = torch.randn(T, H, generator=gen, device="cuda").to(dt)
    if op == "dispatch_bwd":
        st["grad_rows"] = torch.randn(T * k, H, generator=gen, device="cuda", dtype=dt)
    if op in ("combine", "combine_bwd"):
        st["rows"] = torch.randn(T * k, H, generator=gen, device="cuda", dtype=dt)
    if op == "combine_bwd":
        st["grad_out"] = torch.randn(T, H, generator=gen, device="cuda").to(dt)
    return st


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
def _chosen(logits, k):
    """The k largest of each row, ties to the lowest index."""
    return torch.argsort(logits.float(), dim=1, descending=True, stable=True)[:, :k].to(torch.int32)


def _probabilities(logits, mode):
    l = logits.float()
    if mode == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    e = torch.exp(l - l.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_route(st):
    c = st["case"]
    experts = _chosen(st["logits"], c["k"])
    p = _probabilities(st["logits"], c["mode"]).gather(1, experts.long())
    if c["renorm"]:
        p = p / p.sum(1, keepdim=True)
    return p, experts


def _plain_route_bwd(st):
    c = st["case"]
    logits, g, at = st["logits"], st["grad_weights"], st["experts"].long()
    p = _probabilities(logits, c["mode"])
    chosen = p.gather(1, at)
    grad = torch.zeros_like(p)
    if c["renorm"]:
        u = chosen / chosen.sum(1, keepdim=True)
        d = u * (g - (g * u).sum(1, keepdim=True))
        if c["mode"] == "sigmoid":
            d = d * (1.0 / (1.0 + torch.exp(logits.float().gather(1, at))))
        grad.scatter_add_(1, at, d)
    elif c["mode"] == "sigmoid":
        grad.scatter_add_(1, at, g * chosen * (1.0 / (1.0 + torch.exp(logits.float().gather(1, at)))))
    else:
        grad.scatter_add_(1, at, g)
        grad = p * (grad - (g * chosen).sum(1, keepdim=True))
    return grad.to(logits.dtype)


def _place(position):
    """Each slot's row, and whether the slot is in use."""
    p = position.long()
    return torch.where(p >= 0, p, -1 - p), p >= 0


def _plain_spread(x, position, weights):
    """rows[place of (t, j)] = w[t, j] * x[t], zero for unused slots."""
    T, k = position.shape
    place, used = _place(position)
    rows = torch.empty(T * k, x.shape[1], dtype=x.dtype, device=x.device)
    f = x.float()
    for j in range(k):
        v = f if weights is None else f * weights[:, j, None]
        rows[place[:, j]] = torch.where(used[:, j, None], v, torch.zeros_like(v)).to(x.dtype)
    return rows


def _plain_join(rows, position, weights):
    """out[t] = sum over used j of w[t, j] * rows[place of (t, j)]."""
    T, k = position.shape
    place, used = _place(position)
    out = torch.zeros(T, rows.shape[1], dtype=torch.float32, device=rows.device)
    for j in range(k):
        v = rows[place[:, j]].float()
        if weights is not None:
            v = v * weights[:, j, None]
        out += torch.where(used[:, j, None], v, torch.zeros_like(v))
    return out.to(rows.dtype)


def _plain_dots(x, rows, position):
    """<x[t], rows[place of (t, j)]>, zero for unused slots."""
    T, k = position.shape
    place, used = _place(position)
    dots = torch.empty(T, k, dtype=torch.float32, device=x.device)
    f = x.float()
    for j in range(k):
        dots[:, j] = (f * rows[place[:, j]].float()).sum(1)
    return torch.where(used, dots, torch.zeros_like(dots))


def _plain(st):
    op = st["case"]["op"]
    if op == "route":
        return _plain_route(st)
    if op == "route_bwd":
        return _plain_route_bwd(st)
    if op == "sort":
        return _sorted_plain(st["ids"], _first(st["case"]), _local(st["case"]))
    position, w = st["position"], st["weights"]
    if op == "dispatch":
        return _plain_spread(st["x"], position, w)
    if op == "combine":
        return _plain_join(st["rows"], position, w)
    if op == "dispatch_bwd":
        grad_x = _plain_join(st["grad_rows"], position, w)
        return grad_x if w is None else (grad_x, _plain_dots(st["x"], st["grad_rows"], position))
    grad_rows = _plain_spread(st["grad_out"], position, w)
    return grad_rows if w is None else (grad_rows, _plain_dots(st["grad_out"], st["rows"], position))


# ---------------------------------------------------------------------------
# The framework's operators
# ---------------------------------------------------------------------------
def _own(st):
    import lsd_radix_sort_pass_amd as rs

    c = st["case"]
    op = c["op"]
    if op == "route":
        return rs.route_topk(st["logits"], c["k"], mode=c["mode"], renormalize=c["renorm"])
    if op == "route_bwd":
        return rs.route_topk_backward(st["logits"], st["experts"], st["grad_weights"], mode=c["mode"],
                                      renormalize=c["renorm"])
    if op == "sort":
        return rs.sort_experts(st["ids"], _local(c), first_expert=_first(c))
    if op == "dispatch":
        return rs.dispatch_rows(st["x"], st["position"], st["weights"])
    if op == "combine":
        return rs.combine_rows(st["rows"], st["position"], st["weights"])
    if op == "dispatch_bwd":
        if st["weights"] is None:
            return rs.dispatch_rows_backward(st["grad_rows"], st["position"])
        return rs.dispatch_rows_backward(st["grad_rows"], st["position"], st["x"], st["weights"])
    if st["weights"] is None:
        return rs.combine_rows_backward(st["grad_out"], st["position"])
    return rs.combine_rows_backward(st["grad_out"], st["position"], st["rows"], st["weights"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_choice(l, k):
    """k rounds of taking the row's largest value, at its lowest index."""
    left = l.clone()
    index = torch.arange(l.shape[1], device=l.device).expand_as(l)
    chosen = torch.empty(l.shape[0], k, dtype=torch.int64, device=l.device)
    for j in range(k):
        top = left.amax(1, keepdim=True)
        at = torch.where(left == top, index, torch.full_like(index, l.shape[1])).amin(1)
        chosen[:, j] = at
        left.scatter_(1, at[:, None], -math.inf)
    return chosen


def _exact_route(case, st):
    l = st["logits"].double()
    k = case["k"]
    at = st["experts"].long() if case["op"] == "route_bwd" else _exact_choice(l, k)
    top = torch.gather(l, 1, at)
    if case["mode"] == "softmax":
        total = top if case["renorm"] else l
        w = torch.exp(top - torch.logsumexp(total, 1, keepdim=True))
    else:
        w = torch.sigmoid(top)
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
    if case["op"] == "route":
        return w.cpu(), at.to(torch.int32).cpu()
    # d w_j / d l_i, summed against the incoming gradient.
    g = st["grad_weights"].double()
    grad = torch.zeros_like(l)
    mean = (g * w).sum(1, keepdim=True)
    if case["mode"] == "softmax":
        grad.scatter_add_(1, at, g * w)
        if case["renorm"]:
            grad.scatter_add_(1, at, -w * mean)
        else:
            grad -= mean * torch.exp(l - torch.logsumexp(l, 1, keepdim=True))
    else:
        inner = g - mean if case["renorm"] else g
        grad.scatter_add_(1, at, w * torch.sigmoid(-top) * inner)
    return grad.cpu()


def _exact_sort(case, st):
    ids = st["ids"].cpu().numpy().astype(np.int64).ravel() - _first(case)
    n, E = ids.size, _local(case)
    key = np.where((ids < 0) | (ids >= E), E, ids)
    order = np.lexsort((np.arange(n), key))
    position = np.zeros(n, dtype=np.int64)
    position[order] = np.arange(n)
    position[key == E] = ~position[key == E]
    offsets = np.searchsorted(key[order], np.arange(E + 1), side="left")
    return (torch.from_numpy(order.astype(np.int32)),
            torch.from_numpy(position.astype(np.int32).reshape(tuple(st["ids"].shape))),
            torch.from_numpy(offsets.astype(np.int32)))


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("route", "route_bwd"):
        return _exact_route(case, st)
    if op == "sort":
        return _exact_sort(case, st)
    # By rows: row p belongs to slot slot[p] (token slot[p] // k), or to none.
    T, k, H = case["T"], case["k"], case["H"]
    flat = st["position"].cpu().numpy().ravel()
    slot = np.empty(T * k, dtype=np.int64)
    used = np.empty(T * k, dtype=bool)
    at = np.where(flat < 0, ~flat, flat)
    slot[at] = np.arange(T * k)
    used[at] = flat >= 0
    slot = torch.from_numpy(slot).cuda()
    token = slot // k
    scale = torch.from_numpy(used.astype(np.float64)).cuda()
    if st["weights"] is not None:
        scale = scale * st["weights"].double().reshape(-1)[slot]
    live = torch.from_numpy(used).cuda().double()
    block = max(1, (1 << 26) // H)
    spread = op in ("dispatch", "combine_bwd")
    by_token = st.get("grad_out", st.get("x"))
    by_row = st.get("grad_rows", st.get("rows"))
    result = torch.empty(T * k, H, dtype=torch.float64) if spread else torch.zeros(T, H, dtype=torch.float64, device="cuda")
    dots = None
    if op.endswith("_bwd") and st["weights"] is not None:
        dots = torch.zeros(T * k, dtype=torch.float64, device="cuda")
    for a in range(0, T * k, block):
        z = slice(a, min(T * k, a + block))
        if spread:
            result[z] = (by_token[token[z]].double() * scale[z, None]).cpu()
        else:
            result.index_add_(0, token[z], by_row[z].double() * scale[z, None])
        if dots is not None:
            dots[slot[z]] = (by_token[token[z]].double() * by_row[z].double()).sum(1) * live[z]
    result = result.cpu()
    return result if dots is None else (result, dots.reshape(T, k).cpu())
