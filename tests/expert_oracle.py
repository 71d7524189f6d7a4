"""Plain 64-bit definitions of the mixture-of-experts calls (numpy, one loop a
formula), and the bounds on the rounding of float32 evaluations of them."""
import numpy as np

U32 = 2.0 ** -24                                   # half a step of float32, relative
HALF_STEP = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
# Half the smallest positive number (results below the normal range round by it).
TINY = {"float32": 2.0 ** -150, "float16": 2.0 ** -25, "bfloat16": 2.0 ** -134}


def choose(logits, k):
    """k largest of each row, ties to the lowest index, NaN first, -inf never
    (-1)."""
    T, E = logits.shape
    out = np.full((T, k), -1, dtype=np.int64)
    for t in range(T):
        row = logits[t]
        allowed = [i for i in range(E) if not row[i] == -np.inf]
        allowed.sort(key=lambda i: (0 if np.isnan(row[i]) else 1, 0.0 if np.isnan(row[i]) else -row[i], i))
        out[t, :min(k, len(allowed))] = allowed[:k]
    return out


def _gates(row, mode):
    if mode == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-row))
    top = np.max(row)
    if top == -np.inf:
        return np.zeros_like(row)
    with np.errstate(invalid="ignore"):
        e = np.exp(row - top)
    return e / e.sum()


def _chosen_gates(row, at, mode, renorm):
    """Gate values of the experts `at` of a row (no -1 among them)."""
    if not renorm:
        return _gates(row, mode)[at]
    top = np.max(row[at])
    if mode == "softmax":
        with np.errstate(invalid="ignore"):
            e = np.exp(row[at] - top)
    else:
        low = min(top, 0.0)
        e = np.exp(np.minimum(row[at], 0.0) - low) / (1.0 + np.exp(-np.abs(row[at])))
    return e / e.sum()


def route(logits, k, mode, renorm, scale=1.0):
    logits = logits.astype(np.float64)
    at = choose(logits, k)
    w = np.zeros(at.shape)
    for t in range(at.shape[0]):
        m = at[t] >= 0
        if m.any():
            w[t, m] = scale * _chosen_gates(logits[t], at[t, m], mode, renorm)
    return w, at


def route_spread(logits, at):
    """How far below the maximum the chosen logits of a row lie, plus the mean
    of that over the row: each logit's difference from the maximum is rounded
    once, which moves its exponential by that difference in half steps."""
    out = np.zeros(logits.shape[0])
    for t in range(logits.shape[0]):
        row = logits[t].astype(np.float64)
        row = row[np.isfinite(row)]
        if row.size:
            p = np.exp(row - row.max())
            p /= p.sum()
            got = logits[t].astype(np.float64)[at[t][at[t] >= 0]]
            got = got[np.isfinite(got)]
            out[t] = (row.max() - (got.min() if got.size else row.max())) + (p * (row.max() - row)).sum()
    return out


def route_relative(logits, at):
    """Relative bound on a gate value: the spread above, two exponentials (2
    half steps each), a sum over lanes that hold at most E / 16 values, joined
    in at most 6 steps, two divisions, the scale, and a product."""
    E = logits.shape[1]
    return U32 * (route_spread(logits, at) + E / 16 + 24)


def route_backward(logits, at, g, mode, renorm, scale=1.0):
    """(gradient, bound on a float32 evaluation before its last rounding)."""
    logits = logits.astype(np.float64)
    T, E = logits.shape
    k = at.shape[1]
    grad, bound = np.zeros((T, E)), np.zeros((T, E))
    rel = route_relative(logits, np.where((at >= 0) & (at < E), at, -1))
    for t in range(T):
        use = [j for j in range(k) if 0 <= at[t, j] < E and logits[t, at[t, j]] != -np.inf]
        if not use:
            continue
        s, h = at[t, use], g[t, use].astype(np.float64)
        p = _gates(logits[t], mode)
        a, size = np.zeros(E), np.zeros(E)
        np.add.at(a, s, h)
        np.add.at(size, s, np.abs(h))
        r = rel[t] + (k + 8) * U32
        if not renorm and mode == "softmax":
            mean, weight = (h * p[s]).sum(), (np.abs(h) * p[s]).sum()
            grad[t] = scale * p * (a - mean)
            bound[t] = abs(scale) * p * 2 * r * (size + weight)
        elif not renorm:
            d = p * _gates(-logits[t], mode)
            grad[t], bound[t] = scale * a * d, abs(scale) * size * d * r
        else:
            u = _chosen_gates(logits[t], s, mode, True)
            mean, weight = (h * u).sum(), (np.abs(h) * u).sum()
            rest = _gates(-logits[t], mode)[s] if mode == "sigmoid" else np.ones(len(s))
            np.add.at(grad[t], s, scale * u * (h - mean) * rest)
            np.add.at(bound[t], s, abs(scale) * u * rest * 2 * r * (np.abs(h) + weight))
    return grad, bound


def sort_experts(ids, first, experts):
    flat = ids.astype(np.int64).ravel()
    buckets = [[] for _ in range(experts + 1)]
    for s, e in enumerate(flat):
        buckets[e - first if first <= e < first + experts else experts].append(s)
    order = np.array([s for b in buckets for s in b], dtype=np.int64)
    place = np.empty(flat.size, dtype=np.int64)
    place[order] = np.arange(flat.size)
    for s in buckets[experts]:
        place[s] = ~place[s]
    counts = [len(b) for b in buckets]
    offsets = np.concatenate([[0], np.cumsum(counts[:experts])])
    return order, place.reshape(ids.shape), offsets


def spread(x, position, weights, rows):
    """rows (a float64 copy of what is there before the call) with the tokens'
    rows written; a place beyond them is skipped."""
    rows = rows.astype(np.float64).copy()
    T, k = position.shape
    for t in range(T):
        for j in range(k):
            p = int(position[t, j])
            place = p if p >= 0 else ~p
            if place >= rows.shape[0]:
                continue
            w = 1.0 if weights is None else float(weights[t, j])
            rows[place] = w * x[t].astype(np.float64) if p >= 0 else 0.0
    return rows


def join(rows, position, weights):
    """(sums, sums of magnitudes)."""
    T, k = position.shape
    out, size = np.zeros((T, rows.shape[1])), np.zeros((T, rows.shape[1]))
    for t in range(T):
        for j in range(k):
            p = int(position[t, j])
            if 0 <= p < rows.shape[0]:
                v = (1.0 if weights is None else float(weights[t, j])) * rows[p].astype(np.float64)
                out[t] += v
                size[t] += np.abs(v)
    return out, size


def dots(x, rows, position):
    """(products, sums of magnitudes)."""
    T, k = position.shape
    out, size = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            p = int(position[t, j])
            if 0 <= p < rows.shape[0]:
                v = x[t].astype(np.float64) * rows[p].astype(np.float64)
                out[t, j], size[t, j] = v.sum(), np.abs(v).sum()
    return out, size


def spread_bound(exact, dtype):
    """One float32 product, one rounding to dtype."""
    return np.abs(exact) * (HALF_STEP[dtype] + U32) * 1.01 + TINY[dtype]


def join_bound(exact, size, k, dtype):
    """k products added in float32 (two roundings a term), one rounding to
    dtype."""
    return 2 * k * U32 * size * 1.01 + np.abs(exact) * HALF_STEP[dtype] * 1.01 + TINY[dtype]


def dots_bound(size, width):
    """A float32 sum spread over 64 lanes or more: width / 64 terms and the
    16 of a last access each, then joined in at most 8 steps; a product and a
    sum round each term."""
    return 2 * (width / 64 + 24) * U32 * size + TINY["float32"]
