"""Plain 64-bit definitions of the experts' products, of rows in 8 bits and of
gated rows (torch, on any device), and bounds on the rounding of the calls."""
import torch

import expert_oracle as eo

HALF_STEP, TINY = eo.HALF_STEP, eo.TINY
STEP32 = 2.0 ** -23            # a step of float32, relative: what an addition inside a matrix instruction may lose
BLOCK, FP8_MAX, LEAST = 128, 448.0, 2.0 ** -100
# What a matrix instruction may lose of 128 products of 8-bit operands, relative to
# the largest of them: each is aligned to the largest and cut 2^-18 below it.
LOST8 = 2.0 ** -11


def spans(offsets, experts, n):
    if offsets is None:
        return [(0, n)]
    o = [min(max(int(v), 0), n) for v in offsets.tolist()]
    return [(o[e], max(o[e], o[e + 1])) for e in range(experts)]


def product(x, spans_, w, before):
    """(results, sums of sizes) of rows in float64; `before` where there is no expert."""
    out, size = before.double().clone(), torch.zeros_like(before, dtype=torch.float64)
    for (lo, hi), m in zip(spans_, w):
        if hi > lo:
            out[lo:hi] = x[lo:hi].double() @ m.double().t().contiguous()
            size[lo:hi] = x[lo:hi].double().abs() @ m.double().abs().t().contiguous()
    return out, size


def product_rows_backward(g, spans_, w, before):
    return product(g, spans_, [m.t() for m in w], before)


def product_weights_backward(g, spans_, x):
    E, N, K = len(spans_), g.shape[1], x.shape[1]
    out, size = (torch.zeros(E, N, K, dtype=torch.float64, device=g.device) for _ in range(2))
    for e, (lo, hi) in enumerate(spans_):
        a, b = g[lo:hi].double().t().contiguous(), x[lo:hi].double()
        out[e], size[e] = a @ b, a.abs() @ b.abs()
    return out, size


def product_bound(exact, size, terms, dtype):
    """`terms` products added in float32 by instructions that may cut, one rounding
    to dtype."""
    return (terms + 8) * STEP32 * size + exact.abs() * HALF_STEP[dtype] * 1.01 + TINY[dtype]


def expand(q, scales):
    """The values that (n, K) e4m3 and (blocks, n) scales stand for."""
    return q.double() * scales.double().t().repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def expand_weights(q, scales):
    s = scales.double().repeat_interleave(BLOCK, 1)[:, :q.shape[1]].repeat_interleave(BLOCK, 2)[:, :, :q.shape[2]]
    return q.double() * s


def fp8_lost(x, spans_, w, before):
    """Bound on what the matrix instructions lose, of expanded rows and weights: for
    each block the largest product."""
    lost = torch.zeros_like(before, dtype=torch.float64)
    for (lo, hi), m in zip(spans_, w):
        for a in range(lo, hi, 16):
            z = slice(a, min(hi, a + 16))
            for k in range(0, x.shape[1], BLOCK):
                p = x[z, None, k:k + BLOCK].abs() * m[None, :, k:k + BLOCK].abs()
                lost[z] += LOST8 * p.amax(2)
    return lost


def quantized(x):
    """(values before they are rounded, scales) of rows in float64."""
    n, width = x.shape
    blocks = (width + BLOCK - 1) // BLOCK
    wide = torch.zeros(n, blocks * BLOCK, dtype=torch.float64, device=x.device)
    wide[:, :width] = x
    parts = wide.reshape(n, blocks, BLOCK)
    size = torch.where(parts.isfinite(), parts.abs(), torch.zeros_like(parts))
    scale = size.amax(2).clamp(min=LEAST) / FP8_MAX
    return (parts / scale[:, :, None]).reshape(n, -1)[:, :width], scale.t()


def quantized_bound(v):
    """Half a step of e4m3: 2^-4 of the value, at least 2^-10; the value itself
    comes out of three float32 roundings."""
    return torch.clamp(v.abs() * 2.0 ** -4, min=2.0 ** -10) * (1 + 2.0 ** -20) + v.abs() * 4 * STEP32


def act(a, kind):
    """(act(a), act'(a), the sum of the sizes of the latter's terms)."""
    if kind == "silu":
        s, r = torch.sigmoid(a), torch.sigmoid(-a)
        return a * s, s + a * s * r, s + (a * s * r).abs()
    cdf = 0.5 * torch.special.erfc(-a / 2.0 ** 0.5)
    density = torch.exp(-0.5 * a * a) / (2 * torch.pi) ** 0.5
    return a * cdf, cdf + a * density, cdf + (a * density).abs()


def gate(x, kind):
    a, b = x.double().chunk(2, 1)
    return act(a, kind)[0] * b


def gate_backward(g, x, kind):
    """(gradient, sizes of the terms)."""
    a, b = x.double().chunk(2, 1)
    value, slope, size = act(a, kind)
    g = g.double()
    return torch.cat([g * b * slope, g * value], 1), torch.cat([(g * b).abs() * size, (g * value).abs()], 1)


def gate_relative(x, kind):
    """Relative error of the activation in float32: its argument is rounded (twice
    for gelu's square), which moves an exponential by the argument in steps."""
    a = x.double().chunk(2, 1)[0].abs()
    return STEP32 * ((a if kind == "silu" else a * a) + 24)


def gate_bound(exact, size, relative, x, dtype):
    """... and exponentials below the normal range may be taken as zero."""
    top = x.double().abs().amax() + 1
    return size * relative + exact.abs() * HALF_STEP[dtype] * 1.01 + TINY[dtype] + 2.0 ** -125 * top ** 3
