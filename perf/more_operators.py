"""Cases of the experts' own work in a mixture-of-experts layer: the matrix
products of token rows that stand sorted by expert, in 16 and 32 bits and with
8-bit operands, and what stands between and before them.

n rows stand expert by expert: expert e has rows offsets[e] .. offsets[e + 1] - 1,
rows behind the last expert's belong to none.  The operators are

  product    out[r] = weights[e] @ rows[r], weights (E, N, K)
  product_bwd  grad_rows[r] = grad[r] @ weights[e],
             grad_weights[e] = the sum over the expert's rows of grad[r] x rows[r]
  fp8        product of e4m3 rows with a scale for each 128 elements and e4m3
             weights with a scale for each 128 x 128 elements
  quantize   rows to e4m3 with a scale for each 128 elements
  gate       out = silu(first half of a row) * second half
  gate_bwd   its gradient
  gate_quantize  gate, and its result to e4m3 with a scale for each 128 elements

Rows of no expert get zeros.
"""
import math
import random

import torch

own = False

_DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2}
_F8 = torch.float8_e4m3fn
_F8_MAX = 448.0
_BLOCK = 128
_LEAST = 2.0 ** -100      # the least maximum of a block that its scale follows


def _case(name, op, rows, E=1, N=0, K=0, dtype="bf16", pad=0.0):
    c = {"op": op, "rows": rows, "E": E, "N": N, "K": K, "dtype": dtype, "pad": pad}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # One decoded token with 8 choices: the weights of 8 experts are read once.
        _case("product_token", "product", 8, E=64, N=2048, K=2048),
        # A prefill batch of 4096 tokens with 8 choices: the first product of its layer.
        _case("product_prefill", "product", 32768, E=64, N=4096, K=4096),
        # Half-precision rows of odd widths, a fifth of them for no expert here.
        _case("product_odd", "product", 5003, E=7, N=1001, K=1537, dtype="f16", pad=0.2),
        # A training batch's gradients, of rows and of weights.
        _case("product_grad", "product_bwd", 16384, E=16, N=2816, K=2048, pad=0.05),
        # Full-precision training with few experts and odd widths.
        _case("product_grad_f32", "product_bwd", 4093, E=8, N=515, K=1030, dtype="f32"),
        # A decode batch of 32 tokens with 8 choices: 2 rows an expert, weights in 8 bits.
        _case("fp8_decode", "fp8", 256, E=128, N=2048, K=4096),
        # A long prefill with 8-bit weights: the largest product.
        _case("fp8_prefill", "fp8", 32768, E=32, N=4096, K=7168),
        # A decode batch's tokens to 8 bits: latency.
        _case("quantize_decode", "quantize", 64, K=7168),
        # A prefill batch's tokens to 8 bits, at a width that is no multiple of the block.
        _case("quantize_prefill", "quantize", 16384, K=2880),
        # A prefill batch between its two products.
        _case("gate_prefill", "gate", 32768, K=2048, pad=0.05),
        # A training batch's gradient between its two products, odd width.
        _case("gate_grad", "gate_bwd", 16383, K=1411, dtype="f16"),
        # A prefill batch between two products with 8-bit operands.
        _case("gate_quantize", "gate_quantize", 32768, K=2048),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["product", "product", "product_bwd", "fp8", "fp8", "quantize", "gate", "gate_bwd", "gate_quantize"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f16", "f32"])
    pad = rng.choice([0.0, 0.0, rng.uniform(0.0, 0.5)])
    rows = _log(rng, 1, 32768)
    K = _log(rng, 64, 7168)
    if rng.random() < 0.7:
        K = (K + 63) // 64 * 64
    if op in ("quantize", "gate", "gate_bwd", "gate_quantize"):
        return _case(None, op, rows, K=K, dtype=dtype, pad=pad)
    E = _log(rng, 1, 128)
    N = _log(rng, 64, 4096)
    if rng.random() < 0.7:
        N = (N + 63) // 64 * 64
    if op == "product_bwd":               # two products
        rows = min(rows, 16384)
    if dtype == "f32":                    # 32-bit products run at a small share of the 16-bit rate
        rows, N = min(rows, 8192), min(N, 2048)
    E = max(1, min(E, (1 << (28 if op == "product_bwd" else 30)) // (N * K)))
    return _case(None, op, rows, E=E, N=N, K=K, dtype="bf16" if op == "fp8" and dtype == "f32" else dtype, pad=pad)


# ---------------------------------------------------------------------------
# Sizes of a case
# ---------------------------------------------------------------------------
def _used(case):
    """Rows that belong to an expert."""
    return max(1, case["rows"] - int(case["rows"] * case["pad"]))


def _counts(case):
    """Rows of each expert: some are liked, as routers do; whose turn it is, the
    seed says."""
    E, rng = case["E"], random.Random(case["E"] * 1000003 + _used(case))
    liking = [math.exp(0.5 * rng.gauss(0.0, 1.0)) for _ in range(E)]
    counts = [0] * E
    for e in rng.choices(range(E), weights=liking, k=_used(case)):
        counts[e] += 1
    return counts


def _blocks(width):
    return (width + _BLOCK - 1) // _BLOCK


def work(case):
    n, N, K, b, op = case["rows"], case["N"], case["K"], _BYTES[case["dtype"]], case["op"]
    used = _used(case)
    if op == "quantize":
        return {"bytes": used * K * b + n * (K + 4 * _blocks(K)), "flops": 3 * used * K}
    if op == "gate":
        return {"bytes": used * 2 * K * b + n * K * b, "flops": 5 * used * K}
    if op == "gate_bwd":
        return {"bytes": used * 3 * K * b + n * 2 * K * b, "flops": 10 * used * K}
    if op == "gate_quantize":
        return {"bytes": used * 2 * K * b + n * (K + 4 * _blocks(K)), "flops": 8 * used * K}
    active = sum(c > 0 for c in _counts(case))      # the other experts' weights are not read
    if op == "product":
        return {"bytes": used * K * b + active * N * K * b + n * N * b, "flops": 2 * used * N * K}
    if op == "product_bwd":
        return {"bytes": used * (N + K) * b + active * N * K * b + n * K * b + case["E"] * N * K * b,
                "flops": 4 * used * N * K}
    return {"bytes": used * (K + 4 * _blocks(K)) + active * (N * K + 4 * _blocks(N) * _blocks(K)) + n * N * b,
            "flops": 2 * used * N * K}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _outlying(rows, width, gen):
    """Activations: some channels are larger than the others."""
    channel = torch.exp(torch.randn(width, generator=gen, device="cuda"))
    return torch.randn(rows, width, generator=gen, device="cuda") * channel


def _normal(shape, scale, dtype, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype).mul_(scale)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    n, E, N, K, op = case["rows"], case["E"], case["N"], case["K"], case["op"]
    dt = _DTYPES[case["dtype"]]
    st = {"case": case}
    if op in ("quantize", "gate", "gate_bwd", "gate_quantize"):
        st["offsets"] = torch.tensor([0, _used(case)], dtype=torch.int32, device="cuda")
        st["rows"] = _outlying(n, K if op == "quantize" else 2 * K, gen).to(dt)
        if op == "gate_bwd":
            st["grad"] = _normal((n, K), 1.0, dt, gen)
        return st
    counts = _counts(case)
    random.Random(seed).shuffle(counts)
    st["offsets"] = torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32)
    # For the plain form: the experts that have rows, and the most that one has.
    st["active"] = torch.tensor([e for e in range(E) if counts[e]], device="cuda")
    st["most"] = max(counts)
    if op == "fp8":
        st["rows"], st["row_scales"] = _quantized(_outlying(n, K, gen))
        st["weights"] = torch.empty(E, N, K, dtype=_F8, device="cuda")
        st["weight_scales"] = torch.empty(E, _blocks(N), _blocks(K), device="cuda")
        for e in range(E):
            w = torch.randn(N, K, generator=gen, device="cuda") / math.sqrt(K)
            st["weights"][e], st["weight_scales"][e] = _quantized_weights(w)
        return st
    st["rows"] = _outlying(n, K, gen).to(dt)
    st["weights"] = _normal((E, N, K), 1.0 / math.sqrt(K), dt, gen)
    if op == "product_bwd":
        st["grad"] = _normal((n, N), 1.0, dt, gen)
    return st


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
def _in_blocks(x):
    """(rows, blocks, 128) of (rows, width), zeros behind the width."""
    wide = torch.zeros(x.shape[0], _blocks(x.shape[1]) * _BLOCK, device=x.device)
    wide[:, :x.shape[1]] = x
    return wide.reshape(x.shape[0], -1, _BLOCK)


def _quantized(x):
    """e4m3 values (rows, width) and scales (blocks, rows) of 32-bit rows."""
    parts = _in_blocks(x)
    scale = parts.abs().amax(2).clamp(min=_LEAST) / _F8_MAX
    q = (parts / scale[:, :, None]).clamp(-_F8_MAX, _F8_MAX).to(_F8)
    return q.reshape(x.shape[0], -1)[:, :x.shape[1]].contiguous(), scale.t().contiguous()


def _quantized_weights(w):
    """e4m3 values (N, K) and scales (blocks of N, blocks of K) of a 32-bit matrix."""
    N, K = w.shape
    wide = torch.zeros(_blocks(N) * _BLOCK, _blocks(K) * _BLOCK, device=w.device)
    wide[:N, :K] = w
    parts = wide.reshape(_blocks(N), _BLOCK, _blocks(K), _BLOCK)
    scale = parts.abs().amax((1, 3)).clamp(min=_LEAST) / _F8_MAX
    q = (parts / scale[:, None, :, None]).clamp(-_F8_MAX, _F8_MAX).to(_F8)
    return q.reshape(wide.shape)[:N, :K], scale


def _padded(st, rows):
    """The rows of each active expert, (active, most, width) in 32 bits, zeros
    behind its last."""
    lo, hi = st["offsets"][st["active"]].long(), st["offsets"][st["active"] + 1].long()
    at = lo[:, None] + torch.arange(st["most"], device=rows.device)
    own_row = at < hi[:, None]
    return rows[torch.where(own_row, at, torch.zeros_like(at))].float() * own_row[:, :, None]


def _unpadded(st, padded, count, dtype):
    """Back from there: row r of `count`, zeros where it has no expert."""
    at = torch.arange(count, device=padded.device)
    group = torch.searchsorted(st["offsets"][st["active"] + 1].long(), at, right=True)
    has = group < st["active"].numel()
    group = torch.where(has, group, torch.zeros_like(group))
    slot = torch.where(has, at - st["offsets"][st["active"]].long()[group], torch.zeros_like(at))
    rows = padded.reshape(-1, padded.shape[2])[group * st["most"] + slot]
    return (rows * has[:, None]).to(dtype)


def _plain_fp8(st):
    K, N = st["case"]["K"], st["case"]["N"]
    rows = st["rows"].float() * st["row_scales"].t().repeat_interleave(_BLOCK, 1)[:, :K]
    scales = st["weight_scales"][st["active"]].repeat_interleave(_BLOCK, 1)[:, :N]
    weights = st["weights"].view(torch.uint8)[st["active"]].view(_F8).float()
    weights = weights * scales.repeat_interleave(_BLOCK, 2)[:, :, :K]
    product = torch.bmm(_padded(st, rows), weights.transpose(1, 2))
    return _unpadded(st, product, rows.shape[0], _DTYPES[st["case"]["dtype"]])


def _plain_product(st):
    weights = st["weights"][st["active"]].float()
    product = torch.bmm(_padded(st, st["rows"]), weights.transpose(1, 2))
    return _unpadded(st, product, st["rows"].shape[0], st["rows"].dtype)


def _plain_product_bwd(st):
    weights = st["weights"][st["active"]].float()
    grad, rows = _padded(st, st["grad"]), _padded(st, st["rows"])
    grad_rows = _unpadded(st, torch.bmm(grad, weights), st["rows"].shape[0], st["rows"].dtype)
    grad_weights = torch.zeros_like(st["weights"])
    grad_weights[st["active"]] = torch.bmm(grad.transpose(1, 2), rows).to(grad_weights.dtype)
    return grad_rows, grad_weights


def _live(st):
    """1 for a row that has an expert, else 0."""
    return (torch.arange(st["rows"].shape[0], device="cuda") < st["offsets"][-1]).float()[:, None]


def _gated(st):
    f = st["rows"].float()
    a, b = f[:, :f.shape[1] // 2], f[:, f.shape[1] // 2:]
    return a / (1.0 + torch.exp(-a)) * b * _live(st)


def _plain_gate_bwd(st):
    f, g = st["rows"].float(), st["grad"].float()
    a, b = f[:, :f.shape[1] // 2], f[:, f.shape[1] // 2:]
    s = 1.0 / (1.0 + torch.exp(-a))
    grad = torch.cat([g * b * s * (1.0 + a * (1.0 - s)), g * a * s], 1)
    return (grad * _live(st)).to(st["rows"].dtype)


def _plain(st):
    op = st["case"]["op"]
    if op == "product":
        return _plain_product(st)
    if op == "product_bwd":
        return _plain_product_bwd(st)
    if op == "fp8":
        return _plain_fp8(st)
    if op == "quantize":
        return _quantized(st["rows"].float() * _live(st))
    if op == "gate":
        return _gated(st).to(st["rows"].dtype)
    if op == "gate_bwd":
        return _plain_gate_bwd(st)
    return _quantized(_gated(st))


# ---------------------------------------------------------------------------
# The framework's operators
# ---------------------------------------------------------------------------
def _own(st):
    import lsd_radix_sort_pass_amd as rs

    op = st["case"]["op"]
    if op == "product":
        return rs.expert_products(st["rows"], st["offsets"], st["weights"])
    if op == "product_bwd":
        return rs.expert_products_backward(st["grad"], st["offsets"], st["weights"], st["rows"])
    if op == "fp8":
        return rs.expert_products_fp8(st["rows"], st["row_scales"], st["offsets"], st["weights"], st["weight_scales"],
                                      dtype=_DTYPES[st["case"]["dtype"]])
    if op == "quantize":
        return rs.quantize_rows(st["rows"], st["offsets"])
    if op == "gate":
        return rs.gate_rows(st["rows"], st["offsets"])
    if op == "gate_bwd":
        return rs.gate_rows_backward(st["grad"], st["rows"], st["offsets"])
    return rs.gate_quantize_rows(st["rows"], st["offsets"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_products(case, st):
    op, n, N, K = case["op"], case["rows"], case["N"], case["K"]
    bounds = st["offsets"].tolist()
    out = torch.zeros(n, N, dtype=torch.float64)
    grad_rows = torch.zeros(n, K, dtype=torch.float64)
    grad_weights = torch.zeros(case["E"], N, K, dtype=torch.float64) if op == "product_bwd" else None
    for e in range(case["E"]):
        z = slice(bounds[e], bounds[e + 1])
        if z.start == z.stop:
            continue
        x, w = st["rows"][z].double(), st["weights"][e].double()
        if op == "fp8":
            for b in range(_blocks(K)):
                k = slice(b * _BLOCK, min(K, (b + 1) * _BLOCK))
                x[:, k] *= st["row_scales"][b, z].double()[:, None]
                for a in range(_blocks(N)):
                    w[a * _BLOCK:(a + 1) * _BLOCK, k] *= st["weight_scales"][e, a, b].double()
        if op == "product_bwd":
            g = st["grad"][z].double()
            grad_rows[z] = torch.mm(g, w).cpu()
            grad_weights[e] = torch.mm(g.t().contiguous(), x).cpu()
        else:
            out[z] = torch.mm(x, w.t().contiguous()).cpu()
    return (grad_rows, grad_weights) if op == "product_bwd" else out


def _exact_quantized(v):
    """The values before they are rounded to 8 bits, and their scales."""
    n, width = v.shape
    scales = torch.empty(_blocks(width), n, dtype=torch.float64, device=v.device)
    q = torch.empty_like(v)
    for b in range(_blocks(width)):
        k = slice(b * _BLOCK, min(width, (b + 1) * _BLOCK))
        top = torch.maximum(v[:, k].max(1).values, -v[:, k].min(1).values)
        scales[b] = torch.where(top > _LEAST, top, torch.full_like(top, _LEAST)) / _F8_MAX
        q[:, k] = v[:, k] / scales[b][:, None]
    return q.cpu(), scales.cpu()


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("product", "product_bwd", "fp8"):
        return _exact_products(case, st)
    x = st["rows"].double()
    x[int(st["offsets"][-1]):] = 0.0
    if op == "quantize":
        return _exact_quantized(x)
    a, b = torch.chunk(x, 2, 1)
    gate = torch.sigmoid(a)
    if op == "gate":
        return (a * gate * b).cpu()
    if op == "gate_quantize":
        return _exact_quantized(a * gate * b)
    g = st["grad"].double()
    return torch.cat([g * b * (gate + a * gate * torch.sigmoid(-a)), g * a * gate], 1).cpu()
