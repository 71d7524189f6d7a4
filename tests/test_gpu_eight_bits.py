"""GPU tests of what rows and weights become in 8 bits, to the bit, and of the
accuracy of products of 8-bit operands."""
import contextlib

import pytest

import product_oracle as po

torch = pytest.importorskip("torch")
rs = pytest.importorskip("lsd_radix_sort_pass_amd")
from lsd_radix_sort_pass_amd import _lib  # noqa: E402

pytestmark = pytest.mark.gpu

DTYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
FP8 = torch.float8_e4m3fn


def note(msg):
    print(f"\n[case] {msg}", flush=True)


def eight_bits(blocks):
    """(bits, scales) of blocks (count, size) in float32 on the host: the largest
    size times 1 / 448, and quotients.  Those of two float32 numbers that are rounded to
    float64 and then to float32 are the correctly rounded ones (53 >= 2 * 24 + 2 bits)."""
    size = torch.where(blocks.isfinite(), blocks.abs(), torch.zeros_like(blocks))
    scale = size.amax(1).clamp(min=2.0 ** -100) * torch.tensor(1.0 / 448, dtype=torch.float32)
    quotient = (blocks.double() / scale.double()[:, None]).float()
    bits = quotient.clamp(-448, 448).to(FP8).view(torch.uint8)
    return torch.where(blocks.isfinite(), bits, torch.full_like(bits, 0x7F)), scale


def same(bits, want):
    """Whether 8-bit values are the same, NaN of either sign."""
    nan = (want & 0x7F) == 0x7F
    return bool((((bits & 0x7F) == 0x7F) == nan).all() and torch.equal(bits[~nan], want[~nan]))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("n,K", [(700, 128), (400, 640), (300, 200), (64, 3)])
def test_quantize_rows_divide_by_the_scale(n, K, dtype):
    """Numbers of few digits, whose quotients often stand halfway between two
    e4m3, in blocks of all magnitudes."""
    note(f"quantize bits {dtype} n={n} K={K}")
    gen = torch.Generator().manual_seed(n + K)
    whole = torch.randint(-64, 65, (n, K), generator=gen).float()
    top = {"float16": 8, "bfloat16": 120, "float32": 120}[dtype]
    x = whole * torch.exp2(torch.randint(-top - 10, top + 1, (n, 1), generator=gen).float())
    x[:n // 4] = torch.randn(n // 4, K, generator=gen)
    x[0] = 0
    x[1, 0], x[2, K - 1], x[3, K // 2] = float("nan"), float("inf"), float("-inf")
    x[4] = float(torch.finfo(DTYPES[dtype]).max)
    x = x.to(DTYPES[dtype])
    got = rs.quantize_rows(x.cuda())
    for b in range(0, K, 128):
        bits, scale = eight_bits(x[:, b:b + 128].float())
        assert torch.equal(got.scales[b // 128].cpu(), scale)
        assert same(got.values.view(torch.uint8)[:, b:b + 128].cpu(), bits), f"block {b}"


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_quantize_weights_divide_by_the_scale(dtype):
    note(f"quantize weights bits {dtype}")
    gen = torch.Generator().manual_seed(3)
    E, N, K = 5, 200, 300
    w = torch.randint(-64, 65, (E, N, K), generator=gen).float()
    w *= torch.exp2(torch.tensor([0.0, 8.0, -14.0, -30.0, -110.0]))[:, None, None]      # (float16 loses the last two)
    w = w.to(DTYPES[dtype])
    got = rs.quantize_weights(w.cuda())
    for e in range(E):
        for a in range(0, N, 128):
            for b in range(0, K, 128):
                part = w[e, a:a + 128, b:b + 128].float()
                bits, scale = eight_bits(part.reshape(1, -1))
                assert float(got.scales[e, a // 128, b // 128]) == float(scale[0])
                have = got.values.view(torch.uint8)[e, a:a + 128, b:b + 128].cpu().reshape(1, -1)
                assert same(have, bits), (e, a, b)


def test_gate_quantize_rows_divide_by_the_scale():
    """Gated rows that are exact: silu(64) is 64 in float32, times a number of few digits."""
    note("gate_quantize bits")
    gen = torch.Generator().manual_seed(4)
    b = torch.randint(-64, 65, (300, 256), generator=gen).float()
    x = torch.cat([torch.full_like(b, 64.0), b], 1)
    for dtype in DTYPES.values():
        got = rs.gate_quantize_rows(x.to(dtype).cuda())
        for k in (0, 128):
            bits, scale = eight_bits(64.0 * b[:, k:k + 128])
            assert torch.equal(got.scales[k // 128].cpu(), scale)
            assert same(got.values.view(torch.uint8)[:, k:k + 128].cpu(), bits)


@contextlib.contextmanager
def forced(kernel):
    before = rs.prof_product_kernel(kernel)
    try:
        yield
    finally:
        rs.prof_product_kernel(before)


KERNELS = {"square": _lib.RS_PRODUCT_SQUARE, "few": _lib.RS_PRODUCT_FEW, "split": _lib.RS_PRODUCT_SPLIT}


@pytest.mark.parametrize("dtype", ["float32", "float16"])
@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("n,N,K", [(40, 33, 128), (70, 130, 400), (3, 5, 9)])
def test_fp8_sums_in_float32(n, N, K, kernel, dtype):
    """In each block two large products cancel, and what is left is 2^-10 of them and
    less: sums in float32 lose 2^-24 of a partial sum a step."""
    note(f"fp8 sums {kernel} {dtype} n={n} N={N} K={K}")
    gen = torch.Generator().manual_seed(n + K)
    x = torch.randint(-15, 16, (n, K), generator=gen).float() * 2.0 ** -6
    w = torch.randint(-15, 16, (1, N, K), generator=gen).float() * 2.0 ** -6
    for b in range(0, K, 128):
        last = min(b + 128, K) - 1
        x[:, b], x[:, last], w[:, :, b], w[:, :, last] = 8.0, -8.0, 8.0, 8.0
    x, w = x.cuda().to(FP8), w.cuda().to(FP8)
    qs = torch.exp2(torch.rand((K + 127) // 128, n, generator=gen)).cuda()
    ws = torch.exp2(torch.rand(1, (N + 127) // 128, (K + 127) // 128, generator=gen)).cuda()
    spans = [(0, n)]
    exact, size = po.product(po.expand(x, qs), spans, po.expand_weights(w, ws), torch.zeros(n, N, device="cuda"))
    with forced(KERNELS[kernel]):
        got = rs.expert_products_fp8(x, qs, None, w, ws, DTYPES[dtype]).double()
    # K products, a product of scales and one with them for each block.
    bound = po.product_bound(exact, size, K + 2, dtype)
    assert ((got - exact).abs() <= bound).all(), f"{float(((got - exact).abs() / bound).max())} bounds off"


# A kernel each, and the wide one, which serves bfloat16 alone; magnitudes of the scales of rows
# and of matrices, whose products are normal numbers.
@pytest.mark.parametrize("rows,matrix", [(-100, 80), (-90, 110), (100, -100), (50, 48), (-105, -18), (0, 0)])
@pytest.mark.parametrize("kernel,dtype", [(k, d) for k in KERNELS for d in ("float32", "bfloat16")] + [("wide", "bfloat16")])
def test_fp8_scales_of_any_size(kernel, dtype, rows, matrix):
    """Results in float32's range are right, whatever the scales are; rows and blocks of
    zeros, whose scales' product may be too small for float32, give zeros."""
    note(f"fp8 scales {kernel} {dtype} 2^{rows} 2^{matrix}")
    gen = torch.Generator().manual_seed(rows + 200)
    n, N, K = 70, 136, 384
    x, w = torch.randint(-15, 16, (n, K), generator=gen).float(), torch.randint(-15, 16, (1, N, K), generator=gen).float()
    qs, ws = torch.exp2(rows + torch.rand(3, n, generator=gen)), torch.exp2(matrix + torch.rand(1, 2, 3, generator=gen))
    least = 2.0 ** -100 / 448
    x[:, 128:256], qs[1], w[:, 128:], ws[:, 1] = 0, least, 0, least       # as they become in 8 bits
    x, w, qs, ws = x.cuda().to(FP8), w.cuda().to(FP8), qs.cuda(), ws.cuda()
    values, matrices, none = po.expand(x, qs), po.expand_weights(w, ws), torch.zeros(n, N, device="cuda")
    exact, size = po.product(values, [(0, n)], matrices, none)
    with forced({**KERNELS, "wide": _lib.RS_PRODUCT_WIDE}[kernel]):
        got = rs.expert_products_fp8(x, qs, None, w, ws, DTYPES[dtype]).double()
    bound = po.product_bound(exact, size, K + 2, dtype)
    if dtype == "bfloat16":
        bound += po.fp8_lost(values, [(0, n)], matrices, none)
    assert ((got - exact).abs() <= bound).all(), (float(got.abs().max()), float(exact.abs().max()))
    assert (got[:, 128:] == 0).all()


def test_tangents_are_refused():
    """Of every tensor, the 8-bit ones too, which may carry them."""
    note("tangents in 8 bits")
    import torch.autograd.forward_ad as fwd
    x, w = torch.randn(6, 32, device="cuda"), torch.randn(1, 16, 32, device="cuda")
    (q, s), (w8, ws) = rs.quantize_rows(x), rs.quantize_weights(w)
    out = torch.empty(6, 16, device="cuda")
    operands = {"rows": q, "row_scales": s, "weights": w8, "weight_scales": ws, "out": out}
    results = {"rows": x, "out": torch.empty_like(q), "scales_out": torch.empty_like(s)}
    gated = {"rows": torch.randn(6, 64, device="cuda"), "out": torch.empty_like(q), "scales_out": torch.empty_like(s)}
    for call, given in ((lambda **t: rs.expert_products_fp8(offsets=None, **t), operands), (rs.quantize_rows, results),
                        (rs.gate_quantize_rows, gated), (rs.quantize_weights, {"weights": w})):
        with fwd.dual_level():
            call(**given)
            for name, t in given.items():
                dual = fwd.make_dual(t, torch.zeros(t.shape, device="cuda").to(t.dtype))
                with pytest.raises(ValueError, match=f"^{name} carries a tangent"):
                    call(**{**given, name: dual})


@pytest.mark.parametrize("kernel,dtype", [(k, d) for k in KERNELS for d in DTYPES] + [("wide", "bfloat16")])
def test_fp8_every_value(kernel, dtype):
    """Every e4m3 as a row's and as a matrix's element, times 1; a NaN of either sign makes
    NaN of its row or column alone.  (The wide kernel serves bfloat16 alone.)"""
    note(f"fp8 every value {kernel} {dtype}")
    bits = torch.arange(256, dtype=torch.uint8)
    finite = bits[(bits & 0x7F) != 0x7F].cuda().view(FP8)                # 254
    one = torch.eye(254, device="cuda").to(FP8)
    values = torch.zeros(254, 254, device="cuda").to(FP8)
    values[:] = finite
    qs, ws = torch.ones(2, 254, device="cuda"), torch.ones(1, 2, 2, device="cuda")
    pad = torch.zeros(254, 2, device="cuda").to(FP8)                     # (rows of whole 16 bytes)
    one, values = torch.cat([one, pad], 1), torch.cat([values, pad], 1)
    with forced({**KERNELS, "wide": _lib.RS_PRODUCT_WIDE}[kernel]):
        rows = rs.expert_products_fp8(values, qs, None, one[None], ws, DTYPES[dtype])
        matrix = rs.expert_products_fp8(one, qs, None, values[None], ws, DTYPES[dtype])
        assert torch.equal(rows.float(), finite.float().expand(254, 254))
        assert torch.equal(matrix.float(), finite.float()[:, None].expand(254, 254))
        x, w = values.clone(), one.clone()
        x.view(torch.uint8)[7, 200], w.view(torch.uint8)[250, 3] = 0x7F, 0xFF
        got = rs.expert_products_fp8(x, qs, None, w[None], ws, DTYPES[dtype])
    nan = torch.zeros(254, 254, dtype=torch.bool, device="cuda")
    nan[7], nan[:, 250] = True, True
    assert torch.equal(got.isnan(), nan) and torch.equal(got[~nan], rows[~nan])
