"""GPU tests of the experts' products, 8-bit rows and gated rows against their
64-bit definitions (product_oracle)."""
import pytest

import product_oracle as po

torch = pytest.importorskip("torch")
rs = pytest.importorskip("lsd_radix_sort_pass_amd")

pytestmark = pytest.mark.gpu

DTYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
NAMES = {v: k for k, v in DTYPES.items()}
FP8 = torch.float8_e4m3fn


def note(msg):
    print(f"\n[case] {msg}", flush=True)


def close(got, exact, bound, what):
    got = got.double()
    bad = ~(((got - exact).abs() <= bound) | (got.isnan() & exact.isnan()) | (got == exact))
    if bad.any():
        at = bad.nonzero()[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()}, first {at}: {got[tuple(at)]} for "
                             f"{exact[tuple(at)]}, bound {bound.expand_as(got)[tuple(at)]}")


def generator(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return gen


def normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(DTYPES[dtype])


def offsets_of(n, E, kind):
    """Offsets of E experts over n rows: "all" rows have one; "holes": empty
    experts, rows before the first and behind the last without one; "one" expert
    has all; "none" has any."""
    gen = torch.Generator().manual_seed(n * 31 + E)
    if kind == "one":
        e = n % E
        o = [0] * (e + 1) + [n] * (E - e)
    elif kind == "none":
        o = [n // 2] * (E + 1)
    else:
        lo, hi = (0, n) if kind == "all" else (n // 9, n - n // 5)
        cuts = torch.randint(lo, hi + 1, (max(0, E - 1),), generator=gen).tolist()
        if kind == "holes" and E > 3:
            cuts[1] = cuts[0]
        o = [lo] + sorted(cuts) + [hi]
    return torch.tensor(o, dtype=torch.int32, device="cuda")


# (rows, experts, N, K): single elements, odd widths, widths below 16 bytes, one and
# several tiles each way, whole tiles, rows whose starts are aligned and not.
SHAPES = [(1, 1, 1, 1), (3, 2, 5, 7), (17, 4, 33, 64), (40, 5, 3, 2), (130, 3, 129, 65), (300, 5, 136, 200),
          (64, 8, 256, 520), (1000, 6, 304, 1032), (513, 2, 640, 96), (700, 3, 257, 259), (8, 64, 192, 256)]
# Many rows an expert and rows that begin at 16 bytes: contractions of one and several
# stages with and without a rest, tiles of more and fewer than 128 rows.
SHAPES += [(300, 1, 136, 8), (1500, 4, 264, 200), (900, 2, 512, 1032), (520, 3, 1000, 40), (2100, 5, 152, 352)]
KINDS = ["all", "holes", "one", "none"]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,E,N,K", SHAPES)
def test_products(n, E, N, K, kind, dtype):
    note(f"expert_products {dtype} n={n} E={E} N={N} K={K} {kind}")
    gen = generator(n + N + K)
    o = offsets_of(n, E, kind)
    s = po.spans(o, E, n)
    x, w, g = normal(gen, (n, K), dtype), normal(gen, (E, N, K), dtype, K ** -0.5), normal(gen, (n, N), dtype)
    zeros, held = torch.zeros(n, N, device="cuda"), torch.full((n, N), 3.0, dtype=DTYPES[dtype], device="cuda")
    exact, size = po.product(x, s, w, zeros)
    close(rs.expert_products(x, o, w), exact, po.product_bound(exact, size, K, dtype), "product")
    exact, size = po.product(x, s, w, held)
    close(rs.expert_products(x, o, w, out=held), exact, po.product_bound(exact, size, K, dtype), "given out")
    grad_rows, grad_w = rs.expert_products_backward(g, o, w, x)
    exact, size = po.product_rows_backward(g, s, w, torch.zeros(n, K, device="cuda"))
    close(grad_rows, exact, po.product_bound(exact, size, N, dtype), "gradient of rows")
    exact, size = po.product_weights_backward(g, s, x)
    close(grad_w, exact, po.product_bound(exact, size, n, dtype), "gradient of weights")
    assert torch.equal(rs.expert_products_backward(g, o, rows=x), grad_w)
    assert torch.equal(rs.expert_products_backward(g, o, w), grad_rows)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("N,K", [(40, 72), (130, 264), (33, 65), (256, 328)])
def test_products_strided(N, K, dtype):
    """Rows and matrices that are views: wider rows, every other row, experts in
    another order of strides, outputs among other columns; what lies beside them
    stays, NaN there does no harm."""
    note(f"strided {dtype} N={N} K={K}")
    gen = generator(N)
    E = 4
    for extra, n, begin in ((8, 150, 1), (3, 150, 1), (8, 1200, 0), (16, 700, 8)):
        o = offsets_of(n, E, "holes")
        s = po.spans(o, E, n)
        x = torch.full((2 * n, K + extra), float("nan"), dtype=DTYPES[dtype], device="cuda")[::2, begin:K + begin]
        w = torch.full((N, E, K + extra), float("nan"), dtype=DTYPES[dtype], device="cuda")[:, :, :K].transpose(0, 1)
        g = torch.full((n, N + extra), float("nan"), dtype=DTYPES[dtype], device="cuda")[:, :N]
        x.copy_(normal(gen, (n, K), dtype)), w.copy_(normal(gen, (E, N, K), dtype)), g.copy_(normal(gen, (n, N), dtype))
        wide = torch.full((n, N + 2 * extra), 5.0, dtype=DTYPES[dtype], device="cuda")
        rs.expert_products(x, o, w, out=wide[:, extra:extra + N])
        exact, size = po.product(x, s, w, torch.full((n, N), 5.0, device="cuda"))
        close(wide[:, extra:extra + N], exact, po.product_bound(exact, size, K, dtype), "product")
        assert (wide[:, :extra] == 5.0).all() and (wide[:, extra + N:] == 5.0).all()
        grad_rows, grad_w = rs.expert_products_backward(g, o, w, x)
        exact, size = po.product_rows_backward(g, s, w, torch.zeros(n, K, device="cuda"))
        close(grad_rows, exact, po.product_bound(exact, size, N, dtype), "gradient of rows")
        exact, size = po.product_weights_backward(g, s, x)
        close(grad_w, exact, po.product_bound(exact, size, n, dtype), "gradient of weights")


def test_products_broadcast_and_slices():
    """One matrix for all experts by a stride of 0, one row for all rows, and a range
    of experts: their offsets do not begin at 0."""
    note("broadcast and slices")
    gen = generator(5)
    n, E, N, K = 90, 6, 48, 40
    o = offsets_of(n, E, "all")
    x, w = normal(gen, (n, K), "bfloat16"), normal(gen, (E, N, K), "bfloat16")
    shared = w[:1].expand(E, N, K)
    assert torch.equal(rs.expert_products(x, o, shared), rs.expert_products(x, None, w[:1]))
    row = x[:1].expand(n, K)
    assert torch.equal(rs.expert_products(row, o, w), rs.expert_products(row.contiguous(), o, w))
    part = rs.expert_products(x, o[2:5], w[2:4])
    lo, hi = int(o[2]), int(o[4])
    whole = rs.expert_products(x, o, w)
    assert torch.equal(part[lo:hi], whole[lo:hi]) and (part[:lo] == 0).all() and (part[hi:] == 0).all()


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_products_special_values(dtype):
    """NaN and infinities stay in their own rows and columns, and in rows of no
    expert they are not read."""
    note(f"special values {dtype}")
    gen = generator(6)
    n, E, N, K = 70, 3, 40, 100
    o = torch.tensor([5, 30, 30, 60], dtype=torch.int32, device="cuda")
    s = po.spans(o, E, n)
    x, w, g = normal(gen, (n, K), dtype), normal(gen, (E, N, K), dtype), normal(gen, (n, N), dtype)
    x[:5] = x[60:] = g[:5] = g[60:] = float("nan")
    w[1] = float("nan")                                          # an expert without rows
    x[10, 3], x[40, 99], w[2, 7, 0], g[12, 39] = float("inf"), float("nan"), float("nan"), float("-inf")
    exact, size = po.product(x, s, w, torch.zeros(n, N, device="cuda"))
    close(rs.expert_products(x, o, w), exact, po.product_bound(exact, size, K, dtype), "product")
    grad_rows, grad_w = rs.expert_products_backward(g, o, w, x)
    exact, size = po.product_rows_backward(g, s, w, torch.zeros(n, K, device="cuda"))
    close(grad_rows, exact, po.product_bound(exact, size, N, dtype), "gradient of rows")
    exact, size = po.product_weights_backward(g, s, x)
    close(grad_w, exact, po.product_bound(exact, size, n, dtype), "gradient of weights")
    assert (grad_w[1] == 0).all()


def test_products_offsets_out_of_range():
    """Offsets beyond the rows are taken as their end, descending ones as empty."""
    note("offsets out of range")
    gen = generator(7)
    n, N, K = 50, 40, 64
    o = torch.tensor([-7, 20, 10, 10**9], dtype=torch.int32, device="cuda")
    x, w = normal(gen, (n, K), "float32"), normal(gen, (3, N, K), "float32")
    got = rs.expert_products(x, o, w)
    exact, size = po.product(x[:10], [(0, 10)], w[:1], torch.zeros(10, N, device="cuda"))
    close(got[:10], exact, po.product_bound(exact, size, K, "float32"), "rows of the first expert alone")
    exact, size = po.product(x[20:], [(0, 30)], w[2:], torch.zeros(30, N, device="cuda"))
    close(got[20:], exact, po.product_bound(exact, size, K, "float32"), "rows of the last expert alone")
    assert rs.expert_products_backward(x[:, :N].contiguous(), o, w, x)[1].isfinite().all()


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_products_without_rows(dtype):
    note(f"no rows {dtype}")
    w = torch.randn(3, 16, 24, device="cuda").to(DTYPES[dtype])
    o = torch.zeros(4, dtype=torch.int32, device="cuda")
    x, g = w.new_empty(0, 24), w.new_empty(0, 16)
    assert rs.expert_products(x, o, w).shape == (0, 16)
    held = torch.full((3, 16, 24), 7.0, dtype=DTYPES[dtype], device="cuda")
    grad_rows, grad_w = rs.expert_products_backward(g, o, w, x, grad_weights_out=held)
    assert grad_rows.shape == (0, 24) and (grad_w == 0).all()
    assert rs.quantize_rows(x, o).values.shape == (0, 24) and rs.gate_rows(x, o).shape == (0, 12)


def test_products_many_experts():
    """More experts than a wave has lanes, most of them without rows."""
    note("many experts")
    gen = generator(8)
    for E in (65, 200, 1024):
        n, N, K = 400, 24, 32
        o = torch.sort(torch.randint(0, n + 1, (E + 1,), generator=gen, device="cuda", dtype=torch.int32)).values
        s = po.spans(o, E, n)
        x, w, g = normal(gen, (n, K), "bfloat16"), normal(gen, (E, N, K), "bfloat16"), normal(gen, (n, N), "bfloat16")
        exact, size = po.product(x, s, w, torch.zeros(n, N, device="cuda"))
        close(rs.expert_products(x, o, w), exact, po.product_bound(exact, size, K, "bfloat16"), f"product E={E}")
        exact, size = po.product_weights_backward(g, s, x)
        close(rs.expert_products_backward(g, o, rows=x), exact, po.product_bound(exact, size, n, "bfloat16"), f"E={E}")


def test_products_far_offsets():
    """Rows and matrices that begin beyond 2^32 bytes and 2^31 elements."""
    note("far offsets")
    gen = generator(9)
    n, E, N, K, stride = 5, 3, 48, 64, 1 << 30
    x = torch.empty(n * stride, dtype=torch.bfloat16, device="cuda").as_strided((n, K), (stride, 1))
    w = torch.empty(2 * (1 << 31) + N * K, dtype=torch.bfloat16, device="cuda").as_strided((E, N, K), (1 << 31, K, 1))
    x.copy_(normal(gen, (n, K), "bfloat16")), w.copy_(normal(gen, (E, N, K), "bfloat16"))
    o = torch.tensor([0, 2, 3, 5], dtype=torch.int32, device="cuda")
    assert torch.equal(rs.expert_products(x, o, w), rs.expert_products(x.contiguous(), o, w.contiguous()))
    g = normal(gen, (n, N), "bfloat16")
    far = rs.expert_products_backward(g, o, w, x)
    near = rs.expert_products_backward(g, o, w.contiguous(), x.contiguous())
    assert torch.equal(far[0], near[0]) and torch.equal(far[1], near[1])


def test_products_far_offsets_of_tiles():
    """The same for many rows: 1200 of them 8 MiB apart, matrices 4 GiB apart."""
    note("far offsets of tiles")
    gen = generator(10)
    n, E, N, K, stride = 1200, 3, 272, 328, 1 << 22
    x = torch.empty(n * stride, dtype=torch.bfloat16, device="cuda").as_strided((n, K), (stride, 1))
    w = torch.empty(2 * (1 << 31) + N * K, dtype=torch.bfloat16, device="cuda").as_strided((E, N, K), (1 << 31, K, 1))
    x.copy_(normal(gen, (n, K), "bfloat16")), w.copy_(normal(gen, (E, N, K), "bfloat16"))
    o = torch.tensor([0, 500, 510, 1100], dtype=torch.int32, device="cuda")
    assert torch.equal(rs.expert_products(x, o, w), rs.expert_products(x.contiguous(), o, w.contiguous()))
    g = normal(gen, (n, N), "bfloat16")
    far = rs.expert_products_backward(g, o, w, x)
    near = rs.expert_products_backward(g, o, w.contiguous(), x.contiguous())
    assert torch.equal(far[0], near[0]) and torch.equal(far[1], near[1])


# (rows, experts, N, K): few results and a long contraction, whole steps of it, a rest, and
# less than the eight waves have steps; rows whose starts are aligned and not.
LONG = [(70, 1, 130, 4100), (33, 2, 72, 2048), (200, 3, 65, 1537), (40, 1, 264, 520), (129, 1, 8, 8192)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("n,E,N,K", LONG)
def test_products_long_contraction(n, E, N, K, dtype):
    note(f"long contraction {dtype} n={n} E={E} N={N} K={K}")
    gen = generator(n + N + K)
    o = offsets_of(n, E, "holes")
    s = po.spans(o, E, n)
    x, w = normal(gen, (n, K), dtype), normal(gen, (E, N, K), dtype)
    exact, size = po.product(x, s, w, torch.zeros(n, N, device="cuda"))
    close(rs.expert_products(x, o, w), exact, po.product_bound(exact, size, K, dtype), "product")
    # The same lengths the other way round: the rows' gradient over K outputs ...
    g, w = normal(gen, (n, K), dtype), normal(gen, (E, K, N), dtype)
    exact, size = po.product(g, s, w.transpose(1, 2), torch.zeros(n, N, device="cuda"))
    close(rs.expert_products_backward(g, o, w), exact, po.product_bound(exact, size, K, dtype), "gradient of rows")
    # ... and the weights' over K rows.
    o = offsets_of(K, E, "holes")
    s = po.spans(o, E, K)
    g, x = normal(gen, (K, n), dtype), normal(gen, (K, N), dtype)
    exact, size = po.product_weights_backward(g, s, x)
    got = rs.expert_products_backward(g, o, rows=x)
    close(got, exact, po.product_bound(exact, size, K, dtype), "gradient of weights")
    g[:int(o[0])], x[int(o[-1]):] = float("nan"), float("inf")      # rows of no expert
    assert torch.equal(rs.expert_products_backward(g, o, rows=x), got)


@pytest.mark.parametrize("dtype,N,K", [("bfloat16", 1 << 19, 8), ("float32", 1 << 20, 1)])
def test_products_of_many_tiles(dtype, N, K):
    """More tiles than a launch has workgroups: a row of each of 1024 experts, which share
    one matrix.  Small whole numbers, whose sums are exact."""
    note(f"many tiles {dtype}")
    gen = generator(11)
    E = 1024
    x = torch.randint(-2, 3, (E, K), generator=gen, device="cuda").to(DTYPES[dtype])
    w = torch.randint(-2, 3, (1, N, K), generator=gen, device="cuda").to(DTYPES[dtype])
    o = torch.arange(E + 1, dtype=torch.int32, device="cuda")
    got = rs.expert_products(x, o, w.expand(E, N, K))
    for first in range(0, N, 1 << 16):
        part = slice(first, first + (1 << 16))
        want = sum(x[:, k, None].float() * w[0, part, k].float() for k in range(K))
        assert torch.equal(got[:, part].float(), want)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_products_of_one_operand_twice(dtype):
    """Rows that are their results' gradient as well."""
    note(f"one operand twice {dtype}")
    gen = generator(13)
    n, E, N = 700, 2, 264
    x, w = normal(gen, (n, N), dtype), normal(gen, (E, N, N), dtype)
    o = torch.tensor([0, 300, 690], dtype=torch.int32, device="cuda")
    twice, once = rs.expert_products_backward(x, o, w, x), rs.expert_products_backward(x, o, w, x.clone())
    assert torch.equal(twice[0], once[0]) and torch.equal(twice[1], once[1])


def test_products_of_a_shard():
    """A rank that holds few of the experts: most rows are other ranks', NaN here, and
    results for them zeros, or left as they were."""
    note("shard")
    gen = generator(12)
    n, E, N, K = 3000, 2, 264, 136
    o = torch.tensor([0, 300, 430], dtype=torch.int32, device="cuda")
    for dtype in DTYPES:
        x, w = normal(gen, (n, K), dtype), normal(gen, (E, N, K), dtype)
        want = rs.expert_products(x[:430].contiguous(), o, w)
        x[430:] = float("nan")
        got = rs.expert_products(x, o, w)
        s = po.spans(o, E, n)
        exact, size = po.product(x, s, w, torch.zeros(n, N, device="cuda"))
        close(got, exact, po.product_bound(exact, size, K, dtype), "product")
        close(want, exact[:430], po.product_bound(exact, size, K, dtype)[:430], "its rows alone")
        held = torch.full((n, N + 1), 7.0, dtype=DTYPES[dtype], device="cuda")[:, 1:]
        rs.expert_products(x, o, w, out=held)
        assert torch.equal(held[:430], got[:430]) and (held[430:] == 7).all()


# ---------------------------------------------------------------------------
# 8 bits
# ---------------------------------------------------------------------------
FP8_SHAPES = [(1, 1, 1, 1), (5, 2, 130, 16), (20, 3, 40, 127), (130, 4, 129, 300), (300, 5, 264, 512), (77, 2, 33, 1041),
              (9, 40, 256, 384), (600, 2, 384, 256), (1500, 4, 264, 208), (900, 3, 520, 1040), (700, 3, 136, 16)]


def eight_bits(gen, n, E, N, K):
    x = normal(gen, (n, K), "float32") * torch.exp(normal(gen, (1, K), "float32"))
    return rs.quantize_rows(x), rs.quantize_weights(normal(gen, (E, N, K), "float32", K ** -0.5))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,E,N,K", FP8_SHAPES)
def test_products_fp8(n, E, N, K, kind, dtype):
    note(f"expert_products_fp8 {dtype} n={n} E={E} N={N} K={K} {kind}")
    o = offsets_of(n, E, kind)
    s = po.spans(o, E, n)
    (q, qs), (w, ws) = eight_bits(generator(n + N), n, E, N, K)
    x, m = po.expand(q, qs), po.expand_weights(w, ws)
    for before in (None, 2.0):
        out = None if before is None else torch.full((n, N), before, dtype=DTYPES[dtype], device="cuda")
        held = torch.full((n, N), before or 0.0, device="cuda")
        exact, size = po.product(x, s, m, held)
        bound = po.product_bound(exact, size, K // 32 + 8, dtype) + po.fp8_lost(x, s, m, held)
        close(rs.expert_products_fp8(q, qs, o, w, ws, DTYPES[dtype], out=out), exact, bound, f"out {before}")


def test_products_fp8_strided_and_special():
    """Rows and matrices that are views, at any byte; a NaN stays in its row and column."""
    note("fp8 views")
    gen = generator(11)
    n, E, N, K = 60, 3, 50, 200
    o = offsets_of(n, E, "holes")
    (q, qs), (w, ws) = eight_bits(gen, n, E, N, K)
    want = rs.expert_products_fp8(q, qs, o, w, ws)
    for extra in (16, 5):
        x = torch.full((n, K + extra), 0x7F, dtype=torch.uint8, device="cuda").view(FP8)[:, 1:K + 1]
        m = torch.full((N, E, K + extra), 0x7F, dtype=torch.uint8, device="cuda").view(FP8)[:, :, :K].transpose(0, 1)
        x.copy_(q), m.copy_(w)
        assert torch.equal(rs.expert_products_fp8(x, qs, o, m, ws), want)
    r = int(o[0]) + 1
    q.view(torch.uint8)[r, 150] = 0x7F
    got = rs.expert_products_fp8(q, qs, o, w, ws)
    assert got[r].isnan().all()
    got[r] = want[r]
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("n,K", [(1, 1), (3, 127), (17, 128), (40, 129), (100, 520), (33, 2880), (5, 8), (2000, 136)])
def test_quantize(n, K, dtype):
    note(f"quantize {dtype} n={n} K={K}")
    gen = generator(n + K)
    x = normal(gen, (n, K), dtype) * torch.exp(3 * normal(gen, (n, 1), dtype))
    x[n // 2] = 0
    if n > 10:
        x[1] = x[1] * 1e-30                     # (zeros in float16)
        x[2, K // 2], x[3, 0], x[3, K - 1] = float("nan"), float("inf"), float("-inf")
        x[4] = float("nan")
    for q, s in (rs.quantize_rows(x), rs.quantize_rows(torch.cat([x, x], 1)[:, :K])):
        v, scale = po.quantized(x.double())
        close(s, scale, scale * 2 * po.STEP32, "scales")
        finite = x.isfinite()
        assert q.double().isnan().eq(~finite).all()
        v = torch.where(finite, v, torch.zeros_like(v))
        close(torch.where(finite, q.double(), torch.zeros_like(v)), v, po.quantized_bound(v), "values")
    # Rows of no expert: zeros with the least scale, or what was there.
    o = torch.tensor([n // 4, n // 2, n - n // 3], dtype=torch.int32, device="cuda")
    live = slice(n // 4, n - n // 3)
    part = rs.quantize_rows(x, o)
    none = torch.ones(n, dtype=torch.bool, device="cuda")
    none[live] = False
    assert torch.equal(part.values.view(torch.uint8)[live], q.view(torch.uint8)[live])
    assert torch.equal(part.scales[:, live], s[:, live])
    assert (part.values.view(torch.uint8)[none] == 0).all()
    assert (part.scales[:, none] == torch.tensor(po.LEAST / 448, dtype=torch.float32, device="cuda")).all()
    held = (torch.full((n, K + 3), 0x11, dtype=torch.uint8, device="cuda").view(FP8)[:, :K],
            torch.full(s.shape, 6.0, device="cuda"))
    rs.quantize_rows(x, o, out=held[0], scales_out=held[1])
    assert (held[0].view(torch.uint8)[none] == 0x11).all() and (held[1][:, none] == 6.0).all()
    assert torch.equal(held[0].view(torch.uint8)[live], q.view(torch.uint8)[live])
    assert torch.equal(held[1][:, live], s[:, live])


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("E,N,K", [(1, 1, 1), (3, 128, 256), (2, 130, 130), (4, 300, 65)])
def test_quantize_weights(E, N, K, dtype):
    note(f"quantize_weights {dtype} {E} {N} {K}")
    w = normal(generator(N), (E, N, K), dtype)
    w[0, 0, 0] = 50.0
    for m in (w, torch.cat([w, w], 2)[:, :, :K], w.transpose(0, 1).contiguous().transpose(0, 1)):
        q, s = rs.quantize_weights(m)
        nb, kb = s.shape[1:]
        wide = torch.zeros(E, nb * 128, kb * 128, dtype=torch.float64, device="cuda")
        wide[:, :N, :K] = w.double()
        scale = wide.reshape(E, nb, 128, kb, 128).abs().amax((2, 4)).clamp(min=po.LEAST) / 448
        close(s, scale, scale * 2 * po.STEP32, "scales")
        v = w.double() / scale.repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
        close(q, v, po.quantized_bound(v), "values")


# ---------------------------------------------------------------------------
# Gated rows
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("n,F", [(1, 1), (3, 5), (9, 8), (40, 129), (70, 264), (25, 1411), (3000, 40)])
def test_gate(n, F, dtype, act):
    note(f"gate {act} {dtype} n={n} F={F}")
    gen = generator(n + F)
    x, g = normal(gen, (n, 2 * F), dtype, 2.0), normal(gen, (n, F), dtype)
    x[0, 0] = -9.0
    if n > 5:
        x[1, :F] = torch.linspace(-80, 80, F, device="cuda")
        x[2, :F] = torch.linspace(-12, 0, F, device="cuda")
        x[3, 0], x[4, F], x[5, 2] = float("nan"), float("inf"), 0.0
    o = torch.tensor([n // 4, n - n // 3], dtype=torch.int32, device="cuda")
    live = slice(n // 4, n - n // 3)
    none = torch.ones(n, dtype=torch.bool, device="cuda")
    none[live] = False
    fine = torch.nan_to_num(x.float(), posinf=1.0)      # for the bounds alone
    exact, relative = po.gate(x, act), po.gate_relative(x, act)
    bound = po.gate_bound(exact, exact.abs(), relative, fine, dtype)
    got = rs.gate_rows(x, act=act)
    close(got, exact, bound, "gate")
    part = rs.gate_rows(x, o, act)
    assert torch.equal(part[live].nan_to_num(), got[live].nan_to_num()) and (part[none] == 0).all()
    wide = torch.full((n, F + 3), 4.0, dtype=DTYPES[dtype], device="cuda")
    rs.gate_rows(torch.cat([x, x], 1)[:, :2 * F], o, act, out=wide[:, 1:F + 1])
    assert torch.equal(wide[live, 1:F + 1].nan_to_num(), got[live].nan_to_num())
    assert (wide[none] == 4).all() and (wide[:, 0] == 4).all() and (wide[:, F + 1:] == 4).all()
    exact, size = po.gate_backward(g, x, act)
    bound = po.gate_bound(exact, size, torch.cat([relative, relative], 1), fine, dtype)
    got = rs.gate_rows_backward(g, x, act=act)
    close(got, exact, bound, "gradient")
    part = rs.gate_rows_backward(g, x, o, act)
    assert torch.equal(part[live].nan_to_num(), got[live].nan_to_num()) and (part[none] == 0).all()
    # In 8 bits: the gated rows in float32, then as quantize_rows.
    x = torch.nan_to_num(x, posinf=1.0)
    v, scale = po.quantized(po.gate(x, act))
    moved = float((po.gate_relative(x, act)).max()) * 2 + 4 * po.STEP32
    q, s = rs.gate_quantize_rows(x, act=act)
    close(s, scale, scale * moved, "scales")
    close(q, v, po.quantized_bound(v) + v.abs() * moved, "values")
    part = rs.gate_quantize_rows(x, o, act)
    assert torch.equal(part.values.view(torch.uint8)[live], q.view(torch.uint8)[live])
    assert torch.equal(part.scales[:, live], s[:, live]) and (part.values.view(torch.uint8)[none] == 0).all()


# ---------------------------------------------------------------------------
# Refusals that need device tensors
# ---------------------------------------------------------------------------
def test_refusals():
    note("refusals")
    x, w, g = torch.randn(6, 32, device="cuda"), torch.randn(2, 16, 32, device="cuda"), torch.randn(6, 16, device="cuda")
    o = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    (q, qs), (w8, ws) = rs.quantize_rows(x), rs.quantize_weights(w)
    value = [lambda: rs.expert_products(x, None, w), lambda: rs.expert_products(x, o[:2], w),
             lambda: rs.expert_products(x[:, :30], o, w), lambda: rs.expert_products(x, o, w[0]),
             lambda: rs.expert_products(x[:, ::2], o, w[:, :, :16]), lambda: rs.expert_products(x, o, w.transpose(1, 2)),
             lambda: rs.expert_products(x, o, w, out=g[:5]), lambda: rs.expert_products(x, o.cpu(), w),
             lambda: rs.expert_products(x, o, w.cpu()), lambda: rs.expert_products(x, o, w[:0]),
             lambda: rs.expert_products_backward(g, o), lambda: rs.expert_products_backward(g, o, w, x[:5]),
             lambda: rs.expert_products_backward(x, o, w), lambda: rs.expert_products_backward(g, o, w, x[:, :31]),
             lambda: rs.expert_products_backward(g, o, rows=x, out=x), lambda: rs.expert_products_backward(g, o, w, out=g),
             lambda: rs.expert_products_backward(g, o, w, grad_weights_out=w),
             lambda: rs.expert_products_backward(g, o, w, x, grad_weights_out=w[:1]),
             lambda: rs.expert_products_backward(g, o[:1], rows=x), lambda: rs.expert_products_backward(g, o[None], rows=x),
             lambda: rs.expert_products_fp8(q, qs[:, :5], o, w8, ws), lambda: rs.expert_products_fp8(q, qs, o, w8, ws[:1]),
             lambda: rs.expert_products_fp8(q, qs, None, w8, ws), lambda: rs.expert_products_fp8(q[:, :30], qs, o, w8, ws),
             lambda: rs.quantize_rows(x, out=q), lambda: rs.quantize_rows(x, scales_out=qs),
             lambda: rs.quantize_rows(x, out=q[:5], scales_out=qs), lambda: rs.quantize_rows(x[0]),
             lambda: rs.quantize_rows(x, o[:1]), lambda: rs.quantize_weights(w[0]),
             lambda: rs.gate_rows(x[:, :31]), lambda: rs.gate_rows(x, act="relu"), lambda: rs.gate_rows(x, out=x),
             lambda: rs.gate_rows_backward(x, x), lambda: rs.gate_rows(x[:, :0]),
             lambda: rs.gate_quantize_rows(x, act="tanh"), lambda: rs.gate_quantize_rows(x[:, :31])]
    kind = [lambda: rs.expert_products(x, o, w.half()), lambda: rs.expert_products(x, o.long(), w),
            lambda: rs.expert_products(x.double(), o, w.double()), lambda: rs.expert_products(x, o, w, out=g.half()),
            lambda: rs.expert_products_backward(g, o, w.half()), lambda: rs.expert_products_backward(g, o, w, x.half()),
            lambda: rs.expert_products_fp8(x, qs, o, w8, ws), lambda: rs.expert_products_fp8(q, qs, o, w, ws),
            lambda: rs.expert_products_fp8(q, qs.half(), o, w8, ws), lambda: rs.expert_products_fp8(q, qs, o, w8, ws, FP8),
            lambda: rs.quantize_rows(q), lambda: rs.gate_rows(o[None]), lambda: rs.gate_rows(x, [0, 6]),
            lambda: rs.gate_rows_backward(g.half(), x), lambda: rs.quantize_weights([w])]
    status = [lambda: rs.expert_products(x, o, torch.randn(2, 32, 32, device="cuda"), out=x),
              lambda: rs.expert_products_backward(g, o, w, x, out=x),
              lambda: rs.expert_products_backward(g, o, w, x, grad_weights_out=w),
              lambda: rs.gate_rows_backward(x[:, :16], x, out=x),
              lambda: rs.expert_products(x.expand(6, 32), o, w, out=x[:1, :16].expand(6, 16))]
    for error, calls in ((ValueError, value), (TypeError, kind), (rs.RadixSortError, status)):
        for i, call in enumerate(calls):
            with pytest.raises(error):
                print(error, i, call())
    leaf = x.clone().requires_grad_()
    for call in (lambda: rs.expert_products(leaf, o, w), lambda: rs.expert_products(x, o, w.clone().requires_grad_()),
                 lambda: rs.gate_rows(leaf), lambda: rs.quantize_rows(leaf), lambda: rs.gate_quantize_rows(leaf)):
        with pytest.raises(ValueError, match="gradient"):
            call()
        with torch.no_grad():
            call()
    import torch.autograd.forward_ad as fwd
    with fwd.dual_level():
        dual = fwd.make_dual(x, torch.ones_like(x))
        for call in (lambda: rs.expert_products(dual, o, w), lambda: rs.gate_rows(dual), lambda: rs.quantize_rows(dual)):
            with pytest.raises(ValueError, match="tangent"):
                call()


# ---------------------------------------------------------------------------
# A layer, as it is used
# ---------------------------------------------------------------------------
class Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, position):
        ctx.save_for_backward(position)
        return rs.dispatch_rows(x, position)

    @staticmethod
    def backward(ctx, grad):
        return rs.dispatch_rows_backward(grad.contiguous(), *ctx.saved_tensors), None


class Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, position, w):
        ctx.save_for_backward(rows, position, w)
        return rs.combine_rows(rows, position, w)

    @staticmethod
    def backward(ctx, grad):
        rows, position, w = ctx.saved_tensors
        grad_rows, grad_w = rs.combine_rows_backward(grad.contiguous(), position, rows, w)
        return grad_rows, None, grad_w


class Products(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, offsets, weights):
        ctx.save_for_backward(rows, offsets, weights)
        return rs.expert_products(rows, offsets, weights)

    @staticmethod
    def backward(ctx, grad):
        rows, offsets, weights = ctx.saved_tensors
        grad_rows, grad_w = rs.expert_products_backward(grad.contiguous(), offsets, weights, rows)
        return grad_rows, None, grad_w


class Gate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, offsets):
        ctx.save_for_backward(rows, offsets)
        return rs.gate_rows(rows, offsets)

    @staticmethod
    def backward(ctx, grad):
        rows, offsets = ctx.saved_tensors
        return rs.gate_rows_backward(grad.contiguous(), rows, offsets), None


def layer(x, logits, w_up, w_down, k, first=0):
    w, e = rs.route_topk(logits, k, renormalize=True)
    s = rs.sort_experts(e, w_up.shape[0], first_expert=first)
    rows = Dispatch.apply(x, s.position)
    h = Gate.apply(Products.apply(rows, s.offsets, w_up), s.offsets)
    return Combine.apply(Products.apply(h, s.offsets, w_down), s.position, w), (w, e)


@pytest.mark.parametrize("T,E,k,H,F,first", [(50, 6, 2, 40, 24, 0), (33, 5, 3, 17, 9, 2), (300, 4, 2, 96, 128, 1)])
def test_layer_gradients(T, E, k, H, F, first):
    """Output and gradients of a whole layer, some experts another rank's, against
    the same layer in 64 bits by autograd.  Every value passes sums of at most
    H + 2 F + k + 2 E k T terms' depth; their steps bound its relative error in norm."""
    note(f"layer T={T} E={E}")
    gen = generator(T)
    x, logits = normal(gen, (T, H), "float32"), normal(gen, (T, E + first), "float32")
    up, down = normal(gen, (E, 2 * F, H), "float32", H ** -0.5), normal(gen, (E, H, F), "float32", F ** -0.5)
    g = normal(gen, (T, H), "float32")
    mine = [t.clone().requires_grad_() for t in (x, up, down)]
    out, (w, e) = layer(mine[0], logits, mine[1], mine[2], k, first)
    out.backward(g)
    other = [t.double().requires_grad_() for t in (x, up, down)]
    want = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for i in range(E):
        for j in range(k):
            take = (e[:, j] == first + i).nonzero()[:, 0]
            a, b = (other[0][take] @ other[1][i].t()).chunk(2, 1)
            rows = (a * torch.sigmoid(a) * b) @ other[2][i].t()
            want = want.index_add(0, take, rows * w[take, j, None].double())
    want.backward(g.double())
    bound = (H + 2 * F + k * T + 64) * po.STEP32
    for name, a, b in [("out", out, want)] + [(f"gradient {i}", p.grad, q.grad) for i, (p, q) in
                                              enumerate(zip(mine, other))]:
        far = float((a.detach().double() - b.detach()).norm() / b.detach().norm())
        assert far < bound, f"{name}: {far} over {bound}"


def run_all(x, position, offsets, up, down, up8, down8, w, g, b):
    """Forward in both forms and backward, into buffers."""
    rs.dispatch_rows(x, position, out=b["rows"])
    rs.expert_products(b["rows"], offsets, up, out=b["up"])
    rs.gate_rows(b["up"], offsets, out=b["h"])
    rs.expert_products(b["h"], offsets, down, out=b["down"])
    rs.combine_rows(b["down"], position, w, out=b["out"])
    rs.combine_rows_backward(g, position, b["down"], w, out=b["gdown"], grad_weights_out=b["gw"])
    rs.expert_products_backward(b["gdown"], offsets, down, b["h"], out=b["gh"], grad_weights_out=b["gdownw"])
    rs.gate_rows_backward(b["gh"], b["up"], offsets, out=b["gup"])
    rs.expert_products_backward(b["gup"], offsets, up, b["rows"], out=b["grows"], grad_weights_out=b["gupw"])
    rs.dispatch_rows_backward(b["grows"], position, out=b["gx"])
    rs.quantize_rows(b["rows"], offsets, out=b["q"].view(FP8), scales_out=b["qs"])
    rs.expert_products_fp8(b["q"].view(FP8), b["qs"], offsets, *up8, out=b["up8"])
    rs.gate_quantize_rows(b["up8"], offsets, out=b["q2"].view(FP8), scales_out=b["q2s"])
    rs.expert_products_fp8(b["q2"].view(FP8), b["q2s"], offsets, *down8, out=b["down8"])


def buffers(T, k, E, H, F):
    def new(*shape, dtype=torch.bfloat16):
        return torch.zeros(*shape, dtype=dtype, device="cuda")
    n = T * k
    return {"rows": new(n, H), "up": new(n, 2 * F), "h": new(n, F), "down": new(n, H), "out": new(T, H), "gdown": new(n, H),
            "gw": new(T, k, dtype=torch.float32), "gh": new(n, F), "gdownw": new(E, H, F), "gup": new(n, 2 * F),
            "grows": new(n, H), "gupw": new(E, 2 * F, H), "gx": new(T, H), "q": new(n, H, dtype=torch.uint8),
            "qs": new((H + 127) // 128, n, dtype=torch.float32), "up8": new(n, 2 * F), "q2": new(n, F, dtype=torch.uint8),
            "q2s": new((F + 127) // 128, n, dtype=torch.float32), "down8": new(n, H)}


def layer_inputs(gen, T, k, E, H, F):
    w, e = rs.route_topk(normal(gen, (T, E), "float32"), k)
    s = rs.sort_experts(e, E)
    up, down = normal(gen, (E, 2 * F, H), "bfloat16", H ** -0.5), normal(gen, (E, H, F), "bfloat16", F ** -0.5)
    return [normal(gen, (T, H), "bfloat16"), s.position, s.offsets, up, down, rs.quantize_weights(up),
            rs.quantize_weights(down), w, normal(gen, (T, H), "bfloat16")]


LAYERS = [(3, 2, 16, 256, 128), (600, 3, 4, 200, 136)]


@pytest.mark.parametrize("T,k,E,H,F", LAYERS)
def test_layer_in_graphs(T, k, E, H, F):
    """Two captured graphs, replayed in turn with eager work between: every replay
    equals the eager result."""
    note(f"layer in graphs T={T}")
    gen = generator(T)
    stat = layer_inputs(gen, T, k, E, H, F)
    bufs = [buffers(T, k, E, H, F) for _ in range(2)]
    run_all(*stat, buffers(T, k, E, H, F))
    torch.cuda.synchronize()
    graphs = []
    for b in bufs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run_all(*stat, b)
        graphs.append(graph)
    for i in range(5):
        for to, new in zip(stat, layer_inputs(generator(100 + i), T, k, E, H, F)):
            for p, q in zip(to, new) if isinstance(to, tuple) else [(to, new)]:
                p.view(torch.uint8).copy_(q.view(torch.uint8))
        graphs[i % 2].replay()
        eager = buffers(T, k, E, H, F)
        run_all(*stat, eager)
        torch.cuda.synchronize()
        for name in eager:
            assert torch.equal(bufs[i % 2][name], eager[name]), f"replay {i}: {name}"


def test_layer_on_streams_and_threads():
    """Two host threads, a stream each, at once, equal one; and again the same."""
    note("threads and streams")
    import threading
    sizes = (500, 3, 6, 256, 136)
    inputs = [layer_inputs(generator(i), *sizes) for i in range(2)]
    want = [buffers(*sizes) for _ in range(2)]
    for p, b in zip(inputs, want):
        run_all(*p, b)
    torch.cuda.synchronize()
    got = [[buffers(*sizes) for _ in range(4)] for _ in range(2)]
    torch.cuda.synchronize()
    errors = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for b in got[i]:
                    run_all(*inputs[i], b)
                torch.cuda.current_stream().synchronize()
        except Exception as e:      # reported below: a thread's own is only printed
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for i in range(2):
        for b in got[i]:
            for name in b:
                assert torch.equal(b[name], want[i][name]), name


def test_given_stream():
    """A call on a given stream, with outputs that it allocates."""
    note("given stream")
    sizes = (100, 2, 4, 64, 40)
    x, position, offsets, up, down, up8, _, w, g = layer_inputs(generator(1), *sizes)
    rows = rs.dispatch_rows(x, position)
    want = [rs.expert_products(rows, offsets, up), rs.gate_rows(rs.expert_products(rows, offsets, up), offsets),
            *rs.quantize_rows(rows, offsets), *rs.expert_products_backward(rows, offsets, down, g.new_ones(200, 40))]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    ones = g.new_ones(200, 40)
    s.wait_stream(torch.cuda.current_stream())
    y = rs.expert_products(rows, offsets, up, stream=s)
    got = [y, rs.gate_rows(y, offsets, stream=s), *rs.quantize_rows(rows, offsets, stream=s),
           *rs.expert_products_backward(rows, offsets, down, ones, stream=s)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_kernel_timing():
    """The calls' launches are timed under their own kernel kinds."""
    note("kernel timing")
    from lsd_radix_sort_pass_amd import _lib
    x, w = torch.randn(64, 32, device="cuda"), torch.randn(1, 16, 32, device="cuda")
    rs.prof_reset()
    rs.prof_enable(True)
    try:
        y = rs.expert_products(x, None, w)
        rs.gate_rows_backward(rs.gate_rows(y), y)
        q, w8 = rs.quantize_rows(x), rs.quantize_weights(w)
        rs.expert_products_fp8(*q, None, *w8)
        rs.expert_products_backward(y, None, w, x)
    finally:
        rs.prof_enable(False)
    counts = [rs.prof_summary(kind)[0] for kind in (_lib.RS_KERNEL_PRODUCT, _lib.RS_KERNEL_GATE, _lib.RS_KERNEL_QUANTIZE)]
    assert counts[0] >= 4 and counts[1:] == [2, 2]
    rs.prof_reset()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "8 bits"])
@pytest.mark.parametrize("N,K", [(264, 208), (520, 8), (136, 1008)])
def test_products_tiles_of_every_height(N, K, dtype):
    """Experts whose last tile has any number of rows, among many stages and one."""
    note(f"heights {dtype} N={N} K={K}")
    counts = [1, 31, 32, 33, 63, 64, 65, 96, 100, 127, 128, 129, 160, 191, 192, 193, 224, 255, 256, 300, 0, 513]
    E, n, gen = len(counts), sum(counts) + 70, generator(N)
    o = torch.tensor([40] + counts, device="cuda").cumsum(0).to(torch.int32)
    s = po.spans(o, E, n)
    if dtype == "8 bits":
        (q, qs), (w, ws) = eight_bits(gen, n, E, N, K)
        x, m, none = po.expand(q, qs), po.expand_weights(w, ws), torch.zeros(n, N, device="cuda")
        exact, size = po.product(x, s, m, none)
        lost = po.fp8_lost(x, s, m, none)
        for out in DTYPES:
            bound = po.product_bound(exact, size, K // 32 + 8, out) + lost
            close(rs.expert_products_fp8(q, qs, o, w, ws, DTYPES[out]), exact, bound, out)
        return
    x, w, g = normal(gen, (n, K), dtype), normal(gen, (E, N, K), dtype, K ** -0.5), normal(gen, (n, N), dtype)
    exact, size = po.product(x, s, w, torch.zeros(n, N, device="cuda"))
    close(rs.expert_products(x, o, w), exact, po.product_bound(exact, size, K, dtype), "product")
    grad_rows, grad_w = rs.expert_products_backward(g, o, w, x)
    exact, size = po.product_rows_backward(g, s, w, torch.zeros(n, K, device="cuda"))
    close(grad_rows, exact, po.product_bound(exact, size, N, dtype), "gradient of rows")
    exact, size = po.product_weights_backward(g, s, x)
    close(grad_w, exact, po.product_bound(exact, size, n, dtype), "gradient of weights")
