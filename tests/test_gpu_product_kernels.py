"""GPU tests of each kernel of the experts' products by itself, at sizes where it can go
wrong, whichever kernel the library would choose for them; and of the kernels that
it chooses for the sizes that each is made for."""
import contextlib

import pytest

import product_oracle as po

torch = pytest.importorskip("torch")
rs = pytest.importorskip("lsd_radix_sort_pass_amd")
from lsd_radix_sort_pass_amd import _lib  # noqa: E402
from test_gpu_products import DTYPES, FP8, close, generator, normal, note, offsets_of  # noqa: E402

pytestmark = pytest.mark.gpu

SQUARE, FEW, SPLIT, WIDE = _lib.RS_PRODUCT_SQUARE, _lib.RS_PRODUCT_FEW, _lib.RS_PRODUCT_SPLIT, _lib.RS_PRODUCT_WIDE
NAMES = {"square": SQUARE, "few": FEW, "split": SPLIT, "wide": WIDE}
FEW_TAGS = {(rows, strips): FEW + 16 * rows + 256 * strips for rows in (1, 2, 4) for strips in (1, 2)}
HALVES = ["float16", "bfloat16"]


@contextlib.contextmanager
def forced(kernel):
    before = rs.prof_product_kernel(kernel)
    try:
        yield
    finally:
        rs.prof_product_kernel(before)


def launched(call):
    """The call's result and the tags of the product kernels that it launched."""
    rs.prof_reset()
    rs.prof_enable(True)
    try:
        res = call()
    finally:
        rs.prof_enable(False)
    tags = [t for t in (SQUARE, SPLIT, WIDE, *FEW_TAGS.values())
            for _ in range(len(rs.prof_samples(_lib.RS_KERNEL_PRODUCT, t)))]
    assert len(tags) == rs.prof_summary(_lib.RS_KERNEL_PRODUCT)[0]
    rs.prof_reset()
    return res, tags


def runs(call, kernel):
    """The result of a call that is seen to launch nothing but that kernel."""
    res, tags = launched(call)
    assert tags and all(t == kernel or (kernel == FEW and t in FEW_TAGS.values()) for t in tags), (kernel, tags)
    return res


def check_product(kernel, x, o, w, dtype):
    n, N, K = x.shape[0], w.shape[1], x.shape[1]
    s = po.spans(o, w.shape[0], n)
    wide = torch.full((n, N + 3), 5.0, dtype=DTYPES[dtype], device="cuda")
    runs(lambda: rs.expert_products(x, o, w, out=wide[:, 1:N + 1]), kernel)
    exact, size = po.product(x, s, w, torch.full((n, N), 5.0, device="cuda"))
    bound = po.product_bound(exact, size, K, dtype)
    close(wide[:, 1:N + 1], exact, bound, "product to a given out")
    assert (wide[:, 0] == 5.0).all() and (wide[:, N + 1:] == 5.0).all()
    got = runs(lambda: rs.expert_products(x, o, w), kernel)
    none = torch.ones(n, dtype=torch.bool, device="cuda")
    for lo, hi in s:
        none[lo:hi] = False
    assert (got[none] == 0).all()
    assert torch.equal(got[~none].nan_to_num(), wide[:, 1:N + 1][~none].nan_to_num())


def check_gradient_of_rows(kernel, g, o, w, dtype):
    n, K = g.shape[0], w.shape[2]
    exact, size = po.product_rows_backward(g, po.spans(o, w.shape[0], n), w, torch.zeros(n, K, device="cuda"))
    got = runs(lambda: rs.expert_products_backward(g, o, w), kernel)
    close(got, exact, po.product_bound(exact, size, g.shape[1], dtype), "gradient of rows")


def check_gradient_of_weights(kernel, g, o, x, dtype):
    n, E = g.shape[0], len(o) - 1
    exact, size = po.product_weights_backward(g, po.spans(o, E, n), x)
    got = runs(lambda: rs.expert_products_backward(g, o, rows=x), kernel)
    close(got, exact, po.product_bound(exact, size, n, dtype), "gradient of weights")


def check(kernel, n, E, N, K, dtype, kind="holes", gradients=True):
    gen = generator(n + N + K)
    o = offsets_of(n, E, kind)
    x, w, g = normal(gen, (n, K), dtype), normal(gen, (E, N, K), dtype, K ** -0.5), normal(gen, (n, N), dtype)
    with forced(kernel):
        check_product(kernel, x, o, w, dtype)
        if gradients:
            check_gradient_of_rows(kernel, g, o, w, dtype)
            check_gradient_of_weights(kernel, g, o, x, dtype)


# Widths of one part of a stage of 64 elements, its first half, one stage, a rest behind one and
# several; tiles whose last columns are a part, that have waves without columns, several.
WIDE_SHAPES = [(300, 2, 8, 8), (700, 3, 264, 40), (700, 3, 136, 64), (1500, 4, 520, 72), (900, 2, 512, 136),
               (2100, 5, 152, 352), (1300, 1, 256, 1032), (600, 2, 1000, 200)]


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("n,E,N,K", WIDE_SHAPES)
def test_wide_products(n, E, N, K, dtype):
    note(f"wide {dtype} n={n} E={E} N={N} K={K}")
    check(WIDE, n, E, N, K, dtype)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("N,K", [(264, 208), (520, 8), (136, 1008)])
def test_wide_products_of_every_height(N, K, dtype):
    """Experts whose last tile has any number of rows, which is also the number of steps of
    the weights' gradient: tiles of up to 128 rows, and of up to 192 and 256."""
    note(f"wide, heights, {dtype} N={N} K={K}")
    counts = [1, 31, 32, 33, 63, 64, 65, 96, 100, 127, 128, 129, 160, 191, 192, 193, 224, 255, 256, 300, 0, 513]
    E, n, gen = len(counts), sum(counts) + 70, generator(N)
    o = torch.tensor([40] + counts, device="cuda").cumsum(0).to(torch.int32)
    x, w, g = normal(gen, (n, K), dtype), normal(gen, (E, N, K), dtype, K ** -0.5), normal(gen, (n, N), dtype)
    with forced(WIDE):
        check_product(WIDE, x, o, w, dtype)
        check_gradient_of_rows(WIDE, g, o, w, dtype)
        check_gradient_of_weights(WIDE, g, o, x, dtype)


@pytest.mark.parametrize("dtype", HALVES)
def test_wide_products_strided(dtype):
    """Rows and matrices among NaN, and rows of no expert that are NaN."""
    note(f"wide, strided {dtype}")
    gen = generator(3)
    n, E, N, K = 1300, 4, 264, 328
    o = offsets_of(n, E, "holes")
    lo, hi = int(o[0]), int(o[-1])
    for extra, begin in ((8, 0), (16, 8)):
        x = torch.full((2 * n, K + extra), float("nan"), dtype=DTYPES[dtype], device="cuda")[::2, begin:K + begin]
        w = torch.full((N, E, K + extra), float("nan"), dtype=DTYPES[dtype], device="cuda")[:, :, :K].transpose(0, 1)
        g = torch.full((n, N + extra), float("nan"), dtype=DTYPES[dtype], device="cuda")[:, begin:N + begin]
        x[lo:hi], g[lo:hi] = normal(gen, (hi - lo, K), dtype), normal(gen, (hi - lo, N), dtype)
        w.copy_(normal(gen, (E, N, K), dtype))
        with forced(WIDE):
            check_product(WIDE, x, o, w, dtype)
            check_gradient_of_rows(WIDE, g, o, w, dtype)
            check_gradient_of_weights(WIDE, g, o, x, dtype)


def test_wide_products_special_values():
    """NaN and infinities stay in their own rows and columns: others read them in no stage."""
    note("wide, special values")
    gen = generator(6)
    n, E, N, K = 700, 3, 264, 200
    o = torch.tensor([5, 300, 300, 690], dtype=torch.int32, device="cuda")
    x, w, g = normal(gen, (n, K), "bfloat16"), normal(gen, (E, N, K), "bfloat16"), normal(gen, (n, N), "bfloat16")
    x[10, 3], x[299, 199], w[2, 7, 0], w[2, 263, 199] = float("inf"), float("nan"), float("nan"), float("-inf")
    g[12, 39], g[689, 263] = float("-inf"), float("nan")
    w[1] = float("nan")                                          # an expert without rows
    with forced(WIDE):
        check_product(WIDE, x, o, w, "bfloat16")
        check_gradient_of_rows(WIDE, g, o, w, "bfloat16")
        check_gradient_of_weights(WIDE, g, o, x, "bfloat16")


def test_wide_products_far_apart():
    """Rows 2^22 elements apart, as many as the wide kernel takes, matrices 4 GiB apart."""
    note("wide, far apart")
    gen = generator(10)
    n, E, N, K, stride = 1200, 3, 272, 328, 1 << 22
    x = torch.empty((n - 1) * stride + K, dtype=torch.bfloat16, device="cuda").as_strided((n, K), (stride, 1))
    g = torch.empty((n - 1) * stride + N, dtype=torch.bfloat16, device="cuda").as_strided((n, N), (stride, 1))
    w = torch.empty(2 * (1 << 31) + N * K, dtype=torch.bfloat16, device="cuda").as_strided((E, N, K), (1 << 31, K, 1))
    x.copy_(normal(gen, (n, K), "bfloat16")), g.copy_(normal(gen, (n, N), "bfloat16"))
    w.copy_(normal(gen, (E, N, K), "bfloat16"))
    o = torch.tensor([0, 500, 510, 1100], dtype=torch.int32, device="cuda")
    with forced(WIDE):
        check_product(WIDE, x, o, w, "bfloat16")
        check_gradient_of_rows(WIDE, g, o, w, "bfloat16")
        check_gradient_of_weights(WIDE, g, o, x, "bfloat16")


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("n,E,N,K", [(70, 1, 130, 4100), (33, 2, 72, 2048), (200, 3, 65, 1537), (300, 2, 136, 72),
                                     (129, 1, 8, 8192), (1000, 6, 304, 264)])
def test_split_products(n, E, N, K, dtype):
    note(f"split {dtype} n={n} E={E} N={N} K={K}")
    check(SPLIT, n, E, N, K, dtype)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("n,E,N,K", [(1, 1, 1, 1), (130, 3, 129, 65), (300, 5, 136, 200), (513, 2, 640, 96),
                                     (1000, 6, 304, 1032), (40, 5, 3, 2)])
def test_square_products(n, E, N, K, dtype):
    note(f"square {dtype} n={n} E={E} N={N} K={K}")
    check(SQUARE, n, E, N, K, dtype)


# (rows, experts, N), and the kernel's form: rows of a tile / 16, output channels / 16.
FEW_FORMS = {(1, 1): (4, 1, 392), (2, 1): (20, 1, 392), (4, 1): (70, 1, 392), (1, 2): (16, 64, 1040), (2, 2): (320, 16, 1032),
             (4, 2): (800, 16, 1032)}
# Elements of a round of all waves' steps, by the form.
FEW_ROUND = {(1, 1): 16, (2, 1): 16, (4, 1): 8, (1, 2): 4, (2, 2): 4, (4, 2): 4}


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("form", list(FEW_FORMS))
def test_few_rows_products(form, dtype):
    """Several rounds of four steps a wave, which the workgroups begin at different places,
    and a rest of whole steps and a part of one."""
    n, E, N = FEW_FORMS[form]
    step = 32 if dtype == "float32" else 64
    K = 3 * 4 * FEW_ROUND[form] * step + 2 * step + 8
    note(f"few {dtype} {form} n={n} E={E} N={N} K={K}")
    gen = generator(n)
    o = offsets_of(n, E, "all")
    x, w = normal(gen, (n, K), dtype), normal(gen, (1, N, K), dtype, K ** -0.5)
    w = torch.cat([w * (1 + e % 3) for e in range(E)])
    s = po.spans(o, E, n)
    with forced(FEW):
        got, tags = launched(lambda: rs.expert_products(x, o, w))
    assert tags == [FEW_TAGS[form]]
    exact, size = po.product(x, s, w, torch.zeros(n, N, device="cuda"))
    close(got, exact, po.product_bound(exact, size, K, dtype), "product")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("n,E,N,K", [(17, 4, 33, 64), (300, 5, 136, 200), (64, 8, 256, 520), (700, 3, 257, 259), (9, 3, 40, 8)])
def test_few_rows_products_of_short_rows(n, E, N, K, dtype):
    note(f"few {dtype} n={n} E={E} N={N} K={K}")
    check(FEW, n, E, N, K, dtype, gradients=False)


# ---------------------------------------------------------------------------
# 8 bits
# ---------------------------------------------------------------------------
def scaled(gen, n, E, N, K):
    """Operands in 8 bits whose blocks all have scales of their own."""
    def values(*shape):
        return torch.randn(shape, generator=gen, device="cuda").mul_(60).clamp_(-448, 448).to(FP8)

    def scales(*shape):
        return torch.exp2(2 * torch.rand(shape, generator=gen, device="cuda") - 1)
    kb, nb = (K + 127) // 128, (N + 127) // 128
    return values(n, K), scales(kb, n), values(E, N, K), scales(E, nb, kb)


def check_fp8(kernel, n, E, N, K, o, dtype, tag=None):
    gen = generator(n + N + K)
    q, qs, w, ws = scaled(gen, n, E, N, K)
    s = po.spans(o, E, n)
    x, m, none = po.expand(q, qs), po.expand_weights(w, ws), torch.zeros(n, N, device="cuda")
    exact, size = po.product(x, s, m, none)
    bound = po.product_bound(exact, size, K // 32 + 8, dtype) + po.fp8_lost(x, s, m, none)
    if dtype == "float16":      # sizes from 65504 and half its step of 32 on round to infinity
        far = exact.abs() >= 65520
        bound = torch.where((exact.abs() - 65520).abs() <= bound, float("inf"), bound)
        exact = torch.where(far, exact.sign() * float("inf"), exact)
    wide = torch.full((n, N + 3), 5.0, dtype=DTYPES[dtype], device="cuda")
    with forced(kernel):
        got, tags = launched(lambda: rs.expert_products_fp8(q, qs, o, w, ws, DTYPES[dtype]))
        rs.expert_products_fp8(q, qs, o, w, ws, out=wide[:, 1:N + 1])
    assert tags == [tag or kernel], tags
    close(got, exact, bound, "product of 8 bits")
    lo, hi = int(o[0]), int(o[-1])
    assert torch.equal(wide[lo:hi, 1:N + 1], got[lo:hi]) and (got[:lo] == 0).all() and (got[hi:] == 0).all()
    assert (wide[:lo] == 5).all() and (wide[hi:] == 5).all() and (wide[:, 0] == 5).all() and (wide[:, N + 1:] == 5).all()


@pytest.mark.parametrize("n,E,N,K", [(300, 2, 8, 16), (700, 3, 264, 80), (700, 3, 136, 128), (1500, 4, 520, 144),
                                     (900, 2, 512, 272), (2100, 5, 152, 704), (1300, 1, 256, 1040)])
def test_wide_products_fp8(n, E, N, K):
    note(f"wide fp8 n={n} E={E} N={N} K={K}")
    check_fp8(WIDE, n, E, N, K, offsets_of(n, E, "holes"), "bfloat16")


# (The wide kernel serves bfloat16 results alone.)
@pytest.mark.parametrize("N,K", [(264, 400), (520, 16), (136, 1008)])
def test_wide_products_fp8_of_every_height(N, K):
    note(f"wide fp8, heights, N={N} K={K}")
    counts = [1, 31, 32, 33, 63, 64, 65, 96, 100, 127, 128, 129, 160, 191, 192, 193, 224, 255, 256, 300, 0, 513]
    o = torch.tensor([40] + counts, device="cuda").cumsum(0).to(torch.int32)
    check_fp8(WIDE, sum(counts) + 70, len(counts), N, K, o, "bfloat16")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("n,E,N,K", [(70, 1, 130, 4100), (33, 2, 72, 2048), (200, 3, 65, 1537), (300, 2, 136, 144)])
def test_split_products_fp8(n, E, N, K, dtype):
    note(f"split fp8 {dtype} n={n} E={E} N={N} K={K}")
    check_fp8(SPLIT, n, E, N, K, offsets_of(n, E, "holes"), dtype)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("n,E,N,K", [(3, 1, 5, 7), (130, 4, 129, 300), (900, 3, 520, 1040), (700, 3, 136, 16)])
def test_square_products_fp8(n, E, N, K, dtype):
    note(f"square fp8 {dtype} n={n} E={E} N={N} K={K}")
    check_fp8(SQUARE, n, E, N, K, offsets_of(n, E, "holes"), dtype)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("form", list(FEW_FORMS))
def test_few_rows_products_fp8(form, dtype):
    n, E, N = FEW_FORMS[form]
    if form[1] == 2:
        E, n, N = E // 4, n // 4, 4 * N
    K = 3 * 4 * FEW_ROUND[form] * 128 + 2 * 128 + 40
    note(f"few fp8 {dtype} {form} n={n} E={E} N={N} K={K}")
    check_fp8(FEW, n, E, N, K, offsets_of(n, E, "all"), dtype, FEW_TAGS[form])


# ---------------------------------------------------------------------------
# The library's choice
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("what,n,E,N,K,kernel", [
    ("product", 2400, 2, 2056, 1032, WIDE), ("rows", 4800, 4, 2056, 1032, WIDE), ("weights", 2400, 2, 2056, 1032, WIDE),
    ("fp8", 2400, 2, 2056, 1040, WIDE), ("product", 8, 64, 2048, 2088, FEW_TAGS[1, 2]),
    ("fp8", 16, 64, 2048, 4240, FEW_TAGS[1, 2]), ("product", 256, 1, 4096, 4096, SPLIT),
    ("weights", 8192, 1, 1024, 1024, SPLIT), ("product", 1000, 7, 1001, 1537, SPLIT), ("product", 5003, 7, 1001, 1537, SQUARE)])
def test_chosen_kernels(what, n, E, N, K, kernel):
    """The sizes that each kernel is made for."""
    note(f"chosen {what} n={n} E={E} N={N} K={K}")
    gen = generator(n)
    o = offsets_of(n, E, "all")
    s = po.spans(o, E, n)
    if what == "fp8":
        check_fp8(0, n, E, N, K, o, "bfloat16", kernel)
        return
    x, w, g = (normal(gen, shape, "bfloat16") for shape in ((n, K), (E, N, K), (n, N)))
    zeros = torch.zeros(n, K if what == "rows" else N, device="cuda")
    if what == "product":
        got, tags = launched(lambda: rs.expert_products(x, o, w))
        (exact, size), terms = po.product(x, s, w, zeros), K
    elif what == "rows":
        got, tags = launched(lambda: rs.expert_products_backward(g, o, w))
        (exact, size), terms = po.product_rows_backward(g, s, w, zeros), N
    else:
        got, tags = launched(lambda: rs.expert_products_backward(g, o, rows=x))
        (exact, size), terms = po.product_weights_backward(g, s, x), n
    assert tags == [kernel]
    close(got, exact, po.product_bound(exact, size, terms, "bfloat16"), what)


def test_forcing_falls_back():
    """A kernel that cannot serve a call is not taken for it."""
    note("forcing falls back")
    x, w = normal(generator(1), (50, 3), "float32"), normal(generator(2), (1, 5, 3), "float32")
    want = rs.expert_products(x, None, w)
    for kernel in (FEW, SPLIT, WIDE, 99):
        with forced(kernel):
            got, tags = launched(lambda: rs.expert_products(x, None, w))
        assert tags == [SQUARE] and torch.equal(got, want)
    assert rs.prof_product_kernel(0) == 0
