"""Argument checks of the experts' products, 8-bit rows and gated rows that need no
GPU, and their oracle against values worked by hand and differences.  (Pointers
below are fake addresses: every call must return before touching them.)"""
import pytest

from lsd_radix_sort_pass_amd import _lib

torch = pytest.importorskip("torch")
rs = pytest.importorskip("lsd_radix_sort_pass_amd")
import product_oracle as po  # noqa: E402

OK, INVALID = _lib.RS_SUCCESS, _lib.RS_ERROR_INVALID_VALUE
A, B, C, D, E, F = (i << 40 for i in range(1, 7))
n, K, N, EXPERTS = 100, 64, 48, 8
F32, F16, BF16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


GROUPS = (dict(experts=0), dict(experts=1025), dict(experts=-1), dict(offsets=None), dict(offsets=B + 2), dict(rows_n=2**31),
          dict(rows_n=2**30 + 1))


def test_product_checks(lib):
    def call(rows=A, dtype=F16, rows_n=n, width=K, rs_=K, offsets=B, experts=EXPERTS, w=C, wide=N, ws=K, we=K * N, out=D,
             os=N):
        return lib.rs_expert_products(rows, dtype, rows_n, width, rs_, offsets, experts, w, wide, ws, we, out, os, 0, None)
    for bad in GROUPS + (dict(dtype=3), dict(dtype=-1), dict(width=0), dict(width=2**20 + 1), dict(wide=0),
                         dict(wide=2**20 + 1), dict(rows=None), dict(rows=A + 1), dict(w=None), dict(w=C + 1),
                         dict(out=None), dict(out=D + 1), dict(os=N - 1), dict(out=A), dict(out=A + n * K * 2 - 2),
                         dict(out=C + 64), dict(out=B), dict(ws=2**41), dict(we=2**51), dict(rs_=2**41)):
        assert call(**bad) == INVALID, bad
    assert call(rows_n=0, rows=None, out=None) == OK
    assert call(rows_n=0, rows=None, out=None, offsets=None, experts=1) == OK


def test_product_backward_checks(lib):
    def call(g=A, dtype=BF16, rows_n=n, wide=N, gs=N, offsets=B, experts=EXPERTS, w=C, ws=K, we=K * N, x=D, xs=K, width=K,
             gr=E, grs=K, gw=F):
        return lib.rs_expert_products_backward(g, dtype, rows_n, wide, gs, offsets, experts, w, ws, we, x, xs, width, gr,
                                               grs, gw, 0, None)
    for bad in GROUPS + (dict(dtype=3), dict(width=0), dict(width=2**20 + 1), dict(wide=0), dict(wide=2**20 + 1),
                         dict(g=None), dict(g=A + 1), dict(w=None), dict(w=C + 1), dict(x=None), dict(x=D + 1),
                         dict(gr=E + 1), dict(gw=F + 1), dict(grs=K - 1), dict(gr=A), dict(gr=B), dict(gr=C), dict(gr=D),
                         dict(gw=A), dict(gw=B), dict(gw=C + 2), dict(gw=D), dict(gw=E + 2), dict(ws=2**41),
                         dict(we=2**51), dict(xs=2**41)):
        assert call(**bad) == INVALID, bad
    assert call(gr=None, gw=None) == OK
    assert call(rows_n=0, g=None, x=None, gr=E, gw=None) == OK


def test_fp8_checks(lib):
    G = 7 << 40

    def call(rows=A, scales=G, rows_n=n, width=K, rs_=K, offsets=B, experts=EXPERTS, w=C, wscales=F, wide=N, ws=K, we=K * N,
             out=D, dtype=BF16, os=N):
        return lib.rs_expert_products_fp8(rows, scales, rows_n, width, rs_, offsets, experts, w, wscales, wide, ws, we, out,
                                          dtype, os, 0, None)
    for bad in GROUPS + (dict(dtype=3), dict(width=0), dict(wide=0), dict(rows=None), dict(w=None), dict(scales=None),
                         dict(wscales=None), dict(scales=G + 2), dict(wscales=F + 1), dict(out=None), dict(out=D + 1),
                         dict(os=N - 1), dict(out=A), dict(out=C), dict(out=G), dict(out=F), dict(out=B)):
        assert call(**bad) == INVALID, bad
    assert call(rows_n=0, rows=None, out=None, scales=None) == OK


def test_quantize_and_gate_checks(lib):
    def q(x=A, dtype=F32, rows_n=n, width=K, xs=K, offsets=B, experts=EXPERTS, out=C, os=K, scales=D):
        return lib.rs_quantize_rows(x, dtype, rows_n, width, xs, offsets, experts, out, os, scales, 0, None)

    def gq(x=A, dtype=F32, rows_n=n, width=K, xs=2 * K, offsets=B, experts=EXPERTS, out=C, os=K, scales=D, act=0):
        return lib.rs_gate_quantize_rows(x, dtype, rows_n, width, xs, offsets, experts, act, out, os, scales, 0, None)

    def gate(x=A, dtype=F32, rows_n=n, width=K, xs=2 * K, offsets=B, experts=EXPERTS, out=C, os=K, act=0):
        return lib.rs_gate_rows(x, dtype, rows_n, width, xs, offsets, experts, act, out, os, 0, None)

    def back(g=E, x=A, dtype=F32, rows_n=n, width=K, xs=2 * K, offsets=B, experts=EXPERTS, out=C, os=2 * K, act=0, gs=K):
        return lib.rs_gate_rows_backward(g, gs, x, dtype, rows_n, width, xs, offsets, experts, act, out, os, 0, None)
    common = GROUPS + (dict(dtype=3), dict(width=0), dict(x=None), dict(x=A + 2), dict(out=None), dict(out=A), dict(out=B),
                       dict(os=K - 1), dict(xs=2**41))
    for call, more in ((q, (dict(width=2**20 + 1), dict(scales=None), dict(scales=D + 2), dict(scales=C), dict(scales=A))),
                       (gq, (dict(width=2**19 + 1), dict(act=2), dict(act=-1), dict(scales=None), dict(scales=C))),
                       (gate, (dict(width=2**19 + 1), dict(act=2), dict(out=C + 2))),
                       (back, (dict(width=2**19 + 1), dict(act=2), dict(g=None), dict(g=E + 1), dict(out=E),
                               dict(os=2 * K - 1)))):
        for bad in common + more:
            assert call(**bad) == INVALID, (call.__name__, bad)
    assert q(rows_n=0, x=None, out=None, scales=None) == OK
    assert gate(rows_n=0, x=None, out=None) == OK

    def weights(w=A, dtype=BF16, experts=EXPERTS, wide=N, width=K, ws=K, we=N * K, out=B, scales=C):
        return lib.rs_quantize_weights(w, dtype, experts, wide, width, ws, we, out, scales, None)
    for bad in (dict(dtype=3), dict(experts=0), dict(experts=1025), dict(wide=0), dict(width=0), dict(wide=2**20 + 1),
                dict(w=None), dict(w=A + 1), dict(out=None), dict(scales=None), dict(scales=C + 1), dict(out=A),
                dict(scales=B), dict(scales=A), dict(ws=2**41)):
        assert weights(**bad) == INVALID, bad


def test_python_refuses_host_tensors():
    x, o = torch.zeros(4, 8), torch.zeros(3, dtype=torch.int32)
    w = torch.zeros(2, 4, 8)
    q = torch.zeros(4, 8).to(torch.float8_e4m3fn)
    for call in (lambda: rs.expert_products(x, o, w), lambda: rs.expert_products_backward(x, o, w),
                 lambda: rs.expert_products_fp8(q, x, o, w, w), lambda: rs.quantize_rows(x), lambda: rs.quantize_weights(w),
                 lambda: rs.gate_rows(x), lambda: rs.gate_rows_backward(x, x), lambda: rs.gate_quantize_rows(x)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: rs.expert_products([1.0], o, w), lambda: rs.quantize_weights(None), lambda: rs.gate_rows("rows"),
                 lambda: rs.expert_products_fp8(x, x, o, w, w)):
        with pytest.raises((TypeError, ValueError)):
            call()


def test_constants_match_the_header():
    src = open(__file__.replace("tests/test_products_abi.py", "include/rs.h")).read()
    assert f"#define RS_SCALE_BLOCK {rs.SCALE_BLOCK}\n" in src
    assert "#define RS_MAX_PRODUCT_ROWS ((size_t)1 << 30)\n" in src


# The oracle itself.
def test_oracle_products():
    x = torch.tensor([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0], [7.0, 8.0]])
    w = torch.tensor([[[1.0, 0.0]], [[0.0, 2.0]], [[1.0, -1.0]]])
    s = po.spans(torch.tensor([1, 1, 3, 3]), 3, 4)
    assert s == [(1, 1), (1, 3), (3, 3)]
    out, size = po.product(x, s, w, torch.full((4, 1), 9.0))
    assert out[:, 0].tolist() == [9.0, 8.0, 12.0, 9.0] and size[:, 0].tolist() == [0.0, 8.0, 12.0, 0.0]
    assert po.spans(None, 1, 4) == [(0, 4)] and po.spans(torch.tensor([-5, 9, 2]), 2, 4) == [(0, 4), (4, 4)]


def test_oracle_product_gradients_match_differences():
    """The product is linear in rows and in weights: a difference of any step is the
    gradient, but for rounding in 64 bits."""
    gen = torch.Generator().manual_seed(1)
    x, w, g = (torch.randn(s, generator=gen, dtype=torch.float64) for s in ((7, 5), (3, 4, 5), (7, 4)))
    s = po.spans(torch.tensor([1, 3, 3, 6]), 3, 7)
    zero = torch.zeros(7, 4)

    def loss(x, w):
        return float((po.product(x, s, w, zero)[0] * g).sum())
    gx = po.product_rows_backward(g, s, w, torch.zeros(7, 5))[0]
    gw = po.product_weights_backward(g, s, x)[0]
    for i in range(x.numel()):
        d = torch.zeros(x.numel(), dtype=torch.float64)
        d[i] = 1.0
        d = d.reshape(x.shape)
        assert abs(loss(x + d, w) - loss(x, w) - float((gx * d).sum())) < 1e-12
    for i in range(w.numel()):
        d = torch.zeros(w.numel(), dtype=torch.float64)
        d[i] = 1.0
        d = d.reshape(w.shape)
        assert abs(loss(x, w + d) - loss(x, w) - float((gw * d).sum())) < 1e-12


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_oracle_gate_gradient_matches_differences(kind):
    """Central differences with step h: truncation h^2 / 6 times a third derivative
    (below 4 here), rounding 2^-52 / h, both far below 1e-8."""
    gen = torch.Generator().manual_seed(2)
    x, g = torch.randn(3, 10, generator=gen, dtype=torch.float64) * 2, torch.randn(3, 5, generator=gen, dtype=torch.float64)
    grad, h = po.gate_backward(g, x, kind)[0], 1e-5
    for i in range(30):
        d = torch.zeros(30, dtype=torch.float64)
        d[i] = h
        d = d.reshape(x.shape)
        slope = ((po.gate(x + d, kind) - po.gate(x - d, kind)) * g).sum() / (2 * h)
        assert abs(float(slope - grad.reshape(-1)[i])) < 1e-8
    assert abs(float(po.act(torch.tensor(1.0, dtype=torch.float64), "silu")[0]) - 0.7310585786300049) < 1e-15
    assert abs(float(po.act(torch.tensor(1.0, dtype=torch.float64), "gelu")[0]) - 0.8413447460685429) < 1e-15


def test_oracle_quantized():
    x = torch.zeros(2, 130, dtype=torch.float64)
    x[0, 3], x[0, 129], x[1, 5], x[1, 6] = -896.0, 7.0, float("inf"), 1.0
    v, s = po.quantized(x)
    assert s.shape == (2, 2) and s[0].tolist() == [2.0, 1.0 / 448] and s[1].tolist() == [7.0 / 448, 2.0 ** -100 / 448]
    assert v[0, 3] == -448.0 and v[0, 129] == 448.0 and v[1, 6] == 448.0
    assert torch.equal(po.expand(v, s)[0], x[0])
