"""Argument checks of the mixture-of-experts calls that need no GPU: bad
arguments are rejected on the host before any HIP call.  (Pointers below are
fake addresses: every call here must return before touching them.)"""
import numpy as np
import pytest

import expert_oracle as eo
from lsd_radix_sort_pass_amd import _lib

torch = pytest.importorskip("torch")
rs = pytest.importorskip("lsd_radix_sort_pass_amd")

OK, INVALID, INSUFFICIENT = _lib.RS_SUCCESS, _lib.RS_ERROR_INVALID_VALUE, _lib.RS_ERROR_INSUFFICIENT_TEMP
A, B, C, D, E, F = (i << 40 for i in range(1, 7))
T, K, N, H = 100, 4, 400, 64
F32, F16, BF16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def test_route_checks(lib):
    def call(logits=A, dtype=BF16, tokens=T, experts=16, stride=16, k=K, gate=0, weights=B, chosen=C):
        return lib.rs_route_topk(logits, dtype, tokens, experts, stride, k, gate, 0, 1.0, weights, chosen, None)
    assert call(tokens=0, logits=None, weights=None, chosen=None) == OK
    for bad in (dict(dtype=3), dict(dtype=-1), dict(experts=0), dict(experts=1025, stride=1025), dict(k=0), dict(k=17),
                dict(k=65, experts=128, stride=128), dict(gate=2), dict(gate=-1), dict(logits=None), dict(weights=None),
                dict(chosen=None), dict(logits=A + 1), dict(weights=B + 2), dict(chosen=C + 2), dict(weights=A + 8),
                dict(chosen=B), dict(tokens=2**31), dict(stride=2**41), dict(tokens=0, experts=0),
                dict(tokens=2**29, k=1, stride=2**40)):        # no address range holds the rows
        assert call(**bad) == INVALID, bad

    def back(logits=A, dtype=BF16, tokens=T, experts=16, k=K, gate=1, chosen=B, g=C, grad=D, grad_stride=16):
        return lib.rs_route_topk_backward(logits, dtype, tokens, experts, 16, chosen, g, k, gate, 1, 1.0, grad,
                                          grad_stride, None)
    assert back(tokens=0, logits=None, chosen=None, g=None, grad=None) == OK
    for bad in (dict(dtype=3), dict(k=17), dict(gate=5), dict(logits=None), dict(chosen=None), dict(g=None),
                dict(grad=None), dict(grad=A), dict(grad=A + 64), dict(grad=B - 2), dict(grad_stride=15),
                dict(grad=D + 1), dict(g=C + 1)):
        assert back(**bad) == INVALID, bad


def test_sort_checks(lib):
    small, big = 8192, 100_000
    assert lib.rs_temp_bytes_experts(0, 8) == 0
    assert lib.rs_temp_bytes_experts(big, 0) == 0 and lib.rs_temp_bytes_experts(big, 1025) == 0
    assert lib.rs_temp_bytes_experts(2**31, 8) == 0
    need = lib.rs_temp_bytes_experts(big, 128)
    assert need > 0 and need % 256 == 0
    for name, size in (("rs_sort_experts_i32", 4), ("rs_sort_experts_i64", 8)):
        def call(ids=A, n=big, first=0, experts=128, order=B, position=C, offsets=D, temp=E, temp_bytes=need):
            return getattr(lib, name)(ids, n, first, experts, order, position, offsets, temp, temp_bytes, None)
        for bad in (dict(ids=None), dict(order=None), dict(position=None), dict(offsets=None), dict(temp=None),
                    dict(temp=E + 4), dict(experts=0), dict(experts=1025), dict(first=-1), dict(n=2**31),
                    dict(first=2**31 - 127), dict(ids=A + size // 2), dict(order=B + 2), dict(position=C + 1),
                    dict(offsets=D + 2), dict(order=A), dict(order=C + 4), dict(offsets=B + 40), dict(temp=A),
                    dict(temp=C + 256), dict(n=0, offsets=None)):
            assert call(**bad) == INVALID, bad
        assert call(temp_bytes=need - 1) == INSUFFICIENT
        assert call(n=small, ids=A, order=A) == INVALID


def test_row_checks(lib):
    def dispatch(x=A, dtype=F16, tokens=T, width=H, xs=H, position=B, weights=C, k=K, rows=D, num=N, rstride=H):
        return lib.rs_dispatch_rows(x, dtype, tokens, width, xs, position, weights, k, rows, num, rstride, None)

    def combine(rows=A, dtype=F16, num=N, rstride=H, position=B, weights=C, k=K, out=D, tokens=T, width=H, ostride=H):
        return lib.rs_combine_rows(rows, dtype, num, rstride, position, weights, k, out, tokens, width, ostride, None)
    common = (dict(dtype=3), dict(width=0), dict(width=2**20 + 1, ), dict(k=0), dict(k=65), dict(tokens=2**30),
              dict(num=2**31), dict(position=None), dict(position=B + 2), dict(weights=C + 2), dict(rows=None))
    for bad in common + (dict(x=None), dict(x=A + 1), dict(rows=D + 1), dict(rows=A), dict(rows=B - 64),
                         dict(rows=C + 16), dict(rstride=H - 1), dict(xs=2**41)):
        assert dispatch(**bad) == INVALID, bad
    for bad in common + (dict(out=None), dict(out=D + 1), dict(out=A + 128), dict(out=B - 2), dict(out=C),
                         dict(ostride=H - 1), dict(rows=A + 1)):
        assert combine(**bad) == INVALID, bad
    assert dispatch(tokens=0, x=None, position=None) == OK
    assert dispatch(num=0, rows=None) == OK
    assert combine(tokens=0, out=None, position=None) == OK

    def dback(x=E, gx=D, gw=F, **kw):
        a = dict(rows=A, dtype=F16, num=N, position=B, weights=C, k=K, tokens=T, width=H, xs=H, gs=H)
        a.update(kw)
        return lib.rs_dispatch_rows_backward(a["rows"], a["dtype"], a["num"], H, a["position"], a["weights"], a["k"],
                                             x, a["xs"], gx, a["gs"], gw, a["tokens"], a["width"], None)

    def cback(rows=E, gr=D, gw=F, **kw):
        a = dict(g=A, dtype=F16, num=N, position=B, weights=C, k=K, tokens=T, width=H, rs=H, gs=H)
        a.update(kw)
        return lib.rs_combine_rows_backward(a["g"], a["dtype"], a["tokens"], a["width"], H, a["position"],
                                            a["weights"], a["k"], rows, a["rs"], gr, a["gs"], a["num"], gw, None)
    for bad in (dict(x=None), dict(x=E + 1), dict(gw=F + 2), dict(gw=A), dict(gw=D), dict(gw=E + 4), dict(gx=E),
                dict(gx=None), dict(gs=H - 1), dict(rows=None), dict(gw=B), dict(gx=C)):
        assert dback(**bad) == INVALID, bad
    for bad in (dict(rows=None), dict(rows=E + 1), dict(gw=F + 2), dict(gw=A), dict(gw=D), dict(gw=E + 4),
                dict(gr=E), dict(gr=None), dict(gs=H - 1), dict(g=None), dict(gw=B), dict(gr=C)):
        assert cback(**bad) == INVALID, bad


def test_python_refuses_host_tensors():
    x, pos = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: rs.route_topk(x, 2), lambda: rs.sort_experts(pos, 8), lambda: rs.dispatch_rows(x, pos),
                 lambda: rs.combine_rows(x, pos), lambda: rs.combine_rows_backward(x, pos),
                 lambda: rs.dispatch_rows_backward(x, pos), lambda: rs.route_topk_backward(x, pos, x)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: rs.route_topk([1.0], 1), lambda: rs.sort_experts([1], 8), lambda: rs.dispatch_rows(None, pos)):
        with pytest.raises(TypeError):
            call()


def test_limits_match_the_header():
    src = open(__file__.replace("tests/test_experts_abi.py", "include/rs.h")).read()
    assert f"#define RS_MAX_EXPERTS {rs.MAX_EXPERTS} " in src
    assert f"#define RS_MAX_CHOICES {rs.MAX_CHOICES} " in src


# The oracle itself, against values worked by hand.
def test_oracle_choice_and_gates():
    l = np.array([[1.0, 3.0, 3.0, -np.inf], [-np.inf] * 4, [0.0, -0.0, np.nan, 5.0]])
    assert eo.choose(l, 3).tolist() == [[1, 2, 0], [-1, -1, -1], [2, 3, 0]]
    w, at = eo.route(l[:2], 2, "softmax", True, 2.0)
    assert np.allclose(w, [[1.0, 1.0], [0.0, 0.0]])
    w, _ = eo.route(np.array([[0.0, np.log(3.0)]]), 1, "softmax", False)
    assert np.allclose(w, [[0.75]])
    w, _ = eo.route(np.array([[-800.0, -800.0 + np.log(3.0)]]), 2, "sigmoid", True)
    assert np.allclose(w, [[0.75, 0.25]])


def test_oracle_sort():
    order, position, offsets = eo.sort_experts(np.array([[2, 0], [-1, 2], [5, 1]]), 1, 2)
    assert order.tolist() == [5, 0, 3, 1, 2, 4]
    assert position.tolist() == [[1, ~3], [~4, 2], [~5, 0]]
    assert offsets.tolist() == [0, 1, 3]


@pytest.mark.parametrize("mode", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_oracle_gradient_matches_differences(mode, renorm):
    """Central differences in 64 bits with step h: truncation h^2 / 6 times a
    third derivative (below 1 here), rounding 2^-52 / h, both far below 1e-7."""
    rng = np.random.default_rng(3)
    l, g = rng.normal(size=(4, 9)) * 2, rng.normal(size=(4, 3))
    _, at = eo.route(l, 3, mode, renorm)
    grad, _ = eo.route_backward(l, at, g, mode, renorm, 1.7)
    h = 1e-5

    def loss(x):
        w = np.stack([eo._chosen_gates(x[t], at[t], mode, renorm) for t in range(4)])
        return 1.7 * (w * g).sum()
    for t in range(4):
        for i in range(9):
            up, down = l.copy(), l.copy()
            up[t, i] += h
            down[t, i] -= h
            assert abs((loss(up) - loss(down)) / (2 * h) - grad[t, i]) < 1e-7


def test_oracle_rows_are_each_other_transposed():
    """<spread(x), y> = <x, join(y)> for any x and y, and the products are the
    derivative of either side in the weights."""
    rng = np.random.default_rng(4)
    T, k, H = 7, 3, 5
    position = rng.permutation(T * k).reshape(T, k)
    position = np.where(rng.random((T, k)) < 0.3, ~position, position)
    w, x, y = rng.normal(size=(T, k)), rng.normal(size=(T, H)), rng.normal(size=(T * k, H))
    there = (eo.spread(x, position, w, np.zeros((T * k, H))) * y).sum()
    assert abs(there - (x * eo.join(y, position, w)[0]).sum()) < 1e-12
    assert abs(there - (w * eo.dots(x, y, position)[0]).sum()) < 1e-12


def test_row_checks_of_the_whole_gradient(lib):
    """rs_combine_rows_backward_all refuses what rs_combine_rows_backward does."""
    def call(rows=E, gr=D, gw=F, g=A, dtype=F16, num=N, position=B, weights=C, k=K, tokens=T, width=H, stride=H):
        return lib.rs_combine_rows_backward_all(g, dtype, tokens, width, H, position, weights, k, rows, H, gr, stride,
                                                num, gw, None)
    for bad in (dict(rows=None), dict(rows=E + 1), dict(gw=F + 2), dict(gw=A), dict(gw=D), dict(gr=E), dict(gr=None),
                dict(stride=H - 1), dict(g=None), dict(gw=B), dict(gr=C), dict(dtype=3), dict(width=0), dict(k=65),
                dict(tokens=2**30), dict(num=2**31), dict(position=B + 2), dict(weights=C + 2)):
        assert call(**bad) == INVALID, bad
    assert call(tokens=0, num=0, g=None, gr=None, position=None, gw=None) == OK
