"""GPU tests of the mixture-of-experts calls against their 64-bit definitions
(expert_oracle): whole numbers equal, sums within bounds counted from the
roundings that a float32 evaluation makes."""
import numpy as np
import pytest

import expert_oracle as eo

torch = pytest.importorskip("torch")
rs = pytest.importorskip("lsd_radix_sort_pass_amd")

pytestmark = pytest.mark.gpu

DTYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}


def note(msg):
    print(f"\n[case] {msg}", flush=True)


def host(t):
    return t.detach().cpu().double().numpy() if t.dtype.is_floating_point else t.detach().cpu().numpy()


def close(got, exact, bound, what):
    got = host(got)
    with np.errstate(invalid="ignore"):
        bad = ~((np.abs(got - exact) <= bound) | (np.isnan(got) & np.isnan(exact)) | (got == exact))
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, first {np.argwhere(bad)[0]}: " \
        f"{got[bad][0]!r} for {exact[bad][0]!r}, bound {np.broadcast_to(bound, got.shape)[bad][0]!r}"


def rounded(a, dtype):
    """A device tensor of dtype and the values it holds."""
    t = torch.from_numpy(a).to(DTYPES[dtype]).cuda()
    return t, host(t)


# ---------------------------------------------------------------------------
# Routing
# ---------------------------------------------------------------------------
def make_logits(rng, T, E):
    l = rng.normal(size=(T, E)) * 2.0
    l = np.where(rng.random((T, E)) < 0.05, np.round(l), l)        # ties
    for t in range(T):
        kind = t % 7
        if kind == 1:
            l[t, rng.random(E) < 0.5] = -np.inf                    # some experts barred
        elif kind == 2 and T > 3:
            l[t] = -np.inf                                         # all of them
        elif kind == 3:
            l[t] = -60000.0                                        # equal and very low
        elif kind == 4:
            l[t] = np.where(rng.random(E) < 0.5, 0.0, -0.0)        # zeros of both signs
        elif kind == 5:
            l[t] -= 200.0
    return l


ROUTES = [(1, 1, 1), (1, 64, 6), (3, 5, 5), (17, 60, 4), (33, 256, 8), (64, 16, 16), (5, 257, 8), (30, 1000, 64),
          (130, 96, 16), (7, 100, 17), (8, 1024, 1), (259, 31, 3)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("T,E,k", ROUTES)
def test_route(dtype, T, E, k):
    rng = np.random.default_rng(T * 1000 + E + k)
    wide = np.zeros((T, E + 3))
    wide[:, 1:E + 1] = make_logits(rng, T, E)
    store, _ = rounded(wide, dtype)
    for strided in (False, True):
        logits = store[:, 1:E + 1] if strided else store[:, 1:E + 1].contiguous()
        values = host(logits)
        for mode in ("softmax", "sigmoid"):
            for renorm in (False, True):
                note(f"route_topk {dtype} T={T} E={E} k={k} {mode} renorm={renorm} strided={strided}")
                w, e = rs.route_topk(logits, k, mode, renorm, 1.5)
                exact, at = eo.route(values, k, mode, renorm, 1.5)
                assert w.dtype == torch.float32 and e.dtype == torch.int32
                assert np.array_equal(host(e), at)
                rel = eo.route_relative(values, at)[:, None]
                close(w, exact, np.abs(exact) * rel + 2.0 ** -125, "weights")
                if renorm:
                    continue
                assert (host(w)[at < 0] == 0).all()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("T,E,k", ROUTES)
def test_route_backward(dtype, T, E, k):
    rng = np.random.default_rng(T * 1000 + E + k + 7)
    wide = np.zeros((T, E + 2))
    wide[:, 1:E + 1] = make_logits(rng, T, E)
    store, _ = rounded(wide, dtype)
    grads = torch.full((T, E + 5), 3.0, dtype=DTYPES[dtype], device="cuda")
    for strided in (False, True):
        logits = store[:, 1:E + 1] if strided else store[:, 1:E + 1].contiguous()
        values = host(logits)
        at = eo.choose(values, k)
        if k > 2:
            at[T // 2, 1] = at[T // 2, 0]                # one expert named by two slots
            at[T - 1, k - 1] = E + 3                     # and one that is not there
        g = rng.normal(size=(T, k))
        g[(at < 0) | (at >= E)] = np.nan                 # gradients of slots without an expert
        de, dg = torch.from_numpy(at.astype(np.int32)).cuda(), torch.from_numpy(g.astype(np.float32)).cuda()
        for mode in ("softmax", "sigmoid"):
            for renorm in (False, True):
                note(f"route_topk_backward {dtype} T={T} E={E} k={k} {mode} renorm={renorm} strided={strided}")
                out = grads[:, 2:E + 2] if strided else None
                got = rs.route_topk_backward(logits, de, dg, mode, renorm, 1.5, out=out)
                exact, bound = eo.route_backward(values, at, host(dg), mode, renorm, 1.5)
                close(got, exact, bound + np.abs(exact) * eo.HALF_STEP[dtype] * 1.01 + eo.TINY[dtype] + 2.0 ** -125,
                      "gradient")
        assert (grads[:, :2] == 3).all() and (grads[:, E + 2:] == 3).all()


def test_route_special_values():
    note("route_topk NaN, infinities, the lowest value")
    inf, nan = np.inf, np.nan
    rows = np.array([[1.0, nan, 2.0, nan, 0.0], [inf, 1.0, 2.0, 3.0, -inf], [-3.4028234663852886e38] * 5,
                     [-inf, -inf, 7.0, -inf, -inf]])
    for dtype in DTYPES:
        logits, values = rounded(np.clip(rows, -65504, None) if dtype == "float16" else rows, dtype)
        w, e = rs.route_topk(logits, 3)
        assert host(e).tolist() == [[1, 3, 2], [0, 3, 2], [0, 1, 2], [2, -1, -1]] or dtype != "float32"
        assert np.array_equal(host(e), eo.choose(values, 3))
        assert np.isnan(host(w)[0]).all() and np.isnan(host(w)[1, 0])
        if dtype != "bfloat16":        # bfloat16 rounds the lowest float32 to -inf
            assert np.allclose(host(w)[2], 0.2)
        if dtype != "float16":         # where the clip above leaves no -inf
            assert host(w)[3].tolist() == [1.0, 0.0, 0.0]
        w, e = rs.route_topk(logits, 2, "sigmoid")
        assert np.isnan(host(w)[0]).all() and host(w)[1, 0] == 1.0


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_route_lowest_and_barred(dtype):
    """The type's lowest number is a logit like any other; -inf is not."""
    note(f"route_topk {dtype} lowest value beside -inf")
    low, inf = torch.finfo(DTYPES[dtype]).min, float("inf")
    logits = torch.tensor([[low] * 4, [-inf, low, -inf, low], [-inf, -inf, 7.0, -inf], [low, 0.0, low, -inf]],
                          dtype=DTYPES[dtype], device="cuda")
    w, e = rs.route_topk(logits, 3)
    assert e.tolist() == [[0, 1, 2], [1, 3, -1], [2, -1, -1], [1, 0, 2]]
    assert w.tolist() == [[0.25] * 3, [0.5, 0.5, 0.0], [1.0, 0.0, 0.0], [1.0, 0.0, 0.0]]
    w, e = rs.route_topk(logits, 3, "sigmoid", True)
    assert e.tolist() == [[0, 1, 2], [1, 3, -1], [2, -1, -1], [1, 0, 2]]
    assert w[1:].tolist() == [[0.5, 0.5, 0.0], [1.0, 0.0, 0.0], [1.0, 0.0, 0.0]]


def test_route_no_tokens_and_outputs():
    note("route_topk T=0, given outputs")
    empty = torch.empty(0, 16, device="cuda")
    w, e = rs.route_topk(empty, 4)
    assert w.shape == (0, 4) and e.shape == (0, 4)
    assert rs.route_topk_backward(empty, e, w).shape == (0, 16)
    logits = torch.randn(9, 16, device="cuda")
    w, e = torch.empty(9, 4, device="cuda"), torch.empty(9, 4, dtype=torch.int32, device="cuda")
    got = rs.route_topk(logits, 4, weights_out=w, experts_out=e)
    assert got[0] is w and got[1] is e
    fresh = rs.route_topk(logits, 4)
    assert torch.equal(fresh[0], w) and torch.equal(fresh[1], e)


def test_route_many_rows():
    note("route_topk T=300001")
    logits = torch.randn(300_001, 8, device="cuda")
    w, e = rs.route_topk(logits, 2, "softmax", True)
    top = torch.argsort(logits, dim=1, descending=True, stable=True)[:, :2]
    assert torch.equal(e.long(), top)
    exact = torch.softmax(torch.gather(logits, 1, top).double(), 1)
    assert (w.double() - exact).abs().max().item() < 40 * eo.U32


@pytest.mark.parametrize("E,k", [(256, 8), (255, 7), (64, 8), (512, 16), (400, 12), (1024, 32), (1000, 8), (1024, 64)])
def test_route_choice_over_many_rows(E, k):
    """Rows enough for every way of choosing, among them rows with more
    candidates than lanes and rows with a few values that repeat.  Weights
    (softmax over the row) within 20 + E / 16 half steps and the differences
    from the maximum, below 40 here."""
    T = 8192
    note(f"route_topk T={T} E={E} k={k}")
    logits = torch.randn(T, E, device="cuda") * 2
    logits[::5] = (logits[::5] * 2).round() / 2
    logits[1::97] = float("-inf")
    logits[1::97, 3:3 + k // 2] = 1.5
    for dtype in DTYPES.values():
        l = logits.to(dtype)
        w, e = rs.route_topk(l, k)
        top = torch.argsort(l.float(), dim=1, descending=True, stable=True)[:, :k]
        barred = torch.gather(l, 1, top) == float("-inf")
        assert torch.equal(e.long(), top.masked_fill(barred, -1))
        exact = torch.gather(torch.softmax(l.double(), 1), 1, top)
        assert ((w.double() - exact).abs() <= exact * eo.U32 * (60 + E / 16) + 2.0 ** -125).all()


# ---------------------------------------------------------------------------
# Slots sorted by expert
# ---------------------------------------------------------------------------
def check_sort(ids, first, experts, **kw):
    res = rs.sort_experts(ids, experts, first, **kw)
    order, position, offsets = eo.sort_experts(host(ids), first, experts)
    assert res.order.dtype == res.position.dtype == res.offsets.dtype == torch.int32
    assert np.array_equal(host(res.offsets), offsets), "offsets"
    assert np.array_equal(host(res.order), order), "order"
    assert res.position.shape == ids.shape
    assert np.array_equal(host(res.position), position), "position"
    return res


@pytest.mark.parametrize("n", [0, 1, 2, 63, 64, 65, 511, 1023, 1024, 1025, 4097, 8191, 8192, 8193, 16385, 100_003])
@pytest.mark.parametrize("experts", [1, 2, 7, 128, 255, 256, 1024])
def test_sort_experts(n, experts):
    rng = np.random.default_rng(n * 7 + experts)
    for dtype in (np.int32, np.int64):
        note(f"sort_experts n={n} experts={experts} {dtype.__name__}")
        ids = rng.integers(-1, experts + 1, n).astype(dtype)
        check_sort(torch.from_numpy(ids).cuda(), 0, experts)


def test_sort_experts_shapes_of_input():
    rng = np.random.default_rng(5)
    for name, ids in (("all one", np.full(50_000, 3)), ("all dropped", np.full(20_000, -1)),
                      ("sorted", np.sort(rng.integers(0, 64, 30_000))),
                      ("descending", np.sort(rng.integers(0, 64, 30_000))[::-1].copy()),
                      ("one run at the end", np.r_[np.zeros(9000), np.full(9000, 63)])):
        note(f"sort_experts {name}")
        check_sort(torch.from_numpy(ids.astype(np.int32)).cuda(), 0, 64)
    note("sort_experts of another rank's share")
    ids = rng.integers(0, 256, (5000, 8)).astype(np.int32)
    check_sort(torch.from_numpy(ids).cuda(), 192, 64)
    note("sort_experts far numbers")
    far = np.array([-2**31, 2**31 - 1, 5, 6, 4, -5, 0, 5], dtype=np.int32)
    check_sort(torch.from_numpy(far).cuda(), 5, 2)
    far = np.array([-2**63, 2**63 - 1, 2**32 + 5, 5, -2**32 + 5, 6, 2**31, 7], dtype=np.int64)
    check_sort(torch.from_numpy(far).cuda(), 5, 2)
    edge = np.array([2**31 - 1, 2**31 - 2, 2**31 - 1, 0, -1], dtype=np.int32)
    check_sort(torch.from_numpy(edge).cuda(), 2**31 - 2, 2)


@pytest.mark.parametrize("experts", [9, 128, 257, 1024])
@pytest.mark.parametrize("n", [262_144, 1_048_577, 2_097_152, 2_097_153, 5_000_011])
def test_sort_experts_many(n, experts):
    """Tables of few and many counts, one tile and several for a workgroup:
    numpy's stable sort as the definition."""
    note(f"sort_experts n={n} experts={experts}")
    rng = np.random.default_rng(n)
    ids = rng.integers(-3, experts + 43, n).astype(np.int64 if n % 2 else np.int32)
    ids[n // 3:n // 3 + 20_000] = -1
    res = rs.sort_experts(torch.from_numpy(ids).cuda(), experts)
    key = np.where((ids < 0) | (ids >= experts), experts, ids)
    order = np.argsort(key, kind="stable")
    place = np.empty(n, dtype=np.int64)
    place[order] = np.arange(n)
    assert np.array_equal(host(res.order), order)
    assert np.array_equal(host(res.position), np.where(key == experts, ~place, place))
    assert np.array_equal(host(res.offsets), np.searchsorted(key[order], np.arange(experts + 1)))


def test_sort_experts_temp_and_outputs():
    """A given temp buffer's contents do not matter; one that is too small is
    refused; outputs given are the ones returned."""
    note("sort_experts temp")
    ids = torch.randint(0, 100, (40_000,), dtype=torch.int32, device="cuda")
    need = rs.temp_bytes_experts(40_000, 100)
    temp = torch.randint(0, 255, (need,), dtype=torch.uint8, device="cuda")
    a = check_sort(ids, 0, 100, temp=temp)
    outs = dict(order_out=torch.empty_like(a.order), position_out=torch.empty_like(a.position),
                offsets_out=torch.empty_like(a.offsets))
    b = check_sort(ids, 0, 100, temp=temp, **outs)
    assert b.order is outs["order_out"] and b.position is outs["position_out"] and b.offsets is outs["offsets_out"]
    with pytest.raises(rs.RadixSortError):
        rs.sort_experts(ids, 100, temp=temp[:need - 256])


# ---------------------------------------------------------------------------
# Rows
# ---------------------------------------------------------------------------
SHAPES = [(1, 1, 1), (1, 8, 7168), (5, 3, 7), (33, 2, 129), (64, 6, 2048), (7, 64, 33), (150, 4, 1537), (2, 5, 20001),
          (301, 1, 8), (16, 7, 2880), (9, 10, 513), (5, 12, 2051), (4, 16, 1100), (3, 17, 1030), (6, 9, 300)]


def make_places(rng, T, k, dropped):
    """A permutation of the slots' places, some of them marked as dropped."""
    position = rng.permutation(T * k).astype(np.int32).reshape(T, k)
    mask = rng.random((T, k)) < dropped
    if dropped:
        mask[T // 2] = True                       # a token without any slot
    return np.where(mask, ~position, position).astype(np.int32)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("T,k,width", SHAPES)
def test_rows(dtype, T, k, width):
    rng = np.random.default_rng(T * 31 + k + width)
    torch_dtype = DTYPES[dtype]
    for dropped, weighted, pad in ((0.0, False, 0), (0.0, True, 3), (0.4, True, 0), (0.4, False, 1)):
        note(f"rows {dtype} T={T} k={k} width={width} dropped={dropped} weighted={weighted} pad={pad}")
        position = make_places(rng, T, k, dropped)
        dp = torch.from_numpy(position).cuda()
        weights = rng.normal(size=(T, k)).astype(np.float32) if weighted else None
        if weighted:
            weights[position < 0] = np.nan        # a dropped slot's weight counts for nothing
        dw = torch.from_numpy(weights).cuda() if weighted else None
        sx, _ = rounded(rng.normal(size=(T, width + pad)), dtype)
        srows, _ = rounded(rng.normal(size=(T * k, width + pad)), dtype)
        x, rows = sx[:, pad:], srows[:, pad:]
        rows_v = host(rows)
        for p in position[position < 0]:
            rows[~p] = float("nan")               # nor do dropped rows, when read

        def target(n):
            store = torch.full((n, width + pad), 5.0, dtype=torch_dtype, device="cuda")
            return store, (store[:, :width] if pad else None)

        # Forward there, and the gradient that has the same form.
        exact = eo.spread(host(x), position, weights, np.full((T * k, width), 5.0))
        for name, call in (("dispatch_rows", lambda out: rs.dispatch_rows(x, dp, dw, out=out)),
                           ("combine_rows_backward", lambda out: rs.combine_rows_backward(x, dp, weights=dw, out=out))):
            store, out = target(T * k)
            got = call(out)
            assert got.dtype == torch_dtype and got.shape == (T * k, width)
            close(got, exact, eo.spread_bound(exact, dtype), name)
            assert not pad or (store[:, width:] == 5).all()
        # And back.
        exact, size = eo.join(rows_v, position, weights)
        for name, call in (("combine_rows", lambda out: rs.combine_rows(rows, dp, dw, out=out)),
                           ("dispatch_rows_backward",
                            lambda out: rs.dispatch_rows_backward(rows, dp, weights=dw, out=out))):
            store, out = target(T)
            got = call(out)
            close(got, exact, eo.join_bound(exact, size, k, dtype), name)
            assert not pad or (store[:, width:] == 5).all()
        # With the gradient of the weights.
        sums, sizes = eo.dots(host(x), rows_v, position)
        got, grad_w = rs.dispatch_rows_backward(rows, dp, x, dw)
        close(got, exact, eo.join_bound(exact, size, k, dtype), "dispatch_rows_backward")
        close(grad_w, sums, eo.dots_bound(sizes, width), "dispatch_rows_backward weights")
        got, grad_w = rs.combine_rows_backward(x, dp, rows, dw)
        exact = eo.spread(host(x), position, weights, np.full((T * k, width), 5.0))
        close(got, exact, eo.spread_bound(exact, dtype), "combine_rows_backward")
        close(grad_w, sums, eo.dots_bound(sizes, width), "combine_rows_backward weights")


def test_rows_outside():
    """Places beyond the rows are skipped, rows that no slot names stay as
    they were, and a row that two slots name is read by both."""
    note("rows outside")
    x, _ = rounded(np.random.default_rng(1).normal(size=(3, 40)), "float32")
    position = np.array([[0, 9], [2**31 - 1, -2**31], [4, ~3]], dtype=np.int32)
    dp = torch.from_numpy(position).cuda()
    out = torch.full((6, 40), 7.0, device="cuda")
    rs.dispatch_rows(x, dp, out=out)
    exact = np.full((6, 40), 7.0)
    exact[0], exact[4], exact[3] = host(x)[0], host(x)[2], 0.0
    assert np.array_equal(host(out), exact)
    rows, _ = rounded(np.random.default_rng(2).normal(size=(6, 40)), "float32")
    position = np.array([[0, 9], [2**31 - 1, -2**31], [4, 4]], dtype=np.int32)
    dp = torch.from_numpy(position).cuda()
    v = host(rows)
    assert np.array_equal(host(rs.combine_rows(rows, dp)), np.stack([v[0], np.zeros(40), 2 * v[4]]))
    grad, grad_w = rs.combine_rows_backward(x, dp, rows)
    sums, sizes = eo.dots(host(x), v, position)
    close(grad_w, sums, eo.dots_bound(sizes, 40), "weights")
    assert grad.shape == rows.shape
    grad, grad_w = rs.dispatch_rows_backward(rows, dp, x)
    close(grad_w, sums, eo.dots_bound(sizes, 40), "weights")


def test_rows_none():
    note("rows T=0, no rows")
    none = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    x = torch.empty(0, 16, device="cuda")
    assert rs.dispatch_rows(x, none).shape == (0, 16)
    assert rs.combine_rows(x, none).shape == (0, 16)
    assert [t.shape for t in rs.combine_rows_backward(x, none, x)] == [(0, 16), (0, 2)]
    assert [t.shape for t in rs.dispatch_rows_backward(x, none, x)] == [(0, 16), (0, 2)]
    pos = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    assert (rs.combine_rows(x, pos) == 0).all()
    assert (rs.dispatch_rows_backward(x, pos, torch.ones(3, 16, device="cuda"))[1] == 0).all()


def test_rows_broadcast_input():
    """An input row shared by every token (stride 0) is read like any other."""
    note("rows broadcast")
    row = torch.randn(1, 72, device="cuda")
    pos = torch.randperm(12, device="cuda").to(torch.int32).reshape(6, 2)
    assert torch.equal(rs.dispatch_rows(row.expand(6, 72), pos), row.expand(12, 72))
    assert torch.equal(rs.combine_rows(row.expand(12, 72), pos), 2 * row.expand(6, 72))


def test_rows_far_offsets():
    """Rows whose elements lie beyond 2^31, and whose bytes lie beyond 2^32."""
    T, k, width = 70_000, 8, 4096
    note(f"rows T={T} k={k} width={width}: {T * k * width} elements")
    position = torch.randperm(T * k, device="cuda").to(torch.int32).reshape(T, k)
    x = torch.randn(T, width, device="cuda", dtype=torch.bfloat16)
    weights = torch.rand(T, k, device="cuda")
    rows = rs.dispatch_rows(x, position)
    slots = torch.randint(0, T * k, (4000,), device="cuda")
    slots = torch.cat([slots, position.reshape(-1).argsort()[-100:]])        # the last rows among them
    assert torch.equal(rows[position.reshape(-1)[slots].long()], x[slots // k])
    out = rs.combine_rows(rows, position, weights)
    tokens = torch.unique(slots // k)
    exact = x[tokens].double() * weights[tokens].double().sum(1, keepdim=True)
    size = x[tokens].double().abs() * weights[tokens].double().sum(1, keepdim=True)
    bound = eo.join_bound(host(exact), host(size), k, "bfloat16")
    close(out[tokens], host(exact), bound, "combine_rows")
    _, dots = rs.combine_rows_backward(out, position, rows, weights, out=rows.new_empty(rows.shape))
    exact = (out[tokens].double() * x[tokens].double()).sum(1, keepdim=True).expand(-1, k)
    size = (out[tokens].double() * x[tokens].double()).abs().sum(1, keepdim=True).expand(-1, k)
    close(dots[tokens], host(exact), eo.dots_bound(host(size), width), "weights")


# ---------------------------------------------------------------------------
# Refusals that need device tensors
# ---------------------------------------------------------------------------
def test_refusals():
    note("refusals")
    x = torch.randn(6, 32, device="cuda")
    pos = torch.arange(12, dtype=torch.int32, device="cuda").reshape(6, 2)
    w = torch.rand(6, 2, device="cuda")
    rows = torch.randn(12, 32, device="cuda")
    ids = torch.zeros(6, 2, dtype=torch.int32, device="cuda")
    value = [lambda: rs.route_topk(x, 0), lambda: rs.route_topk(x, 33), lambda: rs.route_topk(x, 2, "relu"),
             lambda: rs.route_topk(x.t(), 2), lambda: rs.route_topk(x[0], 2),
             lambda: rs.route_topk(x, 2, weights_out=w.t()), lambda: rs.route_topk(x, 2, experts_out=ids[:5]),
             lambda: rs.route_topk_backward(x, ids[:5], w), lambda: rs.route_topk_backward(x, ids, w[:, :1]),
             lambda: rs.route_topk_backward(x, ids, w, out=x[:5]),
             lambda: rs.sort_experts(ids, 0), lambda: rs.sort_experts(ids, 1025), lambda: rs.sort_experts(ids, 4, -1),
             lambda: rs.sort_experts(ids, 4, 2**31 - 3), lambda: rs.sort_experts(ids.t(), 4),
             lambda: rs.sort_experts(ids, 4, order_out=ids), lambda: rs.sort_experts(ids, 4, offsets_out=ids[0]),
             lambda: rs.dispatch_rows(x, pos[:5]), lambda: rs.dispatch_rows(x, pos, w[:5]),
             lambda: rs.dispatch_rows(x[:, ::2], pos), lambda: rs.dispatch_rows(x, pos.t()),
             lambda: rs.dispatch_rows(x, pos, out=rows[:, :31]), lambda: rs.dispatch_rows(x, pos.reshape(-1)),
             lambda: rs.combine_rows(rows, pos, out=x[:5]), lambda: rs.combine_rows(rows.t(), pos),
             lambda: rs.combine_rows(rows, pos, w.cpu()),
             lambda: rs.combine_rows_backward(x, pos, rows[:, :30]), lambda: rs.combine_rows_backward(x[:5], pos),
             lambda: rs.combine_rows_backward(x, pos, grad_weights_out=w),
             lambda: rs.dispatch_rows_backward(rows, pos, grad_weights_out=w),
             lambda: rs.dispatch_rows_backward(rows, pos, x[:5]),
             lambda: rs.combine_rows_backward(x[:1].expand(6, 32).sum(1, keepdim=True).expand(6, 32), pos)]
    kind = [lambda: rs.route_topk(x.double(), 2), lambda: rs.route_topk(x, 2, weights_out=w.half()),
            lambda: rs.sort_experts(ids.to(torch.int16), 4), lambda: rs.dispatch_rows(x.to(torch.int32), pos),
            lambda: rs.dispatch_rows(x, pos.long()), lambda: rs.dispatch_rows(x, pos, w.half()),
            lambda: rs.dispatch_rows(x, pos, out=rows.half()), lambda: rs.combine_rows(rows, pos, out=x.half()),
            lambda: rs.combine_rows_backward(x, pos, rows.half()),
            lambda: rs.route_topk_backward(x, ids.long(), w)]
    status = [lambda: rs.dispatch_rows(rows[:6], pos, out=rows), lambda: rs.combine_rows(rows, pos, out=rows[:6]),
              lambda: rs.route_topk_backward(x, ids, w, out=x),
              lambda: rs.combine_rows_backward(x, pos, rows, out=rows),
              lambda: rs.sort_experts(ids, 4, position_out=ids),
              lambda: rs.dispatch_rows(x[:, :0], pos), lambda: rs.dispatch_rows(x, pos[:, :0])]
    for error, calls in ((ValueError, value), (TypeError, kind), (rs.RadixSortError, status)):
        for i, call in enumerate(calls):
            with pytest.raises(error):
                print(i, call())
    # A tensor that wants a gradient is refused while gradients are recorded.
    leaf = x.clone().requires_grad_()
    for call in (lambda: rs.route_topk(leaf, 2), lambda: rs.dispatch_rows(leaf, pos),
                 lambda: rs.dispatch_rows(x, pos, w.clone().requires_grad_())):
        with pytest.raises(ValueError, match="gradient"):
            call()
        with torch.no_grad():
            call()


# ---------------------------------------------------------------------------
# A layer, as it is used
# ---------------------------------------------------------------------------
class Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k):
        w, e = rs.route_topk(logits, k, "softmax", True)
        ctx.save_for_backward(logits, e)
        ctx.mark_non_differentiable(e)
        return w, e

    @staticmethod
    def backward(ctx, grad_w, _):
        logits, e = ctx.saved_tensors
        return rs.route_topk_backward(logits, e, grad_w.contiguous(), "softmax", True), None


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


def test_layer_forward_and_gradients():
    """Router, sort, dispatch, one matrix per expert, combine: outputs and
    gradients against the dense layer in 64 bits.  Every float32 step errs by
    some half steps of its magnitude; the sums here hold at most 64 + 48 + 16
    terms of order one through three products, so 2^-24 * 3 * 128 * 8 (their
    largest magnitude) bounds them."""
    note("layer")
    rng = np.random.default_rng(11)
    T, E, k, H = 200, 16, 3, 48
    x0, r0 = rng.normal(size=(T, H)).astype(np.float32), (rng.normal(size=(H, E)) * 0.2).astype(np.float32)
    m0, g0 = (rng.normal(size=(E, H, H)) / 7).astype(np.float32), rng.normal(size=(T, H)).astype(np.float32)

    x, r, m = (torch.from_numpy(a).cuda().requires_grad_() for a in (x0, r0, m0))
    w, e = Route.apply(x @ r, k)
    order, position, offsets = rs.sort_experts(e, E)
    rows = Dispatch.apply(x, position)
    cuts = offsets.tolist()
    rows = torch.cat([rows[a:b] @ m[i] for i, (a, b) in enumerate(zip(cuts, cuts[1:]))])
    out = Combine.apply(rows, position, w)
    out.backward(torch.from_numpy(g0).cuda())

    x1, r1, m1 = (torch.from_numpy(a.astype(np.float64)).requires_grad_() for a in (x0, r0, m0))
    logits = x1 @ r1
    keep = torch.zeros(T, E, dtype=torch.bool).scatter_(1, e.cpu().long(), True)
    dense = torch.softmax(logits.masked_fill(~keep, -float("inf")), 1)
    want = sum(dense[:, i, None] * (x1 @ m1[i]) for i in range(E))
    want.backward(torch.from_numpy(g0.astype(np.float64)))
    assert torch.equal(keep, torch.zeros_like(keep).scatter_(1, torch.topk(logits, k).indices, True))
    for a, b in ((out, want), (x.grad, x1.grad), (r.grad, r1.grad), (m.grad, m1.grad)):
        scale = max(1.0, b.abs().max().item())
        assert (a.detach().cpu().double() - b.detach()).abs().max().item() <= 2.0 ** -24 * 3 * 128 * 8 * scale


def run_layer(logits, x, g, k, E, buf):
    """Every call, forward and backward, into the buffers of buf."""
    w, e = rs.route_topk(logits, k, "sigmoid", True, weights_out=buf["w"], experts_out=buf["e"])
    s = rs.sort_experts(e, E, order_out=buf["order"], position_out=buf["position"], offsets_out=buf["offsets"],
                        temp=buf["temp"])
    rows = rs.dispatch_rows(x, s.position, out=buf["rows"])
    rs.combine_rows(rows, s.position, w, out=buf["out"])
    gr, gw = rs.combine_rows_backward(g, s.position, rows, w, out=buf["grad_rows"], grad_weights_out=buf["gw"])
    rs.dispatch_rows_backward(gr, s.position, out=buf["gx"])
    rs.route_topk_backward(logits, e, gw, "sigmoid", True, out=buf["gl"])


def layer_buffers(T, E, k, H, dtype=torch.bfloat16):
    new = lambda *shape, dtype: torch.zeros(shape, dtype=dtype, device="cuda")
    i32, f32 = torch.int32, torch.float32
    return {"w": new(T, k, dtype=f32), "e": new(T, k, dtype=i32), "order": new(T * k, dtype=i32),
            "position": new(T, k, dtype=i32), "offsets": new(E + 1, dtype=i32), "rows": new(T * k, H, dtype=dtype),
            "out": new(T, H, dtype=dtype), "grad_rows": new(T * k, H, dtype=dtype), "gw": new(T, k, dtype=f32),
            "gx": new(T, H, dtype=dtype), "gl": new(T, E, dtype=dtype),
            "temp": torch.empty(max(256, rs.temp_bytes_experts(T * k, E)), dtype=torch.uint8, device="cuda")}


@pytest.mark.parametrize("T", [5, 3001])
def test_layer_in_graphs(T):
    """Two captured graphs that share the sort's temp storage, replayed in
    turn with eager work between: every replay equals the eager result."""
    note(f"layer in graphs T={T}")
    E, k, H = 32, 4, 200
    stat = {n: torch.empty(T, c, dtype=torch.bfloat16, device="cuda") for n, c in (("logits", E), ("x", H), ("g", H))}
    bufs = [layer_buffers(T, E, k, H) for _ in range(2)]
    bufs[1]["temp"] = bufs[0]["temp"]
    gen = torch.Generator(device="cuda")

    def fill(seed):
        gen.manual_seed(seed)
        for t in stat.values():
            t.copy_(torch.randn(t.shape, generator=gen, device="cuda"))
    fill(0)
    run_layer(stat["logits"], stat["x"], stat["g"], k, E, layer_buffers(T, E, k, H))
    torch.cuda.synchronize()
    graphs = []
    for b in bufs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run_layer(stat["logits"], stat["x"], stat["g"], k, E, b)
        graphs.append(graph)
    for i in range(6):
        fill(100 + i)
        graphs[i % 2].replay()
        eager = layer_buffers(T, E, k, H)
        run_layer(stat["logits"], stat["x"], stat["g"], k, E, eager)
        torch.cuda.synchronize()
        for name in eager:
            if name != "temp":
                assert torch.equal(bufs[i % 2][name], eager[name]), f"replay {i}: {name}"


def test_layer_allocates_in_a_graph():
    """Calls that allocate their outputs and temp storage, captured."""
    note("calls that allocate, captured")
    ids = torch.randint(0, 50, (20_000,), dtype=torch.int32, device="cuda")
    logits = torch.randn(300, 50, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = rs.sort_experts(ids, 50)
        w, e = rs.route_topk(logits, 5)
    for i in range(4):
        ids.copy_(torch.randint(-1, 50, (20_000,), device="cuda"))
        logits.copy_(torch.randn(300, 50, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(s, rs.sort_experts(ids, 50)):
            assert torch.equal(a, b)
        for a, b in zip((w, e), rs.route_topk(logits, 5)):
            assert torch.equal(a, b)


def test_other_streams():
    """Calls on two streams at once, given and current, equal those on one."""
    note("streams")
    T, E, k, H = 2000, 64, 8, 512
    inputs = [(torch.randn(T, E, device="cuda"), torch.randn(T, H, device="cuda")) for _ in range(2)]

    def layer(logits, x, stream=None):
        w, e = rs.route_topk(logits, k, stream=stream)
        s = rs.sort_experts(e, E, stream=stream)
        rows = rs.dispatch_rows(x, s.position, stream=stream)
        return rs.combine_rows(rows, s.position, w, stream=stream)
    want = [layer(*p) for p in inputs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for s, p in zip(streams, inputs):
            s.wait_stream(torch.cuda.current_stream())
            got.append(layer(*p, stream=s))
        with torch.cuda.stream(streams[0]):
            got.append(layer(*inputs[0]))
        torch.cuda.synchronize()
        for a, b in zip(got, want + want[:1]):
            assert torch.equal(a, b)


def test_two_threads():
    """Two host threads, a stream each, at once."""
    note("two threads")
    import threading
    T, E, k, H = 1500, 40, 6, 300
    inputs = [[torch.randn(T, c, device="cuda").bfloat16() for c in (E, H, H)] for _ in range(2)]
    want = [layer_buffers(T, E, k, H) for _ in range(2)]
    for p, b in zip(inputs, want):
        run_layer(p[0], p[1], p[2], k, E, b)
    torch.cuda.synchronize()
    got = [[layer_buffers(T, E, k, H) for _ in range(5)] for _ in range(2)]
    torch.cuda.synchronize()
    errors = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for b in got[i]:
                    run_layer(*inputs[i], k, E, b)
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
                if name != "temp":
                    assert torch.equal(b[name], want[i][name]), name


def test_parameters_under_no_grad():
    """Parameters and tensors that want a gradient, where none is recorded."""
    note("parameters")
    x = torch.nn.Parameter(torch.randn(6, 32, device="cuda"))
    pos = torch.randperm(12, device="cuda").to(torch.int32).reshape(6, 2)
    w = torch.rand(6, 2, device="cuda", requires_grad=True)
    with pytest.raises(ValueError, match="gradient"):
        rs.dispatch_rows(x, pos, w)
    with torch.no_grad():
        rows = rs.dispatch_rows(x, pos, w)
        assert torch.equal(rows, rs.dispatch_rows(x.detach(), pos, w.detach()))
        assert not rows.requires_grad


def test_results_repeat():
    note("results repeat")
    T, E, k, H = 3000, 128, 8, 1000
    buf = [layer_buffers(T, E, k, H) for _ in range(2)]
    logits, x, g = (torch.randn(T, c, device="cuda").bfloat16() for c in (E, H, H))
    for b in buf:
        run_layer(logits, x, g, k, E, b)
    torch.cuda.synchronize()
    for name in buf[0]:
        if name != "temp":
            assert torch.equal(buf[0][name], buf[1][name]), name


def test_kernel_timing():
    """The calls' launches are timed under their own kernel kinds."""
    note("kernel timing")
    from lsd_radix_sort_pass_amd import _lib
    logits, x = torch.randn(64, 16, device="cuda"), torch.randn(64, 256, device="cuda")
    rs.prof_reset()
    rs.prof_enable(True)
    try:
        w, e = rs.route_topk(logits, 2)
        s = rs.sort_experts(e, 16)
        rs.combine_rows(rs.dispatch_rows(x, s.position), s.position, w)
        rs.sort_experts(torch.zeros(100_000, dtype=torch.int32, device="cuda"), 16)
    finally:
        rs.prof_enable(False)
    assert [rs.prof_summary(kind)[0] for kind in (_lib.RS_KERNEL_ROUTE, _lib.RS_KERNEL_EXPERT, _lib.RS_KERNEL_ROWS)] \
        == [1, 3, 2]
    rs.prof_reset()
