"""GPU tests of the mixture-of-experts calls at their edges: rows that no slot
names, and values and tensors that the other tests do not pass."""
import numpy as np
import pytest

import expert_oracle as eo
from test_gpu_experts import DTYPES, close, host, note, rounded

torch = pytest.importorskip("torch")
rs = pytest.importorskip("lsd_radix_sort_pass_amd")

pytestmark = pytest.mark.gpu


def poison(*shapes_and_dtypes):
    """Leaves NaN in the memory that the next allocations of these sizes get."""
    held = [torch.full(shape, float("nan"), dtype=dtype, device="cuda") for shape, dtype in shapes_and_dtypes]
    del held


def places(rng, T, k, num_rows, kind):
    """Places of T * k slots among num_rows rows, some rows without a slot."""
    n = T * k
    if kind == "fewer slots than rows":
        p = rng.permutation(num_rows)[:n]
    elif kind == "a part of a sort":                  # most places lie behind the rows
        p = rng.permutation(4 * n)[:n]
    else:                                             # "skipped": half of them do
        p = rng.permutation(n)
        p = np.where(rng.random(n) < 0.5, p, 2**31 - 1 - p)
    p = np.where(rng.random(n) < 0.2, ~p, p)          # dropped ones among both
    return p.astype(np.int32).reshape(T, k)


# Narrow and wide rows, small and many slots, the 512-byte rule's two sides.
UNNAMED = [(3, 2, 40), (7, 8, 1537), (1, 1, 1), (61, 3, 129), (5, 17, 2051), (2100, 8, 100), (2100, 8, 520),
           (700, 30, 264), (9, 2, 5000)]


@pytest.mark.parametrize("kind", ["fewer slots than rows", "a part of a sort", "skipped"])
@pytest.mark.parametrize("T,k,width", UNNAMED)
def test_gradient_of_unnamed_rows(T, k, width, kind):
    """A row that combine_rows does not read has gradient zero."""
    rng = np.random.default_rng(T + k + width)
    for dtype in DTYPES if T < 100 else ["bfloat16"]:
        note(f"combine_rows_backward {dtype} T={T} k={k} width={width} {kind}")
        num_rows = T * k + (T * k + 5 if kind == "fewer slots than rows" else 0)
        position = places(rng, T, k, num_rows, kind)
        dp = torch.from_numpy(position).cuda()
        g, _ = rounded(rng.normal(size=(T, width)), dtype)
        rows, _ = rounded(rng.normal(size=(num_rows, width)), dtype)
        weights = rng.normal(size=(T, k)).astype(np.float32)
        dw = torch.from_numpy(weights).cuda()
        exact = eo.spread(host(g), position, weights, np.zeros((num_rows, width)))
        poison(((num_rows, width), DTYPES[dtype]))
        grad, _ = rs.combine_rows_backward(g, dp, rows, dw)
        close(grad, exact, eo.spread_bound(exact, dtype), "with the weights' gradient")
        if num_rows == T * k:
            poison(((num_rows, width), DTYPES[dtype]))
            grad = rs.combine_rows_backward(g, dp, weights=dw)
            close(grad, exact, eo.spread_bound(exact, dtype), "rows alone")
        # A given buffer keeps what it has in such rows.
        out = torch.full((num_rows, width), 5.0, dtype=DTYPES[dtype], device="cuda")
        rs.combine_rows_backward(g, dp, rows, dw, out=out)
        exact = eo.spread(host(g), position, weights, np.full((num_rows, width), 5.0))
        close(out, exact, eo.spread_bound(exact, dtype), "given buffer")


def test_gradient_of_rows_without_tokens():
    note("combine_rows_backward T=0")
    poison(((9, 16), torch.float32))
    x = torch.empty(0, 16, device="cuda")
    grad, dots = rs.combine_rows_backward(x, torch.empty(0, 2, dtype=torch.int32, device="cuda"),
                                          torch.randn(9, 16, device="cuda"))
    assert grad.shape == (9, 16) and (grad == 0).all() and dots.shape == (0, 2)


@pytest.mark.parametrize("k,width", [(8, 100), (8, 264), (8, 600), (1, 2100)])
def test_gradient_of_unnamed_rows_among_many(k, width):
    """More slots than 2^16, where narrow rows are cleared otherwise than wide
    ones.  A product of two float32 rounded once is the result to the bit."""
    T = 72_000 // k
    n = T * k
    note(f"combine_rows_backward T={T} k={k} width={width}")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(width)
    position = torch.randperm(n, generator=gen, device="cuda").to(torch.int32)
    position[::3] += n                                            # behind the rows
    position[1::7] = ~position[1::7]                              # dropped
    g = torch.randn(T, width, generator=gen, device="cuda").bfloat16()
    rows = torch.randn(n, width, generator=gen, device="cuda").bfloat16()
    w = torch.rand(T, k, generator=gen, device="cuda")
    want = torch.zeros_like(rows)
    s = torch.nonzero((position >= 0) & (position < n))[:, 0]
    want[position[s].long()] = (g[s // k].float() * w.reshape(-1)[s, None]).bfloat16()
    for with_dots in (True, False):
        poison(((n, width), torch.bfloat16))
        grad = rs.combine_rows_backward(g, position.reshape(T, k), rows if with_dots else None, w)
        assert torch.equal(grad[0] if with_dots else grad, want)


@pytest.mark.parametrize("width", [40, 600])
def test_rows_named_twice(width):
    """A row that two slots name: combine_rows reads it for both, and of the
    gradients the row gets one, the weights each their own."""
    note(f"rows named twice, width {width}")
    rng = np.random.default_rng(width)
    position = torch.tensor([[0, 4], [4, 1], [2, 7]], dtype=torch.int32, device="cuda")
    x, _ = rounded(rng.normal(size=(3, width)), "float32")
    rows, v = rounded(rng.normal(size=(6, width)), "float32")
    w = torch.tensor([[1.0, 2.0], [4.0, 0.5], [1.0, 8.0]], device="cuda")       # products are exact
    exact, size = eo.join(v, host(position), host(w))
    close(rs.combine_rows(rows, position, w), exact, eo.join_bound(exact, size, 2, "float32"), "combine_rows")
    poison(((6, width), torch.float32))
    grad, grad_w = rs.combine_rows_backward(x, position, rows, w)
    sums, sizes = eo.dots(host(x), v, host(position))
    close(grad_w, sums, eo.dots_bound(sizes, width), "weights")
    assert torch.equal(grad[[0, 1, 2, 3, 5]], torch.stack([x[0], x[1] * 0.5, x[2], x[0] * 0, x[0] * 0]))
    assert ((grad[4] == x[0] * 2) | (grad[4] == x[1] * 4)).all()


def test_refusals_of_the_rows_gradient():
    """What is no tensor is a TypeError, a wrong shape a ValueError, whichever
    argument it is."""
    note("refusals of combine_rows_backward")
    g = torch.randn(6, 32, device="cuda")
    pos = torch.arange(12, dtype=torch.int32, device="cuda").reshape(6, 2)
    rows = torch.randn(12, 32, device="cuda")
    for bad in ([1.0], 3, "rows"):
        for kw in (dict(rows=bad), dict(out=bad), dict(rows=rows, out=bad), dict(rows=bad, out=rows),
                   dict(weights=bad), dict(rows=rows, grad_weights_out=bad)):
            with pytest.raises(TypeError):
                rs.combine_rows_backward(g, pos, **kw)
    scalar, empty = torch.zeros((), device="cuda"), torch.empty(0, device="cuda")
    for bad in (scalar, empty, rows[0], rows[None], rows[:, :31], rows.cpu()):
        for kw in (dict(rows=bad), dict(out=bad), dict(rows=rows, out=bad)):
            with pytest.raises(ValueError):
                rs.combine_rows_backward(g, pos, **kw)
    with pytest.raises(ValueError):
        rs.combine_rows_backward(g, pos, rows, out=torch.empty(13, 32, device="cuda"))
    with pytest.raises(TypeError):
        rs.combine_rows_backward(g, pos, rows.half())


def test_refusal_of_tangents():
    """A tensor that carries a forward-mode tangent is refused rather than its
    tangent lost, unless forward gradients are off, as they are inside a
    torch.autograd.Function."""
    note("tangents")
    import torch.autograd.forward_ad as fwad
    x, w = torch.randn(6, 32, device="cuda"), torch.rand(6, 2, device="cuda")
    pos = torch.arange(12, dtype=torch.int32, device="cuda").reshape(6, 2)
    rows = torch.randn(12, 32, device="cuda")
    ids = torch.zeros(6, 2, dtype=torch.int32, device="cuda")
    with fwad.dual_level():
        def dual(t):
            return fwad.make_dual(t, torch.ones_like(t))
        calls = [lambda: rs.route_topk(dual(x), 2), lambda: rs.route_topk_backward(dual(x), ids, w),
                 lambda: rs.route_topk_backward(x, ids, dual(w)), lambda: rs.dispatch_rows(dual(x), pos),
                 lambda: rs.dispatch_rows(x, pos, dual(w)), lambda: rs.combine_rows(dual(rows), pos),
                 lambda: rs.combine_rows(rows, pos, dual(w)), lambda: rs.dispatch_rows_backward(dual(rows), pos),
                 lambda: rs.dispatch_rows_backward(rows, pos, dual(x)), lambda: rs.combine_rows_backward(dual(x), pos),
                 lambda: rs.combine_rows_backward(x, pos, dual(rows), w),
                 lambda: rs.dispatch_rows(x, pos, out=dual(rows))]
        for i, call in enumerate(calls):
            with pytest.raises(ValueError, match="tangent"):
                print(i, call())
        with torch.no_grad(), pytest.raises(ValueError, match="tangent"):
            rs.combine_rows(dual(rows), pos)
        # Tensors without one are as ever, and so is every tensor where none is recorded.
        want = rs.combine_rows(rows, pos, w)
        off = dual(rows)
        with fwad._set_fwd_grad_enabled(False):
            assert torch.equal(rs.combine_rows(off, pos, w), want)
    assert torch.equal(rs.combine_rows(rows, pos, w), want)


class JvpCombine(torch.autograd.Function):
    @staticmethod
    def forward(rows, position, w):
        return rs.combine_rows(rows, position, w)

    @staticmethod
    def setup_context(ctx, inputs, output):
        ctx.save_for_forward(*inputs)

    @staticmethod
    def jvp(ctx, rows_t, _, w_t):
        rows, position, w = ctx.saved_tensors
        return rs.combine_rows(rows_t, position, w) + rs.combine_rows(rows, position, w_t)


def test_tangents_through_a_function():
    """combine_rows is linear in its rows and in its weights."""
    note("tangents through a function")
    import torch.autograd.forward_ad as fwad
    pos = torch.randperm(12, device="cuda").to(torch.int32).reshape(6, 2)
    rows, rows_t = torch.randn(2, 12, 32, device="cuda")
    w, w_t = torch.rand(2, 6, 2, device="cuda")
    with fwad.dual_level():
        out = JvpCombine.apply(fwad.make_dual(rows, rows_t), pos, fwad.make_dual(w, w_t))
        value, tangent = fwad.unpack_dual(out)
    assert torch.equal(value, rs.combine_rows(rows, pos, w))
    assert torch.equal(tangent, rs.combine_rows(rows_t, pos, w) + rs.combine_rows(rows, pos, w_t))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("E", [5, 64, 300])
def test_route_not_finite(dtype, E):
    """A +inf or a NaN in a row: every weight of a softmax is NaN, and every
    element of its gradient but those of barred experts, also those so far
    below the largest that their exponentials are 0."""
    note(f"route_topk {dtype} E={E} with +inf and NaN")
    inf, nan = float("inf"), float("nan")
    l = torch.full((4, E), -300.0)                      # exp(-300 - 0) is 0 in float32
    l[:, 0], l[:, 1], l[:, 2], l[:, 4] = 0.0, 1.0, -inf, -200.0
    l[1, 3], l[2, 3] = inf, nan
    logits = l.to(DTYPES[dtype]).cuda()
    barred = torch.zeros(E, dtype=torch.bool)
    barred[2] = True
    k = 3
    for renorm in (False, True):
        w, e = rs.route_topk(logits, k, "softmax", renorm)
        assert e[[0, 3]].tolist() == [[1, 0, 4]] * 2
        assert e[1:3].tolist() == [[3, 1, 0]] * 2
        assert torch.isfinite(w[[0, 3]]).all() and torch.isnan(w[1:3]).all()
        g = torch.ones(4, k, device="cuda")
        g[3, 1] = nan                                   # a gradient that is not finite, finite logits
        grad = rs.route_topk_backward(logits, e, g, "softmax", renorm).float().cpu()
        assert torch.isfinite(grad[0]).all()
        chosen = torch.zeros(4, E, dtype=torch.bool).scatter_(1, e.cpu().long(), True)
        for t in (1, 2, 3):
            bad = chosen[t] if renorm else ~barred          # renormalized: the others have no part in it
            assert torch.isnan(grad[t][bad]).all() and (grad[t][~bad] == 0).all(), t
    for renorm in (False, True):                        # the sigmoid of +inf is 1, that of NaN a NaN
        w, e = rs.route_topk(logits, k, "sigmoid", renorm)
        assert torch.isfinite(w[[0, 1, 3]]).all()
        assert torch.isnan(w[2] if renorm else w[2, :1]).all() and torch.isfinite(w[2, 1:]).all() != renorm
        if not renorm:
            assert w[1, 0] == 1.0


def expert_patterns(rng, n, experts):
    """Expert numbers whose equal ones stand in every relation to the lanes, the
    half of the patterns with dropped slots between them."""
    lane = np.arange(n) % 64
    some = rng.integers(0, experts, n)
    base = {"uniform": some, "all equal": np.full(n, experts - 1), "two": some % 2, "four": some % 4 * (experts // 4),
            "sixteen": some % 16, "skewed": some & rng.integers(0, experts, n) & rng.integers(0, experts, n),
            "lane mod 4": lane % 4, "lane div 16": lane // 16, "one bank": lane % 8 * 32 % experts,
            "half waves": (lane >= 32) * 3, "reversed lanes": 63 - lane}
    for name, ids in base.items():
        yield name, ids
        yield name + ", dropped between", np.where(rng.random(n) < 0.4, -1, ids)
        yield name + ", odd lanes dropped", np.where(lane % 2 == 1, experts + 7, ids)


@pytest.mark.parametrize("ranker", [0, 1])
@pytest.mark.parametrize("experts", [100, 256, 1024])
def test_sort_experts_lane_order(ranker, experts):
    """The sort is stable whatever the lanes of equal experts, in every form of
    its kernel: 1, 4 and 8 slots a thread of one workgroup, and 256 workgroups
    under contention, with counts summed and scanned.  Ranker 0 takes this from
    the order in which the LDS serves a wave's same-address adds, ranker 1 from
    ballots."""
    rng = np.random.default_rng(experts)
    prev = rs.prof_ranker(ranker)
    try:
        for n in (1000, 4096, 8192, 1_050_000):
            for name, ids in expert_patterns(rng, n, experts):
                note(f"sort_experts ranker={ranker} n={n} experts={experts} {name}")
                key = np.where((ids < 0) | (ids >= experts), experts, ids)
                order = torch.from_numpy(np.argsort(key, kind="stable")).cuda()
                place = torch.empty_like(order)
                place[order] = torch.arange(n, device="cuda")
                place = torch.where(torch.from_numpy(key == experts).cuda(), ~place, place)
                res = rs.sort_experts(torch.from_numpy(ids.astype(np.int32)).cuda(), experts)
                assert torch.equal(res.order.long(), order), name
                assert torch.equal(res.position.long(), place), name
                counts = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=experts + 1)[:experts])])
                assert np.array_equal(host(res.offsets), counts), name
    finally:
        rs.prof_ranker(prev)


# With dots, rows of more than 64 accesses take 1 to 4 chunks in flight together
# for up to two slots a token, 1 or 2 for up to four: widths for each count of
# either element size, most with a last access that is moved back.
FEW_SLOTS = [(9, 1, 1537), (9, 2, 4099), (5, 2, 2500), (5, 1, 4000), (7, 2, 8191), (6, 1, 9001), (40, 2, 700),
             (40, 1, 521), (30, 2, 300), (30, 1, 290), (5, 3, 2500), (6, 4, 4099), (7, 2, 4096), (4, 1, 8192)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("T,k,width", FEW_SLOTS)
def test_rows_of_few_slots(dtype, T, k, width):
    rng = np.random.default_rng(T * 100 + k * 10 + width)
    for dropped, weighted, pad in ((0.0, True, 0), (0.4, False, 3), (0.4, True, 1)):
        note(f"rows {dtype} T={T} k={k} width={width} dropped={dropped} weighted={weighted} pad={pad}")
        position = rng.permutation(T * k).astype(np.int32).reshape(T, k)
        mask = rng.random((T, k)) < dropped
        if dropped:
            mask[T // 2] = True                       # a token without any slot
        position = np.where(mask, ~position, position).astype(np.int32)
        dp = torch.from_numpy(position).cuda()
        weights = rng.normal(size=(T, k)).astype(np.float32) if weighted else None
        dw = torch.from_numpy(weights).cuda() if weighted else None
        x, xv = rounded(rng.normal(size=(T, width + pad)), dtype)
        rows, rv = rounded(rng.normal(size=(T * k, width + pad)), dtype)
        x, xv, rows, rv = x[:, pad:], xv[:, pad:], rows[:, pad:], rv[:, pad:]
        for p in position[position < 0]:
            rows[~p] = float("nan")

        def target(n):
            store = torch.full((n, width + pad + 2), 5.0, dtype=DTYPES[dtype], device="cuda")
            return store, store[:, 1:width + 1]
        sums, sizes = eo.dots(xv, rv, position)
        there = eo.spread(xv, position, weights, np.zeros((T * k, width)))
        back, size = eo.join(rv, position, weights)
        for given in (False, True):
            store, out = target(T)
            gw = torch.full((T, k), 7.0, device="cuda") if given else None
            got, dots = rs.dispatch_rows_backward(rows, dp, x, dw, out=out if given else None, grad_weights_out=gw)
            close(got, back, eo.join_bound(back, size, k, dtype), "dispatch_rows_backward")
            close(dots, sums, eo.dots_bound(sizes, width), "dispatch_rows_backward weights")
            assert (store[:, :1] == 5).all() and (store[:, width + 1:] == 5).all()
            store, out = target(T * k)
            got, dots = rs.combine_rows_backward(x, dp, rows, dw, out=out if given else None, grad_weights_out=gw)
            close(got, there, eo.spread_bound(there, dtype), "combine_rows_backward")
            close(dots, sums, eo.dots_bound(sizes, width), "combine_rows_backward weights")
            assert (store[:, :1] == 5).all() and (store[:, width + 1:] == 5).all()
        close(rs.combine_rows(rows, dp, dw), back, eo.join_bound(back, size, k, dtype), "combine_rows")
        close(rs.dispatch_rows(x, dp, dw), there, eo.spread_bound(there, dtype), "dispatch_rows")


def many_rows(T, k, width, dtype, dropped, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    position = torch.randperm(T * k, generator=gen, device="cuda").to(torch.int32).reshape(T, k)
    if dropped:
        position = torch.where(torch.rand(T, k, generator=gen, device="cuda") < dropped, ~position, position)
    x = torch.randn(T, width, generator=gen, device="cuda", dtype=dtype)
    rows = torch.randn(T * k, width, generator=gen, device="cuda", dtype=dtype)
    return position, x, rows, torch.rand(T, k, generator=gen, device="cuda") - 0.5


def check_many_rows(position, x, rows, w, dtype):
    """All four row calls on many tokens against float64 sums on the device,
    block by block; bounds as in expert_oracle."""
    T, k = position.shape
    width = x.shape[1]
    half, tiny = eo.HALF_STEP[dtype], eo.TINY[dtype]
    joined, dots = rs.dispatch_rows_backward(rows, position, x, w)
    plain = rs.combine_rows(rows, position, w)
    spread, dots2 = rs.combine_rows_backward(x, position, rows, w)
    sent = rs.dispatch_rows(x, position, w)
    assert torch.equal(joined, plain) and torch.equal(spread, sent)
    step = max(1, (1 << 26) // (width * k))
    for a in range(0, T, step):
        p, wt = position[a:a + step], w[a:a + step].double()
        used = (p >= 0).double()
        place = torch.where(p >= 0, p, ~p).long()
        xd = x[a:a + step].double()
        r = rows[place].double()                                            # (step, k, width)
        term = r * (wt * used)[:, :, None]
        exact, size = term.sum(1), term.abs().sum(1)
        bound = (2 * k * eo.U32 * size + exact.abs() * half) * 1.01 + tiny
        assert ((joined[a:a + step].double() - exact).abs() <= bound).all(), f"join, tokens from {a}"
        pr = r * xd[:, None, :] * used[:, :, None]
        bound = 2 * (width / 64 + 24) * eo.U32 * pr.abs().sum(2) + eo.TINY["float32"]
        for d in (dots, dots2):
            assert ((d[a:a + step].double() - pr.sum(2)).abs() <= bound).all(), f"dots, tokens from {a}"
        exact = xd[:, None, :] * (wt * used)[:, :, None]
        bound = exact.abs() * (half + eo.U32) * 1.01 + tiny
        assert ((spread[place].double() - exact).abs() <= bound).all(), f"spread, tokens from {a}"


@pytest.mark.parametrize("T,k,width,dtype", [(12_000, 2, 4099, "bfloat16"), (30_000, 1, 2501, "float32"),
                                             (9_000, 3, 5003, "float16"), (4_000, 17, 2051, "bfloat16")])
def test_rows_beyond_the_last_level_cache(T, k, width, dtype):
    """More than 256 MiB of rows, which are read with non-temporal loads: odd
    widths, few slots, some of them dropped."""
    note(f"rows T={T} k={k} width={width} {dtype}")
    check_many_rows(*many_rows(T, k, width, DTYPES[dtype], 0.3, T), dtype)


@pytest.mark.parametrize("T,k,width", [((1 << 20) + 7, 1, 521), ((1 << 22) + 5, 1, 264), ((1 << 23) + 9, 1, 129),
                                       ((1 << 22) // 17 + 999, 17, 257)])
def test_rows_beyond_one_grid(T, k, width):
    """More tokens (or slots) than the 2^20 workgroups of a launch take at once:
    a workgroup and a wave a token, eight tokens a workgroup, a wave a slot."""
    note(f"rows T={T} k={k} width={width}")
    check_many_rows(*many_rows(T, k, width, torch.bfloat16, 0.1, T), "bfloat16")


def test_route_beyond_one_launch():
    """More rows than the 2^20 workgroups of a launch take: two experts, whose
    softmax is a sigmoid of their difference (12 half steps: the difference,
    which is below 16 and errs by half a step of that, two exponentials, sum,
    quotient; the gradient as many again)."""
    T = (1 << 24) + 21
    note(f"route_topk T={T}")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    logits = torch.randn(T, 2, generator=gen, device="cuda")
    w, e = rs.route_topk(logits, 1)
    d = logits[:, 1].double() - logits[:, 0].double()
    assert torch.equal(e[:, 0].bool(), d > 0)
    p = torch.sigmoid(d.abs())
    assert ((w[:, 0].double() - p).abs() <= 32 * eo.U32 * p).all()
    g = torch.randn(T, 1, generator=gen, device="cuda")
    grad = rs.route_topk_backward(logits, e, g)
    want = torch.where(e[:, 0] == 1, 1.0, -1.0).double() * g[:, 0].double() * p * (1 - p)
    # The chosen one's a - mean = g (1 - p) loses what cancels in 1 - p.
    bound = 64 * eo.U32 * g[:, 0].double().abs()
    assert ((grad[:, 1].double() - want).abs() <= bound).all() and ((grad[:, 0].double() + want).abs() <= bound).all()


@pytest.mark.parametrize("T,k,width,num_rows", [(50, 4, 600, 200), (9000, 8, 80, 72_000), (50, 4, 600, 333)])
def test_gradient_of_unnamed_rows_in_a_graph(T, k, width, num_rows):
    """Captured, replayed with other places and on another stream: the rows that
    were named before and are not now get zeros again."""
    note(f"combine_rows_backward in a graph T={T} k={k} width={width} rows={num_rows}")
    g = torch.randn(T, width, device="cuda").bfloat16()
    rows = torch.randn(num_rows, width, device="cuda").bfloat16()
    w = torch.rand(T, k, device="cuda")
    position = torch.empty(T, k, dtype=torch.int32, device="cuda")

    def fill(seed):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        p = torch.randperm(2 * num_rows, generator=gen, device="cuda")[:T * k].to(torch.int32)
        position.copy_(torch.where(p % 5 == 0, ~p, p).reshape(T, k))
    fill(0)
    rs.combine_rows_backward(g, position, rows, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grad, grad_w = rs.combine_rows_backward(g, position, rows, w)
    side = torch.cuda.Stream()
    for seed in range(1, 5):
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        want = torch.zeros_like(rows)
        s = torch.nonzero((position.reshape(-1) >= 0) & (position.reshape(-1) < num_rows))[:, 0]
        want[position.reshape(-1)[s].long()] = (g[s // k].float() * w.reshape(-1)[s, None]).bfloat16()
        eager = rs.combine_rows_backward(g, position, rows, w)
        side.wait_stream(torch.cuda.current_stream())
        beside = rs.combine_rows_backward(g, position, rows, w, stream=side)
        torch.cuda.synchronize()
        for a, b in ((grad, grad_w), eager, beside):
            assert torch.equal(a, want) and torch.equal(b, eager[1])
