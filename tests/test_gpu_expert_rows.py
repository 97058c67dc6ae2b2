"""Tokens to their experts' rows and back, and the gated activation, against plain 64-bit forms."""
import math

import numpy as np
import pytest

import ops_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
F32, BF16 = torch.float32, torch.bfloat16
TYPES = [F32, BF16]


@pytest.fixture(scope="module")
def ops(cuda_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixture_experts_gemm_gb300 import ops
    return ops


def gen(seed):
    return torch.Generator().manual_seed(seed)


def choice(T, k, E, seed, dropped=0.0, twice=False):
    """idx [T, k] int32: distinct experts, or with `twice` any; some slots dropped by values outside 0..E-1."""
    g = gen(seed)
    idx = torch.randint(0, E, (T, k), generator=g) if twice else torch.rand(T, E, generator=g).topk(k).indices
    out = torch.tensor([-1, E, -2**31, 2**31 - 1])[torch.randint(0, 4, (T, k), generator=g)]
    return torch.where(torch.rand(T, k, generator=g) < dropped, out, idx).to(torch.int32)


def order_of(idx, E):
    """Counts, offsets, row_of and token_of_row by sorting Python tuples."""
    T, k = idx.shape
    flat = idx.reshape(-1).tolist()
    slots = sorted((e, i) for i, e in enumerate(flat) if 0 <= e < E)
    row_of, token = np.full(T * k, -1), np.full(T * k, -1)
    for r, (_, i) in enumerate(slots):
        row_of[i], token[r] = r, i // k
    counts = np.bincount([e for e, _ in slots], minlength=E)
    return counts, np.concatenate([[0], counts.cumsum()]), row_of.reshape(T, k), token


@pytest.mark.parametrize("T,k,E,dropped,twice", [
    (1, 1, 1, 0, False), (1, 8, 256, 0, False), (1, 32, 512, 0.2, False), (3, 2, 8, 1.0, False), (31, 3, 7, 0.1, True),
    (512, 2, 8, 0, False), (513, 2, 8, 0.1, False), (1024, 2, 512, 0, True), (1025, 1, 4, 0, False), (2000, 5, 60, 0.3, True),
    (4099, 4, 60, 0.1, False), (8192, 2, 8, 0, False), (9000, 10, 512, 0.05, False), (20001, 32, 33, 0.5, True),
])
def test_order(ops, T, k, E, dropped, twice):
    idx = choice(T, k, E, T + k, dropped, twice)
    o = ops.dispatch_order(idx.cuda(), E)
    for got, want in zip(o, order_of(idx, E)):
        assert np.array_equal(got.cpu().numpy(), want)


def test_order_of_no_tokens(ops):
    o = ops.dispatch_order(torch.empty(0, 3, dtype=torch.int32, device="cuda"), 5)
    assert o.counts.tolist() == [0] * 5 and o.offsets.tolist() == [0] * 6
    assert o.row_of.shape == (0, 3) and o.token_of_row.shape == (0,)


def test_order_is_routing_s(ops):
    r = ops.route(torch.randn(777, 60, generator=gen(3)).cuda(), 6)
    for got, want in zip(ops.dispatch_order(r.idx, 60), (r.counts, r.offsets, r.row_of, r.token_of_row)):
        assert torch.equal(got, want)


WIDTHS = [1, 7, 8, 64, 200, 1409, 4096, 65536]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", WIDTHS)
def test_rows(ops, dtype, d):
    """Copies: the bits of x, NaN payloads among them, for every alignment of rows and strides."""
    T, R = (3, 5) if d > 5000 else (70, 150)
    token = torch.randint(-1, T, (R,), generator=gen(d), dtype=torch.int32)
    token[0] = T  # outside: a row of zeros, too
    for pad, first in ((0, 0), (8, 0), (3, 1), (8, 8)):
        wide = torch.randn(T, d + pad + first, generator=gen(d + pad)).to(dtype).cuda()
        wide[0, first] = math.nan
        x = wide[:, first:first + d]
        rows = ops.dispatch(x, token.cuda())
        want = torch.where(((token >= 0) & (token < T))[:, None].cuda(), x[token.long().clamp(0, T - 1).cuda()],
                           torch.zeros((), dtype=dtype, device="cuda"))
        ints = torch.int32 if dtype == F32 else torch.int16
        assert torch.equal(rows.view(ints), want.contiguous().view(ints))


def back_bound(dtype, out_dtype, size, k):
    """A sum of k values in fp32, k - 1 additions, each off by half a step of a partial sum that is at most the sum of
    the values' sizes, then one rounding to out_dtype."""
    return (k * 2.0**-24 + ref.half_step(out_dtype) * (out_dtype != F32) * (1 + k * 2.0**-24)) * size


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("out_dtype", TYPES)
@pytest.mark.parametrize("T,k,d", [(1, 1, 1), (1, 8, 4096), (5, 32, 64), (300, 2, 1409), (300, 3, 200), (4, 4, 65536)])
def test_rows_back(ops, dtype, out_dtype, T, k, d):
    E = 40
    idx = choice(T, k, E, d + k, 0.2)
    _, _, row_of, _ = order_of(idx, E)
    g = torch.randn(T * k, d, generator=gen(d)).to(dtype)
    got = ops.dispatch_backward(g.cuda(), torch.from_numpy(row_of).int().cuda(), out_dtype=out_dtype).double().cpu()
    v = np.where((row_of >= 0)[:, :, None], g.double().numpy()[np.maximum(row_of, 0)], 0.0)
    off = (got - torch.from_numpy(v.sum(1))).abs() - back_bound(dtype, out_dtype, torch.from_numpy(np.abs(v).sum(1)), k)
    assert float(off.max()) <= 0


def test_rows_back_is_the_transpose_of_rows(ops):
    """<dispatch(x), g> = <x, dispatch_backward(g)> on whole numbers, where every sum is exact."""
    T, k, E, d = 90, 4, 9, 72
    o = ops.dispatch_order(choice(T, k, E, 5, 0.3, twice=True).cuda(), E)
    x = torch.randint(-8, 9, (T, d), generator=gen(6)).float().cuda()
    g = torch.randint(-8, 9, (T * k, d), generator=gen(7)).float().cuda()
    left = (ops.dispatch(x, o.token_of_row) * g).double().sum()
    assert left == (x * ops.dispatch_backward(g, o.row_of)).double().sum()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("y_dtype", TYPES)
@pytest.mark.parametrize("T,k,d,pad", [(1, 1, 1, 0), (1, 8, 4096, 0), (5, 32, 64, 0), (300, 2, 1409, 0), (300, 3, 200, 8),
                                       (300, 9, 200, 3), (4, 2, 65536, 0)])
def test_combine_backward(ops, dtype, y_dtype, T, k, d, pad):
    """d_y = gate * d_out: one rounded product, one rounding to y's type.  d_gate: d products and d additions in fp32 in
    some order, off by at most 2^-24 of the sum of the products' sizes each, where a thread's sum has at most
    ceil(d / 128) terms, a warp's and the block's 5 + 4 more: (d / 128 + 12) 2^-24."""
    E = 40
    idx = choice(T, k, E, d + k, 0.2)
    _, _, row_of, token = order_of(idx, E)
    d_out = torch.randn(T, d + pad, generator=gen(d)).to(dtype)[:, :d]
    y = torch.randn(T * k, d, generator=gen(d + 1)).to(y_dtype)
    gate = torch.rand(T, k, generator=gen(d + 2))
    wide = torch.empty(T, d + pad, dtype=dtype, device="cuda")
    wide[:, :d] = d_out
    d_y, d_gate = ops.combine_backward(wide[:, :d], y.cuda(), torch.from_numpy(row_of).int().cuda(), gate.cuda(),
                                       torch.from_numpy(token).int().cuda())
    kept, at = torch.from_numpy(row_of >= 0), torch.from_numpy(np.maximum(row_of, 0))
    G, Y = d_out.double(), y.double()
    terms = torch.where(kept[:, :, None], Y[at] * G[:, None, :], 0.0)
    off = (d_gate.double().cpu() - terms.sum(2)).abs() - (d / 128 + 12) * 2.0**-24 * terms.abs().sum(2)
    assert float(off.max()) <= 0
    want = torch.zeros_like(Y)
    want[at[kept]] = (gate.double()[:, :, None] * G[:, None, :])[kept]
    off = (d_y.double().cpu() - want).abs() - (2.0**-24 + ref.half_step(y_dtype) * 1.01 * (y_dtype != F32)) * want.abs()
    assert float(off.max()) <= 0


def test_combine_backward_is_combine_s_gradient(ops):
    """Whole numbers, where every sum is exact: the combine is linear in y and in the gates, so differences are the
    gradients.  One expert twice for a token among them."""
    T, k, E, d = 33, 3, 5, 40
    o = ops.dispatch_order(choice(T, k, E, 8, 0.2, twice=True).cuda(), E)
    ints = lambda seed, *s: torch.randint(-4, 5, s, generator=gen(seed)).float().cuda()  # noqa: E731
    y, gate, d_out, dy, dg = ints(1, T * k, d), ints(2, T, k), ints(3, T, d), ints(4, T * k, d), ints(5, T, k)
    d_y, d_gate = ops.combine_backward(d_out, y, o.row_of, gate, o.token_of_row)
    moved = lambda a, b: ((a - b).double() * d_out).sum()  # noqa: E731
    was = ops.combine(y, o.row_of, gate)
    assert moved(ops.combine(y + dy, o.row_of, gate), was) == (d_y * dy).double().sum()
    assert moved(ops.combine(y, o.row_of, gate + dg), was) == (d_gate * dg).double().sum()


def test_combine_backward_of_a_row_named_twice(ops):
    """Two slots of a token that name one row give it the sum of their gates."""
    row_of = torch.tensor([[0, 0, 1], [2, -1, 2]], dtype=torch.int32, device="cuda")
    token = torch.tensor([0, 0, 1, -1], dtype=torch.int32, device="cuda")
    gate = torch.tensor([[1.0, 2.0, 4.0], [8.0, 16.0, 32.0]], device="cuda")
    d_out = torch.tensor([[1.0] * 16, [3.0] * 16], device="cuda")
    y = torch.ones(4, 16, device="cuda")
    d_y, d_gate = ops.combine_backward(d_out, y, row_of, gate, token)
    assert d_y[:, 0].tolist() == [3.0, 4.0, 120.0, 0.0]
    assert d_gate.tolist() == [[16.0, 16.0, 16.0], [48.0, 0.0, 48.0]]


def test_no_tokens_and_no_rows(ops):
    none = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    x = torch.empty(0, 16, device="cuda")
    t = torch.tensor([-1, 0], dtype=torch.int32, device="cuda")
    assert ops.dispatch(x, t).tolist() == [[0.0] * 16] * 2
    assert ops.dispatch(torch.ones(2, 16, device="cuda"), t[:0]).shape == (0, 16)
    assert ops.dispatch_backward(torch.ones(4, 16, device="cuda"), none).shape == (0, 16)
    assert ops.dispatch_backward(x, torch.full((3, 2), -1, dtype=torch.int32, device="cuda")).eq(0).all()
    d_y, d_gate = ops.combine_backward(x, torch.ones(2, 16, device="cuda"), none, torch.empty(0, 2, device="cuda"), t)
    assert d_y.eq(0).all() and d_gate.shape == (0, 2)
    d_y, d_gate = ops.combine_backward(torch.ones(3, 16, device="cuda"), x, torch.full((3, 2), -1, dtype=torch.int32,
                                       device="cuda"), torch.ones(3, 2, device="cuda"), t[:0])
    assert d_y.shape == (0, 16) and d_gate.eq(0).all()


def test_infinities_behind_dropped_slots(ops):
    """Rows and gates that no slot reads may hold anything."""
    row_of = torch.tensor([[0, -1]], dtype=torch.int32, device="cuda")
    token = torch.tensor([0, -1], dtype=torch.int32, device="cuda")
    y = torch.ones(2, 24, device="cuda")
    y[1] = math.nan
    gate = torch.tensor([[0.5, math.inf]], device="cuda")
    d_y, d_gate = ops.combine_backward(torch.ones(1, 24, device="cuda"), y, row_of, gate, token)
    assert d_y.tolist() == [[0.5] * 24, [0.0] * 24] and d_gate.tolist() == [[24.0, 0.0]]
    assert ops.dispatch_backward(y, row_of).eq(1).all()


# ---- gated activation
def silu_parts(u):
    p = torch.sigmoid(u)
    return u * p, p * (1 + u * (1 - p))


def gated_error(fast):
    """Relative error of p and of 1 - p: exp to 2 ulp of fp32 (the fast one to 4 + 1.2 |u| ulp), one addition, the
    reciprocal to one ulp, a product."""
    return lambda u: ((4 + 1.2 * u.abs()) if fast else 2) * 2.0**-23 + 2.5 * 2.0**-23


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("out_dtype", TYPES)
@pytest.mark.parametrize("R,f,halves", [(1, 1, False), (1, 14336, True), (3, 64, False), (40, 1409, True), (33, 200, True),
                                        (513, 24, False), (2, 65536, False), (70000, 8, False)])
def test_gated(ops, dtype, out_dtype, R, f, halves):
    """h = u p v: the error of p, two products; and one rounding."""
    both = (3 * torch.randn(R, 2 * f, generator=gen(f))).to(dtype)
    u, v = both[:, :f], both[:, f:]
    cu, cv = (both.cuda()[:, :f], both.cuda()[:, f:]) if halves else (u.contiguous().cuda(), v.contiguous().cuda())
    got = ops.gated(cu, cv, out_dtype=out_dtype).double().cpu()
    U, V = u.double(), v.double()
    want = silu_parts(U)[0] * V
    tol = gated_error(out_dtype == BF16)(U) + 2 * 2.0**-24 + ref.half_step(out_dtype) * (out_dtype != F32)
    assert float(((got - want).abs() - tol * 1.01 * want.abs()).max()) <= 1e-36


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("h_dtype", TYPES)
@pytest.mark.parametrize("R,f,halves", [(1, 1, False), (1, 14336, True), (3, 64, False), (40, 1409, True), (33, 200, True),
                                        (513, 24, False), (2, 65536, False), (70000, 8, False)])
def test_gated_backward(ops, dtype, h_dtype, R, f, halves):
    """d_v = g u p: as h.  d_u = g v p (1 + u q): the errors of p and q and four roundings, of 1 + |u| q where u < 0
    cancels, and one rounding to the type."""
    both = (3 * torch.randn(R, 2 * f, generator=gen(f))).to(dtype)
    u, v = both[:, :f], both[:, f:]
    cu, cv = (both.cuda()[:, :f], both.cuda()[:, f:]) if halves else (u.contiguous().cuda(), v.contiguous().cuda())
    g = torch.randn(R, f, generator=gen(f + 1)).to(h_dtype)
    d_u, d_v = ops.gated_backward(g.cuda(), cu, cv)
    U, V, G = u.double(), v.double(), g.double()
    e = gated_error(dtype == BF16)(U) + 4 * 2.0**-24
    half = ref.half_step(dtype) * (dtype != F32)
    silu, slope = silu_parts(U)
    want = G * silu
    assert float(((d_v.double().cpu() - want).abs() - (e + half) * 1.01 * want.abs()).max()) <= 1e-36
    want, p = G * V * slope, torch.sigmoid(U)
    size = (G * V).abs() * p * (1 + U.abs() * (1 - p))
    assert float(((d_u.double().cpu() - want).abs() - 2 * e * 1.01 * size - half * 1.01 * want.abs()).max()) <= 1e-36


def test_gated_backward_is_gated_s_gradient(ops):
    """Differences of h in 64 bits: the step's error is h''' s^2 / 6 with |silu'''| < 1, and h's own error in fp32 over
    the step."""
    g = gen(9)
    u, v, d_h = (torch.randn(50, 33, generator=g).cuda() for _ in range(3))
    d_u, d_v = ops.gated_backward(d_h, u, v)
    s = 2.0**-6
    h = lambda a, b: ops.gated(a, b).double()  # noqa: E731
    for got, up, down, far in ((d_u, h(u + s, v), h(u - s, v), v.double().abs() * s * s / 6),
                               (d_v, h(u, v + s), h(u, v - s), 0.0)):
        want = (up - down) / (2 * s) * d_h
        size = (up.abs() + down.abs()) * 12 * 2.0**-24 / (2 * s) + 2.0**-22 * (u.abs() + v.abs() + 1) / (2 * s)
        assert float(((got - want).abs() - (far + size) * d_h.abs() - 1e-5).max()) <= 0


@pytest.mark.parametrize("pad,first", [(8, 0), (8, 8), (5, 3)])
def test_gated_of_strided_rows(ops, pad, first):
    """Every operand with a stride and an alignment of its own: the bits of the contiguous call."""
    R, f = 21, 264
    u, v, g = (torch.randn(R, f, generator=gen(i)).bfloat16().cuda() for i in range(3))
    wide = [torch.full((R, f + first + (i + 1) * pad), math.nan, dtype=BF16, device="cuda") for i in range(3)]
    for w, t in zip(wide, (u, v, g)):
        w[:, first:first + f] = t
    a, b, c = (w[:, first:first + f] for w in wide)
    assert torch.equal(ops.gated(a, b), ops.gated(u, v))
    for got, want in zip(ops.gated_backward(c, a, b), ops.gated_backward(g, u, v)):
        assert torch.equal(got, want)


def test_gated_at_the_ends(ops):
    """Far from zero silu is 0 or u; nothing overflows on the way."""
    u = torch.tensor([[-3e38, -1e4, -104.0, -88.0, -0.0, 0.0, 88.0, 1e4, 3e38, math.nan]]).cuda()
    v = torch.ones_like(u)
    for out in TYPES:
        h = ops.gated(u, v, out_dtype=out)[0].tolist()
        assert h[:2] == [0.0, 0.0] and h[4:6] == [0.0, 0.0] and math.isnan(h[9])
        assert abs(h[2]) < 1e-40 and abs(h[3] + 88 * math.exp(-88)) < 1e-38
        assert h[6:9] == u[0, 6:9].to(out).tolist()
    d_u, d_v = ops.gated_backward(v, u, v)
    assert d_u[0, :2].eq(0).all() and d_u[0, 4:9].tolist() == [0.5, 0.5, 1.0, 1.0, 1.0] and d_v[0, 8] == u[0, 8]


# ---- streams, graphs
def step(ops, x, idx, E, gate, g):
    o = ops.dispatch_order(idx, E)
    rows = ops.dispatch(x, o.token_of_row)
    h = ops.gated(rows, rows)
    y = ops.combine(h, o.row_of, gate)
    d_h, d_gate = ops.combine_backward(g, h, o.row_of, gate, o.token_of_row)
    d_u, d_v = ops.gated_backward(d_h, rows, rows)
    return y, d_gate, ops.dispatch_backward(d_u + d_v, o.row_of)


def test_step_in_a_graph_and_on_another_stream(ops):
    """The chain as a training step runs it: eagerly, on a stream of its own and replayed with other inputs, the same
    bits."""
    T, k, E, d = 700, 3, 12, 136
    x = [torch.randn(T, d, generator=gen(i)).bfloat16().cuda() for i in (1, 2)]
    idx = [choice(T, k, E, i, 0.1).cuda() for i in (3, 4)]
    gate, g = torch.rand(T, k, generator=gen(5)).cuda(), torch.randn(T, d, generator=gen(6)).bfloat16().cuda()
    want = [step(ops, a, b, E, gate, g) for a, b in zip(x, idx)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(ops, x[0], idx[0], E, gate, g)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    a, b = x[0].clone(), idx[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(ops, a, b, E, gate, g)
    for i in (1, 0, 1):
        a.copy_(x[i]), b.copy_(idx[i])
        graph.replay()
        assert all(torch.equal(p, q) for p, q in zip(out, want[i]))
