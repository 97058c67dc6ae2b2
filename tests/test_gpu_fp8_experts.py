"""Experts in e4m3 with a scale for every block of 128, and their gradients, against the definitions in 64 bits."""
import math

import pytest

import ops_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
F32, BF16, FP8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
B, TOP = 128, 448.0


@pytest.fixture(scope="module")
def ops(cuda_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixture_experts_gemm_gb300 import ops
    yield ops
    assert ops.fp8_status() == 0


def gen(seed):
    return torch.Generator().manual_seed(seed)


def e4m3(v):
    """The nearest e4m3 of fp32 values up to 448 and a little more, ties to even: by their exponents."""
    power = torch.frexp(v.double()).exponent.clamp(min=-5) - 4
    step = torch.ldexp(torch.ones_like(v, dtype=torch.float64), power)
    return ((v.double() / step).round() * step).clamp(-TOP, TOP)


def block_scales(x, down, across):
    """max |x| / 448 in fp32 over blocks of down x across of a matrix, and spread over its elements."""
    n, k = x.shape
    p = torch.zeros(-(-n // down) * down, -(-k // across) * across)
    p[:n, :k] = x.float()
    s = p.view(p.shape[0] // down, down, -1, across).abs().amax((1, 3)) / torch.tensor(TOP)
    return s, s.repeat_interleave(down, 0)[:n].repeat_interleave(across, 1)[:, :k]


def quantised(x, down, across):
    """(q as 64-bit values, scales, scales spread)."""
    s, full = block_scales(x, down, across)
    q = torch.where(full > 0, e4m3(x.float() / torch.where(full > 0, full, 1.0)), 0.0)
    return q, s, full


def weights(E, N, K, seed):
    w = torch.randn(E, N, K, generator=gen(seed)) * 100
    return w.clamp(-TOP, TOP).to(FP8), (0.5 + torch.rand(E, -(-N // B), -(-K // B), generator=gen(seed + 1))) / (100 * K**0.5)


def full(w, s):
    return w.double() * s.double().repeat_interleave(B, 1)[:, :w.shape[1]].repeat_interleave(B, 2)[:, :, :w.shape[2]]


def segments(counts):
    return torch.tensor([0, *counts]).cumsum(0).to(torch.int32)


def bound(size, blocks, out_dtype):
    """A block's sum of 128 exact products in fp32 (fed in four steps of 32: 2^-22 of the products' sizes is more than
    any order of such sums loses), the product of its two scales and that with the sum (2^-24 each, one more where the
    scales multiply one after another), an addition a block, and what 64 bits and the products of these leave: at most
    (4 + 3 + blocks + 1) 2^-24; one rounding to the type."""
    return ((8 + blocks) * 2.0**-24 + ref.half_step(out_dtype) * (out_dtype != F32)) * size


# ---- the quantiser
SHAPES = [(1, 16), (3, 128), (33, 144), (130, 400), (257, 1408)]


def special(n, K, seed, dtype):
    """Values of every size, zeros, middles of two e4m3 and blocks of zeros."""
    g = gen(seed)
    x = torch.randn(n, K, generator=g) * torch.exp(2 * torch.randn(n, 1, generator=g))
    # whole numbers: many are middles where the block's top is 448
    x[:, ::3] = torch.randint(0, 449, (n, len(range(0, K, 3))), generator=g).float()
    x[:, 0] = 448.0
    x[:, 1::7] *= 1e-5
    x[torch.rand(n, K, generator=g) < 0.1] = 0.0
    if n > 2:
        x[2] = 0.0
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,K", SHAPES)
def test_quantize_rows(ops, dtype, n, K):
    for seed, pad in ((1, 0), (2, 5), (3, 8)):
        x = special(n, K, seed, dtype)
        wide = torch.empty(n, K + pad, dtype=dtype, device="cuda")
        wide[:, :K] = x
        q, s = ops.fp8_quantize(wide[:, :K])
        want, scale, _ = quantised(x, 1, B)
        assert torch.equal(s.cpu(), scale) and torch.equal(q.cpu().double(), want)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,K", SHAPES)
def test_quantize_squares(ops, dtype, n, K):
    x = torch.stack([special(n, K, seed, dtype) for seed in (4, 5, 6)])
    q, s = ops.fp8_quantize(x.cuda(), square=True)
    assert s.shape == (3, -(-n // B), -(-K // B))
    for e in range(3):
        want, scale, _ = quantised(x[e], B, B)
        assert torch.equal(s[e].cpu(), scale) and torch.equal(q[e].cpu().double(), want)
    one, s1 = ops.fp8_quantize(x[1].cuda(), square=True)
    assert torch.equal(one.view(torch.uint8), q[1].view(torch.uint8)) and torch.equal(s1, s[1])


def test_quantize_every_quotient(ops):
    """Quotients around every boundary between two e4m3, for scales of every size down to fp32's smallest."""
    values = torch.arange(0, 127, dtype=torch.uint8).view(FP8).float()
    middles = (values[1:] + values[:-1]) / 2
    near = torch.cat([middles, torch.nextafter(middles, torch.tensor(0.0)), torch.nextafter(middles, torch.tensor(1e9))])
    for scale in (1.0, 3.0, 1 / 3, 1.7e-5, 5e30, 3e-33, 1e-38, 3e-43):
        for part in (near * scale).split(96):
            x = torch.zeros(1, 128)
            x[0, :len(part)], x[0, 127] = part, TOP * scale
            q, s = ops.fp8_quantize(x.cuda())
            want, sc, _ = quantised(x, 1, B)
            assert torch.equal(s.cpu(), sc) and torch.equal(q.cpu().double(), want), scale


def test_quantize_what_is_not_finite(ops):
    x = torch.ones(4, 288)
    x[0, 5], x[1, 130], x[2, 287] = math.inf, math.nan, -math.inf
    q, s = ops.fp8_quantize(x.cuda())
    assert torch.isnan(s).tolist() == [[True, False, False], [False, True, False], [False, False, True], [False] * 3]
    assert q[0, :128].float().eq(0).all() and q[0, 128:].float().eq(448).all()


def test_quantize_of_a_copy_on_another_stream(ops):
    """Slices that cannot be viewed as rows, on a stream that does not wait for the current one."""
    w = torch.randn(3, 40, 64, generator=gen(1)).cuda()
    for x in (w[:, :33], w.transpose(1, 2)[:, :48, :32]):
        for square in (False, True):
            want = ops.fp8_quantize(x.contiguous(), square=square)
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            torch.cuda._sleep(10_000_000)  # what the call left to the current stream would come late
            q, s = ops.fp8_quantize(x, square=square, stream=side)
            side.synchronize()
            assert torch.equal(q.view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(s, want[1])


def test_quantize_of_nothing(ops):
    q, s = ops.fp8_quantize(torch.empty(0, 256, device="cuda"))
    assert q.shape == (0, 256) and s.shape == (0, 2)
    q, s = ops.fp8_quantize(torch.empty(3, 0, 256, device="cuda"), square=True)
    assert q.shape == (3, 0, 256) and s.shape == (3, 0, 2)


# ---- products
CASES = [  # counts, N, K
    ([1], 8, 16), ([1], 128, 128), ([2, 0, 1], 200, 272), ([33], 130, 144), ([64, 31, 100], 64, 1024),
    ([128, 129, 0, 3], 257, 400), ([300, 10], 128, 2064), ([0, 0], 16, 16), ([5] * 20, 1409, 256), ([700, 300], 300, 640),
    ([513, 1, 255, 256, 257], 520, 384), ([2000], 1024, 512), ([0, 1100, 0, 900], 129, 1040),
]


def inputs(counts, N, K, dtype, seed=0, tokens=None):
    R = sum(counts)
    n = max(tokens or R, 1)
    x = torch.randn(n, K, generator=gen(seed + 1)).to(dtype)
    rows = torch.randint(0, n, (R,), generator=gen(seed + 2), dtype=torch.int32)
    return x, rows, segments(counts)


def product(x, rows, off, w, s, sizes=False):
    """x's quantised rows times the experts' weights in 64 bits; with `sizes` those of the terms."""
    q, _, scale = quantised(x, 1, B)
    v = q * scale.double()
    y = torch.zeros(len(rows), w.shape[1], dtype=torch.float64)
    W = full(w, s)
    for e in range(len(off) - 1):
        at = rows[off[e]:off[e + 1]].long()
        y[off[e]:off[e + 1]] = v[at].abs() @ W[e].abs().T if sizes else v[at] @ W[e].T
    return y


def worst(excess):
    return float(excess.max()) if excess.numel() else 0.0


@pytest.mark.parametrize("counts,N,K", CASES)
@pytest.mark.parametrize("dtype,out_dtype", [(F32, F32), (BF16, BF16), (BF16, F32)])
def test_product(ops, counts, N, K, dtype, out_dtype):
    x, rows, off = inputs(counts, N, K, dtype, 10)
    w, s = weights(len(counts), N, K, 20)
    got = ops.fp8_experts(x.cuda(), w.cuda(), s.cuda(), off.cuda(), rows=rows.cuda(), out_dtype=out_dtype).double().cpu()
    want, size = product(x, rows, off, w, s), product(x, rows, off, w, s, True)
    assert worst((got - want).abs() - bound(size, -(-K // B), out_dtype)) <= 0


@pytest.mark.parametrize("counts,N,K", CASES)
@pytest.mark.parametrize("dtype,out_dtype", [(F32, F32), (BF16, BF16)])
def test_gated_product(ops, counts, N, K, dtype, out_dtype):
    """silu(v) v3: v's bound moves silu by at most 1.1 times it (|silu'| < 1.1), each factor by the other's size, and
    the activation itself is off by (7 + 1.2 |v|) ulp with the fast exp, 7 without."""
    x, rows, off = inputs(counts, N, K, dtype, 30)
    w, s = weights(len(counts), N, K, 40)
    w3, s3 = weights(len(counts), N, K, 50)
    got = ops.fp8_experts(x.cuda(), w.cuda(), s.cuda(), off.cuda(), rows=rows.cuda(), w3=w3.cuda(), w3_scale=s3.cuda(),
                          out_dtype=out_dtype).double().cpu()
    v, v3 = product(x, rows, off, w, s), product(x, rows, off, w3, s3)
    b, b3 = (bound(product(x, rows, off, *p, True), -(-K // B), F32) for p in ((w, s), (w3, s3)))
    silu = v * torch.sigmoid(v)
    want = silu * v3
    tol = 1.1 * b * (v3.abs() + b3) + b3 * silu.abs() + (7 + 1.2 * v.abs()) * 2.0**-23 * want.abs()
    tol += ref.half_step(out_dtype) * (out_dtype != F32) * (want.abs() + tol)
    assert worst((got - want).abs() - tol) <= 0


@pytest.mark.parametrize("counts,N,K", CASES)
@pytest.mark.parametrize("dtype,weight_dtype", [(F32, F32), (BF16, BF16), (BF16, F32)])
def test_gradients(ops, counts, N, K, dtype, weight_dtype):
    x, rows, off = inputs(counts, N, K, dtype, 60)
    w, s = weights(len(counts), N, K, 70)
    R = len(rows)
    d_y = (torch.randn(R, N, generator=gen(80)) * torch.exp(torch.randn(R, 1, generator=gen(81)))).to(dtype)
    d_rows, d_w = ops.fp8_experts_backward(d_y.cuda(), x.cuda(), w.cuda(), s.cuda(), off.cuda(), rows=rows.cuda(),
                                           weight_dtype=weight_dtype)
    assert d_rows.dtype == dtype and d_w.dtype == weight_dtype
    W = full(w, s)
    for e in range(len(counts)):
        lo, hi = int(off[e]), int(off[e + 1])
        if hi > lo:
            q, _, scale = quantised(d_y[lo:hi], 1, B)
            v, got = q * scale.double(), d_rows[lo:hi].double().cpu()
            assert worst((got - v @ W[e]).abs() - bound(v.abs() @ W[e].abs(), -(-N // B), dtype)) <= 0
            dq, _, ds = quantised(d_y[lo:hi], B, 1)
            xq, _, xs = quantised(x[rows[lo:hi].long()], B, 1)
            D, X = dq * ds.double(), xq * xs.double()
            off_by = (d_w[e].double().cpu() - D.T @ X).abs()
            assert worst(off_by - bound(D.T.abs() @ X.abs(), -(-(hi - lo) // B), weight_dtype)) <= 0
        else:
            assert d_w[e].eq(0).all()
    # one at a time: the same bits
    only, none = ops.fp8_experts_backward(d_y.cuda(), None, w.cuda(), s.cuda(), off.cuda())
    assert none is None and torch.equal(only, d_rows)
    none, only = ops.fp8_experts_backward(d_y.cuda(), x.cuda(), None, None, off.cuda(), rows=rows.cuda(),
                                          weight_dtype=weight_dtype)
    assert none is None and torch.equal(only, d_w)


@pytest.mark.parametrize("counts,N,K", [([3], 200, 8192), ([40, 0, 2], 64, 65536), ([3000], 64, 64), ([1500, 1], 96, 48),
                                        ([130], 131, 144), ([1], 131072, 16)])
def test_split_and_long_products(ops, counts, N, K):
    """Few tiles and long sums (parts of the contraction added in order), few rows of many columns."""
    test_product(ops, counts, N, K, F32, F32)
    test_gradients(ops, counts, N, K, F32, F32)


def exact_inputs(rows, cols, seed):
    """Whole numbers whose blocks along rows and down columns all have the scale 1: 448 on the diagonal of every block of
    128 x 128, small ones elsewhere (e4m3 has whole numbers up to 16)."""
    x = torch.randint(-4, 5, (rows, cols), generator=gen(seed)).float()
    r, c = torch.arange(rows)[:, None] % B, torch.arange(cols)[None] % B
    return torch.where(r == c, 448.0, x)


@pytest.mark.parametrize("counts,N,K", [([128, 256, 0, 384], 384, 256), ([1024, 512], 640, 384), ([4096], 256, 128)])
def test_whole_numbers_are_exact(ops, counts, N, K):
    """Where every scale is a power of two and every sum a whole number below 2^24, results are exact: the product, the
    gradients, and these as differences of the product, which is linear in the weights and in x's values."""
    E, R = len(counts), sum(counts)
    off = segments(counts).cuda()
    x, d_y = exact_inputs(R, K, 1).cuda(), exact_inputs(R, N, 2).cuda()
    w = torch.randint(-8, 9, (E, N, K), generator=gen(3)).float().cuda()
    s = (2.0 ** torch.randint(-2, 3, (E, -(-N // B), -(-K // B)), generator=gen(4))).cuda()
    W = w.double() * s.double().repeat_interleave(B, 1)[:, :N].repeat_interleave(B, 2)[:, :, :K]
    y = ops.fp8_experts(x, w.to(FP8), s, off)
    d_rows, d_w = ops.fp8_experts_backward(d_y, x, w.to(FP8), s, off)
    for e in range(E):
        at = slice(int(off[e]), int(off[e + 1]))
        assert torch.equal(y[at].double(), x[at].double() @ W[e].T)
        assert torch.equal(d_rows[at].double(), d_y[at].double() @ W[e])
        assert torch.equal(d_w[e].double(), d_y[at].double().T @ x[at].double())
    other = torch.randint(-8, 9, (E, N, K), generator=gen(5)).float().cuda()
    moved = (ops.fp8_experts(x, other.to(FP8), torch.ones_like(s), off).double()
             - ops.fp8_experts(x, w.to(FP8), torch.ones_like(s), off).double())
    assert (moved * d_y).sum() == (d_w.double() * (other - w).double()).sum()
    there = x + torch.where(x.abs() < 448, torch.randint(0, 3, x.shape, generator=gen(6)).float().cuda(), 0.0)
    moved = ops.fp8_experts(there, w.to(FP8), s, off).double() - y.double()
    assert (moved * d_y).sum() == (d_rows.double() * (there - x).double()).sum()


def c_forward(ops, x, ldx, n, rows, R, off, w, s, y, config, space):
    L = ops.lib()
    at = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    rc = L.colibri_moe_fp8_experts(ops.ctypes.byref(config), at(x), ldx, n, at(rows), R, at(off), at(w), at(s), None, None,
                                   at(y), at(space), space.numel(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    torch.cuda.synchronize()


def space_for(ops, config, n, R, backward=False):
    size = ops.ctypes.c_size_t()
    f = ops.lib().colibri_moe_fp8_experts_backward_workspace if backward else ops.lib().colibri_moe_fp8_experts_workspace
    assert f(ops.ctypes.byref(config), n, R, ops.ctypes.byref(size)) == 0
    return torch.empty(size.value, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("R,bounds", [(300, [0, 100, 40, 200, 250]), (300, [5, 290, 1000, 2000, -3]), (900, [0, 600, 600, 700, 850]),
                                      (40, [0, 0, 0, 0, 0])])
def test_segments_as_they_come(ops, R, bounds):
    """Offsets outside 0..R are clamped, rows that an earlier segment holds stay with it, and rows of no segment, behind the
    last one too, are left as they were."""
    E, N, K = 4, 136, 160
    x = torch.randn(R, K, generator=gen(R)).cuda()
    w, s = weights(E, N, K, 7)
    off = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    config = ops.Fp8Config(K, N, E, 0, 0, 0, 0)
    y = torch.full((R, N), 7.0, device="cuda")
    c_forward(ops, x, K, R, None, R, off, w.cuda(), s.cuda(), y, config, space_for(ops, config, R, R))
    owner, reach = torch.full((R,), -1), 0
    for e in range(E):
        lo, hi = (min(max(b, 0), R) for b in bounds[e:e + 2])
        owner[max(lo, reach):hi] = e
        reach = max(reach, hi)
    rows = torch.arange(R)
    for e in range(E):
        at = rows[owner == e]
        if len(at):
            # not the bits of a call on these rows alone: that may split its sums otherwise
            args = x.cpu(), at, segments([len(at)]), w[e:e + 1], s[e:e + 1]
            off_by = (y[at.cuda()].double().cpu() - product(*args)).abs()
            assert worst(off_by - bound(product(*args, True), -(-K // B), F32)) <= 0
    assert y[(owner < 0).cuda()].eq(7).all()


@pytest.mark.parametrize("R", [70, 700])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strides_and_tokens(ops, R, dtype):
    """Rows of any stride and alignment, tokens outside x (rows of zeros), no row map: the bits of the plain call."""
    E, N, K = 3, 100, 176
    x, rows, off = inputs([R // 2, 0, R - R // 2], N, K, dtype, R)
    w, s = (t.cuda() for t in weights(E, N, K, 9))
    off, x = off.cuda(), x.cuda()
    rows[::7], rows[3::11] = -1, len(x)
    rows = rows.cuda()
    there = torch.cat([x, torch.zeros(1, K, dtype=dtype, device="cuda")])[torch.where((rows < 0) | (rows >= len(x)), len(x), rows).long()]
    want = ops.fp8_experts(there, w, s, off)
    d_y = torch.randn(R, N, generator=gen(1)).to(dtype).cuda()
    grads = ops.fp8_experts_backward(d_y, there, w, s, off)
    for pad, first in ((0, 0), (8, 8), (5, 3)):
        wide = torch.full((len(x), K + pad + first), math.nan, dtype=dtype, device="cuda")
        wide[:, first:first + K] = x
        deep = torch.full((R, N + pad + first), math.nan, dtype=dtype, device="cuda")
        deep[:, first:first + N] = d_y
        assert torch.equal(ops.fp8_experts(wide[:, first:first + K], w, s, off, rows=rows), want)
        got = ops.fp8_experts_backward(deep[:, first:first + N], wide[:, first:first + K], w, s, off, rows=rows)
        assert all(torch.equal(a, b) for a, b in zip(got, grads))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", ["random", "one token", "half without", "every token alike"])
def test_tokens_of_many_rows(ops, dtype, kind):
    """Enough repeated values that tokens are quantised once and written to all of their rows: the bits of the call on the
    repeated rows themselves, whatever the map: a token of thousands of rows, rows without one, values by division."""
    n, R, K, N, E = 700, 9100, 2064, 72, 3
    x = special(n, K, 3, dtype).cuda()
    g = gen(4)
    rows = {"random": torch.randint(-1, n + 1, (R,), generator=g), "one token": torch.full((R,), 5),
            "half without": torch.where(torch.rand(R, generator=g) < 0.5, torch.randint(0, n, (R,), generator=g), -1),
            "every token alike": torch.arange(R) % n}[kind].int().cuda()
    w, s = (t.cuda() for t in weights(E, N, K, 9))
    off = segments([4000, 100, 5000]).cuda()
    there = torch.cat([x, torch.zeros(1, K, dtype=dtype, device="cuda")])[torch.where((rows < 0) | (rows >= n), n, rows).long()]
    want = ops.fp8_experts(there, w, s, off)
    for _ in range(2):
        assert torch.equal(ops.fp8_experts(x, w, s, off, rows=rows), want)


def test_a_captured_call_follows_its_map(ops):
    """Tokens of many rows in a graph: every replay goes by the map and the values that it finds, with nothing left of the
    last one's."""
    n, R, K, N, E = 700, 9100, 2064, 72, 3
    g = gen(6)
    x, rows = special(n, K, 3, BF16).cuda(), torch.full((R,), 5).int().cuda()
    w, s = (t.cuda() for t in weights(E, N, K, 9))
    off = segments([4000, 100, 5000]).cuda()
    ops.fp8_experts(x, w, s, off, rows=rows)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = ops.fp8_experts(x, w, s, off, rows=rows)
    for map_ in (torch.randint(-1, n + 1, (R,), generator=g), torch.full((R,), -1), torch.arange(R) % n, torch.full((R,), 5)):
        rows.copy_(map_)
        x.copy_(special(n, K, int(map_.sum()) % 97, BF16))
        token = torch.where((rows < 0) | (rows >= n), n, rows).long()
        want = ops.fp8_experts(torch.cat([x, torch.zeros_like(x[:1])])[token], w, s, off)
        graph.replay()
        assert torch.equal(got, want)


@pytest.mark.parametrize("R", [90, 900])
def test_what_is_not_finite_stays_where_it_enters(ops, R):
    """A row with a NaN or an infinity has NaN in all its results; other rows, of the same tile too, and other experts'
    gradients keep their bits.  So do experts beside one whose weights are NaN."""
    E, N, K = 2, 136, 272
    counts = [R // 3, R - R // 3]
    x, rows, off = inputs(counts, N, K, F32, 3)
    x, off = x.cuda()[:R], off.cuda()
    w, s = (t.cuda() for t in weights(E, N, K, 11))
    d_y = torch.randn(R, N, generator=gen(2)).cuda()
    want, (d_rows, d_w) = ops.fp8_experts(x, w, s, off), ops.fp8_experts_backward(d_y, x, w, s, off)
    bad, bad_dy = x.clone(), d_y.clone()
    bad[1, 200], bad[5, 0], bad_dy[2, 100], bad_dy[7, 3] = math.nan, math.inf, -math.inf, math.nan
    y = ops.fp8_experts(bad, w, s, off)
    hit = torch.zeros(R, dtype=torch.bool, device="cuda")
    hit[[1, 5]] = True
    assert torch.isnan(y[hit]).all() and torch.equal(y[~hit], want[~hit])
    got_rows, got_w = ops.fp8_experts_backward(bad_dy, bad, w, s, off)
    hit[:] = False
    hit[[2, 7]] = True
    assert torch.isnan(got_rows[hit]).all() and torch.equal(got_rows[~hit], d_rows[~hit])
    assert torch.equal(got_w[1], d_w[1])
    assert torch.isnan(got_w[0][[100, 3]]).all() and torch.isnan(got_w[0][:, [200, 0]]).all()
    keep_n, keep_k = torch.ones(N, dtype=torch.bool), torch.ones(K, dtype=torch.bool)
    keep_n[[100, 3]], keep_k[[200, 0]] = False, False
    assert torch.equal(got_w[0][keep_n.cuda()][:, keep_k.cuda()], d_w[0][keep_n.cuda()][:, keep_k.cuda()])
    nan_w = w.clone()
    nan_w.view(torch.uint8)[1] = 0x7f
    assert torch.equal(ops.fp8_experts(x, nan_w, s, off)[:counts[0]], want[:counts[0]])
    assert torch.equal(ops.fp8_experts_backward(d_y, None, nan_w, s, off)[0][:counts[0]], d_rows[:counts[0]])


def test_no_rows(ops):
    w, s = (t.cuda() for t in weights(2, 24, 32, 1))
    off, x, none = segments([0, 0]).cuda(), torch.ones(3, 32, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    assert ops.fp8_experts(x, w, s, off, rows=none).shape == (0, 24)
    d_rows, d_w = ops.fp8_experts_backward(torch.empty(0, 24, device="cuda"), x, w, s, off, rows=none)
    assert d_rows.shape == (0, 32) and d_w.shape == (2, 24, 32) and d_w.eq(0).all()
    # rows, but none of an expert: no gradient of a weight
    d_rows, d_w = ops.fp8_experts_backward(torch.ones(3, 24, device="cuda"), x, w, s, off)
    assert d_w.eq(0).all()
    # no tokens: every row is zeros
    y = ops.fp8_experts(x[:0], w, s, segments([2, 1]).cuda(), rows=torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert y.eq(0).all()


# ---- streams, graphs, waits
@pytest.mark.parametrize("counts", [[3, 0, 1], [90, 40, 100], [400, 300, 500]], ids=str)
def test_graphs_and_streams(ops, counts):
    """The same bits from a captured and replayed call with other inputs, from two streams at once, and time after time."""
    N, K = 392, 1040
    data = [inputs(counts, N, K, BF16, i) for i in (1, 2)]
    xs = [d[0][:sum(counts)].cuda() for d in data]
    off = data[0][2].cuda()
    w, s = (t.cuda() for t in weights(3, N, K, 5))
    d_y = torch.randn(sum(counts), N, generator=gen(3)).bfloat16().cuda()

    def step(x, stream=None):
        return (ops.fp8_experts(x, w, s, off, w3=w, w3_scale=s, stream=stream),
                *ops.fp8_experts_backward(d_y, x, w, s, off, stream=stream))

    want = [step(x) for x in xs]
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(step(xs[0]), want[0]))
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[step(x, t) for x, t in zip(xs, streams)] for _ in range(4)]
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for p, q in zip(g, want) for a, b in zip(p, q))
    x = xs[0].clone()
    graphs, outs = [], []
    for _ in range(2):  # two graphs, each with its own workspace
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(step(x))
    for i in (1, 0):
        x.copy_(xs[i])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        for out in outs:
            assert all(torch.equal(a, b) for a, b in zip(out, want[i]))


@pytest.mark.parametrize("counts", [[1, 0, 1], [128, 1, 97], [300, 257, 255]], ids=str)
def test_a_wait_that_runs_out(ops, counts):
    """Products told to wait for a microsecond at most (to within about 20) finish, or stop and say so; the next call, in
    the same workspace, gives what a call without the limit gives."""
    K, N, E, R = 4096, 520, len(counts), sum(counts)
    x = torch.randn(R, K, generator=gen(R)).cuda()
    w, s = (t.cuda() for t in weights(E, N, K, R))
    off = segments(counts).cuda()
    want = ops.fp8_experts(x, w, s, off)
    d_y = torch.randn(R, N, generator=gen(1)).cuda()
    grads = ops.fp8_experts_backward(d_y, x, w, s, off)
    assert ops.fp8_status() == 0
    config = lambda us: ops.Fp8Config(K, N, E, 0, 0, 0, us)  # noqa: E731
    space = [space_for(ops, config(0), R, R, b) for b in (False, True)]

    def call(us):
        y, d_rows, d_w = torch.empty_like(want), torch.empty_like(grads[0]), torch.empty_like(grads[1])
        c_forward(ops, x, K, R, None, R, off, w, s, y, config(us), space[0])
        rc = ops.lib().colibri_moe_fp8_experts_backward(
            ops.ctypes.byref(config(us)), d_y.data_ptr(), N, x.data_ptr(), K, R, None, R, off.data_ptr(), w.data_ptr(),
            s.data_ptr(), d_rows.data_ptr(), d_w.data_ptr(), space[1].data_ptr(), space[1].numel(),
            torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        torch.cuda.synchronize()
        return all(torch.equal(a, b) for a, b in zip((y, d_rows, d_w), (want, *grads)))

    for _ in range(2):
        same = call(1)
        assert ops.fp8_status() == 1 or same
        assert call(0) and ops.fp8_status() == 0
    assert call(10_000_000) and ops.fp8_status() == 0


@pytest.mark.parametrize("R", [10, 600])
def test_a_wait_that_runs_out_is_reported(ops, R):
    """The status word: set once by a call that gave up, from any stream, then clear.  65536 columns of 256 channels are at
    least 64 blocks of each part, 20 us and more that the last tile's takers wait for the first copies and sums."""
    K, N = 65536, 256
    x = torch.randn(R, K, generator=gen(3)).cuda()
    w, s = (t.cuda() for t in weights(1, N, K, 4))
    off = segments([R]).cuda()
    want = ops.fp8_experts(x, w, s, off)
    assert ops.fp8_status() == 0
    real = ops._fp8_config
    config = ops.Fp8Config(K, N, 1, 0, 0, 1, 1)
    for stream in (None, torch.cuda.Stream()):
        ops._fp8_config = lambda *a: (config, ops.ctypes.addressof(config))
        try:
            y = ops.fp8_experts(x, w, s, off, stream=stream)
        finally:
            ops._fp8_config = real
        gave_up = ops.fp8_status()  # waits for the device
        assert gave_up == 1 or torch.equal(y, want)
        y = ops.fp8_experts(x, w, s, off, stream=stream)
        assert ops.fp8_status(0) == 0 and torch.equal(y, want)
