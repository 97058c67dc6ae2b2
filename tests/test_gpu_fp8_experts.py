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
