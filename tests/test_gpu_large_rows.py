"""The expert layer's training operators where element numbers pass 2^31 (buffers of 5 to 9 GB)."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
BF16, FP8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def ops(cuda_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixture_experts_gemm_gb300 import ops
    yield ops
    torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def test_rows_there_and_back(ops):
    T, k, d, E = 20000, 30, 4096, 64  # 600000 rows: 2.46e9 values
    x = torch.randint(-8, 9, (T, d), generator=gen(1), device="cuda").to(BF16)
    idx = torch.rand(T, E, generator=gen(2), device="cuda").topk(k).indices.int()
    o = ops.dispatch_order(idx, E)
    rows = ops.dispatch(x, o.token_of_row)
    at = torch.tensor([0, 1, 2**31 // d - 1, 2**31 // d, 2**31 // d + 1, T * k - 1], device="cuda")
    assert torch.equal(rows[at], x[o.token_of_row[at].long()])
    assert torch.equal(ops.dispatch_backward(rows, o.row_of, out_dtype=torch.float32), k * x.float())
    gate = torch.ones(T, k, device="cuda")
    d_y, d_gate = ops.combine_backward(x, rows, o.row_of, gate, o.token_of_row)
    assert torch.equal(d_y[at], rows[at])
    assert torch.equal(d_gate, x.float().square().sum(1, keepdim=True).expand(T, k))


def test_gated(ops):
    R, f = 40000, 65536
    u = torch.empty(R, f, dtype=BF16, device="cuda").fill_(0.5)
    u[-1], u[0] = 2.0, -1.0
    h = ops.gated(u, u)
    d_u, d_v = ops.gated_backward(u, u, u)
    small = u[[0, 1, R // 2 + 1, R - 1]]
    assert torch.equal(h[[0, 1, R // 2 + 1, R - 1]], ops.gated(small, small))
    for a, b in zip((d_u, d_v), ops.gated_backward(small, small, small)):
        assert torch.equal(a[[0, 1, R // 2 + 1, R - 1]], b)


def weights(E, N, K, seed):
    w = torch.randint(-8, 9, (E, N, K), generator=gen(seed), device="cuda", dtype=torch.int8).to(BF16).to(FP8)
    return w, torch.ones(E, -(-N // 128), -(-K // 128), device="cuda")


def test_product(ops):
    """One block of the contraction: no call splits it, so the last rows alone give the same bits."""
    R, K, N = 40000, 64, 65536
    x = torch.randn(R, K, generator=gen(3), device="cuda")
    w, s = weights(1, N, K, 4)
    off = lambda n: torch.tensor([0, n], dtype=torch.int32, device="cuda")  # noqa: E731
    y = ops.fp8_experts(x, w, s, off(R), out_dtype=BF16)
    assert torch.equal(y[-200:], ops.fp8_experts(x[-200:], w, s, off(200), out_dtype=BF16))
    assert torch.equal(y[32700:32900], ops.fp8_experts(x[32700:32900], w, s, off(200), out_dtype=BF16))
    # and back: d_y of as many values
    d_rows, d_w = ops.fp8_experts_backward(y, x.to(BF16), w, s, off(R))
    small = ops.fp8_experts_backward(y[-200:], None, w, s, off(200))[0]
    scale = small.float().abs().max()
    assert ((d_rows[-200:].float() - small.float()).abs() <= 2.0**-7 * scale).all()  # sums of 512 blocks, split otherwise
    assert torch.isfinite(d_w).all()
    assert ops.fp8_status() == 0


def test_weights_gradient(ops):
    E, N, K = 40, 8192, 8192  # 2.7e9 values
    counts = [0] * (E - 2) + [100, 60]
    off = torch.tensor([0, *counts], device="cuda").cumsum(0).int()
    x, d_y = (torch.randn(160, n, generator=gen(n + 1), device="cuda") for n in (K, N))
    _, d_w = ops.fp8_experts_backward(d_y, x, None, None, off, weight_dtype=BF16)
    for e, at in ((E - 2, slice(0, 100)), (E - 1, slice(100, 160))):
        one = torch.tensor([0, at.stop - at.start], dtype=torch.int32, device="cuda")
        assert torch.equal(d_w[e], ops.fp8_experts_backward(d_y[at], x[at], None, None, one, weight_dtype=BF16)[1][0])
    assert d_w[:E - 2].count_nonzero() == 0
