"""The block operators on the GPU where ranges, host threads and streams meet their limits."""
import math
import threading

import numpy as np
import pytest

import ops_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def ops(cuda_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixture_experts_gemm_gb300 import ops
    return ops


def gen(seed):
    return torch.Generator().manual_seed(seed)


def test_quantize_of_a_copy_on_another_stream(ops):
    """A slice that cannot be viewed as rows, on a stream that does not wait for the current one."""
    w = torch.randn(3, 40, 64, generator=gen(1)).cuda()
    for x in (w[:, :33], w.transpose(1, 2)[:, :48, :32]):
        want = ops.int8_quantize(x.contiguous())
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        torch.cuda._sleep(10_000_000)  # what the call left to the current stream would come late
        got = ops.int8_quantize(x, stream=side)
        side.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# Logits whose scores leave fp32's range one by one or all together.
FAR = {
    "apart": lambda g, T, E: -60 - 80 * torch.rand(T, E, generator=g),          # scores of 1e-26 to 1e-61
    "close": lambda g, T, E: -90 - 0.5 * torch.rand(T, E, generator=g),
    "lowest": lambda g, T, E: -200 - 3 * torch.rand(T, E, generator=g),
    "one near": lambda g, T, E: torch.where(torch.arange(E) % 5 == 0, -20.0, -100 - torch.rand(T, E, generator=g)),
    "one above": lambda g, T, E: torch.where(torch.arange(E) % 5 == 0, 1.0, -88 - torch.rand(T, E, generator=g)),
}


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("far", list(FAR))
def test_renormalised_gates_of_scores_below_fp32(ops, score, far):
    """The chosen scores' ratios, whatever their size.  A gate is expf(l - largest) over a sum of such terms:
    the difference of at most 100 is rounded by 100 * 2^-24, expf is good to 2 ulp, five additions, two
    quotients and a product to 2^-24 each: less than 1e-5 in all; what is below 1e-37 may be lost."""
    T, E, k = 40, 20, 4
    l = FAR[far](gen(21), T, E)
    bias = 0.01 * torch.randperm(E, generator=gen(22)).float()
    if score == "softmax":
        l[:, 3] = 0.0       # the row's largest logit, which the bias keeps out
        bias[3] = -5.0
    r = ops.route(l.cuda(), k, score=score, bias=bias.cuda(), renormalize=True, scale=2.5)
    want = ref.route(l.numpy(), k, score, bias.numpy(), 1, 1, 1, True, 2.5)
    assert np.array_equal(r.idx.cpu().numpy(), want["idx"])
    got = r.gate.double().cpu().numpy()
    off = np.abs(got - want["gate"]) - (1e-5 * np.abs(want["gate"]) + 1e-37)
    assert (off <= 0).all(), (got.flat[off.argmax()], want["gate"].flat[off.argmax()])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("far", list(FAR))
def test_gradient_of_renormalised_gates_of_scores_below_fp32(ops, score, far):
    """scale q_i (g_i - sum q g) (1 - s_i) with q as above: 1e-5 for each of q and the sum."""
    T, E, k = 40, 20, 4
    l = FAR[far](gen(23), T, E)
    idx = torch.rand(T, E, generator=gen(24)).topk(k).indices
    dg = torch.randn(T, k, generator=gen(25))
    got = ops.route_backward(l.cuda(), idx.int().cuda(), dg.cuda(), score=score, renormalize=True, scale=2.5)
    l64 = l.double().requires_grad_(True)
    (ref.gates(l64, idx, score, True, 2.5) * dg.double()).sum().backward()
    off = (got.double().cpu() - l64.grad).abs() - 2e-5 * 2.5 * dg.double().abs().amax(1, keepdim=True)
    assert float(off.max()) <= 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gates_of_logits_masked_by_the_lowest_value(ops, score, dtype):
    """Experts masked by the type's lowest logit, chosen because a bias keeps the others out: their scores are zero, so
    their gates and gradients are, as 0 / 0 of the definition.  A row of nothing but the lowest value masks
    nobody under a softmax."""
    T, E, k = 6, 8, 3
    l = torch.full((T, E), torch.finfo(dtype).min, dtype=dtype)
    l[:4, 0], l[1, 1] = 2.0, -1.0
    bias = torch.zeros(E)
    bias[:2] = -math.inf
    r = ops.route(l.cuda(), k, score=score, bias=bias.cuda())
    dg = torch.randn(T, k, generator=gen(31))
    d = ops.route_backward(l.cuda(), r.idx, dg.cuda(), score=score)
    assert r.idx.tolist() == [[2, 3, 4]] * T
    assert (r.gate[:4] == 0).all() and (d[:4] == 0).all()
    if score == "sigmoid":
        assert (r.gate == 0).all() and (d == 0).all()
    else:
        assert ((r.gate[4:] - 1 / 3).abs() < 1e-6).all()
        want = torch.zeros(2, E, dtype=torch.float64)
        want[:, 2:5] = (dg[4:].double() - dg[4:].double().mean(1, keepdim=True)) / 3
        assert ((d[4:].double().cpu() - want).abs() <= 1e-6 + ref.half_step(dtype) * want.abs()).all()


def test_threads_at_different_widths(ops):
    """Host threads, a stream each, that launch the same kernels with different amounts of shared memory: every
    call is accepted and gives what it gives alone.  The C calls, as fast as they go."""
    import ctypes
    import mixture_experts_gemm_gb300 as moe
    shapes = [(4096, True), (4096, False), (2104, True), (2104, False)]
    f, w = moe.lib().colibri_moe_block_norm, torch.ones(4096, device="cuda")
    data = {d: [torch.randn(2, d, generator=gen(d + i)).cuda() for i in (0, 1)] for d, _ in shapes}

    def caller(d, block, stream):
        x, y = data[d]
        x1, p = torch.empty_like(x), torch.empty_like(x)
        c = moe.NormConfig(d, 0, 0, 0, int(block), 1, 0, 1.0, 1.0, 1e-6, 1)
        v = moe.NormVectors(w.data_ptr() if block else None, None, w.data_ptr(), None, None)
        args = (ctypes.addressof(c), ctypes.addressof(v), x.data_ptr(), d, y.data_ptr() if block else None, d, 2,
                x1.data_ptr() if block else None, p.data_ptr(), stream.cuda_stream)
        return (lambda: f(*args)), p, (c, v, x1)

    alone = {}
    for s in shapes:
        call, p, _ = caller(*s, torch.cuda.current_stream())
        assert call() == 0
        alone[s] = p
    torch.cuda.synchronize()
    failed = []

    def work(mine):
        stream = torch.cuda.Stream()
        many = [caller(*s, stream) for s in mine]
        codes = [call() for _ in range(4000) for call, _, _ in many]
        stream.synchronize()
        if any(codes):
            failed.append(f"{sum(map(bool, codes))} of {len(codes)} calls: {min(codes)}")
        failed.extend(s for s, (_, p, _) in zip(mine, many) if not torch.equal(p, alone[s]))

    torch.cuda.current_stream().synchronize()
    threads = [threading.Thread(target=work, args=(m,)) for m in (shapes[:1], shapes[1:2], shapes[2:3], shapes[3:])]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


def test_as_many_rows_as_a_call_takes(ops):
    """Rows of one value, 2^31 - 2^24 - 1 of them: the first and the last come out as alone."""
    T = 2**31 - 2**24 - 1
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    ends = [slice(0, 500), slice(T - 500, T)]
    w = torch.full((1,), 0.75, dtype=BF16, device="cuda")
    x = torch.empty(T, 1, dtype=BF16, device="cuda").uniform_(0.5, 2.0)
    norm = dict(before="rms", before_weight=w, eps=1.0)
    p = ops.pre_norm(x, w, eps=1.0)
    d = ops.block_norm_backward(None, p, x, **norm)["d_x"]
    for at in ends:
        assert torch.equal(p[at], ops.pre_norm(x[at], w, eps=1.0))
        assert torch.equal(d[at], ops.block_norm_backward(None, p[at], x[at], **norm)["d_x"])
    del p, d
    row = torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda")[:, None]
    out = ops.combine(x, row, torch.ones(T, 1, device="cuda"))
    assert torch.equal(out, x.flip(0))
    del x, row, out
    torch.cuda.empty_cache()


def test_gated_products_in_fp32(ops):
    """silu(v) * u in fp32, with v and u exact (powers of two as scales): expf to 2 ulp, one addition, one
    quotient and one product to half an ulp each, 7 * 2^-24 in all."""
    K, N = 16, 254
    whole = torch.cat([torch.arange(-127, 0), torch.arange(1, 128)])
    w = torch.zeros(1, N, K, dtype=torch.int8)
    w[0, :, 0] = whole.to(torch.int8)
    w3 = torch.zeros_like(w)
    w3[0, :, 0] = whole.flip(0).to(torch.int8)
    x = torch.zeros(6, K)
    x[:, 0] = 127.0 * 2.0 ** torch.arange(-4, 2)
    ws, off = torch.full((1, N), 2.0**-7), torch.tensor([0, 6]).int()
    y = ops.int8_experts(x.cuda(), w.cuda(), ws.cuda(), off.cuda(), w3=w3.cuda(), w3_scale=ws.cuda(), out_dtype=F32)
    scale = x[:, :1].double()  # a row's scale times its one quantised value, 127
    v, u = scale * whole.double() / 128, scale * whole.flip(0).double() / 128
    want = v / (1 + torch.exp(-v)) * u
    off = (y.double().cpu() - want).abs() - (8 * 2.0**-24 * want.abs() + 1e-37 * u.abs())
    i = int(off.argmax())
    assert float(off.max()) <= 0, (float(v.flatten()[i]), float(y.flatten()[i]), float(want.flatten()[i]))

# Rows of every expert, one case for each width of the product's tiles, with and without the second projection.
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("counts", [[1, 0, 1], [40, 30, 36], [128, 1, 97], [300, 257, 255]], ids=str)
def test_a_wait_that_runs_out(ops, counts, gated):
    """A product told to wait for a microsecond at most (to within about 20) finishes, or stops and says so; the next
    call, in the same workspace, gives what a call without the limit gives."""
    import ctypes
    import mixture_experts_gemm_gb300 as moe
    K, N, E, R = 4096, 520, len(counts), sum(counts)
    x = torch.randn(R, K, generator=gen(R)).cuda().to(BF16)
    w = [torch.randint(-127, 128, (E, N, K), generator=gen(R + i)).to(torch.int8).cuda() for i in (1, 2)]
    ws = torch.full((E, N), 1e-3, device="cuda")
    off = torch.tensor([0] + counts, device="cuda").cumsum(0).int()
    kw = dict(w3=w[1], w3_scale=ws) if gated else {}
    want = ops.int8_experts(x, w[0], ws, off, **kw)
    L, at = moe.lib(), ctypes.byref

    def config(us):
        return moe.Int8Config(K, N, E, moe.DTYPE_BF16, moe.DTYPE_BF16, 0, us)

    size = ctypes.c_size_t()
    assert L.colibri_moe_int8_experts_workspace(at(config(0)), R, R, at(size)) == 0
    space = torch.empty(size.value, dtype=torch.uint8, device="cuda")
    w3, s3 = (w[1].data_ptr(), ws.data_ptr()) if gated else (None, None)

    def call(us):
        y = torch.empty(R, N, dtype=BF16, device="cuda")
        s = torch.cuda.current_stream().cuda_stream
        assert L.colibri_moe_int8_experts(at(config(us)), x.data_ptr(), K, R, None, R, off.data_ptr(), w[0].data_ptr(),
                                          ws.data_ptr(), w3, s3, y.data_ptr(), space.data_ptr(), size.value, s) == 0
        torch.cuda.synchronize()
        return y

    for _ in range(2):
        y = call(1)
        assert ops.int8_status() == 1 or torch.equal(y, want)
        assert torch.equal(call(0), want) and ops.int8_status() == 0
    assert torch.equal(call(10_000_000), want)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("R", [10, 40, 100, 600])  # one for each width of the product's tiles
def test_a_wait_that_runs_out_is_reported(ops, R, gated):
    """The status word: clear after calls that finish, set once by one that gave up, from any stream or graph.  A part
    of K is 128 steps of 64 here, at least 20 us of products that the epilogue waits for, two tries and more."""
    K, N = 65536, 256
    x = torch.randn(R, K, generator=gen(3)).cuda()
    w = torch.randint(-127, 128, (1, N, K), generator=gen(4), dtype=torch.int8).cuda()
    ws, off = torch.ones(1, N, device="cuda"), torch.tensor([0, R], device="cuda").int()
    assert ops.int8_status() in (0, 1)
    kw = dict(w3=w, w3_scale=ws) if gated else {}
    want = ops.int8_experts(x, w, ws, off, **kw)
    assert ops.int8_status() == 0

    def short(stream=None):
        """The call with a limit of a microsecond."""
        real = ops._int8_config
        config = ops.Int8Config(K, N, 1, 0, 0, 1, 1)
        ops._int8_config = lambda *a: (config, ops.ctypes.addressof(config))
        try:
            return ops.int8_experts(x, w, ws, off, stream=stream, **kw)
        finally:
            ops._int8_config = real

    for stream in (None, torch.cuda.Stream()):
        short(stream)
        y = ops.int8_experts(x, w, ws, off, stream=stream, **kw)
        assert ops.int8_status() == 1 and ops.int8_status(0) == 0
        assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        short()
    assert ops.int8_status() == 0
    graph.replay()
    assert ops.int8_status("cuda:0") == 1 and ops.int8_status() == 0
