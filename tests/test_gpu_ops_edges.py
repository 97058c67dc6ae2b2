"""The block operators on the GPU where ranges, host threads and streams meet their limits."""
import pytest

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
