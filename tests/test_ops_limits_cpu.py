"""Row counts near 2^31, without a GPU: kernels step past the last row by less than 2^24, so the calls refuse what
would make their 32-bit row numbers wrap."""
import ctypes

import pytest

P = 4096  # an address that is never read
MOST = 2**31 - 1 - 2**24


def far(n):
    return (n + 1) << 44  # addresses whose spans do not meet


@pytest.fixture(scope="module")
def moe(cuda_lib):
    import mixture_experts_gemm_gb300 as m
    return m


def calls(m):
    """Every call that takes a number of rows, as a function of that number."""
    L = m.lib()
    norm = m.NormConfig(1, 1, 1, 1, 1, 1, 0, 1.0, 1.0, 1e-6)
    vec, none = m.NormVectors(P, None, P, None, None), m.NormVectors()
    route = m.RouteConfig(4, 1, 0, 1, 1, 1, 1, 1, 1.0)
    int8 = m.Int8Config(16, 1, 4, 1, 1)
    n, at = ctypes.c_size_t(), ctypes.byref
    big = 1 << 50
    return dict(
        block_norm=lambda T: L.colibri_moe_block_norm(at(norm), at(vec), far(0), 1, far(1), 1, T, far(2), far(3), None),
        block_norm_backward_workspace=lambda T: L.colibri_moe_block_norm_backward_workspace(at(norm), T, at(n)),
        block_norm_backward=lambda T: L.colibri_moe_block_norm_backward(
            at(norm), at(vec), far(0), 1, far(1), 1, far(2), 1, far(3), 1, T, far(4), far(5), at(none), P, big, None),
        route_experts_workspace=lambda T: L.colibri_moe_route_experts_workspace(at(route), T, at(n)),
        route_experts=lambda T: L.colibri_moe_route_experts(at(route), P, 4, None, T, P, P, P, P, P, P, P, big, None),
        route_experts_backward=lambda T: L.colibri_moe_route_experts_backward(at(route), P, 4, P, P, T, P, 4, None),
        int8_experts_workspace=lambda T: L.colibri_moe_int8_experts_workspace(at(int8), T, T, at(n)),
        int8_experts=lambda T: L.colibri_moe_int8_experts(at(int8), P, 16, 8, P, T, P, P, P, None, None, P, P, big, None),
        combine_rows=lambda T: L.colibri_moe_combine_rows(P, 1, 8, P, P, T, 1, 1, P, 1, None))


@pytest.mark.parametrize("name", ["block_norm", "block_norm_backward_workspace", "block_norm_backward",
                                  "route_experts_workspace", "route_experts", "route_experts_backward",
                                  "int8_experts_workspace", "int8_experts", "combine_rows"])
def test_rows_near_2_31_are_refused(moe, name):
    call = calls(moe)[name]
    for T in (MOST + 1, 2**31 - 1):
        assert call(T) == -6
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():  # accepted up to the limit: the next thing that is missing is a device
        assert call(MOST) in (0, -4)


def test_wait_limits(moe):
    for us, code in ((-1, -1), (10_000_001, -1), (10_000_000, 0), (1, 0), (0, 0)):
        c = moe.Int8Config(16, 1, 4, 1, 1, 0, us)
        assert moe.lib().colibri_moe_int8_quantize(ctypes.byref(c), None, 16, 0, None, None, None) == code


def test_status_without_a_device(moe):
    assert moe.lib().colibri_moe_int8_status(None) == -1
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        assert moe.lib().colibri_moe_int8_status(ctypes.byref(ctypes.c_int32())) == -4
