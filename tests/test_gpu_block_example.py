"""The example block (norms, routing to many experts, 8-bit experts) against its unquantised fp32 form."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")


@pytest.fixture(scope="module")
def block(cuda_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("moe_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m, m.Block(d=256, f=128, experts=16, top_k=4, groups=4, top_groups=2, seed=3)


@pytest.mark.parametrize("T", [1, 33, 500])
def test_block_is_near_its_unquantised_form(block, T):
    """An 8-bit value is off by at most half a step of max / 127: about 1 % of a normal row's deviation (max
    near 3.5 sigma: 3.5 / 127 / sqrt(12)), once in the activations and once in the weights of each of two
    products in a row, so the block's result by about 2 % of its root mean square; half of it (block_scale)
    enters x1.  A largest error of five deviations is 0.1; a token whose routing is a close call may differ in
    an expert, so the median over tokens is held to that."""
    m, b = block
    x = torch.randn(T, b.d, generator=torch.Generator().manual_seed(T)).cuda().bfloat16()
    out, want = b.forward(x), b.reference(x)
    for got, ref in zip(out, want):
        err = (got.float() - ref).abs().amax(1) / ref.square().mean().sqrt()
        assert float(err.median()) < 0.1, float(err.median())


def test_gradients_run(block):
    m, b = block
    g = torch.Generator().manual_seed(0)
    T = 20
    x, y = torch.randn(T, b.d, generator=g).cuda().bfloat16(), torch.randn(T, b.d, generator=g).cuda()
    logits = torch.randn(T, 16, generator=g).cuda()
    r = m.ops.route(logits, b.top_k, bias=b.bias, **b.routing)
    norms, d_logits = b.gradients(x, y, logits, r.idx, x, x, torch.randn(T, b.top_k, generator=g).cuda())
    assert sorted(norms) == ["d_wa", "d_wb", "d_x", "d_y"] and torch.isfinite(d_logits).all()
    # renormalised gates sum to a constant: a gradient equal in every slot moves nothing
    same = m.ops.route_backward(logits, r.idx, torch.ones_like(r.gate), score="sigmoid")
    assert float(same.abs().max()) < 1e-6
