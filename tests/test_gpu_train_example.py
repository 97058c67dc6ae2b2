"""The example training step (dispatch, experts in e4m3, gated activation, combine, and back) against fp32."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_train.py")


@pytest.fixture(scope="module")
def example(cuda_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("moe_train", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m, m.Layer(d=256, f=384, experts=8, top_k=2, seed=3)


# An e4m3 value is off by at most 2^-4 of itself, in the mean of a binade by 2^-4 / sqrt(3) of its lower end, 2.6 % of a
# value's root mean square; a product of two such operands with mixed signs by 3.7 % of its own.  Along the chain errors
# of independent steps add as squares: u and v 3.7 %, h 3.7 sqrt(2) times at most 1.4 (silu's slope against its value) and
# its own 2.6 %: 8 %, y and out 9 %; d_h 4.5 %, d_u and d_v 4.5 % with those of u and v: 8 %, the gradients of the first
# weights and of the rows 9 to 10 %, that of w2 9 %, of the gates (with y) and the router 9 %.  bf16 roundings are far
# below.  0.2 is twice the largest.
@pytest.mark.parametrize("T", [1, 37, 900])
def test_step_is_near_fp32(example, T):
    m, layer = example
    g = torch.Generator().manual_seed(T)
    x, d_out = (torch.randn(T, 256, generator=g).cuda().bfloat16() for _ in range(2))
    for n, e in m.errors_of(layer, x, d_out).items():
        assert e < 0.2, (n, e)
    assert m.ops.fp8_status() == 0


def test_a_replayed_choice_with_dropped_slots(example):
    """Slots of -1, tokens with none left, experts without rows: as fp32 for the same choice."""
    m, layer = example
    g = torch.Generator().manual_seed(5)
    x, d_out = (torch.randn(300, 256, generator=g).cuda().bfloat16() for _ in range(2))
    idx = torch.rand(300, 5, generator=g).topk(2).indices.int()  # experts 5, 6 and 7 have no rows
    idx[torch.rand(300, 2, generator=g) < 0.2] = -1
    idx[7] = -1
    for n, e in m.errors_of(layer, x, d_out, idx.cuda()).items():
        assert e < 0.2, (n, e)
    out, saved = layer.forward(x, idx.cuda())
    grads = layer.backward(d_out, saved)
    assert out[7].eq(0).all() and all(grads[n][5:].eq(0).all() for n in ("w1", "w3", "w2"))


def test_the_router_s_choice_replayed(example):
    """The same bits through dispatch_order as through route."""
    m, layer = example
    x = torch.randn(200, 256, generator=torch.Generator().manual_seed(6)).cuda().bfloat16()
    out, saved = layer.forward(x)
    again, replayed = layer.forward(x, saved[3])
    for a, b in zip(saved[5][2:], replayed[5]):
        assert torch.equal(a, b)
    assert torch.equal(saved[9], replayed[9])  # the experts' results
