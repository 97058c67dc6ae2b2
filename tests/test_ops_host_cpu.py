"""The host side of ops.py without a GPU: CPU tensors that say they are on CUDA device 0, and a library that
looks at the arguments it is given instead of launching anything."""
import pytest

torch = pytest.importorskip("torch")


class OnCuda(torch.Tensor):
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0


def cuda(t):
    return t.as_subclass(OnCuda)


class Library:
    """Answers every call with success; `see[name]` is called with the call's arguments."""

    def __init__(self):
        self.see = {}

    def __getattr__(self, name):
        return lambda *args: self.see.get(name, lambda *a: None)(*args) or 0


@pytest.fixture
def host(monkeypatch):
    """(ops, the library, state): state["inside"] is true while a call is under its stream."""
    from mixture_experts_gemm_gb300 import ops
    library, state = Library(), dict(inside=False)

    def run(f, t, dev, stream):
        state["inside"] = True
        try:
            return f(0)
        finally:
            state["inside"] = False

    monkeypatch.setattr(ops, "lib", lambda: library)
    monkeypatch.setattr(ops, "_run", run)
    return ops, library, state


def test_quantize_copies_on_its_stream(host):
    """Rows that cannot be viewed are copied: with the call's stream current, and kept until the call returns."""
    ops, library, state = host
    w = torch.arange(2.0 * 4 * 32).view(2, 32, 4)
    where = []

    class Watched(OnCuda):
        def reshape(self, *shape):
            where.append(state["inside"])
            return super().reshape(*shape)

    seen = []
    library.see["colibri_moe_int8_quantize"] = lambda c, px, ldx, n, *rest: seen.append((px, ldx, n))
    for x in (w.transpose(1, 2), w[:, :3, :], w[0]):
        x = x.as_subclass(Watched)
        del where[:], seen[:]
        q, scale = ops.int8_quantize(x)
        assert where == [True]
        assert q.shape == x.shape and scale.shape == x.shape[:-1]
        (px, ldx, n), = seen
        assert px % 4 == 0 and ldx >= x.shape[-1] and n == scale.numel()
    with pytest.raises(ValueError, match="contiguous"):
        ops.int8_quantize(w[0].t().as_subclass(Watched))
