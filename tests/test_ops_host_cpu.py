"""The host side of ops.py without a GPU: CPU tensors that say they are on CUDA device 0, and a library that
looks at the arguments it is given instead of launching anything."""
import gc
import weakref

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


def calls(ops):
    """One call of each kind, over small tensors."""
    x, y, w = cuda(torch.ones(4, 32)), cuda(torch.ones(4, 32)), cuda(torch.ones(32))
    idx, i32 = cuda(torch.zeros(4, 2, dtype=torch.int32)), torch.int32
    w8, ws = cuda(torch.ones(2, 8, 32, dtype=torch.int8)), cuda(torch.ones(2, 8))
    norms = dict(after="rms", after_weight=w, before="rms", before_weight=w)
    return dict(
        block_norm=lambda: ops.block_norm(x, y, **norms),
        block_norm_backward=lambda: ops.block_norm_backward(x, x, x, y, **norms),
        route=lambda: ops.route(x, 2),
        route_experts_backward=lambda: ops.route_backward(x, idx, cuda(torch.ones(4, 2))),
        int8_quantize=lambda: ops.int8_quantize(x),
        int8_experts=lambda: ops.int8_experts(x, w8, ws, cuda(torch.zeros(3, dtype=i32))))


@pytest.mark.parametrize("name", ["block_norm", "block_norm_backward", "route", "route_experts_backward",
                                  "int8_quantize", "int8_experts"])
def test_configs_outlive_their_call(host, monkeypatch, name):
    """Other threads may bring any number of other configs while a call is in the allocator: what the call gives
    the library stays in memory until the library returns."""
    ops, library, _ = host
    alive = {}

    def watched(kind):
        class Config(kind):
            def __init__(self, *args):
                super().__init__(*args)
                alive.setdefault(ops.ctypes.addressof(self), weakref.ref(self))  # the first one there: the call's
        return Config

    for kind in ("NormConfig", "RouteConfig", "Int8Config"):
        monkeypatch.setattr(ops, kind, watched(getattr(ops, kind)))
    caches = [ops._norm_config, ops._route_config, ops._int8_config]
    for c in caches:
        c.cache_clear()
    real, looked = torch.empty, []

    def empty(*args, **kw):
        for i in range(300):
            ops._norm_config(i + 100, torch.float32, torch.float32, torch.float32, "rms", "rms", 0, 1.0, 1.0, 1e-6)
            ops._route_config(i + 100, 2, "softmax", 1, 1, 1, True, torch.float32, 1.0)
            ops._int8_config(i + 100, 8, 1, torch.float32, torch.float32)
        gc.collect()
        return real(*args, **kw)

    def see(c, *args):
        looked.append(alive[c]() is not None)

    whole = {"route": "route_experts"}.get(name, name)
    library.see["colibri_moe_" + whole] = library.see[f"colibri_moe_{whole}_workspace"] = see
    monkeypatch.setattr(torch, "empty", empty)
    calls(ops)[name]()
    for c in caches:
        c.cache_clear()
    assert looked and all(looked)


def test_scalars_are_read_at_every_call(host):
    """A scalar held in a tensor (a schedule's, a counter's) and changed in place between two calls."""
    ops, library, _ = host
    seen = []
    library.see["colibri_moe_block_norm"] = lambda c, *a: seen.append(
        [getattr(ops.NormConfig.from_address(c), n) for n in ("residual_scale", "block_scale", "eps", "rows_per_gate")])
    library.see["colibri_moe_route_experts"] = lambda c, *a: seen.append(
        [getattr(ops.RouteConfig.from_address(c), n) for n in ("top_k", "groups", "top_groups", "group_top", "scale")])
    x, y, w, logits = cuda(torch.ones(4, 32)), cuda(torch.ones(4, 32)), cuda(torch.ones(2, 32)), cuda(torch.ones(4, 16))
    scalars, counts = [torch.tensor(0.5) for _ in range(4)], [torch.tensor(v) for v in (2, 4, 2, 1)]
    for step in (1, 2):
        for v in scalars:
            v.fill_(0.5 * step)
        ops.block_norm(x, y, gate=w, rows_per_gate=2, residual_scale=scalars[0], block_scale=scalars[1], eps=scalars[2])
        assert seen.pop() == [0.5 * step] * 3 + [2]
        counts[0].fill_(2 * step), counts[3].fill_(step)
        r = ops.route(logits, counts[0], groups=counts[1], top_groups=counts[2], group_top=counts[3], scale=scalars[3])
        assert seen.pop() == [2 * step, 4, 2, step, 0.5 * step] and r.idx.shape == (4, 2 * step)
    with pytest.raises(TypeError):
        ops.route(logits, 2.0)


@pytest.mark.parametrize("backward", [False, True])
def test_calls_inside_a_call(host, monkeypatch, backward):
    """A call that runs while another one of the same thread is in the allocator (a finaliser, a mode's hook) leaves
    the outer call's vectors alone."""
    ops, library, _ = host
    x, y = cuda(torch.ones(4, 32)), cuda(torch.ones(4, 32))
    vectors = [cuda(torch.ones(32)) for _ in range(4)]
    seen, nested = [], []

    def look(address):
        return list(ops.ctypes.cast(address, ops.ctypes.POINTER(ops.ctypes.c_void_p))[:5])

    def one(a, b):
        norms = dict(after="rms", after_weight=a, before="rms", before_weight=b)
        return ops.block_norm_backward(x, x, x, y, **norms) if backward else ops.block_norm(x, y, **norms)

    def see(*args):
        seen.append([look(args[1])] + ([look(args[13])] if backward else []))

    library.see["colibri_moe_block_norm_backward" if backward else "colibri_moe_block_norm"] = see
    real = torch.empty

    def empty(*args, **kw):
        t = real(*args, **kw)
        if not nested:
            nested.append(None)
            nested[0] = one(*vectors[2:])
        return t

    monkeypatch.setattr(torch, "empty", empty)
    out = one(*vectors[:2])
    inner, outer = seen
    for s, v, o in ((inner, vectors[2:], nested[0]), (outer, vectors[:2], out)):
        assert s[0] == [v[0].data_ptr(), None, v[1].data_ptr(), None, None]
        if backward:
            assert s[1] == [o["d_wa"].data_ptr(), None, o["d_wb"].data_ptr(), None, None]


@pytest.mark.parametrize("T", [0, 4])
def test_gate_gradient_has_the_gate_s_shape(host, T):
    ops, library, _ = host
    x, d = cuda(torch.ones(T, 32)), 32
    for shape, per_gate in (((d,), None), ((1, d), None), ((2, d), 2)):
        out = ops.block_norm_backward(x, None, x, x, gate=cuda(torch.ones(shape)), rows_per_gate=per_gate)
        assert out["d_g"].shape == shape


@pytest.mark.parametrize("name", ["block_norm", "route", "int8_quantize", "int8_experts", "combine"])
def test_a_lost_gradient_is_said(host, name):
    """Results are not attached to autograd: a call on tensors that ask for a gradient says so, unless gradients are
    off; it still runs."""
    import warnings
    ops, _, _ = host
    x, y = cuda(torch.ones(4, 32)), cuda(torch.ones(4, 32))
    w8 = cuda(torch.ones(2, 8, 32, dtype=torch.int8))

    def call(x, y):
        if name == "block_norm":
            return ops.block_norm(x, y)
        if name == "route":
            return ops.route(x, 2)
        if name == "int8_quantize":
            return ops.int8_quantize(x)
        if name == "int8_experts":
            return ops.int8_experts(x, w8, cuda(torch.ones(2, 8)), cuda(torch.zeros(3, dtype=torch.int32)))
        return ops.combine(x, cuda(torch.zeros(2, 2, dtype=torch.int32)), cuda(torch.ones(2, 2)))

    leaf = cuda(torch.ones(4, 32)).requires_grad_(True)
    with pytest.warns(UserWarning, match="autograd"):
        call(leaf, y)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        call(x, y)
        with torch.no_grad():
            call(leaf, y)
        call(leaf.detach(), y)
    if name == "block_norm":
        with pytest.warns(UserWarning, match="autograd"):
            call(x, leaf)
        with pytest.warns(UserWarning, match="autograd"):
            ops.pre_norm(x, cuda(torch.ones(32)).requires_grad_(True))
