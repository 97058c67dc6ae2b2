"""Experts in e4m3 without a GPU: what the calls refuse, and the host side of their Python layer."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from test_ops_host_cpu import Library, cuda, host  # noqa: E402,F401

P = 4096  # an address that is never read
MOST = 2**31 - 1 - 2**24


@pytest.fixture(scope="module")
def moe(cuda_lib):
    import mixture_experts_gemm_gb300 as m
    return m


def config(m, kw):
    c = dict(in_features=64, out_features=32, num_experts=4, dtype=1, out_dtype=0, trusted_pointers=1, wait_limit_us=0)
    mine = {k: kw.pop(k) for k in list(kw) if k in c}
    return m.Fp8Config(**{**c, **mine})


CONFIGS = [
    (dict(in_features=0), -1), (dict(in_features=72), -6), (dict(in_features=65552), -6), (dict(out_features=0), -1),
    (dict(out_features=131073), -6), (dict(num_experts=0), -1), (dict(num_experts=513), -6), (dict(dtype=2), -1),
    (dict(out_dtype=2), -1), (dict(trusted_pointers=2), -1), (dict(wait_limit_us=-1), -1), (dict(wait_limit_us=10_000_001), -1),
]


def quantize(m, **kw):
    c = config(m, kw)
    a = {**dict(x=P, ldx=64, n=8, square=0, q=P, scale=P), **kw}
    return m.lib().colibri_moe_fp8_quantize(ctypes.byref(c), *a.values(), None)


def forward(m, **kw):
    c = config(m, kw)
    a = {**dict(x=P, ldx=64, n=8, rows=P, R=8, off=P, w=P, ws=P, w3=None, w3s=None, y=P, space=P, size=1 << 40), **kw}
    return m.lib().colibri_moe_fp8_experts(ctypes.byref(c), *a.values(), None)


def backward(m, **kw):
    c = config(m, kw)
    a = {**dict(d_y=P, ld=32, x=P, ldx=64, n=8, rows=P, R=8, off=P, w=P, ws=P, d_rows=P, d_w=P, space=P, size=1 << 40), **kw}
    return m.lib().colibri_moe_fp8_experts_backward(ctypes.byref(c), *a.values(), None)


@pytest.mark.parametrize("kw,code", CONFIGS + [
    (dict(n=-1), -1), (dict(n=MOST + 1), -6), (dict(x=None), -1), (dict(q=None), -1), (dict(scale=None), -1),
    (dict(ldx=63), -1), (dict(square=2), -1), (dict(square=1, n=6), -1), (dict(q=P + 8), -1), (dict(n=0, x=None, q=None), 0),
])
def test_quantize_refuses(moe, kw, code):
    assert quantize(moe, **dict(kw)) == code


@pytest.mark.parametrize("kw,code", CONFIGS + [
    (dict(n=-1), -1), (dict(R=-1), -1), (dict(R=MOST + 1), -6), (dict(rows=None, R=9), -1), (dict(x=None), -1),
    (dict(ldx=63), -1), (dict(off=None), -1), (dict(w=None), -1), (dict(ws=None), -1), (dict(y=None), -1), (dict(w3=P), -1),
    (dict(w3s=P), -1), (dict(w=P + 8), -1), (dict(w3=P + 8, w3s=P), -1), (dict(space=None), -1), (dict(space=P + 4), -1),
    (dict(size=16), -1), (dict(R=0, x=None, off=None, w=None, y=None, space=None), 0),
])
def test_forward_refuses(moe, kw, code):
    assert forward(moe, **dict(kw)) == code


@pytest.mark.parametrize("kw,code", CONFIGS + [
    (dict(n=-1), -1), (dict(R=-1), -1), (dict(R=MOST + 1), -6), (dict(rows=None, R=9), -1), (dict(d_y=None), -1),
    (dict(ld=31), -1), (dict(x=None), -1), (dict(ldx=63), -1), (dict(off=None), -1), (dict(w=None), -1), (dict(ws=None), -1),
    (dict(d_rows=None), -1), (dict(d_rows=None, d_w=None, w=None, ws=None), -1), (dict(w=P + 8), -1), (dict(d_w=P + 8), -1),
    (dict(space=None), -1), (dict(space=P + 4), -1), (dict(size=16), -1),
])
def test_backward_refuses(moe, kw, code):
    assert backward(moe, **dict(kw)) == code


def test_valid_calls_without_a_gpu_report_cuda_errors(moe):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert quantize(moe) == quantize(moe, square=1) == forward(moe) == backward(moe) == -4
    assert backward(moe, rows=None, x=None, d_w=None) == backward(moe, d_rows=None, w=None, ws=None) == -4
    assert forward(moe, R=MOST, size=1 << 62) == -4
    assert moe.lib().colibri_moe_fp8_status(ctypes.byref(ctypes.c_int32())) == -4


def test_workspaces(moe):
    L, n = moe.lib(), ctypes.c_size_t()
    for f in (L.colibri_moe_fp8_experts_workspace, L.colibri_moe_fp8_experts_backward_workspace):
        assert f(None, 4, 4, ctypes.byref(n)) == -1
        assert f(ctypes.byref(config(moe, {})), 4, 4, None) == -1
        assert f(ctypes.byref(config(moe, {})), 4, -1, ctypes.byref(n)) == -1
        assert f(ctypes.byref(config(moe, {})), 4, MOST + 1, ctypes.byref(n)) == -6
    assert L.colibri_moe_fp8_status(None) == -1


# ---- the Python layer
E4M3 = torch.float8_e4m3fn


def layer(E=2, N=200, K=160):
    return cuda(torch.zeros(E, N, K, dtype=E4M3)), cuda(torch.ones(E, -(-N // 128), -(-K // 128)))


def test_python_layer_checks(host):  # noqa: F811
    ops, _, _ = host
    w, s = layer()
    x, off, d_y = cuda(torch.ones(4, 160)), cuda(torch.zeros(3, dtype=torch.int32)), cuda(torch.ones(4, 200))
    bad = [
        lambda: ops.fp8_experts(x, w.view(torch.uint8), s, off), lambda: ops.fp8_experts(x, w, s[:, :1], off),
        lambda: ops.fp8_experts(x, w, None, off), lambda: ops.fp8_experts(x, w[0], s[0], off),
        lambda: ops.fp8_experts(x[:, :144], w, s, off), lambda: ops.fp8_experts(x, w, s, off[:2]),
        lambda: ops.fp8_experts(x, w, s, off, w3=w), lambda: ops.fp8_experts(x, w, s, off, w3=w, w3_scale=s[:1]),
        lambda: ops.fp8_experts(x, w, s, off.long()), lambda: ops.fp8_experts(x.double(), w, s, off),
        lambda: ops.fp8_experts(x, w, s, off, out_dtype=torch.float16), lambda: ops.fp8_experts(torch.ones(4, 160), w, s, off),
        lambda: ops.fp8_experts(x, w.transpose(1, 2), s, off),
        lambda: ops.fp8_experts_backward(d_y, None, None, None, off), lambda: ops.fp8_experts_backward(d_y, x, None, s, off),
        lambda: ops.fp8_experts_backward(d_y, x, w, None, off), lambda: ops.fp8_experts_backward(d_y[:, 1:], x, w, s, off),
        lambda: ops.fp8_experts_backward(d_y, x[:, :144], w, s, off), lambda: ops.fp8_experts_backward(d_y, x, w, s, off[:0]),
        lambda: ops.fp8_experts_backward(d_y, x.bfloat16(), w, s, off),
        lambda: ops.fp8_experts_backward(d_y, x, w, s, off, weight_dtype=torch.float64),
        lambda: ops.fp8_quantize(cuda(torch.ones(16)), square=True), lambda: ops.fp8_quantize(torch.ones(2, 16)),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()


def test_shapes_and_arguments(host):  # noqa: F811
    ops, library, _ = host
    seen = []
    for name in ("quantize", "experts", "experts_backward"):
        library.see["colibri_moe_fp8_" + name] = lambda c, *a: seen.append((ops.Fp8Config.from_address(c), a))
    x = cuda(torch.ones(3, 5, 160))
    q, s = ops.fp8_quantize(x)
    assert q.shape == (3, 5, 160) and q.dtype == E4M3 and s.shape == (3, 5, 2) and seen[-1][1][2:4] == (15, 0)
    q, s = ops.fp8_quantize(x, square=True)
    assert s.shape == (3, 1, 2) and seen[-1][0].num_experts == 3 and seen[-1][1][2:4] == (15, 1)
    w, s = layer()
    rows, off = cuda(torch.zeros(7, dtype=torch.int32)), cuda(torch.zeros(3, dtype=torch.int32))
    y = ops.fp8_experts(x[0].bfloat16().as_subclass(type(x)), w, s, off, rows=rows, out_dtype=torch.float32)
    c, a = seen[-1]
    assert y.shape == (7, 200) and y.dtype == torch.float32 and a[2] == 5 and a[4] == 7
    assert (c.in_features, c.out_features, c.num_experts, c.dtype, c.out_dtype, c.trusted_pointers) == (160, 200, 2, 1, 0, 1)
    d_y = cuda(torch.ones(7, 200))
    d_rows, d_w = ops.fp8_experts_backward(d_y, x[0], w, s, off, rows=rows, weight_dtype=torch.bfloat16)
    assert d_rows.shape == (7, 160) and d_w.shape == (2, 200, 160) and d_w.dtype == torch.bfloat16
    assert seen[-1][1][4:7:2] == (5, 7)
    d_rows, none = ops.fp8_experts_backward(d_y, None, w, s, off)
    assert none is None and seen[-1][1][11] is None and seen[-1][1][2] is None
    none, d_w = ops.fp8_experts_backward(d_y, x[0], None, None, off, rows=rows)
    assert none is None and seen[-1][1][8:11] == (None, None, None)
    count = len(seen)
    none, d_w = ops.fp8_experts_backward(d_y[:0], x[0], None, None, off, rows=rows[:0])
    assert len(seen) == count + 1 and d_w.shape == (2, 200, 160)  # zeros are written for no rows, too
    ops.fp8_experts_backward(d_y[:0], None, w, s, off)
    assert len(seen) == count + 1


def test_a_lost_gradient_is_said(host):  # noqa: F811
    ops, _, _ = host
    w, s = layer()
    off, leaf = cuda(torch.zeros(3, dtype=torch.int32)), cuda(torch.ones(4, 160)).requires_grad_(True)
    i = cuda(torch.zeros(4, dtype=torch.int32))
    for f in (lambda: ops.fp8_experts(leaf, w, s, off), lambda: ops.fp8_quantize(leaf), lambda: ops.dispatch(leaf, i),
              lambda: ops.gated(leaf, leaf)):
        with pytest.warns(UserWarning, match="autograd"):
            f()
        with torch.no_grad():
            f()


@pytest.mark.parametrize("name", ["quantize", "experts", "experts_backward"])
def test_configs_outlive_their_call(host, monkeypatch, name):  # noqa: F811
    """Other threads may bring any number of configs while a call is in the allocator."""
    import gc
    import weakref
    ops, library, _ = host
    alive, looked = {}, []

    class Config(ops.Fp8Config):
        def __init__(self, *args):
            super().__init__(*args)
            alive.setdefault(ctypes.addressof(self), weakref.ref(self))  # the first one there: the call's

    w, s = layer()
    x, d_y, off = cuda(torch.ones(4, 160)), cuda(torch.ones(4, 200)), cuda(torch.zeros(3, dtype=torch.int32))
    call = dict(quantize=lambda: ops.fp8_quantize(x), experts=lambda: ops.fp8_experts(x, w, s, off),
                experts_backward=lambda: ops.fp8_experts_backward(d_y, x, w, s, off))[name]
    monkeypatch.setattr(ops, "Fp8Config", Config)
    ops._fp8_config.cache_clear()
    real = torch.empty

    def empty(*args, **kw):
        for i in range(300):
            ops._fp8_config(16 * i + 16, 8, 1, torch.float32, torch.float32)
        gc.collect()
        return real(*args, **kw)

    for which in (name, name + "_workspace"):
        library.see["colibri_moe_fp8_" + which] = lambda c, *a: looked.append(alive[c]() is not None)
    monkeypatch.setattr(torch, "empty", empty)
    call()
    ops._fp8_config.cache_clear()
    assert looked and all(looked)
