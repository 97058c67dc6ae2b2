"""What the block operators refuse, without a GPU: every check that needs no device answers first."""
import ctypes

import pytest

P = 4096  # an address that is never read: the checks below fail before any pointer is looked at


@pytest.fixture(scope="module")
def moe(cuda_lib):
    import mixture_experts_gemm_gb300 as m
    return m


def norm_call(m, cfg=(), w=None, x=P, ldx=64, y=1 << 30, ldy=64, T=4, x1=2 << 30, p=3 << 30):
    c = dict(d_model=64, dtype=1, block_dtype=0, param_dtype=0, after=1, before=1, rows_per_gate=0, residual_scale=1.0,
             block_scale=1.0, eps=1e-6)
    c.update(cfg)
    v = dict(after_weight=P, after_bias=None, before_weight=P, before_bias=None, gate=None)
    v.update(w or {})
    return m.lib().colibri_moe_block_norm(ctypes.byref(m.NormConfig(**c)), ctypes.byref(m.NormVectors(**v)), x, ldx, y, ldy,
                                          T, x1, p, None)


@pytest.mark.parametrize("kw,code", [
    (dict(cfg=dict(d_model=0)), -1), (dict(cfg=dict(d_model=16385)), -6), (dict(cfg=dict(dtype=2)), -1),
    (dict(cfg=dict(block_dtype=-1)), -1), (dict(cfg=dict(param_dtype=7)), -1), (dict(cfg=dict(after=3)), -1),
    (dict(cfg=dict(before=-1)), -1), (dict(cfg=dict(eps=-1.0)), -1), (dict(cfg=dict(eps=float("nan"))), -1),
    (dict(T=-1), -1), (dict(x=None), -1), (dict(ldx=63), -1), (dict(ldy=63), -1), (dict(p=None), -1), (dict(x1=None), -1),
    (dict(y=None), -1),                                   # after a block that is not there
    (dict(w=dict(after_weight=None)), -1), (dict(w=dict(before_weight=None)), -1),
    (dict(w=dict(after_bias=P)), -1), (dict(w=dict(before_bias=P)), -1),  # biases belong to layer norms
    (dict(w=dict(gate=P)), -1),                           # a gate without rows_per_gate
    (dict(cfg=dict(before=0)), -1),                       # a weight and a result without their norm
    (dict(p=P), -1), (dict(x1=P + 8), -1), (dict(x1=1 << 30), -1), (dict(x1=3 << 30), -1),  # overlaps
    (dict(x1=P, ldx=72), -1),                             # in place only with contiguous rows
])
def test_block_norm_refuses(moe, kw, code):
    assert norm_call(moe, **kw) == code


def test_block_norm_no_rows(moe):
    assert norm_call(moe, T=0) == 0
    assert moe.lib().colibri_moe_block_norm(None, None, None, 0, None, 0, 0, None, None, None) == -1


def back_call(m, cfg=(), w=None, grads=None, dx1=1 << 30, dp=2 << 30, x1=3 << 30, y=4 << 30, T=4, dx=5 << 30, dy=6 << 30,
              ld=64):
    c = dict(d_model=64, dtype=1, block_dtype=0, param_dtype=0, after=1, before=1, rows_per_gate=0, residual_scale=1.0,
             block_scale=1.0, eps=1e-6)
    c.update(cfg)
    v = dict(after_weight=P, before_weight=P)
    v.update(w or {})
    return m.lib().colibri_moe_block_norm_backward(
        ctypes.byref(m.NormConfig(**c)), ctypes.byref(m.NormVectors(**v)), dx1, ld, dp, ld, x1, ld, y, ld, T, dx, dy,
        ctypes.byref(m.NormVectors(**(grads or {}))), P, 1 << 20, None)


@pytest.mark.parametrize("kw", [
    dict(dp=None), dict(x1=None), dict(dx=None), dict(dy=None), dict(ld=63), dict(T=-2), dict(dx=1 << 30), dict(dy=5 << 30),
    dict(grads=dict(after_bias=P)), dict(grads=dict(gate=P)), dict(w=dict(gate=P), cfg=dict(rows_per_gate=2)),
    dict(cfg=dict(before=0), w=dict(before_weight=None), dp=None, dx1=None),
])
def test_block_norm_backward_refuses(moe, kw):
    assert back_call(moe, **kw) == -1


def route_call(m, T=4, ld=None, ptr=P, ws=P, ws_bytes=1 << 20, **kw):
    c = dict(num_experts=64, top_k=8, score=0, groups=8, top_groups=4, group_top=2, renormalize=1, logits_dtype=0, scale=1.0)
    c.update(kw)
    cfg = m.RouteConfig(**c)
    L = m.lib()
    ld = c["num_experts"] if ld is None else ld
    f = L.colibri_moe_route_experts(ctypes.byref(cfg), ptr, ld, None, T, ptr, ptr, ptr, ptr, ptr, ptr, ws, ws_bytes, None)
    n = ctypes.c_size_t()
    return f, L.colibri_moe_route_experts_workspace(ctypes.byref(cfg), T, ctypes.byref(n)), n.value


@pytest.mark.parametrize("kw,code", [
    (dict(num_experts=0), -1), (dict(top_k=0), -1), (dict(top_k=33), -1), (dict(num_experts=64, top_k=65), -1),
    (dict(score=2), -1), (dict(groups=0), -1), (dict(groups=7), -1), (dict(top_groups=0), -1), (dict(top_groups=9), -1),
    (dict(group_top=0), -1), (dict(group_top=3), -1), (dict(renormalize=2), -1), (dict(logits_dtype=3), -1),
    (dict(num_experts=513, groups=1, top_groups=1), -6), (dict(num_experts=64, groups=64, top_groups=64), -6),
    (dict(num_experts=64, groups=1, top_groups=1, top_k=33), -6), (dict(T=-1), -1), (dict(T=1 << 29), -1),
])
def test_route_refuses(moe, kw, code):
    f, w, _ = route_call(moe, **kw)
    assert f == code and w == code


def test_route_refuses_pointers_and_workspaces(moe):
    assert route_call(moe, ptr=None)[0] == -1
    assert route_call(moe, ld=63)[0] == -1
    assert route_call(moe, T=0, ptr=None)[0] == -1       # counts and offsets are written for no tokens, too
    assert route_call(moe, T=33, ws=None)[0] == -1
    _, rc, need = route_call(moe, T=4096)
    assert rc == 0 and need > 0
    assert route_call(moe, T=4096, ws_bytes=need - 1)[0] == -1
    L = moe.lib()
    cfg = moe.RouteConfig(64, 8, 0, 1, 1, 1, 1, 0, 1.0)
    assert L.colibri_moe_route_experts_backward(ctypes.byref(cfg), P, 64, P, P, 4, P, 63, None) == -1
    assert L.colibri_moe_route_experts_backward(ctypes.byref(cfg), P, 64, None, P, 4, P, 64, None) == -1
    assert L.colibri_moe_route_experts_backward(ctypes.byref(cfg), None, 64, None, None, 0, None, 64, None) == 0
    assert L.colibri_moe_route_experts(None, P, 64, None, 1, P, P, P, P, P, P, None, 0, None) == -1


def int8_call(m, n=8, R=8, rows=P, x=P, ldx=None, off=P, w=P, ws=P, w3=None, w3s=None, y=P, work=4096, size=1 << 40, **kw):
    c = dict(in_features=64, out_features=32, num_experts=4, dtype=1, out_dtype=0)
    c.update(kw)
    return m.lib().colibri_moe_int8_experts(ctypes.byref(m.Int8Config(**c)), x, c["in_features"] if ldx is None else ldx, n,
                                            rows, R, off, w, ws, w3, w3s, y, work, size, None)


@pytest.mark.parametrize("kw,code", [
    (dict(in_features=0), -1), (dict(in_features=72), -6), (dict(in_features=65552), -6), (dict(out_features=0), -1),
    (dict(out_features=131073), -6), (dict(num_experts=0), -1), (dict(num_experts=513), -6), (dict(dtype=2), -1),
    (dict(out_dtype=2), -1), (dict(n=-1), -1), (dict(R=-1), -1), (dict(rows=None, R=9), -1), (dict(x=None), -1),
    (dict(ldx=63), -1), (dict(off=None), -1), (dict(w=None), -1), (dict(ws=None), -1), (dict(y=None), -1),
    (dict(w3=P), -1), (dict(w3s=P), -1), (dict(w=P + 8), -1), (dict(w3=P + 8, w3s=P), -1), (dict(work=None), -1),
    (dict(work=4100), -1), (dict(size=16), -1),
])
def test_int8_refuses(moe, kw, code):
    assert int8_call(moe, **kw) == code


def test_int8_no_rows_and_quantize(moe):
    assert int8_call(moe, R=0) == 0
    L = moe.lib()
    c = moe.Int8Config(64, 32, 4, 1, 0)
    assert L.colibri_moe_int8_quantize(ctypes.byref(c), P, 63, 4, P, P, None) == -1
    assert L.colibri_moe_int8_quantize(ctypes.byref(c), P, 64, -1, P, P, None) == -1
    assert L.colibri_moe_int8_quantize(ctypes.byref(c), None, 64, 4, P, P, None) == -1
    assert L.colibri_moe_int8_quantize(ctypes.byref(c), None, 64, 0, None, None, None) == 0
    for args in ((P, 0, 4, P, P, -1, 2, 8, P, 0), (P, 0, 4, P, P, 1, 0, 8, P, 0), (P, 2, 4, P, P, 1, 2, 8, P, 0),
                 (P, 0, 4, P, P, 1, 2, 0, P, 0), (None, 0, 4, P, P, 1, 2, 8, P, 0), (P, 0, 4, None, P, 1, 2, 8, P, 0)):
        assert L.colibri_moe_combine_rows(*args, None) == -1
    assert L.colibri_moe_combine_rows(P, 0, 4, P, P, 1, 33, 8, P, 0, None) == -6
    assert L.colibri_moe_combine_rows(None, 0, 0, None, None, 0, 2, 8, None, 0, None) == 0


def test_trusted_pointers_is_a_flag(moe):
    assert norm_call(moe, cfg=dict(trusted_pointers=2)) == -1
    assert route_call(moe, trusted_pointers=-1)[0] == -1
    assert int8_call(moe, trusted_pointers=2) == -1
    assert norm_call(moe, cfg=dict(trusted_pointers=1), x=None) == -1  # it does not stand for a NULL


def test_valid_calls_without_a_gpu_report_cuda_errors(moe):
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert norm_call(moe) == -4 and back_call(moe) == -4 and route_call(moe)[0] == -4 and int8_call(moe) == -4


def test_python_layer_checks_shapes(moe):
    torch = pytest.importorskip("torch")
    from mixture_experts_gemm_gb300 import ops
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        ops.pre_norm(x, torch.ones(8))
    with pytest.raises(ValueError, match="CUDA"):
        ops.route(x, 2)
    with pytest.raises(ValueError, match="CUDA"):
        ops.int8_experts(x, torch.zeros(1, 4, 8, dtype=torch.int8), torch.ones(1, 4), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        ops.combine(x[0], torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, 1))
    with pytest.raises(ValueError):
        ops.block_norm_backward(None, None, None)
