"""What the calls that take tokens to their experts' rows and back refuse, without a GPU."""
import pytest

P = 4096  # an address that is never read
MOST = 2**31 - 1 - 2**24


@pytest.fixture(scope="module")
def L(cuda_lib):
    return cuda_lib


def call(L, name, **kw):
    args = {
        "dispatch_order": dict(idx=P, T=4, k=2, E=8, counts=P, offsets=P, row_of=P, token=P, trusted=1),
        "dispatch_rows": dict(x=P, dtype=1, ldx=64, T=4, token=P, R=8, d=64, rows=P, trusted=1),
        "dispatch_backward": dict(d_rows=P, dtype=1, R=8, row_of=P, T=4, k=2, d=64, d_x=P, out=0, trusted=1),
        "combine_backward": dict(d_out=P, dtype=1, ld=64, y=P, y_dtype=1, R=8, row_of=P, gate=P, token=P, T=4, k=2, d=64,
                                 d_y=P, d_gate=P, trusted=1),
        "gated": dict(u=P, ldu=64, v=P, ldv=64, dtype=1, R=4, f=64, h=P, out=0, trusted=1),
        "gated_backward": dict(d_h=P, h_dtype=1, ldh=64, u=P, ldu=64, v=P, ldv=64, dtype=1, R=4, f=64, d_u=P, d_v=P,
                               trusted=1),
    }[name]
    assert set(kw) <= set(args)
    return getattr(L, "colibri_moe_" + name)(*{**args, **kw}.values(), None)


@pytest.mark.parametrize("name,kw,code", [
    ("dispatch_order", dict(T=-1), -1), ("dispatch_order", dict(k=0), -1), ("dispatch_order", dict(E=0), -1),
    ("dispatch_order", dict(k=33), -6), ("dispatch_order", dict(E=513), -6), ("dispatch_order", dict(T=2**30), -6),
    ("dispatch_order", dict(T=MOST + 1, k=1), -6), ("dispatch_order", dict(idx=None), -1),
    ("dispatch_order", dict(counts=None), -1), ("dispatch_order", dict(T=0, offsets=None), -1),
    ("dispatch_order", dict(row_of=None), -1), ("dispatch_order", dict(token=None), -1),
    ("dispatch_order", dict(trusted=2), -1),
    ("dispatch_rows", dict(T=-1), -1), ("dispatch_rows", dict(R=-1), -1), ("dispatch_rows", dict(d=0), -1),
    ("dispatch_rows", dict(dtype=2), -1), ("dispatch_rows", dict(d=65537, ldx=65537), -6),
    ("dispatch_rows", dict(R=MOST + 1), -6), ("dispatch_rows", dict(T=MOST + 1), -6), ("dispatch_rows", dict(ldx=63), -1),
    ("dispatch_rows", dict(x=None), -1), ("dispatch_rows", dict(token=None), -1), ("dispatch_rows", dict(rows=None), -1),
    ("dispatch_rows", dict(trusted=-1), -1), ("dispatch_rows", dict(R=0, x=None, token=None, rows=None), 0),
    ("dispatch_backward", dict(T=-1), -1), ("dispatch_backward", dict(R=-1), -1), ("dispatch_backward", dict(k=0), -1),
    ("dispatch_backward", dict(k=33), -6), ("dispatch_backward", dict(d=0), -1), ("dispatch_backward", dict(d=65537), -6),
    ("dispatch_backward", dict(dtype=2), -1), ("dispatch_backward", dict(out=-1), -1),
    ("dispatch_backward", dict(T=MOST + 1), -6), ("dispatch_backward", dict(R=MOST + 1), -6),
    ("dispatch_backward", dict(d_rows=None), -1), ("dispatch_backward", dict(row_of=None), -1),
    ("dispatch_backward", dict(d_x=None), -1), ("dispatch_backward", dict(trusted=3), -1),
    ("dispatch_backward", dict(T=0, row_of=None, d_x=None), 0),
    ("combine_backward", dict(T=-1), -1), ("combine_backward", dict(R=-1), -1), ("combine_backward", dict(k=0), -1),
    ("combine_backward", dict(k=33), -6), ("combine_backward", dict(d=0), -1), ("combine_backward", dict(d=65537, ld=65537), -6),
    ("combine_backward", dict(dtype=2), -1), ("combine_backward", dict(y_dtype=2), -1), ("combine_backward", dict(ld=63), -1),
    ("combine_backward", dict(T=MOST + 1), -6), ("combine_backward", dict(R=MOST + 1), -6),
    ("combine_backward", dict(trusted=2), -1), ("combine_backward", dict(T=0, R=0), 0),
    *[("combine_backward", {n: None}, -1) for n in ("d_out", "y", "row_of", "gate", "token", "d_y", "d_gate")],
    ("gated", dict(R=-1), -1), ("gated", dict(f=0), -1), ("gated", dict(f=65537, ldu=65537, ldv=65537), -6),
    ("gated", dict(dtype=2), -1), ("gated", dict(out=2), -1), ("gated", dict(ldu=63), -1), ("gated", dict(ldv=63), -1),
    ("gated", dict(R=MOST + 1), -6), ("gated", dict(trusted=2), -1), ("gated", dict(R=0, u=None, v=None, h=None), 0),
    *[("gated", {n: None}, -1) for n in ("u", "v", "h")],
    ("gated_backward", dict(R=-1), -1), ("gated_backward", dict(f=0), -1), ("gated_backward", dict(h_dtype=2), -1),
    ("gated_backward", dict(dtype=-1), -1), ("gated_backward", dict(ldh=63), -1), ("gated_backward", dict(ldu=63), -1),
    ("gated_backward", dict(ldv=63), -1), ("gated_backward", dict(trusted=2), -1), ("gated_backward", dict(R=0, u=None), 0),
    *[("gated_backward", {n: None}, -1) for n in ("d_h", "u", "v", "d_u", "d_v")],
])
def test_refuses(L, name, kw, code):
    assert call(L, name, **kw) == code


def test_untrusted_pointers_are_looked_at(L):
    """Without the caller's word a pointer that is no device memory is refused; without a device that is an error of CUDA."""
    torch = pytest.importorskip("torch")
    want = -1 if torch.cuda.is_available() else -4
    for name in ("dispatch_order", "dispatch_rows", "dispatch_backward", "combine_backward", "gated", "gated_backward"):
        assert call(L, name, trusted=0) == want


def test_python_layer(cuda_lib):
    torch = pytest.importorskip("torch")
    from mixture_experts_gemm_gb300 import ops
    x, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    for f in (lambda: ops.dispatch_order(i, 4), lambda: ops.dispatch(x, i[:, 0]), lambda: ops.dispatch_backward(x, i),
              lambda: ops.combine_backward(x, x, i, x[:, :2], i[:, 0]), lambda: ops.gated(x, x),
              lambda: ops.gated_backward(x, x, x)):
        with pytest.raises(ValueError, match="CUDA"):
            f()
    with pytest.raises(ValueError, match="two dimensions"):
        ops.dispatch_order(i[0], 4)
