"""Operators of the block around the expert layer, and experts in 8-bit integers.

The counterparts of the context-free calls of ``include/colibri_moe.h``: norms before and after a
block with its gate and residual scale (``block_norm``), routing to many experts with the dispatch
order (``route``), experts in 8-bit integers (``int8_experts``) and their combine (``combine``), tokens to
their experts' rows and back for any choice of experts (``dispatch_order``, ``dispatch``), the gated activation
(``gated``), experts in 8-bit floating point (``fp8_experts``), with the backward passes of all but the 8-bit
integers.  Every call runs on CUDA tensors, asynchronously
on ``stream`` (default: the current stream), allocates its outputs and workspace from torch, and can be
captured into a CUDA graph.  Errors raise ``ColibriError`` (checks of the library) or ``ValueError``
(shapes and types that cannot be passed on).  Results are not attached to autograd: the backward passes
are calls of their own, and a call on tensors that ask for a gradient warns.  With a ``stream`` of its own
a call orders nothing: its inputs must be ready there and stay alive until that stream has read them.

    x1, p = block_norm(x, y, after="rms", after_weight=w_a, before="rms", before_weight=w_b)
    r = route(logits, 8, score="sigmoid", bias=b, groups=8, top_groups=4, group_top=2, scale=2.5)
    h = int8_experts(p, w1, s1, r.offsets, rows=r.token_of_row, w3=w3, w3_scale=s3)
    o = combine(int8_experts(h, w2, s2, r.offsets), r.row_of, r.gate)
"""
from __future__ import annotations

import ctypes
import functools
import operator
import struct
import warnings
from typing import NamedTuple, Optional

import torch

from . import DTYPE_BF16, DTYPE_F32, ColibriError, Fp8Config, Int8Config, NormConfig, RouteConfig, _check, lib

__all__ = ["block_norm", "block_norm_backward", "pre_norm", "route", "route_backward", "Routing", "int8_quantize",
           "int8_experts", "int8_status", "combine", "combine_backward", "dispatch_order", "Order", "dispatch",
           "dispatch_backward", "gated", "gated_backward", "fp8_quantize", "fp8_experts", "fp8_experts_backward",
           "fp8_status", "ColibriError"]

_DTYPE = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}
_NORMS = {"none": 0, "rms": 1, "layer": 2}
_SCORES = {"softmax": 0, "sigmoid": 1}


def _dtype(t, name: str) -> int:
    try:
        return _DTYPE[t]
    except KeyError:
        raise ValueError(f"{name}: float32 or bfloat16, not {t}") from None


def _kind(table, key, name: str) -> int:
    try:
        return table[key]
    except KeyError:
        raise ValueError(f"{name}: one of {', '.join(table)}, not {key!r}") from None


def _device(t, name: str) -> int:
    dev = t.get_device()
    if dev < 0 or not t.is_cuda:
        raise ValueError(f"{name}: a CUDA tensor is needed")
    return dev


def _matrix(t, name: str, T: int, d: int, dev: int, dtype=None):
    """(address, row stride) of a [T, d] tensor on CUDA device `dev` whose rows are contiguous."""
    if t.shape != (T, d):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {(T, d)}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, not on CUDA device {dev}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: {dtype} expected, not {t.dtype}")
    s0, s1 = t.stride()
    if s1 != 1 and d > 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    return t.data_ptr(), (s0 if T > 1 else max(d, 1))


def _shape(t, name: str):
    if t.dim() != 2:
        raise ValueError(f"{name}: two dimensions expected, not {tuple(t.shape)}")
    return t.shape


def _vector(t, name: str, shape, dtype, dev: int):
    """Address of a contiguous tensor of the given shape and type on CUDA device `dev`, or None for None."""
    if t is None:
        return None
    if t.shape != shape or t.dtype != dtype or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous tensor {tuple(shape)} of {dtype} on CUDA device {dev} expected, not "
                         f"{tuple(t.shape)} of {t.dtype} on {t.device}")
    return t.data_ptr()


class _on:
    """Makes the tensors' device current for the call, and their stream the caller's.

    Outputs and workspace come from torch's allocator on the stream that the kernels run on, so a block
    freed after the call is handed out again only behind them on that stream."""
    __slots__ = ("guard", "stream", "handle")

    def __init__(self, t, stream):
        dev = t.device.index
        self.guard = torch.cuda.device(dev) if dev != torch.cuda.current_device() else None
        if stream is None:
            self.stream = None
            self.handle = torch.cuda.current_stream(dev).cuda_stream
        else:
            if isinstance(stream, int):
                stream = torch.cuda.ExternalStream(stream, device=t.device)
            self.stream = torch.cuda.stream(stream)
            self.handle = stream.cuda_stream

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        if self.stream is not None:
            self.stream.__enter__()
        return self.handle

    def __exit__(self, *exc):
        if self.stream is not None:
            self.stream.__exit__(*exc)
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _run(f, t, dev: int, stream):
    """f(stream handle) on t's device `dev` and the given or current stream."""
    if stream is None and dev == torch._C._cuda_getDevice():  # the usual case, without the context managers
        return f(torch._C._cuda_getCurrentRawStream(dev))
    with _on(t, stream) as s:
        return f(s)


def _unattached(name: str, gradient: str, *tensors):
    """Says that a call's results leave autograd's graph, where one of its tensors asks for a gradient."""
    for t in tensors:
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            warnings.warn(f"{name}: the result is not attached to autograd and carries no gradient; {gradient}. Under "
                          "torch.no_grad(), or with detached tensors, this is not said", stacklevel=3)
            return


# Five pointers: colibri_moe_norm_params_t and colibri_moe_norm_grads_t.  Every call packs and holds its own.
_five = struct.Struct("5P").pack


def _workspace(n: int, device):
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def _at(t):
    return None if t is None else t.data_ptr()


# ------------------------------------------------------------------------------------------- norms
# The library reads a config through its address.  Every call holds the (struct, address) pair in a local until the
# library has returned: the caches may drop a struct while another thread fills them.  Scalars are plain numbers by
# then: a tensor would be found again by its identity, whatever it holds now.
@functools.lru_cache(maxsize=256)
def _norm_config(d, dtype, block_dtype, param_dtype, after, before, rows_per_gate, residual_scale, block_scale, eps):
    c = NormConfig(d, _dtype(dtype, "x"), _dtype(block_dtype, "y"), _dtype(param_dtype, "the parameters"),
                   _kind(_NORMS, after, "after"), _kind(_NORMS, before, "before"), rows_per_gate, residual_scale,
                   block_scale, eps, 1)
    return c, ctypes.addressof(c)


def _norm_setup(T, d, dev, dtype, block_dtype, after, after_weight, after_bias, before, before_weight, before_bias, gate,
                rows_per_gate, residual_scale, block_scale, eps):
    """(config, the parameters' addresses)."""
    pt = torch.float32
    for p in (after_weight, before_weight, gate):
        if p is not None:
            pt = p.dtype
            break
    rpg = 0
    pg = None
    if gate is not None:
        if gate.dim() == 1:
            gate = gate.unsqueeze(0)
        rpg = max(T, 1) if rows_per_gate is None else int(rows_per_gate)
        if rpg <= 0:
            raise ValueError("rows_per_gate must be positive")
        n_gates = -(-T // rpg) if T else gate.shape[0]
        pg = _vector(gate, "gate", (n_gates, d), pt, dev)
    one = (d,)
    vectors = _five(_vector(after_weight, "after_weight", one, pt, dev) or 0,
                    _vector(after_bias, "after_bias", one, pt, dev) or 0,
                    _vector(before_weight, "before_weight", one, pt, dev) or 0,
                    _vector(before_bias, "before_bias", one, pt, dev) or 0, pg or 0)
    return _norm_config(d, dtype, block_dtype, pt, after, before, rpg, float(residual_scale), float(block_scale),
                        float(eps)), vectors


def block_norm(x, y=None, *, after="none", after_weight=None, after_bias=None, before="none", before_weight=None,
               before_bias=None, gate=None, rows_per_gate=None, residual_scale=1.0, block_scale=1.0, eps=1e-6,
               stream=None):
    """Norms before and after a block, with its gate and the residual scale, in one pass:

        z  = norm_after(y) * after_weight + after_bias
        x1 = residual_scale * x + block_scale * gate * z
        p  = norm_before(x1) * before_weight + before_bias

    x [T, d] is the residual stream, y [T, d] the block's output (its own type: the expert layer gives
    fp32 beside a bf16 stream); after and before are "none", "rms" or "layer"; gate is [d] (every token)
    or [ceil(T / rows_per_gate), d].  Returns (x1, p); p is None without a next norm, and without y
    x1 is None (a norm before a block alone)."""
    T, d = _shape(x, "x")
    dt = x.dtype
    dev = _device(x, "x")
    px, ldx = _matrix(x, "x", T, d, dev)
    py, ldy = _matrix(y, "y", T, d, dev) if y is not None else (None, 0)
    config, vectors = _norm_setup(T, d, dev, dt, y.dtype if y is not None else dt, after, after_weight, after_bias,
                                  before, before_weight, before_bias, gate, rows_per_gate, residual_scale, block_scale,
                                  eps)
    _unattached("block_norm", "block_norm_backward computes it", x, y, after_weight, after_bias, before_weight,
                before_bias, gate)

    def call(s):
        x1 = torch.empty((T, d), dtype=dt, device=x.device) if y is not None else None
        p = torch.empty((T, d), dtype=dt, device=x.device) if before != "none" else None
        _check(lib().colibri_moe_block_norm(config[1], vectors, px, ldx, py, ldy, T, _at(x1), _at(p), s),
               "colibri_moe_block_norm")
        return x1, p
    return _run(call, x, dev, stream)


def pre_norm(x, weight, bias=None, *, kind="rms", eps=1e-6, stream=None):
    """norm(x) * weight (+ bias): the norm before a block, alone."""
    return block_norm(x, before=kind, before_weight=weight, before_bias=bias, eps=eps, stream=stream)[1]


def block_norm_backward(d_x1, d_p, x1, y=None, *, after="none", after_weight=None, after_bias=None, before="none",
                        before_weight=None, before_bias=None, gate=None, rows_per_gate=None, residual_scale=1.0,
                        block_scale=1.0, eps=1e-6, stream=None):
    """Gradients of block_norm from those of its results, as a dict: d_x, d_y, and in fp32 d_wa, d_ba
    (after), d_wb, d_bb (before), d_g (in the gate's shape), whichever the call has.  x1 and y are the
    forward call's (x1: x itself without y); d_x1 may be None where there is a next norm, d_p is None
    where there is none."""
    ref = d_x1 if d_x1 is not None else d_p
    if ref is None:
        raise ValueError("one of d_x1 and d_p is needed")
    T, d = _shape(ref, "d_x1" if d_x1 is not None else "d_p")
    dt = ref.dtype
    on = _device(ref, "d_x1")
    p1, ld1 = _matrix(d_x1, "d_x1", T, d, on, dt) if d_x1 is not None else (None, 0)
    pp, ldp = _matrix(d_p, "d_p", T, d, on, dt) if d_p is not None else (None, 0)
    px, ldx = _matrix(x1, "x1", T, d, on, dt) if x1 is not None else (None, 0)
    py, ldy = _matrix(y, "y", T, d, on) if y is not None else (None, 0)
    config, vectors = _norm_setup(T, d, on, dt, y.dtype if y is not None else dt, after, after_weight, after_bias,
                                  before, before_weight, before_bias, gate, rows_per_gate, residual_scale, block_scale,
                                  eps)

    def call(s):
        dev = ref.device
        out = dict(d_x=torch.empty((T, d), dtype=dt, device=dev))
        if y is not None:
            out["d_y"] = torch.empty((T, d), dtype=y.dtype, device=dev)
        for name, param in (("d_wa", after_weight), ("d_ba", after_bias), ("d_wb", before_weight),
                            ("d_bb", before_bias)):
            if param is not None:
                out[name] = torch.empty(d, dtype=torch.float32, device=dev)
        if gate is not None:
            out["d_g"] = (torch.empty if T else torch.zeros)(gate.shape, dtype=torch.float32, device=dev)
        grads = _five(*[out[n].data_ptr() if n in out else 0 for n in ("d_wa", "d_ba", "d_wb", "d_bb", "d_g")])
        L = lib()
        size = ctypes.c_size_t()
        _check(L.colibri_moe_block_norm_backward_workspace(config[1], T, ctypes.byref(size)),
               "colibri_moe_block_norm_backward")
        n = size.value
        ws = _workspace(n, dev)
        _check(L.colibri_moe_block_norm_backward(config[1], vectors, p1, ld1, pp, ldp, px, ldx, py, ldy, T,
                                                 _at(out["d_x"]), _at(out.get("d_y")), grads, _at(ws), n, s),
               "colibri_moe_block_norm_backward")
        return out
    return _run(call, ref, on, stream)


# ----------------------------------------------------------------------------------------- routing
class Routing(NamedTuple):
    """Experts and gates of every token, and the dispatch order (rows grouped by expert, tokens ascending)."""
    idx: torch.Tensor           # [T, k] int32, best first; -1: none left
    gate: torch.Tensor          # [T, k] fp32
    counts: torch.Tensor        # [E] int32
    offsets: torch.Tensor       # [E + 1] int32
    row_of: torch.Tensor        # [T, k] int32, -1 where idx is
    token_of_row: torch.Tensor  # [T * k] int32, -1 from offsets[E] on


@functools.lru_cache(maxsize=256)
def _route_config(E, k, score, groups, top_groups, group_top, renormalize, dtype, scale):
    c = RouteConfig(E, k, _kind(_SCORES, score, "score"), groups, top_groups, group_top, int(renormalize),
                    _dtype(dtype, "logits"), scale, 1)
    return c, ctypes.addressof(c)


def route(logits, top_k: int, *, score="softmax", bias=None, groups=1, top_groups=1, group_top=1, renormalize=True,
          scale=1.0, stream=None) -> Routing:
    """Routes every row of logits [T, E] (fp32 or bf16, rows may be strided) to top_k of E experts.

    Scores are a softmax over the experts or sigmoids; bias [E] (fp32) is added for the choice only;
    with groups > 1 only the experts of the top_groups best of `groups` equal runs compete, a group
    being worth the sum of its group_top (1 or 2) largest biased scores.  Gates are the chosen scores
    without the bias, divided by their sum if renormalize, times scale.  Ties go to the lowest index; an
    expert with a logit or bias of -inf or NaN is never chosen."""
    T, E = _shape(logits, "logits")
    on = _device(logits, "logits")
    pl, ld = _matrix(logits, "logits", T, E, on)
    pb = _vector(bias, "bias", (E,), torch.float32, on)
    k, index = operator.index(top_k), operator.index
    config = _route_config(E, k, score, index(groups), index(top_groups), index(group_top), bool(renormalize),
                           logits.dtype, float(scale))
    _unattached("route", "route_backward computes that of the gates", logits)

    def call(s):
        L, dev, i32 = lib(), logits.device, torch.int32
        need = ctypes.c_size_t()
        _check(L.colibri_moe_route_experts_workspace(config[1], T, ctypes.byref(need)), "colibri_moe_route_experts")
        size = need.value
        r = Routing(torch.empty((T, k), dtype=i32, device=dev), torch.empty((T, k), dtype=torch.float32, device=dev),
                    torch.empty(E, dtype=i32, device=dev), torch.empty(E + 1, dtype=i32, device=dev),
                    torch.empty((T, k), dtype=i32, device=dev), torch.empty(T * k, dtype=i32, device=dev))
        ws = _workspace(size, dev)
        _check(L.colibri_moe_route_experts(config[1], pl, ld, pb, T, *[t.data_ptr() for t in r], _at(ws), size, s),
               "colibri_moe_route_experts")
        return r
    return _run(call, logits, on, stream)


def route_backward(logits, idx, d_gate, *, score="softmax", renormalize=True, scale=1.0, stream=None):
    """d_logits [T, E] (the logits' type) from the gradient of the gates, the choice idx [T, k] held constant."""
    T, E = _shape(logits, "logits")
    on = _device(logits, "logits")
    pl, ld = _matrix(logits, "logits", T, E, on)
    k = _shape(idx, "idx")[1]
    pi = _vector(idx, "idx", (T, k), torch.int32, on)
    pg = _vector(d_gate, "d_gate", (T, k), torch.float32, on)
    config = _route_config(E, k, score, 1, 1, 1, bool(renormalize), logits.dtype, float(scale))

    def call(s):
        out = torch.empty((T, E), dtype=logits.dtype, device=logits.device)
        _check(lib().colibri_moe_route_experts_backward(config[1], pl, ld, pi, pg, T, out.data_ptr(), E, s),
               "colibri_moe_route_experts_backward")
        return out
    return _run(call, logits, on, stream)


# ----------------------------------------------------------------------------------- 8-bit experts
@functools.lru_cache(maxsize=256)
def _int8_config(K, N, E, dtype, out_dtype):
    c = Int8Config(K, N, E, _dtype(dtype, "x"), _dtype(out_dtype, "out_dtype"), 1)
    return c, ctypes.addressof(c)


def int8_quantize(x, stream=None):
    """(q int8, scale fp32) of the rows of x [..., K]: scale = max |x| / 127, q = round(x / scale).  Rows of
    activations, or the output channels of weights [E, N, K] once ahead of time."""
    K = x.shape[-1]
    on = _device(x, "x")
    config = _int8_config(K, 1, 1, x.dtype, torch.float32)
    _unattached("int8_quantize", "there is no backward pass", x)

    def call(s):
        flat = x.reshape(-1, K)  # a copy where x cannot be viewed so: made, read and freed on this call's stream
        px, ldx = _matrix(flat, "x", flat.shape[0], K, on)
        q = torch.empty(x.shape, dtype=torch.int8, device=x.device)
        scale = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        _check(lib().colibri_moe_int8_quantize(config[1], px, ldx, flat.shape[0], q.data_ptr(), scale.data_ptr(), s),
               "colibri_moe_int8_quantize")
        return q, scale
    return _run(call, x, on, stream)


def int8_experts(x, w, w_scale, offsets, *, rows=None, w3=None, w3_scale=None, out_dtype=None, stream=None):
    """y [R, N]: the rows of every expert times its 8-bit weights.

    x [n, K] (fp32 or bf16) is quantised per row within the call; w [E, N, K] int8 with w_scale [E, N]
    fp32; offsets [E + 1] int32 bounds every expert's rows and rows [R] int32 gives their tokens
    (``Routing.offsets`` and ``.token_of_row``), or None: row r is x[r].  With w3 and w3_scale (same
    shapes) y = silu(v) * v3, the gated pair of projections in one pass.  Rows from offsets[E] on are
    not written.  out_dtype: fp32 or bf16, default x's.  Should a wait inside the product run out (two
    seconds), y is undefined and ``int8_status`` says so."""
    n, K = _shape(x, "x")
    on = _device(x, "x")
    px, ldx = _matrix(x, "x", n, K, on)
    if w.dim() != 3:
        raise ValueError(f"w: [E, N, {K}] expected, not {tuple(w.shape)}")
    E, N, _ = w.shape
    i32, weights, scales = torch.int32, (E, N, K), (E, N)
    pw = _vector(w, "w", weights, torch.int8, on)
    ps = _vector(w_scale, "w_scale", scales, torch.float32, on)
    if (w3 is None) != (w3_scale is None):
        raise ValueError("w3 and w3_scale go together")
    pw3 = _vector(w3, "w3", weights, torch.int8, on)
    ps3 = _vector(w3_scale, "w3_scale", scales, torch.float32, on)
    po = _vector(offsets, "offsets", (E + 1,), i32, on)
    R = n if rows is None else rows.numel()
    pr = _vector(rows, "rows", (R,), i32, on)
    out_dtype = x.dtype if out_dtype is None else out_dtype
    config = _int8_config(K, N, E, x.dtype, out_dtype)
    _unattached("int8_experts", "there is no backward pass", x, w_scale, w3_scale)

    def call(s):
        L = lib()
        need = ctypes.c_size_t()
        _check(L.colibri_moe_int8_experts_workspace(config[1], n, R, ctypes.byref(need)), "colibri_moe_int8_experts")
        size = need.value
        ws = _workspace(size, x.device)
        y = torch.empty((R, N), dtype=out_dtype, device=x.device)
        _check(L.colibri_moe_int8_experts(config[1], px, ldx, n, pr, R, po, pw, ps, pw3, ps3, y.data_ptr(), _at(ws), size,
                                          s), "colibri_moe_int8_experts")
        return y
    return _run(call, x, on, stream)


def int8_status(device=None) -> int:
    """Waits for the device, then reads and clears its status word: 0, or 1 if a wait of any ``int8_experts`` call there
    gave up since the last read (its result is then undefined)."""
    status = ctypes.c_int32()
    with torch.cuda.device(device):
        _check(lib().colibri_moe_int8_status(ctypes.byref(status)), "colibri_moe_int8_status")
    return status.value


def combine(y, row_of, gate, *, out_dtype=None, stream=None):
    """out[t] = sum over a token's slots of gate * y[row_of], in slot order in fp32; rows of -1 are left out."""
    R, d = _shape(y, "y")
    on = _device(y, "y")
    py = _vector(y, "y", (R, d), y.dtype, on)
    T, k = _shape(row_of, "row_of")
    pr = _vector(row_of, "row_of", (T, k), torch.int32, on)
    pg = _vector(gate, "gate", (T, k), torch.float32, on)
    out_dtype = y.dtype if out_dtype is None else out_dtype
    types = _dtype(y.dtype, "y"), _dtype(out_dtype, "out_dtype")
    _unattached("combine", "there is no backward pass", y, gate)

    def call(s):
        out = torch.empty((T, d), dtype=out_dtype, device=y.device)
        _check(lib().colibri_moe_combine_rows(py, types[0], R, pr, pg, T, k, d, out.data_ptr(), types[1], s),
               "colibri_moe_combine_rows")
        return out
    return _run(call, y, on, stream)


# ------------------------------------------------------------------------- tokens to rows and back
class Order(NamedTuple):
    """The dispatch order of a choice of experts (rows grouped by expert, tokens ascending), as Routing has it."""
    counts: torch.Tensor        # [E] int32
    offsets: torch.Tensor       # [E + 1] int32
    row_of: torch.Tensor        # [T, k] int32, -1 where idx names no expert
    token_of_row: torch.Tensor  # [T * k] int32, -1 from offsets[E] on


def dispatch_order(idx, num_experts: int, *, stream=None) -> Order:
    """The dispatch order of any choice idx [T, k] (int32) of experts: a replayed one, another router's, one with slots
    dropped (an index outside 0..num_experts-1 gets no row).  A token may name an expert more than once."""
    T, k = _shape(idx, "idx")
    on = _device(idx, "idx")
    pi = _vector(idx, "idx", (T, k), torch.int32, on)
    E = operator.index(num_experts)
    if E < 1:
        raise ValueError("num_experts must be positive")

    def call(s):
        dev, i32 = idx.device, torch.int32
        o = Order(torch.empty(E, dtype=i32, device=dev), torch.empty(E + 1, dtype=i32, device=dev),
                  torch.empty((T, k), dtype=i32, device=dev), torch.empty(T * k, dtype=i32, device=dev))
        _check(lib().colibri_moe_dispatch_order(pi, T, k, E, *[t.data_ptr() for t in o], 1, s),
               "colibri_moe_dispatch_order")
        return o
    return _run(call, idx, on, stream)


def dispatch(x, token_of_row, *, stream=None):
    """rows [R, d]: x[token_of_row], zeros where the token is -1 (x's rows may be strided)."""
    T, d = _shape(x, "x")
    on = _device(x, "x")
    px, ldx = _matrix(x, "x", T, d, on)
    dt = _dtype(x.dtype, "x")
    R = token_of_row.numel()
    pt = _vector(token_of_row, "token_of_row", (R,), torch.int32, on)
    _unattached("dispatch", "dispatch_backward computes it", x)

    def call(s):
        rows = torch.empty((R, d), dtype=x.dtype, device=x.device)
        _check(lib().colibri_moe_dispatch_rows(px, dt, ldx, T, pt, R, d, rows.data_ptr(), 1, s),
               "colibri_moe_dispatch_rows")
        return rows
    return _run(call, x, on, stream)


def dispatch_backward(d_rows, row_of, *, out_dtype=None, stream=None):
    """d_x [T, d]: the sum of d_rows[row_of] over a token's slots, in slot order in fp32; rows of -1 are left out."""
    R, d = _shape(d_rows, "d_rows")
    on = _device(d_rows, "d_rows")
    pr = _vector(d_rows, "d_rows", (R, d), d_rows.dtype, on)
    T, k = _shape(row_of, "row_of")
    po = _vector(row_of, "row_of", (T, k), torch.int32, on)
    out_dtype = d_rows.dtype if out_dtype is None else out_dtype
    types = _dtype(d_rows.dtype, "d_rows"), _dtype(out_dtype, "out_dtype")

    def call(s):
        d_x = torch.empty((T, d), dtype=out_dtype, device=d_rows.device)
        _check(lib().colibri_moe_dispatch_backward(pr, types[0], R, po, T, k, d, d_x.data_ptr(), types[1], 1, s),
               "colibri_moe_dispatch_backward")
        return d_x
    return _run(call, d_rows, on, stream)


def combine_backward(d_out, y, row_of, gate, token_of_row, *, stream=None):
    """(d_y [R, d] in y's type, d_gate [T, k] fp32): the gradients of ``combine`` from that of its result, d_out [T, d].

    row_of and token_of_row are one dispatch order (``Routing`` or ``Order``).  Rows without a token get zeros, slots
    without a row a gate's gradient of 0."""
    T, d = _shape(d_out, "d_out")
    on = _device(d_out, "d_out")
    pd, ldd = _matrix(d_out, "d_out", T, d, on)
    R = _shape(y, "y")[0]
    py = _vector(y, "y", (R, d), y.dtype, on)
    k = _shape(row_of, "row_of")[1]
    po = _vector(row_of, "row_of", (T, k), torch.int32, on)
    pg = _vector(gate, "gate", (T, k), torch.float32, on)
    pt = _vector(token_of_row, "token_of_row", (R,), torch.int32, on)
    types = _dtype(d_out.dtype, "d_out"), _dtype(y.dtype, "y")

    def call(s):
        d_y = torch.empty((R, d), dtype=y.dtype, device=y.device)
        d_gate = torch.empty((T, k), dtype=torch.float32, device=y.device)
        _check(lib().colibri_moe_combine_backward(pd, types[0], ldd, py, types[1], R, po, pg, pt, T, k, d, d_y.data_ptr(),
                                                  d_gate.data_ptr(), 1, s), "colibri_moe_combine_backward")
        return d_y, d_gate
    return _run(call, d_out, on, stream)


# ------------------------------------------------------------------------------ gated activation
def gated(u, v, *, out_dtype=None, stream=None):
    """silu(u) * v of two [R, f] tensors of one type, whose rows may be strided (the halves of one product, say)."""
    R, f = _shape(u, "u")
    on = _device(u, "u")
    pu, ldu = _matrix(u, "u", R, f, on)
    pv, ldv = _matrix(v, "v", R, f, on, u.dtype)
    out_dtype = u.dtype if out_dtype is None else out_dtype
    types = _dtype(u.dtype, "u"), _dtype(out_dtype, "out_dtype")
    _unattached("gated", "gated_backward computes it", u, v)

    def call(s):
        h = torch.empty((R, f), dtype=out_dtype, device=u.device)
        _check(lib().colibri_moe_gated(pu, ldu, pv, ldv, types[0], R, f, h.data_ptr(), types[1], 1, s), "colibri_moe_gated")
        return h
    return _run(call, u, on, stream)


def gated_backward(d_h, u, v, *, stream=None):
    """(d_u, d_v), in the type of u and v, from the gradient of ``gated``'s result (of its own type)."""
    R, f = _shape(u, "u")
    on = _device(u, "u")
    ph, ldh = _matrix(d_h, "d_h", R, f, on)
    pu, ldu = _matrix(u, "u", R, f, on)
    pv, ldv = _matrix(v, "v", R, f, on, u.dtype)
    types = _dtype(d_h.dtype, "d_h"), _dtype(u.dtype, "u")

    def call(s):
        d_u, d_v = (torch.empty((R, f), dtype=u.dtype, device=u.device) for _ in range(2))
        _check(lib().colibri_moe_gated_backward(ph, types[0], ldh, pu, ldu, pv, ldv, types[1], R, f, d_u.data_ptr(),
                                                d_v.data_ptr(), 1, s), "colibri_moe_gated_backward")
        return d_u, d_v
    return _run(call, u, on, stream)


# ------------------------------------------------------------------------ 8-bit floating-point experts
_FP8, _BLOCK = torch.float8_e4m3fn, 128


@functools.lru_cache(maxsize=256)
def _fp8_config(K, N, E, dtype, out_dtype):
    c = Fp8Config(K, N, E, _dtype(dtype, "x"), _dtype(out_dtype, "out_dtype"), 1)
    return c, ctypes.addressof(c)


def _blocks(n: int) -> int:
    return -(-n // _BLOCK)


def _fp8_weights(w, w_scale, on: int):
    """(E, N, K, address of w [E, N, K], address of its scales)."""
    if w.dim() != 3:
        raise ValueError(f"w: [E, N, K] expected, not {tuple(w.shape)}")
    E, N, K = w.shape
    pw = _vector(w, "w", (E, N, K), _FP8, on)
    if w_scale is None:
        raise ValueError("w and w_scale go together")
    return E, N, K, pw, _vector(w_scale, "w_scale", (E, _blocks(N), _blocks(K)), torch.float32, on)


def fp8_quantize(x, *, square=False, stream=None):
    """(q float8_e4m3fn in x's shape, scale fp32) of x [..., n, K]: scale = max |x| / 448 over a block, q = x / scale
    rounded to e4m3.  Blocks of 128 columns of a row, scale [..., n, ceil(K / 128)]; or with square (weights, once
    ahead of time) of 128 x 128, scale [..., ceil(n / 128), ceil(K / 128)]."""
    if x.dim() < (2 if square else 1):
        raise ValueError(f"x: a matrix or more expected, not {tuple(x.shape)}")
    K = x.shape[-1]
    on = _device(x, "x")
    n = x.shape[-2] if square else 1
    config = _fp8_config(K, 1, max(x.numel() // (n * K), 1) if square and n * K else 1, x.dtype, torch.float32)
    _unattached("fp8_quantize", "there is no backward pass", x)

    def call(s):
        flat = x.reshape(-1, K)  # a copy where x cannot be viewed so: made, read and freed on this call's stream
        px, ldx = _matrix(flat, "x", flat.shape[0], K, on)
        q = torch.empty(x.shape, dtype=_FP8, device=x.device)
        shape = (*x.shape[:-2], _blocks(n), _blocks(K)) if square else (*x.shape[:-1], _blocks(K))
        scale = torch.empty(shape, dtype=torch.float32, device=x.device)
        _check(lib().colibri_moe_fp8_quantize(config[1], px, ldx, flat.shape[0], int(square), q.data_ptr(),
                                              scale.data_ptr(), s), "colibri_moe_fp8_quantize")
        return q, scale
    return _run(call, x, on, stream)


def fp8_experts(x, w, w_scale, offsets, *, rows=None, w3=None, w3_scale=None, out_dtype=None, stream=None):
    """y [R, N]: the rows of every expert times its weights in e4m3, a scale for every block of 128.

    x [n, K] (fp32 or bf16) is quantised within the call, in blocks of 128 columns of a row; w [E, N, K] e4m3 with
    w_scale [E, ceil(N / 128), ceil(K / 128)] fp32 (``fp8_quantize(..., square=True)``, or a checkpoint's); offsets
    and rows as for ``int8_experts``.  With w3 and w3_scale (same shapes) y = silu(v) * v3, the gated pair of
    projections in one pass.  Rows from offsets[E] on are not written.  out_dtype: fp32 or bf16, default x's.
    Should a wait inside the product run out (two seconds), y is undefined and ``fp8_status`` says so."""
    n, K = _shape(x, "x")
    on = _device(x, "x")
    px, ldx = _matrix(x, "x", n, K, on)
    E, N, wk, pw, ps = _fp8_weights(w, w_scale, on)
    if wk != K:
        raise ValueError(f"w: [E, N, {K}] expected, not {tuple(w.shape)}")
    if (w3 is None) != (w3_scale is None):
        raise ValueError("w3 and w3_scale go together")
    pw3 = _vector(w3, "w3", (E, N, K), _FP8, on)
    ps3 = _vector(w3_scale, "w3_scale", w_scale.shape, torch.float32, on)
    po = _vector(offsets, "offsets", (E + 1,), torch.int32, on)
    R = n if rows is None else rows.numel()
    pr = _vector(rows, "rows", (R,), torch.int32, on)
    out_dtype = x.dtype if out_dtype is None else out_dtype
    config = _fp8_config(K, N, E, x.dtype, out_dtype)
    _unattached("fp8_experts", "fp8_experts_backward computes it", x, w_scale, w3_scale)

    def call(s):
        L = lib()
        need = ctypes.c_size_t()
        _check(L.colibri_moe_fp8_experts_workspace(config[1], n, R, ctypes.byref(need)), "colibri_moe_fp8_experts")
        size = need.value
        ws = _workspace(size, x.device)
        y = torch.empty((R, N), dtype=out_dtype, device=x.device)
        _check(L.colibri_moe_fp8_experts(config[1], px, ldx, n, pr, R, po, pw, ps, pw3, ps3, y.data_ptr(), _at(ws), size,
                                         s), "colibri_moe_fp8_experts")
        return y
    return _run(call, x, on, stream)


def fp8_experts_backward(d_y, x, w, w_scale, offsets, *, rows=None, weight_dtype=torch.float32, stream=None):
    """(d_rows [R, K], d_w [E, N, K]): the gradients of ``fp8_experts`` without w3, from that of y, d_y [R, N].

    d_rows, in d_y's type, has a row for each of y's (``dispatch_backward`` adds up a token's; rows from offsets[E]
    on are not written): d_y quantised in blocks of 128 columns times the weights.  d_w, of weight_dtype (fp32 or
    bf16), is that of the weights' values, w * w_scale: d_y and x [n, K] quantised in blocks of 128 rows of an
    expert, summed over its rows (zeros for an expert without any).  With x None there is no d_w, with w and
    w_scale None no d_rows (None in their place; x's type is d_y's)."""
    R, N = _shape(d_y, "d_y")
    on = _device(d_y, "d_y")
    pd, ldd = _matrix(d_y, "d_y", R, N, on)
    E = offsets.numel() - 1
    if E < 1:
        raise ValueError("offsets: [E + 1] expected")
    po = _vector(offsets, "offsets", (E + 1,), torch.int32, on)
    if w is None and x is None:
        raise ValueError("one of x and w is needed")
    n, K, pw, ps, px, ldx, pr = R, None, None, None, None, 0, None
    if w is not None:
        we, wn, K, pw, ps = _fp8_weights(w, w_scale, on)
        if (we, wn) != (E, N):
            raise ValueError(f"w: [{E}, {N}, K] expected, not {tuple(w.shape)}")
    elif w_scale is not None:
        raise ValueError("w and w_scale go together")
    if x is not None:
        n, K = _shape(x, "x")[0], K or x.shape[1]
        px, ldx = _matrix(x, "x", n, K, on, d_y.dtype)
        pr = _vector(rows, "rows", (R,), torch.int32, on)
    config = _fp8_config(K, N, E, d_y.dtype, weight_dtype)

    def call(s):
        L, dev = lib(), d_y.device
        need = ctypes.c_size_t()
        _check(L.colibri_moe_fp8_experts_backward_workspace(config[1], n, R, ctypes.byref(need)),
               "colibri_moe_fp8_experts_backward")
        size = need.value
        ws = _workspace(size, dev)
        d_rows = torch.empty((R, K), dtype=d_y.dtype, device=dev) if w is not None else None
        d_w = torch.empty((E, N, K), dtype=weight_dtype, device=dev) if x is not None else None
        if R or d_w is not None:
            of_w = (pw, ps, _at(d_rows)) if R else (None, None, None)
            _check(L.colibri_moe_fp8_experts_backward(config[1], pd, ldd, px, ldx, n, pr, R, po, *of_w, _at(d_w), _at(ws),
                                                      size, s), "colibri_moe_fp8_experts_backward")
        return d_rows, d_w
    return _run(call, d_y, on, stream)


def fp8_status(device=None) -> int:
    """As ``int8_status``, for the products of ``fp8_experts`` and ``fp8_experts_backward``."""
    status = ctypes.c_int32()
    with torch.cuda.device(device):
        _check(lib().colibri_moe_fp8_status(ctypes.byref(status)), "colibri_moe_fp8_status")
    return status.value
