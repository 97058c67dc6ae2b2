"""The operators of an expert layer's training step and of experts in 8-bit floating point, in their plain
form, and the cases they are measured at.

Tokens to their experts' rows and back (the dispatch order of any choice of experts, the rows, and the
gradients of both ways, with the gates applied), the gated activation between the two projections with its
gradient, and the experts' products in e4m3 with a scale for every block of 128, forward and backward.
Where `own` is true `run` calls the package's kernels, otherwise elementary torch operations compute the
same thing.  Sizes come from the layer shapes this repository is measured on (hidden 256, 2048 and 4096,
inner 512, 1408, 5632 and 14336, 8192 tokens of prefill, 1 to 32 of decode) and, for layers of many
experts, 60, 64 and 256 experts.

    order[e] = the slots (t, s) with idx[t, s] == e, tokens ascending;  rows of all experts one after another
    rows[r] = x[token_of_row[r]],  d_x[t] = sum_s d_rows[row_of[t, s]]
    out[t] = sum_s gate[t, s] y[row_of[t, s]]:  d_y[row] = gate d_out[t],  d_gate[t, s] = <d_out[t], y[row]>
    h = silu(u) v:  d_u = d_h v silu'(u),  d_v = d_h silu(u)
    q = e4m3(x / scale),  scale = max |x| / 448 over a block of 128
    y[r, n] = sum_b sx[r, b] sw[n / 128, b] sum_{k in b} qx[r, k] qw[n, k];  the gradients are the same products
    with d_y in blocks along n (for the rows') and with d_y and x in blocks along the rows (for the weights')
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
B = 128  # elements of a scale's block
TOP = 448.0  # the largest e4m3
DEV = "cuda"


# ------------------------------------------------------------------------------------------ cases
def _named(name, c):
    return dict(c, name=name) if name else c


def _dispatch(name, T, k, E, d, dtype, dropped):
    return _named(name, dict(op="dispatch", T=T, k=k, E=E, d=d, dtype=dtype, dropped=dropped))


def _dispatch_backward(name, T, k, E, d, dtype, out, dropped):
    return _named(name, dict(op="dispatch_backward", T=T, k=k, E=E, d=d, dtype=dtype, out=out, dropped=dropped))


def _combine_backward(name, T, k, E, d, dtype, y_dtype, dropped):
    return _named(name, dict(op="combine_backward", T=T, k=k, E=E, d=d, dtype=dtype, y_dtype=y_dtype, dropped=dropped))


def _gated(name, R, f, dtype, out, backward):
    return _named(name, dict(op="gated_backward" if backward else "gated", R=R, f=f, dtype=dtype, out=out))


def _fp8(name, T, k, E, K, N, swiglu, dtype, out, skew):
    return _named(name, dict(op="fp8", T=T, k=k, E=E, K=K, N=N, swiglu=swiglu, dtype=dtype, out=out, skew=skew))


def _fp8_backward(name, T, k, E, K, N, dtype, out, skew):
    return _named(name, dict(op="fp8_backward", T=T, k=k, E=E, K=K, N=N, dtype=dtype, out=out, skew=skew))


def listed():
    return [
        # one decoded token of a layer with 256 experts, its choice replayed: order and rows, a call's latency
        _dispatch("dispatch-token", 1, 8, 256, 4096, "bf16", 0.0),
        # a prefill batch of the large layer
        _dispatch("dispatch-prefill", 8192, 2, 8, 4096, "bf16", 0.0),
        # the rows' gradients back to an odd batch, an odd width; experts over their capacity dropped some slots
        _dispatch_backward("dispatch-backward-odd", 4099, 4, 60, 1409, "f32", "f32", 0.1),
        # a training step's combine: the gradients of the experts' results and of the gates
        _combine_backward("combine-backward", 8192, 2, 8, 4096, "bf16", "bf16", 0.0),
        # the activation between the projections of small experts, an odd width, fp32
        _gated("gated-odd", 6126, 1409, "f32", "f32", False),
        # the same in a training step of the large layer: both halves of one product, and their gradients
        _gated("gated-backward", 16384, 14336, "bf16", "bf16", True),
        # one decoded token, two experts of the large layer: the weights' bytes
        _fp8("fp8-token", 1, 2, 8, 4096, 14336, True, "bf16", "bf16", 0.0),
        # a batch of 512 tokens, the middle layer's up projections
        _fp8("fp8-batch", 512, 2, 8, 2048, 5632, True, "bf16", "bf16", 0.0),
        # a batch over 64 small experts, unevenly loaded, an odd number of channels and tokens
        _fp8("fp8-many-experts", 1021, 6, 64, 2048, 1409, False, "f32", "f32", 1.0),
        # prefill: 8192 tokens, the large layer's down projection
        _fp8("fp8-prefill", 8192, 2, 8, 14336, 4096, False, "bf16", "bf16", 0.3),
        # a training step over 16 unevenly loaded experts: the gradients of the rows and of the weights
        _fp8_backward("fp8-backward-skewed", 4096, 2, 16, 2048, 1408, "bf16", "f32", 1.5),
        # the large layer's down projection in a training step, gradients of the weights kept in bf16
        _fp8_backward("fp8-backward-large", 8192, 2, 8, 14336, 4096, "bf16", "bf16", 0.3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dispatch", "dispatch_backward", "combine_backward", "gated", "gated_backward", "fp8", "fp8", "fp8",
                     "fp8_backward", "fp8_backward"])
    dtype, out = rng.choice(["f32", "bf16"]), rng.choice(["f32", "bf16"])
    if op in ("dispatch", "dispatch_backward", "combine_backward"):
        E = _log(rng, 1, 512)
        k = rng.randint(1, min(10, E))
        d = _log(rng, 64, 8192)
        if rng.random() < 0.6:
            d = (d + 7) // 8 * 8
        T = _log(rng, 1, max(1, min(16384, 8192 * 4 * 4096 // (d * k))))
        dropped = rng.choice([0.0, 0.0, 0.1, 0.5])
        if op == "dispatch":
            return _dispatch(None, T, k, E, d, dtype, dropped)
        return (_dispatch_backward if op == "dispatch_backward" else _combine_backward)(None, T, k, E, d, dtype, out, dropped)
    if op in ("gated", "gated_backward"):
        f = _log(rng, 64, 14336)
        if rng.random() < 0.6:
            f = (f + 7) // 8 * 8
        return _gated(None, _log(rng, 1, 16384), f, dtype, out, op == "gated_backward")
    K = (_log(rng, 64, 14336) + 15) // 16 * 16
    N = _log(rng, 64, 14336)
    E = rng.choice([1, 4, 8, 16, 60, 64])
    swiglu = op == "fp8" and rng.random() < 0.5
    while E * N * K * (2 if swiglu else 1) > 8 * 14336 * 4096:
        N = (N + 1) // 2
    k = rng.randint(1, min(E, 6))
    T = _log(rng, 1, 8192)
    while T > 1 and T * k * N * K * (2 if swiglu else 1) > 16384 * 14336 * 4096 // 2:
        T //= 2
    skew = rng.choice([0.0, 0.3, 1.0])
    if op == "fp8":
        return _fp8(None, T, k, E, K, N, swiglu, dtype, out, skew)
    return _fp8_backward(None, T, k, E, K, N, dtype, out, skew)


# ----------------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rn = lambda *shape: torch.randn(*shape, generator=g, device=DEV)  # noqa: E731
    s = dict(case)
    if case["op"] in ("gated", "gated_backward"):
        R, f, dt = case["R"], case["f"], DTYPES[case["dtype"]]
        both = (1.5 * rn(R, 2 * f)).to(dt)  # the two projections' results, as one product leaves them
        s["u"], s["v"] = both[:, :f], both[:, f:]
        if case["op"] == "gated_backward":
            s["d_h"] = rn(R, f).to(DTYPES[case["out"]])
        return s
    T, k, E = case["T"], case["k"], case["E"]
    # every token in k distinct experts, an uneven load if `skew`
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=g, device=DEV).clamp(1e-6, 1 - 1e-6)))
    load = -case.get("skew", 0.0) * torch.log(torch.arange(1, E + 1, device=DEV, dtype=torch.float32))
    idx = (noise + load).topk(k).indices.to(torch.int32)
    if case["op"] in ("dispatch", "dispatch_backward", "combine_backward"):
        d, dt = case["d"], DTYPES[case["dtype"]]
        if case["dropped"]:
            idx = idx.masked_fill(torch.rand(T, k, generator=g, device=DEV) < case["dropped"], -1)
        if case["op"] == "dispatch":
            s["x"], s["idx"] = rn(T, d).to(dt), idx
            return s
        _, _, s["row_of"], s["token_of_row"] = _order(idx, E)
        if case["op"] == "dispatch_backward":
            s["d_rows"] = rn(T * k, d).to(dt)
            return s
        s["gate"] = torch.rand(T, k, generator=g, device=DEV)
        s["d_out"], s["y"] = rn(T, d).to(dt), rn(T * k, d).to(DTYPES[case["y_dtype"]])
        return s
    K, N = case["K"], case["N"]
    counts, s["offsets"], _, s["rows"] = _order(idx, E)
    s["x"] = rn(T, K).to(DTYPES[case["dtype"]])
    s["w"], s["ws"] = _weights(E, N, K, g)
    s["w3"], s["w3s"] = _weights(E, N, K, g) if case.get("swiglu") else (None, None)
    if case["op"] == "fp8_backward":
        s["d_y"] = (rn(T * k, N) * torch.exp(rn(T * k, 1))).to(DTYPES[case["dtype"]])
    # the same rows as a rectangle of experts x the fullest expert's rows (whole blocks), for batched products
    s["cap"] = -(-int(counts.max()) // B) * B
    expert = torch.repeat_interleave(torch.arange(E, device=DEV), counts.long())
    s["at"] = expert * s["cap"] + torch.arange(T * k, device=DEV) - s["offsets"].long()[expert]
    return s


def _weights(E, N, K, g):
    """Normal weights of variance 1 / K in e4m3, with a scale for each block of 128 x 128."""
    w = torch.empty(E, N, K, dtype=torch.float8_e4m3fn, device=DEV)
    for e in range(E):
        w[e] = torch.randn(N, K, generator=g, device=DEV).mul_(100).clamp_(-TOP, TOP).to(torch.float8_e4m3fn)
    scale = torch.rand(E, -(-N // B), -(-K // B), generator=g, device=DEV)
    return w, (0.8 + 0.4 * scale) / (100 * math.sqrt(K))


# ------------------------------------------------------------------------------------ plain forms
def _order(idx, E):
    T, k = idx.shape
    flat = torch.where((idx >= 0) & (idx < E), idx, E).reshape(-1).long()
    counts = torch.zeros(E + 1, dtype=torch.int64, device=idx.device).scatter_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat([counts.new_zeros(1), counts[:E].cumsum(0)])
    order = torch.argsort(flat, stable=True)
    place = torch.arange(T * k, device=idx.device)
    row_of = torch.empty_like(flat).scatter_(0, order, place)
    row_of = torch.where(flat < E, row_of, -1).view(T, k)
    token = torch.where(place < offsets[E], order // k, -1)
    i32 = torch.int32
    return counts[:E].to(i32), offsets.to(i32), row_of.to(i32), token.to(i32)


def _plain_dispatch(s):
    counts, offsets, row_of, token = _order(s["idx"], s["E"])
    rows = torch.where((token >= 0)[:, None], s["x"][token.long().clamp(min=0)], 0)
    return dict(counts=counts, offsets=offsets, row_of=row_of, token_of_row=token, rows=rows)


def _taken(v, row_of):
    """v[row_of] in 32 bits, [T, k, d]; zeros where there is no row."""
    return torch.where((row_of >= 0)[:, :, None], v.float()[row_of.long().clamp(min=0)], 0.0)


def _plain_dispatch_backward(s):
    return dict(d_x=_taken(s["d_rows"], s["row_of"]).sum(1).to(DTYPES[s["out"]]))


def _plain_combine_backward(s):
    kept = s["row_of"] >= 0
    d_out = s["d_out"].float()
    d_gate = (_taken(s["y"], s["row_of"]) * d_out[:, None, :]).sum(2)
    weight = torch.zeros(s["T"] * s["k"], device=d_out.device)
    weight[s["row_of"][kept].long()] = s["gate"][kept]
    d_y = torch.where((s["token_of_row"] >= 0)[:, None], weight[:, None] * d_out[s["token_of_row"].long().clamp(min=0)], 0.0)
    return dict(d_y=d_y.to(s["y"].dtype), d_gate=d_gate)


def _plain_gated(s):
    u = s["u"].float()
    return dict(h=(u / (1 + torch.exp(-u)) * s["v"].float()).to(DTYPES[s["out"]]))


def _plain_gated_backward(s):
    u, v, d_h = s["u"].float(), s["v"].float(), s["d_h"].float()
    p = 1 / (1 + torch.exp(-u))
    d_u = d_h * v * (p * (1 + u * (1 - p)))
    return dict(d_u=d_u.to(s["u"].dtype), d_v=(d_h * (u * p)).to(s["v"].dtype))


def _quantised(v, dim):
    """v as e4m3 times a scale for each block of 128 along `dim`, in 32 bits."""
    n = v.shape[dim]
    pad = [0, 0] * (v.dim() - 1 - dim) + [0, -n % B]
    b = torch.nn.functional.pad(v, pad).unflatten(dim, (-1, B))
    # two tensors, so that the quotient is rounded once (by a number, it is a product with 1 / 448)
    scale = b.abs().amax(dim + 1, keepdim=True) / torch.full((1,), TOP, device=v.device)
    q = torch.where(scale > 0, b / scale, 0.0).clamp(-TOP, TOP).to(torch.float8_e4m3fn).float()
    return (q * scale).flatten(dim, dim + 1).narrow(dim, 0, n)


def _full(w, scale):
    return w.float() * scale.repeat_interleave(B, 1)[:, :w.shape[1]].repeat_interleave(B, 2)[:, :, :w.shape[2]]


def _rectangle(s, v):
    """Rows [R, C] as [E, cap, C]."""
    return torch.zeros(s["E"] * s["cap"], v.shape[1], device=v.device).index_copy_(0, s["at"], v).view(s["E"], s["cap"], -1)


def _plain_fp8(s):
    a = _rectangle(s, _quantised(s["x"].float(), 1)[s["rows"].long()])

    def product(w, scale):
        return torch.bmm(a, _full(w, scale).transpose(1, 2)).flatten(0, 1)[s["at"]]

    y = product(s["w"], s["ws"])
    if s["swiglu"]:
        y = y / (1 + torch.exp(-y)) * product(s["w3"], s["w3s"])
    return dict(y=y.to(DTYPES[s["out"]]))


def _plain_fp8_backward(s):
    d_y = s["d_y"].float()
    d_rows = torch.bmm(_rectangle(s, _quantised(d_y, 1)), _full(s["w"], s["ws"])).flatten(0, 1)[s["at"]]
    down = _quantised(_rectangle(s, d_y), 1)
    d_w = torch.bmm(down.transpose(1, 2), _quantised(_rectangle(s, s["x"].float()[s["rows"].long()]), 1))
    return dict(d_rows=d_rows.to(s["x"].dtype), d_w=d_w.to(DTYPES[s["out"]]))


# -------------------------------------------------------------------------------------------- run
def run(s):
    op = s["op"]
    if not own:
        return {"dispatch": _plain_dispatch, "dispatch_backward": _plain_dispatch_backward,
                "combine_backward": _plain_combine_backward, "gated": _plain_gated,
                "gated_backward": _plain_gated_backward, "fp8": _plain_fp8, "fp8_backward": _plain_fp8_backward}[op](s)
    from mixture_experts_gemm_gb300 import ops
    if op == "dispatch":
        o = ops.dispatch_order(s["idx"], s["E"])
        return dict(counts=o.counts, offsets=o.offsets, row_of=o.row_of, token_of_row=o.token_of_row,
                    rows=ops.dispatch(s["x"], o.token_of_row))
    if op == "dispatch_backward":
        return dict(d_x=ops.dispatch_backward(s["d_rows"], s["row_of"], out_dtype=DTYPES[s["out"]]))
    if op == "combine_backward":
        d_y, d_gate = ops.combine_backward(s["d_out"], s["y"], s["row_of"], s["gate"], s["token_of_row"])
        return dict(d_y=d_y, d_gate=d_gate)
    if op == "gated":
        return dict(h=ops.gated(s["u"], s["v"], out_dtype=DTYPES[s["out"]]))
    if op == "gated_backward":
        d_u, d_v = ops.gated_backward(s["d_h"], s["u"], s["v"])
        return dict(d_u=d_u, d_v=d_v)
    if op == "fp8":
        return dict(y=ops.fp8_experts(s["x"], s["w"], s["ws"], s["offsets"], rows=s["rows"], w3=s["w3"],
                                      w3_scale=s["w3s"], out_dtype=DTYPES[s["out"]]))
    d_rows, d_w = ops.fp8_experts_backward(s["d_y"], s["x"], s["w"], s["ws"], s["offsets"], rows=s["rows"],
                                           weight_dtype=DTYPES[s["out"]])
    return dict(d_rows=d_rows, d_w=d_w)


# ------------------------------------------------------------------------------------------- work
def work(case):
    size = {"f32": 4, "bf16": 2}
    c = case
    if c["op"] in ("gated", "gated_backward"):
        n, s, o = c["R"] * c["f"], size[c["dtype"]], size[c["out"]]
        # u, v and h, or those and the two gradients
        return dict(bytes=n * (2 * s + o) if c["op"] == "gated" else n * (4 * s + o),
                    flops=(5 if c["op"] == "gated" else 10) * n)
    R = c["T"] * c["k"]
    if c["op"] in ("dispatch", "dispatch_backward", "combine_backward"):
        s = size[c["dtype"]]
        kept = int(R * (1 - c["dropped"]))
        if c["op"] == "dispatch":  # choice and rows read; rows, row_of, token_of_row, counts and offsets written
            return dict(bytes=c["d"] * s * (c["T"] + R) + 12 * R + 8 * c["E"], flops=R)
        if c["op"] == "dispatch_backward":
            return dict(bytes=c["d"] * (kept * s + c["T"] * size[c["out"]]) + 4 * R, flops=kept * c["d"])
        return dict(bytes=c["d"] * (c["T"] * s + (kept + R) * size[c["y_dtype"]]) + 16 * R, flops=3 * kept * c["d"])
    m = 2 if c.get("swiglu") else 1
    used = min(c["E"], R) if c["T"] > 1 else min(c["E"], c["k"])
    weights = m * used * c["N"] * c["K"] * (1 + 4 / B**2)
    product = 2 * m * R * c["N"] * c["K"]
    if c["op"] == "fp8":
        return dict(bytes=int(weights + c["T"] * c["K"] * size[c["dtype"]] + R * c["N"] * size[c["out"]]), flops=product)
    # d_y, x and the weights read, the gradients of the rows and of the weights (all experts') written
    return dict(bytes=int(weights + (c["T"] * c["K"] + R * (c["N"] + c["K"])) * size[c["dtype"]]
                          + c["E"] * c["N"] * c["K"] * size[c["out"]]), flops=2 * product)


# ------------------------------------------------------------------------------------------ exact
def exact(case, seed):
    """From the definitions in 64 bits; whole numbers are compared with the plain form's for equality.  A block's
    scale and its quotients are rounded to 32 bits, as the format says."""
    s = prepare(case, seed)
    return {"dispatch": _exact_dispatch, "dispatch_backward": _exact_dispatch_backward,
            "combine_backward": _exact_combine_backward, "gated": _exact_gated, "gated_backward": _exact_gated_backward,
            "fp8": _exact_fp8, "fp8_backward": _exact_fp8_backward}[s["op"]](s)


def _exact_dispatch(s):
    """Expert by expert, its tokens as they come."""
    rows, at = torch.zeros(s["T"] * s["k"], s["d"], dtype=torch.float64, device=s["x"].device), 0
    for e in range(s["E"]):
        t = (s["idx"] == e).nonzero()[:, 0]
        rows[at:at + len(t)] = s["x"][t].double()
        at += len(t)
    return dict(rows=rows)


def _exact_dispatch_backward(s):
    d_x = torch.zeros(s["T"], s["d"], dtype=torch.float64, device=s["d_rows"].device)
    t = s["token_of_row"].long()
    d_x.index_add_(0, t[t >= 0], s["d_rows"][t >= 0].double())
    return dict(d_x=d_x)


def _exact_combine_backward(s):
    """Differentiates the combine by torch's own rules, slot by slot."""
    y, gate = s["y"].double().requires_grad_(True), s["gate"].double().requires_grad_(True)
    with torch.enable_grad():
        for j in range(s["k"]):
            row = s["row_of"][:, j].long()
            t = (row >= 0).nonzero()[:, 0]
            part = gate[t, j][:, None] * y.index_select(0, row[t])
            (part * s["d_out"][t].double()).sum().backward()
    return dict(d_y=y.grad, d_gate=gate.grad)


def _exact_gated(s):
    u = s["u"].double()
    return dict(h=u * torch.sigmoid(u) * s["v"].double())


def _exact_gated_backward(s):
    u, v = s["u"].double().requires_grad_(True), s["v"].double().requires_grad_(True)
    with torch.enable_grad():
        (torch.nn.functional.silu(u) * v).backward(s["d_h"].double())
    return dict(d_u=u.grad, d_v=v.grad)


def _rounded(v):
    """v (32 bits) to the nearest e4m3, ties to even: steps of 2^-3 of the power of two below, of 2^-9 at least."""
    power = torch.frexp(v).exponent.clamp(min=-5) - 4
    step = torch.ldexp(torch.ones_like(v), power)
    return ((v / step).round() * step).clamp(-TOP, TOP)


def _blocks(x, lo, hi):
    """Columns lo .. hi of x in 64 bits, each row's as e4m3 times its scale."""
    p = x[:, lo:hi].to(torch.float32)
    scale = torch.div(p.abs().max(1, keepdim=True).values, torch.full((1, 1), TOP, device=x.device))
    q = torch.where(scale > 0, torch.div(p, scale), torch.zeros_like(p))
    return _rounded(q).double() * scale.double()


def _exact_rows(x):
    return torch.cat([_blocks(x, lo, min(lo + B, x.shape[1])) for lo in range(0, x.shape[1], B)], 1)


def _dequantised(w, scale):
    out = w.double()
    for j in range(scale.shape[0]):
        out[j * B:(j + 1) * B] *= scale[j].double().repeat_interleave(B)[:w.shape[1]]
    return out


def _too_long(s, products):
    return 2 * s["T"] * s["k"] * s["N"] * s["K"] * products > 6e12


def _exact_fp8(s):
    if _too_long(s, 2 if s["swiglu"] else 1):
        return None
    x = _exact_rows(s["x"])
    off = s["offsets"].tolist()
    y = torch.zeros(s["T"] * s["k"], s["N"], dtype=torch.float64, device=x.device)
    for e in range(s["E"]):
        if off[e + 1] > off[e]:
            t = s["rows"][off[e]:off[e + 1]].long()
            v = x[t] @ _dequantised(s["w"][e], s["ws"][e]).T
            if s["swiglu"]:
                v = v * torch.sigmoid(v) * (x[t] @ _dequantised(s["w3"][e], s["w3s"][e]).T)
            y[off[e]:off[e + 1]] = v
    return dict(y=y)


def _exact_fp8_backward(s):
    if _too_long(s, 2):
        return None
    d_y = _exact_rows(s["d_y"])
    off = s["offsets"].tolist()
    d_rows = torch.zeros(s["T"] * s["k"], s["K"], dtype=torch.float64, device=d_y.device)
    d_w = torch.zeros(s["E"], s["N"], s["K"], dtype=torch.float64, device=d_y.device)
    for e in range(s["E"]):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            d_rows[lo:hi] = d_y[lo:hi] @ _dequantised(s["w"][e], s["ws"][e])
            t = s["rows"][lo:hi].long()
            d_w[e] = _exact_rows(s["d_y"][lo:hi].T) @ _exact_rows(s["x"][t].T).T
    return dict(d_rows=d_rows, d_w=d_w)


if __name__ == "__main__":
    for c in listed():
        print(c["name"], work(c))
    print(draw(random.Random(0)))
