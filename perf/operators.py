"""The layer-block operators in their plain form, and the cases they are measured at.

A Mixture-of-Experts block around the expert layer: norms before and after the block with its gate
and residual scale, routing to many experts with the dispatch order, and the experts' products in
8-bit integers.  Where `own` is true `run` calls the package's kernels, otherwise elementary torch
operations compute the same thing.  Sizes come from the layer shapes this repository is measured on
(hidden 256, 2048 and 4096, inner 512, 1408, 5632 and 14336, 8192 tokens of prefill, 1 to 32 of
decode) and, for layers of many experts, 60, 64 and 256 experts.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


# ------------------------------------------------------------------------------------------ cases
def _route(name, T, E, k, score, bias, groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0, dtype="f32",
           masked=False, pad=0, backward=False):
    c = dict(op="route_backward" if backward else "route", T=T, E=E, k=k, score=score, bias=bias, groups=groups,
             top_groups=top_groups, group_top=group_top, renorm=renorm, scale=scale, dtype=dtype, masked=masked, pad=pad)
    return dict(c, name=name) if name else c


def _norm(name, T, d, dtype, y_dtype, after, before, gate, per_gate, params, alpha=1.0, beta=1.0, backward=False):
    c = dict(op="norm_backward" if backward else "norm", T=T, d=d, dtype=dtype, y_dtype=y_dtype, after=after,
             before=before, gate=gate, per_gate=per_gate, params=params, alpha=alpha, beta=beta)
    return dict(c, name=name) if name else c


def _int8(name, T, k, E, K, N, swiglu, dtype, out, skew):
    c = dict(op="int8", T=T, k=k, E=E, K=K, N=N, swiglu=swiglu, dtype=dtype, out=out, skew=skew)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decoded token of a layer with 256 grouped experts, balanced by a bias: a call's latency
        _route("route-token", 1, 256, 8, "sigmoid", True, 8, 4, 2, scale=2.5),
        # a prefill batch of the same layer
        _route("route-prefill", 8192, 256, 8, "sigmoid", True, 8, 4, 2, scale=2.5),
        # an odd batch of a layer with 60 experts whose logits are a slice of a wider product; some
        # experts are masked off, some tokens (padding) have none left
        _route("route-odd-masked", 4099, 60, 4, "softmax", False, renorm=False, dtype="bf16", masked=True, pad=4),
        # the router's gradient in a training step
        _route("route-backward", 8192, 64, 6, "softmax", False, renorm=False, backward=True),
        # decode: four tokens between two blocks
        _norm("norm-decode", 4, 4096, "bf16", "f32", "rms", "rms", "none", 1, "bf16"),
        # prefill: the layer's fp32 output normed, added to the stream, and the next block's norm
        _norm("norm-prefill", 8192, 4096, "bf16", "f32", "rms", "rms", "channel", 8192, "bf16", alpha=0.9, beta=0.5),
        # modulated blocks: a gate row for each sample of 1000 tokens, layer norms, an odd width
        _norm("norm-samples-odd", 3001, 1409, "f32", "f32", "layer", "layer", "samples", 1000, "f32"),
        # the training step's backward pass
        _norm("norm-backward", 8192, 4096, "bf16", "bf16", "rms", "rms", "channel", 8192, "f32", alpha=0.9, beta=0.5,
              backward=True),
        # one decoded token, two experts of the large layer: the weights' bytes
        _int8("int8-token", 1, 2, 8, 4096, 14336, True, "bf16", "bf16", 0.0),
        # a batch of 512 tokens, the middle layer's up projections
        _int8("int8-batch", 512, 2, 8, 2048, 5632, True, "bf16", "bf16", 0.0),
        # a batch over 64 small experts, unevenly loaded, an odd number of channels and tokens
        _int8("int8-many-experts", 1021, 6, 64, 2048, 1409, False, "f32", "f32", 1.0),
        # prefill: 8192 tokens, the large layer's down projection
        _int8("int8-prefill", 8192, 2, 8, 14336, 4096, False, "bf16", "f32", 0.3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "route_backward", "norm", "norm", "norm_backward", "int8", "int8", "int8"])
    if op in ("route", "route_backward"):
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * rng.randint(max(1, 8 // groups), 256 // groups)
        top_groups = rng.randint(1, groups)
        k = rng.randint(1, min(10, top_groups * (E // groups)))
        score = rng.choice(["softmax", "sigmoid"])
        return _route(None, _log(rng, 1, 16384), E, k, score, rng.random() < 0.5, groups, top_groups,
                      rng.choice([1, 2]) if E // groups > 1 else 1, rng.random() < 0.6, rng.choice([1.0, 2.5]),
                      rng.choice(["f32", "bf16"]), rng.random() < 0.3, rng.choice([0, 0, 3, 8]), op == "route_backward")
    if op in ("norm", "norm_backward"):
        d = _log(rng, 64, 8192)
        if rng.random() < 0.6:
            d = (d + 7) // 8 * 8
        T = _log(rng, 1, min(16384, 8192 * 4096 // d))
        after = rng.choice(["none", "rms", "layer"])
        before = rng.choice(["none", "rms", "layer"])
        gate = rng.choice(["none", "channel", "samples"])
        dtype = rng.choice(["f32", "bf16"])
        return _norm(None, T, d, dtype, "f32" if dtype == "f32" else rng.choice(["f32", "bf16"]), after, before, gate,
                     rng.randint(max(1, T // 9), T) if gate == "samples" else T, rng.choice(["f32", "bf16"]),
                     rng.choice([1.0, 0.9]), rng.choice([1.0, 0.5]), op == "norm_backward")
    K = (_log(rng, 64, 14336) + 15) // 16 * 16
    N = _log(rng, 64, 14336)
    E = rng.choice([1, 4, 8, 16, 60, 64])
    swiglu = rng.random() < 0.5
    while E * N * K * (2 if swiglu else 1) > 8 * 14336 * 4096:
        N = (N + 1) // 2
    k = rng.randint(1, min(E, 6))
    T = _log(rng, 1, 8192)
    while T > 1 and T * k * N * K * (2 if swiglu else 1) > 16384 * 14336 * 4096 // 2:
        T //= 2
    return _int8(None, T, k, E, K, N, swiglu, rng.choice(["f32", "bf16"]), rng.choice(["f32", "bf16"]),
                 rng.choice([0.0, 0.3, 1.0]))


# ----------------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    s = dict(case)
    if case["op"] in ("route", "route_backward"):
        T, E, k = case["T"], case["E"], case["k"]
        logits = rn(T, E + case["pad"])
        if case["masked"]:
            logits[torch.rand(T, E + case["pad"], generator=g, device="cuda") < 0.05] = -math.inf
            logits[96::97] = -math.inf
        s["logits"] = logits.to(DTYPES[case["dtype"]])[:, :E]
        s["b"] = 0.05 * rn(E) if case["bias"] else None
        if case["op"] == "route_backward":
            # the selection a forward pass kept: distinct experts, none of them a masked one
            free = torch.rand(T, E, generator=g, device="cuda").masked_fill(torch.isneginf(s["logits"]), -1.0)
            v, i = free.topk(k)
            s["idx"] = torch.where(v >= 0, i, -1).to(torch.int32)
            s["d_gate"] = rn(T, k)
    elif case["op"] in ("norm", "norm_backward"):
        T, d = case["T"], case["d"]
        dt, pt = DTYPES[case["dtype"]], DTYPES[case["params"]]
        n_gates = {"none": 0, "channel": 1, "samples": -(-T // case["per_gate"])}[case["gate"]]
        s["x"] = (2 * rn(T, d)).to(dt)
        s["y"] = (0.7 * rn(T, d)).to(DTYPES[case["y_dtype"]])
        one = lambda on, mean: (mean + 0.1 * rn(d)).to(pt) if on else None  # noqa: E731
        s["wa"], s["ba"] = one(case["after"] != "none", 1.0), one(case["after"] == "layer", 0.0)
        s["wb"], s["bb"] = one(case["before"] != "none", 1.0), one(case["before"] == "layer", 0.0)
        s["g"] = (0.5 * rn(n_gates, d)).to(pt) if n_gates else None
        if case["op"] == "norm_backward":
            s["d_x1"] = rn(T, d).to(dt)
            s["d_p"] = rn(T, d).to(dt) if case["before"] != "none" else None
    else:
        T, k, E, K, N = (case[n] for n in ("T", "k", "E", "K", "N"))
        s["x"] = rn(T, K).to(DTYPES[case["dtype"]])
        # the dispatch that routing left: every token in k distinct experts, an uneven load if `skew`
        noise = -torch.log(-torch.log(torch.rand(T, E, generator=g, device="cuda").clamp(1e-6, 1 - 1e-6)))
        load = -case["skew"] * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
        idx = (noise + load).topk(k).indices
        rows = torch.argsort(idx.reshape(-1), stable=True)
        s["rows"] = (rows // k).to(torch.int32)
        counts = torch.bincount(idx.reshape(-1), minlength=E)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        # the same rows as a rectangle of experts x the fullest expert's rows, for batched products
        expert = torch.repeat_interleave(torch.arange(E, device="cuda"), counts)
        s["at"] = expert * int(counts.max()) + torch.arange(T * k, device="cuda") - s["offsets"].long()[expert]
        s["cap"] = int(counts.max())
        s["w"], s["ws"] = _weights(E, N, K, g)
        s["w3"], s["w3s"] = _weights(E, N, K, g) if case["swiglu"] else (None, None)
    return s


def _weights(E, N, K, g):
    """Normal weights of variance 1 / K as 8-bit integers with a scale for each output channel."""
    w = torch.empty(E, N, K, dtype=torch.int8, device="cuda")
    for e in range(E):
        w[e] = torch.randn(N, K, generator=g, device="cuda").mul_(32).round_().clamp_(-127, 127)
    return w, (0.8 + 0.4 * torch.rand(E, N, generator=g, device="cuda")) / (32 * math.sqrt(K))


# ------------------------------------------------------------------------------------ plain forms
def _scores(logits, score):
    """Scores in 64 bits and which experts are admissible (a finite or infinite logit above -inf)."""
    l = logits.double()
    ok = l > -math.inf
    if score == "sigmoid":
        return l, torch.where(ok, 1 / (1 + torch.exp(-l)), 0.0), ok
    m = l.masked_fill(~ok, -math.inf).amax(1, keepdim=True)
    z = torch.where(ok, torch.exp(l - torch.where(torch.isneginf(m), 0.0, m)), 0.0)
    return l, z / z.sum(1, keepdim=True).clamp(min=1e-300), ok


def _plain_route(s):
    T, E, k, G = s["T"], s["E"], s["k"], s["groups"]
    l, p, ok = _scores(s["logits"], s["score"])
    biased = p + s["b"].double() if s["b"] is not None else p
    key = (biased if s["b"] is not None else l).masked_fill(~ok, -math.inf)
    if G > 1:
        per = biased.masked_fill(~ok, -math.inf).view(T, G, E // G)
        if s["group_top"] == 1 and s["b"] is None:
            rank = key.view(T, G, E // G).amax(2)
        else:
            top = per.topk(s["group_top"], dim=2).values
            rank = torch.where(torch.isneginf(top[:, :, 0]), -math.inf, top.masked_fill(torch.isneginf(top), 0.0).sum(2))
        first = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
        kept = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, first, True)
        key = key.masked_fill(~kept.repeat_interleave(E // G, 1), -math.inf)
    v, i = torch.sort(key, dim=1, descending=True, stable=True)
    none = torch.isneginf(v[:, :k])
    idx = i[:, :k].masked_fill(none, -1)
    gate = p.gather(1, i[:, :k]).masked_fill(none, 0.0)
    if s["renorm"]:
        gate = gate / gate.sum(1, keepdim=True).clamp(min=1e-300)
    flat = idx.reshape(-1)
    flat = torch.where(flat < 0, E, flat)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=l.device).scatter_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat([counts.new_zeros(1), counts[:E].cumsum(0)])
    order = torch.argsort(flat, stable=True)
    place = torch.arange(T * k, device=l.device)
    row_of = torch.empty_like(flat).scatter_(0, order, place)
    row_of = torch.where(flat < E, row_of, -1).view(T, k)
    token = torch.where(place < offsets[E], order // k, -1)
    i32 = torch.int32
    return dict(idx=idx.to(i32), gate=(gate * s["scale"]).float(), counts=counts[:E].to(i32), offsets=offsets.to(i32),
                row_of=row_of.to(i32), token_of_row=token.to(i32))


def _plain_route_backward(s):
    _, p, _ = _scores(s["logits"], s["score"])
    sel = s["idx"] >= 0
    at = s["idx"].long().clamp(min=0)
    ps = torch.where(sel, p.gather(1, at), 0.0)
    dg = torch.where(sel, s["d_gate"].double(), 0.0) * s["scale"]
    if s["renorm"]:
        total = ps.sum(1, keepdim=True).clamp(min=1e-300)
        dg = torch.where(sel, (dg - (dg * ps).sum(1, keepdim=True) / total) / total, 0.0)
    dp = torch.zeros_like(p).scatter_add_(1, at, dg)
    if s["score"] == "sigmoid":
        dl = dp * p * (1 - p)
    else:
        dl = p * (dp - (dp * p).sum(1, keepdim=True))
    return dict(d_logits=dl.to(s["logits"].dtype))


def _normed(v, kind):
    """v normed along its rows, and 1 / its deviation."""
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    r = torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)
    return v * r, r


def _gate(s, T):
    """The gate of every token, or None."""
    if s["g"] is None:
        return None
    return s["g"].float()[torch.arange(T, device=s["g"].device) // s["per_gate"]] if s["g"].shape[0] > 1 else s["g"].float()


def _affine(v, w, b):
    v = v * w.float()
    return v + b.float() if b is not None else v


def _plain_norm(s):
    z = s["y"].float()
    if s["after"] != "none":
        z = _affine(_normed(z, s["after"])[0], s["wa"], s["ba"])
    gate = _gate(s, s["T"])
    if gate is not None:
        z = gate * z
    x1 = (s["alpha"] * s["x"].float() + s["beta"] * z).to(s["x"].dtype)
    out = dict(x1=x1)
    if s["before"] != "none":
        out["p"] = _affine(_normed(x1.float(), s["before"])[0], s["wb"], s["bb"]).to(s["x"].dtype)
    return out


def _norm_grad(d_n, n, r, kind):
    """The gradient of a norm's input from that of its result n = (v - mean) * r."""
    t = d_n - n * (d_n * n).mean(1, keepdim=True)
    if kind == "layer":
        t = t - d_n.mean(1, keepdim=True)
    return t * r


def _plain_norm_backward(s):
    out = {}
    D = s["d_x1"].float()
    if s["before"] != "none":
        n, r = _normed(s["x"].float(), s["before"])
        d_p = s["d_p"].float()
        out["d_wb"] = (d_p * n).sum(0)
        if s["bb"] is not None:
            out["d_bb"] = d_p.sum(0)
        D = D + _norm_grad(d_p * s["wb"].float(), n, r, s["before"])
    out["d_x"] = (s["alpha"] * D).to(s["x"].dtype)
    z = s["y"].float()
    if s["after"] != "none":
        ny, ry = _normed(z, s["after"])
        z = _affine(ny, s["wa"], s["ba"])
    d_z = s["beta"] * D
    gate = _gate(s, s["T"])
    if gate is not None:
        n_gates = s["g"].shape[0]
        if n_gates == 1:
            out["d_g"] = (d_z * z).sum(0, keepdim=True)
        else:
            sample = torch.arange(s["T"], device=z.device) // s["per_gate"]
            out["d_g"] = torch.zeros(n_gates, s["d"], device=z.device).index_add_(0, sample, d_z * z)
        d_z = d_z * gate
    if s["after"] != "none":
        out["d_wa"] = (d_z * ny).sum(0)
        if s["ba"] is not None:
            out["d_ba"] = d_z.sum(0)
        d_z = _norm_grad(d_z * s["wa"].float(), ny, ry, s["after"])
    out["d_y"] = d_z.to(s["y"].dtype)
    return out


def _plain_int8(s):
    x = s["x"].float()
    # two tensors, so that the quotient is rounded once (by a number, it is a product with 1 / 127)
    scale = x.abs().amax(1, keepdim=True) / torch.full((1, 1), 127.0, device=x.device)
    q = torch.where(scale > 0, torch.round(x / scale).clamp(-127, 127), 0.0)
    E, cap, K = s["E"], s["cap"], s["K"]
    rows = s["rows"].long()
    a = torch.zeros(E * cap, K, device=x.device).index_copy_(0, s["at"], q[rows]).view(E, cap, K)
    sa = scale[rows]

    def product(w, ws):
        y = torch.bmm(a, w.float().transpose(1, 2)) * ws[:, None, :]
        return y.view(E * cap, -1)[s["at"]] * sa

    y = product(s["w"], s["ws"])
    if s["swiglu"]:
        y = y / (1 + torch.exp(-y)) * product(s["w3"], s["w3s"])
    return dict(y=y.to(DTYPES[s["out"]]))


# -------------------------------------------------------------------------------------------- run
def run(s):
    op = s["op"]
    if not own:
        return {"route": _plain_route, "route_backward": _plain_route_backward, "norm": _plain_norm,
                "norm_backward": _plain_norm_backward, "int8": _plain_int8}[op](s)
    from mixture_experts_gemm_gb300 import ops
    if op == "route":
        r = ops.route(s["logits"], s["k"], score=s["score"], bias=s["b"], groups=s["groups"],
                      top_groups=s["top_groups"], group_top=s["group_top"], renormalize=s["renorm"], scale=s["scale"])
        return r._asdict()
    if op == "route_backward":
        return dict(d_logits=ops.route_backward(s["logits"], s["idx"], s["d_gate"], score=s["score"],
                                                renormalize=s["renorm"], scale=s["scale"]))
    norms = dict(after=s.get("after"), after_weight=s.get("wa"), after_bias=s.get("ba"), before=s.get("before"),
                 before_weight=s.get("wb"), before_bias=s.get("bb"), gate=s.get("g"), rows_per_gate=s.get("per_gate"),
                 residual_scale=s.get("alpha"), block_scale=s.get("beta"), eps=EPS)
    if op == "norm":
        x1, p = ops.block_norm(s["x"], s["y"], **norms)
        return dict(x1=x1, p=p) if p is not None else dict(x1=x1)
    if op == "norm_backward":
        return ops.block_norm_backward(s["d_x1"], s["d_p"], s["x"], s["y"], **norms)
    return dict(y=ops.int8_experts(s["x"], s["w"], s["ws"], s["offsets"], rows=s["rows"], w3=s["w3"],
                                   w3_scale=s["w3s"], out_dtype=DTYPES[s["out"]]))


# ------------------------------------------------------------------------------------------- work
def work(case):
    size = {"f32": 4, "bf16": 2}
    c = case
    if c["op"] == "route":
        # logits read; idx, gate, row_of, token_of_row, counts and offsets written
        return dict(bytes=c["T"] * (c["E"] * size[c["dtype"]] + 16 * c["k"]) + (12 if c["bias"] else 8) * c["E"],
                    flops=4 * c["T"] * c["E"])
    if c["op"] == "route_backward":
        return dict(bytes=c["T"] * (2 * c["E"] * size[c["dtype"]] + 8 * c["k"]), flops=6 * c["T"] * c["E"])
    if c["op"] in ("norm", "norm_backward"):
        n, s, sy, p = c["T"] * c["d"], size[c["dtype"]], size[c["y_dtype"]], size[c["params"]]
        vectors = {"none": 0, "rms": 1, "layer": 2}
        n_gates = {"none": 0, "channel": 1, "samples": -(-c["T"] // c["per_gate"])}[c["gate"]]
        v = vectors[c["after"]] + vectors[c["before"]]
        nb = c["before"] != "none"
        if c["op"] == "norm":
            return dict(bytes=n * (2 * s + sy + (s if nb else 0)) + (v + n_gates) * c["d"] * p, flops=14 * n)
        # d_x1, d_p, x and y read, d_x and d_y written; the stream itself is not needed without a next norm
        return dict(bytes=n * (2 * s + (2 * s if nb else 0) + 2 * sy) + (v + n_gates) * c["d"] * (p + 4), flops=30 * n)
    R = c["T"] * c["k"]
    m = 2 if c["swiglu"] else 1
    used = min(c["E"], R) if c["T"] > 1 else min(c["E"], c["k"])
    return dict(bytes=m * used * c["N"] * (c["K"] + 4) + c["T"] * c["K"] * size[c["dtype"]] + R * c["N"] * size[c["out"]],
                flops=2 * m * R * c["N"] * c["K"])


# ------------------------------------------------------------------------------------------ exact
def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "route_backward": _exact_route_backward, "norm": _exact_norm,
            "norm_backward": _exact_norm_backward, "int8": _exact_int8}[s["op"]](s)


def _exact_route(s):
    """Gates from the definition; the whole numbers are compared with the plain form's for equality."""
    l = s["logits"].double()
    p = torch.sigmoid(l) if s["score"] == "sigmoid" else torch.nan_to_num(torch.softmax(l, 1), nan=0.0)
    dead = torch.isneginf(l)
    select = torch.where(dead, -math.inf, p + (0.0 if s["b"] is None else s["b"].double()))
    if s["groups"] > 1:
        by = select.view(s["T"], s["groups"], -1)
        best = by.sort(2, descending=True).values[:, :, :s["group_top"]]
        worth = best.clamp(min=-1e300).where(best > -math.inf, torch.zeros_like(best)).sum(2)
        worth = worth.masked_fill((best == -math.inf).all(2), -math.inf)
        # equal groups: the lower index first, as a stable order leaves it
        order = worth.argsort(dim=1, descending=True, stable=True).argsort(dim=1)
        select = by.masked_fill((order >= s["top_groups"])[:, :, None], -math.inf).reshape(s["T"], -1)
    best, at = select.topk(s["k"], dim=1)
    gate = p.gather(1, at) * (best > -math.inf)
    if s["renorm"]:
        gate = torch.nan_to_num(gate / gate.sum(1, keepdim=True), nan=0.0)
    return dict(gate=gate * s["scale"])


def _exact_route_backward(s):
    """Differentiates the gates by torch's own rules in 64 bits."""
    dead = torch.isneginf(s["logits"])
    l = s["logits"].double().masked_fill(dead, -1e4).requires_grad_(True)
    with torch.enable_grad():
        p = torch.sigmoid(l) if s["score"] == "sigmoid" else torch.softmax(l, 1)
        kept = s["idx"] >= 0
        gate = p.gather(1, s["idx"].long().clamp(min=0)) * kept
        if s["renorm"]:
            gate = gate / (gate.sum(1, keepdim=True) + (~kept).all(1, keepdim=True))
        (gate * s["d_gate"].double() * kept).sum().mul(s["scale"]).backward()
    return dict(d_logits=l.grad.masked_fill(dead, 0.0))


def _forward64(s, x, y, wa, ba, wb, bb, g):
    def norm(v, kind, w, b):
        if kind == "rms":
            return v / (v.square().mean(1, keepdim=True) + EPS).sqrt() * w
        c = v - v.mean(1, keepdim=True)
        return c / (c.square().mean(1, keepdim=True) + EPS).sqrt() * w + b

    z = y if s["after"] == "none" else norm(y, s["after"], wa, ba)
    if g is not None:
        z = z * torch.repeat_interleave(g, s["per_gate"], 0)[:s["T"]]
    x1 = s["alpha"] * x + s["beta"] * z
    if s["before"] == "none":
        return x1, None
    stored = x1.detach().to(s["x"].dtype).double() if not x1.requires_grad else x1
    return x1, norm(stored, s["before"], wb, bb)


def _doubles(s):
    return [None if s[n] is None else s[n].double() for n in ("y", "wa", "ba", "wb", "bb", "g")]


def _exact_norm(s):
    x1, p = _forward64(s, s["x"].double(), *_doubles(s))
    return dict(x1=x1) if p is None else dict(x1=x1, p=p)


def _exact_norm_backward(s):
    """Differentiates the two steps by torch's own rules in 64 bits: the next norm at the stored stream,
    then the block's side, linear in the stream's gradient."""
    y, wa, ba, wb, bb, g = (None if v is None else v.requires_grad_(True) for v in _doubles(s))
    x = s["x"].double().requires_grad_(True)
    out = {}
    with torch.enable_grad():
        if s["before"] == "none":
            D = s["d_x1"].double()
        else:
            after = dict(s, after="none", alpha=1.0, beta=0.0)
            _, p = _forward64(after, x, torch.zeros_like(x), None, None, wb, bb, None)
            (p * s["d_p"].double()).sum().backward()
            D = s["d_x1"].double() + x.grad
        x1, _ = _forward64(dict(s, before="none"), x.detach(), y, wa, ba, None, None, g)
        (x1 * D).sum().backward()
    out["d_x"], out["d_y"] = s["alpha"] * D, y.grad
    for name, v in (("d_wa", wa), ("d_ba", ba), ("d_wb", wb), ("d_bb", bb), ("d_g", g)):
        if v is not None:
            out[name] = v.grad
    return out


def _exact_int8(s):
    """Whole-number products summed exactly, expert by expert; a row's scale and quotients are rounded to
    32 bits, as the format says."""
    if 2 * s["T"] * s["k"] * s["N"] * s["K"] * (2 if s["swiglu"] else 1) > 6e12:
        return None
    x = s["x"].to(torch.float32)
    top = x.abs().max(1).values
    scale = torch.div(top, torch.full_like(top, 127.0))
    q = torch.div(x, scale.clamp(min=1e-45)[:, None]).round().clamp(-127, 127).double() * (scale > 0)[:, None]
    off = s["offsets"].tolist()
    y = torch.zeros(s["T"] * s["k"], s["N"], dtype=torch.float64, device=x.device)
    for e in range(s["E"]):
        at = slice(off[e], off[e + 1])
        if off[e + 1] > off[e]:
            t = s["rows"][at].long()
            v = q[t] @ s["w"][e].double().T * s["ws"][e].double() * scale[t].double()[:, None]
            if s["swiglu"]:
                v = v * torch.sigmoid(v) * (q[t] @ s["w3"][e].double().T * s["w3s"][e].double() * scale[t].double()[:, None])
            y[at] = v
    return dict(y=y)


if __name__ == "__main__":
    for c in listed():
        print(c["name"], work(c))
    print(draw(random.Random(0)))
