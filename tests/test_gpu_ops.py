"""The block operators on the GPU against plain 64-bit references: norms around a block with their
backward pass, routing to many experts with its gradient, experts in 8-bit integers, the combine."""
import math

import numpy as np
import pytest

import ops_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def ops(cuda_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixture_experts_gemm_gb300 import ops
    return ops


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g).to(dtype)


def within(got, want, bound, what):
    got, want, bound = (torch.as_tensor(v, dtype=torch.float64) for v in (got, want, bound))
    assert got.shape == want.shape, what
    off = (got - want).abs()
    bad = ~(off <= bound)
    if bad.any():
        i = int((off - bound).nan_to_num(nan=math.inf).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, worst at {i}: got "
                             f"{got.flatten()[i]}, want {want.flatten()[i]} +- {bound.expand_as(want).flatten()[i]}")


# ------------------------------------------------------------------------------------------- norms
# (T, d, stream, block, params, after, before, gate, rows_per_gate)
NORMS = [
    (1, 1, F32, F32, F32, "rms", "layer", "channel", 1),
    (1, 4096, BF16, F32, BF16, "rms", "rms", "none", 1),
    (3, 7, BF16, BF16, F32, "layer", "rms", "samples", 2),
    (5, 256, BF16, BF16, BF16, "rms", "none", "channel", 5),
    (37, 1409, F32, F32, F32, "layer", "layer", "samples", 10),
    (64, 2048, BF16, F32, F32, "none", "rms", "channel", 64),
    (301, 520, F32, BF16, BF16, "rms", "layer", "samples", 1),
    (700, 64, BF16, F32, BF16, "layer", "layer", "samples", 300),
    (33, 8192, F32, F32, F32, "rms", "rms", "channel", 33),
    (9, 8200, BF16, BF16, BF16, "layer", "rms", "none", 1),
    (4, 16384, BF16, F32, F32, "rms", "layer", "samples", 3),
    (5, 16383, F32, F32, F32, "layer", "rms", "channel", 5),
    (1500, 1024, BF16, BF16, F32, "none", "none", "samples", 7),
    (2, 4100, F32, F32, BF16, "rms", "rms", "none", 1),
]
EPS = 1e-5
ALPHA, BETA = 0.9, 0.5


def norm_case(case, seed=0, backward=False):
    T, d, dt, yt, pt, after, before, gate, rpg = case
    g = gen(1000 + seed + d)
    v = dict(x=randn(g, T, d, dtype=dt) * 2 + 0.5, y=(randn(g, T, d) * 0.7 - 1.0).to(yt))
    vec = lambda on, mean: (mean + 0.2 * randn(g, d)).to(pt) if on else None  # noqa: E731
    v.update(wa=vec(after != "none", 1.0), ba=vec(after == "layer", 0.0), wb=vec(before != "none", 1.0),
             bb=vec(before == "layer", 0.1))
    v["g"] = None if gate == "none" else randn(g, 1 if gate == "channel" else -(-T // rpg), d, dtype=pt)
    if backward:
        v["dx1"] = randn(g, T, d, dtype=dt)
        v["dp"] = randn(g, T, d, dtype=dt) if before != "none" else None
    kw = dict(after=after, before=before, rows_per_gate=rpg, residual_scale=ALPHA, block_scale=BETA, eps=EPS)
    return v, kw


def cuda(v):
    return None if v is None else v.cuda()


def params(v):
    return dict(after_weight=cuda(v["wa"]), after_bias=cuda(v["ba"]), before_weight=cuda(v["wb"]),
                before_bias=cuda(v["bb"]), gate=cuda(v["g"]))


def dbl(v):
    return None if v is None else v.double()


def norm_slack(v, kind, w, b):
    """What fp32 statistics may move a norm's result by: a relative 1e-5 of the terms, the mean's rounding
    (against the deviation) among them.  Row sums of up to 16384 values in a tree of 16 + 10 additions are
    off by at most 26 * 2^-24 = 1.6e-6, the reciprocal root by 2^-22."""
    if kind == "none":
        return torch.zeros_like(v)
    n = norm_of(v, kind)
    size = 1 + n.abs() + (v.mean(1, keepdim=True).abs() / v.std(1, keepdim=True, unbiased=False).clamp(min=1e-2)
                          if kind == "layer" else 0.0)
    return 1e-5 * (size * w.abs() + (b.abs() if b is not None else 0.0))


def norm_of(v, kind):
    one = torch.ones(v.shape[1], dtype=torch.float64)
    return ref.norm(v, kind, one, None, EPS)


@pytest.mark.parametrize("case", NORMS, ids=lambda c: f"{c[0]}x{c[1]}-{c[5]}-{c[6]}-{c[7]}")
def test_block_norm(ops, case):
    T, d, dt, yt, pt, after, before, gate, rpg = case
    v, kw = norm_case(case)
    x1, p = ops.block_norm(cuda(v["x"]), cuda(v["y"]), **params(v), **kw)
    x, y = v["x"].double(), v["y"].double()
    want = ref.block(x, y, after, dbl(v["wa"]), dbl(v["ba"]), dbl(v["g"]), rpg if gate == "samples" else T, ALPHA, BETA, EPS)
    z = ref.norm(y, after, dbl(v["wa"]), dbl(v["ba"]), EPS)
    zs = norm_slack(y, after, dbl(v["wa"]), dbl(v["ba"]))
    if v["g"] is not None:
        rows = ref.gate_rows(v["g"].double(), rpg if gate == "samples" else T, T)
        z, zs = z * rows, zs * rows.abs()
    slack = BETA * zs + 2.0**-22 * ((ALPHA * x).abs() + (BETA * z).abs())
    within(x1.cpu(), want, (1 + 2.0**-8) * ref.half_step(dt) * want.abs() + 2 * slack, "x1")
    if before == "none":
        assert p is None
        return
    stored = x1.double().cpu()
    want = ref.norm(stored, before, dbl(v["wb"]), dbl(v["bb"]), EPS)
    slack = norm_slack(stored, before, dbl(v["wb"]), dbl(v["bb"]))
    within(p.cpu(), want, (1 + 2.0**-8) * ref.half_step(dt) * want.abs() + 2 * slack, "p")


def norm_reference_grads(v, kw, T):
    """64-bit gradients by torch's rules, and for every column sum the sum of its terms' magnitudes."""
    lv = {n: dbl(v[n]).requires_grad_(True) for n in ("x", "y", "wa", "ba", "wb", "bb", "g") if v[n] is not None}
    D = v["dx1"].double()
    if kw["before"] != "none":
        p = ref.norm(lv["x"], kw["before"], lv["wb"], lv.get("bb"), EPS)
        p.backward(v["dp"].double())
        D = D + lv["x"].grad
    rpg = kw["rows_per_gate"] if v["g"] is not None and v["g"].shape[0] > 1 else T
    x1 = ref.block(torch.zeros_like(D), lv["y"], kw["after"], lv.get("wa"), lv.get("ba"), lv.get("g"), rpg, ALPHA, BETA, EPS)
    x1.backward(D)
    return D, {n: t.grad for n, t in lv.items()}, rpg


@pytest.mark.parametrize("case", NORMS, ids=lambda c: f"{c[0]}x{c[1]}-{c[5]}-{c[6]}-{c[7]}")
def test_block_norm_backward(ops, case):
    """Against the 64-bit gradients.  fp32 terms are off by a few 2^-24 of the largest term of their row
    (2e-5 with the row sums), column sums by 2e-5 of the sum of their terms' magnitudes (up to about 60
    additions in a block and 40 across blocks at 2^-24 each)."""
    T, d, dt, yt, pt, after, before, gate, rpg = case
    v, kw = norm_case(case, 1, backward=True)
    out = ops.block_norm_backward(cuda(v["dx1"]), cuda(v["dp"]), cuda(v["x"]), cuda(v["y"]), **params(v), **kw)
    D, grad, rpg = norm_reference_grads(v, kw, T)
    x, y = v["x"].double(), v["y"].double()

    def deviation(t, kind):
        c = t - t.mean(1, keepdim=True) if kind == "layer" else t
        return torch.sqrt((c * c).mean(1, keepdim=True) + EPS)

    size = v["dx1"].double().abs().amax(1, keepdim=True)
    if before != "none":
        dn = (v["dp"].double() * v["wb"].double()).abs().amax(1, keepdim=True)
        size = size + dn * (2 + norm_of(x, before).abs().amax(1, keepdim=True)) / deviation(x, before)
    within(out["d_x"].cpu(), ALPHA * D, ref.half_step(dt) * 1.01 * (ALPHA * D).abs() + 2e-5 * size, "d_x")
    dz_size = BETA * size
    rows = ref.gate_rows(v["g"].double(), rpg, T) if v["g"] is not None else torch.ones(1, d, dtype=torch.float64)
    dn_size = dz_size * rows.abs().amax(1, keepdim=True)
    ysize = dn_size
    if after != "none":
        ysize = dn_size * v["wa"].double().abs().max() * (2 + norm_of(y, after).abs().amax(1, keepdim=True)) / deviation(y, after)
    within(out["d_y"].cpu(), grad["y"], ref.half_step(yt) * 1.01 * grad["y"].abs() + 2e-5 * ysize, "d_y")
    terms = {}
    if before != "none":
        terms["wb"] = (v["dp"].double() * norm_of(x, before)).abs().sum(0) + v["dp"].double().abs().sum(0)
        terms["bb"] = v["dp"].double().abs().sum(0)
    if after != "none":
        terms["wa"] = (dn_size * (1 + norm_of(y, after).abs())).sum(0)
        terms["ba"] = dn_size.sum(0).expand(d)
    for n, t in terms.items():
        if v[n] is not None:
            assert out["d_" + n].dtype == F32
            within(out["d_" + n].cpu(), grad[n], 2e-5 * t, "d_" + n)
    if v["g"] is not None:
        z = ref.norm(y, after, dbl(v["wa"]), dbl(v["ba"]), EPS).abs() + 1
        t = torch.zeros_like(grad["g"]).index_add_(0, torch.arange(T) // rpg, dz_size * z)
        within(out["d_g"].cpu(), grad["g"], 2e-5 * t, "d_g")
    assert sorted(out) == sorted(["d_x", "d_y"] + ["d_" + n for n in ("wa", "ba", "wb", "bb", "g") if v[n] is not None])


@pytest.mark.parametrize("case", [NORMS[4], NORMS[6], NORMS[8]], ids=["layer", "mixed", "rms"])
def test_block_norm_gradient_against_differences(ops, case):
    """The kernel's gradients along random directions against central differences of the 64-bit forward."""
    T, d, _, _, _, after, before, gate, rpg = case
    case = (T, d, F32, F32, F32, after, before, gate, rpg)
    v, kw = norm_case(case, 2)
    x1, _ = ops.block_norm(cuda(v["x"]), cuda(v["y"]), **params(v), **kw)
    v["dx1"], v["dp"] = randn(gen(5), T, d), randn(gen(6), T, d)
    out = {n: t.double().cpu() for n, t in ops.block_norm_backward(cuda(v["dx1"]), cuda(v["dp"]), x1, cuda(v["y"]), **params(v), **kw).items()}
    rpg = rpg if gate == "samples" else T
    names = [n for n in ("x", "y", "wa", "ba", "wb", "bb", "g") if v[n] is not None]

    def loss(p):
        x1 = ref.block(p["x"], p["y"], after, p.get("wa"), p.get("ba"), p.get("g"), rpg, ALPHA, BETA, EPS)
        return float((x1 * v["dx1"]).sum() + (ref.norm(x1, before, p["wb"], p.get("bb"), EPS) * v["dp"]).sum())

    for n in names:
        base = {m: v[m].double() for m in names}
        u = torch.randn(base[n].shape, generator=gen(7), dtype=torch.float64)
        h = 1e-5
        lo, hi = dict(base), dict(base)
        lo[n], hi[n] = base[n] - h * u, base[n] + h * u
        num = (loss(hi) - loss(lo)) / (2 * h)
        got = float((out["d_" + n] * u).sum())
        # the sum of |gradient * direction| bounds what fp32 gradients can add up to
        assert abs(got - num) <= 1e-4 * float((out["d_" + n] * u).abs().sum()) / math.sqrt(u.numel()) + 1e-4 * abs(num) + 1e-3, n


def test_block_norm_forms(ops):
    """A norm before a block alone, strided rows, in-place streams, empty batches, another stream, repeats."""
    g = gen(3)
    x = randn(g, 40, 264, dtype=BF16).cuda()
    w = (1 + 0.1 * randn(g, 256)).cuda()
    p = ops.pre_norm(x[:, 8:], w, eps=EPS)
    assert torch.equal(p, ops.pre_norm(x[:, 8:].contiguous(), w, eps=EPS))
    odd = ops.pre_norm(x[:, 3:259], w, eps=EPS)  # rows that start off 16 bytes
    want = ref.norm(x[:, 3:259].double().cpu(), "rms", w.double().cpu(), None, EPS)
    within(odd.cpu(), want, 1.01 * ref.half_step(BF16) * want.abs() + 1e-5, "odd")
    y = randn(g, 40, 256).cuda()
    b = ops.block_norm_backward(None, p, x[:, 8:].contiguous(), before="rms", before_weight=w, eps=EPS)
    assert sorted(b) == ["d_wb", "d_x"]
    for T in (0, 1, 40):
        x1, q = ops.block_norm(x[:T, :256], y[:T], after="rms", after_weight=w, before="rms", before_weight=w)
        assert x1.shape == (T, 256) and q.shape == (T, 256)
    e = ops.block_norm_backward(x[:0, :256], x[:0, :256], x[:0, :256], y[:0], after="rms", after_weight=w, before="rms", before_weight=w)
    assert e["d_x"].shape == (0, 256) and float(e["d_wa"].abs().sum()) == 0 and float(e["d_wb"].abs().sum()) == 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = ops.pre_norm(x[:, 8:], w, eps=EPS, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(again, p)
    big = randn(g, 700, 512, dtype=BF16).cuda()
    one = [ops.block_norm_backward(big, big, big, big, after="layer", after_weight=torch.ones(512, device="cuda"),
                                   before="layer", before_weight=torch.ones(512, device="cuda"),
                                   gate=torch.ones(7, 512, device="cuda"), rows_per_gate=100) for _ in range(2)]
    assert all(torch.equal(one[0][n], one[1][n]) for n in one[0])


def test_block_norm_in_place_and_specials(ops):
    import ctypes
    import mixture_experts_gemm_gb300 as moe
    g = gen(4)
    x, y = randn(g, 9, 128, dtype=BF16).cuda(), randn(g, 9, 128, dtype=BF16).cuda()
    y[2, 5], y[4, 7], x[6, 1] = math.nan, math.inf, -math.inf
    w = torch.ones(128, dtype=BF16, device="cuda")
    x1, p = ops.block_norm(x, y, after="rms", after_weight=w, before="rms", before_weight=w)
    clean = [0, 1, 3, 5, 7, 8]
    assert torch.isfinite(x1[clean].float()).all() and torch.isfinite(p[clean].float()).all()
    assert torch.isnan(p[2].float()).all() and torch.isnan(p[6, 1].float())
    # the C call may write x1 over x
    c = moe.NormConfig(128, 1, 1, 1, 1, 1, 0, 1.0, 1.0, 1e-6)
    v = moe.NormVectors(w.data_ptr(), None, w.data_ptr(), None, None)
    inplace, q = x.clone(), torch.empty_like(x)
    rc = moe.lib().colibri_moe_block_norm(ctypes.byref(c), ctypes.byref(v), inplace.data_ptr(), 128, y.data_ptr(), 128, 9,
                                          inplace.data_ptr(), q.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    assert torch.equal(inplace[clean], x1[clean]) and torch.equal(q[clean], p[clean])


# ----------------------------------------------------------------------------------------- routing
# (T, E, k, score, bias, groups, top_groups, group_top, renorm, dtype, mask, pad)
ROUTES = [
    (1, 1, 1, "softmax", False, 1, 1, 1, True, F32, 0.0, 0),
    (1, 256, 8, "sigmoid", True, 8, 4, 2, True, F32, 0.0, 0),
    (2, 8, 2, "softmax", False, 1, 1, 1, True, BF16, 0.0, 0),
    (31, 60, 4, "softmax", False, 1, 1, 1, False, BF16, 0.3, 4),
    (32, 64, 6, "softmax", True, 1, 1, 1, False, F32, 0.0, 0),
    (33, 33, 32, "sigmoid", True, 3, 3, 2, True, F32, 0.5, 1),
    (100, 96, 5, "sigmoid", False, 32, 5, 2, True, F32, 0.7, 0),
    (129, 512, 22, "softmax", True, 16, 3, 1, True, BF16, 0.0, 0),
    (257, 255, 3, "sigmoid", True, 5, 2, 1, False, F32, 0.9, 7),
    (640, 128, 8, "softmax", False, 8, 2, 2, True, F32, 0.2, 0),
    (1000, 16, 2, "sigmoid", True, 4, 2, 2, True, BF16, 0.97, 0),
    (1500, 20, 3, "softmax", False, 4, 2, 1, True, F32, 0.1, 0),
]


def route_case(case, seed=0):
    T, E, k, score, bias, groups, top_groups, group_top, renorm, dt, mask, pad = case
    g = gen(2000 + seed + E)
    wide = randn(g, T, E + pad)
    if mask:
        wide[torch.rand(T, E + pad, generator=g) < mask] = -math.inf
        wide[::17] = -math.inf
        wide[5::23, :2] = math.nan
        wide[7::29] = torch.finfo(torch.bfloat16).min
    b = 0.05 * randn(g, E) if bias else None
    if bias and mask:
        b[E // 2] = -math.inf
    kw = dict(score=score, groups=groups, top_groups=top_groups, group_top=group_top, renormalize=renorm, scale=2.5)
    return wide.to(dt), b, kw


def check_route(r, want, what=""):
    for n in ("idx", "counts", "offsets", "row_of", "token_of_row"):
        got = getattr(r, n).cpu().numpy()
        assert np.array_equal(got, want[n]), f"{what}{n}: {np.argwhere(got != want[n])[:4].tolist()}"
    # scores: exp to 2 ulp and its argument's rounding, sums of up to 512 terms, two quotients
    within(r.gate.cpu(), want["gate"], 1e-5 * np.abs(want["gate"]) + 1e-37, what + "gate")


@pytest.mark.parametrize("case", ROUTES, ids=lambda c: f"{c[0]}x{c[1]}k{c[2]}-{c[3]}-g{c[5]}")
def test_route(ops, case):
    T, E, k = case[:3]
    wide, b, kw = route_case(case)
    r = ops.route(wide.cuda()[:, :E], k, bias=cuda(b), **kw)
    want = ref.route(wide[:, :E].float().numpy(), k, kw["score"], None if b is None else b.numpy(), kw["groups"],
                     kw["top_groups"], kw["group_top"], kw["renormalize"], 2.5)
    check_route(r, want)
    again = ops.route(wide.cuda()[:, :E], k, bias=cuda(b), **kw)
    assert all(torch.equal(a, c) for a, c in zip(r, again))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top,group_top", [(1, 1, 1), (8, 3, 1), (8, 3, 2)])
def test_route_close_calls(ops, score, groups, top, group_top):
    """Keys closer than fp32 can tell apart: the ranking is that of the 64-bit keys; equal ones by index."""
    E, k, T = 64, 6, 96
    g = gen(9)
    l = randn(g, T, E)
    l[:, 32:] = l[:, :32]                               # equal logits
    l[::2, 1::2] = l[::2, ::2] * (1 + 2.0**-23)          # and neighbours one ulp away
    b = torch.zeros(E)
    b[::3] = 2.0**-25
    b[1::7] = -2.0**-26
    kw = dict(score=score, groups=groups, top_groups=top, group_top=group_top, renormalize=True, scale=1.0)
    for bias in (b, torch.zeros(E), None):
        r = ops.route(l.cuda(), k, bias=cuda(bias), **kw)
        want = ref.route(l.numpy(), k, score, None if bias is None else bias.numpy(), groups, top, group_top, True, 1.0)
        check_route(r, want, f"bias {bias is not None} ")


def test_route_peaked_and_empty(ops):
    l = torch.zeros(70, 32)
    l[:, 3] = 80.0
    l[10] = math.inf
    l[11, 5] = math.inf
    l[12] = -math.inf
    l[13] = math.nan
    want = {}
    for score in ("softmax", "sigmoid"):
        r = ops.route(l.cuda(), 2, score=score, renormalize=False)
        assert r.idx[10].tolist() == [0, 1] and r.idx[11].tolist()[0] == 5
        assert r.idx[12].tolist() == [-1, -1] and r.gate[12].tolist() == [0.0, 0.0] and r.row_of[13].tolist() == [-1, -1]
        g = r.gate[11].tolist()
        assert g[0] == 1.0 and g[1] == (0.0 if score == "softmax" else 1.0)
        assert torch.isfinite(r.gate).all()
        want[score] = r
    assert want["softmax"].gate[10].tolist() == [1 / 32, 1 / 32]
    e = ops.route(l[:0].cuda(), 2)
    assert e.idx.shape == (0, 2) and e.counts.tolist() == [0] * 32 and e.offsets.tolist() == [0] * 33
    dead = ops.route(l.cuda(), 2, bias=torch.full((32,), -math.inf, device="cuda"))
    assert (dead.idx == -1).all() and (dead.counts == 0).all() and (dead.token_of_row == -1).all()


@pytest.mark.parametrize("case", ROUTES, ids=lambda c: f"{c[0]}x{c[1]}k{c[2]}-{c[3]}-g{c[5]}")
def test_route_backward(ops, case):
    T, E, k, score, _, _, _, _, renorm, dt, mask, pad = case
    g = gen(3000 + E)
    wide = randn(g, T, E + pad).to(dt)
    l = wide[:, :E]
    idx = torch.rand(T, E, generator=g).topk(k).indices
    if mask:
        idx[torch.rand(T, k, generator=g) < 0.2] = -1
        idx[::13] = -1
    dg = randn(g, T, k)
    got = ops.route_backward(wide.cuda()[:, :E], idx.int().cuda(), dg.cuda(), score=score, renormalize=renorm, scale=2.5)
    l64 = l.double().requires_grad_(True)
    (ref.gates(l64, idx, score, renorm, 2.5) * dg.double()).sum().backward()
    # each term is a product of a score (at most 1) and gate gradients: a few 2^-24 of the row's largest
    size = 2.5 * dg.double().abs().amax(1, keepdim=True)
    within(got.cpu(), l64.grad, 1.01 * ref.half_step(dt) * l64.grad.abs() + 2e-6 * size, "d_logits")
    u = torch.randn(T, E, generator=g, dtype=torch.float64)
    f = lambda h: float((ref.gates(l.double() + h * u, idx, score, renorm, 2.5) * dg.double()).sum())  # noqa: E731
    num = (f(1e-5) - f(-1e-5)) / 2e-5
    slop = float((1.01 * ref.half_step(dt) * l64.grad.abs() * u.abs() + 2e-6 * size * u.abs()).sum())
    assert abs(float((got.double().cpu() * u).sum()) - num) <= slop + 1e-6 * abs(num) + 1e-6


def test_route_backward_masked(ops):
    """Masked experts and rows get zero; a saturated sigmoid keeps its small slope."""
    l = torch.randn(6, 8, generator=gen(1))
    l[0] = -math.inf
    l[1, 2] = -math.inf
    l[2, 3] = math.nan
    l[3, 4] = 30.0
    idx = torch.tensor([[0, 1], [2, 3], [3, 1], [4, 5], [-1, 0], [6, 7]], dtype=torch.int32)
    dg = torch.ones(6, 2)
    for score in ("softmax", "sigmoid"):
        got = ops.route_backward(l.cuda(), idx.cuda(), dg.cuda(), score=score, renormalize=False).cpu()
        assert torch.isfinite(got).all()
        assert (got[0] == 0).all() and got[1, 2] == 0 and got[2, 3] == 0
    assert abs(float(got[3, 4]) / math.exp(-30.0) - 1) < 1e-5


# ----------------------------------------------------------------------------------- 8-bit experts
# (rows of every expert, K, N, dtype, out, swiglu)
INT8 = [
    ([1], 16, 1, F32, F32, False),
    ([1, 0, 1], 256, 128, BF16, BF16, True),
    ([0, 0, 3, 0], 512, 130, BF16, F32, False),
    ([17, 1, 0, 33], 208, 65, F32, F32, True),
    ([64, 128, 0, 129, 1], 1024, 256, BF16, BF16, False),
    ([300], 2048, 96, F32, BF16, True),
    ([16, 15, 32, 31, 0, 2, 40, 7], 4096, 300, BF16, F32, False),
    ([260, 257, 5], 80, 513, BF16, F32, True),
    ([2, 1], 14336, 260, BF16, F32, False),
]


def int8_case(case, seed=0):
    counts, K, N, dt, out, swiglu = case
    g = gen(4000 + seed + K + N)
    E, R = len(counts), sum(counts)
    n = max(1, R // 2 + 3)
    x = randn(g, n, K) * torch.exp(randn(g, n, 1))
    if n > 4:
        x[3] = 0
    rows = torch.randint(0, n, (R,), generator=g).int()
    off = torch.tensor([0] + list(np.cumsum(counts))).int()
    w = [(32 * randn(g, E, N, K)).round().clamp(-127, 127).to(torch.int8) for _ in range(2 if swiglu else 1)]
    ws = [0.01 + 0.02 * torch.rand(E, N, generator=g) / math.sqrt(K) for _ in w]
    return x.to(dt), rows, off, w, ws


def check_int8(y, x, rows, off, w, ws, out):
    want, slack = ref.int8_experts(x.float().numpy(), w[0].numpy(), ws[0].numpy(), off.numpy(), rows.numpy(),
                                   *((w[1].numpy(), ws[1].numpy()) if len(w) > 1 else ()))
    live = ~np.isnan(want)
    got = y.double().cpu().numpy()
    half = ref.half_step(out) if out != F32 else 0.0
    within(got[live], want[live], (1.01 * half * np.abs(want) + 1.01 * slack + 1e-37)[live], "y")


@pytest.mark.parametrize("case", INT8, ids=lambda c: f"E{len(c[0])}R{sum(c[0])}K{c[1]}N{c[2]}{'s' if c[5] else ''}")
def test_int8_experts(ops, case):
    counts, K, N, dt, out, swiglu = case
    x, rows, off, w, ws = int8_case(case)
    kw = dict(w3=w[1].cuda(), w3_scale=ws[1].cuda()) if swiglu else {}
    y = ops.int8_experts(x.cuda(), w[0].cuda(), ws[0].cuda(), off.cuda(), rows=rows.cuda(), out_dtype=out, **kw)
    check_int8(y, x, rows, off, w, ws, out)
    again = ops.int8_experts(x.cuda(), w[0].cuda(), ws[0].cuda(), off.cuda(), rows=rows.cuda(), out_dtype=out, **kw)
    assert torch.equal(y, again)


def test_int8_largest_sums(ops):
    """All products at their largest, with one sign: sums far above 2^24."""
    K, N = 4096, 128
    x = torch.full((20, K), 3.0)
    w = torch.full((1, N, K), 127, dtype=torch.int8)
    w[0, 1::2] = -127
    ws = torch.full((1, N), 0.5)
    off, rows = torch.tensor([0, 20]).int(), torch.arange(20).int()
    y = ops.int8_experts(x.cuda(), w.cuda(), ws.cuda(), off.cuda())
    check_int8(y, x, rows, off, [w], [ws], F32)


def test_int8_forms(ops):
    """Rows outside the tokens, segments that are cut, strided inputs, rows with an infinity or NaN, no rows."""
    g = gen(8)
    x = randn(g, 12, 96)
    x[4, 7], x[5, 0] = math.inf, math.nan
    w, ws = int8_weights(g, 3, 40, 64)
    rows = torch.tensor([0, 1, -1, 12, 4, 5, 2, 3, 2, 2**31 - 1]).int()
    for off in ([0, 4, 4, 9], [0, 3, 50, 10], [-5, 2, 1, 6], [2, 5, 7, 8]):
        off = torch.tensor(off).int()
        for swiglu in (False, True):
            kw = dict(w3=w.cuda(), w3_scale=ws.cuda()) if swiglu else {}
            y = ops.int8_experts(x.cuda()[:, 16:80], w.cuda(), ws.cuda(), off.cuda(), rows=rows.cuda(), **kw).cpu()
            want, slack = ref.int8_experts(x[:, 16:80].numpy(), w.numpy(), ws.numpy(), off.numpy(), rows.numpy(),
                                           *((w.numpy(), ws.numpy()) if swiglu else ()))
            for r in range(10):
                e = [i for i in range(3) if max(int(off[i]), 0) <= r < min(max(int(off[i + 1]), max(int(off[i]), 0)), 10)]
                if not e:
                    continue
                if int(rows[r]) in (4, 5) and not torch.isfinite(x[rows[r], 16:80]).all():
                    assert torch.isnan(y[r]).all()
                elif len(e) == 1:
                    within(y[r], want[r], 1.01 * slack[r] + 1e-37, f"row {r}")
    q, s = ops.int8_quantize(x.cuda()[:, 16:80])
    wq, wsc = ref.quantize(x[:, 16:80].numpy())
    assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(s.cpu().numpy(), wsc, equal_nan=True)
    qw, sw = ops.int8_quantize(torch.randn(2, 5, 64, device="cuda", dtype=BF16))
    assert qw.shape == (2, 5, 64) and sw.shape == (2, 5)
    assert ops.int8_experts(x.cuda()[:0, :64].contiguous(), w.cuda(), ws.cuda(), torch.zeros(4, dtype=torch.int32, device="cuda")).shape == (0, 40)


@pytest.mark.parametrize("K,n,first", [(64, 3, 1), (96, 70, 3), (16400, 2, 0), (2064, 130, 5)])
def test_int8_rows_off_16_bytes(ops, K, n, first):
    """Rows that start off 16 bytes, or are wider than the quantiser's registers: read value by value."""
    g = gen(K)
    x = randn(g, n, K + first, dtype=BF16)
    w, ws = int8_weights(g, 2, 24, K)
    off = torch.tensor([0, n // 2, n]).int()
    rows = torch.randperm(n, generator=g).int()
    y = ops.int8_experts(x.cuda()[:, first:], w.cuda(), ws.cuda(), off.cuda(), rows=rows.cuda(), out_dtype=F32)
    check_int8(y, x[:, first:], rows, off, [w], [ws], F32)


def int8_weights(g, E, N, K):
    return (32 * randn(g, E, N, K)).round().clamp(-127, 127).to(torch.int8), (0.5 + torch.rand(E, N, generator=g)) / 64


@pytest.mark.parametrize("yt,ot", [(F32, F32), (BF16, F32), (F32, BF16), (BF16, BF16)])
@pytest.mark.parametrize("T,k,d", [(1, 1, 1), (5, 2, 257), (40, 8, 512), (3, 32, 4096)])
def test_combine(ops, yt, ot, T, k, d):
    g = gen(d)
    R = T * k
    y, gate = randn(g, R, d, dtype=yt), randn(g, T, k)
    row = torch.randperm(R, generator=g).view(T, k).int()
    row[torch.rand(T, k, generator=g) < 0.2] = -1
    got = ops.combine(y.cuda(), row.cuda(), gate.cuda(), out_dtype=ot)
    terms = y.double()[row.long().clamp(min=0)] * (gate.double() * (row >= 0))[:, :, None]
    want = terms.sum(1)
    within(got.cpu(), want, ref.half_step(ot) * 1.01 * want.abs() + (k + 1) * 2.0**-24 * terms.abs().sum(1), "out")


# ------------------------------------------------------------------------------- the block, together
def test_block_in_a_graph(ops):
    """norm -> route -> gated 8-bit experts -> combine -> norm, eagerly, on a side stream and as a replayed
    graph: the same bits each time; and new inputs through the captured graph."""
    g = gen(12)
    T, d, f, E, k = 50, 256, 128, 16, 4
    x = randn(g, T, d, dtype=BF16).cuda()
    wr = (randn(g, E, d) / 16).cuda()
    (w1, s1), (w3, s3), (w2, s2) = [tuple(t.cuda() for t in int8_weights(g, E, n, m)) for n, m in ((f, d), (f, d), (d, f))]
    wb = torch.ones(d, device="cuda")
    bias = (0.05 * randn(g, E)).cuda()

    def block(x):
        p = ops.pre_norm(x, wb)
        r = ops.route(p.float() @ wr.t(), k, score="sigmoid", bias=bias, groups=4, top_groups=2, group_top=2)
        h = ops.int8_experts(p, w1, s1, r.offsets, rows=r.token_of_row, w3=w3, w3_scale=s3)
        y = ops.combine(ops.int8_experts(h, w2, s2, r.offsets), r.row_of, r.gate, out_dtype=F32)
        return ops.block_norm(x, y, after="rms", after_weight=wb, before="rms", before_weight=wb)

    eager = block(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(x)
    torch.cuda.current_stream().wait_stream(side)
    static = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block(static)
    for seed in (0, 1):
        new = x if seed == 0 else randn(gen(77), T, d, dtype=BF16).cuda()
        static.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        want = eager if seed == 0 else block(new)
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
