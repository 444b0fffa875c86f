"""The operators around the forward on the GPU, against plain 64-bit implementations.

Tolerances count roundings: a rounding to type t is off by at most finfo(t).eps / 2
relative to the value (BF16 2^-8, FP32 2^-24, E4M3 2^-4).
"""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle as orc

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(scope="module")
def nvm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import nvfp4_weight_quantized_moe_b200 as nvm
    return nvm


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _guarded(rows, cols, dtype, fill):
    """[rows, cols] inside a larger buffer whose rest must stay as it is."""
    pad = 64
    flat = torch.full((rows * cols + 2 * pad,), fill, device="cuda").to(dtype)
    view = flat[pad:pad + rows * cols].view(rows, cols)

    def check():
        want = torch.full((pad,), fill, device="cuda").to(dtype)
        assert torch.equal(flat[:pad], want) and torch.equal(flat[-pad:], want)
    return view, check


# --------------------------------------------------------------------------- #
# Routing
# --------------------------------------------------------------------------- #
def _route_ref(logits, bias, topk, score, groups, keep, top, renorm, scale):
    """ids and weights row by row in numpy float64, ties to the lower index."""
    l = logits.float().cpu().numpy().astype(np.float64)
    m, e = l.shape
    b = None if bias is None else bias.cpu().numpy().astype(np.float64)
    ids = np.full((m, topk), -1, np.int64)
    w = np.zeros((m, topk))
    big = float(np.finfo(np.float32).max)
    for t in range(m):
        x = np.where(np.isnan(l[t]), -np.inf, np.minimum(l[t], big))
        can = x > -np.inf
        if not can.any():
            continue
        with np.errstate(over="ignore", invalid="ignore"):
            if score == "softmax":
                p = np.exp(x - x.max())
                p = p / p.sum()
            else:
                p = 1.0 / (1.0 + np.exp(-x))
        c = x.copy() if b is None else p + b
        c[np.isnan(c)] = -np.inf
        can &= c > -np.inf
        if groups > 1:
            size = e // groups
            v = p if b is None and top > 1 else c
            best = []
            for g in range(groups):
                inside = np.sort(v[g * size:(g + 1) * size][can[g * size:(g + 1) * size]])[::-1]
                best.append(inside[:top].sum() if inside.size else -np.inf)
            order = sorted((g for g in range(groups) if best[g] > -np.inf), key=lambda g: (-best[g], g))
            for g in set(range(groups)) - set(order[:keep]):
                can[g * size:(g + 1) * size] = False
        order = sorted(np.nonzero(can)[0], key=lambda i: (-c[i], i))[:topk]
        ids[t, :len(order)] = order
        sel = x[order]
        if len(order) == 0:
            continue
        if renorm:
            if score == "softmax":
                u = np.exp(sel - sel.max())
            else:
                # Scores relative to e^base: ratios stay when the scores underflow.
                base = min(0.0, sel.max())
                low = np.minimum(sel, 0.0)
                u = np.where(sel > 0, 1.0 / (1.0 + np.exp(-np.abs(sel))), np.exp(low - base) / (1.0 + np.exp(low)))
            u = u / u.sum()
        else:
            u = p[order]
        w[t, :len(order)] = u * scale
    return ids, w


def _check_route(nvm, logits, topk, bias=None, score="softmax", groups=1, keep=1, top=1, renorm=True,
                 scale=1.0):
    m = logits.shape[0]
    ids, ids_ok = _guarded(m, topk, torch.int32, -7)
    w, w_ok = _guarded(m, topk, F32, -7.0)
    nvm.route_topk(logits, ids, w, score=score, bias=bias, num_groups=groups, topk_groups=keep,
                   group_top=top, renormalize=renorm, scale=scale)
    torch.cuda.synchronize()
    ids_ok(), w_ok()
    want_ids, want_w = _route_ref(logits, bias, topk, score, groups, keep, top, renorm, scale)
    np.testing.assert_array_equal(ids.cpu().numpy(), want_ids)
    got = w.cpu().numpy().astype(np.float64)
    # exp of a difference: the difference is rounded (2^-24 of up to 2^7 here), exp,
    # quotient and scale a few 2^-24, a sum of at most 64 roundings.  Below the
    # smallest normal FP32 number there is no relative accuracy.
    assert np.all(np.abs(got - want_w) <= 2.0 ** -16 * np.abs(want_w) + 2.0 ** -126), \
        np.abs(got - want_w).max()


@pytest.mark.parametrize("e,topk", [(1, 1), (2, 2), (8, 2), (31, 5), (33, 32), (128, 8), (129, 7), (256, 8),
                                    (500, 3), (1000, 10), (1024, 32)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_route_matches_the_definition(nvm, e, topk, score, dtype):
    g = _gen(e * 64 + topk)
    logits = (torch.randn(37, e, generator=g, device="cuda") * 2).to(dtype)
    _check_route(nvm, logits, topk, score=score, renorm=True, scale=2.5)
    _check_route(nvm, logits, topk, score=score, renorm=False)
    bias = torch.randn(e, generator=g, device="cuda") * 0.1
    _check_route(nvm, logits, topk, bias=bias, score=score)


@pytest.mark.parametrize("m", [1, 2, 7, 8, 9, 592, 593, 1500])
def test_route_batch_sizes(nvm, m):
    g = _gen(m)
    logits = torch.randn(m, 128, generator=g, device="cuda")
    _check_route(nvm, logits, 8, bias=torch.randn(128, generator=g, device="cuda") * 0.05, score="sigmoid")
    _check_route(nvm, logits.to(BF16), 8)


@pytest.mark.parametrize("e,groups,keep", [(8, 2, 1), (256, 8, 4), (256, 8, 8), (60, 4, 3), (96, 32, 5), (1024, 32, 7),
                                           (12, 3, 2), (32, 32, 9), (250, 5, 2)])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_groups(nvm, e, groups, keep, top, biased, score):
    if top > e // groups:
        pytest.skip("a group of one expert has no two best")
    g = _gen(e + 7 * groups + keep)
    logits = torch.randn(64, e, generator=g, device="cuda") * 2
    bias = torch.randn(e, generator=g, device="cuda") * 0.2 if biased else None
    topk = min(8, keep * (e // groups), 32)
    _check_route(nvm, logits, topk, bias=bias, score=score, groups=groups, keep=keep, top=top)
    _check_route(nvm, logits.to(BF16), topk, bias=bias, score=score, groups=groups, keep=keep, top=top,
                 renorm=False, scale=0.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", ["none", "zero", "steps"])
@pytest.mark.parametrize("groups,keep,top", [(1, 1, 1), (8, 3, 1), (8, 3, 2)])
def test_route_ties_go_to_the_lower_index(nvm, score, bias, groups, keep, top):
    """Logits from a few values: most choices are ties, +0 and -0 among them."""
    g = _gen(11)
    logits = torch.randint(-2, 3, (200, 128), generator=g, device="cuda").float() * 0.5
    logits = torch.where(logits == 0, torch.where(torch.rand(200, 128, generator=g, device="cuda") < 0.5, -0.0, 0.0),
                         logits)
    b = {"none": None, "zero": torch.zeros(128, device="cuda"),
         "steps": torch.randint(0, 2, (128,), generator=g, device="cuda").float() * 0.25}[bias]
    _check_route(nvm, logits, 8, bias=b, score=score, groups=groups, keep=keep, top=top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_orders_values_that_fp32_cannot(nvm, score):
    """Neighbouring logits whose scores (plus bias) round to the same FP32 value, in
    descending, ascending and mixed order of their index."""
    base = torch.tensor([3.0, 5.0, 2.0, 7.0], device="cuda")
    steps = torch.arange(32, device="cuda").float()
    ulp = 2.0 ** -21  # of values in [4, 8); larger than an FP32 step of the rest
    rows = [base[:, None] + steps * ulp, base[:, None] - steps * ulp,
            base[:, None] + ((steps * 11) % 32) * ulp]
    logits = torch.cat([r.expand(4, 32) for r in rows]).contiguous()
    for bias in (torch.zeros(32, device="cuda"), torch.full((32,), 0.75, device="cuda"),
                 torch.full((32,), -40.0, device="cuda")):
        _check_route(nvm, logits, 8, bias=bias, score=score)
        _check_route(nvm, logits, 4, bias=bias, score=score, groups=4, keep=2, top=2)
    _check_route(nvm, logits, 8, score=score, groups=4, keep=2, top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups,keep,top", [(1, 1, 1), (4, 2, 1), (4, 2, 2)])
def test_route_masked_and_odd_values(nvm, score, biased, groups, keep, top):
    g = _gen(5)
    logits = torch.randn(24, 64, generator=g, device="cuda") * 3
    inf = float("inf")
    logits[0] = -inf                         # nothing to choose: a padding token
    logits[1, 3:] = -inf                     # fewer experts than slots
    logits[2, ::2] = float("nan")
    logits[3, 5] = inf
    logits[4, 5] = logits[4, 9] = inf
    logits[5] = torch.finfo(F32).min         # the type's lowest value masks nothing
    logits[6, 1:] = torch.finfo(F32).min
    logits[7] = float("nan")
    logits[8, :60] = -inf
    logits[9] = torch.finfo(F32).max
    logits[10] = -60.0                       # sigmoid scores near 1e-26
    logits[11, 32:] = -inf                   # whole groups masked
    bias = None
    if biased:
        bias = torch.randn(64, generator=g, device="cuda") * 0.3
        bias[7], bias[8], bias[9] = -inf, float("nan"), inf
    for renorm in (True, False):
        _check_route(nvm, logits, 6, bias=bias, score=score, groups=groups, keep=keep, top=top, renorm=renorm)


def test_route_strided_logits(nvm):
    g = _gen(3)
    wide = torch.randn(50, 300, generator=g, device="cuda")
    _check_route(nvm, wide[:, 17:145], 8)
    _check_route(nvm, wide[::3, 1:65].to(BF16), 4, score="sigmoid")
    _check_route(nvm, wide.to(BF16)[::2, 3:260], 4, score="sigmoid", bias=torch.zeros(257, device="cuda"))


def test_route_feeds_the_sort_and_the_forward(nvm):
    """Padding tokens (all logits masked) drop out of the sort and of the output."""
    from workloads import make_problem
    from workloads.device import upload_inputs, upload_layer
    from workloads.generators import MoEConfig

    prob = make_problem(MoEConfig("padded", 256, 512, 8, 2, 9, "uniform", 77))
    layer = upload_layer(prob)
    x, _, _ = upload_inputs(prob)
    logits = torch.randn(9, 8, generator=_gen(1), device="cuda")
    logits[3] = logits[8] = float("-inf")
    ids = torch.empty(9, 2, dtype=torch.int32, device="cuda")
    w = torch.empty(9, 2, device="cuda")
    nvm.route_topk(logits, ids, w)
    for ws in (None, layer.workspace(9)):
        bufs = layer.buffers(9)
        layer.forward(x, ids, w, bufs, workspace=ws)
        torch.cuda.synchronize()
        assert bool((ids[3] == -1).all()) and bool((ids[8] == -1).all())
        assert int(bufs.expert_offsets[-1]) == 14 and int(bufs.status) == 1
        assert float(bufs.out[3].abs().max()) == 0.0 and float(bufs.out[8].abs().max()) == 0.0
        fns = [lambda e, mm=mm: prob.expert_weight(mm, e) for mm in (0, 1, 2)]
        ref = orc.moe_forward(prob.x_bf16, ids.cpu().numpy(), w.cpu().numpy(), 8, *fns, hidden=256, inter=512)
        assert orc.relative_l2(bufs.out.cpu().numpy().astype(np.float64), ref["out"]) <= 1e-3


@pytest.mark.parametrize("kind", ["shared", "nongated", "steps"])
def test_forward_logits_is_routing_then_forward(nvm, kind):
    from workloads import make_problem
    from workloads.device import upload_inputs, upload_layer
    from workloads.generators import MoEConfig

    prob = make_problem(MoEConfig("routed", 256, 512, 8, 2, 21, "uniform", 88))
    layer = upload_layer(prob, shared=kind == "shared", activation="relu2" if kind == "nongated" else None)
    x, _, _ = upload_inputs(prob)
    router = nvm.MoERouter(2, score="sigmoid", bias=torch.linspace(-0.1, 0.1, 8, device="cuda"), scale=2.0)
    logits = torch.randn(21, 8, generator=_gen(2), device="cuda").to(BF16)
    ids, w = torch.empty(21, 2, dtype=torch.int32, device="cuda"), torch.empty(21, 2, device="cuda")
    router.route(logits, ids, w)
    opts = dict(steps=True) if kind == "steps" else {}
    want = layer.forward(x, ids, w, workspace=layer.workspace(21), **opts)
    got = layer.forward_logits(x, logits, router, layer.buffers(30), workspace=layer.workspace(21), **opts)
    torch.cuda.synchronize()
    assert torch.equal(got.routed_ids[:21], ids) and torch.equal(got.routed_weights[:21], w)
    assert torch.equal(got.out[:21], want.out[:21]) and float(want.out.abs().max()) > 0
    for bad in (dict(logits=logits[:20]), dict(router=nvm.MoERouter(3))):
        with pytest.raises(ValueError):
            layer.forward_logits(x, bad.get("logits", logits), bad.get("router", router))


# --------------------------------------------------------------------------- #
# Norm
# --------------------------------------------------------------------------- #
E4M3, INT8 = torch.float8_e4m3fn, torch.int8
# Relative error of an FP32 y: a sum of up to 32 terms per thread and 10 tree steps
# of positive numbers, halved by the root, rsqrt 2 ulp, r, its two products: under
# 32 roundings.
Y32 = 32 * 2.0 ** -24


def _norm_ref(x, res, weight, eps):
    r = x.double() if res is None else x.double() + res.double()
    return r, r / torch.sqrt((r * r).mean(dim=1, keepdim=True) + eps) * weight.double()


def _check_norm(nvm, x, weight, res=None, eps=1e-6, want_out=True, code=None, in_place=False):
    m, h = x.shape
    r, y = _norm_ref(x, res, weight, eps)
    out, out_ok = _guarded(m, h, BF16, -7.0) if want_out else (None, lambda: None)
    r_out, r_ok = (None, lambda: None)
    if res is not None:
        r_out, r_ok = (res, lambda: None) if in_place else _guarded(m, h, res.dtype, -7.0)
    q = scale = None
    q_ok = s_ok = lambda: None
    if code is not None:
        q, q_ok = _guarded(m, h, torch.uint8, 7)
        q = q.view(code)
        scale, s_ok = _guarded(1, m, F32, -7.0)
        scale = scale[0]
    nvm.add_rms_norm(x, weight, eps, out=out, residual=res, residual_out=r_out, q=q, q_scale=scale)
    torch.cuda.synchronize()
    out_ok(), r_ok(), q_ok(), s_ok()
    if res is not None:
        # r in FP32, then the type: two roundings.
        assert bool(((r_out.double() - r).abs() <= r.abs() * (HALF[res.dtype] + 2.0 ** -23)).all())
    if want_out:
        assert bool(((out.double() - y).abs() <= y.abs() * (HALF[BF16] * 1.01 + Y32) + 2.0 ** -133).all())
    if code is not None:
        most = 127.0 if code == INT8 else 448.0
        s = y.abs().amax(dim=1) / most
        assert bool(((scale.double() - s).abs() <= s * Y32).all())
        t = torch.where(s[:, None] > 0, y / s[:, None], torch.zeros_like(y))
        v = q.double() if code == INT8 else q.float().double()
        # t is formed with five roundings; half a step of the code's type on top:
        # 1/2 for int8; E4M3 2^-4 of the value, 2^-10 below its normal range.
        step = torch.full_like(t, 0.5) if code == INT8 else torch.clamp(t.abs() * 2.0 ** -4, min=2.0 ** -10)
        assert bool(((v - t).abs() <= step + t.abs() * 5 * 2.0 ** -24).all()), float((v - t).abs().max())
        assert bool((v.abs().amax(dim=1)[s > 0] == most).all())


def _hidden(g, m, h, dtype, scale=1.0):
    loud = 1.0 + 15.0 * (torch.rand(h, generator=g, device="cuda") < 0.01)
    return (torch.randn(m, h, generator=g, device="cuda") * loud * scale).to(dtype)


@pytest.mark.parametrize("m,h", [(1, 1), (3, 7), (5, 32), (1, 256), (9, 255), (17, 1000), (4, 1024), (3, 1025),
                                 (2, 2048), (33, 4096), (5, 4100), (3, 7168), (2, 8192), (3, 8200), (2, 16384),
                                 (2, 16392), (1, 16391), (2, 32768), (1, 32767), (1500, 96)])
@pytest.mark.parametrize("xt,rt", [(BF16, None), (BF16, BF16), (F32, None), (F32, BF16), (F32, F32), (BF16, F32)])
def test_norm_matches_the_definition(nvm, m, h, xt, rt):
    g = _gen(m * 40000 + h)
    x = _hidden(g, m, h, xt)
    res = None if rt is None else _hidden(g, m, h, rt, 2.0)
    wt = F32 if (m + h) % 2 else BF16
    weight = (1 + 0.2 * torch.randn(h, generator=g, device="cuda")).to(wt)
    _check_norm(nvm, x, weight, res)
    _check_norm(nvm, x, weight, res, code=INT8)
    _check_norm(nvm, x, weight, res, code=E4M3, want_out=False)


@pytest.mark.parametrize("shift", [1, 2, 4])
@pytest.mark.parametrize("code", [INT8, E4M3])
def test_norm_views_and_alignments(nvm, shift, code):
    """Column slices at every alignment, row strides, an odd row distance."""
    g = _gen(shift)
    for width in (600, 601):
        wide = torch.randn(12, width, generator=g, device="cuda")
        for h in (512, 264, 77):
            x = wide[:, shift:shift + h]
            weight = torch.randn(h + shift, generator=g, device="cuda")[shift:]
            _check_norm(nvm, x, weight, wide.to(BF16)[:, 8:8 + h], code=code)
            _check_norm(nvm, wide.to(BF16)[::3, shift:shift + h], weight.to(BF16), wide[::3, :h], code=code)


def test_norm_in_place(nvm):
    g = _gen(2)
    for h in (256, 1001, 20000):
        x = _hidden(g, 6, h, BF16)
        weight = torch.ones(h, device="cuda")
        _check_norm(nvm, x, weight, _hidden(g, 6, h, BF16), in_place=True, code=INT8)
        # The residual's output on x, and the norm's output on the residual.
        x2, res = x.clone(), _hidden(g, 6, h, BF16)
        r, y = _norm_ref(x, res, weight, 1e-6)
        nvm.add_rms_norm(x2, weight, 1e-6, out=res, residual=res, residual_out=x2)
        torch.cuda.synchronize()
        assert bool(((x2.double() - r).abs() <= r.abs() * (HALF[BF16] + 2.0 ** -23)).all())
        assert bool(((res.double() - y).abs() <= y.abs() * (HALF[BF16] * 1.01 + Y32)).all())


@pytest.mark.parametrize("code", [INT8, E4M3])
def test_norm_rows_of_extreme_values(nvm, code):
    h = 512
    g = _gen(9)
    x = torch.randn(8, h, generator=g, device="cuda")
    x[0] = 0.0
    x[1] *= 1e-30           # squares vanish: eps carries the norm
    x[2] = 0.0
    x[2, 17] = 3e15         # one value alone
    x[3] *= 1e15
    x[4] = 1e-44            # subnormal
    weight = torch.ones(h, device="cuda")
    rows = [0, 1, 2, 3, 5, 6, 7]
    _check_norm(nvm, x[rows].contiguous(), weight, code=code)
    weight[3:200] = 0.0
    _check_norm(nvm, x[rows].contiguous(), weight, code=code)
    q = torch.empty(8, h, dtype=code, device="cuda")
    s = torch.empty(8, device="cuda")
    nvm.add_rms_norm(x, weight, 1e-6, q=q, q_scale=s)
    assert bool(torch.isfinite(q.float()).all()) and bool(torch.isfinite(s).all())
    assert float(s[0]) == 0.0 and float(q[0].float().abs().max()) == 0.0


def test_norm_keeps_bad_rows_to_themselves(nvm):
    g = _gen(4)
    x = torch.randn(6, 300, generator=g, device="cuda").to(BF16)
    res = torch.randn(6, 300, generator=g, device="cuda").to(BF16)
    x[1, 7] = float("nan")
    x[3, 299] = float("inf")
    weight = torch.ones(300, device="cuda")
    out, r_out = torch.empty_like(x), torch.empty_like(res)
    q, s = torch.empty(6, 300, dtype=INT8, device="cuda"), torch.empty(6, device="cuda")
    nvm.add_rms_norm(x, weight, 1e-6, out=out, residual=res, residual_out=r_out, q=q, q_scale=s)
    assert bool(torch.isnan(out[1]).all()) and bool(torch.isnan(out[3, 299])) and bool(torch.isnan(s[[1, 3]]).all())
    assert bool(torch.isinf(r_out[3, 299])) and bool(torch.isfinite(r_out[1, :7]).all())
    good = [0, 2, 4, 5]
    assert bool(torch.isfinite(out[good]).all()) and bool(torch.isfinite(s[good]).all())
    r, y = _norm_ref(x[good], res[good], weight, 1e-6)
    assert bool(((out[good].double() - y).abs() <= y.abs() * (HALF[BF16] * 1.01 + Y32)).all())


# --------------------------------------------------------------------------- #
# int8 product
# --------------------------------------------------------------------------- #
def _codes(g, m, k):
    return torch.randint(-128, 128, (m, k), generator=g, device="cuda", dtype=torch.int8)


def _check_matmul(nvm, x, w, dtype=BF16, bias=None, seed=0, strided=False):
    (m, k), n = x.shape, w.shape[0]
    g = _gen(seed)
    xs = torch.rand(m, generator=g, device="cuda") + 0.01
    ws = torch.rand(n, generator=g, device="cuda") * 1e-3
    if strided:
        store = torch.full((m, n + 13), -7.0, device="cuda").to(dtype)
        out, ok = store[:, 5:5 + n], lambda: None
    else:
        out, ok = _guarded(m, n, dtype, -7.0)
    nvm.int8_matmul(x, xs, w, ws, out, bias=bias)
    torch.cuda.synchronize()
    assert nvm.device_error() == 0
    ok()
    if strided:
        rest = torch.cat([store[:, :5], store[:, 5 + n:]], dim=1)
        assert bool((rest == -7.0).all())
    sums = x.double() @ w.double().T  # whole numbers below 2^53: exact
    prod = sums * xs.double()[:, None] * ws.double()
    want = prod if bias is None else prod + bias.double()
    # The sum to FP32 and two products; the bias' addition; the output's rounding.
    off = prod.abs() * 4 * 2.0 ** -24 + want.abs() * (HALF[dtype] * 1.01 if dtype == BF16 else 2.0 ** -24)
    assert bool(((out.double() - want).abs() <= off).all()), float(((out.double() - want).abs() - off).max())


@pytest.mark.parametrize("m", [1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 64, 65, 100, 128, 129, 200, 256, 257, 300, 513])
@pytest.mark.parametrize("n,k", [(256, 256), (200, 208), (1, 16), (33, 48), (129, 1040), (515, 144), (1024, 2048)])
def test_matmul_matches_the_definition(nvm, m, n, k):
    g = _gen(m * 7 + n + k)
    x, w = _codes(g, m, k), _codes(g, n, k)
    _check_matmul(nvm, x, w, seed=m)
    _check_matmul(nvm, x, w, F32, bias=torch.randn(n, generator=g, device="cuda"), seed=n)


@pytest.mark.parametrize("m,n,k", [(1, 4096, 2048), (32, 5120, 4096), (5, 1536, 16), (256, 2048, 7168), (1000, 4099, 2048),
                                   (2048, 1536, 4096), (700, 8192, 512), (4097, 1111, 272)])
def test_matmul_larger_sizes(nvm, m, n, k):
    g = _gen(m + n)
    _check_matmul(nvm, _codes(g, m, k), _codes(g, n, k), seed=k)
    _check_matmul(nvm, _codes(g, m, k), _codes(g, n, k), F32, bias=torch.randn(n, generator=g, device="cuda"), seed=k)


# Shapes that take each of the forms (register-fed with 8 and 16 tokens and short and
# long k; tiles of 64 and 128 channels, k whole or split over 2, 4, 8 CTAs; CTA
# pairs), with n a multiple of 8, even and odd, batches below and above a tile's 128
# rows, and k that ends inside a stage.
FORMS = [(1, 1, 4480), (243, 1, 4384), (138, 8, 4480), (26, 288, 5264), (5, 3686, 4640), (6, 9791, 1072),
         (1330, 1, 1920), (4027, 2, 672), (110, 2426, 48), (49, 1870, 1472), (92, 1479, 1296), (1428, 465, 96),
         (231, 3924, 96), (226, 3489, 112), (230, 3640, 112), (64, 4711, 512), (110, 3356, 576), (79, 3696, 896),
         (772, 1457, 544), (4442, 326, 784),
         (4239, 40, 1584), (33, 4206, 1952), (4194, 46, 1520), (4204, 51, 1472), (45, 4432, 1792), (2331, 139, 1664),
         (3580, 17, 2848), (3817, 50, 944), (84, 1589, 1440), (166, 944, 1360), (127, 1254, 1472), (126, 1256, 1712),
         (1717, 19, 4480), (1198, 34, 4464), (65, 774, 4000), (113, 639, 2880), (625, 184, 1888), (89, 960, 3936),
         (268, 4456, 1520), (140, 4991, 2608), (653, 2830, 1200),
         (17, 3874, 3216), (2866, 66, 1376), (1470, 131, 1408), (49, 3960, 1408), (72, 2651, 1472), (2260, 72, 2176),
         (1431, 2413, 80), (2396, 1526, 80), (1832, 2008, 80), (1025, 2305, 2064), (511, 8191, 2048), (2091, 2259, 96),
         (153, 7921, 944), (243, 6941, 1424), (488, 2964, 2304), (1, 6934, 6096), (2, 7667, 5584), (9, 5993, 5040),
         (1, 3989, 6016), (14, 2939, 6352), (2064, 71, 5504), (420, 8198, 64), (3988, 6446, 16), (474, 7623, 256),
         (642, 1896, 128), (784, 1388, 224), (494, 4471, 208), (1, 7839, 2928), (63, 3679, 688), (1770, 181, 896),
         (9, 4585, 3392), (2244, 79, 3120), (487, 729, 2320), (4989, 19, 6128), (9, 1568, 6384), (2137, 55, 1904),
         (579, 250, 2336), (813, 18, 6016), (209, 190, 3904), (408, 98, 4912), (98, 67, 1024), (189, 2708, 48),
         (16, 1008, 8192), (63, 1024, 1664)]


@pytest.mark.parametrize("m,n,k", FORMS)
def test_matmul_forms(nvm, m, n, k):
    g = _gen(m * n)
    x, w = _codes(g, m, k), _codes(g, n, k)
    bias = torch.randn(n, generator=g, device="cuda")
    _check_matmul(nvm, x, w, seed=1)
    _check_matmul(nvm, x, w, bias=bias, seed=2)
    _check_matmul(nvm, x, w, F32, seed=3)
    _check_matmul(nvm, x, w, F32, bias=bias, seed=4)
    _check_matmul(nvm, x, w, bias=bias, seed=5, strided=True)
    _check_matmul(nvm, x, w, F32, seed=6, strided=True)


@pytest.mark.parametrize("m", [1, 20, 150, 600])
def test_matmul_strided_rows(nvm, m):
    g = _gen(m)
    for n, k in ((128, 256), (77, 336), (512, 512)):
        wide = _codes(g, 2 * m, k + 64)
        w = _codes(g, n, k)
        _check_matmul(nvm, wide[::2, 16:16 + k], w, strided=True)
        _check_matmul(nvm, wide[:m, 48:48 + k], w, F32, strided=True)


@pytest.mark.parametrize("m", [1, 40, 130])
def test_matmul_largest_sums(nvm, m):
    """All codes -128 at the longest K: the sums reach 2^31 - 2^18."""
    k = 131056  # the limit
    x = torch.full((m, k), -128, dtype=torch.int8, device="cuda")
    w = torch.full((48, k), -128, dtype=torch.int8, device="cuda")
    w[1] = 127
    _check_matmul(nvm, x, w, F32)


def test_matmul_scales_of_zero_and_nan(nvm):
    """A row of zeros arrives with scale 0; a poisoned row stays to itself."""
    g = _gen(1)
    for m in (4, 40, 300):
        x, w = _codes(g, m, 128), _codes(g, 64, 128)
        xs, ws = torch.ones(m, device="cuda"), torch.ones(64, device="cuda")
        xs[1], xs[2] = 0.0, float("nan")
        out = torch.empty(m, 64, device="cuda")
        nvm.int8_matmul(x, xs, w, ws, out)
        torch.cuda.synchronize()
        assert float(out[1].abs().max()) == 0.0 and bool(torch.isnan(out[2]).all())
        rest = [i for i in range(m) if i != 2]
        assert torch.equal(out[rest].double(), (x.double() @ w.double().T * xs.double()[:, None])[rest])


# --------------------------------------------------------------------------- #
# Together, streams and graphs
# --------------------------------------------------------------------------- #
class _Block:
    """One layer's way through the operators: norm to BF16 and int8, router logits from
    the int8 rows, routing, the experts, the next norm over their FP32 output, and the
    next projection on its int8 rows."""

    def __init__(self, nvm, m, seed):
        from workloads import make_problem
        from workloads.device import upload_layer
        from workloads.generators import MoEConfig

        self.nvm, self.m = nvm, m
        self.prob = make_problem(MoEConfig("block", 256, 512, 8, 2, m, "uniform", 1000))
        self.layer = upload_layer(self.prob)
        self.router = nvm.MoERouter(2, score="sigmoid", bias=torch.randn(8, generator=_gen(1), device="cuda") * 0.1,
                                    num_groups=4, topk_groups=2, group_top=2, scale=1.5)
        g = _gen(seed)
        cuda = dict(device="cuda")
        self.x = torch.randn(m, 256, generator=g, **cuda).to(BF16)
        self.res = torch.randn(m, 256, generator=g, **cuda).to(BF16)
        self.gain = (1 + 0.1 * torch.randn(256, generator=g, **cuda)).to(BF16)
        self.wr, self.wrs = _codes(g, 8, 256), torch.full((8,), 0.001, **cuda)
        self.wp, self.wps = _codes(g, 320, 256), torch.full((320,), 0.001, **cuda)
        self.res1, self.h = torch.empty_like(self.res), torch.empty_like(self.x)
        self.res2 = torch.empty_like(self.res)
        self.q, self.s = torch.empty(m, 256, dtype=INT8, **cuda), torch.empty(m, **cuda)
        self.q2, self.s2 = torch.empty(m, 256, dtype=INT8, **cuda), torch.empty(m, **cuda)
        self.logits = torch.empty(m, 8, **cuda)
        self.bufs, self.ws = self.layer.buffers(m), self.layer.workspace(m)
        self.y = torch.empty(m, 320, dtype=BF16, **cuda)

    def run(self):
        nvm = self.nvm
        nvm.add_rms_norm(self.x, self.gain, 1e-6, out=self.h, residual=self.res, residual_out=self.res1,
                         q=self.q, q_scale=self.s)
        nvm.int8_matmul(self.q, self.s, self.wr, self.wrs, self.logits)
        self.layer.forward_logits(self.h, self.logits, self.router, self.bufs, workspace=self.ws)
        nvm.add_rms_norm(self.bufs.out, self.gain, 1e-6, residual=self.res1, residual_out=self.res2,
                         q=self.q2, q_scale=self.s2)
        nvm.int8_matmul(self.q2, self.s2, self.wp, self.wps, self.y)

    def outputs(self):
        return [self.res1, self.h, self.q, self.s, self.logits, self.bufs.routed_ids, self.bufs.routed_weights,
                self.bufs.out, self.res2, self.q2, self.s2, self.y]

    def check(self):
        """Each step against 64 bits, from what the step before it wrote."""
        torch.cuda.synchronize()
        assert self.nvm.device_error() == 0
        r, y = _norm_ref(self.x, self.res, self.gain, 1e-6)
        assert bool(((self.h.double() - y).abs() <= y.abs() * (HALF[BF16] * 1.01 + Y32)).all())
        want = (self.q.double() @ self.wr.double().T) * self.s.double()[:, None] * self.wrs.double()
        assert bool(((self.logits.double() - want).abs() <= want.abs() * 4 * 2.0 ** -24).all())
        ids, w = _route_ref(self.logits, self.router.bias, 2, "sigmoid", 4, 2, 2, True, 1.5)
        np.testing.assert_array_equal(self.bufs.routed_ids.cpu().numpy(), ids)
        assert np.abs(self.bufs.routed_weights.cpu().numpy() - w).max() <= 2.0 ** -16
        fns = [lambda e, mm=mm: self.prob.expert_weight(mm, e) for mm in (0, 1, 2)]
        bits = self.h.view(torch.int16).cpu().numpy().view(np.uint16)
        ref = orc.moe_forward(bits, ids.astype(np.int32), w.astype(np.float32), 8, *fns, hidden=256, inter=512)
        out = self.bufs.out[:self.m]
        assert orc.relative_l2(out.cpu().numpy().astype(np.float64), ref["out"]) <= 1e-3
        r2, y2 = _norm_ref(out, self.res1, self.gain, 1e-6)
        assert bool(((self.res2.double() - r2).abs() <= r2.abs() * (HALF[BF16] + 2.0 ** -23)).all())
        t = y2 / (y2.abs().amax(dim=1, keepdim=True) / 127.0)
        assert bool(((self.q2.double() - t).abs() <= 0.5 + t.abs() * 5 * 2.0 ** -24).all())
        want = (self.q2.double() @ self.wp.double().T) * self.s2.double()[:, None] * self.wps.double()
        assert bool(((self.y.double() - want).abs() <= want.abs() * (HALF[BF16] * 1.01)).all())


@pytest.mark.parametrize("m", [1, 5, 40, 200])
def test_block_matches_step_by_step(nvm, m):
    b = _Block(nvm, m, m)
    b.run()
    b.check()


def test_block_captured_and_replayed(nvm):
    """Two captured blocks of different sizes, replayed after one another and again on new
    inputs, give what eager runs give, bit for bit."""
    blocks = [_Block(nvm, 5, 1), _Block(nvm, 70, 2)]
    eager = []
    for b in blocks:
        b.run()
        torch.cuda.synchronize()
        eager.append([t.clone() for t in b.outputs()])
    side = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(side):
        for b in blocks:
            b.run()
            side.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                b.run()
            graphs.append(graph)
    torch.cuda.synchronize()
    for _ in range(2):
        for b in blocks:
            for t in b.outputs():
                t.zero_()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for b, want in zip(blocks, eager):
            for t, u in zip(b.outputs(), want):
                assert torch.equal(t.view(torch.uint8), u.view(torch.uint8))
    blocks[0].x.copy_(torch.randn_like(blocks[0].x))
    graphs[0].replay()
    blocks[0].check()


FIRST_CALL_CAPTURED = """
import torch
import nvfp4_weight_quantized_moe_b200 as nvm
g = torch.Generator(device="cuda").manual_seed(1)
m, n, k = 256, 2048, 7168
x = torch.randint(-127, 128, (m, k), dtype=torch.int8, device="cuda", generator=g)
w = torch.randint(-127, 128, (n, k), dtype=torch.int8, device="cuda", generator=g)
xs, ws, out = torch.rand(m, device="cuda"), torch.rand(n, device="cuda"), torch.zeros(m, n, device="cuda")
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    nvm.int8_matmul(x, xs, w, ws, out)
graph.replay()
torch.cuda.synchronize()
captured = out.clone()
nvm.int8_matmul(x, xs, w, ws, out)
torch.cuda.synchronize()
assert torch.equal(captured, out) and out.abs().max() > 0
assert nvm.device_error() == 0
print("captured")
"""


def test_the_first_call_of_a_process_may_be_captured(nvm):
    """What a launch asks the device once (shared-memory limits, clusters) is asked during a capture."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", FIRST_CALL_CAPTURED], cwd=root, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and "captured" in res.stdout, res.stderr[-2000:]


def test_calls_on_two_streams_at_once(nvm):
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    blocks = [_Block(nvm, 64, 3), _Block(nvm, 33, 4)]
    for b in blocks:
        b.run()
    torch.cuda.synchronize()
    want = [[t.clone() for t in b.outputs()] for b in blocks]
    for b in blocks:
        for t in b.outputs():
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        for b, s in zip(blocks, streams):
            with torch.cuda.stream(s):
                b.run()
    torch.cuda.synchronize()
    for b, w in zip(blocks, want):
        for t, u in zip(b.outputs(), w):
            assert torch.equal(t.view(torch.uint8), u.view(torch.uint8))


def test_a_given_stream_is_the_one_used(nvm):
    """The stream argument wins over the current one: the call waits for that stream's work."""
    s = torch.cuda.Stream()
    x = torch.zeros(64, 512, device="cuda")
    weight = torch.ones(512, device="cuda")
    out = torch.empty(64, 512, dtype=BF16, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        x.fill_(2.0)
    nvm.add_rms_norm(x, weight, 1e-6, out=out, stream=s)
    s.synchronize()
    assert float((out.float() - 1.0).abs().max()) <= 2.0 ** -8


# --------------------------------------------------------------------------- #
# Refusals that need CUDA tensors
# --------------------------------------------------------------------------- #
def test_the_binding_refuses_wrong_tensors(nvm):
    cuda = dict(device="cuda")
    l, ids, w = torch.zeros(4, 16, **cuda), torch.zeros(4, 2, dtype=torch.int32, **cuda), torch.zeros(4, 2, **cuda)
    for args in ((l.half(), ids, w), (l, ids.long(), w), (l, ids, w.double())):
        with pytest.raises(TypeError):
            nvm.route_topk(*args)
    for args in ((l, ids[:3], w), (l, ids, w[:, :1]), (l, ids.T.contiguous().T, w), (l, ids.cpu(), w), (l.T, ids, w)):
        with pytest.raises(ValueError):
            nvm.route_topk(*args)
    with pytest.raises(ValueError):
        nvm.route_topk(l, ids, w, bias=torch.zeros(15, **cuda))
    with pytest.raises(nvm.NVFP4MoEError):
        nvm.route_topk(l, ids, w, num_groups=3)
    for bad in (dict(num_groups=-1), dict(topk_groups=1 << 40), dict(scale=1e300)):
        with pytest.raises((ValueError, nvm.NVFP4MoEError)):
            nvm.route_topk(l, ids, w, **bad)
    with pytest.raises(AttributeError):
        nvm.route_topk(None, ids, w)

    x, g, out = torch.zeros(4, 16, **cuda), torch.ones(16, **cuda), torch.zeros(4, 16, dtype=BF16, **cuda)
    q, s = torch.zeros(4, 16, dtype=INT8, **cuda), torch.zeros(4, **cuda)
    for kw in (dict(out=out.float()), dict(out=out, residual=x.half()), dict(q=q.float(), q_scale=s),
               dict(q=q, q_scale=s.double()), dict(out=out, residual=x, residual_out=out)):
        with pytest.raises(TypeError):
            nvm.add_rms_norm(x, g, 1e-6, **kw)
    for kw in (dict(out=out[:2]), dict(out=out, residual=x[:2]), dict(out=out, residual_out=x), dict(q=q),
               dict(out=out, q_scale=s), dict(q=q, q_scale=s[:3]), dict(out=out.cpu())):
        with pytest.raises(ValueError):
            nvm.add_rms_norm(x, g, 1e-6, **kw)
    with pytest.raises(ValueError):
        nvm.add_rms_norm(x, g[:15], 1e-6, out=out)
    with pytest.raises(nvm.NVFP4MoEError):
        nvm.add_rms_norm(x, g, 0.0, out=out)
    with pytest.raises(nvm.NVFP4MoEError):
        nvm.add_rms_norm(x, g, 1e-6)

    wq, o = torch.zeros(8, 16, dtype=INT8, **cuda), torch.zeros(4, 8, **cuda)
    ws = torch.ones(8, **cuda)
    for args in ((q.float(), s, wq, ws, o), (q, s, wq.float(), ws, o), (q, s.double(), wq, ws, o), (q, s, wq, ws, o.half())):
        with pytest.raises(TypeError):
            nvm.int8_matmul(*args)
    for args in ((q, s[:3], wq, ws, o), (q, s, wq[:, :8], ws, o), (q, s, wq, ws[:7], o), (q, s, wq, ws, o[:, :7]),
                 (q, s, wq.cpu(), ws, o)):
        with pytest.raises(ValueError):
            nvm.int8_matmul(*args)
    with pytest.raises(nvm.NVFP4MoEError):
        nvm.int8_matmul(q[:, :8], s, wq[:, :8].contiguous(), ws, o)


def test_arguments_that_have_no_truth_value(nvm):
    cuda = dict(device="cuda")
    l, ids, w = torch.zeros(4, 16, **cuda), torch.zeros(4, 2, dtype=torch.int32, **cuda), torch.zeros(4, 2, **cuda)
    with pytest.raises(RuntimeError):  # of a tensor of two values, as everywhere in Python
        nvm.route_topk(l, ids, w, renormalize=torch.ones(2))
    nvm.route_topk(l, ids, w, renormalize=torch.ones(1))
    torch.cuda.synchronize()
    assert torch.equal(w, torch.full_like(w, 0.5))


def test_empty_batches(nvm):
    cuda = dict(device="cuda")
    nvm.route_topk(torch.empty(0, 16, **cuda), torch.empty(0, 2, dtype=torch.int32, **cuda), torch.empty(0, 2, **cuda))
    nvm.add_rms_norm(torch.empty(0, 64, **cuda), torch.ones(64, **cuda), 1e-6, out=torch.empty(0, 64, dtype=BF16, **cuda))
    nvm.int8_matmul(torch.empty(0, 64, dtype=INT8, **cuda), torch.empty(0, **cuda),
                    torch.zeros(8, 64, dtype=INT8, **cuda), torch.ones(8, **cuda), torch.empty(0, 8, **cuda))
    torch.cuda.synchronize()
