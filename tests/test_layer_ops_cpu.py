"""CPU checks of the operators around the forward (routing, RMS norm, int8
product): the library refuses bad arguments on the host, before any CUDA call,
and the binding refuses tensors it cannot hand over.  No compute runs."""

import ctypes
import os
import re

import pytest
import torch

OK, EINVAL, ESHAPE = 0, 1, 2
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def B():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import nvfp4_weight_quantized_moe_b200._binding as binding
    return binding


P = [(1 + i) << 32 for i in range(8)]  # device addresses far apart; never read


def test_the_packed_structs_are_the_header_s(B):
    """Field by field, against the header's declarations laid out by ctypes."""
    text = open(os.path.join(ROOT, "include", "nvfp4_moe.h")).read()
    plain = {"uint64_t": ctypes.c_uint64, "uint32_t": ctypes.c_uint32, "int32_t": ctypes.c_int32,
             "float": ctypes.c_float}
    for name, layout in (("route", B._ROUTE_ARGS), ("norm", B._NORM_ARGS), ("int8", B._INT8_ARGS)):
        body = re.search(r"typedef struct \{([^}]*)\} nvfp4_moe_%s_args;" % name, text).group(1)
        fields = []
        for line in filter(None, (part.strip() for part in body.split(";"))):
            kind, field = line.rsplit(" ", 1)
            fields.append((field, ctypes.c_void_p if kind.endswith("*") else plain[kind]))
        struct_type = type(name, (ctypes.Structure,), {"_fields_": fields})
        values = [1000 + i for i in range(len(fields))]
        raw = layout.pack(*values).ljust(ctypes.sizeof(struct_type), b"\0")
        got = struct_type.from_buffer_copy(raw)
        assert [getattr(got, f) for f, _ in fields] == values, name


# --------------------------------------------------------------------------- #
# Routing
# --------------------------------------------------------------------------- #
def _route(B, tokens=4, ld=None, kind=1, logits=P[0], ids=P[1], weights=P[2], bias=0, num_experts=16, topk=2,
           num_groups=1, topk_groups=1, group_top=1, score=1, renormalize=1, scale=1.0):
    args = B._ROUTE_ARGS.pack(logits, bias, ids, weights, num_experts if ld is None else ld, tokens, num_experts,
                              topk, num_groups, topk_groups, group_top, kind, score, renormalize, scale)
    return B._lib.nvfp4_moe_route_topk(args, None)


def test_no_arguments_at_all(B):
    for name in ("route_topk", "add_rms_norm", "int8_matmul"):
        assert getattr(B._lib, "nvfp4_moe_" + name)(None, None) == EINVAL


@pytest.mark.parametrize("kw", [
    dict(num_experts=0), dict(num_experts=1025), dict(topk=0), dict(topk=33, num_experts=64),
    dict(topk=17), dict(ld=15), dict(num_groups=0), dict(num_groups=3), dict(num_experts=66, num_groups=33),
    dict(num_groups=4, topk_groups=0), dict(num_groups=4, topk_groups=5), dict(group_top=0),
    dict(group_top=3), dict(num_groups=16, topk_groups=2, group_top=2),
    dict(num_groups=4, topk_groups=1, topk=5), dict(tokens=(1 << 23) + 1), dict(ld=1 << 41),
])
def test_route_refuses_shapes(B, kw):
    assert _route(B, **kw) == ESHAPE


@pytest.mark.parametrize("kw", [
    dict(kind=2), dict(kind=7), dict(score=0), dict(score=3), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(logits=0), dict(ids=0), dict(weights=0),
    dict(weights=P[1]), dict(ids=P[0]), dict(weights=(1 << 32) + 64),   # overlapping outputs / input
    dict(logits=(1 << 32) + 2), dict(bias=(2 << 32) + 4), dict(ids=(2 << 32) + 2),
])
def test_route_refuses_arguments(B, kw):
    assert _route(B, **kw) == EINVAL


def test_route_without_tokens_launches_nothing(B):
    assert _route(B, tokens=0, logits=0, ids=0, weights=0) == OK
    assert _route(B, tokens=0, topk=0) == ESHAPE  # the router is still checked


# --------------------------------------------------------------------------- #
# Norm
# --------------------------------------------------------------------------- #
def _norm(B, x=P[0], x_type=0, ldx=64, res=0, res_type=0, ldr=64, res_out=0, w=P[2], w_type=0,
          eps=1e-6, rows=4, hidden=64, out=P[3], q=0, q_type=2, q_scale=0):
    args = B._NORM_ARGS.pack(x, res, res_out, w, out, q, q_scale, ldx, ldr, rows, hidden, x_type, res_type,
                             w_type, q_type, eps)
    return B._lib.nvfp4_moe_add_rms_norm(args, None)


@pytest.mark.parametrize("kw", [
    dict(hidden=0), dict(hidden=32769, ldx=32769), dict(ldx=63), dict(res=P[1], ldr=63),
    dict(rows=1 << 31), dict(ldx=1 << 41),
])
def test_norm_refuses_shapes(B, kw):
    assert _norm(B, **kw) == ESHAPE


@pytest.mark.parametrize("kw", [
    dict(x_type=2), dict(w_type=3), dict(res=P[1], res_type=2), dict(eps=0.0), dict(eps=-1.0),
    dict(eps=float("nan")), dict(eps=float("inf")), dict(x=0), dict(w=0), dict(out=0),
    dict(q=P[4]), dict(q_scale=P[5]), dict(q=P[4], q_scale=P[5], q_type=1),
    dict(res_out=P[1]),                                       # a residual's output without a residual
    dict(res=P[1], res_out=(2 << 32) + 128),              # one row further on
    dict(res=P[1], ldr=72, res_out=P[1]),                     # the same start, another row distance
    dict(res=P[1], res_type=1, res_out=P[0]),                 # on x, another element size
    dict(out=P[2]), dict(q=P[0], q_scale=P[5]), dict(q=P[4], q_scale=P[4]), dict(res=P[1], res_out=P[3]),
    dict(x=(1 << 32) + 1), dict(x=(1 << 32) + 2, x_type=1), dict(q=P[4], q_scale=(6 << 32) + 2),
])
def test_norm_refuses_arguments(B, kw):
    assert _norm(B, **kw) == EINVAL


def test_norm_without_rows_launches_nothing(B):
    assert _norm(B, rows=0) == OK
    assert _norm(B, rows=0, hidden=0) == ESHAPE


# --------------------------------------------------------------------------- #
# int8 product
# --------------------------------------------------------------------------- #
def _matmul(B, x=P[0], ldx=64, xs=P[1], w=P[2], ws=P[3], bias=0, out=P[4], kind=0, ldo=32, m=4, n=32, k=64):
    return B._lib.nvfp4_moe_int8_matmul(B._INT8_ARGS.pack(x, xs, w, ws, bias, out, ldx, ldo, m, n, k, kind), None)


@pytest.mark.parametrize("kw", [
    dict(n=0), dict(k=0), dict(k=24, ldx=32), dict(k=131072, ldx=131072), dict(ldx=48), dict(ldx=72),
    dict(ldo=31), dict(ldx=1 << 40), dict(ldo=1 << 41), dict(m=0x7fffff01), dict(n=0x7fffff01, ldo=1 << 32),
])
def test_matmul_refuses_shapes(B, kw):
    assert _matmul(B, **kw) == ESHAPE


@pytest.mark.parametrize("kw", [
    dict(kind=2), dict(x=0), dict(xs=0), dict(w=0), dict(ws=0), dict(out=0),
    dict(x=(1 << 32) + 8), dict(w=(3 << 32) + 8), dict(out=(5 << 32) + 1),
    dict(out=(5 << 32) + 2, kind=1), dict(bias=(6 << 32) + 2), dict(out=P[0]), dict(out=P[2]),
    dict(out=P[1]), dict(bias=P[4]),
])
def test_matmul_refuses_arguments(B, kw):
    assert _matmul(B, **kw) == EINVAL


def test_matmul_without_tokens_launches_nothing(B):
    assert _matmul(B, m=0) == OK
    assert _matmul(B, m=0, k=24, ldx=32) == ESHAPE


# --------------------------------------------------------------------------- #
# Binding
# --------------------------------------------------------------------------- #
def test_the_binding_takes_cuda_tensors_only(B):
    f, i = torch.zeros(4, 16), torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        B.route_topk(f, i, torch.zeros(4, 2))
    with pytest.raises(ValueError, match="score"):
        B.route_topk(f, i, torch.zeros(4, 2), score="relu")
    with pytest.raises(ValueError, match="CUDA"):
        B.add_rms_norm(f, torch.ones(16), 1e-6, out=torch.zeros(4, 16, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="CUDA"):
        B.int8_matmul(torch.zeros(4, 16, dtype=torch.int8), torch.ones(4),
                      torch.zeros(8, 16, dtype=torch.int8), torch.ones(8), torch.zeros(4, 8))


def test_rows_of_strided_views(B):
    t = torch.zeros(6, 40)
    assert B._rows(t, "t") == (6, 40, 40)
    assert B._rows(t[:, 8:24], "t") == (6, 16, 40)
    assert B._rows(t[::2], "t") == (3, 40, 80)
    assert B._rows(t[:1, :16], "t") == (1, 16, 16)
    for bad in (t.T, t[:, ::2], t[0], t[:1].expand(6, 40)):
        with pytest.raises(ValueError):
            B._rows(bad, "t")
