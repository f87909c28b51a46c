"""The operators around the layer (include/cb_serve.h) against their definitions in 64 bits: the norm with the
residual's addition and 8-bit rows, routing from logits, and products of a few rows with 4-bit
weights in groups.

Tolerances count roundings, each at most half a step of its type (EPS):
  * norm: h is one fp32 addition (its result is compared after one more rounding, to its type).  The sum of
    squares of up to 32768 terms, in at most 32 + 5 + 32 steps of order (a thread's, a warp's, the block's),
    is off by at most 70 EPS32 of itself, its square root by half of that, the division, the root and two
    products by one each: 40 EPS32 of |y|, then the result's own rounding.  An e4m3 code may be the
    neighbour's where the quotient, off by 50 EPS32, lies next to a border.
  * routing: ids are equal to those of the 64-bit order.  A weight is an expf (2 ulp), a sum of at most 16 of
    them and a division, a product: 16 EPS32.  (The softmax that is not renormalised has an argument l - m that
    is rounded: |l - m| EPS32 more, and a sum over the experts: 16 more.)
  * product: a group's products are added in fp32 by the tensor core, which loses at most 2^-22 of the
    magnitudes per instruction of 16 of them: up to 8 instructions a group; then one fused addition per group, joins of
    8 warps, and the weighted sum over slots: (8 + k / group + 8 + 16) 2^-22 of the terms' magnitudes, then the
    result's rounding.  SwiGLU: that relative to its operands, plus 8 EPS32.
"""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import mixture_experts_router_gb300 as cb
from mixture_experts_router_gb300 import build as cbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16, F32 = torch.bfloat16, torch.float32
EPS = {t: torch.finfo(t).eps / 2 for t in (BF16, F32)}
TINY = 1e-37  # below it fp32 products lose bits


# ------------------------------------------------------------------ no GPU
@pytest.fixture(scope="module")
def lib():
    cbuild.build()
    return cb.load_library()


def header():
    return open(os.path.join(ROOT, "include", "cb_serve.h")).read()


def test_header_declares_what_the_library_exports(lib):
    declared = sorted(set(re.findall(r"CB_API\s+[\w\s\*]*?\b(cb_\w+)\s*\(", header())))
    assert declared == sorted(cb.SERVE_SYMBOLS)
    raw = ctypes.CDLL(cb.LIB_PATH)
    assert all(hasattr(raw, name) for name in declared)
    enums = dict(re.findall(r"\b(CB_(?:SCORE|GROUP)_\w+)\s*=\s*(\d+)", header()))
    enums.update(re.findall(r"#define (CB_(?:NORM|FP8|ROUTE|INT4)_\w+)\s+(\d+)", header()))
    assert len(enums) == 8 and all(getattr(cb, n) == int(v) for n, v in enums.items()), enums
    assert cb.CB_INT4_MAX_ROWS == cb.CB_MOE_MAX_FEW


def test_structs_are_laid_out_as_in_the_header(lib):
    """Fields of each struct in the header's order (their sizes are checked where they are packed)."""
    for name, t in (("cb_rms_norm_t", cb.cb_rms_norm_t), ("cb_route_t", cb.cb_route_t), ("cb_int4_matmul_t", cb.cb_int4_matmul_t)):
        body = re.search(r"typedef struct \{([^}]*)\} " + name, header()).group(1)
        body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
        fields = [w for line in body.split(";") for w in re.findall(r"(\w+)\s*(?:,|$)", line.strip())]
        assert fields == [f for f, _ in t._fields_], name


def norm_args(**kw):
    a = dict(rows=4, cols=64, x=0x10000, ld_x=64, residual=None, ld_residual=0, weight=0x20000, sum=None, ld_sum=0,
             out=0x30000, ld_out=64, codes=None, scales=None, eps=1e-6, x_type=0, weight_type=0, out_type=0)
    a.update(kw)
    return cb.cb_rms_norm_t(*(a[n] for n, _ in cb.cb_rms_norm_t._fields_))


def test_norm_refuses_bad_arguments_before_cuda(lib):
    assert lib.cb_rms_norm(None, None) == cb.CB_ERR_INVALID_ARG
    for kw in (dict(rows=-1), dict(cols=0), dict(ld_x=63), dict(ld_out=63), dict(x=None), dict(weight=None), dict(out=None),
               dict(x_type=2), dict(weight_type=2), dict(out_type=-1), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(codes=0x40000), dict(scales=0x40000), dict(residual=0x50000, ld_residual=63),
               dict(sum=0x50000, ld_sum=63), dict(out=0x10010), dict(out=0x10000, ld_out=72), dict(out=0x10000, out_type=1),
               dict(out=0x20000), dict(sum=0x10002, ld_sum=64), dict(residual=0x50000, ld_residual=64, sum=0x50000, ld_sum=65),
               dict(residual=0x30000, ld_residual=64), dict(codes=0x10000, scales=0x40000), dict(codes=0x40000, scales=0x10000),
               dict(codes=0x30000, scales=0x40000), dict(codes=0x40000, scales=0x40010), dict(sum=0x30000, ld_sum=64)):
        assert cb.cb_rms_norm(norm_args(**kw)) == cb.CB_ERR_INVALID_ARG, kw
    for kw in (dict(x=0x10001), dict(x_type=1, x=0x10002), dict(weight=0x20001), dict(out=0x30001), dict(sum=0x50001, ld_sum=64),
               dict(codes=0x40000, scales=0x50002)):
        assert cb.cb_rms_norm(norm_args(**kw)) == cb.CB_ERR_ALIGNMENT, kw
    for kw in (dict(cols=32769, ld_x=40000, ld_out=40000), dict(rows=1 << 31), dict(ld_x=1 << 60)):
        assert cb.cb_rms_norm(norm_args(**kw)) == cb.CB_ERR_UNSUPPORTED, kw
    assert cb.cb_rms_norm(norm_args(rows=0, x=None, weight=None, out=None)) == cb.CB_OK


def route_args(**kw):
    a = dict(n_tokens=4, logits=0x10000, ld_logits=16, bias=None, ids=0x20000, w=0x30000, scale=1.0, logits_type=1,
             n_experts=16, top_k=4, score=0, n_groups=1, top_groups=1, group_score=0, renormalise=1)
    a.update(kw)
    return cb.cb_route_t(*(a[n] for n, _ in cb.cb_route_t._fields_))


def test_route_refuses_bad_arguments_before_cuda(lib):
    assert lib.cb_route(None, None) == cb.CB_ERR_INVALID_ARG
    for kw in (dict(n_tokens=-1), dict(n_experts=0), dict(top_k=0), dict(top_k=17), dict(ld_logits=15), dict(logits=None),
               dict(ids=None), dict(w=None), dict(score=2), dict(group_score=2), dict(logits_type=2), dict(n_groups=3),
               dict(n_groups=0), dict(n_groups=4, top_groups=5), dict(top_groups=0), dict(n_groups=8, top_groups=1),
               dict(renormalise=2), dict(scale=float("nan")), dict(scale=float("inf")), dict(ids=0x10000), dict(w=0x10020),
               dict(w=0x20000), dict(bias=0x20000), dict(bias=0x30010)):
        assert cb.cb_route(route_args(**kw)) == cb.CB_ERR_INVALID_ARG, kw
    for kw in (dict(logits=0x10002), dict(logits_type=0, logits=0x10001), dict(bias=0x40002), dict(ids=0x20002), dict(w=0x30001)):
        assert cb.cb_route(route_args(**kw)) == cb.CB_ERR_ALIGNMENT, kw
    for kw in (dict(n_experts=257, ld_logits=257), dict(n_experts=64, ld_logits=64, top_k=17),
               dict(n_experts=66, ld_logits=66, n_groups=33, top_groups=33), dict(n_tokens=1 << 31), dict(ld_logits=1 << 60)):
        assert cb.cb_route(route_args(**kw)) == cb.CB_ERR_UNSUPPORTED, kw
    assert cb.cb_route(route_args(n_tokens=0, logits=None, ids=None, w=None)) == cb.CB_OK


def int4_args(**kw):
    a = dict(x=0x100000, x_scales=None, codes=0x200000, scales=0x300000, zeros=None, ids=None, w=None, out=0x400000,
             status=None, ld_x=256, ld_out=64, n=64, k=256, n_tokens=2, top_k=1, n_experts=1, group=64, x_per_slot=0,
             swiglu=0, out_type=0)
    a.update(kw)
    return cb.cb_int4_matmul_t(*(a[n] for n, _ in cb.cb_int4_matmul_t._fields_))


def test_int4_refuses_bad_arguments_before_cuda(lib):
    assert lib.cb_int4_matmul_few(None, None) == cb.CB_ERR_INVALID_ARG
    by = dict(ids=0x500000, n_experts=8, top_k=2)
    for kw in (dict(n_tokens=-1), dict(n=0), dict(n=24), dict(n=48, swiglu=1, ld_out=64), dict(k=0), dict(k=96), dict(group=16),
               dict(group=256), dict(ld_x=255), dict(ld_out=63), dict(out_type=2), dict(x=None), dict(codes=None),
               dict(scales=None), dict(out=None), dict(top_k=2), dict(n_experts=2), dict(w=0x600000), dict(x_per_slot=1),
               dict(w=0x600000, swiglu=1, **by), dict(out=0x100000), dict(out=0x200010), dict(out=0x300000), dict(out=0x500000, **by),
               dict(out=0x600000, w=0x600000, **by), dict(zeros=0x400000), dict(x_scales=0x400000), dict(status=0x400004)):
        assert cb.cb_int4_matmul_few(int4_args(**kw)) == cb.CB_ERR_INVALID_ARG, kw
    for kw in (dict(x=0x100008), dict(codes=0x200004), dict(scales=0x300004), dict(zeros=0x700008), dict(x_scales=0x700002),
               dict(ids=0x500002, n_experts=8), dict(out=0x400001), dict(ld_x=260), dict(status=0x700002)):
        assert cb.cb_int4_matmul_few(int4_args(**kw)) == cb.CB_ERR_ALIGNMENT, kw
    for kw in (dict(n_tokens=17), dict(by, n_experts=257), dict(by, top_k=17), dict(n=(1 << 24) + 16, ld_out=1 << 25),
               dict(k=1 << 25, ld_x=1 << 25), dict(k=393216 + 64, ld_x=1 << 20), dict(by, k=49152 + 64, ld_x=1 << 16), dict(ld_out=1 << 50)):
        assert cb.cb_int4_matmul_few(int4_args(**kw)) == cb.CB_ERR_UNSUPPORTED, kw
    assert cb.cb_int4_matmul_few(int4_args(n_tokens=0, x=None, codes=None, scales=None, out=None)) == cb.CB_OK


def test_python_refusals(lib):
    x, g = torch.zeros(2, 64, dtype=BF16), torch.ones(64, dtype=BF16)
    for args, kw in (((x.half(), g), {}), ((x, g.half()), {}), ((x, g[:32]), {}), ((x, g), dict(want="fp4")),
                     ((x, g), dict(residual=x.float())), ((x, g), dict(residual=x[:1])), ((x, g), dict(sum=x)),
                     ((x, g), dict(out=x, want="fp8")), ((x, g), dict(dtype=torch.float16)), ((x.T, g), {}), ((x, g), {})):
        with pytest.raises(ValueError):        # the last one: not on a GPU
            cb.rms_norm(*args, **kw)
    l = torch.zeros(2, 16)
    for kw in (dict(score="tanh"), dict(group_score="sum"), dict(bias=torch.zeros(15)), dict(bias=torch.zeros(16, dtype=BF16)), {}):
        with pytest.raises(ValueError):
            cb.route(l, 2, **kw)
    with pytest.raises(ValueError):
        cb.route(l.half(), 2)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    m = cb.Int4Matrix(u8(32, 64), torch.ones(2, 32), u8(2, 32))
    assert (m.rows, m.cols, m.group, m.experts) == (32, 128, 64, None)
    e = cb.Int4Matrix(u8(4, 32, 64), torch.ones(4, 1, 32))
    assert (e.rows, e.cols, e.group, e.experts) == (32, 128, 128, 4)
    for args in ((u8(32, 64), torch.ones(32, 2)), (u8(32, 64), torch.ones(2, 31)), (u8(32, 64), torch.ones(8, 32)),
                 (u8(32, 64), torch.ones(3, 32)), (u8(32, 64), torch.ones(2, 32).double()), (u8(32, 64), torch.ones(0, 32)),
                 (u8(32, 64), torch.ones(2, 32), u8(2, 16)), (u8(4, 32, 64), torch.ones(2, 32)),
                 (u8(32, 128)[:, ::2], torch.ones(2, 32)), (torch.zeros(32, 64), torch.ones(2, 32))):
        with pytest.raises(ValueError):
            cb.Int4Matrix(*args)
    rows = cb.Fp8Rows(u8(3, 200), torch.ones(3, 2))
    assert (rows.rows, rows.cols) == (3, 200)
    for args in ((u8(3, 200), torch.ones(3, 1)), (u8(3, 200).float(), torch.ones(3, 2)), (u8(3, 400)[:, ::2], torch.ones(3, 2))):
        with pytest.raises(ValueError):
            cb.Fp8Rows(*args)
    x = torch.zeros(2, 128, dtype=BF16)
    ids, w = torch.zeros(2, 3, dtype=torch.int32), torch.ones(2, 3)
    for args, kw in (((x.float(), m), {}), ((x[:, :64], m), {}), ((x, m), dict(ids=ids)), ((x, e), {}), ((x, m), dict(weights=w)),
                     ((x, e), dict(ids=ids.long())), ((x, e), dict(ids=ids, weights=w.double())), ((x, e), dict(ids=ids[:1])),
                     ((x, e), dict(ids=ids, weights=w, swiglu=True)), ((x, e), dict(ids=ids, weights=w[:, :2])),
                     ((x.view(1, 2, 128), m), {}), ((torch.zeros(2, 2, 128, dtype=BF16), e), dict(ids=ids)),
                     ((x, m), dict(out=torch.zeros(2, 31, dtype=BF16))), ((x, m), dict(dtype=torch.float16)), ((x, m), {})):
        with pytest.raises(ValueError):
            cb.int4_matmul_few(*args, **kw)


# ---------------------------------------------------------------- the norm
def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, std=1.0, dtype=F32):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def e4m3_64(v):
    e = torch.frexp(v.abs().clamp_min(2.0 ** -6)).exponent.double() - 1
    step = torch.exp2(e - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def check_norm(x, weight, residual, r, eps, want, dtype=None):
    h32 = x.float() if residual is None else x.float() + residual.float()
    h = h32.double()
    if residual is not None:
        assert r.sum.dtype == x.dtype and torch.equal(r.sum, h32.to(x.dtype))   # one fp32 addition, one rounding
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + eps) * weight.double()
    err = 40 * EPS[F32] * y.abs() + TINY
    if want != "fp8":
        kind = dtype or x.dtype
        assert r.out.dtype == kind
        assert ((r.out.double() - y).abs() <= err + EPS[kind] * (y.abs() + err) + TINY).all()
    else:
        assert r.out is None
    if want == "out":
        assert r.fp8 is None
        return
    rows, cols = x.shape
    codes, scales = r.fp8.codes.view(torch.float8_e4m3fn).double(), r.fp8.scales.double()
    for b in range(-(-cols // 128)):
        part = slice(b * 128, min(cols, b * 128 + 128))
        s = y[:, part].abs().amax(-1) / 448
        assert ((scales[:, b] - s).abs() <= 42 * EPS[F32] * s + 2.0 ** -149).all()
        q = torch.where(s[:, None] > 0, y[:, part] / s[:, None].clamp_min(1e-300), 0.0)
        tol = 90 * EPS[F32] * q.abs() + (1e-2 * q.abs() if (s < 1e-36).any() else 0)
        lo, hi = e4m3_64(q - tol), e4m3_64(q + tol)
        got = codes[:, part]
        assert ((got >= lo) & (got <= hi)).all()
        # and hardly any is the neighbour's
        assert (got != e4m3_64(q)).double().mean() <= 0.01 or (s < 1e-36).any()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (1, 256), (2, 128), (5, 130), (4, 1000), (17, 2050), (1, 4096), (33, 4096),
                                       (300, 96), (2, 9000), (3, 16384), (2, 32768), (2, 32767)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("want", ["out", "fp8", "both"])
def test_norm_against_64_bits(rows, cols, dtype, want):
    g = gen(rows * 100003 + cols)
    x, weight = randn(g, rows, cols, dtype=dtype), 1 + randn(g, cols, std=0.3)
    residual = randn(g, rows, cols, std=3.0, dtype=dtype) if want != "out" else None
    r = cb.rms_norm(x, weight, eps=1e-5, residual=residual, want=want)
    check_norm(x, weight, residual, r, 1e-5, want)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(2432, 1032), (5000, 2048), (2500, 2056), (4871, 4096), (2600, 4104), (2433, 8192), (2500, 96),
                                       (2500, 1024), (2500, 1031), (3000, 8200)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_norm_many_rows(rows, cols, dtype):
    g = gen(rows + cols)
    wide = randn(g, rows, cols + 8, dtype=dtype)
    x, res, weight = wide[:, :cols], randn(g, rows, cols, std=2.0, dtype=dtype), 1 + randn(g, cols, std=0.3, dtype=dtype)
    r = cb.rms_norm(x, weight, residual=res, want="both", dtype=F32)
    check_norm(x, weight, res, r, 1e-6, "both", F32)
    bare = cb.rms_norm(x, weight)
    check_norm(x, weight, None, bare, 1e-6, "out")
    x2, res2 = x.clone(), res.clone()
    again = cb.rms_norm(x2, weight, residual=res2, sum=res2, out=x2, want="both")
    check_norm(x, weight, res, again, 1e-6, "both")
    assert torch.equal(res2, r.sum) and torch.equal(x2, again.out)
    # a few of the rows alone: another way through the kernels, the same definition
    check_norm(x[-5:], weight, None, cb.rms_norm(x[-5:], weight), 1e-6, "out")


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(607, 4096), (608, 4096), (609, 1032), (456, 8192), (1217, 520), (1500, 2048), (700, 6258), (650, 770)])
def test_norm_rows_about_the_number_of_blocks(rows, cols):
    """As many rows as blocks that stay, one more, one less; and pairs of columns."""
    g = gen(rows + cols)
    for dtype in (BF16, F32):
        x, r = randn(g, rows, cols, dtype=dtype), randn(g, rows, cols, dtype=dtype)
        w = (1 + randn(g, cols, std=0.2)).to(dtype)
        check_norm(x, w, r, cb.rms_norm(x, w, residual=r, want="both"), 1e-6, "both")
        check_norm(x, w, None, cb.rms_norm(x, w, want="fp8"), 1e-6, "fp8")


@pytest.mark.gpu
def test_norm_types_strides_and_places():
    g = gen(5)
    wide = randn(g, 9, 700, dtype=BF16)
    for start, cols in ((0, 512), (1, 512), (3, 333), (8, 640)):   # rows on 16 bytes and not
        x = wide[:, start:start + cols]
        res = randn(g, 9, cols + 24, dtype=BF16)[:, 8:8 + cols]
        weight = (1 + randn(g, cols, std=0.2)).to(BF16)
        for dtype in (BF16, F32):
            out = torch.full((9, cols + 5), 7.0, dtype=dtype, device="cuda")
            total = torch.full((9, cols + 8), 7.0, dtype=BF16, device="cuda")
            r = cb.rms_norm(x, weight, residual=res, want="both", out=out[:, :cols], sum=total[:, :cols])
            check_norm(x, weight, res, r, 1e-6, "both", dtype)
            assert r.out.data_ptr() == out.data_ptr() and (out[:, cols:] == 7).all() and (total[:, cols:] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("cols", [100, 4096, 16384])
def test_norm_in_place(cols):
    g = gen(cols)
    for dtype in (BF16, F32):
        x, res, weight = randn(g, 50, cols, dtype=dtype), randn(g, 50, cols, dtype=dtype), 1 + randn(g, cols, std=0.2, dtype=dtype)
        want = cb.rms_norm(x, weight, residual=res)
        for over in ("residual", "x"):
            x2, res2 = x.clone(), res.clone()
            r = cb.rms_norm(x2, weight, residual=res2, sum=res2 if over == "residual" else x2)
            assert torch.equal(r.sum, want.sum) and torch.equal(r.out, want.out)
            assert torch.equal(res2 if over == "residual" else x2, want.sum)
        x2, res2 = x.clone(), res.clone()
        r = cb.rms_norm(x2, weight, residual=res2, sum=res2, out=x2)
        assert torch.equal(x2, want.out) and torch.equal(res2, want.sum)
        with pytest.raises(cb.CbMoeError):
            cb.rms_norm(x2, weight, residual=res2, out=res2)


@pytest.mark.gpu
def test_norm_of_zeros_extremes_and_what_is_no_number():
    for cols in (256, 250):
        weight = torch.ones(cols, device="cuda")
        x = torch.zeros(8, cols, device="cuda")
        x[1, 200] = 3.0
        x[2] = 1e-20
        x[3, 5] = float("nan")
        x[4, 5] = float("inf")
        x[5] = 1e15
        x[6, :128] = 1.0       # its second group is all zeros
        x[7] = 2.0 ** -149
        r = cb.rms_norm(x, weight, eps=1e-30, want="both")
        ok = [0, 1, 2, 5, 6, 7]
        sub = cb.RmsNormed(r.out[ok], cb.Fp8Rows(r.fp8.codes[ok].contiguous(), r.fp8.scales[ok].contiguous()), None)
        assert (r.out[0] == 0).all() and (r.fp8.codes.view(torch.uint8)[0] == 0).all() and (r.fp8.scales[0] == 0).all()
        assert r.fp8.scales[6, 1] == 0 and (r.fp8.codes.view(torch.uint8)[6, 128:] == 0).all()
        # 1e-20 squared leaves fp32's range: eps decides there, as the documented range says
        keep = [0, 1, 3, 4]
        check_norm(x[[0, 1, 5, 6]], weight, None, cb.RmsNormed(sub.out[keep], cb.Fp8Rows(sub.fp8.codes[keep].contiguous(),
                                                               sub.fp8.scales[keep].contiguous()), None), 1e-30, "both")
        assert r.out[3].isnan().all() and r.fp8.scales[3].isnan().all() and (r.fp8.codes.view(torch.uint8)[3] == 0).all()
        assert r.fp8.scales[4, 0].isnan()
        small = cb.rms_norm(x[1:2], weight * 1e-42, eps=1e-6, want="fp8").fp8     # a scale that is no normal number
        assert (small.codes.float().abs() <= 448).all() and not small.codes.float().isnan().any()


@pytest.mark.gpu
def test_norm_empty_streams_graphs():
    g = gen(1)
    weight = torch.ones(512, device="cuda", dtype=BF16)
    r = cb.rms_norm(torch.empty(0, 512, device="cuda", dtype=BF16), weight, want="both")
    assert r.out.shape == (0, 512) and r.fp8.codes.shape == (0, 512)
    x = randn(g, 64, 512, dtype=BF16)
    want = cb.rms_norm(x, weight).out
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = cb.rms_norm(x, weight, stream=side).out
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = cb.rms_norm(x, weight, residual=x, want="both")
    x.copy_(randn(g, 64, 512, dtype=BF16))
    graph.replay()
    again = cb.rms_norm(x, weight, residual=x, want="both")
    assert torch.equal(out.out, again.out) and torch.equal(out.fp8.scales, again.fp8.scales)
    assert torch.equal(out.fp8.codes.view(torch.uint8), again.fp8.codes.view(torch.uint8))


# ----------------------------------------------------------------- routing
def choose64(l, top_k, score, bias, groups, top_groups, group_score):
    """The documented order in 64 bits, one token at a time."""
    l = l.astype(np.float64)
    T, E = l.shape
    l = np.where(l == np.inf, np.finfo(np.float32).max, l)
    ids = np.zeros((T, top_k), np.int64)
    scores = np.zeros((T, E))
    for t in range(T):
        row = l[t]
        b = np.zeros(E) if bias is None else bias.astype(np.float64)
        nan, out = np.isnan(row) | np.isnan(b), row == -np.inf
        fine = ~np.isnan(row) & ~out
        s = np.full(E, np.nan)
        with np.errstate(over="ignore"):
            if score == "sigmoid":
                s[fine] = 1 / (1 + np.exp(-row[fine]))
            elif fine.any():
                e = np.exp(row[fine] - row[fine].max())
                s[fine] = e / e.sum()
        s[out & ~np.isnan(row)] = 0
        scores[t] = s
        c = s + b
        rank = np.where(nan, 1, np.where(out, 2, 3))
        allowed = np.ones(E, bool)
        if groups > 1:
            size = E // groups
            value = []
            for gi in range(groups):
                part = range(gi * size, (gi + 1) * size)
                by = row if bias is None and (group_score == "max" or size == 1) else c   # the logits' own order, as below
                v = sorted((by[e] for e in part if rank[e] == 3), reverse=True)
                value.append((0, 0.0) if not v else (1, v[0] if group_score == "max" or len(v) == 1 else v[0] + v[1]))
            order = sorted(range(groups), key=lambda i: (-value[i][0], -value[i][1], i))[:top_groups]
            allowed = np.isin(np.arange(E) // size, order)
        key = lambda e: (-rank[e], -c[e] if rank[e] == 3 else 0.0, e)  # noqa: E731
        if bias is None:    # the logits' own order, where 64 bits no longer tell the scores
            key = lambda e: (-rank[e], -row[e] if rank[e] == 3 else 0.0, e)  # noqa: E731
        ids[t] = sorted((e for e in range(E) if allowed[e]), key=key)[:top_k]
    return ids, scores


def weights64(l, ids, scores, renormalise, score, scale):
    l = np.where(l == np.inf, np.finfo(np.float32).max, l.astype(np.float64))
    w = np.take_along_axis(scores, ids, 1)
    if renormalise:
        chosen = np.take_along_axis(l, ids, 1)
        for t in range(len(w)):
            if np.isnan(w[t]).any():
                w[t] = np.nan
            elif (chosen[t] == -np.inf).all():
                w[t] = 0
            else:   # from the logits, so that nothing vanishes
                m = chosen[t].max()
                with np.errstate(over="ignore"):
                    e = w[t] if score == "sigmoid" and m > -600 else np.exp(chosen[t] - m)
                w[t] = e / e.sum()
    return w * scale


def check_route(l, top_k, bias=None, score="sigmoid", groups=1, top_groups=None, group_score="top2", renormalise=True, scale=1.0):
    ids, w = cb.route(l, top_k, score=score, bias=bias, groups=groups, top_groups=top_groups, group_score=group_score,
                      renormalise=renormalise, scale=scale)
    l64 = l.double().cpu().numpy()
    b64 = None if bias is None else bias.double().cpu().numpy()
    want, scores = choose64(l64, top_k, score, b64, groups, top_groups or groups, group_score)
    wrong = np.flatnonzero((ids.cpu().numpy() != want).any(1))
    assert ids.dtype == torch.int32 and not len(wrong), (wrong[:4], ids[wrong[0]].tolist(), want[wrong[0]].tolist())
    ww, got = weights64(l64, want, scores, renormalise, score, scale), w.double().cpu().numpy()
    finite = np.where(np.isfinite(l64), l64, np.nan)
    span = 0.0 if score == "sigmoid" or not np.isfinite(finite).any() else np.nanmax(finite) - np.nanmin(finite)
    tol = (16 if renormalise else 32) * EPS[F32] + (min(span, 200.0) * EPS[F32])
    assert np.array_equal(np.isnan(got), np.isnan(ww))
    far = np.nan_to_num(np.abs(got - ww)) > np.nan_to_num(tol * np.abs(ww)) + TINY
    assert not far.any(), (got[far][:4], ww[far][:4])


ROUTINGS = [  # experts, top, groups, top groups
    (1, 1, 1, 1), (8, 2, 1, 1), (16, 16, 1, 1), (37, 5, 1, 1), (64, 6, 8, 3), (96, 7, 6, 2), (60, 4, 4, 4), (128, 8, 4, 1),
    (160, 6, 8, 3), (256, 8, 8, 4), (256, 16, 1, 1), (255, 3, 5, 2), (32, 8, 32, 9), (256, 8, 32, 5), (200, 8, 2, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("experts,top,groups,top_groups", ROUTINGS)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_route_against_64_bits(experts, top, groups, top_groups, score, dtype):
    g = gen(experts * 31 + groups)
    l = randn(g, 203, experts, std=2.0, dtype=dtype)
    for i, bias in enumerate((None, randn(g, experts, std=0.1 if score == "sigmoid" else 0.01))):
        for group_score in ("top2", "max")[:2 if groups > 1 else 1]:
            check_route(l, top, bias, score, groups, top_groups, group_score, renormalise=(i == 0) == (group_score == "max"), scale=2.5)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_ties_and_near_ties(score):
    """Few distinct values, equal biases, and scores that 32 bits cannot tell apart."""
    g = gen(8)
    l = torch.randint(-2, 3, (64, 64), generator=g, device="cuda").float()
    for bias in (None, torch.zeros(64, device="cuda"), torch.randint(0, 2, (64,), generator=g, device="cuda").float() / 8):
        for groups, top_groups in ((1, 1), (8, 3)):
            check_route(l, 8, bias, score, groups, top_groups)
            check_route(l, 8, bias, score, groups, top_groups, "max")
    # logits a step or two of fp32 apart, the same bias: the order is still the logits'
    base = torch.full((40, 256), 0.7, device="cuda")
    steps = torch.randint(0, 5, (40, 256), generator=g, device="cuda", dtype=torch.int32)
    near = (base.view(torch.int32) + steps).view(F32)
    for bias in (None, torch.full((256,), 0.25, device="cuda")):
        for groups, top_groups in ((1, 1), (8, 4), (32, 7), (4, 1)):
            check_route(near, 8, bias, score, groups, top_groups, "max")
            check_route(near, 8, bias, score, groups, top_groups, "top2")
    # groups whose values meet, and values of one expert each that do
    twin = randn(g, 30, 64)
    twin[:, 16:32] = twin[:, :16]
    for bias in (None, torch.zeros(64, device="cuda")):
        for groups, top_groups in ((4, 1), (4, 2), (8, 3)):
            check_route(twin, 4, bias, score, groups, top_groups, "max")
            check_route(twin, 4, bias, score, groups, top_groups, "top2")
            check_route(twin.to(BF16), 4, bias, score, groups, top_groups, "top2")
    # biases that nearly undo the scores' differences
    s = 1 / (1 + torch.exp(-l.double()))
    if score == "softmax":
        s = torch.softmax(l.double(), -1)
    for t in range(0, 64, 9):
        check_route(l[t:t + 1], 8, (0.5 - s[t]).float(), score)
        check_route(l[t:t + 1], 4, (0.5 - s[t]).float(), score, 8, 3)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalise", [True, False])
def test_route_masks_and_what_is_no_number(score, dtype, renormalise):
    g = gen(3)
    l = randn(g, 24, 32, dtype=dtype)
    inf, lowest = float("inf"), torch.finfo(dtype).min
    l[0] = -inf                       # nothing left
    l[1, :30] = -inf                  # fewer than k left
    l[2, 3:] = -inf
    l[3] = lowest                     # a mask of the lowest value everywhere
    l[4, 5:] = lowest
    l[5] = float("nan")
    l[6, ::2] = float("nan")
    l[7, 4] = inf
    l[8, 4:9] = inf
    l[9] = inf
    l[10, :31] = -inf
    l[10, 31] = float("nan")
    l[11, :16] = -inf
    l[12] = -100.0 - torch.arange(32, device="cuda").to(dtype)   # scores that vanish in 32 bits
    l[13] = 100.0
    l[14, 1:] = -inf
    l[15, ::2] = -inf
    l[15, 1::4] = float("nan")
    for bias in (None, randn(g, 32, std=0.1)):
        for groups, top_groups, k in ((1, 1, 4), (1, 1, 16), (8, 2, 4), (8, 8, 5)):
            for group_score in ("top2", "max"):
                check_route(l, k, bias, score, groups, top_groups, group_score, renormalise)
    bias = torch.zeros(32, device="cuda")
    bias[3], bias[7], bias[9] = -inf, inf, float("nan")
    check_route(randn(g, 8, 32, dtype=dtype), 6, bias, score, renormalise=renormalise)


@pytest.mark.gpu
def test_route_strides_sizes_streams_graphs():
    g = gen(2)
    wide = randn(g, 3000, 300)
    check_route(wide[:, 3:131], 4, None, "softmax")
    check_route(wide[::7, 1:257], 8, randn(g, 256, std=0.1), "sigmoid", 8, 4)
    check_route(wide[:1, :128], 8, None)
    ids, w = cb.route(wide[:0, :64], 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)
    l = wide[:, :64].contiguous()
    want = cb.route(l, 6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = cb.route(l, 6, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = cb.route(l, 6)
    l.copy_(randn(g, 3000, 64))
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(out, cb.route(l, 6)))
    for kw in (dict(groups=5), dict(top_groups=2), dict(groups=8, top_groups=0)):
        with pytest.raises(cb.CbMoeError):
            cb.route(l, 6, **kw)


# ------------------------------------------------------- 4-bit weights in groups
def int4_weights(g, n, k, group, experts=None, zeros=True, scale=0.01):
    lead = () if experts is None else (experts,)
    codes = torch.randint(0, 256, (*lead, n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.rand((*lead, k // group, n), generator=g, device="cuda") * scale + scale / 2
    scales = scales * torch.where(torch.rand(scales.shape, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    z = torch.randint(0, 16, (*lead, k // group, n), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    return cb.Int4Matrix(codes, scales, z)


def int4_values(m, e=None):
    codes, scales = (m.codes, m.scales) if e is None else (m.codes[e], m.scales[e])
    q = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double()
    z = torch.full_like(scales, 8.0).double() if m.zeros is None else (m.zeros if e is None else m.zeros[e]).double()
    return (q - z.T.repeat_interleave(m.group, -1)) * scales.double().T.repeat_interleave(m.group, -1)


def fp8_rows(g, rows, cols):
    codes = randn(g, rows, cols, std=60.0).clamp(-448, 448).to(torch.float8_e4m3fn)
    return cb.Fp8Rows(codes, torch.rand((rows, -(-cols // 128)), generator=g, device="cuda") * 0.02 + 0.001)


def values_of(x):
    if isinstance(x, cb.Fp8Rows):
        return x.codes.view(torch.float8_e4m3fn).double() * x.scales.double().repeat_interleave(128, -1)[:, :x.cols]
    return x.double()


def int4_64(x, m, ids=None, weights=None, swiglu=False):
    """(result, the terms' magnitudes summed) in 64 bits, magnitudes as an error of the result."""
    v = values_of(x)
    loss = (8 + m.cols // m.group + 8 + 16) * 2.0 ** -22
    if ids is None:
        w = int4_values(m)
        y, mag = v @ w.T, v.abs() @ w.abs().T
    else:
        t, k = ids.shape
        rows = v.reshape(t, k, -1) if v.numel() == t * k * m.cols and (v.dim() == 3 or v.shape[0] != t) else v[:, None].expand(t, k, -1)
        y = torch.full((t, k, m.rows), float("nan"), dtype=torch.float64, device="cuda")
        mag = torch.zeros_like(y)
        for e in set(ids.flatten().tolist()):
            if 0 <= e < m.experts:
                a, b = torch.nonzero(ids == e, as_tuple=True)
                w = int4_values(m, e)
                y[a, b], mag[a, b] = rows[a, b] @ w.T, rows[a, b].abs() @ w.abs().T
    err = loss * mag
    if swiglu:
        (a, b), (ea, eb) = y.chunk(2, -1), err.chunk(2, -1)
        s = torch.sigmoid(a)
        y = a * s * b
        err = ea * 1.1 * b.abs() + (a * s).abs() * eb + ea * eb * 1.1 + 8 * EPS[F32] * y.abs()   # |silu'| < 1.1
    if weights is not None:
        w = weights.double()[..., None]
        err = (err * w.abs()).sum(1) + 16 * EPS[F32] * (y.abs() * w.abs()).sum(1)
        y = (y * w).sum(1)
    return y, err


def check_int4(x, m, **kw):
    dtype = kw.pop("dtype", BF16)
    got = cb.int4_matmul_few(x, m, dtype=dtype, **kw)
    want, err = int4_64(x, m, **kw)
    assert got.dtype == dtype and got.shape == want.shape
    nan = want.isnan()
    assert torch.equal(got.isnan(), nan)
    assert ((got.double() - want).abs()[~nan] <= (err + EPS[dtype] * (want.abs() + err) + TINY)[~nan]).all()
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("n,groups", [(16, 1), (48, 2), (96, 3), (512, 8), (1008, 5), (4096, 12)])
def test_int4_one_matrix(group, kind, n, groups):
    g = gen(group * 7 + n)
    k = group * groups
    m = int4_weights(g, n, k, group, zeros=n != 512)
    for rows in (1, 2, 5, 8, 9, 16):
        x = randn(g, rows, k, dtype=BF16) if kind == "bf16" else fp8_rows(g, rows, k)
        check_int4(x, m, dtype=F32)
        check_int4(x, m)
        if n % 32 == 0:
            check_int4(x, m, swiglu=True, dtype=F32 if rows % 2 else BF16)


@pytest.mark.gpu
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("experts,top,n,k", [(1, 1, 32, 256), (4, 2, 160, 384), (16, 3, 96, 640), (256, 8, 32, 128), (5, 16, 64, 256), (64, 6, 544, 1152)])
def test_int4_by_expert(group, kind, experts, top, n, k):
    g = gen(experts * 13 + group)
    m = int4_weights(g, n, k, group, experts)
    for rows in (1, 3, 8, 16):
        ids = torch.randint(0, experts, (rows, top), generator=g, device="cuda", dtype=torch.int32)   # experts may come twice
        w = randn(g, rows, top)
        x = randn(g, rows, k, dtype=BF16) if kind == "bf16" else fp8_rows(g, rows, k)
        slots = randn(g, rows, top, k, dtype=BF16) if kind == "bf16" else fp8_rows(g, rows * top, k)
        check_int4(x, m, ids=ids, dtype=F32)
        check_int4(x, m, ids=ids, swiglu=True)
        check_int4(x, m, ids=ids, weights=w, dtype=F32)
        check_int4(slots, m, ids=ids, weights=w)
        check_int4(slots, m, ids=ids, dtype=F32)


@pytest.mark.gpu
@pytest.mark.parametrize("n,k,group,kind,rows", [(80, 16384, 128, "bf16", (16, 9, 3)), (4128, 14336, 64, "fp8", (16, 8)),
                                                 (48, 65536, 64, "fp8", (5, 16)), (32, 53248, 32, "bf16", (16, 1)), (16, 393216, 128, "bf16", (2,))])
def test_int4_long_rows(n, k, group, kind, rows):
    """Rows of x that several blocks share."""
    g = gen(n)
    m = int4_weights(g, n, k, group)
    for r in rows:
        x = randn(g, r, k, dtype=BF16) if kind == "bf16" else fp8_rows(g, r, k)
        check_int4(x, m, dtype=F32)
        if n % 32 == 0:
            check_int4(x, m, swiglu=True)


@pytest.mark.gpu
@pytest.mark.parametrize("experts,k,group", [(3, 16384, 128), (2, 49152, 32)])
def test_int4_long_rows_by_expert(experts, k, group):
    g = gen(experts)
    m = int4_weights(g, 64, k, group, experts)
    for rows, top in ((16, 2), (3, 1)):
        ids = torch.randint(0, experts, (rows, top), generator=g, device="cuda", dtype=torch.int32)
        x = randn(g, rows, k, dtype=BF16)
        check_int4(x, m, ids=ids)
        check_int4(x, m, ids=ids, swiglu=True)
        check_int4(x, m, ids=ids, weights=randn(g, rows, top), dtype=F32)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,n,k,group,experts,top", [
    (12, 96, 2304, 32, 4, 2), (7, 736, 6656, 128, 4, 1), (16, 2048, 1408, 128, 64, 6), (16, 6400, 512, 64, 64, 8), (3, 16, 8192, 64, 2, 2)])
def test_int4_weighted_sum_by_clusters(rows, n, k, group, experts, top):
    """Few tiles of columns, whose experts and k several blocks share; and many, in rounds."""
    g = gen(rows * n)
    m = int4_weights(g, n, k, group, experts)
    ids = torch.randint(0, experts, (rows, top), generator=g, device="cuda", dtype=torch.int32)
    w, x = randn(g, rows, top), randn(g, rows, k, dtype=BF16)
    check_int4(x, m, ids=ids, weights=w, dtype=F32)
    check_int4(fp8_rows(g, rows * top, k), m, ids=ids, weights=w)
    got = cb.int4_matmul_few(x, m, ids=ids, weights=w)
    assert torch.equal(got, cb.int4_matmul_few(x, m, ids=ids, weights=w))
    ids[rows // 2, 0] = experts
    bad = cb.int4_matmul_few(x, m, ids=ids, weights=w)
    keep = torch.arange(rows, device="cuda") != rows // 2
    assert bad[rows // 2].isnan().all() and torch.isfinite(bad[keep].float()).all()
    check_int4(x, m, ids=ids, weights=w, dtype=F32)


@pytest.mark.gpu
def test_int4_sizes_of_x():
    """Large and small elements, up to the documented limits."""
    g = gen(14)
    m = int4_weights(g, 64, 512, 64)
    for power in (-30, -10, 0, 20, 50):
        check_int4((randn(g, 5, 512) * 2.0 ** power).to(BF16), m, dtype=F32)
    x = randn(g, 3, 512, dtype=BF16)
    x[1] = x[1] * 2.0 ** -100          # far below what can be told from 0
    got = cb.int4_matmul_few(x, m, dtype=F32)
    assert (got[1].abs() <= 512 * 15 * 0.02 * 2.0 ** -56).all()
    x[1, 7] = 2.0 ** 100
    got = cb.int4_matmul_few(x, m, dtype=F32)
    assert not got[1].isfinite().any() and got[[0, 2]].isfinite().all()


@pytest.mark.gpu
def test_int4_everyone_at_one_expert():
    g = gen(4)
    m = int4_weights(g, 64, 512, 64, 12)
    ids = torch.full((16, 16), 7, dtype=torch.int32, device="cuda")
    x = randn(g, 16, 512, dtype=BF16)
    check_int4(x, m, ids=ids)
    check_int4(x, m, ids=ids, weights=randn(g, 16, 16))


@pytest.mark.gpu
def test_int4_experts_that_do_not_exist():
    g = gen(6)
    m = int4_weights(g, 96, 384, 128, 6)
    x = randn(g, 4, 384, dtype=BF16)
    ids = torch.tensor([[0, 5], [6, 1], [2, -1], [3, 3]], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = cb.int4_matmul_few(x, m, ids=ids, status=status)
    want, _ = int4_64(x, m, ids)
    assert status.item() == cb.CB_ERR_DEVICE and torch.equal(got.isnan(), want.isnan())
    check_int4(x, m, ids=ids, weights=torch.ones(4, 2, device="cuda"))
    none = torch.full((4, 2), 99, dtype=torch.int32, device="cuda")
    assert cb.int4_matmul_few(x, m, ids=none).isnan().all()
    assert cb.int4_matmul_few(x, m, ids=none, weights=torch.ones(4, 2, device="cuda")).isnan().all()
    assert cb.int4_matmul_few(x, m, ids=none, swiglu=True).isnan().all()
    status.zero_()
    cb.int4_matmul_few(x, m, ids=ids.clamp(0, 5), status=status)
    assert status.item() == 0


@pytest.mark.gpu
def test_int4_strides_and_rows_left_alone():
    g = gen(9)
    m = int4_weights(g, 80, 256, 32)
    x = randn(g, 7, 512, dtype=BF16)[:, 128:384]
    out = torch.full((9, 100), 7.0, dtype=BF16, device="cuda")
    got = cb.int4_matmul_few(x, m, out=out[1:8, 5:85])
    assert torch.equal(got, cb.int4_matmul_few(x.contiguous(), m))
    assert (out[0] == 7).all() and (out[8] == 7).all() and (out[:, :5] == 7).all() and (out[:, 85:] == 7).all()
    with pytest.raises(cb.CbMoeError):
        cb.int4_matmul_few(randn(g, 4, 260, dtype=BF16)[:, :256], m)     # rows that do not start on 16 bytes
    with pytest.raises(cb.CbMoeError):
        cb.int4_matmul_few(randn(g, 17, 256, dtype=BF16), m)
    assert cb.int4_matmul_few(x[:0], m).shape == (0, 80)


@pytest.mark.gpu
def test_int4_one_row_has_no_stride():
    """A single row of a matrix whose rows do not start on 16 bytes is a row on 16 bytes like any other."""
    g = gen(77)
    m, by = int4_weights(g, 80, 256, 32), int4_weights(g, 48, 256, 32, 3)
    x = randn(g, 3, 261, dtype=BF16)[:1, :256]
    assert x.stride(0) == 261
    check_int4(x, m, dtype=F32)
    check_int4(x, by, ids=torch.tensor([[2, 0]], dtype=torch.int32, device="cuda"))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_int4_what_is_no_number_stays_in_its_row(kind):
    g = gen(10)
    m = int4_weights(g, 64, 512, 64)
    x = randn(g, 6, 512, dtype=BF16) if kind == "bf16" else fp8_rows(g, 6, 512)
    clean = cb.int4_matmul_few(x, m)
    if kind == "bf16":
        x[2, 100], x[4, 3] = float("nan"), float("inf")
    else:
        x.codes.view(torch.uint8)[2, 100] = 0x7F
        x.scales[4, 1] = float("nan")
    got = cb.int4_matmul_few(x, m)
    assert got[2].isnan().all() and not got[4].isfinite().any()
    assert torch.equal(got[[0, 1, 3, 5]], clean[[0, 1, 3, 5]])
    scales = m.scales.clone()
    scales[3, 17] = float("nan")
    again = cb.int4_matmul_few(x, cb.Int4Matrix(m.codes, scales, m.zeros))
    assert again[:, 17].isnan().all() and torch.equal(again[[0, 1, 3, 5]][:, :17], clean[[0, 1, 3, 5]][:, :17])
    assert torch.equal(again[[0, 1, 3, 5]][:, 18:], clean[[0, 1, 3, 5]][:, 18:])


@pytest.mark.gpu
def test_int4_streams_graphs_and_two_at_once():
    g = gen(11)
    m = int4_weights(g, 1024, 1024, 128, 8)
    x = randn(g, 6, 1024, dtype=BF16)
    ids = torch.randint(0, 8, (6, 2), generator=g, device="cuda", dtype=torch.int32)
    want = cb.int4_matmul_few(x, m, ids=ids, swiglu=True)
    sides = [torch.cuda.Stream() for _ in range(4)]
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
    got = [cb.int4_matmul_few(x, m, ids=ids, swiglu=True, stream=s) for s in sides for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(t, want) for t in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = cb.int4_matmul_few(x, m, ids=ids, swiglu=True)
    x.copy_(randn(g, 6, 1024, dtype=BF16))
    ids.copy_(torch.randint(0, 8, (6, 2), generator=g, device="cuda", dtype=torch.int32))
    graph.replay()
    assert torch.equal(out, cb.int4_matmul_few(x, m, ids=ids, swiglu=True))


@pytest.mark.gpu
@pytest.mark.parametrize("k", [256, 512, 640])
@pytest.mark.parametrize("rows", [1, 3, 16])
def test_int4_many_short_tiles_repeat(k, rows):
    """Warps that share a tile of a stage each, and are done with the next while one still adds this one's sums up."""
    g = gen(k + rows)
    m = int4_weights(g, 65536, k, 128)
    x = randn(g, rows, k, dtype=BF16)
    want = check_int4(x, m)
    assert all(torch.equal(cb.int4_matmul_few(x, m), want) for _ in range(40))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_int4_clusters_on_streams_and_in_graphs(kind):
    """Sums that blocks exchange, and a last stage of one group, several calls at once and replayed."""
    g = gen(12)
    k = 14368
    by, one = int4_weights(g, 160, k, 32, 4), int4_weights(g, 48, k, 32)
    x = randn(g, 12, k, dtype=BF16) if kind == "bf16" else fp8_rows(g, 12, k)
    ids = torch.randint(0, 4, (12, 2), generator=g, device="cuda", dtype=torch.int32)
    w = randn(g, 12, 2)
    want = [check_int4(x, by, ids=ids, weights=w), check_int4(x, one)]
    sides = [torch.cuda.Stream() for _ in range(4)]
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
    got = [(cb.int4_matmul_few(x, by, ids=ids, weights=w, stream=s), cb.int4_matmul_few(x, one, stream=s)) for s in sides for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, want[0]) and torch.equal(b, want[1]) for a, b in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b = cb.int4_matmul_few(x, by, ids=ids, weights=w), cb.int4_matmul_few(x, one)
    ids.copy_(ids.flip(0))
    w.copy_(w.flip(0) * 2)
    for _ in range(2):
        graph.replay()
    assert torch.equal(a, cb.int4_matmul_few(x, by, ids=ids, weights=w)) and torch.equal(b, want[1])


@pytest.mark.gpu
def test_int4_first_call_of_a_form_in_a_capture():
    """Nothing that a first launch asks the driver for is refused while a stream is captured."""
    g = gen(15)
    m = int4_weights(g, 64, 16384, 32)
    x = fp8_rows(g, 16, 16384)        # clusters; no other test takes this form
    out = torch.empty(16, 64, dtype=F32, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cb.int4_matmul_few(x, m, out=out)
    graph.replay()
    want, err = int4_64(x, m)
    assert ((out.double() - want).abs() <= err + EPS[F32] * want.abs() + TINY).all()


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """The last rows of arrays of more than 2^32 bytes."""
    g = gen(16)
    E, n, k = 256, 8192, 4352
    codes = torch.empty(E, n, k // 2, dtype=torch.uint8, device="cuda")     # 4.6 GB, of which two experts are used
    scales, zeros = torch.empty(E, k // 128, n, device="cuda"), torch.empty(E, k // 128, n, dtype=torch.uint8, device="cuda")
    for e in (0, E - 1):
        one = int4_weights(g, n, k, 128)
        codes[e], scales[e], zeros[e] = one.codes, one.scales, one.zeros
    m = cb.Int4Matrix(codes, scales, zeros)
    ids = torch.tensor([[0, E - 1], [E - 1, 0], [E - 1, E - 1]], dtype=torch.int32, device="cuda")
    x = randn(g, 3, k, dtype=BF16)
    check_int4(x, m, ids=ids, swiglu=True)
    check_int4(x, m, ids=ids, weights=randn(g, 3, 2))
    del m, codes, scales, zeros
    rows, cols = 540000, 4096                                               # 4.4 GB each
    x = torch.empty(rows, cols, dtype=BF16, device="cuda").normal_(generator=g)
    weight = torch.ones(cols, dtype=BF16, device="cuda")
    r = cb.rms_norm(x, weight, residual=x, want="both", sum=x)
    assert torch.isfinite(r.fp8.scales).all()
    last = cb.rms_norm(x[-3:].clone(), weight, want="both", eps=1e-6)
    assert torch.equal(r.out[-3:], last.out) or (r.out[-3:].float() - last.out.float()).abs().max() <= 0.02   # x is rounded in between
    assert torch.equal(r.fp8.scales[-3:] > 0, last.fp8.scales > 0)
    del r
    l = x.view(-1, 256)                                                     # 8.6 M tokens
    ids, w = cb.route(l, 6, groups=8, top_groups=3)
    for at in (slice(0, 50), slice(-50, None)):
        want, _ = choose64(l[at].double().cpu().numpy(), 6, "sigmoid", None, 8, 3, "top2")
        assert np.array_equal(ids[at].cpu().numpy(), want)


@pytest.mark.gpu
def test_launch_failures_are_reported(monkeypatch):
    g = gen(12)
    m = int4_weights(g, 64, 256, 64)
    x = randn(g, 2, 256, dtype=BF16)
    monkeypatch.setenv("CB_MOE_INJECT_FAULT", "launch")
    for call in (lambda: cb.int4_matmul_few(x, m), lambda: cb.rms_norm(x, torch.ones(256, device="cuda")), lambda: cb.route(x, 4)):
        with pytest.raises(cb.CbMoeError) as e:
            call()
        assert e.value.status == cb.CB_ERR_CUDA


@pytest.mark.gpu
def test_norm_routing_and_experts_together():
    """A decode step of a block as it is used: the norm writes 16-bit rows for the router and 8-bit rows for
    the experts, whose gate and up product, down product and weighted sum follow the routing."""
    g = gen(13)
    T, d, f, E, k = 5, 512, 384, 16, 4
    up, down = int4_weights(g, 2 * f, d, 128, E), int4_weights(g, d, f, 64, E)
    x, res, weight = randn(g, T, d, dtype=BF16), randn(g, T, d, dtype=BF16), (1 + randn(g, d, std=0.1)).to(BF16)
    wr, bias = randn(g, E, d, std=0.05, dtype=BF16), randn(g, E, std=0.05)

    def step():
        n = cb.rms_norm(x, weight, residual=res, want="both")
        ids, w = cb.route(n.out @ wr.T, k, bias=bias, groups=4, top_groups=2, scale=2.5)
        h = cb.int4_matmul_few(n.fp8, up, ids=ids, swiglu=True)
        return n, ids, w, h, cb.int4_matmul_few(h, down, ids=ids, weights=w)

    n, ids, w, h, out = step()
    check_norm(x, weight, res, n, 1e-6, "both")
    want, scores = choose64((n.out @ wr.T).double().cpu().numpy(), k, "sigmoid", bias.double().cpu().numpy(), 4, 2, "top2")
    assert np.array_equal(ids.cpu().numpy(), want)
    want_h, err = int4_64(n.fp8, up, ids, swiglu=True)
    assert ((h.double() - want_h).abs() <= err + EPS[BF16] * (want_h.abs() + err) + TINY).all()
    want_out, err = int4_64(h, down, ids, weights=w)
    assert ((out.double() - want_out).abs() <= err + EPS[BF16] * (want_out.abs() + err) + TINY).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    x.copy_(randn(g, T, d, dtype=BF16))
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(held[1:], step()[1:]))


@pytest.mark.gpu
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("n,k", [(28672, 4096), (65536, 640), (8192, 14336)], ids=["wide", "short", "clusters"])
def test_int4_without_zero_points_over_many_tiles(group, kind, n, k):
    """Each warp takes several tiles, so that stages which have held sums are read again: the 8s have to be there."""
    g = gen(n + group)
    m = int4_weights(g, n, k, group, zeros=False)
    for rows in (1, 8, 9, 15, 16):
        x = randn(g, rows, k, dtype=BF16) if kind == "bf16" else fp8_rows(g, rows, k)
        check_int4(x, m, dtype=F32)
        if rows > 8:
            check_int4(x, m, swiglu=True)


@pytest.mark.gpu
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_int4_without_zero_points_by_expert(group, kind):
    """Parts of 16 rows and fewer, several of them, by rows, SwiGLU and the weighted sum."""
    g = gen(group)
    n, k, experts = 28672, 768, 3
    m = int4_weights(g, n, k, group, experts, zeros=False)
    for rows, top in ((16, 1), (15, 2), (16, 3), (8, 2), (1, 2)):
        x = randn(g, rows, k, dtype=BF16) if kind == "bf16" else fp8_rows(g, rows, k)
        for ids in (torch.full((rows, top), 1, dtype=torch.int32, device="cuda"),
                    torch.randint(0, experts, (rows, top), generator=g, device="cuda", dtype=torch.int32)):
            check_int4(x, m, ids=ids, dtype=F32)
            check_int4(x, m, ids=ids, swiglu=True)
            check_int4(x, m, ids=ids, weights=randn(g, rows, top), dtype=F32)


@pytest.mark.gpu
@pytest.mark.parametrize("experts,groups,top_groups,top", [
    (8, 1, 1, 8), (32, 1, 1, 16), (64, 8, 3, 8), (64, 8, 8, 16), (256, 1, 1, 12), (256, 8, 4, 16), (256, 32, 5, 9)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_route_near_ties_beside_what_is_no_number(experts, groups, top_groups, top, score, dtype):
    """A few numbers a step apart (bf16: with scores far below the bias) among NaN and -inf, fewer than are chosen."""
    g = gen(experts + top)
    T, nan, inf = 60, float("nan"), float("inf")
    rand = lambda *s: torch.rand(s, generator=g, device="cuda")  # noqa: E731
    l = torch.where(rand(T, experts) < 0.5, nan, -inf)
    l[:20], l[20:40] = nan, -inf
    near = torch.full((T, experts), 0.5 if dtype is F32 else -12.0, dtype=dtype, device="cuda")
    bits = torch.int32 if dtype is F32 else torch.int16
    near = (near.view(bits) + torch.randint(0, 2, near.shape, generator=g, device="cuda").to(bits)).view(dtype)
    count = torch.randint(2, 7, (T, 1), generator=g, device="cuda")
    l = torch.where(rand(T, experts).argsort(-1).argsort(-1) < count, near.float(), l)
    if dtype is BF16:
        l[:, 0] = 0.0
    l = l.to(dtype)
    for bias in (None, torch.full((experts,), 0.9, device="cuda"), torch.full((experts,), -0.25, device="cuda")):
        for group_score in ("top2", "max")[:2 if groups > 1 else 1]:
            check_route(l, top, bias, score, groups, top_groups, group_score)
            check_route(l, top, bias, score, groups, top_groups, group_score, renormalise=False)


def nearly_level(g, T, experts, dtype, base):
    """Rows of one value, a few elements of which are a step away from it."""
    bits = torch.int32 if dtype is F32 else torch.int16
    l = torch.full((T, experts), base, dtype=dtype, device="cuda").view(bits)
    share = torch.tensor([0.0, 0.02, 0.1, 0.4], device="cuda")[torch.arange(T, device="cuda") % 4]
    return (l + (torch.rand((T, experts), generator=g, device="cuda") < share[:, None]).to(bits)).view(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("experts,groups,top_groups", [(8, 1, 1), (37, 1, 1), (64, 8, 2), (256, 1, 1), (256, 8, 4), (256, 32, 7)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_the_last_choice_among_equals_and_near_ones(experts, groups, top_groups, score):
    """Equal values at the last choice, and behind them one that is a step larger: it belongs before them."""
    g = gen(experts * 3 + groups)
    l = nearly_level(g, 120, experts, F32, 1.0)
    l[0, :3] = torch.tensor([1.0, 1.0, 1.0 + 2.0 ** -23], device="cuda")
    l[1] = 1.0
    l[1, experts - 1] = 1.0 + 2.0 ** -23
    low = nearly_level(g, 120, experts, F32, -12.0)                      # scores far below the bias
    low16 = nearly_level(g, 120, experts, BF16, -12.0)
    low[:, experts // 2], low16[:, experts // 2] = 0.0, 0.0
    steps = torch.full((experts,), 0.25, device="cuda")
    steps[experts // 3] += 2.0 ** -20
    for top in (1, 2, 3, 5):
        for group_score in ("top2", "max")[:2 if groups > 1 else 1]:
            for bias in (None, torch.full((experts,), 0.25, device="cuda"), steps):
                check_route(l, top, bias, score, groups, top_groups, group_score)
                check_route(low, top, bias, score, groups, top_groups, group_score)
                check_route(low16, top, bias, score, groups, top_groups, group_score)


@pytest.mark.gpu
@pytest.mark.parametrize("experts,top", [(8, 1), (8, 4), (256, 2), (256, 5)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_the_last_choice_beside_what_is_no_number(experts, top, score):
    g = gen(experts + top)
    l = nearly_level(g, 90, experts, F32, 0.5)
    rand = torch.rand(l.shape, generator=g, device="cuda")
    l[30:60] = torch.where(rand[30:60] < 0.7, float("nan"), l[30:60])
    l[60:] = torch.where(rand[60:] < 0.4, float("nan"), torch.where(rand[60:] < 0.8, -float("inf"), l[60:]))
    for bias in (None, torch.full((experts,), 0.9, device="cuda")):
        check_route(l, top, bias, score)
        check_route(l, top, bias, score, 4, 2)


@pytest.mark.gpu
@pytest.mark.parametrize("experts,groups", [(16, 4), (64, 32), (256, 32), (256, 8), (12, 3)])
@pytest.mark.parametrize("group_score", ["top2", "max"])
def test_route_experts_masked_by_their_bias(experts, groups, group_score):
    """A bias of -inf makes a choice the last of the numbers: behind it come experts and groups that are out."""
    g = gen(experts + groups)
    size = experts // groups
    l = randn(g, 40, experts)
    l[:, :size] = -float("inf")                           # the first group is out
    l[20:, size:2 * size] = float("nan")
    for masked in (size, size - 1):                       # of the last two groups all, or all but one
        bias = randn(g, experts, std=0.1)
        for last in (1, 2):
            at = experts - last * size
            bias[at:at + masked] = -float("inf")
        for top_groups in sorted({1, groups // 2, groups - 1, groups}):
            for top in sorted({1, min(size * top_groups, 4), min(size * top_groups, 16)}):
                for score in ("sigmoid", "softmax"):
                    check_route(l, top, bias, score, groups, top_groups, group_score)


def check_codes(r):
    """Codes of an fp32 result and its scales: the e4m3 nearest the fp32 quotient (a double quotient of two
    floats, rounded to fp32, is the rounded quotient), bit for bit."""
    rows, cols = r.out.shape
    s = r.fp8.scales.double().repeat_interleave(128, -1)[:, :cols]
    q = torch.where(s > 0, (r.out.double() / s.clamp_min(1e-300)).float().double(), 0.0)
    assert torch.equal(r.fp8.codes.view(torch.float8_e4m3fn).double(), e4m3_64(q))


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(1, 128), (40, 500), (3000, 1025), (700, 4096), (5000, 2048), (3000, 8192), (9, 16384)])
def test_norm_codes_are_the_nearest_of_the_quotient(rows, cols):
    """Quotients at and beside the borders between two codes: weights that are such borders, times what a row gives."""
    g = gen(rows + cols)
    step = torch.arange(8, 16, device="cuda", dtype=F32)
    border = torch.cat([(step[None] + 0.5) * torch.exp2(torch.arange(-9.0, 6.0, device="cuda"))[:, None],
                        (torch.arange(0, 8, device="cuda")[None] + 0.5) * 2.0 ** -9]).flatten()
    border = border[border < 448]
    weight = border[torch.randint(0, border.numel(), (cols,), generator=g, device="cuda")]
    weight[::128] = 448.0                             # the largest of each group
    x = randn(g, rows, 1) * (randn(g, rows, cols) > 0).float().mul(2).sub(1)      # a row's elements differ in sign alone
    for w in (weight, weight * 0.7, 1 + randn(g, cols, std=0.3)):
        check_codes(cb.rms_norm(x, w, want="both", eps=1e-12))
    check_codes(cb.rms_norm(x.to(BF16), weight, want="both", dtype=F32))
    check_codes(cb.rms_norm(randn(g, rows, cols), weight, residual=x, want="both"))
    check_codes(cb.rms_norm(x, weight * 1e-40, want="both"))                       # scales that are no normal numbers


@pytest.mark.gpu
def test_int4_ranges_of_x_and_of_the_scales():
    """What the header promises: x up to 2^64, scales up to 2^58, and NaN rows for infinite elements."""
    g = gen(23)
    for rows in (3, 16):
        m = int4_weights(g, 96, 512, 64)
        big = randn(g, rows, 512).clamp(-1.9, 1.9).to(BF16) * 2.0 ** 63
        check_int4(big, m, dtype=F32)
        for scale in (2.0 ** 57, 2.0 ** -100):
            for zeros in (True, False):
                check_int4((randn(g, rows, 512) * 2.0 ** -20).to(BF16), int4_weights(g, 96, 512, 64, zeros=zeros, scale=scale), dtype=F32)
        check_int4(fp8_rows(g, rows, 512), int4_weights(g, 96, 512, 64, scale=2.0 ** 57), dtype=F32)
        by = int4_weights(g, 96, 512, 64, 4)
        ids = torch.randint(0, 4, (rows, 2), generator=g, device="cuda", dtype=torch.int32)
        w = torch.ones(rows, 2, device="cuda")
        x = randn(g, rows, 512, dtype=BF16)
        clean = cb.int4_matmul_few(x, m), cb.int4_matmul_few(x, by, ids=ids), cb.int4_matmul_few(x, by, ids=ids, weights=w)
        x[1, 77], x[2, 5], x[2, 6] = -float("inf"), float("inf"), float("inf")
        got = cb.int4_matmul_few(x, m), cb.int4_matmul_few(x, by, ids=ids), cb.int4_matmul_few(x, by, ids=ids, weights=w)
        rest = [t for t in range(rows) if t not in (1, 2)]
        for a, b in zip(got, clean):
            assert a[[1, 2]].isnan().all() and torch.equal(a[rest], b[rest])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_route_weights_of_scores_far_below_the_largest(dtype):
    """Sigmoid scores that vanish in 32 bits beside larger ones that are small too: what remains after the division
    by their sum does not."""
    g = gen(31)
    l = randn(g, 120, 16, std=40.0) - torch.linspace(0, 100, 120, device="cuda")[:, None]
    l[0, :4] = torch.tensor([-20.0, -95.0, -59.5, -100.25], device="cuda")
    l[0, 4:] = -float("inf")
    l[1], l[2, 1:] = -90.0, -float("inf")
    for bias in (None, randn(g, 16) * 2):
        for top in (1, 2, 5, 16):
            check_route(l.to(dtype), top, bias, "sigmoid")
            check_route(l.to(dtype), top, bias, "sigmoid", scale=2.5)


@pytest.mark.gpu
@pytest.mark.parametrize("experts,groups", [(64, 16), (128, 32), (256, 16), (40, 8)])
@pytest.mark.parametrize("infinity", [-float("inf"), float("inf")], ids=["masked", "forced"])
def test_route_groups_of_infinite_values(experts, groups, infinity):
    """Groups whose values are infinite tie, whether one of their two best is or both; behind -inf come those that are out."""
    g = gen(experts + 7)
    l = randn(g, 30, experts)
    rand = torch.rand(l.shape, generator=g, device="cuda")
    l[10:20] = torch.where(rand[10:20] < 0.4, -float("inf"), l[10:20])
    l[20:] = torch.where(rand[20:] < 0.5, float("nan"), torch.where(rand[20:] < 0.7, -float("inf"), l[20:]))
    for share in (0.1, 0.3, 0.7):
        bias = torch.where(torch.rand((experts,), generator=g, device="cuda") < share, infinity, randn(g, experts, std=0.1))
        for top_groups in (1, groups // 2, groups - 3, groups):
            for score in ("sigmoid", "softmax"):
                for group_score in ("top2", "max"):
                    check_route(l, min(8, top_groups * experts // groups), bias, score, groups, top_groups, group_score)
