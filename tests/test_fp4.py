"""4-bit floats with block scales: quantisation, the way back, and the product, against their
definitions in 64 bits.

Quantisation and its way back are exact functions of their inputs, so codes, scales, padding and
values are compared bit for bit.  The product is compared bit for bit where every partial sum fits
fp32's 24 bits, whatever the order of the additions.  Elsewhere its tolerance counts roundings: a
tensor-core instruction adds 64 products to its accumulator and loses at most 2^-22 of the sum of
the magnitudes; a row of k elements is k / 64 of them, and the joins of up to 8 partial sums and
the two matrix scales are a few roundings more: (k / 64 + 12) 2^-22 of the sum of the terms'
magnitudes, then half a step of the output's type.
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
BLOCK = {"mx": 32, "nv": 16}
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
E4M3 = np.array([m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127])


# ------------------------------------------------------------------ no GPU
@pytest.fixture(scope="module")
def lib():
    cbuild.build()
    return cb.load_library()


def header():
    return open(os.path.join(ROOT, "include", "cb_fp4.h")).read()


def test_header_declares_what_the_library_exports(lib):
    declared = sorted(set(re.findall(r"CB_API\s+[\w\s\*]*?\b(cb_\w+)\s*\(", header())))
    assert declared == sorted(cb.FP4_SYMBOLS)
    raw = ctypes.CDLL(cb.LIB_PATH)
    assert all(hasattr(raw, name) for name in declared)
    enums = dict(re.findall(r"\b(CB_(?:FP4|T)_\w+)\s*=\s*(\d+)", header()))
    assert enums and all(getattr(cb, n) == int(v) for n, v in enums.items()), enums


def test_scale_bytes(lib):
    assert cb.cb_fp4_scale_bytes(0, 1, 32) == (cb.CB_OK, 512)
    assert cb.cb_fp4_scale_bytes(0, 128, 128) == (cb.CB_OK, 512)
    assert cb.cb_fp4_scale_bytes(0, 129, 160) == (cb.CB_OK, 2 * 2 * 512)
    assert cb.cb_fp4_scale_bytes(1, 129, 160) == (cb.CB_OK, 2 * 3 * 512)
    assert cb.cb_fp4_scale_bytes(1, 0, 64) == (cb.CB_OK, 0)
    for bad in ((2, 1, 32), (0, -1, 32), (0, 1, 0), (0, 1, 48), (0, 1, -32)):
        assert cb.cb_fp4_scale_bytes(*bad)[0] == cb.CB_ERR_INVALID_ARG
    assert lib.cb_fp4_scale_bytes(0, 1, 32, None) == cb.CB_ERR_INVALID_ARG


def test_quantiser_refuses_bad_arguments_before_cuda(lib):
    ok = dict(fmt=0, x=0x1000, typ=0, rows=4, cols=64, ld=64, g=None, codes=0x2000, scales=0x3000)

    def both(**kw):
        a = {**ok, **kw}
        return {cb.cb_fp4_quantize(a["fmt"], a["x"], a["typ"], a["rows"], a["cols"], a["ld"], a["g"], a["codes"], a["scales"]),
                cb.cb_fp4_dequantize(a["fmt"], a["codes"], a["scales"], a["g"], a["rows"], a["cols"], a["x"], a["typ"], a["ld"])}

    for kw in (dict(fmt=2), dict(fmt=-1), dict(typ=2), dict(rows=-1), dict(cols=0), dict(cols=40), dict(ld=63),
               dict(x=None), dict(codes=None), dict(scales=None), dict(g=64), dict(fmt=1), dict(x=0x2000),
               dict(x=0x3010), dict(codes=0x1010), dict(scales=0x2010), dict(x=0x1f00, ld=600)):
        assert both(**kw) == {cb.CB_ERR_INVALID_ARG}, kw
    for kw in (dict(x=0x1001), dict(typ=1, x=0x1002), dict(codes=0x2008), dict(scales=0x3008), dict(fmt=1, g=66)):
        assert both(**kw) == {cb.CB_ERR_ALIGNMENT}, kw
    for kw in (dict(cols=1 << 31, ld=1 << 31), dict(rows=1 << 60), dict(rows=1 << 36, cols=1 << 20, ld=1 << 20), dict(ld=1 << 61)):
        assert both(**kw) == {cb.CB_ERR_UNSUPPORTED}, kw
    assert both(rows=0, x=None, codes=None, scales=None) == {cb.CB_OK}


def product_args(**kw):
    a = dict(format=0, out_type=0, m=4, n=8, k=64, a_codes=0x10000, a_scales=0x20000, a_tensor_scale=None,
             b_codes=0x30000, b_scales=0x40000, b_tensor_scale=None, n_groups=1, tile_offsets=None, out=0x50000,
             ld_out=8, status=None)
    a.update(kw)
    return cb.cb_fp4_matmul_t(*(a[n] for n, _ in cb.cb_fp4_matmul_t._fields_))


def test_product_refuses_bad_arguments_before_cuda(lib):
    assert lib.cb_fp4_matmul(None, None) == cb.CB_ERR_INVALID_ARG
    for kw in (dict(format=2), dict(out_type=3), dict(m=-1), dict(n=-1), dict(k=0), dict(k=40), dict(ld_out=7),
               dict(a_codes=None), dict(a_scales=None), dict(b_codes=None), dict(b_scales=None), dict(out=None),
               dict(a_tensor_scale=64), dict(b_tensor_scale=64), dict(format=1), dict(format=1, a_tensor_scale=64),
               dict(n_groups=0), dict(n_groups=2), dict(out=0x10000), dict(out=0x30000), dict(out=0x20000),
               dict(out=0x40010)):
        assert cb.cb_fp4_matmul(product_args(**kw)) == cb.CB_ERR_INVALID_ARG, kw
    for kw in (dict(a_codes=0x10008), dict(b_codes=0x30004), dict(a_scales=0x20008), dict(b_scales=0x40004),
               dict(out=0x50002), dict(tile_offsets=0x60002), dict(status=0x60001),
               dict(format=1, a_tensor_scale=0x60002, b_tensor_scale=0x60000)):
        assert cb.cb_fp4_matmul(product_args(**kw)) == cb.CB_ERR_ALIGNMENT, kw
    for kw in (dict(m=1 << 31), dict(n=1 << 31, ld_out=1 << 31), dict(k=1 << 31),
               dict(n=1 << 21, ld_out=1 << 21, n_groups=1024, tile_offsets=0x60000)):
        assert cb.cb_fp4_matmul(product_args(**kw)) == cb.CB_ERR_UNSUPPORTED, kw
    for kw in (dict(m=0), dict(n=0)):
        assert cb.cb_fp4_matmul(product_args(**kw)) == cb.CB_OK, kw


def test_python_refusals(lib):
    with pytest.raises(ValueError):
        cb.fp4_quantize(torch.zeros(2, 64), "e2m1")
    with pytest.raises(ValueError):
        cb.fp4_quantize(torch.zeros(2, 64, dtype=torch.float16), "mx")
    with pytest.raises(ValueError):
        cb.fp4_quantize(torch.zeros(2, 64), "mx")                       # not on a GPU
    u = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    m = cb.Fp4Matrix("mx", 2, 64, u(2, 32), u(512))
    assert m.groups == 1
    for args in (("mx", 2, 64, u(2, 16), u(512)), ("mx", 2, 64, u(2, 32), u(511)), ("nv", 2, 64, u(2, 32), u(512)),
                 ("mx", 2, 64, u(2, 32), u(512), torch.ones(1)), ("mx", 2, 64, u(2, 64)[:, ::2], u(512))):
        with pytest.raises(ValueError):
            cb.Fp4Matrix(*args)
    with pytest.raises(cb.CbMoeError):
        cb.Fp4Matrix("mx", 2, 40, u(2, 20), u(512))
    class Elsewhere:
        device = "cuda:1"

        def get_device(self):
            return 1

    for t in (torch.zeros(2), Elsewhere()):
        with pytest.raises(ValueError):
            cb._check_device(0, None, t)
    cb._check_device(1, None, Elsewhere())
    with pytest.raises(ValueError):
        cb.fp4_matmul(m, cb.Fp4Matrix("mx", 2, 96, u(2, 48), u(512)))
    with pytest.raises(ValueError):
        cb.fp4_matmul(m, cb.Fp4Matrix("nv", 2, 64, u(2, 32), u(512), torch.ones(1)))


# ----------------------------------------------------------- definitions
def nearest(grid, v):
    """Index of the grid value nearest to each v >= 0, ties to the even index, past the end the last."""
    i = np.clip(np.searchsorted(grid, v), 1, len(grid) - 1)
    low, high = v - grid[i - 1], grid[i] - v
    return np.where((low < high) | ((low == high) & ((i - 1) % 2 == 0)), i - 1, i)


def quantise64(x, fmt, g):
    """Codes [rows][cols] and scale bytes [rows][blocks] of float64 x holding fp32 values."""
    v = x.reshape(x.shape[0], -1, BLOCK[fmt])
    top = np.abs(v).max(-1)
    finite = np.isfinite(v).all(-1)
    top = np.where(finite, top, 0)
    with np.errstate(all="ignore"):
        if fmt == "mx":
            byte = np.clip(np.where(top > 0, np.frexp(top)[1] - 1 - 2 + 127, 0), 0, 252)
            unit = np.ldexp(1.0, byte - 127)
        else:
            byte = nearest(E4M3, top / (6 * g))
            unit = E4M3[byte] * g
        w = np.where(unit[..., None] > 0, np.abs(v) / unit[..., None], 0)
    code = np.where(finite[..., None], nearest(E2M1, np.nan_to_num(w, nan=0, posinf=7)), 0)
    byte = np.where(finite, byte, 255 if fmt == "mx" else 127)
    return code.reshape(x.shape), byte.astype(np.uint8)


def tile(scales):
    r, c = -(-scales.shape[0] // 128), -(-scales.shape[1] // 4)
    out = np.zeros((r, c, 32, 4, 4), np.uint8)
    for i, j in np.ndindex(scales.shape):
        out[i // 128, j // 4, i % 32, i // 32 % 4, j % 4] = scales[i, j]
    return out.ravel()


def decode64(m, fmt, e=None):
    """An Fp4Matrix's values (one of its groups) without its own scale, in 64 bits."""
    codes = (m.codes if e is None else m.codes[e]).cpu().numpy()
    scales = m.scales.view(m.groups, -1)[0 if e is None else e].cpu().numpy()
    c = np.stack([codes & 15, codes >> 4], -1).reshape(m.rows, m.cols)
    v = E2M1[c & 7] * np.where(c & 8, -1.0, 1.0)
    blocks = m.cols // BLOCK[fmt]
    s = scales.reshape(-1, -(-blocks // 4), 32, 4, 4).transpose(0, 3, 2, 1, 4)
    s = s.reshape(s.shape[0] * 128, -1)[:m.rows, :blocks].astype(int)
    s = np.ldexp(1.0, s - 127) if fmt == "mx" else E4M3[s]
    return v * s.repeat(BLOCK[fmt], -1)


def dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)


def check_quantised(x, fmt, g=None):
    """x (CUDA tensor) through the library and the definition."""
    scale = None if g is None else torch.tensor([g], dtype=torch.float32, device="cuda")
    m = cb.fp4_quantize(x, fmt, scale)
    g64 = None if g is None else float(scale.double().item())
    v = x.double().cpu().numpy()
    code, byte = quantise64(v, fmt, g64)
    got = m.codes.cpu().numpy()
    got = np.stack([got & 15, got >> 4], -1).reshape(x.shape)
    assert np.array_equal(m.scales.cpu().numpy(), tile(byte))
    assert np.array_equal(got & 7, code)
    negative = v < 0
    assert np.array_equal((got >> 3)[code > 0] == 1, negative[code > 0])
    return m, code, byte


# -------------------------------------------------------------- quantiser
@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 4096), (3, 96), (16, 512), (127, 160), (129, 256), (300, 288), (257, 1184)])
def test_quantise_matches_the_definition(fmt, dtype, rows, cols):
    rng = np.random.default_rng(rows * cols)
    x = rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((rows, 1)) * 2)
    x = dev(x, dtype)
    g = None if fmt == "mx" else float(x.abs().max()) / (6 * 448)
    m, code, byte = check_quantised(x, fmt, g)
    assert (code > 0).mean() > 0.5
    for out_type in (torch.float32, torch.bfloat16):
        want = torch.from_numpy(decode64(m, fmt)).float()
        if g is not None:
            want = want * m.tensor_scale.cpu()
        got = cb.fp4_dequantize(m, out_type)
        assert torch.equal(got.cpu(), want.to(out_type))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("g", [1.0, 0.25, 1 / 3])
def test_ties_and_borders(fmt, dtype, g):
    """Values on the borders of e2m1 and e4m3, and one step to each side of them."""
    top = 6.0 * 2.0 ** np.arange(-6, 6)[:, None] * (1 + np.arange(8) / 16)[None]      # block maxima, on e4m3 borders
    marks = np.array([0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 5.5, 6])
    scale = top.ravel()[:, None] / 6 * (g if fmt == "nv" else 1)
    rows = []
    for off in (-1, 0, 1):
        v = torch.from_numpy(marks[None] * scale).to(dtype)
        bits = v.view(torch.int16 if dtype == torch.bfloat16 else torch.int32)
        v = torch.where(v > 0, (bits + off).view(dtype), v)
        v[:, -1] = torch.from_numpy(top.ravel() * (g if fmt == "nv" else 1)).to(dtype)
        rows += [v, -v]
    x = torch.cat(rows)
    x = torch.cat([x, x.flip(0)], 1).contiguous().cuda()         # 32 columns
    check_quantised(x, fmt, g if fmt == "nv" else None)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_extreme_magnitudes(fmt):
    rng = np.random.default_rng(4)
    rows = [rng.standard_normal(64) * s for s in (1e-45, 1e-42, 1e-38, 1e-30, 1e-3, 1e30, 1e38)]
    rows += [np.zeros(64), np.r_[np.zeros(63), 1e-45], np.full(64, 3.4028234663852886e38), np.full(64, 2.0 ** -126)]
    x = dev(np.clip(np.stack(rows), -3.4028234663852886e38, 3.4028234663852886e38), torch.float32)
    for g in ([None] if fmt == "mx" else [1.0, 1e-38, 2.0 ** -100, 1e-10, 1e30, 1e37]):
        check_quantised(x, fmt, g)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_blocks_that_are_not_finite(fmt):
    """A NaN or an infinity turns its own block, and nothing else, into NaN."""
    x = torch.randn(5, 128, device="cuda")
    x[1, 3], x[2, 70], x[4, 127] = float("nan"), float("inf"), float("-inf")
    m, _, byte = check_quantised(x, fmt, None if fmt == "mx" else 0.01)
    y = cb.fp4_dequantize(m, torch.float32)
    bad = torch.zeros_like(x, dtype=torch.bool).view(5, -1, BLOCK[fmt])
    for r, c in ((1, 3), (2, 70), (4, 127)):
        bad[r, c // BLOCK[fmt]] = True
    assert torch.equal(torch.isnan(y), bad.view(5, 128))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pitch,offset", [(167, 0), (168, 8), (161, 1), (192, 3)])
def test_strided_rows(dtype, pitch, offset):
    """Rows at any stride and start are read and written alike; the gaps between them stay."""
    base = torch.randn(40, pitch, device="cuda").to(dtype)
    x = base[:, offset:offset + 160] if offset + 160 <= pitch else base.view(-1)[offset:offset + 39 * pitch + 160].as_strided((40, 160), (pitch, 1))
    m, _, _ = check_quantised(x, "mx")
    plain = cb.fp4_dequantize(m, dtype)
    out = torch.full((40, pitch), 9.0, device="cuda", dtype=dtype)
    view = out.as_strided((40, 160), (pitch, 1), 0)
    cb.fp4_dequantize(m, out=view)
    assert torch.equal(view, plain)
    if pitch > 160:
        assert (out.as_strided((39, pitch - 160), (pitch, 1), 160) == 9.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_every_code_and_scale_reads_back(fmt):
    bytes_ = np.arange(255 if fmt == "mx" else 127)
    n = len(bytes_)
    codes = np.tile(np.arange(256, dtype=np.uint8)[:16], (n, 1))
    codes = np.stack([(np.arange(16) | (np.roll(np.arange(16), 3) << 4)).astype(np.uint8)] * n)   # 32 columns
    s = np.tile(bytes_[:, None], (1, 32 // BLOCK[fmt])).astype(np.uint8)
    m = cb.Fp4Matrix(fmt, n, 32, torch.from_numpy(codes).cuda(), torch.from_numpy(tile(s)).cuda(),
                     torch.ones(1, device="cuda") if fmt == "nv" else None)
    got = cb.fp4_dequantize(m, torch.float32).double().cpu().numpy()
    with np.errstate(over="ignore"):
        want = decode64(m, fmt).astype(np.float32).astype(np.float64)
    assert np.array_equal(got, want)


# ---------------------------------------------------------------- product
def random_matrix(rng, rows, cols, fmt, exact, groups=None):
    """Any codes; `exact`: scales of 1 and 2 (or 1.5), else over a wide range."""
    lead = () if groups is None else (groups,)
    codes = torch.from_numpy(rng.integers(0, 256, lead + (rows, cols // 2), dtype=np.uint8)).cuda()
    blocks = cols // BLOCK[fmt]
    if fmt == "mx":
        pick = np.array([127, 128]) if exact else np.arange(112, 140)
    else:
        pick = np.array([0x38, 0x3C]) if exact else np.arange(1, 0x7F)
    parts = [tile(pick[rng.integers(0, len(pick), (rows, blocks))].astype(np.uint8)) for _ in range(groups or 1)]
    scale = None
    if fmt == "nv":
        scale = np.ones(groups or 1) if exact else rng.uniform(0.001, 0.01, groups or 1)
        scale = torch.from_numpy(scale).float().cuda()
    return cb.Fp4Matrix(fmt, rows, cols, codes, torch.from_numpy(np.concatenate(parts)).cuda(), scale)


def expected(a, b, fmt, e=None, rows=slice(None)):
    x, y = decode64(a, fmt)[rows], decode64(b, fmt, e)
    g = 1.0 if fmt == "mx" else float(a.tensor_scale.double()) * float(b.tensor_scale.double()[e or 0])
    return g * (x @ y.T), g * (np.abs(x) @ np.abs(y).T)


def check_product(got, ref, mag, k):
    got64 = got.double().cpu().numpy()
    step = torch.finfo(got.dtype).eps / 2
    tol = (k / 64 + 12) * 2.0 ** -22 * mag
    assert np.all(np.abs(got64 - ref) <= tol + step * (np.abs(ref) + tol)), np.max(np.abs(got64 - ref) / (mag + 1e-300))


SIZES = [(1, 1, 32), (1, 128, 64), (1, 1000, 4096), (2, 130, 96), (16, 256, 256), (17, 300, 1184), (33, 64, 2048),
         (64, 129, 288), (65, 500, 800), (128, 256, 1024), (129, 1, 32), (129, 257, 160), (200, 8, 4096),
         (256, 384, 512), (333, 1000, 1184), (1500, 700, 96)]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_product_is_exact_where_its_sums_are(fmt, m, n, k):
    """Products of scales 1, 2 (1.5) and e2m1 values are multiples of 1/16 whose sums stay below 2^20."""
    rng = np.random.default_rng(m + n + k)
    a, b = random_matrix(rng, m, k, fmt, True), random_matrix(rng, n, k, fmt, True)
    ref, mag = expected(a, b, fmt)
    assert mag.max() < 2.0 ** 20
    got = cb.fp4_matmul(a, b, dtype=torch.float32)
    assert np.array_equal(got.double().cpu().numpy(), ref)
    assert torch.equal(cb.fp4_matmul(a, b), torch.from_numpy(ref).to(torch.bfloat16).cuda())


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("m,n,k", SIZES + [(3, 256, 14336), (700, 300, 14336), (40, 4096, 4096), (2048, 1024, 512)])
def test_product_within_its_roundings(fmt, m, n, k):
    rng = np.random.default_rng(m * n + k)
    a, b = random_matrix(rng, m, k, fmt, False), random_matrix(rng, n, k, fmt, False)
    ref, mag = expected(a, b, fmt)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        check_product(cb.fp4_matmul(a, b, dtype=dtype, status=status), ref, mag, k)
    assert int(status) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("counts,n,k", [([128], 64, 64), ([1, 0, 300, 129], 200, 160), ([0, 0, 5], 128, 512),
                                        ([0, 0], 64, 64), ([70] * 20 + [0] * 5 + [600], 384, 1184)])
def test_experts_products(fmt, counts, n, k):
    rng = np.random.default_rng(len(counts) + n)
    ends = np.r_[0, np.cumsum([-(-c // 128) for c in counts])]
    m = int(ends[-1]) * 128 + 40      # rows past the last expert's: not touched
    a = random_matrix(rng, m, k, fmt, True)
    b = random_matrix(rng, n, k, fmt, True, groups=len(counts))
    offsets = torch.from_numpy(ends.astype(np.int32)).cuda()
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.full((m, n), 7.0, dtype=dtype, device="cuda")
        cb.fp4_matmul(a, b, out=out, tile_offsets=offsets)
        for e in range(len(counts)):
            rows = slice(int(ends[e]) * 128, int(ends[e + 1]) * 128)
            if rows.stop > rows.start:
                ref, _ = expected(a, b, fmt, e, rows)
                assert torch.equal(out[rows], torch.from_numpy(ref).to(dtype).cuda()), e
        assert (out[int(ends[-1]) * 128:] == 7.0).all()


# sizes of 152 tiles of 128 x 256 and more: odd numbers of 128-row tiles, ends inside each kind of
# tile, rows of 8 bytes and of 16, k inside and past a stage of 256
LARGE = [(2432, 2304, 96), (2500, 4008, 544), (5100, 1030, 1184), (129, 20000, 32), (19600, 130, 288), (4100, 4097, 256)]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("m,n,k", LARGE)
def test_large_products_are_exact(fmt, m, n, k):
    """As above, against 64-bit products on the GPU."""
    rng = np.random.default_rng(m + n + k)
    a, b = random_matrix(rng, m, k, fmt, True), random_matrix(rng, n, k, fmt, True)
    x, y = (torch.from_numpy(decode64(t, fmt)).cuda() for t in (a, b))
    ref = x @ y.T
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.full((m, n + 24), 7.0, dtype=dtype, device="cuda")
        cb.fp4_matmul(a, b, out=out[:, :n], status=status)
        assert torch.equal(out[:, :n], ref.to(dtype)) and (out[:, n:] == 7.0).all()
    assert int(status) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_many_experts_products_are_exact(fmt):
    rng = np.random.default_rng(8)
    counts, n, k = [130, 0, 5, 700, 128, 1] * 5, 2100, 416
    ends = np.r_[0, np.cumsum([-(-c // 128) for c in counts])]
    a, b = random_matrix(rng, int(ends[-1]) * 128, k, fmt, True), random_matrix(rng, n, k, fmt, True, groups=len(counts))
    got = cb.fp4_matmul(a, b, dtype=torch.float32, tile_offsets=torch.from_numpy(ends.astype(np.int32)).cuda())
    x = torch.from_numpy(decode64(a, fmt)).cuda()
    for e in range(len(counts)):
        rows = slice(int(ends[e]) * 128, int(ends[e + 1]) * 128)
        assert torch.equal(got[rows].double(), x[rows] @ torch.from_numpy(decode64(b, fmt, e)).cuda().T), e


@pytest.mark.gpu
def test_tensors_on_several_devices_are_refused():
    x = torch.randn(4, 64, device="cuda")
    m, u = cb.fp4_quantize(x, "mx"), cb.fp4_quantize(x, "nv", torch.ones(1, device="cuda"))
    on_cpu = cb.Fp4Matrix("mx", 4, 64, m.codes.cpu(), m.scales.cpu())
    for call in (lambda: cb.Fp4Matrix("mx", 4, 64, m.codes, m.scales.cpu()),
                 lambda: cb.Fp4Matrix("nv", 4, 64, u.codes, u.scales, u.tensor_scale.cpu()),
                 lambda: cb.fp4_quantize(x, "nv", torch.ones(1)), lambda: cb.fp4_dequantize(m, out=torch.zeros(4, 64)),
                 lambda: cb.fp4_matmul(m, on_cpu), lambda: cb.fp4_matmul(on_cpu, m),
                 lambda: cb.fp4_matmul(m, m, out=torch.zeros(4, 4))):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
def test_one_expert_of_few_rows_and_short_a():
    """tile_offsets may name more tiles than A has rows for: rows past m are not written."""
    rng = np.random.default_rng(1)
    a, b = random_matrix(rng, 100, 96, "nv", True), random_matrix(rng, 40, 96, "nv", True, groups=1)
    out = cb.fp4_matmul(a, b, dtype=torch.float32, tile_offsets=torch.tensor([0, 3], dtype=torch.int32, device="cuda"))
    assert np.array_equal(out.double().cpu().numpy(), expected(a, b, "nv", 0)[0])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m", [5, 130])
def test_output_with_a_row_stride(dtype, m):
    rng = np.random.default_rng(m)
    a, b = random_matrix(rng, m, 160, "mx", True), random_matrix(rng, 77, 160, "mx", True)
    want = cb.fp4_matmul(a, b, dtype=dtype)
    for pitch in (80, 83, 128):
        out = torch.full((m, pitch), 3.0, dtype=dtype, device="cuda")
        cb.fp4_matmul(a, b, out=out[:, :77])
        assert torch.equal(out[:, :77], want) and (out[:, 77:] == 3.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("m", [3, 140])
def test_a_nan_block_reaches_its_own_row_only(fmt, m):
    x, w = torch.randn(m, 192, device="cuda"), torch.randn(70, 192, device="cuda")
    x[1, 100] = float("nan")
    w[5, 191] = float("inf")
    g = None if fmt == "mx" else torch.tensor([0.002], device="cuda")
    y = cb.fp4_matmul(cb.fp4_quantize(x, fmt, g), cb.fp4_quantize(w, fmt, g), dtype=torch.float32)
    want = torch.zeros(m, 70, dtype=torch.bool, device="cuda")
    want[1], want[:, 5] = True, True
    assert torch.equal(torch.isnan(y), want)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [4, 200])
def test_other_stream_and_graph(m):
    x = torch.randn(m, 1024, device="cuda").bfloat16()
    w = cb.fp4_quantize(torch.randn(512, 1024, device="cuda").bfloat16(), "mx")
    want = cb.fp4_matmul(cb.fp4_quantize(x, "mx"), w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = cb.fp4_matmul(cb.fp4_quantize(x, "mx", stream=side), w, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = cb.fp4_matmul(cb.fp4_quantize(x, "mx"), w)
    x.copy_(x.flip(0))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want.flip(0))


@pytest.mark.gpu
def test_zero_rows():
    x = torch.empty(0, 64, device="cuda")
    m = cb.fp4_quantize(x, "mx")
    w = cb.fp4_quantize(torch.randn(3, 64, device="cuda"), "mx")
    assert cb.fp4_dequantize(m).shape == (0, 64)
    assert cb.fp4_matmul(m, w).shape == (0, 3) and cb.fp4_matmul(w, m).shape == (3, 0)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """A matrix of more than 2^32 elements: its last rows go through as a small matrix's do."""
    rows, cols = 300000, 14336
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-200:] = torch.randn(200, cols, device="cuda").bfloat16()
    big, small = cb.fp4_quantize(x, "mx"), cb.fp4_quantize(x[-200:], "mx")
    assert torch.equal(big.codes[-200:], small.codes) and int(big.codes[:-200].max()) == 0
    back = cb.fp4_dequantize(big)
    assert torch.equal(back[-200:], cb.fp4_dequantize(small))
    w = cb.fp4_quantize(torch.randn(24, cols, device="cuda").bfloat16(), "mx")
    del x, back
    assert torch.equal(cb.fp4_matmul(big, w)[-128:], cb.fp4_matmul(small, w)[-128:])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("top", [0.0, 2.0 ** -140])
@pytest.mark.parametrize("rows,cols", [(3, 96), (140, 320)])
def test_nv_scale_of_zeros(dtype, top, rows, cols):
    """max|x| / (6 * 448) is 0 for zeros, and for values that it cannot tell from them: zeros
    throughout, and a product with them is 0; a block that is not finite is NaN as ever."""
    x = torch.full((rows, cols), top, device="cuda").to(dtype)
    g = (x.float().abs().amax() / (6 * 448)).reshape(1)
    assert float(g) == 0.0
    q = cb.fp4_quantize(x, "nv", g)
    assert int(q.codes.max()) == 0 and int(q.scales.max()) == 0
    assert torch.equal(cb.fp4_dequantize(q, dtype), torch.zeros_like(x))
    w = cb.fp4_quantize(torch.randn(40, cols, device="cuda"), "nv", torch.tensor([0.002], device="cuda"))
    for a, b, shape in ((q, w, (rows, 40)), (w, q, (40, rows))):
        assert torch.equal(cb.fp4_matmul(a, b), torch.zeros(shape, dtype=torch.bfloat16, device="cuda"))
    x[1, 40] = float("nan")
    y = cb.fp4_dequantize(cb.fp4_quantize(x, "nv", g), torch.float32)
    want = torch.zeros_like(x, dtype=torch.bool)
    want[1, 32:48] = True
    assert torch.equal(torch.isnan(y), want)


@pytest.mark.gpu
@pytest.mark.parametrize("ga,gb", [(0.01, 0.003), (1e-23, 1e-23), (1e-23, -1e-23), (1e20, 1e20), (3e38, 3e38), (1e-40, 1e-5),
                                   (2.0 ** -140, 2.0 ** -100), (1e-45, 1e-45), (0.0, 1e30), (1e-30, 1e37)])
@pytest.mark.parametrize("m,n,k,gap", [(4, 130, 160, 0), (200, 256, 96, 0), (200, 77, 96, 0), (2500, 1030, 96, 2), (2500, 2000, 1024, 0),
                                       (2500, 2001, 1024, 0)])
def test_matrix_scales_whose_product_leaves_fp32(m, n, k, gap, ga, gb):
    """The sums themselves are exact here.  Rounded after them: the product of the two scales and the
    scaled sum to fp32 (a smallest step apart at most where it is not normal), then to the output's
    type.  Sums of 0 stay 0, whatever the scales."""
    rng = np.random.default_rng(m + n + k)
    a, b = random_matrix(rng, m, k, "nv", True), random_matrix(rng, n, k, "nv", True)
    a.codes[1] = 0
    sums = torch.from_numpy(decode64(a, "nv")).cuda() @ torch.from_numpy(decode64(b, "nv")).cuda().T
    a.tensor_scale.fill_(ga)
    b.tensor_scale.fill_(gb)
    ref = sums * (a.tensor_scale.double() * b.tensor_scale.double())
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.empty((m, n + gap), dtype=dtype, device="cuda")[:, :n]
        got = cb.fp4_matmul(a, b, out=out).double()
        step, tiny = torch.finfo(dtype).eps / 2, 2.0 ** -149 + (2.0 ** -134 if dtype == torch.bfloat16 else 0)
        tol = ref.abs() * (step + 3 * 2.0 ** -24) + tiny
        top = torch.finfo(dtype).max
        past, within = ref.abs() > top + tol, ref.abs() < top - tol
        assert ((got - ref).abs() <= tol)[within].all()
        assert torch.equal(got[past], torch.copysign(torch.full_like(ref, float("inf")), ref)[past])
        assert (got[1] == 0).all()


# ------------------------------------------- forms that only large matrices take
def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def nearest_on_gpu(grid, v):
    """nearest() as torch operations, in 64 bits."""
    g = torch.tensor(grid, dtype=torch.float64, device=v.device)
    i = torch.searchsorted(g, v.contiguous()).clamp_(1, len(g) - 1)
    low, high = v - g[i - 1], g[i] - v
    return torch.where((low < high) | ((low == high) & ((i - 1) % 2 == 0)), i - 1, i)


def two_to(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def quantise_on_gpu(x, fmt, g):
    """quantise64() as torch operations: codes, and scale bytes in their stored order."""
    v = x.double().view(x.shape[0], -1, BLOCK[fmt])
    finite = torch.isfinite(v).all(-1)
    v = torch.where(finite[..., None], v, 0.0)
    top = v.abs().amax(-1)
    if fmt == "mx":
        byte = torch.where(top > 0, torch.frexp(top).exponent.long() - 1 - 2 + 127, 0).clamp(0, 252)
        unit = two_to(byte - 127)
    else:
        byte = nearest_on_gpu(E4M3, top / (6 * g))
        unit = torch.tensor(E4M3, device=x.device)[byte] * g
    code = nearest_on_gpu(E2M1, torch.where(unit[..., None] > 0, v.abs() / unit[..., None], 0.0))
    byte = torch.where(finite, byte, 255 if fmt == "mx" else 127)
    r, c = -(-byte.shape[0] // 128), -(-byte.shape[1] // 4)
    tiles = torch.zeros((r * 128, c * 4), dtype=torch.uint8, device=x.device)
    tiles[:byte.shape[0], :byte.shape[1]] = byte.to(torch.uint8)
    return code.view(x.shape), tiles.view(r, 4, 32, c, 4).permute(0, 3, 2, 1, 4).reshape(-1), v.view(x.shape) < 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols,gap", [(1300, 14336, 0), (19600, 544, 0), (19600, 544, 1), (39000, 32, 3)])
def test_matrices_of_whole_tiles(fmt, dtype, rows, cols, gap):
    """Two tiles of 128 x 256 and more per SM, each by one block: rows that start on 16 bytes and
    rows that do not, tiles cut at the ends, both ways, bit for bit."""
    assert -(-rows // 128) * -(-cols // 256) >= 2 * sms()
    gen = torch.Generator(device="cuda").manual_seed(rows + cols + gap)
    x = torch.randn((rows, cols), generator=gen, device="cuda") * torch.exp(2 * torch.randn((rows, 1), generator=gen, device="cuda"))
    x[:, ::3] = torch.round(x[:, ::3] * 4) / 4                      # ties among them
    x[rows // 2] = 0
    x[rows - 1, cols - 1], x[5, 17] = float("nan"), float("-inf")
    wide = torch.full((rows, cols + gap), 9.0, device="cuda", dtype=dtype)
    wide[:, :cols] = x.to(dtype)
    x = wide[:, :cols]
    scale = None if fmt == "mx" else (x.float().abs().nan_to_num(0, 0).amax() / (6 * 448)).reshape(1)
    m = cb.fp4_quantize(x, fmt, scale)
    code, scales, negative = quantise_on_gpu(x, fmt, None if fmt == "mx" else scale.double())
    got = torch.stack([m.codes & 15, m.codes >> 4], -1).view(rows, cols)
    assert torch.equal(m.scales, scales)
    assert torch.equal(got.long() & 7, code)
    assert torch.equal((got >> 3 == 1)[code > 0], negative[code > 0])
    # and back: the values of the form for few tiles, 512 rows at a time (its tests are above)
    back = torch.full((rows, cols + gap), 9.0, device="cuda", dtype=dtype)
    cb.fp4_dequantize(m, out=back[:, :cols])
    assert (back[:, cols:] == 9.0).all()
    per = m.scales.numel() // -(-rows // 128)
    assert 4 * -(-cols // 256) < 2 * sms()
    for r in range(0, rows, 512):
        end = min(r + 512, rows)
        part = cb.Fp4Matrix(fmt, end - r, cols, m.codes[r:end], m.scales[r // 128 * per:-(-end // 128) * per], scale)
        assert torch.equal(cb.fp4_dequantize(part, dtype).nan_to_num(-1), back[r:end, :cols].nan_to_num(-1)), r


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("m,n,k,gap", [
    (2400, 2304, 1024, 24),      # 19 row tiles: the last pair's odd CTA has none; whole column tiles; rows on 16 bytes
    (2432, 2344, 1120, 24),      # the last column tile ends in its first half; k ends inside an instruction
    (2300, 2504, 1312, 24),      # ... in its second half; 18 row tiles, the last one cut
    (2400, 2501, 1056, 24),      # rows on any byte
    (2400, 2304, 1024, 0),       # no gap between the rows
])
def test_products_on_cta_pairs_are_exact(fmt, m, n, k, gap):
    """Dense products of k >= 1024 and more tiles of 128 x 256 than SMs run on pairs of SMs (the large
    products above, but for 5100 x 1030 x 1184, are shorter and run on single ones); more tiles of
    256 x 256 than pairs, so that accumulators are handed on."""
    assert k >= 1024 and -(-m // 128) * -(-n // 256) > sms() and -(-m // 256) * -(-n // 256) > sms() // 2
    rng = np.random.default_rng(m + n + k)
    a, b = random_matrix(rng, m, k, fmt, True), random_matrix(rng, n, k, fmt, True)
    x, y = (torch.from_numpy(decode64(t, fmt)).cuda() for t in (a, b))
    ref = x @ y.T
    assert float((x.abs() @ y.abs().T).max()) < 2.0 ** 20
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.full((m, n + gap), 7.0, dtype=dtype, device="cuda")
        cb.fp4_matmul(a, b, out=out[:, :n], status=status)
        assert torch.equal(out[:, :n], ref.to(dtype)) and (out[:, n:] == 7.0).all()
    assert int(status) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(4, 256, 256), (200, 256, 256), (2400, 2304, 1024)])
def test_a_wait_that_runs_out_is_reported(monkeypatch, m, n, k):
    """The library's stall makes the epilogues wait, for 1 ms, for a tile that is never said to be
    done (swapped products, single CTAs, pairs).  The call ends and the status says why: the
    caller's own word, or without one the device's; the next product is right."""
    rng = np.random.default_rng(m)
    a, b = random_matrix(rng, m, k, "mx", True), random_matrix(rng, n, k, "mx", True)
    want = cb.fp4_matmul(a, b)
    assert cb.fp4_last_error() == cb.CB_OK
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    monkeypatch.setenv("CB_MOE_INJECT_FAULT", "stall")
    cb.fp4_matmul(a, b, status=status)
    assert cb.fp4_last_error() == cb.CB_OK and int(status) == cb.CB_ERR_TIMEOUT
    cb.fp4_matmul(a, b)
    monkeypatch.delenv("CB_MOE_INJECT_FAULT")
    assert cb.fp4_last_error() == cb.CB_ERR_TIMEOUT and cb.fp4_last_error() == cb.CB_OK
    assert torch.equal(cb.fp4_matmul(a, b), want) and cb.fp4_last_error() == cb.CB_OK
