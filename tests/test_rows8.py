"""8-bit rows: the root-mean-square norm with the residual's addition, and rows as they are.

Both are compared with their definition in 64 bits.  Rows without a norm match bit for bit, as the
quantised cache write does.  With a norm, the sum of squares is held in fp32: a thread adds up to 16
squares in each of two sums, the two, and five times its warp's (the warps' sums are added without loss), 22 roundings of
at most 2^-24 each, half of which reach 1 / sqrt; with the rounding of h * weight, and of r and s, v / s is off by less
than 14 * 2^-24 < 2^-20.  So a code lies between those of v / s (1 - 2^-20) and v / s (1 + 2^-20).
"""
import ctypes
import math

import pytest
import torch

import dsa_sparse_attention_li_gb300 as dsa
from test_cache_quant import hard_rows, nearest_code

TYPES = [torch.bfloat16, torch.float16, torch.float32]
OFF = 2.0 ** -20


def group_scales(v):
    """fp32(a / 448) of every group of 128 columns of v (64 bits), a its largest finite magnitude."""
    n, d = v.shape
    v = torch.nn.functional.pad(v, (0, -d % 128)).view(n, -1, 128)
    a = torch.where(torch.isfinite(v), v.abs(), 0.0).amax(2)
    return torch.where(a > 0, (a / 448).clamp(min=2.0 ** -126), 1.0).float()


def columns(s, d):
    return s.double().repeat_interleave(128, 1)[:, :d]


def same_codes(got, q):
    """Whether e4m3 codes are those nearest to the quotients q (64 bits), bit for bit but for a NaN's sign."""
    code, sign = nearest_code(q)
    raw = got.view(torch.uint8).long()
    want = code + 128 * sign.long()
    return torch.where(code == 127, (raw & 127) == 127, raw == want)


def check_norm(x, w, residual, eps, codes, scale, total, y):
    """All outputs (on the CPU) of one call against the definition."""
    kind, d = x.dtype, x.shape[1]
    h = x
    if residual is not None:
        h = (x.float() + residual.float()).to(kind)
        assert torch.equal(torch.nan_to_num(total), torch.nan_to_num(h)) and torch.equal(total.isnan(), h.isnan())
    h = h.double()
    r = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    v = h * w.double() * r
    under = r * 2.0 ** -149    # h * w below fp32's normal range is off by half its smallest step, twice that here
    want = group_scales(v).double()
    assert torch.all((scale.double() - want).abs() <= want * OFF + under + 2.0 ** -149)
    q = v / columns(scale, d)
    off = q.abs() * OFF + under / columns(scale, d)
    low, _ = nearest_code((q.abs() - off).clamp(min=0))
    high, _ = nearest_code(q.abs() + off)
    got = codes.view(torch.uint8).long() & 127
    assert torch.all((got >= low) & (got <= high))
    assert torch.all((torch.signbit(codes.float()) == torch.signbit(v)) | (got == 127))
    if y is not None:
        # (below the type's normal range a rounding is off by half its smallest step)
        step = torch.finfo(kind).eps / 2
        off = v.abs() * (step + OFF) + torch.finfo(kind).smallest_normal * step + under
        good = torch.isfinite(v) & (v.abs() < torch.finfo(kind).max)
        assert torch.all(((y.double() - v).abs() <= off)[good])
        assert torch.equal(y.isnan(), v.isnan())


def strided(t, pad):
    wide = torch.full((t.shape[0], t.shape[1] + pad), 3.0, device=t.device).to(t.dtype)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("n,d", [(1, 8), (3, 64), (5, 120), (37, 128), (6, 136), (9, 256), (4, 264), (7, 512), (3, 520),
                                 (5, 576), (11, 1536), (2, 4104), (33, 7168), (3, 16384), (2, 16392), (2, 32768)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_matches_the_definition(cuda_lib, n, d, dtype, residual):
    g = torch.Generator().manual_seed(n * 7 + d)
    x = (torch.randn((n, d), generator=g) * torch.exp(torch.randn((n, 1), generator=g))).to(dtype)
    r = (3 * torch.randn((n, d), generator=g)).to(dtype) if residual else None
    w = (1 + 0.3 * torch.randn(d, generator=g)).to(torch.float32 if n % 2 else dtype)
    pad = 8 * (n % 3)
    y = strided(torch.zeros((n, d), dtype=dtype, device="cuda"), pad)
    got = dsa.rms_norm_quant(strided(x.cuda(), pad), w.cuda(), eps=1e-6, y=y,
                             residual=None if r is None else strided(r.cuda(), 8))
    codes, scale = got[:2]
    assert codes.dtype == torch.float8_e4m3fn and codes.shape == (n, d) and scale.shape == (n, -(-d // 128))
    check_norm(x, w, r, 1e-6, codes.cpu(), scale.cpu(), got[2].cpu() if residual else None, y.cpu())
    if pad:  # nothing beyond a row's columns is written
        assert torch.all(y.as_strided((n, pad), (y.stride(0), 1), d)[:, :].float() == 3.0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("d", [72, 576, 2048])
def test_norm_of_hard_rows(cuda_lib, d, dtype):
    """Rows of zeros, of the type's smallest and largest values, with infinities and NaN."""
    g = torch.Generator().manual_seed(d)
    x = hard_rows(24, d, dtype, g)
    w = (1 + 0.3 * torch.randn(d, generator=g)).to(dtype)
    y = torch.empty((24, d), dtype=dtype, device="cuda")
    codes, scale = dsa.rms_norm_quant(x.cuda(), w.cuda(), eps=1e-5, y=y)
    codes, scale, y = codes.cpu().view(torch.uint8), scale.cpu(), y.cpu()
    # rows whose sum of squares fits fp32; the others have r = 0, or are all NaN
    squares = (x.double() ** 2).sum(1)
    fits = squares < 2.0 ** 127
    check_norm(x[fits], w, None, 1e-5, codes[fits].view(torch.float8_e4m3fn), scale[fits], None, y[fits])
    nan = torch.isnan(x).any(1)
    assert torch.all((codes[nan] & 127) == 127) and torch.all(y[nan].isnan())
    assert torch.all(scale[nan] == 1.0)
    over = ~nan & ~(squares < 2.0 ** 130)
    finite = torch.isfinite(x[over])
    assert torch.all((codes[over] & 127)[finite] == 0) and torch.all(scale[over] == 1.0)
    assert torch.all((codes[over] & 127)[~finite] == 127)


@pytest.mark.gpu
def test_norm_of_zero_rows_without_epsilon(cuda_lib):
    """0 / 0: NaN, as the formula has it, in that row alone."""
    x = torch.randn((3, 200), generator=torch.Generator().manual_seed(0)).bfloat16()
    x[1] = 0
    w = torch.ones(200, dtype=torch.bfloat16)
    codes, scale = dsa.rms_norm_quant(x.cuda(), w.cuda(), eps=0.0)
    codes = codes.cpu().view(torch.uint8)
    assert torch.all((codes[1] & 127) == 127) and torch.all(scale[1] == 1.0)
    check_norm(x[[0, 2]], w, None, 0.0, codes[[0, 2]].view(torch.float8_e4m3fn), scale.cpu()[[0, 2]], None, None)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [128, 7168])
def test_norm_in_place(cuda_lib, d):
    """The sum in the residual's place, and the normed rows in x's."""
    g = torch.Generator().manual_seed(d)
    x, r = (torch.randn((19, d), generator=g).bfloat16().cuda() for _ in range(2))
    w = torch.rand(d, generator=g).bfloat16().cuda()
    y = torch.empty_like(x)
    want = dsa.rms_norm_quant(x, w, residual=r, y=y)
    x2, r2 = x.clone(), r.clone()
    got = dsa.rms_norm_quant(x2, w, residual=r2, residual_out=r2, y=x2)
    assert got[2] is r2 and torch.equal(r2, want[2]) and torch.equal(x2, y)
    assert torch.equal(got[0].view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(got[1], want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("n,d", [(1, 8), (16, 64), (9, 200), (203, 128), (24, 576), (8, 16384), (1, 40000)])
def test_rows_match_the_definition(cuda_lib, n, d, dtype):
    g = torch.Generator().manual_seed(n + d)
    x = hard_rows(n, d, dtype, g)
    codes = strided(torch.zeros((n, d), device="cuda").to(torch.float8_e4m3fn), 8)
    scale = strided(torch.zeros((n, -(-d // 128)), device="cuda"), 3)
    dsa.quant_rows(strided(x.cuda(), 16), codes=codes, scale=scale)
    s = group_scales(x.double())
    assert torch.equal(scale.cpu(), s)
    assert torch.all(same_codes(codes.cpu().contiguous(), x.double() / columns(s, d)))
    assert torch.all(codes.as_strided((n, 8), (d + 8, 1), d).float() == 3.0)


@pytest.mark.gpu
def test_many_rows_and_far_rows(cuda_lib):
    """Rows that lie 2 GB apart, and more rows than a wave of blocks, one by one as all at once."""
    g = torch.Generator().manual_seed(4)
    values = torch.randn((5, 1024), generator=g).bfloat16().cuda()
    far = torch.zeros(4 * 2 ** 30 + 1024, dtype=torch.bfloat16, device="cuda").as_strided((5, 1024), (2 ** 30, 1))
    far.copy_(values)
    w = torch.ones(1024, device="cuda")
    for call in (dsa.quant_rows, lambda x: dsa.rms_norm_quant(x, w)):
        a, b = call(far), call(values)
        assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and torch.equal(a[1], b[1])
    codes = torch.zeros(4 * 2 ** 30 + 1024, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    codes = codes.as_strided((5, 1024), (2 ** 30, 1))
    dsa.quant_rows(values, codes=codes)
    assert torch.equal(codes.contiguous().view(torch.uint8), dsa.quant_rows(values)[0].view(torch.uint8))
    del far, codes
    x = torch.randn((30011, 136), generator=g).cuda()
    w = torch.rand(136, generator=g).cuda()
    for call in (dsa.quant_rows, lambda x: dsa.rms_norm_quant(x, w)):
        a = call(x)
        b = [call(x[i:i + 977]) for i in range(0, len(x), 977)]
        assert torch.equal(a[0].view(torch.uint8), torch.cat([p[0].view(torch.uint8) for p in b]))
        assert torch.equal(a[1], torch.cat([p[1] for p in b]))


@pytest.mark.gpu
def test_no_rows(cuda_lib):
    x = torch.zeros((0, 256), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    assert dsa.quant_rows(x)[0].shape == (0, 256)
    assert [tuple(t.shape) for t in dsa.rms_norm_quant(x, w, residual=x)] == [(0, 256), (0, 2), (0, 256)]


def _norm(**over):
    a = dsa.RmsNormQuantArgs()
    a.n_rows, a.dim, a.elem, a.weight_elem, a.eps = 4, 576, 0, 0, 1e-6
    a.x_stride = a.residual_stride = a.sum_stride = a.y_stride = a.codes_stride = 576
    a.scale_stride = 5
    for n in ("x", "weight", "residual", "sum", "codes", "scale"):
        setattr(a, n, 4096)  # fake, aligned, never dereferenced on these error paths
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,code", [
    ({"n_rows": -1}, dsa.DSA_ERR_INVALID_ARG),
    ({"dim": 0}, dsa.DSA_ERR_INVALID_ARG),
    ({"dim": 580}, dsa.DSA_ERR_UNSUPPORTED),
    ({"dim": 32776}, dsa.DSA_ERR_UNSUPPORTED),
    ({"elem": 3}, dsa.DSA_ERR_INVALID_ARG),
    ({"weight_elem": 1}, dsa.DSA_ERR_UNSUPPORTED),
    ({"elem": 2, "weight_elem": 0}, dsa.DSA_ERR_UNSUPPORTED),
    ({"eps": -1e-6}, dsa.DSA_ERR_INVALID_ARG),
    ({"eps": math.inf}, dsa.DSA_ERR_INVALID_ARG),
    ({"eps": math.nan}, dsa.DSA_ERR_INVALID_ARG),
    ({"x": None}, dsa.DSA_ERR_INVALID_ARG),
    ({"codes": None}, dsa.DSA_ERR_INVALID_ARG),
    ({"sum": None}, dsa.DSA_ERR_INVALID_ARG),
    ({"residual": None}, dsa.DSA_ERR_INVALID_ARG),
    ({"x": 4104}, dsa.DSA_ERR_INVALID_ARG),
    ({"y": 4104}, dsa.DSA_ERR_INVALID_ARG),
    ({"weight": 4104}, dsa.DSA_ERR_INVALID_ARG),
    ({"codes": 4100}, dsa.DSA_ERR_INVALID_ARG),
    ({"x_stride": 568}, dsa.DSA_ERR_INVALID_ARG),
    ({"residual_stride": 580}, dsa.DSA_ERR_INVALID_ARG),
    ({"codes_stride": 580}, dsa.DSA_ERR_INVALID_ARG),
    ({"scale_stride": 4}, dsa.DSA_ERR_INVALID_ARG),
])
def test_norm_host_validation(over, code):
    lib = dsa.load()
    assert lib.dsa_rms_norm_quant(ctypes.byref(_norm(**over)), None) == code, dsa.last_error()
    assert dsa.last_error()
    assert lib.dsa_rms_norm_quant(None, None) == dsa.DSA_ERR_INVALID_ARG
    assert lib.dsa_rms_norm_quant(ctypes.byref(_norm(n_rows=0)), None) == dsa.DSA_OK


def _rows(**over):
    a = dsa.QuantRowsArgs()
    a.n_rows, a.dim, a.elem, a.x_stride, a.codes_stride, a.scale_stride = 4, 576, 0, 576, 576, 5
    a.x = a.codes = a.scale = 4096
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,code", [
    ({"n_rows": -1}, dsa.DSA_ERR_INVALID_ARG),
    ({"dim": -8}, dsa.DSA_ERR_INVALID_ARG),
    ({"dim": 12}, dsa.DSA_ERR_UNSUPPORTED),
    ({"elem": -1}, dsa.DSA_ERR_INVALID_ARG),
    ({"scale": None}, dsa.DSA_ERR_INVALID_ARG),
    ({"x": 4104}, dsa.DSA_ERR_INVALID_ARG),
    ({"x_stride": 572}, dsa.DSA_ERR_INVALID_ARG),
    ({"codes_stride": 568}, dsa.DSA_ERR_INVALID_ARG),
    ({"scale": 4098}, dsa.DSA_ERR_INVALID_ARG),
])
def test_rows_host_validation(over, code):
    lib = dsa.load()
    assert lib.dsa_quant_rows(ctypes.byref(_rows(**over)), None) == code, dsa.last_error()
    assert dsa.last_error()
    assert lib.dsa_quant_rows(None, None) == dsa.DSA_ERR_INVALID_ARG
    assert lib.dsa_quant_rows(ctypes.byref(_rows(n_rows=0)), None) == dsa.DSA_OK


def test_struct_layouts():
    assert ctypes.sizeof(dsa.RmsNormQuantArgs) == 5 * 4 + 4 + 6 * 8 + 7 * 8
    assert ctypes.sizeof(dsa.QuantRowsArgs) == 3 * 4 + 4 + 3 * 8 + 3 * 8


def test_binding_refuses_cpu_tensors_and_shapes():
    x, w = torch.zeros((4, 576), dtype=torch.bfloat16), torch.ones(576, dtype=torch.bfloat16)
    for bad in (dict(x=x), dict(x=x.double()), dict(x=x[0])):
        with pytest.raises(ValueError):
            dsa.quant_rows(**bad)
        with pytest.raises(ValueError):
            dsa.rms_norm_quant(weight=w, **bad)


@pytest.mark.gpu
def test_binding_refuses_what_does_not_fit(cuda_lib):
    x, w = torch.zeros((4, 576), dtype=torch.bfloat16, device="cuda"), torch.ones(576, dtype=torch.bfloat16, device="cuda")
    codes, scale = torch.zeros((4, 576), device="cuda").to(torch.float8_e4m3fn), torch.zeros((4, 5), device="cuda")
    for bad in (dict(weight=w[:512]), dict(weight=w.half()), dict(weight=w.cpu()), dict(residual=x.float()),
                dict(residual=x[:3]), dict(residual_out=x), dict(residual=x, residual_out=x[:, :512]),
                dict(y=x.float()), dict(codes=codes[:, :512]), dict(codes=x), dict(scale=scale[:, :4]),
                dict(scale=scale.T.contiguous().T), dict(residual=x[:1].expand(4, 576)), dict(residual=x.cpu())):
        kw = dict(x=x, weight=w)
        kw.update(bad)
        with pytest.raises(ValueError):
            dsa.rms_norm_quant(**kw)
    for bad in (dict(codes=codes[:3]), dict(codes=codes.view(torch.uint8)), dict(scale=scale.double()),
                dict(x=x.T), dict(x=x[:, ::2])):
        kw = dict(x=x)
        kw.update(bad)
        with pytest.raises(ValueError):
            dsa.quant_rows(**kw)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("d", [136, 4096, 16384])
def test_norm_of_hard_sums(cuda_lib, d, dtype):
    """The sum with a residual of values across the type's whole range, subnormal ones and infinities among them, in
    place and out of it."""
    g = torch.Generator().manual_seed(d + 1)
    x, r = hard_rows(24, d, dtype, g), hard_rows(24, d, dtype, g)[torch.randperm(24, generator=g)]
    w = (1 + 0.3 * torch.randn(d, generator=g)).to(dtype)
    want = (x.float() + r.float()).to(dtype)
    xd, rd = x.cuda(), r.cuda()
    codes, scale, total = dsa.rms_norm_quant(xd, w.cuda(), eps=1e-5, residual=rd)
    same = lambda a, b: torch.equal(a.isnan(), b.isnan()) and torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))
    assert same(total.cpu(), want)
    # the same rows without a residual, and with the sum in the residual's or in x's place
    c2, s2 = dsa.rms_norm_quant(total, w.cuda(), eps=1e-5)
    assert torch.equal(codes.view(torch.uint8), c2.view(torch.uint8)) and torch.equal(scale, s2)
    for place in (rd, xd):
        a, b = xd.clone(), rd.clone()
        at = a if place is xd else b
        c3, s3, t3 = dsa.rms_norm_quant(a, w.cuda(), eps=1e-5, residual=b, residual_out=at, y=b if place is xd else a)
        assert t3 is at and same(t3.cpu(), want)
        assert torch.equal(codes.view(torch.uint8), c3.view(torch.uint8)) and torch.equal(scale, s3)


@pytest.mark.gpu
def test_rows_on_another_stream_and_in_a_graph(cuda_lib):
    """New outputs of a given stream, and a captured norm in place, replayed."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((300, 7168), generator=g, device="cuda").bfloat16()
    w = torch.rand(7168, generator=g, device="cuda").bfloat16()
    want = dsa.rms_norm_quant(x, w, residual=x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [dsa.rms_norm_quant(x, w, residual=x, stream=side) for _ in range(3)]
    rows = [dsa.quant_rows(x, stream=side) for _ in range(3)]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for a in got:
        assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(a, want))
    for a in rows:
        assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(a, dsa.quant_rows(x)))
    r = x.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        codes, scale, _ = dsa.rms_norm_quant(x, w, residual=r, residual_out=r)
    total = x.clone()
    for _ in range(3):
        graph.replay()
        c, s, total = dsa.rms_norm_quant(x, w, residual=total)
        assert torch.equal(r, total) and torch.equal(codes.view(torch.uint8), c.view(torch.uint8)) and torch.equal(scale, s)


def test_more_groups_than_a_launch_numbers_are_refused():
    lib = dsa.load()
    a = _rows(n_rows=1 << 27, dim=576)
    assert lib.dsa_quant_rows(ctypes.byref(a), None) == dsa.DSA_ERR_UNSUPPORTED and "2^29" in dsa.last_error()


LARGEST = torch.finfo(torch.float32).max


def check_beyond_fp32(x, w, eps, codes, scale, y, off=OFF):
    """Codes and scales where some values are beyond fp32: they count as infinite, saturate and leave the others of
    their group alone.  `off`: what the scale may be off by, beside OFF of the quotients."""
    h, d = x.double(), x.shape[1]
    v = h * w.double() / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    assert torch.all((v.abs() / LARGEST - 1).abs() > 2.0 ** -16)   # (none that a rounding could take across)
    beyond = v.abs() > LARGEST
    v = torch.where(beyond, torch.copysign(torch.full_like(v, math.inf), v), v)
    want = group_scales(v).double()
    assert torch.all((scale.double() - want).abs() <= want * off)
    q = v / columns(want, d)
    low, sign = nearest_code(torch.copysign((q.abs() * (1 - OFF)).clamp(min=0), q))
    high, _ = nearest_code(q.abs() * (1 + OFF))
    raw = codes.view(torch.uint8).long()
    assert torch.all(((raw & 127) >= low) & ((raw & 127) <= high) & ((raw >> 7) == sign.long()))
    assert torch.all(y.isinf()[beyond]) and not y.isnan().any()
    return beyond


@pytest.mark.gpu
@pytest.mark.parametrize("d", [256, 4096])
@pytest.mark.parametrize("dtype,wtype", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                         (torch.float16, torch.float32), (torch.float32, torch.float32)], ids=str)
def test_norm_of_values_beyond_fp32(cuda_lib, dtype, wtype, d):
    """Weights near fp32's largest value, whose products with h are finite and whose products with h r are not: in some
    columns of a group, in all of them, and in none."""
    g = torch.Generator().manual_seed(d)
    x = (0.25 * torch.randn((7, d), generator=g)).to(dtype)
    x[3, :128] = 0.5            # (r is some 3.7 there)
    x[3, 64:128] = -0.5
    w = torch.ones(d)
    w[:128] = 3.2e38            # |h| below 1: h w is finite
    w[128:192:3] = 1e38
    w = w.to(wtype)
    x[:, :192] = x[:, :192].clamp(-0.96875, 0.96875)
    y = torch.empty_like(x, device="cuda")
    codes, scale = dsa.rms_norm_quant(x.cuda(), w.cuda(), eps=1e-6, y=y)
    beyond = check_beyond_fp32(x, w, 1e-6, codes.cpu(), scale.cpu(), y.cpu())
    assert beyond[3, :128].all() and beyond[0, :128].any() and not beyond[0, :128].all()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [256, 4096])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_norm_without_epsilon_of_rows_whose_squares_are_below_fp32(cuda_lib, dtype, d):
    """Squares of 2^-200 and 2^-152 .. 2^-150 round to 0: r is infinite, as of a row of zeros, so every value is infinite,
    or NaN in a column of zeros.  Squares of 2^-140 keep some bits: d of them, each off by 2^-150 at most, the mean by as
    much again twice over, so that 1 / sqrt is off by half of 3 * 2^-10 and a scale by less than 2^-9; r is one for the row,
    so the quotients are as close as ever."""
    g = torch.Generator().manual_seed(d + 2)
    ones = torch.ones(d).to(dtype)
    sign = torch.where(torch.rand((4, d), generator=g) < 0.5, -1.0, 1.0)
    mantissa = (1 + torch.randint(0, 125, (4, d), generator=g) / 128).double()
    x = sign * mantissa * torch.tensor([2.0 ** -100, 2.0 ** -76, 2.0 ** -70, 1.0], dtype=torch.float64)[:, None]
    x = x.to(dtype)
    x[0, 5], x[1, 200] = 0.0, -0.0
    y = torch.empty_like(x, device="cuda")
    codes, scale = (t.cpu() for t in dsa.rms_norm_quant(x.cuda(), ones.cuda(), eps=0.0, y=y))
    y, raw = y.cpu(), codes.view(torch.uint8).long()
    zero = x[:2] == 0
    assert torch.all(scale[:2] == 1.0)
    assert torch.all((raw[:2] & 127) == torch.where(zero, 127, 126)) and torch.equal(y[:2].isnan(), zero)
    assert torch.all((raw[:2] >> 7 == torch.signbit(x[:2]).long()) | zero) and torch.all(y[:2].isinf() | zero)
    for row, off in ((2, 2.0 ** -9), (3, OFF)):
        at = slice(row, row + 1)
        assert not check_beyond_fp32(x[at], ones, 0.0, codes[at], scale[at], y[at], off).any()


@pytest.mark.parametrize("call,args,code", [
    ("dsa_quant_rows", lambda: _rows(n_rows=1, dim=2 ** 30 + 8), dsa.DSA_ERR_UNSUPPORTED),
    ("dsa_quant_rows", lambda: _rows(x_stride=2 ** 40 + 8), dsa.DSA_ERR_INVALID_ARG),
    ("dsa_quant_rows", lambda: _rows(scale_stride=2 ** 40 + 1), dsa.DSA_ERR_INVALID_ARG),
    ("dsa_rms_norm_quant", lambda: _norm(sum_stride=2 ** 40 + 8), dsa.DSA_ERR_INVALID_ARG),
    ("dsa_rms_norm_quant", lambda: _norm(codes_stride=2 ** 40 + 8), dsa.DSA_ERR_INVALID_ARG),
])
def test_limits_of_the_header_are_refused(call, args, code):
    assert getattr(dsa.load(), call)(ctypes.byref(args()), None) == code and dsa.last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("n,d", [(3, 64), (5, 264), (9, 1024), (4, 1536), (3, 7168), (2, 16392)])
def test_norm_with_rows_of_every_tensor_apart(cuda_lib, n, d, dtype):
    """Each tensor with a padding of its own, which stays as it is; then in place."""
    g = torch.Generator().manual_seed(n * 3 + d)
    x, r = ((1 + i) * torch.randn((n, d), generator=g) for i in range(2))
    x, r, w = x.to(dtype), r.to(dtype), (1 + 0.3 * torch.randn(d, generator=g)).to(dtype)
    groups = -(-d // 128)
    e4m3 = torch.float8_e4m3fn
    new = lambda cols, pad, kind: strided(torch.zeros((n, cols), device="cuda").to(kind), pad)
    total, y, codes, scale = new(d, 40, dtype), new(d, 24, dtype), new(d, 56, e4m3), new(groups, 3, torch.float32)
    xs, rs = strided(x.cuda(), 8), strided(r.cuda(), 16)
    got = dsa.rms_norm_quant(xs, w.cuda(), eps=1e-6, residual=rs, residual_out=total, codes=codes, scale=scale, y=y)
    assert got[0] is codes and got[1] is scale and got[2] is total
    check_norm(x, w, r, 1e-6, codes.cpu().contiguous(), scale.cpu(), total.cpu(), y.cpu())
    for t, pad in ((xs, 8), (rs, 16), (total, 40), (y, 24), (codes, 56), (scale, 3)):
        cols = t.shape[1]
        assert torch.all(t.as_strided((n, pad), (t.stride(0), 1), cols).float() == 3.0)
    c2, s2 = new(d, 8, e4m3), new(groups, 1, torch.float32)
    dsa.rms_norm_quant(xs, w.cuda(), eps=1e-6, residual=rs, residual_out=rs, codes=c2, scale=s2, y=xs)
    assert torch.equal(rs, total) and torch.equal(xs, y) and torch.equal(s2, scale)
    assert torch.equal(c2.contiguous().view(torch.uint8), codes.contiguous().view(torch.uint8))
    for t, pad in ((xs, 8), (rs, 16), (c2, 8), (s2, 1)):
        assert torch.all(t.as_strided((n, pad), (t.stride(0), 1), t.shape[1]).float() == 3.0)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [576, 2048])
def test_norm_with_rows_of_every_tensor_far_apart(cuda_lib, d):
    """Rows 4 GB apart in every tensor, one buffer: offsets beyond 32 bits in bytes and in elements."""
    g = torch.Generator().manual_seed(d)
    x, r = (torch.randn((3, d), generator=g).bfloat16().cuda() for _ in range(2))
    w = torch.rand(d, generator=g).cuda()
    y = torch.empty_like(x)
    want = (*dsa.rms_norm_quant(x, w, residual=r, y=y), y)
    raw = torch.zeros(2 * 2 ** 32 + 7 * 65536, dtype=torch.uint8, device="cuda")
    def far(like, place):
        size = like.element_size()
        return raw.view(like.dtype)[place * 65536 // size:].as_strided(like.shape, (2 ** 32 // size, 1))
    fx, fr, codes, scale, total, fy = (far(t, i) for i, t in enumerate((x, r, *want)))
    fx.copy_(x), fr.copy_(r)
    dsa.rms_norm_quant(fx, w, residual=fr, residual_out=total, codes=codes, scale=scale, y=fy)
    for a, b in zip((codes, scale, total, fy), want):
        assert torch.equal(a.contiguous().view(torch.uint8), b.view(torch.uint8))
    dsa.quant_rows(x, codes=codes, scale=scale)
    for a, b in zip((codes, scale), dsa.quant_rows(x)):
        assert torch.equal(a.contiguous().view(torch.uint8), b.view(torch.uint8))
