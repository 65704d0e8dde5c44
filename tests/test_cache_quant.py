"""Writing the quantised caches from rows of activations, and reading cache rows back.

The definition is evaluated here in 64 bits: the scale in fp32 (it is stored so), each code the
e4m3 value nearest to the exact quotient, found by a search among all codes.  Codes and scales of a
write must then match bit for bit.  A read rounds one fp32 product to the output's type, so it is
compared with that rounding done by torch on the CPU, bit for bit as well.
"""
import ctypes
import math

import pytest
import torch

import dsa_inputs as di
import dsa_sparse_attention_li_gb300 as dsa

E4M3 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()  # 0 .. 448
WIDTH = {"latent": 128, "mx": 32}


def nearest_code(y):
    """Code bytes of the e4m3 values nearest to y (64 bits): ties to even, saturated, NaN kept."""
    a = torch.nan_to_num(y, nan=0.0, posinf=1e300, neginf=-1e300).abs().clamp(max=448.0)
    up = torch.searchsorted(E4M3, a.contiguous()).clamp(1, 126)
    lo, hi = E4M3[up - 1], E4M3[up]
    mid = (lo + hi) / 2
    code = torch.where((a > mid) | ((a == mid) & (up % 2 == 0)), up, up - 1)
    code = torch.where(torch.isnan(y), 127, code)
    return code, torch.signbit(y)


def reference(rows, form):
    """(code magnitudes, signs, scales or E8M0 bytes) of rows [n, d], one scale per group."""
    x = rows.double()
    n, d = x.shape
    w = WIDTH.get(form, d)
    codes, signs, scales = [], [], []
    for c in range(0, d, w):
        part = x[:, c:c + w]
        a = torch.where(torch.isfinite(part), part.abs(), 0.0).amax(1)
        if form == "mx":
            e = torch.tensor([max(math.frexp(v)[1] - 9, -127) if v > 0 else 0 for v in a.tolist()])
            scales.append((e + 127).to(torch.uint8))
            s = torch.tensor([math.ldexp(1.0, int(v)) for v in e], dtype=torch.float64)
        else:
            s = torch.where(a > 0, (a / 448).clamp(min=2.0 ** -126), 1.0).float()
            scales.append(s)
            s = s.double()
        code, sign = nearest_code(part / s[:, None])
        codes.append(code)
        signs.append(sign)
    return torch.cat(codes, 1), torch.cat(signs, 1), torch.stack(scales, 1)


def make_cache(form, dim, pages, page_size, g):
    """A cache of random bytes, and the keyword arguments that go with its pool."""
    if form == "latent":
        return torch.randint(0, 256, (pages, page_size, 608), generator=g).to(torch.uint8), {}
    pool = torch.randint(0, 127, (pages, page_size, dim), generator=g).to(torch.uint8).view(torch.float8_e4m3fn)
    if form == "fp8":
        return pool, {"scale_pool": torch.rand((pages, page_size), generator=g)}
    return pool, {"sf_pool": torch.randint(0, 255, (pages, page_size, dim // 32), generator=g).to(torch.uint8)}


def places(n, B, max_pages, page_size, g):
    """n different (sequence, position) pairs in random order."""
    pick = torch.randperm(B * max_pages * page_size, generator=g)[:n]
    return ((pick // (max_pages * page_size)).to(torch.int32), (pick % (max_pages * page_size)).to(torch.int32))


def slots(pt, seq, pos, page_size):
    return pt[seq.long(), (pos // page_size).long()].long() * page_size + pos.long() % page_size


def cuda(x):
    return {k: v.cuda() for k, v in x.items()} if isinstance(x, dict) else x.cuda()


def hard_rows(n, d, dtype, g):
    """Rows with what a quantiser can get wrong: plain values; all zero; one large value; values at
    and beside the borders between codes (their group's largest value is 448); values near the
    type's limits and in its subnormal range; infinities and NaN beside finite values."""
    x = torch.randn((n, d), generator=g) * torch.exp(2 * torch.randn((n, 1), generator=g))
    border = ((E4M3[:-1] + E4M3[1:]) / 2).float()
    for r in range(n):
        kind = r % 8
        if kind == 1:
            x[r] = 0
        elif kind == 2:
            x[r, torch.randint(0, d, (1,), generator=g)] *= 1e3
        elif kind == 3:
            x[r] = border[torch.randint(0, 126, (d,), generator=g)]
            if dtype == torch.float32:  # one step of fp32 beside the border
                x[r] *= 1 + torch.randint(-1, 2, (d,), generator=g) * 2.0 ** -23
            x[r] *= torch.randint(0, 2, (d,), generator=g) * 2 - 1
            x[r, ::32] = 448
        elif kind == 4:
            x[r] = torch.rand(d, generator=g) * torch.finfo(dtype).max
        elif kind == 5:
            tiny = torch.finfo(dtype).smallest_normal
            x[r] = torch.randn(d, generator=g) * tiny * 0.25
        elif kind == 6:
            x[r, torch.randint(0, d, (3,), generator=g)] = math.inf
            x[r, torch.randint(0, d, (3,), generator=g)] = -math.inf
            x[r, torch.randint(0, d, (3,), generator=g)] = math.nan
        elif kind == 7:
            x[r, d // 2:] = math.inf
    return x.to(dtype)


FORMS = [("latent", 576), ("fp8", 128), ("fp8", 64), ("fp8", 32), ("fp8", 256), ("mx", 128), ("mx", 32), ("mx", 256)]
TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("form,dim", FORMS)
@pytest.mark.parametrize("n,page_size,pad", [(1, 64, 0), (5, 64, 8), (203, 64, 24), (64, 7, 0)])
def test_write_matches_the_definition(cuda_lib, form, dim, dtype, n, page_size, pad):
    g = torch.Generator().manual_seed(n * 1000 + dim)
    B, max_pages = 3, 40 if page_size == 7 else 4
    pages = B * max_pages + 3
    pt = torch.randperm(pages, generator=g)[:B * max_pages].to(torch.int32).view(B, max_pages)
    seq, pos = places(n, B, max_pages, page_size, g)
    rows = hard_rows(n, dim, dtype, g)
    wide = torch.full((n, dim + pad), 7.0, dtype=dtype)
    wide[:, :dim] = rows
    pool, kw = make_cache(form, dim, pages, page_size, g)
    want_pool, want_kw = pool.view(torch.uint8).clone(), {k: v.clone() for k, v in kw.items()}

    dpool, dkw = cuda(pool), cuda(kw)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dsa.cache_write_quant(dpool, pt.cuda(), seq.cuda(), pos.cuda(), wide.cuda()[:, :dim], status=status, **dkw)
    torch.cuda.synchronize()
    assert int(status) == 0

    at = slots(pt, seq, pos, page_size)
    code, sign, scale = reference(rows, form)
    # zeros carry the sign of the quotient, NaN codes any sign
    byte = torch.where(code == 127, 127, code + 128 * sign).to(torch.uint8)
    want = want_pool.view(-1, want_pool.shape[-1])
    got = dpool.cpu().view(torch.uint8).view(-1, want.shape[1]).clone()
    nan = torch.zeros_like(got, dtype=torch.bool)
    nan[at, :dim] = code == 127
    got[nan] &= 127
    want[at, :dim] = byte
    if form == "latent":
        want[at, 576:596] = scale.contiguous().view(torch.uint8)
        want[at, 596:] = 0
    else:
        name = "scale_pool" if form == "fp8" else "sf_pool"
        want_kw[name].view(-1, scale.shape[1])[at] = scale
        assert torch.equal(dkw[name].cpu(), want_kw[name])
    assert torch.equal(got, want)  # rows that were not written keep their bytes


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("form,dim", FORMS + [("bf16", 576), ("bf16", 128), ("bf16", 8)])
@pytest.mark.parametrize("n,page_size,pad", [(1, 64, 0), (203, 64, 16), (64, 5, 0)])
def test_read_rounds_the_product_once(cuda_lib, form, dim, dtype, n, page_size, pad):
    g = torch.Generator().manual_seed(n + dim)
    B, max_pages = 2, 30 if page_size == 5 else 4
    pages = B * max_pages
    pt = torch.randperm(pages, generator=g).to(torch.int32).view(B, max_pages)
    seq, pos = places(n, B, max_pages, page_size, g)
    if n > 3:
        seq[1], pos[1] = seq[0], pos[0]  # the same place twice
    at = slots(pt, seq, pos, page_size)
    if form == "bf16":
        pool, kw = torch.randn((pages, page_size, dim), generator=g).bfloat16(), {}
        want = pool.view(-1, dim)[at].to(dtype)
    else:
        pool, kw = make_cache(form, dim, pages, page_size, g)
        raw = pool.view(torch.uint8).view(pages * page_size, -1)
        if form == "latent":
            raw[:, 576:596] = (torch.rand((raw.shape[0], 5), generator=g) * 3).view(torch.uint8)
            scale = raw[at, 576:596].contiguous().view(torch.float32).repeat_interleave(128, 1)[:, :576]
        elif form == "fp8":
            scale = kw["scale_pool"].view(-1, 1)[at]
        else:
            e = kw["sf_pool"].view(raw.shape[0], -1)[at].repeat_interleave(32, 1).double() - 127
            scale = torch.pow(2.0, e).float()
        want = (raw[at, :dim].contiguous().view(torch.float8_e4m3fn).float() * scale).to(dtype)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((n, dim + pad), 9.0, dtype=dtype, device="cuda")
    got = dsa.cache_read(pool.cuda(), pt.cuda(), seq.cuda(), pos.cuda(), out=out[:, :dim], status=status, **cuda(kw))
    torch.cuda.synchronize()
    assert int(status) == 0
    got = got.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))
    assert torch.all(out.cpu()[:, dim:] == 9.0)


@pytest.mark.gpu
@pytest.mark.parametrize("form,dim", [("latent", 576), ("fp8", 128), ("mx", 128)])
def test_rows_out_of_range_are_reported(cuda_lib, form, dim):
    g = torch.Generator().manual_seed(5)
    pt = torch.tensor([[1, 0, 99], [2, -1, 3]], dtype=torch.int32)   # pages 99 and -1 do not exist
    seq = torch.tensor([0, 0, 1, 1, 2, -1, 0, 0, 0], dtype=torch.int32)
    pos = torch.tensor([3, 130, 64, 130, 0, 0, 192, -1, 2 ** 31 - 1], dtype=torch.int32)
    good = torch.tensor([0, 3])
    rows = torch.randn((9, dim), generator=g)
    pool, kw = make_cache(form, dim, 4, 64, g)
    dpool, dkw = cuda(pool), cuda(kw)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dsa.cache_write_quant(dpool, pt.cuda(), seq.cuda(), pos.cuda(), rows.cuda(), status=status, **dkw)
    assert int(status) == dsa.DSA_ERR_DEVICE_CHECK
    at = slots(pt, seq[good], pos[good], 64)
    same = dpool.cpu().view(torch.uint8).view(256, -1) == pool.view(torch.uint8).view(256, -1)
    touched = ~same.all(1)
    assert touched[at].all() and int(touched.sum()) == 2
    status.zero_()
    out = dsa.cache_read(dpool, pt.cuda(), seq.cuda(), pos.cuda(), dtype=torch.float32, status=status, **dkw)
    assert int(status) == dsa.DSA_ERR_DEVICE_CHECK
    bad = torch.ones(9, dtype=torch.bool)
    bad[good] = False
    assert torch.all(out.cpu()[bad] == 0) and torch.all(out.cpu()[~bad].abs().amax(1) > 0)
    # without a status word the same call still leaves the caches alone
    dsa.cache_write_quant(dpool, pt.cuda(), seq.cuda(), pos.cuda(), rows.cuda(), **dkw)
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_write_then_read_on_another_stream_and_in_a_graph(cuda_lib):
    g = torch.Generator().manual_seed(11)
    n, pt = 70, torch.tensor([[1, 0]], dtype=torch.int32).cuda()
    seq = torch.zeros(n, dtype=torch.int32, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    rows = torch.randn((n, 576), generator=g).cuda()
    pool = torch.zeros((2, 64, 608), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        dsa.cache_write_quant(pool, pt, seq, pos, rows)
        first = dsa.cache_read(pool, pt, seq, pos)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    out = torch.empty_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.cache_write_quant(pool, pt, seq, pos, rows)
        dsa.cache_read(pool, pt, seq, pos, out=out)
    for k in (1.0, 3.0):
        rows.mul_(k)
        graph.replay()
        torch.cuda.synchronize()
        # half an e4m3 step of the value (2^-4), or of the smallest normal code (2^-10 scales; a
        # scale is amax/448), and half a bf16 step
        tile = torch.nn.functional.pad(rows, (0, 64)).view(n, 5, 128).abs().amax(2).repeat_interleave(128, 1)[:, :576]
        err = (out.float() - rows).abs()
        assert torch.all(err <= rows.abs() * (2 ** -4 + 2 ** -8 + 2 ** -11) + tile / 448 * 2 ** -10)
        if k == 1.0:
            assert torch.equal(out, first)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("form,dim", FORMS)
def test_many_rows_are_written_and_read_as_few_are(cuda_lib, form, dim, dtype):
    """More than a wave of warps of 512 columns each, in one call and a few rows at a time."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n = sms * 64 * 512 // dim + 1003
    g = torch.Generator().manual_seed(dim)
    max_pages = n // 64 + 1
    pt = torch.randperm(max_pages, generator=g).to(torch.int32)[None].cuda()
    pos = torch.randperm(n, generator=g).to(torch.int32).cuda()
    seq = torch.zeros_like(pos)
    rows = hard_rows(1000, dim, dtype, g).cuda()[torch.arange(n, device="cuda") * 7 % 1000]
    pool, kw = make_cache(form, dim, max_pages, 64, g)
    one, one_kw, few, few_kw = cuda(pool), cuda(kw), cuda(pool), cuda(kw)
    dsa.cache_write_quant(one, pt, seq, pos, rows, **one_kw)
    step = n // 9
    for at in range(0, n, step):
        part = slice(at, at + step)
        dsa.cache_write_quant(few, pt, seq[part], pos[part], rows[part], **few_kw)
    assert torch.equal(one.view(torch.uint8), few.view(torch.uint8))
    assert all(torch.equal(one_kw[k], few_kw[k]) for k in one_kw)
    got = dsa.cache_read(one, pt, seq, pos, dtype=dtype, **one_kw)
    again = torch.cat([dsa.cache_read(one, pt, seq[k:k + step], pos[k:k + step], dtype=dtype, **one_kw)
                       for k in range(0, n, step)])
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(again))
    assert torch.equal(torch.isnan(got), torch.isnan(again))


@pytest.mark.gpu
def test_offsets_beyond_32_bits(cuda_lib):
    """A cache of 4.7 GB and rows that lie 2 GB apart."""
    g = torch.Generator().manual_seed(8)
    pages = 120001
    pool = torch.zeros((pages, 64, 608), dtype=torch.uint8, device="cuda")
    pt = torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32, device="cuda")
    pos = torch.tensor([63, 64, 191, 0, 130], dtype=torch.int32, device="cuda")
    seq = torch.zeros_like(pos)
    values = torch.randn((5, 576), generator=g).bfloat16().cuda()
    far = torch.zeros(4 * 2 ** 30 + 576, dtype=torch.bfloat16, device="cuda").as_strided((5, 576), (2 ** 30, 1))
    far.copy_(values)
    dsa.cache_write_quant(pool, pt, seq, pos, far)
    small = torch.zeros((3, 64, 608), dtype=torch.uint8, device="cuda")
    dsa.cache_write_quant(small, torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda"), seq, pos, values)
    assert torch.equal(pool[0], small[0]) and torch.equal(pool[-2:], small[1:])
    far.zero_()
    dsa.cache_read(pool, pt, seq, pos, out=far)
    want = dsa.cache_read(small, torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda"), seq, pos)
    assert torch.equal(far, want) and bool(want.any())


@pytest.mark.gpu
def test_the_written_latent_rows_are_the_generators(cuda_lib):
    """The format is the one that dsa_sfa_* are tested on: the generator's rows, from the same fp32
    values, up to codes whose quotient its fp32 division rounds onto a border (about one in 2^20)."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn((128, 576), generator=g)
    want = di._quant_kv8(x)
    pool = torch.zeros((2, 64, 608), dtype=torch.uint8, device="cuda")
    pt = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    pos = torch.arange(128, dtype=torch.int32, device="cuda")
    dsa.cache_write_quant(pool, pt, torch.zeros_like(pos), pos, x.cuda())
    got = pool.cpu().view(128, 608)
    assert torch.equal(got[:, 576:], want[:, 576:])
    assert int((got[:, :576] != want[:, :576]).sum()) <= 2


def _args(**over):
    a = dsa.CacheRowsArgs()
    a.n_rows, a.dim, a.B, a.page_size, a.max_pages, a.num_pages = 4, 576, 1, 64, 2, 2
    a.format, a.elem, a.row_stride = dsa.ROW_LATENT_FP8, 0, 576
    for n in ("rows", "pool", "scale_pool", "sf_pool", "page_table", "seq", "pos"):
        setattr(a, n, 4096)  # fake, aligned, never dereferenced on these error paths
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("entry", ["dsa_cache_write_quant", "dsa_cache_read"])
@pytest.mark.parametrize("over,code", [
    ({"n_rows": -1}, dsa.DSA_ERR_INVALID_ARG),
    ({"B": 0}, dsa.DSA_ERR_INVALID_ARG),
    ({"page_size": 0}, dsa.DSA_ERR_INVALID_ARG),
    ({"elem": 3}, dsa.DSA_ERR_INVALID_ARG),
    ({"format": 4}, dsa.DSA_ERR_INVALID_ARG),
    ({"dim": 512}, dsa.DSA_ERR_UNSUPPORTED),
    ({"dim": 96, "format": dsa.ROW_FP8}, dsa.DSA_ERR_UNSUPPORTED),
    ({"dim": 128, "format": dsa.ROW_FP8, "scale_pool": None}, dsa.DSA_ERR_INVALID_ARG),
    ({"dim": 128, "format": dsa.ROW_MXFP8, "sf_pool": None}, dsa.DSA_ERR_INVALID_ARG),
    ({"row_stride": 568}, dsa.DSA_ERR_INVALID_ARG),
    ({"row_stride": 580}, dsa.DSA_ERR_UNSUPPORTED),          # rows not 16-byte aligned
    ({"rows": None}, dsa.DSA_ERR_INVALID_ARG),
    ({"pool": 4104}, dsa.DSA_ERR_INVALID_ARG),
    ({"pos": None}, dsa.DSA_ERR_INVALID_ARG),
])
def test_cache_rows_host_validation(entry, over, code):
    lib = dsa.load()
    assert getattr(lib, entry)(ctypes.byref(_args(**over)), None) == code, dsa.last_error()
    assert dsa.last_error()
    assert getattr(lib, entry)(None, None) == dsa.DSA_ERR_INVALID_ARG
    assert getattr(lib, entry)(ctypes.byref(_args(n_rows=0)), None) == dsa.DSA_OK


def test_bf16_caches_are_read_only_here():
    lib = dsa.load()
    a = _args(format=dsa.ROW_BF16)
    assert lib.dsa_cache_write_quant(ctypes.byref(a), None) == dsa.DSA_ERR_UNSUPPORTED
    a = _args(format=dsa.ROW_BF16, dim=12, row_stride=16)
    assert lib.dsa_cache_read(ctypes.byref(a), None) == dsa.DSA_ERR_UNSUPPORTED


def test_struct_layout():
    assert ctypes.sizeof(dsa.CacheRowsArgs) == 8 * 4 + 8 + 8 * 8


def test_binding_refuses_what_does_not_fit():
    pt = torch.zeros((1, 2), dtype=torch.int32)
    at = torch.zeros(4, dtype=torch.int32)
    kv8 = torch.zeros((2, 64, 608), dtype=torch.uint8)
    k8 = torch.zeros((2, 64, 128), dtype=torch.uint8).view(torch.float8_e4m3fn)
    rows = torch.zeros((4, 576))
    for bad in (dict(rows=torch.zeros((4, 512))), dict(rows=torch.zeros((4, 576), dtype=torch.float64)),
                dict(rows=torch.zeros((576, 4)).T), dict(seq=at.long()), dict(pos=at[:3]),
                dict(pool=kv8[..., :600].contiguous()), dict(pool=k8), dict(scale_pool=torch.zeros((2, 64))),
                dict(pool=kv8[:, ::2]), dict(rows=rows[:1].expand(4, 576)), dict()):  # the last: CPU tensors
        kw = dict(pool=kv8, page_table=pt, seq=at, pos=at, rows=rows)
        kw.update(bad)
        with pytest.raises(ValueError):
            dsa.cache_write_quant(**kw)
    for bad in (dict(), dict(scale_pool=torch.zeros((2, 64)), sf_pool=torch.zeros((2, 64, 4), dtype=torch.uint8)),
                dict(sf_pool=torch.zeros((2, 64, 3), dtype=torch.uint8)), dict(scale_pool=torch.zeros((2, 32)))):
        with pytest.raises(ValueError):
            dsa.cache_write_quant(k8, pt, at, at, torch.zeros((4, 128)), **bad)
