"""Product of 8-bit rows with block-scaled e4m3 weights, and the calls around the attention in a run.

Small whole codes with scales that are powers of two make every product and every sum exact in fp32, so those
outputs match the definition bit for bit after its one rounding to the output's type.  With any codes and scales, a
block's 128 products are added by the tensor cores: at most 4 instructions, each of which aligns 33 terms to the largest
and may cut each at 2^-24 of it: 132 * 2^-24 of the block's sum of magnitudes, below 2^-16.  Per block the scales'
product and the multiply-add round by 2^-24 of what they give, up to 128 blocks of them here: below 2^-16 again.  So an
output is off by less than 2^-15 of its sum of magnitudes, and half a step of its type.
"""
import ctypes
import math

import pytest
import torch

import dsa_sparse_attention_li_gb300 as dsa

TYPES = [torch.bfloat16, torch.float16, torch.float32]
OFF = 2.0 ** -15


def definition(a, a_scale, b, b_scale):
    """The product, and the sum of its terms' magnitudes, in 64 bits."""
    n, k = b.shape
    x = a.double() * a_scale.double().repeat_interleave(128, 1)[:, :k]
    w = b.double() * b_scale.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    return x @ w.T, x.abs() @ w.abs().T


def whole(m, n, k, g):
    """Operands whose every sum is exact in fp32: codes in -3 .. 3 (a 7168-column sum is below 2^16), scales 2^-1, 1, 2."""
    blocks = -(-k // 128)
    a = torch.randint(-3, 4, (m, k), generator=g, device="cuda").float().to(torch.float8_e4m3fn)
    b = torch.randint(-3, 4, (n, k), generator=g, device="cuda").float().to(torch.float8_e4m3fn)
    a_scale = torch.exp2(torch.randint(-1, 2, (m, blocks), generator=g, device="cuda").float())
    b_scale = torch.exp2(torch.randint(-1, 2, (-(-n // 128), blocks), generator=g, device="cuda").float())
    return a, a_scale, b, b_scale


def any_values(m, n, k, g):
    blocks = -(-k // 128)
    a, b = ((110 * torch.randn((r, k), generator=g, device="cuda")).clamp_(-448, 448).to(torch.float8_e4m3fn) for r in (m, n))
    a_scale, b_scale = (torch.exp(torch.randn((r, blocks), generator=g, device="cuda")) / 110 for r in (m, -(-n // 128)))
    return a, a_scale, b, b_scale / math.sqrt(k)


def gen(*seed):
    return torch.Generator(device="cuda").manual_seed(sum(s * 31 ** i for i, s in enumerate(seed)))


SIZES = [(1, 1, 16), (1, 128, 128), (1, 2112, 7168), (2, 130, 144), (3, 576, 112), (7, 100, 256), (8, 1000, 1536), (16, 64, 7168),
         (17, 129, 272), (31, 2112, 512), (32, 7168, 2048), (33, 257, 400), (64, 200, 576), (65, 640, 16384), (100, 5000, 640),
         (127, 1111, 1024), (128, 128, 128), (129, 4096, 528), (200, 8192, 1536), (255, 576, 7168), (256, 256, 256),
         (257, 2050, 384), (500, 3000, 1008), (777, 1536, 1536), (1000, 130, 96), (1025, 7168, 512), (2048, 576, 1024),
         (4097, 320, 640), (3001, 2500, 272)]


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", SIZES)
def test_whole_products_are_exact(cuda_lib, m, n, k):
    a, a_scale, b, b_scale = whole(m, n, k, gen(m, n, k))
    want, _ = definition(a, a_scale, b, b_scale)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for dtype in TYPES:
        out = dsa.matmul_fp8(a, a_scale, b, b_scale, dtype=dtype, status=status)
        assert out.dtype == dtype and torch.equal(out, want.float().to(dtype)), dtype
    assert int(status) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("m,n,k", SIZES)
def test_any_values(cuda_lib, m, n, k, dtype):
    a, a_scale, b, b_scale = any_values(m, n, k, gen(n, m, k))
    want, size = definition(a, a_scale, b, b_scale)
    out = dsa.matmul_fp8(a, a_scale, b, b_scale, dtype=dtype)
    tiny = torch.finfo(dtype).smallest_normal
    off = size * OFF + (want.abs() + tiny) * torch.finfo(dtype).eps / 2
    assert torch.all((out.double() - want).abs() <= off)
    # the same call gives the same bits
    assert torch.equal(out, dsa.matmul_fp8(a, a_scale, b, b_scale, dtype=dtype))


def spread(t, rows_apart, fill):
    """The same rows, `rows_apart` elements from one to the next, in memory filled with `fill`."""
    wide = torch.full((t.shape[0], rows_apart), fill, device=t.device).to(t.dtype)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("m,n,k", [(5, 100, 144), (130, 384, 208), (300, 515, 640), (700, 2000, 512)])
def test_strided_rows(cuda_lib, m, n, k, dtype):
    """Operands inside NaN, scales inside NaN, outputs inside memory that has to stay as it is."""
    a, a_scale, b, b_scale = whole(m, n, k, gen(m, k))
    want = definition(a, a_scale, b, b_scale)[0].float().to(dtype)
    blocks = a_scale.shape[1]
    out = torch.full((m + 1, n + 3), 5.0, dtype=dtype, device="cuda")
    dsa.matmul_fp8(spread(a, k + 48, math.nan), spread(a_scale, blocks + 3, math.nan), spread(b, k + 32, math.nan),
                   spread(b_scale, blocks + 1, math.nan), out=out[:m, :n])
    assert torch.equal(out[:m, :n], want)
    assert torch.all(out[m:] == 5.0) and torch.all(out[:, n:] == 5.0)
    # an output that starts on an odd element
    odd = torch.full((m, n + 1), 5.0, dtype=dtype, device="cuda")
    dsa.matmul_fp8(a, a_scale, b, b_scale, out=odd[:, 1:])
    assert torch.equal(odd[:, 1:], want) and torch.all(odd[:, 0] == 5.0)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 20, 130, 600])
def test_what_is_not_finite_stays_in_its_row(cuda_lib, m):
    n, k = 300, 400
    a, a_scale, b, b_scale = whole(m, n, k, gen(m))
    clean = dsa.matmul_fp8(a, a_scale, b, b_scale, dtype=torch.float32)
    row, col = m // 2, 133
    a2, b2, a_scale2 = a.clone(), b.clone(), a_scale.clone()
    a2.view(torch.uint8)[row, k - 1] = 0x7f
    got = dsa.matmul_fp8(a2, a_scale, b, b_scale, dtype=torch.float32)
    keep = torch.arange(m, device="cuda") != row
    assert torch.all(got[row].isnan()) and torch.equal(got[keep], clean[keep])
    b2.view(torch.uint8)[col, 0] = 0xff
    got = dsa.matmul_fp8(a, a_scale, b2, b_scale, dtype=torch.float32)
    cols = torch.arange(n, device="cuda") != col
    assert torch.all(got[:, col].isnan()) and torch.equal(got[:, cols], clean[:, cols])
    a_scale2[row, 1] = math.nan
    got = dsa.matmul_fp8(a, a_scale2, b, b_scale, dtype=torch.float32)
    assert torch.all(got[row].isnan()) and torch.equal(got[keep], clean[keep])
    a_scale2[row, 1] = math.inf
    got = dsa.matmul_fp8(a, a_scale2, b, b_scale, dtype=torch.float32)
    assert not torch.isfinite(got[row]).any() and torch.equal(got[keep], clean[keep])


@pytest.mark.gpu
def test_largest_codes_and_small_scales(cuda_lib):
    """Sums of 448 * 448 at their largest, beside scales that make fp16 overflow or vanish."""
    m, n, k = 40, 256, 2048
    a = torch.full((m, k), 448.0, device="cuda").to(torch.float8_e4m3fn)
    b = torch.full((n, k), 448.0, device="cuda").to(torch.float8_e4m3fn)
    a_scale, b_scale = torch.ones((m, 16), device="cuda"), torch.ones((2, 16), device="cuda")
    out = dsa.matmul_fp8(a, a_scale, b, b_scale, dtype=torch.float32)
    assert torch.all(out == 448.0 * 448.0 * k)
    assert torch.all(dsa.matmul_fp8(a, a_scale, b, b_scale, dtype=torch.float16).isinf())
    a_scale.fill_(2.0 ** -126)
    out = dsa.matmul_fp8(a, a_scale, b, b_scale, dtype=torch.float32)
    assert torch.all(out == 448.0 * 448.0 * k * 2.0 ** -126)


@pytest.mark.gpu
def test_rows_of_an_fp8_latent_cache(cuda_lib):
    """The rows' first 512 codes and their scales, as they lie in the pages that cache_write_quant wrote."""
    g = torch.Generator(device="cuda").manual_seed(2)
    L, n = 500, 768
    pool = torch.full((9, 64, 608), 0xff, dtype=torch.uint8, device="cuda")
    pt = torch.arange(9, dtype=torch.int32, device="cuda")[None]
    pos = torch.arange(L, dtype=torch.int32, device="cuda")
    dsa.cache_write_quant(pool, pt, torch.zeros_like(pos), pos, torch.randn((L, 576), generator=g, device="cuda"))
    a = pool.view(torch.float8_e4m3fn).view(-1, 608)[:L, :512]
    a_scale = pool.view(torch.float32).view(-1, 152)[:L, 144:148]
    _, _, b, b_scale = any_values(1, n, 512, g)
    want, size = definition(a, a_scale, b, b_scale)
    out = dsa.matmul_fp8(a, a_scale, b, b_scale)
    assert torch.all((out.double() - want).abs() <= size * OFF + want.abs() * 2.0 ** -8)


@pytest.mark.gpu
def test_offsets_beyond_32_bits(cuda_lib):
    """Rows that lie 1 GB apart in every tensor."""
    m, n, k = 5, 9, 256
    a, a_scale, b, b_scale = whole(m, n, k, gen(3))
    want = dsa.matmul_fp8(a, a_scale, b, b_scale)
    raw = torch.zeros(9 * 2 ** 30, dtype=torch.uint8, device="cuda")
    far = lambda t, size, at: raw.view(t.dtype)[at:].as_strided(t.shape, (2 ** 30 // size, 1))
    fa, fb, fs, fo = far(a, 1, 0), far(b, 1, 4096), far(a_scale, 4, 4096), far(want, 2, 16384)
    fa.copy_(a), fb.copy_(b), fs.copy_(a_scale)
    dsa.matmul_fp8(fa, fs, fb, b_scale, out=fo)
    assert torch.equal(fo, want)


@pytest.mark.gpu
def test_an_output_beyond_32_bits(cuda_lib):
    """2.2e9 outputs: the last rows are those of a call of their own."""
    m, n, k = 33000, 66000, 16
    a, a_scale, b, b_scale = whole(m, n, k, gen(4))
    out = dsa.matmul_fp8(a, a_scale, b, b_scale)
    assert torch.equal(out[-300:], dsa.matmul_fp8(a[-300:], a_scale[-300:], b, b_scale))
    assert torch.equal(out[:50], dsa.matmul_fp8(a[:50], a_scale[:50], b, b_scale))


@pytest.mark.gpu
def test_no_rows(cuda_lib):
    a, a_scale, b, b_scale = whole(4, 64, 128, gen(5))
    assert dsa.matmul_fp8(a[:0], a_scale[:0], b, b_scale).shape == (0, 64)


@pytest.mark.gpu
def test_streams_and_graphs(cuda_lib):
    """Calls on four streams at once, and a captured run of the three operators, replayed on new inputs."""
    streams = [torch.cuda.Stream() for _ in range(4)]
    cases = [whole(m, n, k, gen(m)) for m, n, k in ((1, 2112, 7168), (32, 1024, 2048), (200, 640, 512), (900, 1536, 768))]
    want = [definition(*c)[0].float().bfloat16() for c in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for s, c in zip(streams, cases):
            with torch.cuda.stream(s):
                got.append(dsa.matmul_fp8(*c))
    outs = [dsa.matmul_fp8(*c, stream=s) for s, c in zip(streams, cases)]
    torch.cuda.synchronize()
    for i, o in enumerate(got + outs):
        assert torch.equal(o, want[i % 4])

    g = torch.Generator(device="cuda").manual_seed(9)
    x, r = (torch.randn((40, 1536), generator=g, device="cuda").bfloat16() for _ in range(2))
    w = torch.rand(1536, generator=g, device="cuda").bfloat16()
    _, _, b, b_scale = any_values(1, 1536, 1536, g)

    def step():
        codes, scale, total = dsa.rms_norm_quant(x, w, residual=r)
        y = dsa.matmul_fp8(codes, scale, b, b_scale)
        return dsa.matmul_fp8(*dsa.quant_rows(y), b, b_scale, dtype=torch.float32), total

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, total = step()
    for _ in range(3):
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        graph.replay()
        again = step()
        assert torch.equal(out, again[0]) and torch.equal(total, again[1])


@pytest.mark.gpu
def test_a_layer_around_the_attention(cuda_lib):
    """One decode step of a layer: norm, down-projection, the cache rows' write, the up-projections, dense latent attention
    in the expanded form on rows that the product reads from the cache, and the output projection; against the same
    steps in 64 bits on the values that each step got.  (Each step's own tolerance is derived where it is tested
    alone: here a wrong row, scale or stride would be off by the size of the values.)"""
    g = torch.Generator(device="cuda").manual_seed(12)
    L, T, H, D, DQ = 200, 5, 4, 1024, 512
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
    weights = lambda n, k: any_values(1, n, k, g)[2:]
    wd, wq, wkv, wo = weights(DQ + 576, D), weights(H * 192, DQ), weights(H * 256, 512), weights(D, H * 128)
    value = lambda b, s: b.double() * s.double().repeat_interleave(128, 0)[:b.shape[0]].repeat_interleave(128, 1)[:, :b.shape[1]]
    near = lambda got, want, tol: bool((got.double() - want).norm() <= tol * want.norm())
    x, res, gamma, gamma_q = rnd(L, D).bfloat16(), rnd(L, D).bfloat16(), rnd(D).abs() + 0.5, rnd(DQ).abs() + 0.5
    codes, scale, h = dsa.rms_norm_quant(x, gamma, residual=res)
    down = dsa.matmul_fp8(codes, scale, *wd, dtype=torch.float32)
    hd = h.double()
    v = hd / torch.sqrt((hd * hd).mean(1, keepdim=True) + 1e-6) * gamma.double()
    assert near(down, v @ value(*wd).T, 0.06)     # e4m3 rows: half a step is 2^-4 at most, 2^-5.4 in the mean square
    qc, qs = dsa.rms_norm_quant(down[-T:, :DQ], gamma_q)
    q = dsa.matmul_fp8(qc, qs, *wq).view(T, H, 192)
    pool = torch.zeros((4, 64, 608), dtype=torch.uint8, device="cuda")
    pt, pos = torch.arange(4, dtype=torch.int32, device="cuda")[None], torch.arange(L, dtype=torch.int32, device="cuda")
    dsa.cache_write_quant(pool, pt, torch.zeros_like(pos), pos, down[:, DQ:])
    rows = pool.view(-1, 608)
    kv = dsa.matmul_fp8(rows.view(torch.float8_e4m3fn)[:L, :512], pool.view(torch.float32).view(-1, 152)[:L, 144:148], *wkv)
    back = dsa.cache_read(pool, pt, torch.zeros_like(pos), pos)
    # bf16 copies of the rows, then bf16 outputs: 2^-8 each at most
    assert near(kv, back[:, :512].double() @ value(*wkv).T, 2.0 ** -7)
    at = lambda *n: torch.tensor(n, dtype=torch.int32, device="cuda")
    o, _ = dsa.mla_prefill(q, kv.view(L, H, 256), back[:, 512:], at(0, T), at(0, L), softmax_scale=0.07, max_q_per_seq=T)
    y = dsa.matmul_fp8(*dsa.quant_rows(o.view(T, H * 128)), *wo)
    z = 0.07 * (torch.einsum("thd,jhd->htj", q[..., :128].double(), kv.view(L, H, 256)[..., :128].double())
                + torch.einsum("thd,jd->htj", q[..., 128:].double(), back[:, 512:].double()))
    z.masked_fill_(pos[None] > pos[-T:, None], -math.inf)
    want = torch.einsum("htj,jhd->thd", z.softmax(-1), kv.view(L, H, 256)[..., 128:].double())
    assert near(y, want.reshape(T, -1) @ value(*wo).T, 0.06)


def _args(**over):
    a = dsa.MatmulFp8Args()
    a.M, a.N, a.K, a.elem = 4, 256, 512, 0
    a.a_stride, a.a_scale_stride, a.b_stride, a.b_scale_stride, a.out_stride = 512, 4, 512, 4, 256
    for n in ("a", "a_scale", "b", "b_scale", "out"):
        setattr(a, n, 4096)  # fake, aligned, never dereferenced on these error paths
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,code", [
    ({"M": -1}, dsa.DSA_ERR_INVALID_ARG),
    ({"N": 0}, dsa.DSA_ERR_INVALID_ARG),
    ({"K": 0}, dsa.DSA_ERR_INVALID_ARG),
    ({"K": 520}, dsa.DSA_ERR_UNSUPPORTED),
    ({"M": 0x7fffff80}, dsa.DSA_ERR_UNSUPPORTED),
    ({"elem": 3}, dsa.DSA_ERR_INVALID_ARG),
    ({"a": None}, dsa.DSA_ERR_INVALID_ARG),
    ({"b_scale": None}, dsa.DSA_ERR_INVALID_ARG),
    ({"out": None}, dsa.DSA_ERR_INVALID_ARG),
    ({"a": 4104}, dsa.DSA_ERR_INVALID_ARG),
    ({"b": 4097}, dsa.DSA_ERR_INVALID_ARG),
    ({"out": 4097}, dsa.DSA_ERR_INVALID_ARG),
    ({"a_scale": 4098}, dsa.DSA_ERR_INVALID_ARG),
    ({"a_stride": 496}, dsa.DSA_ERR_INVALID_ARG),
    ({"b_stride": 520}, dsa.DSA_ERR_INVALID_ARG),
    ({"b_stride": 1 << 40}, dsa.DSA_ERR_INVALID_ARG),
    ({"a_scale_stride": 3}, dsa.DSA_ERR_INVALID_ARG),
    ({"out_stride": 255}, dsa.DSA_ERR_INVALID_ARG),
])
def test_host_validation(over, code):
    lib = dsa.load()
    assert lib.dsa_matmul_fp8(ctypes.byref(_args(**over)), None) == code, dsa.last_error()
    assert dsa.last_error()
    assert lib.dsa_matmul_fp8(None, None) == dsa.DSA_ERR_INVALID_ARG
    assert lib.dsa_matmul_fp8(ctypes.byref(_args(M=0)), None) == dsa.DSA_OK


def test_struct_layout():
    assert ctypes.sizeof(dsa.MatmulFp8Args) == 4 * 4 + 5 * 8 + 6 * 8


def test_binding_refuses_cpu_tensors():
    a, s = torch.zeros((4, 256)).to(torch.float8_e4m3fn), torch.ones((4, 2))
    with pytest.raises(ValueError):
        dsa.matmul_fp8(a, s, a, s[:1])


@pytest.mark.gpu
def test_binding_refuses_what_does_not_fit(cuda_lib):
    a, a_scale, b, b_scale = whole(4, 256, 512, gen(6))
    out = torch.empty((4, 256), device="cuda")
    for bad in (dict(a=a.view(torch.uint8)), dict(a=a[0]), dict(a=a[:, :256]), dict(a=a[:1].expand(4, 512)),
                dict(a=a.T.contiguous().T), dict(a_scale=a_scale[:, :3]), dict(a_scale=a_scale.double()),
                dict(a_scale=a_scale.cpu()), dict(b=b[:, :256]), dict(b=b.float()), dict(b_scale=b_scale[:1]),
                dict(b_scale=b_scale.T.contiguous().T), dict(out=out.double()), dict(out=out[:, :255]),
                dict(out=out.T.contiguous().T), dict(dtype=torch.float64), dict(dtype=torch.int32),
                dict(status=torch.zeros(1, device="cuda"))):
        kw = dict(a=a, a_scale=a_scale, b=b, b_scale=b_scale)
        kw.update(bad)
        with pytest.raises(ValueError):
            dsa.matmul_fp8(**kw)
    with pytest.raises(dsa.DsaError):
        dsa.matmul_fp8(a[:, 8:264], a_scale[:, :2], b[:, :256], b_scale[:, :2])   # rows that start on 8 bytes


# Sizes that large calls divide into wide tiles: blocks below, at and above the eight whose scales are multiplied at a time,
# last blocks of 16 columns, a last tile of one row or column, rows of out that a TMA store cannot reach
WIDE = [(2500, 2500, 16), (2300, 2560, 896), (2300, 2561, 1024), (2049, 2304, 1152), (5000, 1537, 2192), (20000, 256, 144),
        (4100, 5121, 400), (700, 7000, 2064), (257, 16000, 1200), (130, 20000, 640), (8193, 2049, 1040)]
# ... and into narrow ones of every width and number of splits
NARROW = [(9, 2112, 7168), (40, 7168, 16384), (100, 7168, 7168), (16, 24576, 1536), (5, 1000, 400), (64, 100, 16384),
          (128, 640, 3600), (90, 2000, 2048), (128, 576, 7168), (1, 7168, 1040), (64, 7168, 1040), (200, 8192, 1024),
          (160, 2112, 3584), (120, 5000, 3600)]


def test_the_sizes_reach_every_variant():
    plan = dsa.load_testhooks().dsa_test_matmul_plan
    assert all(plan(*s, 152) == 0 for s in WIDE)
    got = {plan(*s, 152) for s in NARROW + SIZES}
    assert {divmod(v, 16)[0] for v in got} >= {32, 64, 96, 128} and {v % 16 for v in got} == {0, 1, 2, 4, 8}


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", WIDE + NARROW)
def test_whole_products_of_every_variant_are_exact(cuda_lib, m, n, k):
    a, a_scale, b, b_scale = whole(m, n, k, gen(m, n, k))
    want = definition(a, a_scale, b, b_scale)[0].float()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for dtype in TYPES:
        out = torch.full((m, n), math.nan, dtype=dtype, device="cuda")
        dsa.matmul_fp8(a, a_scale, b, b_scale, out=out, status=status)
        assert torch.equal(out, want.to(dtype)), dtype
    assert int(status) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [WIDE[1], WIDE[2], WIDE[4], NARROW[0], NARROW[2], NARROW[5]])
def test_any_values_of_every_variant(cuda_lib, m, n, k):
    a, a_scale, b, b_scale = any_values(m, n, k, gen(n, k, m))
    want, size = definition(a, a_scale, b, b_scale)
    out = dsa.matmul_fp8(a, a_scale, b, b_scale, dtype=torch.float32)
    assert torch.all((out.double() - want).abs() <= size * OFF + want.abs() * 2.0 ** -24)
    assert torch.equal(out, dsa.matmul_fp8(a, a_scale, b, b_scale, dtype=torch.float32))


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(2300, 2560, 896), (700, 7000, 2064)])
def test_wide_tiles_with_strided_rows(cuda_lib, m, n, k):
    """As test_strided_rows: operands and scales inside NaN, and what is not written stays, with a TMA store and without."""
    a, a_scale, b, b_scale = whole(m, n, k, gen(m, k))
    want = definition(a, a_scale, b, b_scale)[0].float()
    args = (spread(a, k + 48, math.nan), spread(a_scale, a_scale.shape[1] + 3, math.nan), spread(b, k + 32, math.nan),
            spread(b_scale, b_scale.shape[1] + 1, math.nan))
    for dtype in TYPES:
        for left, right in ((0, 16), (8, 8), (1, 2)):
            out = torch.full((m + 1, left + n + right), 5.0, dtype=dtype, device="cuda")
            dsa.matmul_fp8(*args, out=out[:m, left:left + n])
            assert torch.equal(out[:m, left:left + n], want.to(dtype))
            out[:m, left:left + n] = 5.0
            assert torch.all(out == 5.0)


@pytest.mark.gpu
def test_what_is_not_finite_stays_in_its_row_of_a_wide_tile(cuda_lib):
    m, n, k = 2300, 2560, 896
    a, a_scale, b, b_scale = whole(m, n, k, gen(8))
    clean = dsa.matmul_fp8(a, a_scale, b, b_scale, dtype=torch.float32)
    a.view(torch.uint8)[777, 500], b.view(torch.uint8)[1300, 3], a_scale[2299, 6] = 0x7f, 0xff, math.nan
    got = dsa.matmul_fp8(a, a_scale, b, b_scale, dtype=torch.float32)
    bad = torch.zeros((m, n), dtype=torch.bool, device="cuda")
    bad[777], bad[2299], bad[:, 1300] = True, True, True
    assert torch.all(got[bad].isnan()) and torch.equal(got[~bad], clean[~bad])


@pytest.mark.gpu
def test_wide_and_narrow_calls_at_once(cuda_lib):
    """Both kinds on four streams: each keeps tensor memory that the other waits for."""
    sizes = [(2300, 2560, 896), (9, 2112, 7168), (2049, 2304, 1152), (100, 7168, 1024)]
    cases = [whole(m, n, k, gen(m, n)) for m, n, k in sizes]
    want = [definition(*c)[0].float().bfloat16() for c in cases]
    streams = [torch.cuda.Stream() for _ in sizes]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for s, c in zip(streams, cases):
            with torch.cuda.stream(s):
                got.append(dsa.matmul_fp8(*c))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i % 4]) for i, o in enumerate(got))


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(2300, 2562, 400), (2300, 2566, 272), (100, 7166, 272), (9, 2110, 7168), (33, 258, 640)])
def test_rows_of_out_that_start_on_even_elements(cuda_lib, m, n, k):
    """Rows that are not 16-byte aligned, with an even and with an odd number of columns inside an even stride."""
    a, a_scale, b, b_scale = whole(m, n, k, gen(m, n))
    want = definition(a, a_scale, b, b_scale)[0].float()
    for dtype in TYPES:
        for cols in (n, n - 1):
            for left in (0, 2, 1):
                out = torch.full((m, n + 2 + (n & 1)), 5.0, dtype=dtype, device="cuda")
                dsa.matmul_fp8(a, a_scale, b[:cols], b_scale[:-(-cols // 128)], out=out[:, left:left + cols])
                assert torch.equal(out[:, left:left + cols], want[:, :cols].to(dtype)), (dtype, cols, left)
                out[:, left:left + cols] = 5.0
                assert torch.all(out == 5.0)


@pytest.mark.gpu
def test_products_beside_the_indexer(cuda_lib):
    """Narrow products, whose CTAs share SMs, and the indexer, whose clusters hold tensor memory too, on two streams."""
    import dsa_inputs as di
    wl = di.small("decode_32k_fp8", seq_lens=[2000] * 24, n_new=[4] * 24)
    inp = di.to_device(di.generate(wl), "cuda")
    li = lambda: dsa.li_topk(inp["q_li"], inp["w"], inp["k_pool"], inp["pt_k"], inp["seq_lens"], inp["q_start"], wl.K,
                             q_scale=inp["q_scale"], k_scale=inp["k_scale"], max_seq_len=2000, max_q_per_seq=4)[0]
    case = whole(9, 2112, 7168, gen(1))
    idx, out = li(), dsa.matmul_fp8(*case)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(30):
        with torch.cuda.stream(streams[0]):
            a = li()
        with torch.cuda.stream(streams[1]):
            b = dsa.matmul_fp8(*case)
        got.append((a, b))
    torch.cuda.synchronize()
    assert all(torch.equal(a, idx) and torch.equal(b, out) for a, b in got)


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(2300, 2560, 9232), (700, 7000, 16384)])
def test_scales_of_long_rows_in_wide_tiles(cuda_lib, m, n, k):
    """Many sets of eight blocks' scales, each in the place of one that all warps must have read; again and again.
    (Terms are multiples of 2^-2 and at most 9 * 4, so sums of 16,384 are below 2^24 of them: exact.)"""
    assert dsa.load_testhooks().dsa_test_matmul_plan(m, n, k, 152) == 0
    case = whole(m, n, k, gen(m, n, k))
    want = definition(*case)[0].float()
    for _ in range(10):
        assert torch.equal(dsa.matmul_fp8(*case, dtype=torch.float32), want)


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(1, 300, 400), (130, 2112, 1040), (2300, 2560, 896)])
def test_a_scale_of_b_that_is_not_finite_reaches_its_128_columns(cuda_lib, m, n, k):
    a, a_scale, b, b_scale = whole(m, n, k, gen(m, n))
    clean = dsa.matmul_fp8(a, a_scale, b, b_scale, dtype=torch.float32)
    b_scale[1, 2] = math.nan
    got = dsa.matmul_fp8(a, a_scale, b, b_scale, dtype=torch.float32)
    assert torch.all(got[:, 128:256].isnan())
    assert torch.equal(got[:, :128], clean[:, :128]) and torch.equal(got[:, 256:], clean[:, 256:])


@pytest.mark.parametrize("over", [{"N": 2 ** 31 - 255}, {"K": 2 ** 31 - 128}])
def test_limits_of_the_header_are_refused(over):
    """(More tiles than a launch numbers are refused after the device is asked, so not here.)"""
    a = _args(a_stride=2 ** 39, b_stride=2 ** 39, out_stride=2 ** 37, **over)
    assert dsa.load().dsa_matmul_fp8(ctypes.byref(a), None) == dsa.DSA_ERR_UNSUPPORTED and "2^31" in dsa.last_error()


# Every width of narrow tiles with every number of CTAs that share a tile's blocks, one row of tiles (where the plan gives
# it) and several
PAIRS = {(32, 1): [(5, 33, 144), (137, 34, 144)], (32, 2): [(95, 1226, 1760), (2442, 33, 2080)],
         (32, 4): [(5, 34, 784), (1187, 33, 1296)], (32, 8): [(5, 33, 1104), (134, 35, 1248)],
         (64, 1): [(71, 8998, 144), (130, 2889, 144)], (64, 2): [(5, 7733, 1200), (132, 1879, 3488)],
         (64, 4): [(5, 2361, 832), (131, 711, 2560)], (64, 8): [(5, 1025, 1056), (1449, 33, 4816)],
         (96, 1): [(129, 5583, 160)], (96, 2): [(5, 7279, 1440), (129, 2698, 4224)],
         (96, 4): [(5, 3235, 928), (140, 1247, 2960)], (96, 8): [(5, 1223, 1072), (139, 642, 3680)],
         (128, 1): [(133, 7755, 144)], (128, 2): [(87, 7857, 4256), (129, 4093, 6048)],
         (128, 4): [(5, 4745, 992), (129, 1901, 4528)], (128, 8): [(5, 2092, 1040), (130, 871, 10400)]}


def test_the_pairs_are_what_the_plan_gives():
    plan = dsa.load_testhooks().dsa_test_matmul_plan
    assert set(PAIRS) == {(bn, s) for bn in (32, 64, 96, 128) for s in (1, 2, 4, 8)}
    for pair, sizes in PAIRS.items():
        assert all(divmod(plan(*s, 152), 16) == pair for s in sizes)


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [s for sizes in PAIRS.values() for s in sizes])
def test_every_pair_of_width_and_splits_is_exact(cuda_lib, m, n, k):
    """Rows of out that start 16-byte aligned, on an even element and on an odd one, with an odd number of columns and
    with an even one; what lies around them stays."""
    a, a_scale, b, b_scale = whole(m, n, k, gen(m, n, k))
    want = definition(a, a_scale, b, b_scale)[0].float()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    wide = (n + 23) // 8 * 8
    for dtype in TYPES:
        for cols in (n, n - 1):
            for left, apart in ((0, wide), (8, wide), (2, wide), (1, wide), (0, wide + 1), (0, wide + 2)):
                out = torch.full((m, apart), 5.0, dtype=dtype, device="cuda")
                dsa.matmul_fp8(a, a_scale, b[:cols], b_scale[:-(-cols // 128)], out=out[:, left:left + cols], status=status)
                assert torch.equal(out[:, left:left + cols], want[:, :cols].to(dtype)), (dtype, cols, left, apart)
                out[:, left:left + cols] = 5.0
                assert torch.all(out == 5.0)
    assert int(status) == 0
