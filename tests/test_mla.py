"""Dense latent attention, absorbed (mla_decode) and expanded (mla_prefill), against its definition
in 64 bits.

Tolerances, element by element, from what the kernels round.  With p the exact softmax weights and
A = sum p |v| of an output element:
  - the output is rounded to bf16:                        2^-8 A  (|out| <= A)
  - each weight is rounded to bf16 before P.V:            2^-8 A, and 2^-8 A more where the sum of
    weights that divides it is not the sum of the rounded ones
  - the logits are fp32 sums of exact bf16 products: an error of at most n 2^-24 sum |q k| scale for
    n products, which moves a weight by twice that, relatively (itself and the divisor); so do the
    2 ulp of the exponential and the additions of the fp32 accumulators (2^-24 each, n of them at
    most, of values that sum to A).
lse: the logits' error, and 2^-24 per addition of a positive sum.
"""
import ctypes
import math

import pytest
import torch

import dsa_sparse_attention_li_gb300 as dsa

SCALE = 192 ** -0.5


def definition(q, k, v, seen, scale):
    """q [n, d], k [L, d], v [L, dv], seen [n, L] -> out, lse, A, and the logits' magnitude."""
    z = (q @ k.T) * scale
    z = torch.where(seen, z, -math.inf)
    lse = torch.logsumexp(z, 1)
    p = torch.where(seen, torch.exp(z - lse[:, None]), 0.0)
    p = torch.nan_to_num(p)  # rows that see nothing
    mag = torch.where(seen, (q.abs() @ k.abs().T) * scale, 0.0).amax(1) if k.shape[0] else lse * 0
    return p @ v, lse, p @ v.abs(), mag


def check(got, lse, want, want_lse, A, mag, n_products, length):
    err_z = n_products * 2.0 ** -24 * mag
    rel = 3 * 2.0 ** -8 + 2 * err_z + 2.0 ** -21 + length * 2.0 ** -24
    tol = A * rel[:, None] + 1e-30
    bad = (got.double() - want).abs() > tol
    assert not bad.any(), ((got.double() - want).abs() / tol).max()
    empty = torch.isneginf(want_lse)
    assert torch.equal(torch.isneginf(lse), empty)
    tol = err_z + 2.0 ** -21 + length * 2.0 ** -24 + want_lse.abs() * 2.0 ** -22
    bad = (lse.double() - want_lse).abs()[~empty] > tol[~empty]
    assert not bad.any(), ((lse.double() - want_lse).abs() / tol)[~empty].max()


# ------------------------------------------------------------------------------------------
# absorbed form
# ------------------------------------------------------------------------------------------

def page_tables(lens, extra, g):
    """A page table of random pages for the lengths, `extra` unused columns (an id out of range in
    them) and 2 pages that no sequence owns."""
    counts = [-(-n // 64) for n in lens]
    order = torch.randperm(sum(counts) + 2, generator=g).to(torch.int32)
    pt = torch.full((len(lens), max(1, max(counts)) + extra), 2 ** 30, dtype=torch.int32)
    at = 0
    for b, c in enumerate(counts):
        pt[b, :c] = order[at:at + c]
        at += c
    return pt, sum(counts) + 2


def kv8_rows(rows):
    """FP8 latent rows of random codes and scales, and the values they stand for."""
    g = torch.Generator(device=rows.device).manual_seed(1)
    n = rows.shape[0]
    packed = torch.full((n, 608), 0xAB, dtype=torch.uint8, device=rows.device)
    codes = (rows * 32).clamp(-448, 448).to(torch.float8_e4m3fn)
    scale = (torch.rand((n, 5), generator=g, device=rows.device) + 0.5) / 32
    packed[:, :576] = codes.view(torch.uint8)
    packed[:, 576:596] = scale.view(torch.uint8)
    return packed, (codes.float() * scale.repeat_interleave(128, 1)[:, :576]).bfloat16()


def make_decode(lens, new, H, fp8, seed=0, extra=1, grow=0.0, tail=3, q_scale=1.0):
    """A batch whose cache rows past a sequence's end, and whose unowned pages, hold NaN and
    infinities; `tail` query rows behind the last sequence.  With `grow` the keys turn towards the
    queries along the sequence, so that the running maximum moves all the way."""
    g = torch.Generator().manual_seed(seed)
    pt, pages = page_tables(lens, extra, g)
    gd = torch.Generator(device="cuda").manual_seed(seed)
    n_q = sum(new)
    q = (torch.randn((n_q + tail, H, 576), generator=gd, device="cuda") * q_scale).bfloat16()
    pool = torch.full((pages * 64, 576), math.nan, dtype=torch.bfloat16, device="cuda")
    pool[::2] = math.inf
    pool8 = torch.full((pages * 64, 608), 0x7F, dtype=torch.uint8, device="cuda") if fp8 else None
    rows = []
    for b, L in enumerate(lens):
        x = torch.randn((L, 576), generator=gd, device="cuda")
        if grow and L:
            x += grow * torch.linspace(0, 1, L, device="cuda")[:, None] * q[0, 0].float().sign()
        at = (pt[b, :-(-L // 64)].long()[:, None] * 64 + torch.arange(64)).view(-1)[:L].cuda()
        if fp8:
            pool8[at], x = kv8_rows(x)
        pool[at] = x.bfloat16()
        rows.append(pool[at].double())
    q_start = torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int32)
    return {"q": q, "pool": (pool8.view(pages, 64, 608) if fp8 else pool.view(pages, 64, 576)), "pt": pt.cuda(),
            "seq_lens": torch.tensor(lens, dtype=torch.int32).cuda(), "q_start": q_start.cuda(), "rows": rows,
            "new": new, "lens": lens, "H": H, "tail": tail}


def run_decode(c, **kw):
    n = c["q"].shape[0]
    out = torch.full((n, c["H"], 512), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n, c["H"]), 6.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = {"softmax_scale": SCALE, "max_q_per_seq": max(1, max(c["new"])), "out": out, "lse": lse,
          "status": status, **kw}
    dsa.mla_decode(c["q"], c["pool"], c["pt"], c["seq_lens"], c["q_start"], **kw)
    torch.cuda.synchronize()
    return out, lse, int(status)


def verify_decode(c, out, lse, scale=SCALE):
    t = 0
    for b, n in enumerate(c["new"]):
        L, kv = c["lens"][b], c["rows"][b]
        if n == 0:
            continue
        q = c["q"][t:t + n].double().view(n * c["H"], 576)
        last = (L - n + torch.arange(n, device="cuda")).repeat_interleave(c["H"])
        seen = torch.arange(L, device="cuda")[None] <= last[:, None]
        want = definition(q, kv, kv[:, :512], seen, scale)
        check(out[t:t + n].view(n * c["H"], 512), lse[t:t + n].view(-1), *want, 576, L)
        t += n
    if c["tail"]:
        assert torch.all(out[t:] == 5.0) and torch.all(lse[t:] == 6.0)


DECODE = [
    (1, [1], [1]), (16, [63], [1]), (128, [64], [1]), (128, [65], [1]), (1, [129], [1]), (5, [128, 1, 192], [1, 1, 1]),
    (128, [4096], [1]), (16, [4096], [1]), (100, [777, 5000], [1, 1]), (64, [300, 1000], [2, 2]),
    (16, [200, 1, 0, 9, 513], [3, 1, 0, 9, 8]),       # an empty sequence; a sequence that is all new
    (48, [130, 64, 0], [130, 5, 0]), (128, [150], [150]), (7, [400], [40]),
    (32, [3, 0, 70], [5, 2, 1]),                      # more tokens than positions: some see nothing
    (128, [20011, 77, 4096, 640], [1, 1, 1, 1]), (24, [60000], [4]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("H,lens,new", DECODE, ids=lambda v: str(v).replace(" ", "")[:28])
def test_decode_matches_the_definition(cuda_lib, H, lens, new, fp8):
    c = make_decode(lens, new, H, fp8, seed=H + len(lens))
    out, lse, status = run_decode(c)
    assert status == 0
    verify_decode(c, out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_decode_many_sequences(cuda_lib, fp8):
    g = torch.Generator().manual_seed(2)
    lens = torch.randint(0, 700, (300,), generator=g).tolist()
    new = [min(n, k) for n, k in zip(lens, torch.randint(0, 4, (300,), generator=g).tolist())]
    c = make_decode(lens, new, 40, fp8, seed=9)
    out, lse, status = run_decode(c)
    assert status == 0
    verify_decode(c, out, lse)
    # a bound of the tokens that is too small, or larger than any sequence has, changes the grouping only
    for bound in (1, 3, 50):
        out, lse, status = run_decode(c, max_q_per_seq=bound)
        assert status == 0
        verify_decode(c, out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("grow,q_scale", [(4.0, 1.0), (-4.0, 1.0), (0.0, 12.0), (0.0, 0.0)])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_decode_moving_maximum(cuda_lib, grow, q_scale, fp8):
    """Logits that grow (or fall) by thousands along the sequence, peaked ones, and all-equal ones."""
    c = make_decode([3000, 500], [1, 3], 20, fp8, grow=grow, q_scale=q_scale)
    out, lse, status = run_decode(c)
    assert status == 0
    verify_decode(c, out, lse)


@pytest.mark.gpu
def test_decode_repeats_bit_for_bit_and_captures(cuda_lib):
    c = make_decode([9000, 100, 3333], [2, 1, 2], 64, False)
    first = run_decode(c)
    second = run_decode(c, workspace=torch.full((dsa.mla_decode_workspace_bytes(8, 64, 2) + 256,), 0xFF,
                                                dtype=torch.uint8, device="cuda"))
    assert torch.equal(first[0], second[0]) and torch.equal(first[1], second[1])
    out, lse = torch.zeros_like(first[0]), torch.zeros_like(first[1])
    ws = torch.empty(dsa.mla_decode_workspace_bytes(c["q"].shape[0], 64, 2), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for _ in range(2):  # back to back: the second reads what the first may still be using
            dsa.mla_decode(c["q"], c["pool"], c["pt"], c["seq_lens"], c["q_start"], softmax_scale=SCALE,
                           max_q_per_seq=2, out=out, lse=lse, workspace=ws)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    n = sum(c["new"])
    assert torch.equal(out[:n], first[0][:n]) and torch.equal(lse[:n], first[1][:n])
    # the lengths are read on the device: a replay sees the ones that are there then
    c["seq_lens"][0] -= 70
    graph.replay()
    torch.cuda.synchronize()
    c["lens"][0] -= 70
    c["rows"][0] = c["rows"][0][:-70]
    c["tail"] = 0
    verify_decode(c, out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_decode_hidden_rows_may_hold_anything(cuda_lib, fp8):
    """A draft token's own cache row is NaN or infinite: the tokens before it do not see it."""
    for bad in ((math.nan, 0x7F), (math.inf, 0x7F)):
        c = make_decode([191, 130], [2, 3], 16, fp8)
        for b, j in ((0, 190), (1, 128), (1, 129)):
            page = int(c["pt"][b, j // 64])
            c["pool"][page, j % 64] = bad[1] if fp8 else bad[0]
        out, lse, status = run_decode(c)
        assert status == 0
        ok = torch.tensor([True, False, True, False, False], device="cuda")
        assert torch.isfinite(out[:5][ok].float()).all() and torch.isfinite(lse[:5][ok]).all()
        assert torch.isnan(out[:5][~ok].float()).any(-1).all()
        for b, t, L in ((0, 0, 190), (1, 2, 128)):
            want = definition(c["q"][t].double(), c["rows"][b][:L], c["rows"][b][:L, :512],
                              torch.ones((16, L), dtype=torch.bool, device="cuda"), SCALE)
            check(out[t], lse[t], *want, 576, L)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_decode_on_two_streams_with_tokens_of_no_sequence(cuda_lib, fp8):
    """Two calls at once, each with its workspace; the first sequence starts behind four query rows
    that no sequence owns; both sequences share their first pages."""
    cases = []
    for seed in (1, 2):
        c = make_decode([1500, 4000], [1, 2], 32, fp8, seed=seed, tail=0)
        c["pt"][1, :8] = c["pt"][0, :8]
        c["rows"][1] = torch.cat([c["rows"][0][:512], c["rows"][1][512:]])
        lead = torch.full((4, 32, 576), math.nan, dtype=torch.bfloat16, device="cuda")
        c["q"] = torch.cat([lead, c["q"]])
        c["q_start"] += 4
        cases.append(c)
    streams = [torch.cuda.Stream() for _ in cases]
    outs = []
    torch.cuda.synchronize()
    for c, s in zip(cases, streams):
        out = torch.full((7, 32, 512), 5.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((7, 32), 6.0, device="cuda")
        outs.append((out, lse))
        for t in outs[-1]:
            t.record_stream(s)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(3):
                dsa.mla_decode(c["q"], c["pool"], c["pt"], c["seq_lens"], c["q_start"], softmax_scale=SCALE,
                               max_q_per_seq=2, out=out, lse=lse)
    torch.cuda.synchronize()
    for c, (out, lse) in zip(cases, outs):
        assert torch.all(out[:4] == 5.0) and torch.all(lse[:4] == 6.0)
        c["q"] = c["q"][4:]
        verify_decode(c, out[4:], lse[4:])


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
def test_stream_argument_while_the_current_stream_works_on(cuda_lib, handle):
    """What a call allocates for another stream is that stream's memory: tensors that the current stream
    makes and fills right after the call, while the launch still waits its turn, are not the call's
    workspace or outputs."""
    c, f = make_decode([9000, 100, 3333], [2, 1, 2], 64, False), make_prefill([200, 30], [500, 30], 4)
    want = run_decode(c) + run_prefill(f)
    rows = dsa.cache_read(c["pool"], c["pt"], torch.zeros(100, dtype=torch.int32, device="cuda"),
                          torch.arange(100, dtype=torch.int32, device="cuda"))
    side = torch.cuda.Stream()
    stream = side.cuda_stream if handle else side
    seq, pos = torch.zeros(100, dtype=torch.int32, device="cuda"), torch.arange(100, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    got = dsa.mla_decode(c["q"], c["pool"], c["pt"], c["seq_lens"], c["q_start"], softmax_scale=SCALE,
                         max_q_per_seq=2, stream=stream)
    got += dsa.mla_prefill(f["q"], f["kv"], f["rope"], f["q_start"], f["kv_start"], softmax_scale=SCALE,
                           max_q_per_seq=200, stream=stream)
    got += (dsa.cache_read(c["pool"], c["pt"], seq, pos, stream=stream),)
    ws = dsa.mla_decode_workspace_bytes(c["q"].shape[0], 64, 2)
    others = [torch.zeros(n, dtype=torch.uint8, device="cuda")
              for n in [ws] + [t.numel() * t.element_size() for t in got] for _ in range(2)]
    torch.cuda.synchronize()
    n, m = sum(c["new"]), 230
    assert torch.equal(got[0][:n], want[0][:n]) and torch.equal(got[1][:n], want[1][:n])
    assert torch.equal(got[2][:m], want[3][:m]) and torch.equal(got[3][:m], want[4][:m])
    assert torch.equal(got[4], rows)
    assert all(not bool(t.any()) for t in others)


@pytest.mark.gpu
def test_decode_reports_what_is_out_of_range(cuda_lib):
    c = make_decode([400, 200], [1, 1], 16, False, extra=0, tail=0)
    c["pt"][0, 2] = 10 ** 6
    out, lse, status = run_decode(c)
    assert status == dsa.DSA_ERR_DEVICE_CHECK
    keep = torch.ones(400, dtype=torch.bool)
    keep[128:192] = False            # the positions of the bad page are skipped
    c["rows"][0] = c["rows"][0][keep.cuda()]
    c["lens"][0] = 336
    verify_decode(c, out, lse)
    # a length beyond the page table is clamped to it, one below zero to nothing
    c = make_decode([448, 200], [1, 1], 16, False, extra=0, tail=0)
    c["seq_lens"][0] = 10 ** 6
    c["seq_lens"][1] = -5
    out, lse, status = run_decode(c)
    assert status == dsa.DSA_ERR_DEVICE_CHECK
    c["lens"], c["rows"][1] = [448, 0], c["rows"][1][:0]
    verify_decode(c, out, lse)
    # q_start outside the query rows, or falling: those sequences are skipped
    for starts in ([0, 1, 99], [0, 1, 0], [-1, 0, 2]):
        c = make_decode([100, 200], [1, 1], 16, False, tail=0)
        c["q_start"] = torch.tensor(starts, dtype=torch.int32).cuda()
        out, lse, status = run_decode(c)
        assert status == dsa.DSA_ERR_DEVICE_CHECK


@pytest.mark.gpu
def test_decode_offsets_beyond_32_bits(cuda_lib):
    """The sequence's pages lie at the end of a cache of more than 2^32 bytes and 2^31 elements."""
    pages = 60000
    c = make_decode([1000], [2], 16, False, tail=0)
    pool = torch.empty((pages, 64, 576), dtype=torch.bfloat16, device="cuda")
    own = c["pt"][0, :16].long()
    pool[pages - 1 - own] = c["pool"][own]
    c["pt"][0, :16] = (pages - 1 - own).int()
    c["pool"] = pool
    out, lse, status = run_decode(c)
    assert status == 0
    verify_decode(c, out, lse)


# ------------------------------------------------------------------------------------------
# expanded form
# ------------------------------------------------------------------------------------------

def make_prefill(new, keys, H, seed=0, stride=576, tail=2, grow=0.0, q_scale=1.0):
    """A packed batch; `tail` query rows, and NaN keys and values, behind the last sequence."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n_q, n_kv = sum(new), sum(keys)
    q = (torch.randn((n_q + tail, H, 192), generator=g, device="cuda") * q_scale).bfloat16()
    kv = torch.randn((n_kv + tail, H, 256), generator=g, device="cuda")
    if grow:
        kv[..., :128] += grow * torch.linspace(0, 1, n_kv + tail, device="cuda")[:, None, None] * \
            q[0, 0, :128].float().sign()
    kv = kv.bfloat16()
    wide = torch.randn((n_kv + tail, stride), generator=g, device="cuda").bfloat16()
    rope = wide[:, stride - 64:]
    kv[n_kv:] = math.nan
    rope[n_kv:] = math.nan
    cum = lambda x: torch.tensor([0] + list(torch.tensor(x).cumsum(0)), dtype=torch.int32).cuda()
    return {"q": q, "kv": kv, "rope": rope, "q_start": cum(new), "kv_start": cum(keys), "new": new, "keys": keys,
            "H": H, "tail": tail}


def run_prefill(c, **kw):
    n, H = c["q"].shape[:2]
    out = torch.full((n, H, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n, H), 6.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = {"softmax_scale": SCALE, "max_q_per_seq": max(1, max(c["new"])), **kw}
    dsa.mla_prefill(c["q"], c["kv"], c["rope"], c["q_start"], c["kv_start"], out=out, lse=lse, status=status, **kw)
    torch.cuda.synchronize()
    return out, lse, int(status)


def verify_prefill(c, out, lse):
    t = k = 0
    for n, L in zip(c["new"], c["keys"]):
        seen = torch.arange(L, device="cuda")[None] <= (L - n + torch.arange(n, device="cuda"))[:, None]
        for h in range(c["H"]):
            if n == 0:
                continue
            kv = c["kv"][k:k + L, h].double()
            keys = torch.cat([kv[:, :128], c["rope"][k:k + L].double()], 1)
            want = definition(c["q"][t:t + n, h].double(), keys, kv[:, 128:], seen, SCALE)
            check(out[t:t + n, h], lse[t:t + n, h], *want, 192, L)
        t, k = t + n, k + L
    assert torch.all(out[t:] == 5.0) and torch.all(lse[t:] == 6.0)


PREFILL = [
    (1, [1], [1]), (1, [1], [500]), (3, [128], [128]), (2, [129], [129]), (4, [127, 1, 0, 65], [127, 1, 0, 200]),
    (2, [300], [1000]), (16, [64, 17], [64, 129]), (1, [1000], [1000]), (5, [5, 3], [2, 0]),  # some see nothing
    (2, [257, 256, 255], [257, 512, 300]), (128, [33], [400]), (3, [700, 2, 0, 130], [700, 2, 44, 131]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("H,new,keys", PREFILL, ids=lambda v: str(v).replace(" ", "")[:28])
def test_prefill_matches_the_definition(cuda_lib, H, new, keys):
    c = make_prefill(new, keys, H, seed=H, stride=64 if H == 2 else 576)
    out, lse, status = run_prefill(c)
    assert status == 0
    verify_prefill(c, out, lse)
    again = run_prefill(c)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.gpu
@pytest.mark.parametrize("grow,q_scale", [(6.0, 1.0), (-6.0, 1.0), (0.0, 12.0), (0.0, 0.0)])
def test_prefill_moving_maximum(cuda_lib, grow, q_scale):
    c = make_prefill([400, 90], [1300, 90], 2, grow=grow, q_scale=q_scale)
    out, lse, status = run_prefill(c)
    assert status == 0
    verify_prefill(c, out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("where", ["key", "rope", "value"])
def test_prefill_hidden_keys_may_hold_anything(cuda_lib, bad, where):
    """Sequence 0's last token, and everything of sequence 2, is bad: the tokens that do not see
    it give what they give without it."""
    c = make_prefill([200, 70, 40], [200, 300, 40], 2)
    good = run_prefill(c)
    for rows in (slice(199, 200), slice(500, 540)):
        if where == "rope":
            c["rope"][rows] = bad
        else:
            cols = slice(0, 128) if where == "key" else slice(128, 256)
            c["kv"][rows, :, cols] = bad
    out, lse, status = run_prefill(c)
    assert status == 0
    ok = torch.ones(312, dtype=torch.bool, device="cuda")
    ok[199] = False
    ok[270:310] = False
    assert torch.equal(out[ok], good[0][ok]) and torch.equal(lse[ok], good[1][ok])


@pytest.mark.gpu
def test_prefill_reports_what_is_out_of_range(cuda_lib):
    for key, starts, fine in (("kv_start", [0, 300, 200], [0]), ("kv_start", [0, 300, 10 ** 6], [0]),
                              ("q_start", [0, 100, 50], [0]), ("q_start", [-3, 100, 150], [1])):
        c = make_prefill([100, 50], [300, 50], 2)
        c[key] = torch.tensor(starts, dtype=torch.int32).cuda()
        out, lse, status = run_prefill(c)
        assert status == dsa.DSA_ERR_DEVICE_CHECK
        rows = slice(0, 100) if fine == [0] else slice(100, 150)
        assert torch.isfinite(out[rows].float()).all() and not torch.any((out[rows] == 5.0).all(-1))
    # more tokens than the host's bound: reported, and computed all the same
    c = make_prefill([600, 50], [600, 50], 2)
    out, lse, status = run_prefill(c, max_q_per_seq=50)
    assert status == dsa.DSA_ERR_DEVICE_CHECK
    assert torch.all(lse[:50] != 6.0) and torch.all(lse[600:650] != 6.0)
    verify_prefill(c, out, lse)


@pytest.mark.gpu
def test_prefill_many_sequences(cuda_lib):
    """More sequences than a warp has lanes, empty ones among them, and tokens of no sequence."""
    g = torch.Generator().manual_seed(4)
    new = torch.randint(0, 300, (77,), generator=g).tolist()
    new[::5] = [0] * len(new[::5])
    keys = [n + k for n, k in zip(new, torch.randint(0, 200, (77,), generator=g).tolist())]
    c = make_prefill(new, keys, 2, seed=77)
    out, lse, status = run_prefill(c)
    assert status == 0
    verify_prefill(c, out, lse)
    # without the first three sequences: their tokens are no one's
    c["q_start"], c["kv_start"] = c["q_start"][3:].contiguous(), c["kv_start"][3:].contiguous()
    rest, lse2, status = run_prefill(c)
    n = sum(new[:3])
    assert status == 0 and torch.all(rest[:n] == 5.0) and torch.equal(rest[n:], out[n:]) and torch.equal(lse2[n:], lse[n:])


@pytest.mark.gpu
def test_prefill_without_any_key(cuda_lib):
    q = torch.randn((5, 3, 192), device="cuda").bfloat16()
    kv = torch.empty((0, 3, 256), dtype=torch.bfloat16, device="cuda")
    rope = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda")
    out, lse = dsa.mla_prefill(q, kv, rope, at, torch.zeros_like(at), softmax_scale=SCALE, max_q_per_seq=3)
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse))


@pytest.mark.gpu
def test_prefill_captures_and_replays_with_other_lengths(cuda_lib):
    c = make_prefill([300, 500, 40], [300, 700, 41], 20, tail=0)
    first = run_prefill(c)
    out, lse = torch.full_like(first[0], 5.0), torch.full_like(first[1], 6.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for _ in range(2):
            dsa.mla_prefill(c["q"], c["kv"], c["rope"], c["q_start"], c["kv_start"], softmax_scale=SCALE,
                            max_q_per_seq=840, out=out, lse=lse)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    # the ranges are read on the device
    c["new"], c["keys"] = [100, 640, 100], [150, 800, 91]
    for key, x in (("q_start", c["new"]), ("kv_start", c["keys"])):
        c[key].copy_(torch.tensor([0] + list(torch.tensor(x).cumsum(0)), dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    verify_prefill(c, out, lse)


@pytest.mark.gpu
def test_prefill_offsets_beyond_32_bits(cuda_lib):
    """Keys and values, and query rows, past 2^31 elements of their arrays."""
    H, n = 128, 70000
    kv = torch.zeros((n, H, 256), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((90000, H, 192), dtype=torch.bfloat16, device="cuda")
    c = make_prefill([30], [100], H, tail=0)
    kv[n - 100:], q[-30:] = c["kv"], c["q"]
    rope = torch.zeros((n, 64), dtype=torch.bfloat16, device="cuda")
    rope[n - 100:] = c["rope"]
    out = torch.empty((90000, H, 128), dtype=torch.bfloat16, device="cuda")
    starts = [torch.tensor(x, dtype=torch.int32).cuda() for x in ([90000 - 30, 90000], [n - 100, n])]
    out, lse = dsa.mla_prefill(q, kv, rope, *starts, softmax_scale=SCALE, max_q_per_seq=30, out=out)
    want = dsa.mla_prefill(c["q"], c["kv"], c["rope"], c["q_start"], c["kv_start"], softmax_scale=SCALE,
                           max_q_per_seq=30)
    assert torch.equal(out[-30:], want[0]) and torch.equal(lse[-30:], want[1])


# ------------------------------------------------------------------------------------------
# the operators together
# ------------------------------------------------------------------------------------------

@pytest.mark.gpu
def test_all_kernels_at_once_and_a_capture_that_allocates(cuda_lib):
    """Calls on four streams at the same time give what they give alone; a captured call that makes its
    own workspace and outputs, replayed between other work, too."""
    cases = [make_decode([5000, 64, 900], [1, 2, 1], 32, fp8, seed=3) for fp8 in (False, True)]
    fills = [make_prefill([300, 1, 700], [900, 1, 700], 6, seed=s) for s in (1, 2)]
    decode = lambda c: dsa.mla_decode(c["q"], c["pool"], c["pt"], c["seq_lens"], c["q_start"], softmax_scale=SCALE,
                                      max_q_per_seq=2)
    fill = lambda c: dsa.mla_prefill(c["q"], c["kv"], c["rope"], c["q_start"], c["kv_start"], softmax_scale=SCALE,
                                     max_q_per_seq=700)
    calls = [(decode, c, sum(c["new"])) for c in cases] + [(fill, c, sum(c["new"])) for c in fills]
    alone = [f(c) for f, c, _ in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = []
    for _ in range(6):
        for (f, c, n), s in zip(calls, streams):
            with torch.cuda.stream(s):
                got.append(f(c))
    torch.cuda.synchronize()
    for k, (out, lse) in enumerate(got):
        n = calls[k % 4][2]
        assert torch.equal(out[:n], alone[k % 4][0][:n]) and torch.equal(lse[:n], alone[k % 4][1][:n])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = [f(c) for f, c, _ in calls]
    for _ in range(2):
        for out, lse in kept:
            out.zero_()
            lse.zero_()
        graph.replay()
        got = [f(c) for f, c, _ in calls]
        torch.cuda.synchronize()
        for a, b, (_, _, n) in zip(kept, got, calls):
            assert torch.equal(a[0][:n], b[0][:n]) and torch.equal(a[1][:n], b[1][:n])


@pytest.mark.gpu
def test_cache_round_trip_absorbed_and_expanded_agree(cuda_lib):
    """A prompt's latent rows enter the FP8 cache; the rows that come back, expanded, give in
    mla_prefill what mla_decode gives on the cache with the up-projections absorbed; and with a top-K
    that covers the context, sparse attention over the same cache gives mla_decode's output."""
    H, lens, new = 128, [300, 190], [3, 190]
    g = torch.Generator(device="cuda").manual_seed(0)
    total = sum(lens)
    pt, pages = page_tables(lens, 0, torch.Generator().manual_seed(1))
    pt = torch.where(pt == 2 ** 30, 0, pt).cuda()
    pool = torch.zeros((pages, 64, 608), dtype=torch.uint8, device="cuda")
    seq = torch.repeat_interleave(torch.arange(2), torch.tensor(lens)).to(torch.int32).cuda()
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32).cuda()
    latent = torch.randn((total, 576), generator=g, device="cuda")
    dsa.cache_write_quant(pool, pt, seq, pos, latent)
    back = dsa.cache_read(pool, pt, seq, pos)
    w_uk = (torch.randn((H, 128, 512), generator=g, device="cuda") / 512 ** 0.5).bfloat16()
    w_uv = (torch.randn((H, 128, 512), generator=g, device="cuda") / 512 ** 0.5).bfloat16()
    q = torch.randn((sum(new), H, 192), generator=g, device="cuda").bfloat16()
    c = back[:, :512].double()
    kv = torch.cat([torch.einsum("nc,hdc->nhd", c, w_uk.double()), torch.einsum("nc,hdc->nhd", c, w_uv.double())], 2)
    cum = lambda x: torch.tensor([0] + list(torch.tensor(x).cumsum(0)), dtype=torch.int32).cuda()
    q_start, kv_start = cum(new), cum(lens)
    out_e, lse_e = dsa.mla_prefill(q, kv.bfloat16(), back[:, 512:], q_start, kv_start, softmax_scale=SCALE,
                                   max_q_per_seq=190)
    q_abs = torch.cat([torch.einsum("nhd,hdc->nhc", q[..., :128].double(), w_uk.double()), q[..., 128:].double()], 2)
    q_abs = q_abs.bfloat16()
    seq_lens = torch.tensor(lens, dtype=torch.int32).cuda()
    out_a, lse_a = dsa.mla_decode(q_abs, pool, pt, seq_lens, q_start, softmax_scale=SCALE, max_q_per_seq=190)
    # both forms round other intermediates (K, V and out; q and out) to bf16: 2^-8 of each, and a
    # logit's error of 2^-8 |q||k| scale on either side, at most exp of their sum
    out_l = torch.einsum("nhc,hdc->nhd", out_a.double(), w_uv.double())
    assert (lse_a - lse_e).abs().max() <= 2 * 2 ** -8 * float((q.float().norm(dim=-1).max() *
                                                               kv[..., :128].norm(dim=-1).max() * SCALE))
    num, den = (out_l - out_e.double()).norm(), out_l.norm()
    assert num <= 4 * 2 ** -8 * den
    # sparse attention with every visible position selected
    K = 300
    last = torch.cat([L - n + torch.arange(n) for n, L in zip(new, lens)]).cuda()
    idx = torch.arange(K, device="cuda")[None].expand(sum(new), K)
    idx = torch.where(idx <= last[:, None], idx, -1).to(torch.int32).contiguous()
    out_s, lse_s = dsa.sfa_prefill(q_abs, pool, pt, seq_lens, q_start, idx, softmax_scale=SCALE, max_seq_len=300,
                                   max_q_per_seq=190)
    # each kernel is within 3 2^-8 A of the exact output (see above); |out| / A is a few percent here
    A = back[:, :512].float().abs().mean()
    assert (out_s.float() - out_a.float()).abs().max() <= 6 * 2 ** -8 * 8 * A
    assert (lse_s - lse_a).abs().max() <= 1e-4


# ------------------------------------------------------------------------------------------
# refusals
# ------------------------------------------------------------------------------------------

def _decode_args(**over):
    a = dsa.MlaDecodeArgs()
    a.B, a.n_q, a.H, a.d_qk, a.d_v, a.page_size, a.max_pages, a.num_pages = 1, 2, 128, 576, 512, 64, 8, 8
    a.max_q_per_seq, a.softmax_scale, a.kv_dtype = 2, 0.07, dsa.DSA_BF16
    for n in ("q", "kv_pool", "page_table", "seq_lens", "q_start", "out", "workspace"):
        setattr(a, n, 4096)  # fake, aligned, never dereferenced on these error paths
    a.workspace_bytes = 1 << 40
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,code", [
    ({"B": 0}, dsa.DSA_ERR_INVALID_ARG), ({"n_q": -1}, dsa.DSA_ERR_INVALID_ARG), ({"H": 0}, dsa.DSA_ERR_INVALID_ARG),
    ({"max_q_per_seq": 0}, dsa.DSA_ERR_INVALID_ARG), ({"softmax_scale": 0.0}, dsa.DSA_ERR_INVALID_ARG),
    ({"softmax_scale": float("nan")}, dsa.DSA_ERR_INVALID_ARG), ({"softmax_scale": float("inf")}, dsa.DSA_ERR_INVALID_ARG),
    ({"softmax_scale": 3.0e38}, dsa.DSA_ERR_INVALID_ARG), ({"out": 4112}, dsa.DSA_ERR_INVALID_ARG),
    ({"H": 129}, dsa.DSA_ERR_UNSUPPORTED), ({"d_qk": 512}, dsa.DSA_ERR_UNSUPPORTED), ({"d_v": 576}, dsa.DSA_ERR_UNSUPPORTED),
    ({"page_size": 32}, dsa.DSA_ERR_UNSUPPORTED), ({"kv_dtype": dsa.DSA_MXFP8_E4M3}, dsa.DSA_ERR_UNSUPPORTED),
    ({"num_pages": 1 << 25}, dsa.DSA_ERR_UNSUPPORTED), ({"q_start": None}, dsa.DSA_ERR_INVALID_ARG),
    ({"out": 4104}, dsa.DSA_ERR_INVALID_ARG), ({"workspace": 4112}, dsa.DSA_ERR_INVALID_ARG),
])
def test_mla_decode_host_validation(over, code):
    lib = dsa.load()
    assert lib.dsa_mla_decode(ctypes.byref(_decode_args(**over)), None) == code, dsa.last_error()
    assert dsa.last_error()


def test_mla_decode_null_empty_and_workspace():
    lib = dsa.load()
    assert lib.dsa_mla_decode(None, None) == dsa.DSA_ERR_INVALID_ARG
    assert lib.dsa_mla_decode(ctypes.byref(_decode_args(n_q=0)), None) == dsa.DSA_OK
    assert lib.dsa_mla_decode_workspace_bytes(None) == 0
    need = lib.dsa_mla_decode_workspace_bytes(ctypes.byref(_decode_args()))
    assert need == dsa.mla_decode_workspace_bytes(2, 128, 2)
    if need:
        for over in ({"workspace_bytes": need - 1}, {"workspace": None}):
            assert lib.dsa_mla_decode(ctypes.byref(_decode_args(**over)), None) == dsa.DSA_ERR_INVALID_ARG


def _prefill_args(**over):
    a = dsa.MlaPrefillArgs()
    a.B, a.n_q, a.n_kv, a.H, a.d_nope, a.d_rope, a.d_v, a.max_q_per_seq = 1, 2, 4, 16, 128, 64, 128, 2
    a.softmax_scale, a.k_rope_stride = 0.07, 576
    for n in ("q", "kv", "k_rope", "q_start", "kv_start", "out"):
        setattr(a, n, 4096)
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,code", [
    ({"B": 0}, dsa.DSA_ERR_INVALID_ARG), ({"n_kv": -1}, dsa.DSA_ERR_INVALID_ARG), ({"H": 0}, dsa.DSA_ERR_INVALID_ARG),
    ({"max_q_per_seq": 0}, dsa.DSA_ERR_INVALID_ARG), ({"softmax_scale": -1.0}, dsa.DSA_ERR_INVALID_ARG),
    ({"d_nope": 64}, dsa.DSA_ERR_UNSUPPORTED), ({"d_rope": 32}, dsa.DSA_ERR_UNSUPPORTED), ({"d_v": 192}, dsa.DSA_ERR_UNSUPPORTED),
    ({"H": 1025}, dsa.DSA_ERR_UNSUPPORTED), ({"k_rope_stride": 32}, dsa.DSA_ERR_INVALID_ARG),
    ({"k_rope_stride": 68}, dsa.DSA_ERR_UNSUPPORTED), ({"kv": None}, dsa.DSA_ERR_INVALID_ARG), ({"k_rope": 4104}, dsa.DSA_ERR_INVALID_ARG),
])
def test_mla_prefill_host_validation(over, code):
    lib = dsa.load()
    assert lib.dsa_mla_prefill(ctypes.byref(_prefill_args(**over)), None) == code, dsa.last_error()
    assert dsa.last_error()
    assert lib.dsa_mla_prefill(None, None) == dsa.DSA_ERR_INVALID_ARG
    assert lib.dsa_mla_prefill(ctypes.byref(_prefill_args(n_q=0)), None) == dsa.DSA_OK


@pytest.mark.parametrize("over", [{"B": 1 << 28, "H": 1}, {"n_q": 0x7fffffff, "H": 512}, {"B": 1 << 21, "H": 1024}])
def test_mla_prefill_refuses_more_blocks_than_it_can_number(over):
    assert dsa.load().dsa_mla_prefill(ctypes.byref(_prefill_args(**over)), None) == dsa.DSA_ERR_UNSUPPORTED
    assert "2^31" in dsa.last_error()


def test_struct_layouts():
    assert ctypes.sizeof(dsa.MlaDecodeArgs) == 11 * 4 + 4 + 9 * 8 + 8
    assert ctypes.sizeof(dsa.MlaPrefillArgs) == 9 * 4 + 4 + 8 + 8 * 8


def test_bindings_refuse_a_stream_of_another_device():
    class Stream:
        cuda_stream, device = 0, torch.device("cuda", 1)

    with pytest.raises(ValueError, match="stream"):
        dsa._empty(Stream(), (1,), torch.uint8, torch.device("cuda", 0))
    with pytest.raises(ValueError, match="stream"):
        dsa._launch_stream(Stream(), torch.device("cuda", 0))


def test_bindings_refuse_what_does_not_fit():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    good = dict(q=bf(2, 16, 576), kv_pool=bf(2, 64, 576), page_table=i32(1, 2), seq_lens=i32(1), q_start=i32(2))
    for bad in (dict(q=bf(2, 16, 512)), dict(q=good["q"].float()), dict(kv_pool=good["kv_pool"].half()),
                dict(kv_pool=bf(2, 64, 608)), dict(page_table=i32(2, 2)), dict(seq_lens=i32(1).long()),
                dict(q_start=i32(3)), dict(out=bf(2, 16, 576)), dict(lse=bf(2, 16)), dict()):  # last: CPU tensors
        with pytest.raises(ValueError):
            dsa.mla_decode(**{**good, **bad}, softmax_scale=1.0)
    good = dict(q=bf(2, 16, 192), kv=bf(4, 16, 256), k_rope=bf(4, 64), q_start=i32(2), kv_start=i32(2))
    for bad in (dict(q=bf(2, 16, 128)), dict(kv=bf(4, 8, 256)), dict(k_rope=bf(64, 4).T), dict(k_rope=bf(1, 64).expand(4, 64)),
                dict(kv_start=i32(3)), dict(q_start=i32(2).long()), dict(out=bf(2, 16, 192)), dict()):
        with pytest.raises(ValueError):
            dsa.mla_prefill(**{**good, **bad}, softmax_scale=1.0)
