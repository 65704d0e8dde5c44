"""Dense latent attention at the borders of what it may read and of what a token sees: page tables that end
inside a tile, sequences whose bounds are out of order, values that are not finite, and whether every tile
of a long context counts once.  (tests/test_mla.py holds the definition and its tolerances.)
"""
import math

import pytest
import torch

import dsa_sparse_attention_li_gb300 as dsa
from test_mla import (SCALE, check, definition, make_decode, make_prefill, run_decode, run_prefill,
                      verify_decode, verify_prefill)


@pytest.mark.parametrize("owned", [False, True], ids=["padding", "token"])
@pytest.mark.parametrize("length", [129, 150, 192])
def test_a_query_row_looks_up_only_pages_of_its_sequence(owned, length):
    """A tile is two pages.  Three pages of a sequence end inside its second tile, and the page table may end
    there: the number behind it (a guard of either kind) must not count for any row.  On the host, with the
    kernel's own rule; a row that belongs to no token counts as seeing 2^31 - 1 positions."""
    f = dsa.load_testhooks().dsa_test_mla_visible_columns
    got = []
    for guard in (0, -1, 10 ** 6):
        table = torch.tensor([0, 10 ** 6, 1, guard], dtype=torch.int32)
        seen = length if owned else 2 ** 31 - 1
        got.append([f(owned, seen, pos0, 1, table.data_ptr(), 2) for pos0 in (0, 64, 128, 192)])
    assert got[0] == got[1] == got[2]
    assert got[0] == ([64, 0, length - 128, length - 192] if owned else [64] * 4)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("bad", [0, 1, 2])
def test_decode_page_that_does_not_exist_in_a_table_that_ends_inside_a_tile(cuda_lib, fp8, bad):
    """The last sequence has three pages and the table no room for more; one of them does not exist."""
    c = make_decode([100, 170], [1, 1], 16, fp8, extra=1, tail=0)
    assert c["pt"].shape[1] == 4
    guarded = torch.full((7,), 10 ** 6, dtype=torch.int32, device="cuda")
    table = guarded[:6].view(2, 3)
    table.copy_(c["pt"][:, :3])
    table[1, bad] = (-1, 10 ** 6, 2 ** 31 - 1)[bad]
    c["pt"] = table
    out, lse, status = run_decode(c)
    assert status == dsa.DSA_ERR_DEVICE_CHECK
    keep = torch.ones(170, dtype=torch.bool)
    keep[64 * bad:64 * bad + 64] = False
    c["rows"][1] = c["rows"][1][keep.cuda()]
    c["lens"][1] = int(keep.sum())
    verify_decode(c, out, lse)


# ------------------------------------------------------------------------------------------
# infinities among what a token sees
# ------------------------------------------------------------------------------------------

def put_inf(c, b, j, col, fp8):
    """Column `col` of cache row j of sequence b becomes -inf, in the cache and in the reference's rows."""
    row = c["pool"][int(c["pt"][b, j // 64]), j % 64]
    if fp8:   # the only code of its 128 columns that is not zero, times a scale that overflows
        tile = slice(col // 128 * 128, min(576, col // 128 * 128 + 128))
        row[tile] = 0
        row[col] = 0xFE   # -448
        row[576 + col // 128 * 4:580 + col // 128 * 4] = torch.tensor([3.0e38], device="cuda").view(torch.uint8)
        c["rows"][b][j, tile] = 0
    else:
        row[col] = -math.inf
    c["rows"][b][j, col] = -math.inf


def ieee(q, k, v):
    """Attention of every row of q [n, d] over all of k [L, d], v [L, dv], in 64 bits as the formula stands: a
    weight of 0 times an infinite value is NaN, and so is the difference of two infinities."""
    z = (q @ k.T) * SCALE
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    s = e.sum(1, keepdim=True)
    mag = (q.abs() @ k.abs().nan_to_num(0, 0, 0).T * SCALE).amax(1)
    return (e / s) @ v, (m + torch.log(s))[:, 0], torch.nan_to_num(e / s) @ v.abs().nan_to_num(0, 0, 0), mag


def check_seen(got, lse, want, want_lse, A, mag, n_products, length):
    """Where the definition gives NaN, so does the kernel; what it gives else is right, unless the row holds a
    NaN or an infinity, which may make all of it NaN."""
    odd = ~torch.isfinite(want).all(1)
    assert torch.isnan(got[~torch.isfinite(want)]).all()
    check(got[~odd], lse[~odd], want[~odd], want_lse[~odd], A[~odd], mag[~odd], n_products, length)
    tol = A * (3 * 2.0 ** -8 + 2 * n_products * 2.0 ** -24 * mag + 2.0 ** -21 + length * 2.0 ** -24)[:, None] + 1e-30
    fine = torch.isfinite(want) & ~torch.isnan(got)
    assert torch.all((got.double() - want).abs()[fine] <= tol[fine])


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("col", [7, 300, 520], ids=["value0", "value1", "rope"])
@pytest.mark.parametrize("j", [100, 400, 450, 497])
def test_decode_infinity_that_a_token_sees(cuda_lib, fp8, col, j):
    """Row j holds -inf: a score of -inf for the even heads, of +inf for the odd ones.  j lies in a tile that
    all tokens see to its end (100), or in the last one, seen by all (400, 450) or by the last three
    tokens only: what a token gets does not depend on that."""
    c = make_decode([500], [4], 16, fp8)
    c["q"][..., col] = torch.tensor([1.0, -1.0], device="cuda").repeat(8)
    clean = run_decode(c)
    put_inf(c, 0, j, col, fp8)
    out, lse, status = run_decode(c)
    assert status == 0
    for t in range(4):
        seen = 497 + t
        if j >= seen:
            assert torch.equal(out[t], clean[0][t]) and torch.equal(lse[t], clean[1][t])
            continue
        kv = c["rows"][0][:seen]
        want = ieee(c["q"][t].double(), kv, kv[:, :512])
        assert torch.isnan(want[0][1::2]).all()
        assert torch.isnan(want[0][::2]).any(1).all() == (col < 512)
        check_seen(out[t], lse[t], *want, 576, seen)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_decode_scores_that_are_all_minus_infinity(cuda_lib, fp8):
    """A token that sees positions but no finite score has no softmax: NaN, and not the zeros of a token
    that sees nothing.  Positions that score -inf beside others have a weight of 0."""
    lens, new = [1, 70, 9000, 3, 4000, 9000], [1, 2, 1, 5, 1, 1]
    c = make_decode(lens, new, 16, fp8, tail=0)
    c["q"][..., 520] = 1.0
    for b, part in ((0, (0, 1)), (1, (0, 70)), (2, (0, 9000)), (3, (0, 3)), (4, (0, 2500)), (5, (4444, 9000))):
        c["rows"][b][part[0]:part[1], 512:] = 0     # as put_inf, for many rows at once
        c["rows"][b][part[0]:part[1], 520] = -math.inf
        j = torch.arange(*part, device="cuda")
        pool, at = c["pool"].view(-1, c["pool"].shape[-1]), c["pt"][b].long()[j // 64] * 64 + j % 64
        if fp8:
            row = pool[at]
            row[:, 512:576] = 0
            row[:, 520] = 0xFE
            row[:, 592:596] = torch.tensor([3.0e38], device="cuda").view(torch.uint8)
            pool[at] = row
        else:
            pool[at, 512:] = 0
            pool[at, 520] = -math.inf
    out, lse, status = run_decode(c)
    assert status == 0
    for t in (0, 1, 2, 3, 6, 7, 8):
        assert torch.isnan(out[t]).all() and torch.isnan(lse[t]).all(), t
    assert torch.all(out[4:6] == 0) and torch.isneginf(lse[4:6]).all()
    for t, b, part in ((9, 4, slice(2500, 4000)), (10, 5, slice(0, 4444))):
        kv = c["rows"][b][part]
        want = definition(c["q"][t].double(), kv, kv[:, :512], torch.ones((16, len(kv)), dtype=torch.bool, device="cuda"),
                          SCALE)
        check(out[t], lse[t], *want, 576, lens[b])
    # none of whose pages exist: nothing is seen, whatever the scores
    c["pt"][2], c["pt"][0] = -1, 2 ** 30
    out, lse, status = run_decode(c)
    assert status == dsa.DSA_ERR_DEVICE_CHECK
    for t in (0, 3):
        assert torch.all(out[t] == 0) and torch.isneginf(lse[t]).all()
    # some of them do, with scores of -inf only
    c["pt"][2, 3] = c["pt"][5, 100]
    out, lse, status = run_decode(c)
    assert torch.isnan(out[3]).all() and torch.isnan(lse[3]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_decode_scores_beyond_fp32_give_nan(cuda_lib, fp8):
    """Logits of 1e39 and more are infinite in fp32: the output says so."""
    out, lse, status = run_decode(make_decode([5000, 90], [1, 2], 16, fp8, tail=0), softmax_scale=1.9e38)
    assert status == 0
    assert torch.isnan(out).all() and torch.isnan(lse).all()


@pytest.mark.gpu
def test_prefill_scores_beyond_fp32_give_nan(cuda_lib):
    out, lse, status = run_prefill(make_prefill([130], [400], 2, tail=0), softmax_scale=1.9e38)
    assert status == 0
    assert torch.isnan(out).all() and torch.isnan(lse).all()


@pytest.mark.gpu
def test_prefill_scores_that_are_all_minus_infinity(cuda_lib):
    """As for decode: sequence 1 has no finite score, 2 has some, two tokens of 3 see nothing and the others
    no finite score."""
    new, keys = [40, 300, 200, 5], [40, 400, 200, 3]
    c = make_prefill(new, keys, 3, tail=0)
    c["q"][..., 130] = 1.0
    for rows in (slice(40, 440), slice(440, 500), slice(640, 643)):
        c["rope"][rows, 2] = -math.inf
    out, lse, status = run_prefill(c)
    assert status == 0
    nan = torch.cat([torch.arange(40, 340), torch.arange(340, 400), torch.arange(542, 545)]).cuda()
    assert torch.isnan(out[nan]).all() and torch.isnan(lse[nan]).all()
    assert torch.all(out[540:542] == 0) and torch.isneginf(lse[540:542]).all()
    ok = torch.cat([torch.arange(0, 40), torch.arange(400, 540)]).cuda()
    assert torch.isfinite(out[ok].float()).all() and torch.isfinite(lse[ok]).all()
    for h in range(3):
        kv, rope = c["kv"][500:640, h].double(), c["rope"][500:640].double()
        seen = torch.arange(140, device="cuda")[None] <= torch.arange(140, device="cuda")[:, None]
        want = definition(c["q"][400:540, h].double(), torch.cat([kv[:, :128], rope], 1), kv[:, 128:], seen, SCALE)
        check(out[400:540, h], lse[400:540, h], *want, 192, 200)


# ------------------------------------------------------------------------------------------
# bounds out of order
# ------------------------------------------------------------------------------------------

def starts(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check_prefill_rows(c, out, lse, t, n, k, L):
    """Tokens t .. t + n - 1 as the last ones of the keys k .. k + L - 1."""
    seen = torch.arange(L, device="cuda")[None] <= (L - n + torch.arange(n, device="cuda"))[:, None]
    for h in range(c["H"]):
        kv = c["kv"][k:k + L, h].double()
        keys = torch.cat([kv[:, :128], c["rope"][k:k + L].double()], 1)
        want = definition(c["q"][t:t + n, h].double(), keys, kv[:, 128:], seen, SCALE)
        check(out[t:t + n, h], lse[t:t + n, h], *want, 192, L)


@pytest.mark.gpu
@pytest.mark.parametrize("more", [0, 40], ids=["few", "many"])
def test_prefill_falling_q_start(cuda_lib, more):
    """A token belongs to the first sequence that claims it; sequences that fall, and those that start
    before another's end, are skipped, and the others are whole.  `more` empty sequences in front take
    the batch beyond the lanes of a warp."""
    c = make_prefill([1000, 600], [1000, 600], 2)

    def run(q_start, kv_start, owned):
        c["q_start"], c["kv_start"] = (starts(*x[:1] * more, *x) for x in (q_start, kv_start))
        out, lse, status = run_prefill(c, max_q_per_seq=1600)
        assert status == dsa.DSA_ERR_DEVICE_CHECK
        free = torch.ones(1602, dtype=torch.bool, device="cuda")
        for t, n, k, L in owned:
            check_prefill_rows(c, out, lse, t, n, k, L)
            free[t:t + n] = False
        assert torch.all(out[free] == 5.0) and torch.all(lse[free] == 6.0)

    run([0, 1000, 0, 1000], [0, 1000, 1000, 1600], [(0, 1000, 0, 1000)])
    run([0, 1000, 0, 1000, 0, 1000, 0, 1000], [0, 1000, 1000, 1000, 1000, 1000, 1000, 1000], [(0, 1000, 0, 1000)])
    run([0, 300, 200, 1600], [0, 300, 300, 1600], [(0, 300, 0, 300)])
    run([0, 300, 250, 300, 900], [0, 300, 300, 300, 900], [(0, 300, 0, 300), (300, 600, 300, 600)])
    run([500, 0, 1000], [0, 0, 1000], [(0, 1000, 0, 1000)])
    run([0, 300, 10 ** 6, 300, 900], [0, 300, 300, 300, 900], [(0, 300, 0, 300), (300, 600, 300, 600)])
    run([-7, 300, 900], [0, 300, 900], [(300, 600, 300, 600)])
    run([0, 1000, 1600], [0, 1000, 900], [(0, 1000, 0, 1000)])


@pytest.mark.gpu
def test_prefill_falling_q_start_in_front_of_many_sequences(cuda_lib):
    """An error in the first 32 sequences is remembered in the following ones."""
    new = [40] * 100
    c = make_prefill(new, new, 1)
    q_start = [40 * i for i in range(101)]
    q_start[5] = 3900      # sequence 4 claims 160 .. 3899, sequence 5 falls, the ones up to 3899 come too late
    c["q_start"] = starts(*q_start)
    out, lse, status = run_prefill(c, max_q_per_seq=4000)
    assert status == dsa.DSA_ERR_DEVICE_CHECK
    for b in (0, 3, 98, 99):
        check_prefill_rows(c, out, lse, 40 * b, 40, 40 * b, 40)
    # of sequence 4's 3,740 tokens the last 40 see its 40 keys, the others nothing
    assert torch.all(out[160:3860] == 0) and torch.isneginf(lse[160:3860]).all()
    check_prefill_rows(c, out, lse, 3860, 40, 160, 40)
    assert torch.all(out[3900:3920] == 5.0) and torch.all(lse[3900:3920] == 6.0)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("q_start,owned", [([0, 1, 99], 0), ([0, 1, 0], 0), ([-1, 1, 2], 1), ([5, 1, 2], 1)])
def test_decode_skips_a_sequence_whose_q_start_is_out_of_order(cuda_lib, fp8, q_start, owned):
    """Its rows stay as they were, and the other sequence is whole."""
    c = make_decode([100, 1200], [1, 1], 16, fp8, tail=0)
    c["q_start"] = starts(*q_start)
    out, lse, status = run_decode(c)
    assert status == dsa.DSA_ERR_DEVICE_CHECK
    assert torch.all(out[1 - owned] == 5.0) and torch.all(lse[1 - owned] == 6.0)
    kv = c["rows"][owned]
    want = definition(c["q"][owned].double(), kv, kv[:, :512],
                      torch.ones((16, len(kv)), dtype=torch.bool, device="cuda"), SCALE)
    check(out[owned], lse[owned], *want, 576, len(kv))


@pytest.mark.gpu
@pytest.mark.parametrize("page", [4, 5, 30], ids=["first", "second", "last"])
def test_decode_fp8_page_that_does_not_exist(cuda_lib, page):
    """The first or the second page of a tile, or the last page of the sequence: page 0, which stands in for it,
    belongs to the other sequence and must not count."""
    c = make_decode([1980, 640], [1, 2], 16, True, tail=0)
    assert int((c["pt"][1, :10] == 0).sum()) + int((c["pt"][0, :31] == 0).sum()) <= 1
    c["pt"][0, page] = -3
    out, lse, status = run_decode(c)
    assert status == dsa.DSA_ERR_DEVICE_CHECK
    keep = torch.ones(1980, dtype=torch.bool, device="cuda")
    keep[64 * page:64 * page + 64] = False
    c["rows"][0] = c["rows"][0][keep]
    c["lens"][0] = int(keep.sum())
    verify_decode(c, out, lse)


@pytest.mark.gpu
def test_decode_fp8_length_beyond_the_page_table_and_below_zero(cuda_lib):
    c = make_decode([448, 200], [1, 1], 16, True, extra=0, tail=0)
    c["seq_lens"][0] = 10 ** 6
    c["seq_lens"][1] = -5
    out, lse, status = run_decode(c)
    assert status == dsa.DSA_ERR_DEVICE_CHECK
    c["lens"], c["rows"][1] = [448, 0], c["rows"][1][:0]
    verify_decode(c, out, lse)


@pytest.mark.gpu
def test_decode_fp8_offsets_beyond_32_bits(cuda_lib):
    """The sequence's pages lie at the end of a cache of 4.7 GB."""
    pages = 120001
    c = make_decode([1000], [2], 16, True, tail=0)
    pool = torch.full((pages, 64, 608), 0x7F, dtype=torch.uint8, device="cuda")
    own = c["pt"][0, :16].long()
    pool[pages - 1 - own] = c["pool"][own]
    c["pt"][0, :16] = (pages - 1 - own).int()
    c["pool"] = pool
    out, lse, status = run_decode(c)
    assert status == 0
    verify_decode(c, out, lse)


# ------------------------------------------------------------------------------------------
# every tile counts once
# ------------------------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("H,lens,new", [(1, [60001], [3]), (24, [65536, 20011, 777], [4, 1, 2]),
                                        (128, [40000, 129, 30000], [1, 1, 1])], ids=str)
def test_decode_weight_of_every_tile(cuda_lib, fp8, H, lens, new):
    """Value column c is 1 in tile c of 128 positions and 0 elsewhere, so that an output element is the weight
    of one tile: nothing cancels in it, and a tile lost or counted twice is an error of all of it.  The
    scores are the rope columns'."""
    c = make_decode(lens, new, H, fp8)
    c["q"][..., :512] = 0
    pool = c["pool"].view(-1, c["pool"].shape[-1])
    for b, L in enumerate(lens):
        j = torch.arange(L, device="cuda")
        at = c["pt"][b].long()[j // 64] * 64 + j % 64
        one = torch.zeros((L, 512), device="cuda")
        one[j, j // 128] = 1.0
        c["rows"][b][:, :512] = one.double()
        if fp8:
            pool[at, :512] = one.to(torch.float8_e4m3fn).view(torch.uint8)
            row = pool[at]
            row[:, 576:592] = torch.ones((L, 4), device="cuda").view(torch.uint8)
            pool[at] = row
        else:
            pool[at, :512] = one.bfloat16()
    out, lse, status = run_decode(c)
    assert status == 0
    verify_decode(c, out, lse)


@pytest.mark.gpu
def test_prefill_weight_of_every_tile(cuda_lib):
    """The same in the expanded form: 128 tiles of 128 keys, and a prompt of its own."""
    new, keys = [300, 700], [16384, 700]
    c = make_prefill(new, keys, 2)
    tile = torch.cat([torch.arange(n, device="cuda") // 128 for n in keys])
    c["kv"][:sum(keys), :, 128:] = torch.nn.functional.one_hot(tile, 128)[:, None].bfloat16()
    out, lse, status = run_prefill(c)
    assert status == 0
    verify_prefill(c, out, lse)


@pytest.mark.gpu
def test_prefill_value_that_is_nan_reaches_the_tokens_that_see_it(cuda_lib):
    """A few NaN values per head, in tiles that all tokens of a block see and in those that only some do, with
    several items a CTA, so that the marks of one tile follow on another's: NaN in that column for every
    token that sees it, and every other token as without it."""
    new, keys = [500, 130, 300], [500, 400, 300]
    c = make_prefill(new, keys, 128)
    good = run_prefill(c)
    g = torch.Generator().manual_seed(6)
    t = k = 0
    nan = torch.zeros((932, 128, 128), dtype=torch.bool)
    hit = torch.zeros((932, 128), dtype=torch.bool)
    for n, L in zip(new, keys):
        for h in range(128):
            for _ in range(h % 4):    # every fourth head has none
                j, col = int(torch.randint(L, (1,), generator=g)), int(torch.randint(128, (1,), generator=g))
                c["kv"][k + j, h, 128 + col] = math.nan
                first = t + max(0, j - (L - n))    # the first token that sees key j
                nan[first:t + n, h, col] = True
                hit[first:t + n, h] = True
        t, k = t + n, k + L
    out, lse, status = run_prefill(c)
    assert status == 0
    out, lse = out.cpu(), lse.cpu()
    assert torch.isnan(out[nan]).all()
    assert torch.equal(out[~hit], good[0].cpu()[~hit]) and torch.equal(lse[~hit], good[1].cpu()[~hit])


# ------------------------------------------------------------------------------------------
# waits that run out
# ------------------------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("new,keys,H", [([700, 300], [900, 300], 4), ([900], [900], 4), ([300, 20], [3000, 20], 128),
                                        ([257, 129, 2], [257, 400, 90], 128)], ids=str)
def test_prefill_waits_that_run_out_at_any_moment(cuda_lib, monkeypatch, new, keys, H):
    """The first CTA's products never start, so that all its other waits give up, each at its own moment: the
    loads with part of the ring on its way, the edge tiles' warps ahead of them.  Each launch ends and reports
    it, whatever the order, and the next call is right."""
    c = make_prefill(new, keys, H)
    hooks = dsa.load_testhooks()
    with monkeypatch.context() as m:
        m.setattr(dsa, "_lib", hooks)
        for _ in range(12):
            hooks.dsa_test_inject_stall(4)
            try:
                assert run_prefill(c)[2] == dsa.DSA_ERR_TIMEOUT
            finally:
                hooks.dsa_test_inject_stall(0)
        out, lse, status = run_prefill(c)
    assert status == 0
    verify_prefill(c, out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("what,case", [
    (5, ([9000, 700], [1, 2], 64)), (5, ([100], [1], 16)), (6, ([9000, 700], [1, 2], 64)), (6, ([100], [1], 16)),
    (7, ([700, 300], [900, 300], 128)), (8, ([700, 300], [900, 300], 128)), (8, ([100], [100], 4)),
    (9, ([700, 300], [900, 300], 128))], ids=str)
def test_a_load_that_never_comes(cuda_lib, monkeypatch, what, case):
    """The first CTA leaves a load out: keys, values (of a tile that all tokens see to its end, and of an edge
    tile) or queries.  Whoever waits for its bytes gives up, nothing is loaded into what still waits for
    them, and the launch ends with the error; the next call is right."""
    c, run, verify = ((make_decode(*case, False), run_decode, verify_decode) if what < 7 else
                      (make_prefill(*case), run_prefill, verify_prefill))
    hooks = dsa.load_testhooks()
    with monkeypatch.context() as m:
        m.setattr(dsa, "_lib", hooks)
        for _ in range(3):
            hooks.dsa_test_inject_stall(what)
            try:
                assert run(c)[2] == dsa.DSA_ERR_TIMEOUT
            finally:
                hooks.dsa_test_inject_stall(0)
            out, lse, status = run(c)
            assert status == 0
            verify(c, out, lse)


# ------------------------------------------------------------------------------------------
# the host's bound of the tokens
# ------------------------------------------------------------------------------------------

@pytest.mark.gpu
def test_the_bound_of_the_tokens_is_asked_for(cuda_lib):
    """It cannot come from q_start: on the device that would be a synchronisation, on the host the kernels
    could not read it."""
    c, f = make_decode([100], [1], 16, False), make_prefill([5], [9], 2)
    for at in ("cuda", "cpu"):
        for op, kw in ((dsa.mla_decode, dict(q=c["q"], kv_pool=c["pool"], page_table=c["pt"], seq_lens=c["seq_lens"],
                                             q_start=c["q_start"].to(at))),
                       (dsa.mla_prefill, dict(q=f["q"], kv=f["kv"], k_rope=f["rope"], q_start=f["q_start"].to(at),
                                              kv_start=f["kv_start"]))):
            with pytest.raises(ValueError, match="max_q_per_seq" if at == "cuda" else "q_start is on cpu"):
                op(**kw, softmax_scale=SCALE)
