"""Workloads of the latent-cache operators: writing a quantised cache, reading it back, and dense
latent attention over it in the absorbed and in the expanded form.

``run`` computes a case with elementary torch operations where ``own`` is false and with this
package's operators where it is true; ``exact`` gives the same outputs in 64 bits.
"""
import math
import random

import torch

own = False

PAGE = 64
D_LATENT, D_ROPE = 512, 64
D_ROW = D_LATENT + D_ROPE
KV8_ROW = 608                    # 576 e4m3 codes, 5 fp32 tile scales, 12 unused bytes
D_HEAD = 128                     # expanded keys (without rope) and values
SCALE = (D_HEAD + D_ROPE) ** -0.5
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step of 32 sequences: their new latent rows enter the FP8 cache
        {"name": "write_latent_step", "op": "write", "format": "latent", "rows": 32, "dim": D_ROW, "type": "bf16"},
        # the latent rows of a 64k-token prompt, as an fp32 projection leaves them
        {"name": "write_latent_64k", "op": "write", "format": "latent", "rows": 65536, "dim": D_ROW, "type": "fp32"},
        # the index keys of a prompt of odd length into the MXFP8 key cache
        {"name": "write_keys_mx", "op": "write", "format": "mx", "rows": 35003, "dim": 128, "type": "bf16"},
        # the index keys of many prompts into the per-row FP8 key cache
        {"name": "write_keys_fp8", "op": "write", "format": "fp8", "rows": 262144, "dim": 128, "type": "fp16"},
        # a short shared prefix comes back from the FP8 latent cache
        {"name": "read_latent_short", "op": "read", "format": "latent", "rows": 100, "dim": D_ROW, "type": "bf16"},
        # the 60k-token prefix of a prefill chunk comes back for the expanded form
        {"name": "read_latent_60k", "op": "read", "format": "latent", "rows": 61440, "dim": D_ROW, "type": "bf16"},
        # one token of one 4k-token sequence, 16 heads (a tensor-parallel share): latency
        {"name": "decode_4k", "op": "decode", "heads": 16, "lens": "4096", "new": "1", "cache": "bf16"},
        # the decode batch of the benchmark, dense: 32 sequences of 32k tokens
        {"name": "decode_32k", "op": "decode", "heads": 128, "lens": "32768x32", "new": "1x32", "cache": "bf16"},
        # verified and draft token of ragged sequences over the FP8 cache
        {"name": "decode_ragged_fp8", "op": "decode", "heads": 64, "new": "2x16", "cache": "fp8",
         "lens": "1024 1777 2500 3333 4999 6001 8192 10007 14001 20011 29000 40009 57001 80021 111111 131072"},
        # a few tokens appended to short cached contexts
        {"name": "prefill_short", "op": "prefill", "heads": 16, "new": "1 65 17", "prefix": "500 0 129"},
        # ragged prompts from their first token
        {"name": "prefill_ragged", "op": "prefill", "heads": 16, "new": "777 2049 128 4000 1 3001 513 1500", "prefix": "0x8"},
        # a prefill chunk behind a cached prefix of the same length, all heads
        {"name": "prefill_chunk", "op": "prefill", "heads": 128, "new": "4096", "prefix": "4096"},
    ]


def _counts(text):
    """The whole numbers of a text: "5 7x2" is [5, 7, 7]."""
    parts = [(w + "x1").split("x")[:2] for w in text.split()]
    return [int(n) for n, times in parts for _ in range(int(times))]


def _text(counts):
    return " ".join(str(n) for n in counts)


def _log(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["write", "read", "decode", "prefill"])
    if op in ("write", "read"):
        form = rng.choice(["latent", "latent", "fp8", "mx"])
        dim = D_ROW if form == "latent" else rng.choice([64, 128])
        return {"op": op, "format": form, "rows": _log(rng, 1, 65536 if form == "latent" else 262144),
                "dim": dim, "type": rng.choice(["bf16", "fp16", "fp32"])}
    if op == "decode":
        heads = rng.choice([1, 5, 16, 24, 32, 64, 96, 128])
        b = _log(rng, 1, 32)
        lens = [_log(rng, 1, 32768 if b > 16 else 131072) for _ in range(b)]
        return {"op": op, "heads": heads, "lens": _text(lens), "cache": rng.choice(["bf16", "fp8"]),
                "new": _text(min(n, rng.randint(1, 4)) for n in lens)}
    heads = rng.choice([1, 3, 8, 16, 32, 128])
    b = rng.randint(1, 4)
    most = 4096 // b if heads == 128 else 4096
    return {"op": op, "heads": heads, "new": _text(_log(rng, 1, most) for _ in range(b)),
            "prefix": _text(rng.choice([0, _log(rng, 1, most)]) for _ in range(b))}


def work(case):
    op = case["op"]
    if op in ("write", "read"):
        n, d = case["rows"], case["dim"]
        cached = d + {"latent": 20, "fp8": 4, "mx": d // 32}[case["format"]]
        return {"bytes": n * (d * (4 if case["type"] == "fp32" else 2) + cached + 8), "flops": n * d * 2}
    h, new = case["heads"], _counts(case["new"])
    tokens = sum(new)
    if op == "decode":
        lens = _counts(case["lens"])
        seen = sum(n * (L - n) + n * (n + 1) // 2 for L, n in zip(lens, new))
        row = 2 * D_ROW if case["cache"] == "bf16" else D_ROW + 20
        return {"bytes": sum(lens) * row + tokens * h * (2 * D_ROW + 2 * D_LATENT + 4),
                "flops": 2 * seen * h * (D_ROW + D_LATENT)}
    prefix = _counts(case["prefix"])
    keys = tokens + sum(prefix)
    seen = sum(n * p + n * (n + 1) // 2 for n, p in zip(new, prefix))
    return {"bytes": 2 * (tokens * h * (D_HEAD + D_ROPE) + keys * (h * 2 * D_HEAD + D_ROPE) + tokens * h * D_HEAD)
            + 4 * tokens * h, "flops": 2 * seen * h * (2 * D_HEAD + D_ROPE)}


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------

def _starts(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device=DEV)


def _activations(n, dim, g):
    """Rows as a projection leaves them: normal values, channels of different sizes, and rows of
    different sizes."""
    x = torch.randn((n, dim), generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn((1, dim), generator=g, device=DEV))
    return x.mul_(torch.exp(0.3 * torch.randn((n, 1), generator=g, device=DEV)))


def _pages(lens, g):
    """A page table whose pages lie in random order, and the number of pages."""
    counts = [max(1, -(-n // PAGE)) for n in lens]
    order = torch.randperm(sum(counts), generator=g, device=DEV).to(torch.int32)
    table = torch.zeros((len(lens), max(counts)), dtype=torch.int32, device=DEV)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    return table, at


def _tokens(lens):
    """(sequence, position) of every position of every sequence."""
    n = torch.tensor(lens, device=DEV)
    seq = torch.repeat_interleave(torch.arange(len(lens), device=DEV), n)
    pos = torch.arange(int(n.sum()), device=DEV) - torch.repeat_interleave(n.cumsum(0) - n, n)
    return seq.to(torch.int32), pos.to(torch.int32)


def _codes(shape, g):
    """e4m3 codes as a quantiser leaves them: no NaN, most of them of middling size."""
    return (32 * torch.randn(shape, generator=g, device=DEV)).clamp_(-448, 448).to(torch.float8_e4m3fn)


def _scales(shape, g):
    return torch.exp(0.3 * torch.randn(shape, generator=g, device=DEV)) / 32


def _latent_pool(pages, g):
    pool = torch.zeros((pages, PAGE, KV8_ROW), dtype=torch.uint8, device=DEV)
    pool[..., :D_ROW] = _codes((pages, PAGE, D_ROW), g).view(torch.uint8)
    pool[..., D_ROW:D_ROW + 20] = _scales((pages, PAGE, 5), g).view(torch.uint8)
    return pool


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    st = {"case": case}
    if op in ("write", "read"):
        n = case["rows"]
        # rows of up to 8 sequences, in order, as a batch of chunks has them
        b = min(8, n)
        lens = [n // b + (i < n % b) for i in range(b)]
        st["page_table"], pages = _pages(lens, g)
        st["seq"], st["pos"] = _tokens(lens)
        form, dim = case["format"], case["dim"]
        if form == "latent":
            st["pool"] = _latent_pool(pages, g)
        else:
            st["pool"] = _codes((pages, PAGE, dim), g)
            if form == "fp8":
                st["scale_pool"] = _scales((pages, PAGE), g)
            else:
                st["sf_pool"] = torch.randint(118, 126, (pages, PAGE, dim // 32), generator=g,
                                              device=DEV).to(torch.uint8)
        if op == "write":
            st["rows"] = _activations(n, dim, g).to(TYPES[case["type"]])
        return st
    h = case["heads"]
    st["new"] = _counts(case["new"])
    st["q_start"] = _starts(st["new"])
    st["most"] = max(st["new"])
    tokens = sum(st["new"])
    if op == "decode":
        st["lens"] = _counts(case["lens"])
        st["page_table"], pages = _pages(st["lens"], g)
        if case["cache"] == "fp8":
            st["pool"] = _latent_pool(pages, g)
        else:
            st["pool"] = torch.randn((pages, PAGE, D_ROW), generator=g, device=DEV, dtype=torch.bfloat16)
        st["seq_lens"] = torch.tensor(st["lens"], dtype=torch.int32, device=DEV)
        st["q"] = torch.randn((tokens, h, D_ROW), generator=g, device=DEV, dtype=torch.bfloat16)
        return st
    lens = [n + p for n, p in zip(st["new"], _counts(case["prefix"]))]
    st["lens"] = lens
    st["kv_start"] = _starts(lens)
    # the latent rows (their last columns are the shared rope key), and the up-projection's output
    st["latent"] = torch.randn((sum(lens), D_ROW), generator=g, device=DEV, dtype=torch.bfloat16)
    st["kv"] = torch.randn((sum(lens), h, 2 * D_HEAD), generator=g, device=DEV, dtype=torch.bfloat16)
    st["q"] = 1.5 * torch.randn((tokens, h, D_HEAD + D_ROPE), generator=g, device=DEV, dtype=torch.bfloat16)
    return st


# ------------------------------------------------------------------------------------------
# the operators in their plain form
# ------------------------------------------------------------------------------------------

def _slots(st):
    pos = st["pos"].long()
    return st["page_table"][st["seq"].long(), pos // PAGE].long() * PAGE + pos % PAGE


def _pow2(e):
    """2^e in 64 bits, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3(y):
    """The e4m3 value nearest to y (64 bits; ties to the even code, saturated)."""
    _, e = torch.frexp(y)
    step = _pow2((e - 1).clamp(min=-6) - 3)
    return ((y / step).round() * step).clamp(-448, 448)


def _quantise(x, group):
    """fp32 rows [n, d] -> e4m3 codes [n, d] and one fp32 scale per group."""
    n, d = x.shape
    x = torch.nn.functional.pad(x, (0, -d % group)).view(n, -1, group)
    amax = x.abs().amax(-1, keepdim=True)
    scale = torch.where(amax > 0, (amax / torch.full_like(amax, 448)).clamp(min=2.0 ** -126), 1.0)
    # 64 bits: a quotient next to the border between two codes
    codes = _e4m3(x.double() / scale.double()).to(torch.float8_e4m3fn)
    return codes.view(n, -1)[:, :d], scale.squeeze(-1)


def _quantise_mx(x):
    n, d = x.shape
    x = x.view(n, -1, 32)
    amax = x.abs().amax(-1, keepdim=True)
    _, e = torch.frexp(amax)
    e = torch.where(amax > 0, e - 9, 0).clamp(-127, 127)
    codes = _e4m3(x.double() * _pow2(-e)).to(torch.float8_e4m3fn)
    return codes.view(n, d), (e.squeeze(-1) + 127).to(torch.uint8)


def _latent_values(rows):
    """FP8 latent rows [n, 608] -> fp32 products of codes and tile scales [n, 576]."""
    codes = rows[:, :D_ROW].view(torch.float8_e4m3fn).float()
    scale = rows[:, D_ROW:D_ROW + 20].contiguous().view(torch.float32)
    return codes * scale.repeat_interleave(128, 1)[:, :D_ROW]


def _plain_write(st):
    case, at = st["case"], _slots(st)
    x = st["rows"].float()
    if case["format"] == "mx":
        codes, sf = _quantise_mx(x)
        st["sf_pool"].view(-1, sf.shape[1])[at] = sf
        st["pool"].view(torch.uint8).view(-1, case["dim"])[at] = codes.view(torch.uint8)
    elif case["format"] == "fp8":
        codes, scale = _quantise(x, case["dim"])
        st["scale_pool"].view(-1)[at] = scale[:, 0]
        st["pool"].view(torch.uint8).view(-1, case["dim"])[at] = codes.contiguous().view(torch.uint8)
    else:
        codes, scale = _quantise(x, 128)
        rows = torch.cat([codes.view(torch.uint8), scale.view(torch.uint8),
                          torch.zeros((x.shape[0], 12), dtype=torch.uint8, device=DEV)], 1)
        st["pool"].view(-1, KV8_ROW)[at] = rows


def _plain_read(st):
    case, at = st["case"], _slots(st)
    if case["format"] == "latent":
        y = _latent_values(st["pool"].view(-1, KV8_ROW)[at])
    else:
        c = st["pool"].view(torch.uint8).view(-1, case["dim"])[at].view(torch.float8_e4m3fn).float()
        if case["format"] == "fp8":
            y = c * st["scale_pool"].view(-1)[at][:, None]
        else:
            e = st["sf_pool"].view(-1, case["dim"] // 32)[at].int() - 127
            y = (c * _pow2(e).repeat_interleave(32, 1)).float()
    return y.to(TYPES[case["type"]])


def _softmax(z, hidden):
    """Softmax weights over the last dimension, and the log of their sum."""
    z = z.masked_fill(hidden, -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - m)
    s = p.sum(-1, keepdim=True)
    return p / s, (m + torch.log(s)).squeeze(-1)


def _hidden(n, length):
    """Which positions of a sequence its last n tokens do not see."""
    return torch.arange(length, device=DEV) > torch.arange(length - n, length, device=DEV)[:, None]


def _plain_decode(st):
    case = st["case"]

    def sequence(b, q, length):
        rows = st["pool"][st["page_table"][b, :max(1, -(-length // PAGE))].long()]
        rows = rows.view(-1, rows.shape[-1])[:length]
        # an element of an FP8 row stands for its product rounded to bf16
        kv = rows.float() if case["cache"] == "bf16" else _latent_values(rows).bfloat16().float()
        n, h, _ = q.shape
        z = (q.float().view(n * h, -1) @ kv.T).view(n, h, -1) * SCALE
        p, lse = _softmax(z, _hidden(n, length)[:, None])
        return (p.view(n * h, -1) @ kv[:, :D_LATENT]).view(n, h, -1).bfloat16(), lse

    # sequences of different lengths share no dimension to batch over
    parts = [sequence(b, q, st["lens"][b]) for b, q in enumerate(st["q"].split(st["new"]))]
    return torch.cat([o for o, _ in parts]), torch.cat([s for _, s in parts])


def _plain_prefill(st):
    new, lens = st["new"], st["lens"]

    def sequence(q, kv, rope):
        q, kv, rope = (t.float() for t in (q.transpose(0, 1), kv.transpose(0, 1), rope))
        z = q[..., :D_HEAD] @ kv[..., :D_HEAD].transpose(1, 2) + q[..., D_HEAD:] @ rope.T
        p, lse = _softmax(z * SCALE, _hidden(q.shape[1], kv.shape[1]))
        return (p @ kv[..., D_HEAD:]).transpose(0, 1).bfloat16(), lse.T

    parts = [sequence(*x) for x in zip(st["q"].split(new), st["kv"].split(lens),
                                       st["latent"][:, D_LATENT:].split(lens))]
    return torch.cat([o for o, _ in parts]), torch.cat([s for _, s in parts])


def _caches(st):
    """The written cache: codes and scales."""
    if st["case"]["format"] == "latent":
        return [st["pool"][..., :D_ROW].view(torch.float8_e4m3fn),
                st["pool"][..., D_ROW:D_ROW + 20].view(torch.float32)]
    return [st["pool"], st["scale_pool"] if "scale_pool" in st else st["sf_pool"]]


def run(state):
    op = state["case"]["op"]
    if own:
        return _call(state, op)
    if op == "write":
        _plain_write(state)
        return _caches(state)
    if op == "read":
        return [_plain_read(state)]
    return list(_plain_decode(state) if op == "decode" else _plain_prefill(state))


def _call(st, op):
    import dsa_sparse_attention_li_gb300 as dsa
    if op in ("write", "read"):
        kw = {k: st[k] for k in ("scale_pool", "sf_pool") if k in st}
        if op == "write":
            dsa.cache_write_quant(st["pool"], st["page_table"], st["seq"], st["pos"], st["rows"], **kw)
            return _caches(st)
        return [dsa.cache_read(st["pool"], st["page_table"], st["seq"], st["pos"],
                               dtype=TYPES[st["case"]["type"]], **kw)]
    if op == "decode":
        return list(dsa.mla_decode(st["q"], st["pool"], st["page_table"], st["seq_lens"], st["q_start"],
                                   softmax_scale=SCALE, max_q_per_seq=st["most"]))
    return list(dsa.mla_prefill(st["q"], st["kv"], st["latent"][:, D_LATENT:], st["q_start"], st["kv_start"],
                                softmax_scale=SCALE, max_q_per_seq=st["most"]))


# ------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------

_E4M3 = None


def _nearest_code(y):
    """Value of the e4m3 code nearest to each y, by a search among all of them; a tie goes to the
    even code."""
    global _E4M3
    if _E4M3 is None:
        _E4M3 = torch.arange(127, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).double()
    a = y.abs().clamp(max=448.0)
    up = torch.searchsorted(_E4M3, a.contiguous()).clamp(1, 126)
    lo, hi = _E4M3[up - 1], _E4M3[up]
    middle = (lo + hi) / 2
    take = (a > middle) | ((a == middle) & (up % 2 == 0))
    return torch.where(take, hi, lo) * torch.where(y < 0, -1.0, 1.0)


def _exact_write(st):
    case, at = st["case"], _slots(st)
    d = case["dim"]
    x = st["rows"].double()
    codes, scales = (t.double() if t.is_floating_point() else t.clone() for t in _caches(st))
    flat = codes.view(-1, d)
    per_row = scales.view(flat.shape[0], -1)
    width = {"latent": 128, "fp8": d, "mx": 32}[case["format"]]
    for i, c in enumerate(range(0, d, width)):
        part = x[:, c:c + width]
        top = part.abs().amax(1)
        if case["format"] == "mx":
            powers = torch.tensor([2.0 ** (i - 119) for i in range(255)], dtype=torch.float64, device=DEV)
            byte = (torch.searchsorted(powers, top, right=True) - 1).clamp(0, 254)
            byte = torch.where(top > 0, byte, 127)
            stored, scale = byte.to(torch.uint8), powers[byte] * 2.0 ** -8
        else:
            stored = torch.where(top > 0, (top / 448).clamp(min=2.0 ** -126), 1.0)
            scale = stored.float().double()       # the scale is kept in 32 bits
        flat[at, c:c + width] = _nearest_code(part / scale[:, None])
        per_row[at, i] = stored
    return [codes, scales]


def _exact_rows(codes, scales, width):
    y = codes.view(torch.float8_e4m3fn).double()
    for i, c in enumerate(range(0, y.shape[1], width)):
        y[:, c:c + width] *= scales[:, i:i + 1]
    return y


def _exact_read(st):
    case, at = st["case"], _slots(st)
    if case["format"] == "latent":
        rows = st["pool"].view(-1, KV8_ROW)[at]
        return _exact_rows(rows[:, :D_ROW], rows[:, D_ROW:D_ROW + 20].contiguous().view(torch.float32).double(), 128)
    codes = st["pool"].view(torch.uint8).view(-1, case["dim"])[at]
    if case["format"] == "fp8":
        return _exact_rows(codes, st["scale_pool"].view(-1, 1)[at].double(), case["dim"])
    return _exact_rows(codes, torch.exp2(st["sf_pool"].view(-1, case["dim"] // 32)[at].double() - 127), 32)


def _exact_attention(q, k, v, first):
    """One head's rows q over keys k and values v; row i sees the keys before first + i."""
    z = SCALE * (q @ k.T)
    seen = torch.arange(k.shape[0], device=DEV)[None] < (first + torch.arange(q.shape[0], device=DEV))[:, None]
    lse = torch.logsumexp(torch.where(seen, z, -math.inf), 1)
    return torch.where(seen, torch.exp(z - lse[:, None]), 0.0) @ v, lse


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "write":
        return _exact_write(st)
    if case["op"] == "read":
        return [_exact_read(st)]
    tokens, h = st["q"].shape[:2]
    width = D_LATENT if case["op"] == "decode" else D_HEAD
    out = torch.empty((tokens, h, width), dtype=torch.float64, device=DEV)
    lse = torch.empty((tokens, h), dtype=torch.float64, device=DEV)
    t0 = k0 = 0
    for b, n in enumerate(st["new"]):
        if case["op"] == "decode":
            length = st["lens"][b]
            pages = st["page_table"][b, :max(1, -(-length // PAGE))].long()
            rows = st["pool"][pages].flatten(0, 1)[:length]
            if case["cache"] == "bf16":
                kv = rows.double()
            else:
                scales = rows[:, D_ROW:D_ROW + 20].contiguous().view(torch.float32).double()
                kv = _exact_rows(rows[:, :D_ROW], scales, 128).float().bfloat16().double()
            for i in range(n):
                o, s = _exact_attention(st["q"][t0 + i].double(), kv[:length - n + i + 1],
                                        kv[:length - n + i + 1, :D_LATENT], length + 1)
                out[t0 + i], lse[t0 + i] = o, s
        else:
            length = st["lens"][b]
            rope = st["latent"][k0:k0 + length, D_LATENT:].double()
            for j in range(h):
                kv = st["kv"][k0:k0 + length, j].double()
                o, s = _exact_attention(st["q"][t0:t0 + n, j].double(), torch.cat([kv[:, :D_HEAD], rope], 1),
                                        kv[:, D_HEAD:], length - n + 1)
                out[t0:t0 + n, j], lse[t0:t0 + n, j] = o, s
            k0 += length
        t0 += n
    return [out, lse]


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(i)) for i in range(6)]:
        print(c.get("name", "drawn"), c["op"], work(c))
