"""Workloads of the operators between the residual stream and the attention, in 8 bits: the
root-mean-square norm with the residual's addition, the quantisation of rows without a norm, and the
matrix product of e4m3 operands with a scale for each block of 128.

``run`` computes a case with elementary torch operations where ``own`` is false and with this
package's operators where it is true; ``exact`` gives the same outputs in 64 bits.
"""
import math
import random

import torch

own = False

BLOCK = 128                       # columns of a scale; a weight's scale covers 128 rows of them too
D_MODEL = 7168                    # hidden state
D_Q = 1536                        # query latent
D_ROW, D_LATENT = 576, 512        # cache row, and its part that the up-projection takes
KV8_ROW = 608                     # FP8 cache row: 576 e4m3 codes, 5 fp32 scales, 12 unused bytes
EPS = 1e-6
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step of 32 sequences: the residual stream before the attention; the indexer
        # takes the normed rows in 16 bits too
        {"name": "norm_step", "op": "norm", "rows": 32, "dim": D_MODEL, "type": "bf16", "residual": True, "y": True},
        # the same for the tokens of several prompts
        {"name": "norm_prompts", "op": "norm", "rows": 16384, "dim": D_MODEL, "type": "bf16", "residual": True,
         "y": False},
        # the query latents of ragged prompts, as an fp32 projection leaves them
        {"name": "norm_query_latent", "op": "norm", "rows": 11969, "dim": D_Q, "type": "fp32", "residual": False,
         "y": True},
        # a decode step's attention output (128 heads of 128) before the output projection
        {"name": "quant_step", "op": "quant", "rows": 32, "dim": 128 * 128, "type": "bf16"},
        # the same of a prefill chunk of odd length
        {"name": "quant_chunk", "op": "quant", "rows": 4095, "dim": 128 * 128, "type": "bf16"},
        # one token's query latent and cache row, projected in one product
        {"name": "down_token", "op": "matmul", "m": 1, "n": D_Q + D_ROW, "k": D_MODEL, "type": "bf16", "a": "rows"},
        # a decode step's output projection
        {"name": "out_step", "op": "matmul", "m": 32, "n": D_MODEL, "k": 128 * 128, "type": "bf16", "a": "rows"},
        # two tokens of each of 100 sequences: the indexer's queries (64 heads of 128)
        {"name": "index_q_pairs", "op": "matmul", "m": 200, "n": 64 * 128, "k": D_Q, "type": "fp16", "a": "rows"},
        # ragged prompts: the queries of 128 heads (192 columns each) from the query latents
        {"name": "up_q_ragged", "op": "matmul", "m": 777, "n": 128 * 192, "k": D_Q, "type": "bf16", "a": "rows"},
        # a prompt's cache rows in 32 bits, which the quantised write takes
        {"name": "down_rows", "op": "matmul", "m": 16384, "n": D_ROW, "k": D_MODEL, "type": "fp32", "a": "rows"},
        # keys and values of 128 heads from the rows of an FP8 latent cache, as they lie there
        {"name": "up_kv_cache", "op": "matmul", "m": 8192, "n": 128 * 256, "k": D_LATENT, "type": "bf16", "a": "cache"},
        # a prefill chunk's output projection
        {"name": "out_chunk", "op": "matmul", "m": 4096, "n": D_MODEL, "k": 128 * 128, "type": "bf16", "a": "rows"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["norm", "quant", "matmul", "matmul"])
    kind = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op != "matmul":
        dim = 8 * _log(rng, 8, (D_MODEL if op == "norm" else 128 * 128) // 8)
        most = (16384 * D_MODEL if op == "norm" else 4095 * 128 * 128) // (2 if kind == "fp32" else 1)
        case = {"op": op, "rows": _log(rng, 1, min(65536, most // dim)), "dim": dim, "type": kind}
        if op == "norm":
            case.update(residual=rng.random() < 0.6, y=rng.random() < 0.4)
        return case
    if rng.random() < 0.2:
        return {"op": op, "m": _log(rng, 64, 8192), "n": 256 * rng.choice([1, 8, 16, 64, 128]), "k": D_LATENT,
                "type": rng.choice(["bf16", "fp16"]), "a": "cache"}
    k = 16 * _log(rng, 4, 128 * 128 // 16)
    n = _log(rng, 64, 24576)
    m = _log(rng, 1, max(1, min(16384, 4096 * D_MODEL * 128 * 128 // (n * k), (1 << 28) // n)))
    return {"op": op, "m": m, "n": n, "k": k, "type": kind, "a": "rows"}


def work(case):
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        blocks = -(-k // BLOCK)
        return {"bytes": (m + n) * k + 4 * blocks * (m + -(-n // BLOCK)) + m * n * BYTES[case["type"]],
                "flops": 2 * m * n * k}
    n, d, size = case["rows"], case["dim"], BYTES[case["type"]]
    moved = size                                       # the rows
    if case["op"] == "norm":
        moved += 2 * size * case["residual"] + size * case["y"]
    return {"bytes": n * (d * (moved + 1) + 4 * -(-d // BLOCK)) + (size * d if case["op"] == "norm" else 0),
            "flops": n * d * (6 if case["op"] == "norm" else 3)}


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------

def _activations(n, dim, g):
    """Rows as they stand in a network: normal values, channels of different sizes, and rows of
    different sizes."""
    x = torch.randn((n, dim), generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn((1, dim), generator=g, device=DEV))
    return x.mul_(torch.exp(0.3 * torch.randn((n, 1), generator=g, device=DEV)))


def _codes(n, dim, g):
    """e4m3 codes as a quantiser leaves them: no NaN, most of them of middling size."""
    out = torch.empty((n, dim), dtype=torch.float8_e4m3fn, device=DEV)
    for at in range(0, n, 4096):
        part = torch.randn((min(4096, n - at), dim), generator=g, device=DEV)
        out[at:at + 4096] = part.mul_(110).clamp_(-448, 448).to(torch.float8_e4m3fn)
    return out


def _scales(rows, blocks, size, g):
    return size / 110 * torch.exp(0.3 * torch.randn((rows, blocks), generator=g, device=DEV))


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    st = {"case": case}
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        blocks = -(-k // BLOCK)
        if case["a"] == "cache":
            # the cache's pages of 64 rows: the product takes the first 512 columns of each row
            pool = torch.zeros((-(-m // 64), 64, KV8_ROW), dtype=torch.uint8, device=DEV)
            rows = pool.view(-1, KV8_ROW)
            rows[:, :D_ROW] = _codes(rows.shape[0], D_ROW, g).view(torch.uint8)
            rows[:, D_ROW:D_ROW + 20] = _scales(rows.shape[0], 5, 1.0, g).view(torch.uint8)
            st["pool"] = pool
        else:
            st["a"], st["a_scale"] = _codes(m, k, g), _scales(m, blocks, 1.0, g)
        st["b"] = _codes(n, k, g)
        st["b_scale"] = _scales(-(-n // BLOCK), blocks, k ** -0.5, g)
        return st
    n, d, kind = case["rows"], case["dim"], TYPES[case["type"]]
    st["x"] = _activations(n, d, g).to(kind)
    if case["op"] == "norm":
        st["weight"] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(kind)
        if case["residual"]:
            st["residual"] = (4 * _activations(n, d, g)).to(kind)
    return st


def _left(st):
    """The product's left operand, and its scales."""
    if "pool" not in st:
        return st["a"], st["a_scale"]
    m = st["case"]["m"]
    codes = st["pool"].view(torch.float8_e4m3fn).view(-1, KV8_ROW)[:m, :D_LATENT]
    scales = st["pool"].view(torch.float32).view(-1, KV8_ROW // 4)[:m, D_ROW // 4:D_ROW // 4 + D_LATENT // BLOCK]
    return codes, scales


# ------------------------------------------------------------------------------------------
# the operators in their plain form
# ------------------------------------------------------------------------------------------

def _e4m3(y):
    """The e4m3 value nearest to y (64 bits; ties to the even code, saturated)."""
    _, e = torch.frexp(y)
    step = torch.exp2(((e - 1).clamp(min=-6) - 3).double())
    return ((y / step).round() * step).clamp(-448, 448)


def _quantise(v):
    """fp32 rows [n, d] -> e4m3 codes [n, d] and one fp32 scale per group of 128 columns."""
    n, d = v.shape
    v = torch.nn.functional.pad(v, (0, -d % BLOCK)).view(n, -1, BLOCK)
    amax = v.abs().amax(-1, keepdim=True)
    scale = torch.where(amax > 0, (amax / torch.full_like(amax, 448)).clamp(min=2.0 ** -126), 1.0)
    # 64 bits: a quotient next to the border between two codes
    codes = _e4m3(v.double() / scale.double()).to(torch.float8_e4m3fn)
    return codes.view(n, -1)[:, :d].contiguous(), scale.squeeze(-1)


def _plain_norm(st):
    x, kind = st["x"], st["x"].dtype
    out = []
    if "residual" in st:
        x = (x.float() + st["residual"].float()).to(kind)
        out.append(x)
    h = x.float()
    v = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * st["weight"].float()
    if st["case"]["y"]:
        out.append(v.to(kind))
    return list(_quantise(v)) + out


def _plain_matmul(st):
    a, a_scale = _left(st)
    n, k = st["b"].shape
    x = a.float() * a_scale.repeat_interleave(BLOCK, 1)[:, :k]
    w = st["b"].float() * st["b_scale"].repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]
    return [(x @ w.T).to(TYPES[st["case"]["type"]])]


def run(state):
    op = state["case"]["op"]
    if own:
        return _call(state, op)
    if op == "norm":
        return _plain_norm(state)
    if op == "quant":
        return list(_quantise(state["x"].float()))
    return _plain_matmul(state)


def _call(st, op):
    import dsa_sparse_attention_li_gb300 as dsa
    if op == "quant":
        return list(dsa.quant_rows(st["x"]))
    if op == "matmul":
        a, a_scale = _left(st)
        return [dsa.matmul_fp8(a, a_scale, st["b"], st["b_scale"], dtype=TYPES[st["case"]["type"]])]
    y = [torch.empty_like(st["x"])] if st["case"]["y"] else []
    out = dsa.rms_norm_quant(st["x"], st["weight"], residual=st.get("residual"), eps=EPS, y=y[0] if y else None)
    return list(out) + y                     # codes, scales, and with a residual the sum


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
    return torch.where((a > middle) | ((a == middle) & (up % 2 == 0)), hi, lo) * torch.where(y < 0, -1.0, 1.0)


def _exact_rows(v):
    """Codes and scales of rows in 64 bits; a scale is kept in 32."""
    codes, scales = [], []
    for c in range(0, v.shape[1], BLOCK):
        part = v[:, c:c + BLOCK]
        top = part.abs().amax(1, keepdim=True)
        s = torch.where(top > 0, (top / 448).clamp(min=2.0 ** -126), 1.0)
        scales.append(s)
        codes.append(_nearest_code(part / s.float().double()))
    return [torch.cat(codes, 1), torch.cat(scales, 1)]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quant":
        return _exact_rows(st["x"].double())
    if case["op"] == "norm":
        h, more = st["x"].double(), []
        if case["residual"]:
            h = (h + st["residual"].double())
            more.append(h)
            h = h.to(st["x"].dtype).double()      # the norm is of the sum as it is kept
        v = h / torch.sqrt((h * h).sum(1, keepdim=True) / case["dim"] + EPS) * st["weight"].double()
        return _exact_rows(v) + more + ([v] if case["y"] else [])
    a, a_scale = _left(st)
    m, n, k = case["m"], case["n"], case["k"]
    out = torch.zeros((m, n), dtype=torch.float64, device=DEV)
    for i, c in enumerate(range(0, k, BLOCK)):
        w = st["b"][:, c:c + BLOCK].double() * st["b_scale"][:, i].double().repeat_interleave(BLOCK)[:n, None]
        out.addmm_(a[:, c:c + BLOCK].double() * a_scale[:, i:i + 1].double(), w.T)
    return [out]


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(i)) for i in range(6)]:
        print(c.get("name", "drawn"), c["op"], work(c))
