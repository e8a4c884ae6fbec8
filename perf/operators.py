"""What is measured of the 8-bit floating point linear layer and of the token read-out.

Five operators: the activation quantizer with a scale for each 128 values of a row, the weight quantizer with a scale for
each 128 x 128 tile, SwiGLU with the same row quantizer behind it, the matrix product on those codes and scales, and the
log probabilities of given tokens with the entropy and the top alternatives.

``run`` computes them in plain torch operations, or through this package's own calls where ``own`` is true.  Codes are
returned as float8_e4m3fn tensors, that is as the values they stand for.
"""
import math

import torch

own = False

BLOCK = 128
FP8_MAX = 448.0
FP8 = torch.float8_e4m3fn
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
LARGEST_FLOPS = 2 * 8192 * 5120 * 5120   # of a product
LARGEST_VALUES = 17408 * 5120            # of a quantizer's input
LARGEST_LOGITS = 2048 * 100003


def listed():
    return [
        # one token's attention output projection while decoding: latency
        {"name": "gemm_decode_1", "op": "gemm", "m": 1, "n": 5120, "k": 5120, "out": "bf16"},
        # an odd number of running requests, each one token, through a 4B-class MLP up-projection
        {"name": "gemm_decode_33", "op": "gemm", "m": 33, "n": 9728, "k": 2560, "out": "bf16"},
        # a short prompt, down-projection: few output tiles, long sums, K not a whole number of blocks
        {"name": "gemm_prompt_500", "op": "gemm", "m": 500, "n": 2560, "k": 9680, "out": "bf16"},
        # a prefill chunk through a 27B-class MLP up-projection
        {"name": "gemm_prefill_2048", "op": "gemm", "m": 2048, "n": 17408, "k": 5120, "out": "bf16"},
        # a full prefill batch, square projection, fp32 out for a residual kept in fp32
        {"name": "gemm_prefill_8192", "op": "gemm", "m": 8192, "n": 5120, "k": 5120, "out": "f32"},
        # the activations of one decoding step of 16 requests: latency
        {"name": "quant_rows_16", "op": "quant", "m": 16, "k": 5120, "in": "f32"},
        # the activations of a full prefill batch
        {"name": "quant_rows_8192", "op": "quant", "m": 8192, "k": 5120, "in": "bf16"},
        # a weight matrix brought to 8 bits at load time, rows not a whole number of tiles
        {"name": "quant_tiles_17400", "op": "tiles", "m": 17400, "k": 5120, "in": "bf16"},
        # between the two products of an MLP, one decoding step of 4 requests
        {"name": "swiglu_4", "op": "swiglu", "m": 4, "k": 9728, "in": "bf16"},
        # the same for a prefill chunk, the intermediate width not a whole number of blocks
        {"name": "swiglu_2048", "op": "swiglu", "m": 2048, "k": 17360, "in": "bf16"},
        # one question's answer read off a vocabulary of 128 Ki: latency
        {"name": "logprobs_1", "op": "logprobs", "m": 1, "v": 131072, "in": "f32", "t": 4, "top": 20, "keep": 1.0},
        # a scored prompt, every position's next token, rows of an odd vocabulary, some of it masked
        {"name": "logprobs_2048", "op": "logprobs", "m": 2048, "v": 100003, "in": "bf16", "t": 1, "top": 8, "keep": 0.9},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "gemm", "quant", "tiles", "swiglu", "logprobs", "logprobs"])
    kind = rng.choice(["f32", "f16", "bf16"])
    if op == "gemm":
        n, k = _log(rng, 16, 17408), 16 * _log(rng, 4, 1088)
        m = min(_log(rng, 1, 8192), max(1, LARGEST_FLOPS // (2 * n * k)))
        return {"op": op, "m": m, "n": n, "k": k, "out": kind}
    if op == "logprobs":
        v = _log(rng, 1000, 200000)
        m = min(_log(rng, 1, 2048), LARGEST_LOGITS // v)
        return {"op": op, "m": m, "v": v, "in": kind, "t": rng.choice([1, 2, 5, 8]), "top": rng.randrange(0, 21),
                "keep": rng.choice([1.0, 1.0, 0.9, 0.02])}
    k = 16 * _log(rng, 4, 1088)
    m = min(_log(rng, 1, 17408 if op == "tiles" else 8192), LARGEST_VALUES // k)
    return {"op": op, "m": m, "k": k, "in": kind}


# ------------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _activations(g, m, k):
    """N(0, 1) with one column in a hundred twenty times larger, as the projections' inputs have it."""
    x = torch.randn((m, k), generator=g, device="cuda")
    loud = torch.rand((k,), generator=g, device="cuda") < 0.01
    return x * torch.where(loud, 20.0, 1.0)


def _to_blocks(x):
    """The blocks of 128 columns, zeros behind the last one: [rows, KB, 128]."""
    rows, k = x.shape
    return torch.nn.functional.pad(x, (0, -k % BLOCK)).view(rows, -1, BLOCK)


def _to_tiles(x):
    """The 128 x 128 tiles, zeros behind the last rows and columns: [NB, 128, KB, 128]."""
    rows, k = x.shape
    x = torch.nn.functional.pad(x, (0, -k % BLOCK, 0, -rows % BLOCK))
    return x.view(x.shape[0] // BLOCK, BLOCK, x.shape[1] // BLOCK, BLOCK)


def _codes(values, scale):
    """values / scale to the nearest e4m3 value, 0 where the scale is 0."""
    ratio = torch.where(scale > 0, values / scale, 0.0).clamp(-FP8_MAX, FP8_MAX)
    return ratio.to(FP8)


def _quantize_rows(x):
    blocks = _to_blocks(x.float())
    scale = blocks.abs().amax(2) / FP8_MAX
    q = _codes(blocks, scale[:, :, None]).view(x.shape[0], -1)
    return q[:, :x.shape[1]].contiguous(), scale.t().contiguous()


def _quantize_tiles(x):
    tiles = _to_tiles(x.float())
    scale = tiles.abs().amax((1, 3)) / FP8_MAX
    q = _codes(tiles, scale[:, None, :, None]).view(tiles.shape[0] * BLOCK, -1)
    return q[:x.shape[0], :x.shape[1]].contiguous(), scale


def prepare(case, seed):
    g = _generator(seed)
    op, m = case["op"], case["m"]
    state = {"case": case}
    if op == "gemm":
        n, k = case["n"], case["k"]
        state["q"], state["s_a"] = _quantize_rows(_activations(g, m, k))
        state["w"], state["s_w"] = _quantize_tiles(torch.randn((n, k), generator=g, device="cuda") * 0.02)
    elif op == "quant":
        state["x"] = _activations(g, m, case["k"]).to(TYPES[case["in"]])
    elif op == "tiles":
        state["x"] = (torch.randn((m, case["k"]), generator=g, device="cuda") * 0.02).to(TYPES[case["in"]])
    elif op == "swiglu":
        # gate and up side by side, as one product with both weights leaves them
        state["gu"] = (2 * torch.randn((m, 2 * case["k"]), generator=g, device="cuda")).to(TYPES[case["in"]])
    else:
        v = case["v"]
        z = 3 * torch.randn((m, v), generator=g, device="cuda")
        if case["keep"] < 1:
            # tokens that a grammar forbids; one row in eight has none left
            z = torch.where(torch.rand((m, v), generator=g, device="cuda") < case["keep"], z, -math.inf)
            z[7::8] = -math.inf
        state["z"] = z.to(TYPES[case["in"]])
        state["tokens"] = torch.randint(0, v, (m, case["t"]), generator=g, device="cuda")
    return state


# -------------------------------------------------------------- the operators

def _plain_gemm(s, out):
    a = _to_blocks(s["q"].float()) * s["s_a"].t()[:, :, None]
    w = _to_tiles(s["w"].float()) * s["s_w"][:, None, :, None]
    a = a.view(a.shape[0], -1)
    w = w.view(w.shape[0] * BLOCK, -1)[:s["w"].shape[0]]
    return (a @ w.t()).to(out)


def _plain_swiglu(gu):
    gate, up = gu.float().chunk(2, dim=1)
    return _quantize_rows(gate / (1 + torch.exp(-gate)) * up)


def _plain_logprobs(z, tokens, top):
    z = z.float()
    rows, v = z.shape
    most = z.amax(1)
    empty = most == -math.inf
    base = torch.where(empty, 0.0, most)[:, None]
    z0 = z - base
    e = torch.exp(z0)
    total = e.sum(1)
    log_total = torch.log(total)
    entropy = torch.where(empty, 0.0, log_total - (e * torch.where(e > 0, z0, 0.0)).sum(1) / total)
    picked = torch.where(empty[:, None], -math.inf, z0.gather(1, tokens) - log_total[:, None])
    # a larger value first, of equal ones the lower index: one whole number that orders both
    bits = z.view(torch.int32).to(torch.int64)
    order = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
    key = order * (1 << 31) + (v - 1 - torch.arange(v, device=z.device))
    at = torch.topk(key, top, dim=1).indices
    top_lp = torch.where(empty[:, None], -math.inf, z0.gather(1, at) - log_total[:, None])
    at = torch.where(top_lp == -math.inf, -1, at)
    return {"logprobs": picked, "lse": most + torch.where(empty, 0.0, log_total), "entropy": entropy, "top_ids": at,
            "top_logprobs": top_lp}


def _run_own(s):
    from exact_int8_gemm_amd import prism
    case = s["case"]
    op = case["op"]
    if op == "gemm":
        return prism.gemm_fp8_blockscale(s["q"], s["s_a"], s["w"], s["s_w"], out_dtype=TYPES[case["out"]])
    if op == "quant":
        return prism.quantize_blocks_fp8(s["x"])
    if op == "tiles":
        return prism.quantize_tiles_fp8(s["x"])
    if op == "swiglu":
        return prism.swiglu_quantize_fp8(s["gu"][:, :case["k"]], s["gu"][:, case["k"]:])
    r = prism.token_logprobs(s["z"], s["tokens"], top=case["top"])
    return {"logprobs": r.logprobs, "lse": r.lse, "entropy": r.entropy, "top_ids": r.top_ids,
            "top_logprobs": r.top_logprobs}


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    op = case["op"]
    if op == "gemm":
        return _plain_gemm(state, TYPES[case["out"]])
    if op == "quant":
        return _quantize_rows(state["x"])
    if op == "tiles":
        return _quantize_tiles(state["x"])
    if op == "swiglu":
        return _plain_swiglu(state["gu"])
    return _plain_logprobs(state["z"], state["tokens"], case["top"])


def work(case):
    op, m = case["op"], case["m"]
    if op == "logprobs":
        v, t, top = case["v"], case["t"], case["top"]
        return {"bytes": m * v * SIZE[case["in"]] + m * (8 * t + 4 * t + 8 + 12 * top), "flops": 8 * m * v}
    k = case["k"]
    kb = -(-k // BLOCK)
    if op == "gemm":
        n = case["n"]
        nb = -(-n // BLOCK)
        return {"bytes": m * k + n * k + 4 * m * kb + 4 * nb * kb + m * n * SIZE[case["out"]], "flops": 2 * m * n * k}
    if op == "tiles":
        return {"bytes": m * k * (SIZE[case["in"]] + 1) + 4 * -(-m // BLOCK) * kb, "flops": 5 * m * k}
    if op == "quant":
        return {"bytes": m * k * (SIZE[case["in"]] + 1) + 4 * m * kb, "flops": 5 * m * k}
    return {"bytes": m * k * (2 * SIZE[case["in"]] + 1) + 4 * m * kb, "flops": 15 * m * k}


# ------------------------------------------------------------- in 64 bits

def _group_max(x, rows):
    """max |x| over groups of `rows` rows by 128 columns, spread back over x's shape, and the groups' own."""
    m, k = x.shape
    mp, kp = -(-m // rows) * rows, -(-k // BLOCK) * BLOCK
    full = torch.zeros((mp, kp), dtype=torch.float64, device=x.device)
    full[:m, :k] = x.abs()
    groups = full.reshape(mp // rows, rows, kp // BLOCK, BLOCK).amax(dim=(1, 3))
    row = torch.arange(m, device=x.device) // rows
    col = torch.arange(k, device=x.device) // BLOCK
    return groups[row][:, col], groups


def _exact_quant(x, rows):
    """The quotients before their rounding to 8 bits, and the scales."""
    spread, groups = _group_max(x, rows)
    ratio = torch.zeros_like(x)
    some = spread > 0
    ratio[some] = x[some] * FP8_MAX / spread[some]
    return ratio, groups / FP8_MAX


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gemm":
        n, k = case["n"], case["k"]
        col = torch.arange(k, device="cuda") // BLOCK
        row = torch.arange(n, device="cuda") // BLOCK
        a = s["q"].double() * s["s_a"].double()[col].transpose(0, 1)
        w = s["w"].double() * s["s_w"].double()[row][:, col]
        return torch.mm(a, w.transpose(0, 1).contiguous())
    if op == "tiles":
        return _exact_quant(s["x"].double(), BLOCK)
    if op in ("quant", "swiglu"):
        if op == "quant":
            x = s["x"].double()
        else:
            gate, up = s["gu"][:, :case["k"]].double(), s["gu"][:, case["k"]:].double()
            x = gate * torch.sigmoid(gate) * up
        ratio, scale = _exact_quant(x, 1)
        return ratio, scale.transpose(0, 1).contiguous()
    z = s["z"].double()
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    lp = z - lse[:, None]
    lp[lse == -math.inf] = -math.inf
    entropy = -torch.where(z == -math.inf, 0.0, p * lp).sum(1)
    top_lp = lp.topk(case["top"], dim=1).values
    return {"logprobs": lp.gather(1, s["tokens"]), "lse": lse, "entropy": entropy, "top_ids": None, "top_logprobs": top_lp}
