"""The operators of a mixture-of-experts serving step around the block-scaled FP8 products, as cases to measure.

  norm   residual addition, root-mean-square norm, and its output as e4m3 codes with 1x128 scales
         (dg_fp8_rmsnorm_quantize_1x128)
  gate   the k largest router logits of each token, and their softmax or sigmoid weights (dg_moe_gate_topk)
  layer  gate and up projection, SwiGLU, down projection and weighted sum over the chosen experts, for a few
         tokens (dg_fp8_moe_layer)

`run` takes the plain form (elementary torch operations in 32 bits, one rounding at the end) where `own` is false and
the framework's entry points where it is true; `exact` computes the same outputs in 64 bits.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def _norm(M, K, x="bf16", residual="bf16", weight="bf16", normed=True):
    """residual: the residual stream's type, or "none"; normed: the bf16 rows that a router reads are wanted too."""
    return {"op": "norm", "M": M, "K": K, "x": x, "residual": residual, "weight": weight, "normed": normed}


def _gate(T, E, k, logits="f32", score="softmax", renormalize=True, masked=False):
    """masked: a quarter of the logits are -inf (experts that a token may not use), and every 17th token has no expert."""
    return {"op": "gate", "T": T, "E": E, "k": k, "logits": logits, "score": score, "renormalize": renormalize,
            "masked": masked}


def _layer(T, k, E, H, I, shards=1):  # noqa: E741
    """shards: the E experts are one of so many equal shares of the model's; other experts' slots hold -1."""
    return {"op": "layer", "T": T, "k": k, "E": E, "H": H, "I": I, "shards": shards}


def listed():
    cases = {
        # One token of a decoding request: the launch and one row's latency.
        "norm_1x7168": _norm(1, 7168),
        # A batch of decoding requests, an fp32 residual stream.
        "norm_64x7168_f32_residual": _norm(64, 7168, residual="f32"),
        # A first norm (no residual yet) over odd sizes, fp32 activations and weight, no router behind it.
        "norm_613x1152_f32": _norm(613, 1152, x="f32", residual="none", weight="f32", normed=False),
        # The tokens of a prefill, as the contiguous grouped product takes them.
        "norm_8192x7168": _norm(8192, 7168),
        # One token's router, 32 experts.
        "gate_1x32_top8": _gate(1, 32, 8),
        # A ragged batch, bf16 logits (ties), sigmoid scores, masked experts and tokens without any.
        "gate_203x96_top6_masked": _gate(203, 96, 6, logits="bf16", score="sigmoid", masked=True),
        # A prefill's router over many experts.
        "gate_8192x256_top8": _gate(8192, 256, 8, renormalize=False),
        # One token through 8 of 32 experts: eight experts' weights are the whole cost.
        "layer_1_top8_e32": _layer(1, 8, 32, 7168, 2048),
        # A few requests on a small layer: latency.
        "layer_5_top2_e8_small": _layer(5, 2, 8, 1024, 384),
        # A batch on one of four shares of the experts, odd block counts (23 and 9): most slots belong elsewhere.
        "layer_33_top6_e16_shard": _layer(33, 6, 16, 2944, 1152, shards=4),
        # A batch that uses all of eight experts, each by half of the tokens.
        "layer_32_top4_e8": _layer(32, 4, 8, 7168, 2048),
        # The largest batch: every one of 32 experts is read.
        "layer_64_top8_e32": _layer(64, 8, 32, 7168, 2048),
    }
    return [{"name": name, **case} for name, case in cases.items()]


def _log_uniform(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["norm", "gate", "layer", "layer"])
    if op == "norm":
        return _norm(_log_uniform(rng, 1, 8192), BLOCK * _log_uniform(rng, 1, 56), x=rng.choice(["bf16", "bf16", "f32"]),
                     residual=rng.choice(["bf16", "f32", "none"]) if rng.random() < 0.7 else "bf16",
                     weight=rng.choice(["bf16", "f32"]), normed=rng.random() < 0.6)
    if op == "gate":
        E = _log_uniform(rng, 2, 512)
        return _gate(_log_uniform(rng, 1, 8192), E, rng.randint(1, min(E, 16)), logits=rng.choice(["f32", "bf16"]),
                     score=rng.choice(["softmax", "sigmoid"]), renormalize=rng.random() < 0.6,
                     masked=rng.random() < 0.4)
    E = _log_uniform(rng, 2, 64)
    H, I = BLOCK * _log_uniform(rng, 2, 56), BLOCK * _log_uniform(rng, 1, 16)  # noqa: E741
    while E * H * I > 32 * 7168 * 2048:
        E -= 1
    shards = rng.choice([1, 1, 2, 4])
    return _layer(_log_uniform(rng, 1, 64), rng.randint(1, min(E, 8)), E, H, I, shards=shards)


# ---------------------------------------------------------------- inputs

def _normal_with_outliers(shape, gen, share=1e-3, factor=50.0):
    """N(0, 1) with one value in a thousand 50 times as large, as activations have them."""
    x = torch.randn(shape, generator=gen, device="cuda")
    x[torch.rand(shape, generator=gen, device="cuda") < share] *= factor
    return x


def _quantize_rows(x):
    """e4m3 codes [M, K] of fp32 rows, and the scales of their 1x128 blocks, as a view of an M-major table."""
    M, K = x.shape
    blocks = x.view(M, K // BLOCK, BLOCK)
    s = blocks.abs().amax(-1) / E4M3_MAX
    codes = (blocks / s[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.view(M, K), s.t().contiguous().t()


def _expert_weights(E, N, K, gen):
    """e4m3 codes [E, N, K] of normal weights of variance 1/K, and the scales of their 128x128 blocks."""
    codes = torch.empty((E, N, K), dtype=torch.uint8, device="cuda")
    scales = torch.empty((E, N // BLOCK, K // BLOCK), device="cuda")
    for e in range(E):
        w = torch.randn((N // BLOCK, BLOCK, K // BLOCK, BLOCK), generator=gen, device="cuda") * K ** -0.5
        scales[e] = w.abs().amax((1, 3)) / E4M3_MAX
        w = (w / scales[e][:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
        codes[e] = w.to(torch.float8_e4m3fn).view(torch.uint8).view(N, K)
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    state = {"case": case}
    if case["op"] == "norm":
        M, K = case["M"], case["K"]
        state["x"] = _normal_with_outliers((M, K), gen).to(DTYPES[case["x"]])
        state["weight"] = (1 + 0.2 * torch.randn(K, generator=gen, device="cuda")).to(DTYPES[case["weight"]])
        state["residual"] = None
        if case["residual"] != "none":
            state["residual"] = (3 * _normal_with_outliers((M, K), gen)).to(DTYPES[case["residual"]])
    elif case["op"] == "gate":
        T, E = case["T"], case["E"]
        logits = 2 * torch.randn((T, E), generator=gen, device="cuda") + torch.randn(E, generator=gen, device="cuda")
        if case["masked"]:
            logits[torch.rand((T, E), generator=gen, device="cuda") < 0.25] = -math.inf
            logits[::17] = -math.inf
        state["logits"] = logits.to(DTYPES[case["logits"]])
    else:
        T, k, E, H, I = (case[n] for n in ("T", "k", "E", "H", "I"))  # noqa: E741
        state["x"], state["sx"] = _quantize_rows(_normal_with_outliers((T, H), gen))
        state["w13"], state["s13"] = _expert_weights(E, 2 * I, H, gen)
        state["w2"], state["s2"] = _expert_weights(E, H, I, gen)
        # k different experts of the model for each token; this share holds the first E of them.
        order = torch.rand((T, E * case["shards"]), generator=gen, device="cuda").argsort(dim=1)[:, :k]
        state["ids"] = torch.where(order < E, order, -1).to(torch.int32)
        weights = torch.rand((T, k), generator=gen, device="cuda") + 0.1
        state["weights"] = weights / weights.sum(1, keepdim=True)
    return state


# ---------------------------------------------------------------- plain forms

def _plain_norm(case, x, weight, residual):
    h = x.float()
    out = {}
    if residual is not None:
        h = h + residual.float()
        out["residual"] = h.to(residual.dtype)
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * weight.float()
    if case["normed"]:
        out["y"] = y.to(torch.bfloat16)
    blocks = y.view(y.shape[0], -1, BLOCK)
    amax = blocks.abs().amax(-1)
    s = torch.where(amax == 0, torch.ones_like(amax), amax / E4M3_MAX)
    q = (blocks / s[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return {**out, "q": q.view(y.shape), "s": s}


def _plain_gate(case, logits):
    l = logits.float()  # noqa: E741
    top, ids = torch.sort(l, dim=1, descending=True, stable=True)
    top, ids = top[:, :case["k"]], ids[:, :case["k"]]
    chosen = top > -math.inf
    if case["score"] == "softmax":
        largest = torch.where(chosen[:, :1], top[:, :1], 0)
        score = torch.exp(top - largest)
        if case["renormalize"]:
            weights = score / score.sum(1, keepdim=True).clamp_min(1e-30)
        else:
            weights = score / torch.exp(l - largest).sum(1, keepdim=True).clamp_min(1e-30)
    else:
        weights = 1 / (1 + torch.exp(-top))
        if case["renormalize"]:
            weights = weights / weights.sum(1, keepdim=True).clamp_min(1e-30)
    return {"ids": torch.where(chosen, ids, -1).to(torch.int32), "weights": torch.where(chosen, weights, 0)}


def _dequantize(codes, scales):
    """fp32 values of e4m3 codes [E, N, K] with a scale for each 128x128 block."""
    E, N, K = codes.shape
    values = codes.view(torch.float8_e4m3fn).float().view(E, N // BLOCK, BLOCK, K // BLOCK, BLOCK)
    return (values * scales[:, :, None, :, None]).view(E, N, K)


def _plain_layer(case, x, sx, w13, s13, w2, s2, ids, weights):
    T, k, E, H, I = (case[n] for n in ("T", "k", "E", "H", "I"))  # noqa: E741
    xf = (x.view(torch.float8_e4m3fn).float().view(T, H // BLOCK, BLOCK) * sx[:, :, None]).view(T, H)
    chosen, ids = ids >= 0, ids.clamp_min(0).long()
    if T * k < E:
        # Few pairs of token and expert: each pair reads its expert.
        pair = ids.view(-1)
        rows = xf.repeat_interleave(k, 0)
        gu = (_dequantize(w13[pair], s13[pair]) * rows[:, None, :]).sum(2)
        g, u = gu[:, :I], gu[:, I:]
        h = g / (1 + torch.exp(-g)) * u
        y = (_dequantize(w2[pair], s2[pair]) * h[:, None, :]).sum(2).view(T, k, H)
        return (torch.where(chosen, weights, 0)[:, :, None] * y).sum(1).to(torch.bfloat16)
    # Every token through every expert, as two products, with a weight of zero where the token did not choose it.
    combine = torch.zeros((T, E), device=x.device).scatter_add(1, ids, torch.where(chosen, weights, 0))
    gu = (xf @ _dequantize(w13, s13).view(E * 2 * I, H).t()).view(T, E, 2 * I)
    g, u = gu[:, :, :I], gu[:, :, I:]
    h = g / (1 + torch.exp(-g)) * u * combine[:, :, None]
    down = _dequantize(w2, s2).transpose(1, 2).reshape(E * I, H)
    return (h.view(T, E * I) @ down).to(torch.bfloat16)


# ---------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if own:
        import fp8_block_scaled_sa_amd as dg
    if case["op"] == "norm":
        args = (state["x"], state["weight"])
        if not own:
            return _plain_norm(case, *args, state["residual"])
        q, s, residual, y = dg.dg_fp8_rmsnorm_quantize_1x128(*args, EPS, residual=state["residual"],
                                                             normed=case["normed"])
        out = {"q": q.view(torch.float8_e4m3fn), "s": s}
        if residual is not None:
            out["residual"] = residual
        if y is not None:
            out["y"] = y
        return out
    if case["op"] == "gate":
        if not own:
            return _plain_gate(case, state["logits"])
        ids, weights = dg.dg_moe_gate_topk(state["logits"], case["k"], score=case["score"],
                                           renormalize=case["renormalize"])
        return {"ids": ids, "weights": weights}
    args = [state[n] for n in ("x", "sx", "w13", "s13", "w2", "s2", "ids", "weights")]
    if not own:
        return _plain_layer(case, *args)
    if "workspace" not in state:
        # A serving program keeps one for all of its steps.
        state["workspace"] = dg.workspace(dg.dg_fp8_moe_layer_workspace_bytes(case["T"], case["k"], case["H"],
                                                                              case["I"]))
    return dg.dg_fp8_moe_layer(*args, state["workspace"])


# ---------------------------------------------------------------- bytes and operations

def work(case):
    if case["op"] == "norm":
        n = case["M"] * case["K"]
        size = {"bf16": 2, "f32": 4, "none": 0}
        per = size[case["x"]] + 2 * size[case["residual"]] + 2 * case["normed"] + 1 + 4 / BLOCK
        return {"bytes": n * per + case["K"] * size[case["weight"]], "flops": 8 * n}
    if case["op"] == "gate":
        n = case["T"] * case["E"]
        return {"bytes": n * (4 if case["logits"] == "f32" else 2) + 8 * case["T"] * case["k"], "flops": 4 * n}
    T, k, E, H, I = (case[n] for n in ("T", "k", "E", "H", "I"))  # noqa: E741
    share = k / (E * case["shards"])                    # how likely a token is to choose an expert
    experts = E * (1 - (1 - share) ** T)                # experts that some token chose, on average
    per_expert = 3 * H * I * (1 + 4 / BLOCK ** 2)
    return {"bytes": experts * per_expert + T * H * (1 + 4 / BLOCK + 2) + 8 * T * k,
            "flops": 2 * 3 * H * I * T * k / case["shards"]}


# ---------------------------------------------------------------- 64 bits

def _e4m3_values():
    """The value of each e4m3 code from its bits: sign, 4 exponent bits with bias 7, 3 mantissa bits, no infinity."""
    values = []
    for code in range(256):
        exponent, mantissa = (code >> 3) & 15, code & 7
        v = math.ldexp(8 + mantissa, exponent - 10) if exponent else math.ldexp(mantissa, -9)
        values.append(math.nan if code & 0x7F == 0x7F else -v if code & 0x80 else v)
    return torch.tensor(values, dtype=torch.float64, device="cuda")


def _exact_norm(case, state):
    h = state["x"].double()
    out = {}
    if state["residual"] is not None:
        h = h + state["residual"].double()
        out["residual"] = h
    scale = (torch.linalg.vector_norm(h, dim=1).square() / case["K"] + EPS).sqrt()
    y = h / scale[:, None] * state["weight"].double()
    if case["normed"]:
        out["y"] = y
    amax = torch.stack([b.abs().max(1).values for b in y.split(BLOCK, 1)], 1)
    s = torch.where(amax > 0, amax / E4M3_MAX, 1.0)
    # The code stands for y / s; its own rounding is part of how far a code is from that.
    return {**out, "q": y / s.repeat_interleave(BLOCK, 1), "s": s}


def _exact_gate(case, state):
    l = state["logits"].double()  # noqa: E741
    T, k = case["T"], case["k"]
    ids = torch.full((T, k), -1, dtype=torch.int32, device=l.device)
    picked = torch.full((T, k), -math.inf, dtype=torch.float64, device=l.device)
    left = l.clone()
    at = torch.arange(l.shape[1], device=l.device)
    for j in range(k):
        most = left.max(1).values
        # the lowest index of those that hold the largest value
        first = torch.where(left == most[:, None], at, l.shape[1]).min(1).values
        some = most > -math.inf
        ids[:, j] = torch.where(some, first, -1).to(torch.int32)
        picked[:, j] = most
        left[at == first[:, None]] = -math.inf
    none = picked == -math.inf
    if case["score"] == "softmax":
        over = torch.logsumexp(picked if case["renormalize"] else l, dim=1)
        weights = torch.exp(picked - torch.where(over > -math.inf, over, 0)[:, None])
    else:
        weights = torch.sigmoid(picked)
        if case["renormalize"]:
            total = weights.sum(1)
            weights = weights / torch.where(total > 0, total, 1)[:, None]
    return {"ids": ids, "weights": torch.where(none, 0, weights)}


def _exact_layer(case, state):
    T, H, I = case["T"], case["H"], case["I"]  # noqa: E741
    values = _e4m3_values()
    spread = lambda s: s.double().repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)  # noqa: E731
    x = values[state["x"].long()] * state["sx"].double().repeat_interleave(BLOCK, 1)
    out = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        t, slot = torch.nonzero(state["ids"] == e, as_tuple=True)
        if not len(t):
            continue
        both = x[t] @ (values[state["w13"][e].long()] * spread(state["s13"][e])).t()
        h = torch.sigmoid(both[:, :I]) * both[:, :I] * both[:, I:]
        y = h @ (values[state["w2"][e].long()] * spread(state["s2"][e])).t()
        out.index_add_(0, t, state["weights"][t, slot].double()[:, None] * y)
    return out


def exact(case, seed):
    state = prepare(case, seed)
    return {"norm": _exact_norm, "gate": _exact_gate, "layer": _exact_layer}[case["op"]](case, state)
