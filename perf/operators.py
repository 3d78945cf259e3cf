"""What is measured of the FP8 operators and the router's balance loss: cases, inputs, one pass of each, and its work.

Where ``own`` is false ``run`` computes an operator in its plain form, from elementary torch operations in fp32;
where it is true it makes the calls that a user of the framework makes.
"""
import math

import torch

own = False

BLOCK = 128        # values that share a scale
E4M3_MAX = 448.0
FLOOR = 2.0 ** -100
FP8 = torch.float8_e4m3fn
FLOATS = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}

# (E, k, H, I): the layer families of this repository's workloads
LAYERS = {"tiny": (8, 2, 256, 512), "main": (128, 8, 2048, 768), "slots": (512, 10, 2048, 512),
          "wide": (32, 4, 2880, 2880)}


def listed():
    return [
        # activations of a decode batch, and of a prefill of 8192 tokens of the wide layer (22.5 blocks in a row)
        {"name": "quant_decode", "op": "quant", "M": 64, "K": 2048, "dtype": "bf16"},
        {"name": "quant_prefill", "op": "quant", "M": 8192, "K": 2880, "dtype": "bf16"},
        # a dense projection beside the experts: one token, a decode batch, a ragged chunk, a prefill
        {"name": "gemm_one_token", "op": "gemm", "M": 1, "N": 2048, "K": 2048, "out": "bf16"},
        {"name": "gemm_decode", "op": "gemm", "M": 64, "N": 5760, "K": 2880, "out": "bf16"},
        {"name": "gemm_ragged", "op": "gemm", "M": 1037, "N": 1234, "K": 1100, "out": "fp32"},
        {"name": "gemm_prefill", "op": "gemm", "M": 8192, "N": 8192, "K": 2048, "out": "bf16"},
        # the expert FFN: one token, a decode batch, a skewed prefill, a prefill of few wide experts
        {"name": "ffn_one_token", "op": "ffn", "T": 1, "layer": "main", "zipf": False},
        {"name": "ffn_decode", "op": "ffn", "T": 64, "layer": "main", "zipf": False},
        {"name": "ffn_prefill", "op": "ffn", "T": 4096, "layer": "main", "zipf": True},
        {"name": "ffn_wide", "op": "ffn", "T": 1500, "layer": "wide", "zipf": False},
        # a training step's router: a small batch, and a long one whose last tokens are padding
        {"name": "balance_small", "op": "balance", "T": 64, "E": 128, "k": 8, "padded": 0},
        {"name": "balance_large", "op": "balance", "T": 8192, "E": 512, "k": 10, "padded": 700},
    ]


def _log(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op = rng.choice(["quant", "gemm", "gemm", "ffn", "ffn", "balance"])
    if op == "quant":
        return {"op": op, "M": _log(rng, 1, 8192), "K": _log(rng, 64, 2880), "dtype": rng.choice(["bf16", "fp16", "fp32"])}
    if op == "gemm":
        while True:
            M, N, K = _log(rng, 1, 8192), _log(rng, 16, 8192), _log(rng, 64, 4096)
            if M * N * K <= 8192 * 8192 * 2048:
                return {"op": op, "M": M, "N": N, "K": K, "out": rng.choice(["bf16", "fp32"])}
    if op == "ffn":
        layer = rng.choice(sorted(LAYERS))
        most = {"tiny": 8192, "main": 4096, "slots": 4096, "wide": 1500}[layer]
        return {"op": op, "T": _log(rng, 1, most), "layer": layer, "zipf": rng.random() < 0.5}
    E = _log(rng, 2, 512)
    T = _log(rng, 1, 8192)
    return {"op": op, "T": T, "E": E, "k": min(E, rng.randint(1, 10)), "padded": rng.randint(0, T // 4)}


# ------------------------------------------------------------- inputs ---

def _blocks(n):
    return -(-n // BLOCK)


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _quant_rows(x):
    """fp32 [..., K] -> (codes, scales): one scale for each 128 values of a row."""
    K = x.shape[-1]
    padded = torch.nn.functional.pad(x, (0, _blocks(K) * BLOCK - K))
    groups = padded.view(*x.shape[:-1], _blocks(K), BLOCK)
    top = groups.abs().amax(-1).clamp(min=FLOOR)
    codes = (groups * E4M3_MAX / top[..., None]).to(FP8)
    return codes.view(*x.shape[:-1], -1)[..., :K], top / E4M3_MAX


def _quant_weight(w):
    """fp32 [..., N, K] -> (codes, scales [..., ceil(N/128), ceil(K/128)]): one scale for each 128 x 128 block."""
    N, K = w.shape[-2:]
    nb, kb = _blocks(N), _blocks(K)
    padded = torch.nn.functional.pad(w, (0, kb * BLOCK - K, 0, nb * BLOCK - N))
    tiles = padded.view(*w.shape[:-2], nb, BLOCK, kb, BLOCK)
    top = tiles.abs().amax((-3, -1)).clamp(min=FLOOR)
    codes = (tiles * E4M3_MAX / top[..., None, :, None]).to(FP8)
    return codes.view(*w.shape[:-2], nb * BLOCK, kb * BLOCK)[..., :N, :K], top / E4M3_MAX


def _rows16(codes):
    """The codes in rows that start on 16 bytes."""
    K = codes.shape[-1]
    out = torch.zeros(*codes.shape[:-1], -(-K // 16) * 16, dtype=torch.uint8, device=codes.device)
    out[..., :K] = codes.view(torch.uint8)
    return out.view(FP8)[..., :K]


def _slot_layout(H, I):
    """Offsets of gate, up and down in an FP8 expert slot: codes [N, K], fp32 scales in rows of ld bytes."""
    off, codes, scales, ld = 0, [], [], []
    for N, K in ((I, H), (I, H), (H, I)):
        codes.append(off)
        off = -(-(off + N * K) // 256) * 256
        scales.append(off)
        ld.append(-(-4 * _blocks(K) // 16) * 16)
        off = -(-(off + _blocks(N) * ld[-1]) // 256) * 256
    return codes, scales, ld, -(-(off + 12) // 256) * 256


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    randn = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    if op == "quant":
        # rows of unlike magnitude, as a residual stream has them
        x = randn(case["M"], case["K"]) * torch.exp(randn(case["M"], 1))
        return {"case": case, "x": x.to(FLOATS[case["dtype"]])}
    if op == "gemm":
        a, a_scales = _quant_rows(randn(case["M"], case["K"]))
        b, b_scales = _quant_weight(randn(case["N"], case["K"]) * 0.02)
        return {"case": case, "a": _rows16(a), "a_scales": a_scales, "b": _rows16(b), "b_scales": b_scales}
    if op == "balance":
        T, E, k = case["T"], case["E"], case["k"]
        logits = randn(T, E) + randn(E)
        w, ids = torch.softmax(logits, -1).topk(k, dim=-1)
        valid = torch.arange(T, device="cuda") < T - case["padded"]
        return {"case": case, "logits": logits, "ids": ids.int(), "w": w / w.sum(-1, keepdim=True), "dw": randn(T, k) / T,
                "valid": valid, "dloss": 0.5 + torch.rand(1, generator=g, device="cuda"), "coef": 0.01}
    E, k, H, I = LAYERS[case["layer"]]
    T = case["T"]
    slots = E + 3
    codes, scales, ld, slot_bytes = _slot_layout(H, I)
    pool = torch.zeros(slots, slot_bytes, dtype=torch.uint8, device="cuda")
    for m, (N, K) in enumerate(((I, H), (I, H), (H, I))):
        c, s = _quant_weight(randn(slots, N, K) * 0.02)
        pool[:, codes[m]:codes[m] + N * K] = c.contiguous().view(torch.uint8).view(slots, -1)
        pool[:, scales[m]:scales[m] + _blocks(N) * ld[m]].view(slots, _blocks(N), ld[m])[..., :4 * _blocks(K)] = \
            s.contiguous().view(torch.uint8).view(slots, _blocks(N), -1)
        del c, s
    logits = randn(T, E)
    if case["zipf"]:   # a few experts are much asked for
        rank = torch.randperm(E, generator=g, device="cuda") + 1.0
        logits = logits + 2.0 - 4.0 * rank.log() / math.log(E)
    ids = logits.topk(k, dim=-1).indices.flatten()
    perm_src = ids.sort(stable=True).indices.int()
    rows = torch.bincount(ids, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = rows.cumsum(0)
    table = torch.randperm(slots, generator=g, device="cuda")[:E].int()
    return {"case": case, "x": randn(T, H).bfloat16(), "pool": pool.view(-1), "table": table, "perm_src": perm_src,
            "offsets": offsets, "active": rows.nonzero().flatten(), "most": int(rows.max()), "slots": slots}


# --------------------------------------------------------- plain forms ---

def _dequant_rows(codes, scales):
    return codes.float() * scales.repeat_interleave(BLOCK, -1)[..., :codes.shape[-1]]


def _dequant_weight(codes, scales):
    N, K = codes.shape[-2:]
    return codes.float() * scales.repeat_interleave(BLOCK, -2)[..., :N, :].repeat_interleave(BLOCK, -1)[..., :K]


def _expert_tensor(state, mat, experts):
    """(codes, scales) of one of the three tensors of the given experts, from their slots."""
    E, k, H, I = LAYERS[state["case"]["layer"]]
    codes, scales, ld, slot_bytes = _slot_layout(H, I)
    N, K = (H, I) if mat == 2 else (I, H)
    slots = state["pool"].view(-1, slot_bytes)
    at = state["table"].long()[experts]
    c = slots[:, codes[mat]:codes[mat] + N * K][at].view(FP8).view(-1, N, K)
    s = slots[:, scales[mat]:scales[mat] + _blocks(N) * ld[mat]][at].view(torch.float32).view(-1, _blocks(N), ld[mat] // 4)
    return c, s[..., :_blocks(K)]


def _plain_ffn(state):
    E, k, H, I = LAYERS[state["case"]["layer"]]
    x, active, offsets, perm_src = state["x"], state["active"], state["offsets"].long(), state["perm_src"].long()
    P = perm_src.numel()
    xq = _dequant_rows(*_quant_rows(x.float()))
    row = torch.arange(P, device=x.device)
    at = torch.searchsorted(offsets[active], row, right=True) - 1      # which active expert a row is of
    place = row - offsets[active][at]                                    # and its place in that group
    grid = (offsets[active][:, None] + torch.arange(state["most"], device=x.device)).clamp(max=P - 1)
    rows = xq[perm_src[grid] // k]
    gate = rows @ _dequant_weight(*_expert_tensor(state, 0, active)).transpose(1, 2)
    up = rows @ _dequant_weight(*_expert_tensor(state, 1, active)).transpose(1, 2)
    h = _dequant_rows(*_quant_rows(gate / (1.0 + torch.exp(-gate)) * up))
    out = h @ _dequant_weight(*_expert_tensor(state, 2, active)).transpose(1, 2)
    return out[at, place].bfloat16()


def _plain_balance(state):
    logits, ids, w, dw, valid = (state[n] for n in ("logits", "ids", "w", "dw", "valid"))
    T, E = logits.shape
    k = ids.shape[1]
    live = valid[:, None].float()
    z = torch.exp(logits - logits.amax(-1, keepdim=True))
    p = z / z.sum(-1, keepdim=True)
    counts = torch.zeros(E, dtype=torch.int32, device=logits.device)
    counts.index_add_(0, ids.flatten().long(), valid[:, None].expand(T, k).flatten().int())
    n = valid.sum().float().clamp(min=1.0)
    c = counts.float()
    loss = state["coef"] * E / (n * n * k) * (c * (p * live).sum(0)).sum()
    dlogits = state["dloss"] * state["coef"] * E / (n * n * k) * p * (c - (p * c).sum(-1, keepdim=True))
    dlogits = dlogits.scatter_add(1, ids.long(), w * (dw - (w * dw).sum(-1, keepdim=True)))
    return {"loss": loss.reshape(1), "counts": counts, "dlogits": dlogits * live}


def run(state):
    case = state["case"]
    if own:
        return _own(state)
    if case["op"] == "quant":
        codes, scales = _quant_rows(state["x"].float())
        return {"codes": codes, "scales": scales}
    if case["op"] == "gemm":
        a, b = _dequant_rows(state["a"], state["a_scales"]), _dequant_weight(state["b"], state["b_scales"])
        return (a @ b.T).to(FLOATS[case["out"]])
    return _plain_balance(state) if case["op"] == "balance" else _plain_ffn(state)


def _own(state):
    from moe_expert_layer_renorm_b200 import _lib, balance, fp8, layer
    case = state["case"]
    if case["op"] == "quant":
        codes, scales = fp8.quantize_rows(state["x"])
        return {"codes": codes, "scales": scales}
    if case["op"] == "gemm":
        if "linear" not in state:
            state["linear"] = fp8.Fp8Linear(state["b"], state["b_scales"])
        return state["linear"].matmul(state["a"], state["a_scales"], out_dtype=FLOATS[case["out"]])
    if case["op"] == "balance":
        if "balance" not in state:
            state["balance"] = balance.RouterBalance(case["T"], case["E"], case["k"], state["coef"])
        b = state["balance"]
        loss = b.forward(state["logits"], state["ids"], valid=state["valid"])
        dlogits = b.backward(state["logits"], state["ids"], dloss=state["dloss"], w=state["w"], dw=state["dw"], valid=state["valid"])
        return {"loss": loss, "counts": b.counts, "dlogits": dlogits}
    if "layer" not in state:
        E, k, H, I = LAYERS[case["layer"]]
        state["experts"] = layer.ExpertPool(H, I, state["slots"], fmt=_lib.FT_SCALE_FP8, buf=state["pool"])
        state["layer"] = layer.MoELayer(case["T"], E, k, H, I, out_dtype=torch.bfloat16)
        state["layer"].perm_src, state["layer"].offsets = state["perm_src"], state["offsets"]
    state["layer"].ffn(state["x"], state["table"], state["experts"])
    return state["layer"].out_perm


# ---------------------------------------------------------------- work ---

def work(case):
    op = case["op"]
    if op == "quant":
        M, K = case["M"], case["K"]
        return {"bytes": M * K * (4 if case["dtype"] == "fp32" else 2) + M * K + 4 * M * _blocks(K), "flops": 2 * M * K}
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        scales = 4 * _blocks(K) * (M + _blocks(N))
        return {"bytes": M * K + N * K + scales + M * N * (4 if case["out"] == "fp32" else 2), "flops": 2 * M * N * K}
    if op == "balance":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": 8 * T * E + 12 * T * k + T + 4 * E, "flops": 12 * T * E}
    E, k, H, I = LAYERS[case["layer"]]
    T = case["T"]
    experts = E * (1.0 - (1.0 - k / E) ** T)     # expected, for even routing
    weights = 3 * H * I + 4 * 3 * _blocks(H) * _blocks(I)
    return {"bytes": experts * weights + 2 * T * H + 2 * T * k * H + 4 * T * k, "flops": 6 * T * k * H * I}


# --------------------------------------------------------------- exact ---

def _e4m3_64(v):
    """fp64 values to the nearest E4M3 value (ties to even), at most 448 in magnitude."""
    exponent = torch.frexp(v.abs().clamp(min=2.0 ** -6)).exponent - 1
    step = torch.ldexp(torch.ones_like(v), exponent - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _codes_64(x):
    """fp64 rows -> (values of the codes, scales of each 128 spread over their values, one scale for each 128)."""
    K = x.shape[1]
    codes, spread, scales = torch.empty_like(x), torch.empty_like(x), []
    for k0 in range(0, K, BLOCK):
        part = x[:, k0:k0 + BLOCK]
        top = part.abs().max(dim=1, keepdim=True).values.clamp(min=FLOOR)
        codes[:, k0:k0 + BLOCK], spread[:, k0:k0 + BLOCK] = _e4m3_64(E4M3_MAX * part / top), top / E4M3_MAX
        scales.append(top / E4M3_MAX)
    return codes, spread, torch.cat(scales, 1)


def _weight_64(codes, scales):
    w = codes.double()
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            w[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK] *= scales[i, j].double()
    return w


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "quant":
        codes, _, scales = _codes_64(state["x"].double())
        return {"codes": codes, "scales": scales}
    if case["op"] == "gemm":
        a = state["a"].double()
        for j in range(state["a_scales"].shape[1]):
            a[:, j * BLOCK:(j + 1) * BLOCK] *= state["a_scales"][:, j:j + 1].double()
        return torch.matmul(a, _weight_64(state["b"], state["b_scales"]).t())
    if case["op"] == "balance":
        live = state["valid"].nonzero().flatten()
        l = state["logits"][live].double().requires_grad_()
        ids = state["ids"][live].long()
        counts = torch.bincount(ids.flatten(), minlength=case["E"])
        share = torch.softmax(l, 1).mean(0) if len(live) else l.sum(0)
        loss = state["coef"] * case["E"] * (counts.double() / max(1, len(live) * case["k"]) * share).sum()
        # the router's weights: softmax of the selected logits
        chosen = torch.softmax(torch.gather(l, 1, ids), 1)
        grad, = torch.autograd.grad(state["dloss"].double()[0] * loss + (chosen * state["dw"][live].double()).sum(), l)
        dlogits = torch.zeros(case["T"], case["E"], dtype=torch.float64, device=l.device)
        dlogits[live] = grad
        return {"loss": loss.detach().reshape(1), "counts": counts.int(), "dlogits": dlogits}
    E, k, H, I = LAYERS[case["layer"]]
    codes, spread, _ = _codes_64(state["x"].double())
    x = codes * spread
    out = torch.empty(case["T"] * k, H, dtype=torch.float64, device=x.device)
    offsets = state["offsets"].tolist()
    for e in state["active"].tolist():
        one = torch.tensor([e], device=x.device)
        gate, up, down = (_weight_64(c[0], s[0]) for c, s in (_expert_tensor(state, m, one) for m in range(3)))
        rows = x[state["perm_src"][offsets[e]:offsets[e + 1]].long() // k]
        pre = rows @ gate.T
        codes, spread, _ = _codes_64(pre * torch.sigmoid(pre) * (rows @ up.T))
        out[offsets[e]:offsets[e + 1]] = (codes * spread) @ down.T
    return out
