"""Cases of the 8-bit and feed-forward operators: what a pass is, its inputs and its plain form.

    quantize_int8      rows of activations -> int8 values and one fp32 scale a row
    decode_int8        trellis bitstreams -> int8 weights (one scale for all)
    int8_matmul        int8 x int8 product with scales for each token and channel
    gated_ffn          act(x Wg^T) * (x Wu^T) on 16-bit weights, and its gradients
    int8_gated_ffn     the same block on int8 tokens and weights

``own`` false computes them from elementary torch operations; true calls the
package.  Sizes are the package's own (1024, 2048 and 8192 wide matrices, L =
12 and 16 streams), with ragged token counts.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
LCG_MUL, LCG_ADD = 34038481, 76625530        # the 1MAD code's generator


def listed():
    return [
        # the activations of one token in front of an 8-bit product: latency
        {"name": "quantize_token_f16", "op": "quantize", "M": 1, "K": 8192, "dtype": "f16"},
        # a prefill batch's activations, bound by HBM traffic
        {"name": "quantize_prefill_bf16", "op": "quantize", "M": 4096, "K": 8192, "dtype": "bf16"},
        # a whole 8192 x 8192 matrix from its tail-biting tiles, once per load of a model
        {"name": "decode_int8_l16_8192sq", "op": "decode", "L": 16, "layout": 0, "tiles": True,
         "rows": 8192, "cols": 8192, "n": 262144, "T": 256},
        # 1,024 free-start sequences, the batch that the L = 12 encode works on
        {"name": "decode_int8_l12_seq", "op": "decode", "L": 12, "layout": 1, "tiles": False,
         "rows": 0, "cols": 0, "n": 1024, "T": 256},
        # one new token against an 8192 x 8192 weight: the weight's bytes count
        {"name": "int8_matmul_token", "op": "matmul", "M": 1, "N": 8192, "K": 8192, "out": "f16",
         "bias": False},
        # a prefill of ragged length, bound by the tensor cores
        {"name": "int8_matmul_prefill", "op": "matmul", "M": 3001, "N": 8192, "K": 8192, "out": "bf16",
         "bias": True},
        # one new token through a feed-forward block of decoded fp16 weights
        {"name": "gated_ffn_token_f16", "op": "gated", "M": 1, "K": 2048, "F": 8192, "dtype": "f16",
         "act": "silu"},
        # a prefill of ragged length
        {"name": "gated_ffn_prefill_bf16", "op": "gated", "M": 3001, "K": 2048, "F": 8192,
         "dtype": "bf16", "act": "silu"},
        # a step of quantisation-aware training: block output and all three gradients
        {"name": "gated_ffn_train_bf16", "op": "train", "M": 4096, "K": 2048, "F": 8192,
         "dtype": "bf16", "act": "silu"},
        # the same on a small block whose hidden width is no multiple of 8
        {"name": "gated_ffn_train_odd_f16", "op": "train", "M": 777, "K": 1024, "F": 2731,
         "dtype": "f16", "act": "gelu"},
        # a decode batch of sixteen requests on 8-bit weights
        {"name": "int8_gated_ffn_batch", "op": "gated8", "M": 16, "K": 2048, "F": 8192, "out": "f16",
         "act": "silu"},
        # a prefill on 8-bit weights
        {"name": "int8_gated_ffn_prefill", "op": "gated8", "M": 2048, "K": 2048, "F": 8192,
         "out": "bf16", "act": "gelu_tanh"},
    ]


def _log(rng, lo, hi):
    """A whole number spread evenly over its logarithm, lo..hi; about a third are multiples of 16."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v > 16 and rng.random() < 1 / 3:
        v -= v % 16
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["quantize", "decode", "matmul", "gated", "train", "gated8"])
    act = rng.choice(["silu", "gelu", "gelu_tanh", "relu"])
    if op == "quantize":
        return {"op": op, "M": _log(rng, 1, 4096), "K": _log(rng, 16, 8192),
                "dtype": rng.choice(["f16", "bf16", "f32"])}
    if op == "decode":
        L, layout = rng.choice([8, 12, 16]), rng.choice([0, 1])
        if rng.random() < 0.5:
            r, c = _log(rng, 1, 512), _log(rng, 1, 512)
            return {"op": op, "L": L, "layout": layout, "tiles": True, "rows": 16 * r, "cols": 16 * c,
                    "n": r * c, "T": 256}
        # a tail-biting stream holds whole words
        T = 16 * rng.randint(1, 16) if layout == 0 else rng.randint(1, 256)
        return {"op": op, "L": L, "layout": layout, "tiles": False, "rows": 0, "cols": 0,
                "n": _log(rng, 1, 65536), "T": T}
    if op == "matmul":
        return {"op": op, "M": _log(rng, 1, 3001), "N": _log(rng, 16, 8192), "K": _log(rng, 16, 8192),
                "out": rng.choice(["f16", "bf16", "f32"]), "bias": rng.random() < 0.5}
    if op == "gated8":
        return {"op": op, "M": _log(rng, 1, 2048), "K": _log(rng, 16, 2048), "F": _log(rng, 16, 8192),
                "out": rng.choice(["f16", "bf16", "f32"]), "act": act}
    least = 128 if op == "train" else 16          # a training step has more than a handful of tokens
    return {"op": op, "M": _log(rng, least if op == "train" else 1, 3001), "K": _log(rng, least, 2048),
            "F": _log(rng, least, 8192), "dtype": rng.choice(["f16", "bf16"]), "act": act}


def _words(case):
    kT = 2 * case["T"]
    return kT // 32 if case["layout"] == 0 else (kT + case["L"] - 2 + 31) // 32


def _int8_rows(g, rows, cols):
    """int8 rows as a row quantiser leaves them: near Gaussian, every row's largest at 127."""
    q = torch.randn(rows, cols, device="cuda", generator=g).mul_(32).round_().clamp_(-127, 127).to(torch.int8)
    q[torch.arange(rows, device="cuda"),
      torch.randint(0, cols, (rows,), device="cuda", generator=g)] = 127
    return q


def _scales(g, n, centre):
    return torch.exp(torch.randn(n, device="cuda", generator=g) * 0.3) * centre


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if op == "quantize":
        M, K = case["M"], case["K"]
        x = torch.randn(M, K, device="cuda", generator=g)
        # activations have a few channels far larger than the rest, and rows of very different size
        x[:, torch.randint(0, K, (max(1, K // 256),), device="cuda", generator=g)] *= 20
        x *= _scales(g, M, 1.0)[:, None]
        s["x"] = x.to(DTYPES[case["dtype"]])
    elif op == "decode":
        s["bits"] = torch.randint(-2 ** 31, 2 ** 31, (case["n"], _words(case)), device="cuda",
                                  generator=g).to(torch.int32).view(torch.uint32)
    elif op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        s["a"], s["w"] = _int8_rows(g, M, K), _int8_rows(g, N, K)
        s["a_scale"], s["w_scale"] = _scales(g, M, 1 / 32), _scales(g, N, 1 / (32 * math.sqrt(K)))
        s["bias"] = torch.randn(N, device="cuda", generator=g) if case["bias"] else None
    elif op == "gated8":
        M, K, F = case["M"], case["K"], case["F"]
        s["a"], s["wg"], s["wu"] = _int8_rows(g, M, K), _int8_rows(g, F, K), _int8_rows(g, F, K)
        s["a_scale"] = _scales(g, M, 1 / 32)
        s["wg_scale"], s["wu_scale"] = (_scales(g, F, 1 / (32 * math.sqrt(K))) for _ in range(2))
    else:
        M, K, F = case["M"], case["K"], case["F"]
        dt = DTYPES[case["dtype"]]
        s["x"] = torch.randn(M, K, device="cuda", generator=g).to(dt)
        s["wg"], s["wu"] = (torch.randn(F, K, device="cuda", generator=g).div_(math.sqrt(K)).to(dt)
                            for _ in range(2))
        if op == "train":
            s["grad"] = torch.randn(M, F, device="cuda", generator=g).mul_(0.1).to(dt)
    return s


# ---------------------------------------------------------------- plain forms

def _act(v, act):
    """The activation and its derivative."""
    if act == "silu":
        p = 1 / (1 + torch.exp(-v))
        return v * p, p * (1 + v * (1 - p))
    if act == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v)), (v > 0).to(v.dtype)
    if act == "gelu":
        c = 0.5 * (1 + torch.erf(v * math.sqrt(0.5)))
        return v * c, c + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)
    a, b = math.sqrt(2 / math.pi), 0.044715
    t = torch.tanh(a * (v + b * v ** 3))
    return 0.5 * v * (1 + t), 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * a * (1 + 3 * b * v * v)


def _plain_quantize(x):
    # the division in 64 bits: next to a border between two integers, 32 lose the side
    amax = x.float().abs().amax(dim=1)
    scale = (amax.double() / 127).float()
    by = torch.where(scale > 0, scale, torch.ones_like(scale)).double()
    return torch.round(x.double() / by[:, None]).to(torch.int8), scale


def _plain_decode(case, bits):
    T, L, W = case["T"], case["L"], bits.shape[1]
    w = bits.view(torch.int32).to(torch.int64) & 0xFFFFFFFF
    t = 2 * torch.arange(T, device=bits.device)
    hi = w[:, t // 32]
    nxt = t // 32 + 1
    lo = w[:, nxt % W] if case["layout"] == 0 else w[:, nxt.clamp(max=W - 1)] * (nxt < W)
    x = ((hi << 32 | lo) >> (64 - L - t % 32)) & ((1 << L) - 1)
    x = (x * LCG_MUL + LCG_ADD) & 0xFFFFFFFF
    k = (x & 255) + (x >> 8 & 255) + (x >> 16 & 255) + (x >> 24) - 510
    q = torch.round(k.float() / 4).to(torch.int8)          # ties to the even integer
    if case["tiles"]:
        r, c = case["rows"] // 16, case["cols"] // 16
        q = q.view(r, c, 16, 16).permute(0, 2, 1, 3).reshape(case["rows"], case["cols"])
    return q


def _plain_product8(a, a_scale, w, w_scale):
    # sums of whole numbers that pass 2^24: 64 bits keep them whole
    return (a.double() @ w.double().t()) * a_scale.double()[:, None] * w_scale.double()


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        import trellis_coded_weight_bitshift_b200 as tcq
        act = {"silu": tcq.ACT_SILU, "gelu": tcq.ACT_GELU, "gelu_tanh": tcq.ACT_GELU_TANH,
               "relu": tcq.ACT_RELU}.get(case.get("act"))
        if op == "quantize":
            return tcq.quantize_int8(s["x"])
        if op == "decode":
            return tcq.decode_int8(s["bits"], case["L"], case["T"], case["layout"],
                                   tcq.OUT_TILE16 if case["tiles"] else tcq.OUT_SEQ, case["rows"],
                                   case["cols"])
        if op == "matmul":
            return tcq.int8_matmul(s["a"], s["a_scale"], s["w"], s["w_scale"], bias=s["bias"],
                                   out_dtype=DTYPES[case["out"]])
        if op == "gated8":
            return tcq.int8_gated_ffn(s["a"], s["a_scale"], s["wg"], s["wg_scale"], s["wu"],
                                      s["wu_scale"], act=act, out_dtype=DTYPES[case["out"]])
        if op == "gated":
            return tcq.gated_ffn(s["x"], s["wg"], s["wu"], act=act)
        leaves = [s[k].detach().requires_grad_() for k in ("x", "wg", "wu")]
        h = tcq.GatedFfn.apply(*leaves, act)
        return (h.detach(), *torch.autograd.grad(h, leaves, s["grad"]))
    if op == "quantize":
        return _plain_quantize(s["x"])
    if op == "decode":
        return _plain_decode(case, s["bits"])
    if op == "matmul":
        y = _plain_product8(s["a"], s["a_scale"], s["w"], s["w_scale"])
        return (y if s["bias"] is None else y + s["bias"].double()).to(DTYPES[case["out"]])
    if op == "gated8":
        gate = _plain_product8(s["a"], s["a_scale"], s["wg"], s["wg_scale"]).float()
        up = _plain_product8(s["a"], s["a_scale"], s["wu"], s["wu_scale"]).float()
        return (_act(gate, case["act"])[0] * up).to(DTYPES[case["out"]])
    x, wg, wu = s["x"].float(), s["wg"].float(), s["wu"].float()
    gate, up = x @ wg.t(), x @ wu.t()
    a, da = _act(gate, case["act"])
    h = (a * up).to(s["x"].dtype)
    if op == "gated":
        return h
    grad = s["grad"].float()
    dgate, dup = grad * up * da, grad * a
    return (h, (dgate @ wg + dup @ wu).to(h.dtype), (dgate.t() @ x).to(h.dtype), (dup.t() @ x).to(h.dtype))


def work(case):
    op = case["op"]
    size = {"f16": 2, "bf16": 2, "f32": 4}
    if op == "quantize":
        M, K = case["M"], case["K"]
        return {"bytes": M * K * (size[case["dtype"]] + 1) + 4 * M, "flops": 2 * M * K}
    if op == "decode":
        return {"bytes": case["n"] * (4 * _words(case) + case["T"]), "flops": 0}
    if op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K + N * K + 4 * (M + N + N * case["bias"]) + M * N * size[case["out"]],
                "flops": 2 * M * N * K}
    M, K, F = case["M"], case["K"], case["F"]
    if op == "gated8":
        return {"bytes": M * K + 2 * F * K + 4 * (M + 2 * F) + M * F * size[case["out"]],
                "flops": 4 * M * F * K}
    if op == "gated":
        return {"bytes": 2 * (M * K + 2 * F * K + M * F), "flops": 4 * M * F * K}
    # inputs, the output and its gradient, three gradients; forward, then twice the products
    return {"bytes": 2 * (2 * M * K + 4 * F * K + 2 * M * F), "flops": 12 * M * F * K}


# ------------------------------------------------------- the definition, 64 bits

def _exact_decode(case, bits):
    """By bytes: the window of weight t lies in the three bytes from byte t / 4 on."""
    n, L, T = bits.shape[0], case["L"], case["T"]
    table = [sum(((i * LCG_MUL + LCG_ADD) & 0xFFFFFFFF).to_bytes(4, "little")) - 510 for i in range(1 << L)]
    table = torch.tensor([(k // 4) + ((k % 4 == 3) or (k % 4 == 2 and (k // 4) % 2 == 1)) for k in table],
                         dtype=torch.int8, device=bits.device)
    by = bits.view(torch.uint8).view(n, -1, 4).flip(2).reshape(n, -1)          # most significant byte first
    by = torch.cat([by, by[:, :3] if case["layout"] == 0 else torch.zeros_like(by[:, :1]).expand(n, 3)], 1).int()
    t = torch.arange(T, device=bits.device)
    three = by[:, t // 4] * 65536 + by[:, t // 4 + 1] * 256 + by[:, t // 4 + 2]
    q = table[(three.bitwise_right_shift(24 - L - 2 * (t % 4)) & ((1 << L) - 1)).long()]
    if case["tiles"]:
        q = q.view(-1, case["cols"] // 16, 16, 16).transpose(1, 2).reshape(case["rows"], case["cols"])
    return q


def _exact_gate(v, act):
    """Value and slope of the activation, by torch's own 64-bit functions and closed forms of the slopes."""
    if act == "silu":
        p = torch.sigmoid(v)
        return v * p, p + v * p * torch.sigmoid(-v)
    if act == "relu":
        return v.clamp(min=0), torch.heaviside(v, torch.zeros((), dtype=v.dtype, device=v.device))
    if act == "gelu":
        p = 0.5 * torch.special.erfc(-v / math.sqrt(2))
        return v * p, p + v * torch.exp(v.square() / -2) * (0.5 * math.sqrt(2 / math.pi))
    # (1 + tanh z) / 2 is the logistic function of 2 z
    k = 2 * math.sqrt(2 / math.pi)
    p = torch.sigmoid(k * v * (1 + 0.044715 * v.square()))
    return v * p, p + v * p * (1 - p) * k * (1 + 0.134145 * v.square())


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = s["x"].double()
        scale = (x.abs().max(dim=1, keepdim=True).values / 127).float().double()   # the scale is kept in fp32
        y = x / torch.where(scale > 0, scale, 1.0)
        low = torch.floor(y)
        up = (y - low > 0.5) | ((y - low == 0.5) & (low % 2 == 1))
        return (low + up).to(torch.int8), scale[:, 0]
    if op == "decode":
        return _exact_decode(case, s["bits"])
    if op in ("matmul", "gated8"):
        a = s["a"].double() * s["a_scale"].double()[:, None]
        if op == "matmul":
            y = a @ (s["w"].double() * s["w_scale"].double()[:, None]).t()
            return y if s["bias"] is None else y + s["bias"].double()
        gate, up = (a @ (s[k].double() * s[k + "_scale"].double()[:, None]).t() for k in ("wg", "wu"))
        return _exact_gate(gate, case["act"])[0] * up
    x, wg, wu = (s[k].double() for k in ("x", "wg", "wu"))
    gate, up = torch.matmul(x, wg.mT), torch.matmul(x, wu.mT)
    value, slope = _exact_gate(gate, case["act"])
    if op == "gated":
        return value * up
    grad = s["grad"].double()
    dgate, dup = grad * slope * up, grad * value
    return (value * up, torch.cat([dgate, dup], 1) @ torch.cat([wg, wu], 0), torch.matmul(dgate.mT, x),
            torch.matmul(dup.mT, x))
