"""Cases of the products with GPTQ-packed layers that carry their epilogue.

Two operators, each in three forms:

* linear  Y = act(X W^T + bias) + residual, one packed layer W;
* gated   Y = act(X Wg^T) * (X Wu^T), two packed layers that share their input
  (and so their act-order permutation), the first half of a gated
  feed-forward block.

The forms are "decode" (a few tokens; the weight is s (q - z) in fp32), "many"
(the tensor cores; the weight is the 16-bit value bf16(s (q - z)), which the
packed layer stands for there, as in gptq_dequant_gemm) and "backward" (the
gradients of the "many" form for given dY and saved pre-activations, with the
same 16-bit weight).

A packed layer holds `bits`-bit codes q as each row's little-endian bit stream
in quantization order: position k belongs to input column perm[k] and to group
k // g, whose scale s and zero point z are stored group-major.
"""
import math

import torch

own = False

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


# ------------------------------------------------------------------- cases
def listed():
    def case(name, op, form, n, d_col, d_row, bits, g, perm, act, extras=False):
        return {"name": name, "op": op, "form": form, "n": n, "d_col": d_col, "d_row": d_row, "bits": bits,
                "g": g, "perm": perm, "act": act, "extras": extras}

    return [
        # one generated token through an attention output projection, added to the residual stream
        case("decode o_proj 1 token", "linear", "decode", 1, 4096, 4096, 4, 128, False, "none", True),
        # eight sequences decoded together through the largest layer, act-order
        case("decode down_proj 8 tokens", "linear", "decode", 8, 28672, 8192, 4, 128, True, "none", True),
        # one token through the first half of a 3-bit feed-forward block
        case("decode ffn 3-bit 1 token", "gated", "decode", 1, 4096, 11008, 3, 128, False, "silu"),
        # a batch of 32 sequences decoded together, the larger block, act-order
        case("decode ffn 32 tokens", "gated", "decode", 32, 8192, 28672, 4, 128, True, "silu"),
        # a ragged prompt through a fine-grained act-order down projection, added to the residual stream
        case("prompt down_proj g32 500", "linear", "many", 500, 11008, 4096, 4, 32, True, "none", True),
        # a batch of prompts through a projection with bias and activation (plain feed-forward blocks)
        case("prompt fc 4096 tokens", "linear", "many", 4096, 8192, 8192, 4, 128, False, "gelu_tanh", True),
        # a training step's forward pass: the projections' outputs are kept for the backward pass
        case("train ffn 2048 tokens", "gated", "many", 2048, 4096, 11008, 4, 128, False, "silu", True),
        # a short ragged prompt through a 3-bit block
        case("prompt ffn 3-bit 77", "gated", "many", 77, 4096, 11008, 3, 128, False, "silu"),
        # the gradient of an act-order down projection (fine-tuning next to frozen packed weights)
        case("backward down_proj 2048", "linear", "backward", 2048, 11008, 4096, 4, 32, True, "none"),
        # the gradients of an 8-bit layer with bias and activation, ragged tokens
        case("backward fc 8-bit 333", "linear", "backward", 333, 4096, 4096, 8, 128, False, "gelu", True),
        # the gradients of a feed-forward block's first half
        case("backward ffn 2048", "gated", "backward", 2048, 4096, 11008, 4, 128, False, "silu"),
        # the same at two bits with act-order and a short ragged batch
        case("backward ffn 2-bit 150", "gated", "backward", 150, 4096, 11008, 2, 64, True, "gelu_tanh"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "gated"))
    form = rng.choice(("decode", "many", "backward"))
    bits = rng.choice((4, 4, 4, 2, 3, 8))
    unit = 128 if bits == 3 else 64
    d_col = unit * _log(rng, 256 // unit, 16384 // unit)
    d_row = _log(rng, 100, 16384)
    n = _log(rng, 1, 32) if form == "decode" else _log(rng, 17, 3000)
    # no more work than the largest listed case
    while 2 * n * d_col * d_row * (2 if op == "gated" else 1) > 4e11 and n > 17:
        n = n // 2 + 1
    g = rng.choice((128, 128, 128, 128, 64, 32, 16, 8, 256, 1024, -1))
    act = rng.choice(ACTS)
    return {"op": op, "form": form, "n": n, "d_col": d_col, "d_row": d_row, "bits": bits, "g": g,
            "perm": rng.random() < 0.5, "act": act, "extras": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs
def _groups(c):
    g = c["d_col"] if c["g"] == -1 or c["g"] > c["d_col"] else c["g"]
    return g, -(-c["d_col"] // g)


def _pack(codes, bits):
    """uint8 codes (rows x d, d a multiple of 32) -> int32 words, each row's little-endian bit stream."""
    at = torch.arange(32, device=codes.device)
    if 32 % bits == 0:
        per = 32 // bits
        w = (codes.view(codes.shape[0], -1, per).long() << (bits * at[:per])).sum(-1)
    else:
        b = (codes.view(codes.shape[0], -1, 32, 1) >> torch.arange(bits, device=codes.device, dtype=torch.uint8)) & 1
        w = (b.view(codes.shape[0], -1, 32).long() << at).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).int()


def _layer(c, gen, dev):
    """A layer as the quantizer leaves it: Gaussian weights of 0.02, each group's range cut into 2^bits levels."""
    rows, d, top = c["d_row"], c["d_col"], 2 ** c["bits"] - 1
    _, ng = _groups(c)
    mid, std = top / 2, top / 5.4
    codes = torch.randn(rows, d, generator=gen, device=dev).mul_(std).add_(mid).round_().clamp_(0, top).to(torch.uint8)
    scales = 0.02 * 5.4 / top * (1 + 0.15 * torch.randn(ng, rows, generator=gen, device=dev)).clamp_(0.5, 2.0)
    zeros = (mid + 0.06 * top * torch.randn(ng, rows, generator=gen, device=dev)).round_().clamp_(0, top).int()
    return _pack(codes, c["bits"]), scales, zeros


def _activations(n, d, gen, dev):
    """Heavy-tailed activations (Student-t, 4 degrees of freedom) with a few outlier channels."""
    u = 1.0 - torch.rand(2, n, d, generator=gen, device=dev)
    x = torch.randn(n, d, generator=gen, device=dev) / torch.sqrt(-0.5 * torch.log(u[0] * u[1]))
    x[:, torch.randperm(d, generator=gen, device=dev)[:max(1, d // 200)]] *= 10.0
    return x.bfloat16()


def prepare(case, seed):
    c = dict(case)
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 1000003 + 17)
    n, d, r = c["n"], c["d_col"], c["d_row"]
    s = {"case": c, "layers": [_layer(c, gen, dev) for _ in range(2 if c["op"] == "gated" else 1)],
         "perm": torch.randperm(d, generator=gen, device=dev).int() if c["perm"] else None}
    bf = dict(dtype=torch.bfloat16, device=dev)

    def normal(std, *shape):
        return (torch.randn(*shape, generator=gen, device=dev) * std).bfloat16()

    if c["form"] != "backward":
        s["X"] = _activations(n, d, gen, dev)
        s["Y"] = torch.empty(n, r, **bf)
        if c["op"] == "linear":
            s["bias"] = 0.3 * torch.randn(r, generator=gen, device=dev) if c["extras"] else None
            s["residual"] = normal(1.0, n, r) if c["extras"] else None
        elif c["extras"] and c["form"] == "many":
            s["gate"], s["up"] = torch.empty(n, r, **bf), torch.empty(n, r, **bf)
    else:
        s["dY"] = normal(1e-2, n, r)
        s["dX"] = torch.empty(n, d, **bf)
        # gradients of the products that the tensor memory accelerator reads: rows of whole 16 bytes
        ld = -(-r // 8) * 8
        if c["op"] == "linear":
            plain = c["act"] == "none"
            s["pre"] = None if plain else normal(1.5, n, r)
            s["dPre"] = None if plain and r % 8 == 0 else torch.empty(n, ld, **bf)[:, :r]
            s["dbias"] = torch.empty(r, device=dev) if c["extras"] else None
        else:
            s["gate"], s["up"] = normal(1.5, n, r), normal(1.5, n, r)
            s["dGate"], s["dUp"] = torch.empty(n, ld, **bf)[:, :r], torch.empty(n, ld, **bf)[:, :r]
    s["st"] = torch.zeros(1, dtype=torch.int32, device=dev)
    # more than any of the calls asks for (the *_workspace_size functions say how much that is)
    s["ws"] = torch.empty(2 * n * (d + 2 * r) + (64 << 20), dtype=torch.uint8, device=dev)
    return s


# -------------------------------------------------------------- plain form
def _weights(c, layer, rounded):
    """W_hat (d_row x d_col, fp32) in quantization order."""
    packed, scales, zeros = layer
    d, bits = c["d_col"], c["bits"]
    g, ng = _groups(c)
    if 32 % bits == 0:
        at = bits * torch.arange(32 // bits, device=packed.device, dtype=torch.int32)
        q = ((packed.unsqueeze(-1) >> at) & (2 ** bits - 1)).view(-1, d)
    else:
        k = torch.arange(32, device=packed.device) * bits
        w = packed.view(packed.shape[0], -1, bits).long() & 0xFFFFFFFF
        w = torch.cat((w, torch.zeros_like(w[..., :1])), -1)
        q = (((w[..., k >> 5] | (w[..., (k >> 5) + 1] << 32)) >> (k & 31)) & (2 ** bits - 1)).view(-1, d)
    s, z = (t.t().repeat_interleave(g, 1)[:, :d] for t in (scales, zeros))
    w = s * (q - z).float()
    # the 16-bit weight that the packed layer stands for in the tensor-core forms
    return w.bfloat16().float() if rounded else w


def _act(x, act):
    if act == "relu":
        return x.clamp(min=0)
    if act == "gelu":
        return 0.5 * x * (1 + torch.erf(x * 0.7071067811865476))
    if act == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(0.7978845608028654 * (x + 0.044715 * x * x * x)))
    if act == "silu":
        return x / (1 + torch.exp(-x))
    return x


def _act_slope(x, act):
    if act == "relu":
        return (x > 0).to(x.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(x * 0.7071067811865476)) + x * 0.3989422804014327 * torch.exp(-0.5 * x * x)
    if act == "gelu_tanh":
        t = torch.tanh(0.7978845608028654 * (x + 0.044715 * x * x * x))
        return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * 0.7978845608028654 * (1 + 0.134145 * x * x)
    if act == "silu":
        s = 1 / (1 + torch.exp(-x))
        return s * (1 + x * (1 - s))
    return torch.ones_like(x)


def _plain(s):
    c = s["case"]
    W = [_weights(c, layer, c["form"] != "decode") for layer in s["layers"]]
    if c["form"] != "backward":
        X = s["X"].float()
        if s["perm"] is not None:
            X = X[:, s["perm"].long()]
        P = [X @ w.t() for w in W]
        if c["op"] == "linear":
            y = _act(P[0] + s["bias"] if s["bias"] is not None else P[0], c["act"])
            return {"Y": (y + s["residual"].float() if s["residual"] is not None else y).bfloat16()}
        out = {"Y": (_act(P[0], c["act"]) * P[1]).bfloat16()}
        if "gate" in s:
            out["gate"], out["up"] = P[0].bfloat16(), P[1].bfloat16()
        return out
    dY = s["dY"].float()
    out = {}
    if c["op"] == "linear":
        D = [dY if s["pre"] is None else dY * _act_slope(s["pre"].float(), c["act"])]
        if s["dPre"] is not None:
            out["dPre"] = D[0].bfloat16()
        if s["dbias"] is not None:
            out["dbias"] = D[0].sum(0)
    else:
        g, u = s["gate"].float(), s["up"].float()
        D = [dY * u * _act_slope(g, c["act"]), dY * _act(g, c["act"])]
        out["dGate"], out["dUp"] = D[0].bfloat16(), D[1].bfloat16()
    dX = D[0] @ W[0]
    if len(W) > 1:
        dX += D[1] @ W[1]
    if s["perm"] is not None:
        dX = dX[:, torch.argsort(s["perm"])]
    out["dX"] = dX.bfloat16()
    return out


# ------------------------------------------------------------------- calls
def _own(s):
    import post_weight_quantization_gptq_b200 as q
    c = s["case"]
    layers = [t for layer in s["layers"] for t in layer] + [s["perm"], c["bits"], c["g"]]
    if c["form"] == "decode" and c["op"] == "linear":
        q.gptq_dequant_matmul_linear(s["X"], *layers, s["Y"], s["ws"], bias=s["bias"], activation=c["act"], residual=s["residual"])
        return {"Y": s["Y"]}
    if c["form"] == "decode":
        q.gptq_dequant_matmul_gated(s["X"], *layers, c["act"], s["Y"], s["ws"])
        return {"Y": s["Y"]}
    if c["form"] == "many" and c["op"] == "linear":
        q.gptq_dequant_gemm_linear(s["X"], *layers, s["Y"], s["ws"], bias=s["bias"], activation=c["act"], residual=s["residual"], dev_status=s["st"])
        return {"Y": s["Y"]}
    if c["form"] == "many":
        q.gptq_dequant_gemm_gated(s["X"], *layers, c["act"], s["Y"], s["ws"], gate=s.get("gate"), up=s.get("up"), dev_status=s["st"])
        return {k: s[k] for k in ("Y", "gate", "up") if k in s}
    if c["op"] == "linear":
        q.gptq_dequant_gemm_linear_backward(s["dY"], *layers, s["dX"], s["ws"], activation=c["act"], pre=s["pre"], dPre=s["dPre"], dbias=s["dbias"], dev_status=s["st"])
        return {k: s[k] for k in ("dX", "dPre", "dbias") if s[k] is not None}
    q.gptq_dequant_gemm_gated_backward(s["dY"], s["gate"], s["up"], *layers, c["act"], s["dGate"], s["dUp"], s["dX"], s["ws"], dev_status=s["st"])
    return {k: s[k] for k in ("dX", "dGate", "dUp")}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    c = case
    n, d, r = c["n"], c["d_col"], c["d_row"]
    _, ng = _groups(c)
    mats = 2 if c["op"] == "gated" else 1
    size = mats * (r * d * c["bits"] / 8 + ng * r * 8) + (4 * d if c["perm"] else 0)
    if c["form"] != "backward":
        size += 2 * n * (d + r)
        if c["extras"]:
            size += 2 * n * r + 4 * r if c["op"] == "linear" else 4 * n * r if c["form"] == "many" else 0
    elif c["op"] == "gated":
        size += 2 * n * (5 * r + d)
    else:
        wide = c["act"] == "none"
        size += 2 * n * (r + d) + (0 if wide and r % 8 == 0 else 2 * n * r) + (0 if wide else 2 * n * r) + (4 * r if c["extras"] else 0)
    return {"bytes": size, "flops": 2 * mats * n * d * r}


# ------------------------------------------------------------------- exact
def _exact_weights(c, layer):
    """The definition's weights in float64, in quantization order; bits are read one by one."""
    packed, scales, zeros = layer
    d, bits = c["d_col"], c["bits"]
    k = torch.arange(d, device=packed.device)
    group = k // _groups(c)[0]
    q = torch.zeros(packed.shape[0], d, dtype=torch.int32, device=packed.device)
    for b in range(bits):
        place = k * bits + b
        q += ((packed[:, place // 32] >> (place % 32).int()) & 1) << b
    q -= zeros.t()[:, group]
    s = scales.t()[:, group]
    if c["form"] == "decode":
        return s.double() * q.double()
    # the weight is a 16-bit number: one fp32 product, rounded to bf16
    return torch.mul(s, q.to(torch.float32)).to(torch.bfloat16).double()


def _exact_act(x, act):
    """(act(x), act'(x)) in float64."""
    if act == "none":
        return x, torch.ones_like(x)
    if act == "relu":
        return torch.where(x > 0, x, 0.0), torch.where(x > 0, 1.0, 0.0).double()
    if act == "silu":
        s = torch.where(x >= 0, 1 / (1 + torch.exp(-x.abs())), torch.exp(-x.abs()) / (1 + torch.exp(-x.abs())))
        return x * s, s + x * s * (1 - s)
    if act == "gelu":
        cdf = 0.5 * torch.special.erfc(-x / math.sqrt(2.0))
        return x * cdf, cdf + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    inner = math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)
    half = 1 / (1 + torch.exp(-2 * inner))  # (1 + tanh(inner)) / 2
    return x * half, half + 2 * x * half * (1 - half) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * x ** 2)


def exact(case, seed):
    c = dict(case)
    s = prepare(case, seed)
    order = s["perm"].long() if s["perm"] is not None else None
    mats = []
    for layer in s["layers"]:
        w = _exact_weights(c, layer)
        if order is not None:
            full = torch.empty_like(w)
            full[:, order] = w
            w = full
        mats.append(w)
    if c["form"] != "backward":
        sums = [s["X"].double() @ w.T for w in mats]
        if c["op"] == "linear":
            if s["bias"] is not None:
                sums[0] = sums[0] + s["bias"].double()
            y = _exact_act(sums[0], c["act"])[0]
            return {"Y": y if s["residual"] is None else y + s["residual"].double()}
        found = {"Y": _exact_act(sums[0], c["act"])[0] * sums[1]}
        if "gate" in s:
            found.update(gate=sums[0], up=sums[1])
        return found
    dY = s["dY"].double()
    if c["op"] == "linear":
        d = dY if s["pre"] is None else dY * _exact_act(s["pre"].double(), c["act"])[1]
        found = {"dX": d @ mats[0]}
        if s["dPre"] is not None:
            found["dPre"] = d
        if s["dbias"] is not None:
            found["dbias"] = d.sum(0)
        return found
    value, slope = _exact_act(s["gate"].double(), c["act"])
    d_gate, d_up = dY * s["up"].double() * slope, dY * value
    return {"dX": d_gate @ mats[0] + d_up @ mats[1], "dGate": d_gate, "dUp": d_up}
