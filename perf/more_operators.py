"""The gated feed-forward block of the experts, its backward pass, and the clipping of the gradients that it leaves, as cases
that can be timed and compared.

Four operators, each reached through the package's public calls:

* gated -- ``grouped_gated_mm``: both projections of block-quantized rows with block-quantized stacked weights (E, 2, N, K),
  the activation of the first and the product with the second, one expert per token group: bf16 rows, e4m3 rows with one
  scale per 1x128 block for the next product, or both, and for training the two projections as well;
* backward -- ``gated_backward``: the gradients of the two projections from the gradient of their gated product, in the
  rows' own type, quantized per 1x128 block, or both;
* grad -- ``grouped_gated_grad``: grad_input, the sum of the two projections' products with their transposed weights;
* clip -- ``grad_norm`` (the norm over all of a list of tensors) and ``clip_grads`` (the tensors scaled to a largest norm).

The activations are x * sigmoid(z): z = x (silu), or z = 2 sqrt(2 / pi) (x + 0.044715 x^3) (gelu, the tanh form).  The
stored scale is the multiplier 448 / max(amax, 1e-12); the quantized value divided by it is the value it stands for.  With
``own`` false, ``run`` computes the same in elementary torch operations in 32 bits, rounded once at the end.
"""
import math
import random

import torch

own = False

BLOCK = 128
E4M3 = torch.float8_e4m3fn
GELU_A = 2.0 * math.sqrt(2.0 / math.pi)
GELU_B = GELU_A * 0.044715


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one token of a decoding step: the weights of eight experts are read for one row each
        {"name": "gated one token", "op": "gated", "tokens": 1, "top_k": 8, "experts": 64, "local": 64, "n": 2048, "k": 4096,
         "activation": "silu", "form": "fp8", "keep": False},
        # a decoding batch: every expert's weights for a handful of rows, ragged N and K
        {"name": "gated decode batch", "op": "gated", "tokens": 64, "top_k": 8, "experts": 64, "local": 64, "n": 1424,
         "k": 2064, "activation": "gelu", "form": "bf16", "keep": False},
        # prefill where this GPU holds 40 of 160 experts: rows behind the last group stay as they are
        {"name": "gated prefill local experts", "op": "gated", "tokens": 16381, "top_k": 6, "experts": 160, "local": 40,
         "n": 1360, "k": 2064, "activation": "silu", "form": "fp8", "keep": False},
        # the benchmark's training shape: 16640 tokens in 16 groups; the projections are kept for the backward pass, the
        # bf16 rows for the weight gradient of the second layer, the quantized ones for its product
        {"name": "gated training", "op": "gated", "tokens": 16640, "top_k": 1, "experts": 16, "local": 16, "n": 4096,
         "k": 4096, "activation": "silu", "form": "both", "keep": True},
        # fp32 activations of a small odd batch
        {"name": "backward fp32 odd", "op": "backward", "rows": 513, "n": 1040, "activation": "gelu", "dtype": "fp32",
         "form": "both"},
        # the training shape: bf16 for the weight gradients, quantized for grad_input
        {"name": "backward training", "op": "backward", "rows": 16640, "n": 4096, "activation": "silu", "dtype": "bf16",
         "form": "both"},
        # a small uneven layer of which this GPU holds 9 of 24 experts, ragged N and K
        {"name": "grad local experts odd", "op": "grad", "tokens": 2047, "top_k": 3, "experts": 24, "local": 9, "n": 1040,
         "k": 1360},
        # grad_input of the training shape
        {"name": "grad training", "op": "grad", "tokens": 16640, "top_k": 1, "experts": 16, "local": 16, "n": 4096, "k": 4096},
        # a router's weight and two vectors: latency
        {"name": "clip three small", "op": "clip", "kind": "many", "count": 3, "most": 60000, "sizes": 3, "write": True},
        # the norms, biases and small matrices of a whole model, both types, odd sizes and addresses: the norm for the log
        {"name": "norm many small", "op": "clip", "kind": "many", "count": 400, "most": 200000, "sizes": 5, "write": False},
        # the gradients of the training shape's layer
        {"name": "clip training", "op": "clip", "kind": "layer", "experts": 16, "n": 4096, "k": 4096, "dtype": "bf16",
         "write": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _wide(rng, lo, hi):
    return max(lo, _log(rng, lo, hi) // 16 * 16)


def draw(rng):
    op = rng.choice(["gated", "gated", "backward", "grad", "clip"])
    if op in ("gated", "grad"):
        top_k = rng.randint(1, 10)
        experts = _log(rng, max(top_k, 2), 128)
        local = experts if rng.random() < 0.6 else rng.randint(1, experts)
        n, k = _wide(rng, 64, 8192), _wide(rng, 64, 8192)
        while local * n * k > 16 * 4096 * 4096:
            n, k = max(64, n // 32 * 16), max(64, k // 32 * 16)
        tokens = min(_log(rng, 1, 16384), max(1, (16640 * 4096 * 4096) // (top_k * n * k)),
                     max(1, (4 * 16640 * 4096) // (top_k * max(n, k))))
        case = {"op": op, "tokens": tokens, "top_k": top_k, "experts": experts, "local": local, "n": n, "k": k}
        if op == "gated":
            case.update(activation=rng.choice(["silu", "gelu"]), form=rng.choice(["bf16", "fp8", "both"]),
                        keep=rng.random() < 0.4)
        return case
    if op == "backward":
        n, dtype = _wide(rng, 64, 16384), rng.choice(["bf16", "bf16", "fp32"])
        rows = min(_log(rng, 1, 65536), (16640 * 4096) // (n * (2 if dtype == "fp32" else 1)))
        return {"op": op, "rows": rows, "n": n, "activation": rng.choice(["silu", "gelu"]), "dtype": dtype,
                "form": rng.choice(["bf16", "fp8", "both"])}
    if rng.random() < 0.5:
        return {"op": op, "kind": "many", "count": _log(rng, 1, 600), "most": _log(rng, 10, 300000),
                "sizes": rng.randint(0, 10 ** 6), "write": rng.random() < 0.6}
    dtype = rng.choice(["bf16", "fp32"])
    n, k = _wide(rng, 64, 8192), _wide(rng, 64, 8192)
    room = (16 * 4096 * 4096) // (n * k * (2 if dtype == "fp32" else 1))
    return {"op": op, "kind": "layer", "experts": max(1, min(_log(rng, 1, 128), room)), "n": n, "k": k, "dtype": dtype,
            "write": rng.random() < 0.6}


def _blocks(v):
    return -(-v // BLOCK)


def _sizes(case):
    """(elements, type) of every tensor of a clip case."""
    if case["kind"] == "layer":
        dtype, e, n, k = case["dtype"], case["experts"], case["n"], case["k"]
        return [(e * 2 * n * k, dtype), (e * k * n, dtype), (e * k, "fp32"), (k, "fp32")]
    r = random.Random(case["sizes"])
    return [(int(round(math.exp(r.uniform(0.0, math.log(case["most"]))))), r.choice(["bf16", "fp32"]))
            for _ in range(case["count"])]


def work(case):
    c = case
    if c["op"] == "clip":
        data = sum(n * (2 if t == "bf16" else 4) for n, t in _sizes(c))
        count = sum(n for n, _ in _sizes(c))
        return {"bytes": data * (2 if c["write"] else 1) + 4, "flops": count * (3 if c["write"] else 2)}
    if c["op"] == "backward":
        size = 2 if c["dtype"] == "bf16" else 4
        data = 3 * size + (2 * size if c["form"] != "fp8" else 0) + (2 * (1 + 4 / BLOCK) if c["form"] != "bf16" else 0)
        return {"bytes": c["rows"] * c["n"] * data, "flops": 20 * c["rows"] * c["n"]}
    n, k = c["n"], c["k"]
    touched = c["local"] * (1 - (1 - c["top_k"] / c["experts"]) ** c["tokens"])
    live = c["tokens"] * c["top_k"] * c["local"] / c["experts"]
    weights = touched * 2 * n * k * (1 + 4 / BLOCK ** 2) + 4 * c["local"]
    if c["op"] == "grad":
        return {"bytes": weights + live * (2 * n * (1 + 4 / BLOCK) + 2 * k), "flops": 4 * live * n * k}
    row = k * (1 + 4 / BLOCK) + (2 * n if c["form"] != "fp8" else 0) + (n * (1 + 4 / BLOCK) if c["form"] != "bf16" else 0)
    return {"bytes": weights + live * (row + (4 * n if c["keep"] else 0)), "flops": 4 * live * n * k}


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _activations(gen, rows, cols):
    """Rows of differing size with a few strong channels, as the residual stream of a trained model has."""
    channel = torch.exp(0.5 * torch.randn(cols, device="cuda", generator=gen))
    channel *= 1 + 15 * (torch.rand(cols, device="cuda", generator=gen) < 0.01)
    size = torch.exp(0.3 * torch.randn(rows, 1, device="cuda", generator=gen))
    return torch.randn(rows, cols, device="cuda", generator=gen) * channel * size


def _weights(gen, rows, cols):
    w = torch.empty(rows, cols, device="cuda").normal_(generator=gen)
    spread = torch.exp(0.4 * torch.randn(rows, 1, device="cuda", generator=gen))
    return w.mul_(spread).mul_(cols ** -0.5)


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _layer(c, gen):
    """Quantized weights of the experts held here, and the end offsets of their rows."""
    popular = 0.5 * torch.randn(c["experts"], device="cuda", generator=gen)
    logits = torch.randn(c["tokens"], c["experts"], device="cuda", generator=gen) + popular
    ids = torch.topk(logits, c["top_k"], dim=1).indices.reshape(-1)
    sizes = torch.zeros(c["experts"], dtype=torch.int64, device="cuda")
    sizes = sizes.scatter_add(0, ids, torch.ones_like(ids))[:c["local"]]
    n, k = c["n"], c["k"]
    qb = torch.empty(c["local"], 2, n, k, dtype=E4M3, device="cuda")
    sb = torch.empty(c["local"], 2, _blocks(n), _blocks(k), device="cuda")
    for e in range(c["local"]):
        for j in range(2):
            qb[e, j], sb[e, j] = _quantize_tiles(_weights(gen, n, k))
    return {"case": c, "qb": qb, "sb": sb, "offs": sizes.cumsum(0).to(torch.int32), "sizes": sizes.tolist()}


def prepare(case, seed):
    c = case
    gen = _gen(seed)
    if c["op"] == "backward":
        dtype = _dtype(c["dtype"])
        pre = 1.5 * torch.randn(c["rows"], 2, c["n"], device="cuda", generator=gen)
        pre *= torch.exp(0.3 * torch.randn(c["rows"], 1, 1, device="cuda", generator=gen))
        return {"case": c, "g": (1e-3 * _activations(gen, c["rows"], c["n"])).to(dtype), "pre": pre.to(dtype)}
    if c["op"] == "clip":
        sizes = _sizes(c)
        flat, out = {}, {}
        for t in ("bf16", "fp32"):
            total = sum(n for n, d in sizes if d == t)
            flat[t] = torch.empty(total, device="cuda").normal_(generator=gen).mul_(0.01).to(_dtype(t))
            out[t] = torch.zeros(total if c["write"] else 0, dtype=_dtype(t), device="cuda")
        at = {"bf16": 0, "fp32": 0}
        grads, outs = [], []
        for n, t in sizes:  # one behind the other, as views of a step's gradient buffer are
            grads.append(flat[t][at[t]:at[t] + n])
            outs.append(out[t][at[t]:at[t] + n])
            at[t] += n
        # a norm that most steps of this case exceed
        most = 0.005 * math.sqrt(sum(n for n, _ in sizes))
        return {"case": c, "grads": grads, "outs": outs, "flat": flat, "out": out, "most": most}
    state = _layer(c, gen)
    slots = c["tokens"] * c["top_k"]
    n, k, part = c["n"], c["k"], c["local"] < c["experts"]
    if c["op"] == "grad":
        d = 1e-3 * _activations(gen, slots * 2, n)
        qd, sd = _quantize_rows(d)
        state["qd"], state["sd"] = qd.view(slots, 2, n), sd.view(slots, 2, _blocks(n))
        # rows behind the last group are not written: the buffers that a program keeps hold zeros there
        state["out"] = torch.zeros(slots, k, dtype=torch.bfloat16, device="cuda") if part else None
        return state
    state["qa"], state["sa"] = _quantize_rows(_activations(gen, slots, k))
    state["out"] = state["q"] = state["scales"] = state["pre"] = None
    if part:
        if c["form"] != "fp8":
            state["out"] = torch.zeros(slots, n, dtype=torch.bfloat16, device="cuda")
        if c["form"] != "bf16":
            state["q"] = torch.zeros(slots, n, dtype=torch.uint8, device="cuda").view(E4M3)
            state["scales"] = torch.zeros(slots, _blocks(n), device="cuda")
        if c["keep"]:
            state["pre"] = torch.zeros(slots, 2, n, dtype=torch.bfloat16, device="cuda")
    return state


# ------------------------------------------------------------ plain forms --

def _quantize_rows(x):
    rows, cols = x.shape
    nb = _blocks(cols)
    b = torch.nn.functional.pad(x.float(), (0, nb * BLOCK - cols)).view(rows, nb, BLOCK)
    s = 448.0 / b.abs().amax(2).clamp_min(1e-12)
    q = (b * s[:, :, None]).clamp(-448.0, 448.0).view(rows, nb * BLOCK)[:, :cols]
    return q.to(E4M3), s


def _quantize_tiles(w):
    n, k = w.shape
    nb, kb = _blocks(n), _blocks(k)
    b = torch.nn.functional.pad(w, (0, kb * BLOCK - k, 0, nb * BLOCK - n)).view(nb, BLOCK, kb, BLOCK)
    s = 448.0 / b.abs().amax((1, 3)).clamp_min(1e-12)
    q = (b * s[:, None, :, None]).clamp(-448.0, 448.0).view(nb * BLOCK, kb * BLOCK)[:n, :k]
    return q.to(E4M3), s


def _values(q, s, rows_per_scale):
    """The values that block-quantized (..., rows, cols) data stands for, in 32 bits."""
    r = 1.0 / s
    if rows_per_scale > 1:
        r = r.repeat_interleave(rows_per_scale, -2)[..., : q.shape[-2], :]
    return q.float() * r.repeat_interleave(BLOCK, -1)[..., : q.shape[-1]]


def _sigmoid_of(x, activation):
    """sigmoid(z(x)) and dz/dx of the activation x * sigmoid(z(x))."""
    if activation == "silu":
        return 1.0 / (1.0 + torch.exp(-x)), torch.ones_like(x)
    x2 = x * x
    return 1.0 / (1.0 + torch.exp(-x * (GELU_A + GELU_B * x2))), GELU_A + 3.0 * GELU_B * x2


def _gated_plain(s):
    c = s["case"]
    a = _values(s["qa"], s["sa"], 1)
    pre = torch.zeros(a.shape[0], 2, c["n"], device="cuda")
    at = 0
    # a product per group: elementary torch has no form for groups of differing length
    for e, size in enumerate(s["sizes"]):
        if size:
            w = _values(s["qb"][e], s["sb"][e], BLOCK)
            pre[at:at + size] = torch.matmul(a[at:at + size], w.view(2 * c["n"], c["k"]).t()).view(size, 2, c["n"])
            at += size
    x, up = pre[:, 0], pre[:, 1]
    h = x * _sigmoid_of(x, c["activation"])[0] * up
    q = scales = None
    if c["form"] != "bf16":
        q, scales = _quantize_rows(h)
        scales = torch.where((torch.arange(a.shape[0], device="cuda") < at)[:, None], scales, torch.zeros((), device="cuda"))
    return (h.to(torch.bfloat16) if c["form"] != "fp8" else None, q, scales,
            pre.to(torch.bfloat16) if c["keep"] else None)


def _backward_plain(s):
    c = s["case"]
    g, x, up = s["g"].float(), s["pre"][:, 0].float(), s["pre"][:, 1].float()
    sig, dz = _sigmoid_of(x, c["activation"])
    d = torch.stack([g * up * (sig + x * sig * (1.0 - sig) * dz), g * (x * sig)], dim=1)
    q = scales = None
    if c["form"] != "bf16":
        q, scales = _quantize_rows(d.view(-1, c["n"]))
        q, scales = q.view(d.shape), scales.view(d.shape[0], 2, -1)
    return d.to(s["g"].dtype) if c["form"] != "fp8" else None, q, scales


def _grad_plain(s):
    c = s["case"]
    d = _values(s["qd"], s["sd"], 1)
    out = torch.zeros(d.shape[0], c["k"], device="cuda")
    at = 0
    for e, size in enumerate(s["sizes"]):
        if size:
            w = _values(s["qb"][e], s["sb"][e], BLOCK).view(2 * c["n"], c["k"])
            torch.matmul(d[at:at + size].view(size, 2 * c["n"]), w, out=out[at:at + size])
            at += size
    return out.to(torch.bfloat16)


def _clip_plain(s):
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for t in s["grads"]:
        total += t.float().square().sum(dtype=torch.float64)
    norm = total.sqrt()
    if not s["case"]["write"]:
        return norm.float()
    factor = (s["most"] / norm).clamp_max(1.0).float()
    for t, o in zip(s["grads"], s["outs"]):
        o.copy_(t.float() * factor)
    return norm.float(), s["out"]["bf16"], s["out"]["fp32"]


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"gated": _gated_plain, "backward": _backward_plain, "grad": _grad_plain, "clip": _clip_plain}[c["op"]](s)

    import fp8_quantization_moe_gb300 as gq

    if c["op"] == "gated":
        r = gq.grouped_gated_mm(s["qa"], s["sa"], s["qb"], s["sb"], s["offs"], activation=c["activation"],
                                plain=c["form"] != "fp8", fp8=c["form"] != "bf16", keep=c["keep"], out=s["out"], q=s["q"],
                                scales=s["scales"], pre=s["pre"])
        return r.out, r.q, r.scales, r.pre
    if c["op"] == "backward":
        r = gq.gated_backward(s["g"], s["pre"], activation=c["activation"], plain=c["form"] != "fp8",
                              fp8=c["form"] != "bf16")
        return r.out, r.q, r.scales
    if c["op"] == "grad":
        return gq.grouped_gated_grad(s["qd"], s["sd"], s["qb"], s["sb"], s["offs"], out=s["out"])
    if not c["write"]:
        return gq.grad_norm(s["grads"])
    norm = gq.clip_grads(s["grads"], s["most"], out=s["outs"])
    return norm, s["out"]["bf16"], s["out"]["fp32"]


# ------------------------------------------------------------ in 64 bits --

def _e4m3_exact(v):
    """Nearest e4m3 value, ties to even, saturating: three mantissa bits, smallest normal exponent -6."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -20))).clamp(-6, 8) - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _rows_exact(x, live):
    """Quantized values and scales of the first `live` rows of x; zeros behind them."""
    q, s = torch.zeros_like(x), x.new_zeros(x.shape[0], _blocks(x.shape[1]))
    for j in range(s.shape[1]):
        part = x[:live, j * BLOCK:(j + 1) * BLOCK]
        s[:live, j] = 448.0 / torch.clamp(part.abs().max(1).values, min=1e-12)
        q[:live, j * BLOCK:(j + 1) * BLOCK] = _e4m3_exact(part * s[:live, j, None])
    return q, s


def _widen(q, s):
    """The values of one quantized matrix in 64 bits; s has a row per row of q, or per 128 of them."""
    v = q.double()
    tall = 1 if s.shape[0] == q.shape[0] else BLOCK
    for i in range(s.shape[0]) if tall > 1 else [slice(None)]:
        at = slice(i * BLOCK, (i + 1) * BLOCK) if tall > 1 else i
        for j in range(s.shape[1]):
            v[at, j * BLOCK:(j + 1) * BLOCK] /= s[i, j].double() if tall > 1 else s[:, j, None].double()
    return v


def _act_exact(x, activation):
    """The activation and its derivative, gelu by its tanh form."""
    if activation == "silu":
        sig = torch.sigmoid(x)
        return x * sig, sig * (1 + x * (1 - sig))
    t = torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3))
    return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * x * x)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "clip":
        norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(t.double()) for t in s["grads"]]))
        if not c["write"]:
            return norm
        factor = min(1.0, s["most"] / float(norm))
        return norm, s["flat"]["bf16"].double() * factor, s["flat"]["fp32"].double() * factor
    if c["op"] == "backward":
        x, up, g = s["pre"][:, 0].double(), s["pre"][:, 1].double(), s["g"].double()
        act, slope = _act_exact(x, c["activation"])
        d = torch.empty(s["pre"].shape, dtype=torch.float64, device="cuda")
        d[:, 0], d[:, 1] = g * up * slope, g * act
        q = scales = None
        if c["form"] != "bf16":
            q, scales = _rows_exact(d.view(-1, c["n"]), 2 * c["rows"])
            q, scales = q.view(d.shape), scales.view(c["rows"], 2, -1)
        return d if c["form"] != "fp8" else None, q, scales
    slots, n, k = c["tokens"] * c["top_k"], c["n"], c["k"]
    if 4.0 * slots * n * k > 8e12:  # 64-bit products of that size take too long
        return None
    ends = s["offs"].tolist()
    if c["op"] == "grad":
        out = torch.zeros(slots, k, dtype=torch.float64, device="cuda")
        for e, (start, end) in enumerate(zip([0] + ends[:-1], ends)):
            for j in range(2):
                if end > start:
                    out[start:end] += _widen(s["qd"][start:end, j], s["sd"][start:end, j]) @ _widen(s["qb"][e, j], s["sb"][e, j])
        return out
    pre = torch.zeros(2, slots, n, dtype=torch.float64, device="cuda")
    a = _widen(s["qa"], s["sa"])
    for e, (start, end) in enumerate(zip([0] + ends[:-1], ends)):
        for j in range(2):
            if end > start:
                pre[j, start:end] = a[start:end] @ _widen(s["qb"][e, j], s["sb"][e, j]).mT
    h = _act_exact(pre[0], c["activation"])[0] * pre[1]
    q, scales = _rows_exact(h, ends[-1]) if c["form"] != "bf16" else (None, None)
    return h if c["form"] != "fp8" else None, q, scales, pre.transpose(0, 1) if c["keep"] else None
