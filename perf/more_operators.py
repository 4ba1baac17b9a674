"""Cases of the router with its balance loss and of the 8-bit products with a scale for each block of 128, their plain
forms and their calls.

Three kinds of pass:

router   logits to the top_k experts of each token and their weights; with `train` also the balance loss, the slots of each
         expert, and the logits' gradient from the weights' and the loss's.
linear   y = W . Q(x): rows quantized to E4M3 with one fp32 scale per 128 columns, times E4M3 weights with one fp32 scale per
         block of 128 x 128; dense, or rows grouped by expert.
train    a training step through such a product: the weights quantized from their 16-bit masters, y, and both gradients.

`own` selects the framework's calls; without it `run` computes the same in elementary torch operations in 32 bits.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}
TOP = 448.0           # largest E4M3 value
FLOOR = 2.0 ** -116   # the least maximum that a block is scaled by


def listed():
    return [
        # one decode token's router: what the call itself costs
        {"name": "router 1x32", "kind": "router", "tokens": 1, "experts": 32, "top_k": 4, "score": "softmax", "renorm": True, "scale": 1.0, "dtype": "bf16", "dead": 0.0, "train": False},
        # a ragged, padded batch before 256 experts with sigmoid scores
        {"name": "router 777x256 sigmoid", "kind": "router", "tokens": 777, "experts": 256, "top_k": 8, "score": "sigmoid", "renorm": True, "scale": 2.5, "dtype": "f32", "dead": 0.2, "train": False},
        # a training step's router of the benchmarked layer, rows not a multiple of anything
        {"name": "router 8191x32 train", "kind": "router", "tokens": 8191, "experts": 32, "top_k": 4, "score": "softmax", "renorm": True, "scale": 1.0, "dtype": "bf16", "dead": 0.0, "train": True},
        # a long batch before many experts, forward and backward
        {"name": "router 16384x256 train", "kind": "router", "tokens": 16384, "experts": 256, "top_k": 8, "score": "softmax", "renorm": False, "scale": 1.0, "dtype": "f32", "dead": 0.1, "train": True},
        # one decode token through a projection
        {"name": "linear 1x2880x2880", "kind": "linear", "rows": 1, "experts": 1, "n": 2880, "k": 2880, "dtype": "bf16"},
        # a decode batch through a wide projection
        {"name": "linear 16x7168x7168", "kind": "linear", "rows": 16, "experts": 1, "n": 7168, "k": 7168, "dtype": "bf16"},
        # a ragged chunk of a prompt through a down projection
        {"name": "linear 1001x7168x2048 f16", "kind": "linear", "rows": 1001, "experts": 1, "n": 7168, "k": 2048, "dtype": "f16"},
        # a long prompt through a square projection
        {"name": "linear 8192x7168x7168", "kind": "linear", "rows": 8192, "experts": 1, "n": 7168, "k": 7168, "dtype": "bf16"},
        # a decode batch's 128 slots over 256 experts, many of them without a row
        {"name": "linear 128 of 256 experts", "kind": "linear", "rows": 128, "experts": 256, "n": 2048, "k": 7168, "dtype": "bf16"},
        # a prompt's slots over 32 experts
        {"name": "linear 16384 of 32 experts", "kind": "linear", "rows": 16384, "experts": 32, "n": 2880, "k": 2880, "dtype": "bf16"},
        # a small training step with odd sizes
        {"name": "train 333x1001x2880", "kind": "train", "rows": 333, "experts": 1, "n": 1001, "k": 2880, "dtype": "f16"},
        # a training step of an expert projection
        {"name": "train 16384 of 32 experts", "kind": "train", "rows": 16384, "experts": 32, "n": 2880, "k": 2880, "dtype": "bf16"},
    ]


def draw(rng):
    def size(lo, hi, unit=1):
        return unit * min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))

    kind = rng.choice(("router", "linear", "linear", "train"))
    dtype = rng.choice(("bf16", "bf16", "f16"))
    if kind == "router":
        experts = size(2, 512)
        return {"kind": kind, "tokens": min(size(1, 16384), 16384 * 256 // experts), "experts": experts,
                "top_k": rng.randint(1, min(8, experts)), "score": rng.choice(("softmax", "sigmoid")), "renorm": rng.random() < 0.6,
                "scale": rng.choice((1.0, 2.5)), "dtype": rng.choice((dtype, "f32")), "dead": rng.choice((0.0, 0.0, 0.3)),
                "train": rng.random() < 0.6}
    n, k, experts = size(8, 7168), size(1, 448, 16), rng.choice((1, 1, size(2, 256)))
    experts = max(1, min(experts, 16384 * 2880 * 2880 * 3 // (512 * n * k)))
    most = 8192 * 7168 * 7168 if kind == "linear" else 16384 * 2880 * 2880
    return {"kind": kind, "rows": min(size(1, 16384), max(1, most // (n * k))), "experts": experts, "n": n, "k": k, "dtype": dtype}


# ------------------------------------------------------------------ inputs


def randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def rand(g, *shape):
    return torch.rand(shape, generator=g, device=DEV)


def activations(g, rows, width, dtype, spread=0.5):
    """Normal values whose columns differ in scale, a few of them by much: what a residual stream looks like."""
    scale = torch.exp(spread * randn(g, width))
    scale = torch.where(rand(g, width) < 0.01, scale * 16, scale)
    return (randn(g, rows, width) * scale).to(TYPES[dtype])


def master(g, n, k):
    """Weights whose rows differ in scale."""
    return randn(g, n, k) * (0.03 * torch.exp(0.3 * randn(g, n, 1)))


def prepare(case, seed):
    g, kind = torch.Generator(device=DEV).manual_seed(seed), case["kind"]
    s = dict(case)
    if kind == "router":
        tokens, experts = case["tokens"], case["experts"]
        s["logits"] = (0.5 * randn(g, experts) + randn(g, tokens, experts)).to(TYPES[case["dtype"]])
        s["live"] = (rand(g, tokens) >= case["dead"]).to(torch.uint8) if case["dead"] else None
        if case["train"]:
            s["dweights"] = 1e-2 * randn(g, tokens, case["top_k"])
            s["dloss"] = 1e-2 * (1 + rand(g, 1))
        return s
    rows, experts, n, k = case["rows"], case["experts"], case["n"], case["k"]
    s["x"] = activations(g, rows, k, case["dtype"])
    # rows of each expert, as a router whose experts differ in popularity gives them
    expert = torch.topk(0.5 * randn(g, experts) + randn(g, rows, experts), 1).indices.flatten()
    each = torch.bincount(expert, minlength=experts)
    s["offsets"] = torch.nn.functional.pad(torch.cumsum(each, 0), (1, 0)).to(torch.int32) if experts > 1 else None
    s["cap"] = max(1, int(each.max()))   # rows that the plain form keeps room for in each expert
    if kind == "linear":
        s["w"] = torch.empty(experts, n, k, dtype=torch.uint8, device=DEV)
        s["w_scales"] = torch.empty(experts, -(-n // 128), -(-k // 128), device=DEV)
        for e in range(experts):
            q, s["w_scales"][e] = quantized_blocks(master(g, n, k)[None])
            s["w"][e] = q[0].to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        s["w"] = torch.empty(experts, n, k, dtype=TYPES[case["dtype"]], device=DEV)
        for e in range(experts):
            s["w"][e] = master(g, n, k)
        # gradient rows start on 16-byte boundaries, whatever their width is
        s["dy"] = torch.zeros(rows, -(-n // 8) * 8, dtype=TYPES[case["dtype"]], device=DEV)
        s["dy"][:, :n] = activations(g, rows, n, case["dtype"]) * 0.02
    return s


# ------------------------------------------------------------------ plain forms


def scales_of(top):
    """(scale, its inverse) of blocks with these maxima, each one fp32 division."""
    a = top.clamp(min=FLOOR)
    return a / torch.full_like(a, TOP), torch.full_like(a, TOP) / a


def element(v):
    return v.clamp(-TOP, TOP).to(torch.float8_e4m3fn).float()


def quantized_rows(x):
    """(element values, scales [rows][groups]) of rows x, in groups of 128 columns."""
    width = x.shape[1]
    v = torch.nn.functional.pad(x.float(), (0, -width % 128)).view(x.shape[0], -1, 128)
    scale, inverse = scales_of(v.abs().amax(-1))
    return element(v * inverse[..., None]).flatten(1)[:, :width], scale


def quantized_blocks(w):
    """(element values, scales [experts][row blocks][column blocks]) of matrices w [experts][n][k]."""
    experts, n, k = w.shape
    v = torch.nn.functional.pad(w.float(), (0, -k % 128, 0, -n % 128)).unflatten(2, (-1, 128)).unflatten(1, (-1, 128))
    scale, inverse = scales_of(v.abs().amax((2, 4)))
    return element(v * inverse[:, :, None, :, None]).flatten(3, 4).flatten(1, 2)[:, :n, :k], scale


def requantized(x):
    q, scale = quantized_rows(x)
    return q * torch.repeat_interleave(scale, 128, 1)[:, :x.shape[1]]


def decoded(codes, scales):
    """Matrices of E4M3 values or codes [experts][n][k] and their blocks' scales."""
    v = codes.view(torch.float8_e4m3fn).float() if codes.dtype == torch.uint8 else codes
    n, k = v.shape[1:]
    return v * torch.repeat_interleave(torch.repeat_interleave(scales, 128, 1)[:, :n], 128, 2)[:, :, :k]


def blocks(s):
    """Each expert's rows in a padded block: (row of each place, whether it is one, place of each row)."""
    rows, experts = s["rows"], s["experts"]
    if experts == 1:
        at = torch.arange(rows, device=DEV)
        return at[None], torch.ones(1, rows, dtype=torch.bool, device=DEV), at
    offsets = s["offsets"].long()
    row = torch.arange(s["cap"], device=DEV)[None] + offsets[:-1, None]
    live = row < offsets[1:, None]
    expert = torch.searchsorted(offsets[1:], torch.arange(rows, device=DEV), right=True)
    return torch.where(live, row, 0), live, expert * s["cap"] + torch.arange(rows, device=DEV) - offsets[expert]


def scores(s):
    """(logits, scores, scores as the balance loss takes them) in 32 bits."""
    l = s["logits"].float()
    if s["score"] == "softmax":
        p = torch.exp(l - l.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
        return l, p, p
    p = 1 / (1 + torch.exp(-l))
    return l, p, p / p.sum(1, keepdim=True)


def plain(s):
    kind, out = s["kind"], TYPES[s["dtype"]]
    if kind == "router":
        experts, top_k, c = s["experts"], s["top_k"], s["scale"]
        l, p, share = scores(s)
        live = s["live"][:, None] > 0 if s["live"] is not None else torch.ones_like(l[:, :1], dtype=torch.bool)
        index = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :top_k]   # ties to the lowest index
        chosen = torch.gather(p, 1, index)
        weights = c * (chosen / chosen.sum(1, keepdim=True) if s["renorm"] else chosen)
        got = {"ids": torch.where(live, index, -1).to(torch.int32), "weights": torch.where(live, weights, 0.0)}
        if not s["train"]:
            return got
        n = live.sum().clamp(min=1)   # without a live token everything is 0
        hits = torch.zeros(s["tokens"], experts, device=DEV).scatter_(1, index, 1.0)
        counts = torch.where(live, hits, 0.0).double().sum(0)
        f = (counts / (top_k * n)).float()
        means = torch.where(live, share, 0.0).sum(0) / n
        got |= {"counts": torch.cat([counts, live.sum()[None].double()]).to(torch.int32), "means": means, "loss": experts * (f * means).sum()}
        # the weights' part of the gradient, over the chosen experts
        g = c * s["dweights"]
        sigmoid = s["score"] == "sigmoid"
        other = 1 / (1 + torch.exp(l)) if sigmoid else 1.0   # 1 - s
        if s["renorm"]:
            q = chosen / chosen.sum(1, keepdim=True)
            d = torch.zeros_like(l).scatter_(1, index, q * (g - (g * q).sum(1, keepdim=True))) * other
        elif sigmoid:
            d = torch.zeros_like(l).scatter_(1, index, g * chosen) * other
        else:
            d = torch.zeros_like(l).scatter_(1, index, g * chosen) - p * (g * chosen).sum(1, keepdim=True)
        d = d + s["dloss"] * experts / n * share * (f - (share * f).sum(1, keepdim=True)) * other
        return got | {"dlogits": torch.where(live, d, 0.0).to(out)}
    row, live, place = blocks(s)
    x = requantized(s["x"])
    if kind == "linear":
        w = decoded(s["w"], s["w_scales"])
        return {"y": torch.bmm(x[row], w.transpose(1, 2)).flatten(0, 1)[place].to(out)}
    q, scale = quantized_blocks(s["w"])
    w, dy = decoded(q, scale), s["dy"][:, :s["n"]]
    y = torch.bmm(x[row], w.transpose(1, 2)).flatten(0, 1)[place]
    dx = torch.bmm(requantized(dy)[row], w).flatten(0, 1)[place]
    block = torch.where(live[..., None], dy.float()[row], 0.0)
    return {"codes": q.to(torch.float8_e4m3fn), "scales": scale, "y": y.to(out), "dx": dx.to(out),
            "dw": torch.bmm(block.transpose(1, 2), s["x"].float()[row])}


# ------------------------------------------------------------------ the framework's calls


def new(*shape, dtype=torch.uint8):
    return torch.empty(shape, dtype=dtype, device=DEV)


def called(s):
    import bit_quantized_moe_gb300 as qmv

    kind, dt, out = s["kind"], s["dtype"], TYPES[s["dtype"]]
    if kind == "router":
        tokens, experts, top_k, i32, f32 = s["tokens"], s["experts"], s["top_k"], torch.int32, torch.float32
        ids, weights = new(tokens, top_k, dtype=i32), new(tokens, top_k, dtype=f32)
        qmv.qmv_moe_router(dt, s["logits"], experts, s["live"], tokens, experts, top_k, s["score"], s["renorm"], s["scale"], ids, weights)
        got = {"ids": ids, "weights": weights}
        if s["train"]:
            counts, means, loss = new(experts + 1, dtype=i32), new(experts, dtype=f32), new(1, dtype=f32)
            ws = new(qmv.qmv_moe_balance_workspace_bytes(tokens, experts))
            qmv.qmv_moe_balance(dt, s["logits"], experts, s["live"], ids, tokens, experts, top_k, s["score"], counts, means, loss, ws)
            dlogits = new(tokens, experts, dtype=out)
            qmv.qmv_moe_router_grad(dt, s["logits"], experts, s["live"], ids, s["dweights"], counts, s["dloss"], tokens, experts, top_k,
                                    s["score"], s["renorm"], s["scale"], dlogits, experts)
            got |= {"counts": counts, "means": means, "loss": loss.view(()), "dlogits": dlogits}
        return got
    rows, experts, n, k, offsets = s["rows"], s["experts"], s["n"], s["k"], s["offsets"]
    ws, y = new(qmv.qmv_b128_linear_workspace_bytes(rows, k)), new(rows, n, dtype=out)
    if kind == "linear":
        qmv.qmv_b128_linear(s["w"], s["w_scales"], experts, n, k, dt, s["x"], k, rows, offsets, ws, y)
        return {"y": y}
    codes, scales = new(experts, n, k), new(experts, -(-n // 128), -(-k // 128), dtype=torch.float32)
    qmv.qmv_quantize_weights_b128(dt, s["w"], experts, n, k, codes, scales)
    qmv.qmv_b128_linear(codes, scales, experts, n, k, dt, s["x"], k, rows, offsets, ws, y)
    ld = s["dy"].shape[1]
    dyq, dx, dw = new(qmv.qmv_act_b128_bytes(rows, n)), new(rows, k, dtype=out), new(experts, n, k, dtype=torch.float32)
    qmv.qmv_quantize_act_b128(dt, s["dy"], ld, rows, n, dyq)
    qmv.qmv_b128_grad_x(codes, scales, experts, n, k, dyq, rows, offsets, dt, dx)
    qmv.qmv_b128_grad_w(dt, s["dy"], ld, s["x"], k, experts, n, k, rows, offsets, "f32", dw)
    return {"codes": codes.view(torch.float8_e4m3fn), "scales": scales, "y": y, "dx": dx, "dw": dw}


def run(state):
    return called(state) if own else plain(state)


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    kind, size = case["kind"], SIZES[case["dtype"]]
    if kind == "router":
        table, slots = case["tokens"] * case["experts"], case["tokens"] * case["top_k"]
        # logits in, ids and weights out; with the gradient dweights in and dlogits out
        return {"bytes": table * size + 8 * slots + (table * size + 4 * slots + 8 * case["experts"] if case["train"] else 0),
                "flops": 4 * table * (3 if case["train"] else 1)}
    rows, n, k = case["rows"], case["n"], case["k"]
    matrices = min(case["experts"], rows)   # at most so many experts have rows
    if kind == "linear":
        return {"bytes": matrices * n * k + rows * (n + k) * size, "flops": 2 * rows * n * k}
    # masters in, codes out; x and dy in, y and dx out; the weights' gradient out in 32 bits
    return {"bytes": case["experts"] * n * k * (size + 1 + 4) + 2 * rows * (n + k) * size, "flops": 6 * rows * n * k}


# ------------------------------------------------------------------ the definitions in 64 bits


def exponent(v):
    """floor(log2 v) of positive float64 values, from their bits."""
    return (v.view(torch.int64) >> 52) - 1023


def power(e):
    """2^e of whole e as float64, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def to_f32(v):
    return v.to(torch.float32).double()


def nearest(v):
    """The nearest E4M3 value of float64 v, ties to even."""
    a = v.abs().clamp(max=TOP)
    unit = power(exponent(a).clamp(min=-6) - 3)
    return torch.copysign(torch.round(a / unit) * unit, v)


def cut(v, tall):
    """(values, scales) of one matrix in blocks of `tall` x 128: the scale and its inverse are rounded to 32 bits, and so is the
    scaled number before it takes its nearest E4M3 value."""
    values, columns = torch.empty_like(v), []
    for c in range(0, v.shape[1], 128):
        part = v[:, c:c + 128]
        top = part.abs().amax(1)
        top = torch.stack([b.max() for b in top.split(tall)]) if tall > 1 else top
        top = top.clamp(min=FLOOR)
        inverse = torch.repeat_interleave(to_f32(TOP / top), tall)[:len(v), None]
        values[:, c:c + 128] = nearest(to_f32(part * inverse))
        columns.append(to_f32(top / TOP))
    return values, torch.stack(columns, 1)


def spread(values, scales, tall):
    return values * torch.repeat_interleave(torch.repeat_interleave(scales, tall, 0)[:len(values)], 128, 1)[:, :values.shape[1]]


def e4m3(codes):
    m, ex = (codes & 7).double(), codes >> 3 & 15
    v = torch.where(ex > 0, (8 + m) * power(ex.int() - 10), m * 2.0 ** -9)
    return torch.where(codes >= 128, -v, v)


def exact_router(case, s):
    l, experts, top_k, c = s["logits"].double(), case["experts"], case["top_k"], case["scale"]
    soft = case["score"] == "softmax"
    l.requires_grad_()
    p = torch.softmax(l, 1) if soft else torch.sigmoid(l)
    share = p if soft else p / p.sum(1, keepdim=True)
    alive = torch.ones(case["tokens"], device=DEV, dtype=torch.float64) if s["live"] is None else s["live"].double()
    # an expert's place: those above it, and the equal ones before it
    picked, left = [], l.detach().clone()
    for _ in range(top_k):
        best = (left == left.amax(1, keepdim=True)).to(torch.uint8).argmax(1)
        picked.append(best)
        left.scatter_(1, best[:, None], -math.inf)
    index = torch.stack(picked, 1)
    chosen = p.gather(1, index)
    weights = c * (chosen / chosen.sum(1, keepdim=True) if case["renorm"] else chosen) * alive[:, None]
    got = {"ids": None, "weights": weights.detach()}
    if not case["train"]:
        return got
    n = alive.sum().clamp(min=1)
    f = torch.zeros(experts, dtype=torch.float64, device=DEV).index_add(0, index.flatten(), alive.repeat_interleave(top_k)) / (top_k * n)
    means = (share * alive[:, None]).sum(0) / n
    loss = experts * (f * means).sum()
    total = (weights * s["dweights"].double()).sum() + loss * s["dloss"].double().sum()
    (d,) = torch.autograd.grad(total, l)
    return got | {"counts": None, "means": means.detach(), "loss": loss.detach(), "dlogits": d}


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "router":
        return exact_router(case, s)
    rows, experts, n, k = case["rows"], case["experts"], case["n"], case["k"]
    ends = [0, rows] if experts == 1 else s["offsets"].tolist()
    x = spread(*cut(s["x"].double(), 1), 1)
    y = torch.zeros(rows, n, dtype=torch.float64, device=DEV)
    if case["kind"] == "linear":
        for e in range(experts):
            a, b = ends[e], ends[e + 1]
            if b > a:
                y[a:b] = x[a:b] @ spread(e4m3(s["w"][e]), s["w_scales"][e].double(), 128).T
        return {"y": y}
    dy = s["dy"][:, :n].double()
    dyq, dx = spread(*cut(dy, 1), 1), torch.zeros(rows, k, dtype=torch.float64, device=DEV)
    dw = torch.zeros(experts, n, k, dtype=torch.float64, device=DEV)
    codes, scales = torch.zeros_like(dw), torch.zeros(experts, -(-n // 128), -(-k // 128), dtype=torch.float64, device=DEV)
    for e in range(experts):
        a, b = ends[e], ends[e + 1]
        codes[e], scales[e] = cut(s["w"][e].double(), 128)
        w = spread(codes[e], scales[e], 128)
        y[a:b], dx[a:b], dw[e] = x[a:b] @ w.T, dyq[a:b] @ w, dy[a:b].T @ s["x"][a:b].double()
    return {"codes": codes, "scales": scales, "y": y, "dx": dx, "dw": dw}
