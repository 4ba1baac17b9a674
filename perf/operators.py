"""Cases of the many-token operators beside the decode matvec, their plain forms and their calls.

Four kinds of pass, each over the range from one token to a long prompt:

norm     y = (x + r) / sqrt(mean((x + r)^2) + eps) * gain, the sum kept for the next layer,
         y as it is or in 8 bits (E4M3 codes, one E8M0 scale per 32 columns).
product  y = W . Q(x): activations quantized to the weights' microscaled format (E2M1 or E4M3,
         one E8M0 scale per 32 along K), then a product of two microscaled matrices.
routing  tokens sorted by expert, their rows brought into that order, the experts' rows brought
         back and summed with the router's weights; with `train` also every gradient.
experts  a whole expert layer on many tokens: sort, rows, gate/up with SwiGLU, down, weighted sum.

`own` selects the framework's calls; without it `run` computes the same in elementary torch
operations in 32 bits.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BITS = {"mxfp4": 4, "mxfp8": 8}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
EMAX = {"mxfp4": 2, "mxfp8": 8}       # exponent of the element type's largest power of two
TOP = {"mxfp4": 6.0, "mxfp8": 448.0}  # its largest value
WEIGHT_SCALES = {"mxfp4": (112, 122), "mxfp8": (107, 117)}   # E8M0 bytes: weights of about 0.03 rms
EPS = 1e-5


def listed():
    return [
        # one decode token into an MXFP8 layer: what the call itself costs
        {"name": "norm 1x2880 mxfp8", "kind": "norm", "rows": 1, "width": 2880, "dtype": "bf16", "residual": True, "out": "mxfp8"},
        # the first norm of a model, no residual yet, the output kept in the activations' type; odd rows and width
        {"name": "norm 513x2881 f16", "kind": "norm", "rows": 513, "width": 2881, "dtype": "f16", "residual": False, "out": "plain"},
        # a long prompt through a wide model
        {"name": "norm 8192x7168 mxfp8", "kind": "norm", "rows": 8192, "width": 7168, "dtype": "bf16", "residual": True, "out": "mxfp8"},
        # a projection just past the decode calls' 16 tokens
        {"name": "product 17x2880x2880 fp4", "kind": "product", "fmt": "mxfp4", "rows": 17, "n": 2880, "k": 2880, "dtype": "bf16"},
        # a ragged chunk of a prompt through an 8-bit down projection
        {"name": "product 1001x7168x2048 fp8", "kind": "product", "fmt": "mxfp8", "rows": 1001, "n": 7168, "k": 2048, "dtype": "f16"},
        # a long prompt through a square dense projection
        {"name": "product 8192x7168x7168 fp4", "kind": "product", "fmt": "mxfp4", "rows": 8192, "n": 7168, "k": 7168, "dtype": "bf16"},
        # a decode batch over many experts, some slots dropped
        {"name": "routing 16x8 of 256", "kind": "routing", "tokens": 16, "top_k": 8, "experts": 256, "width": 7168, "dtype": "bf16", "drop": 0.05, "train": False},
        # a prompt through 32 experts
        {"name": "routing 4096x4 of 32", "kind": "routing", "tokens": 4096, "top_k": 4, "experts": 32, "width": 2880, "dtype": "bf16", "drop": 0.0, "train": False},
        # a training step's routing, forward and backward
        {"name": "routing 8191x4 train", "kind": "routing", "tokens": 8191, "top_k": 4, "experts": 32, "width": 2880, "dtype": "bf16", "drop": 0.02, "train": True},
        # the first size that the decode layer no longer takes (132 routed slots)
        {"name": "experts 33x4 of 32 fp4", "kind": "experts", "fmt": "mxfp4", "tokens": 33, "top_k": 4, "experts": 32, "hidden": 2880, "inner": 2880, "dtype": "bf16", "drop": 0.0},
        # an 8-bit layer with few, wide experts and ragged rows
        {"name": "experts 777x2 of 8 fp8", "kind": "experts", "fmt": "mxfp8", "tokens": 777, "top_k": 2, "experts": 8, "hidden": 7168, "inner": 2048, "dtype": "bf16", "drop": 0.02},
        # a long prompt through the benchmarked layer
        {"name": "experts 4096x4 of 32 fp4", "kind": "experts", "fmt": "mxfp4", "tokens": 4096, "top_k": 4, "experts": 32, "hidden": 2880, "inner": 2880, "dtype": "bf16", "drop": 0.0},
    ]


def draw(rng):
    def size(lo, hi, unit=1):
        got = unit * min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))
        return got if got != 3072 else got - unit   # not a size that this repository has

    kind = rng.choice(("norm", "product", "routing", "experts"))
    dtype = rng.choice(("bf16", "bf16", "f16"))
    if kind == "norm":
        out = rng.choice(("mxfp8", "mxfp8", "plain"))
        width = size(1, 256, 32) if out == "mxfp8" else size(1, 8192)
        rows = min(size(1, 16384), 8192 * 7168 // width)
        return {"kind": kind, "rows": rows, "width": width, "dtype": rng.choice((dtype, "f32")), "residual": rng.random() < 0.7, "out": out}
    if kind == "product":
        n, k = size(16, 8192), size(1, 256, 32)
        rows = min(size(1, 8192), max(1, 8192 * 7168 * 7168 // (n * k)))
        return {"kind": kind, "fmt": rng.choice(("mxfp4", "mxfp8")), "rows": rows, "n": n, "k": k, "dtype": dtype}
    if kind == "routing":
        experts, width = size(2, 512), size(8, 7168)
        top_k = rng.randint(1, min(8, experts))
        tokens = min(size(1, 8192), max(1, 8191 * 4 * 2880 // (top_k * width)))
        return {"kind": kind, "tokens": tokens, "top_k": top_k, "experts": experts, "width": width, "dtype": rng.choice((dtype, "f32")),
                "drop": rng.choice((0.0, 0.0, 0.1)), "train": rng.random() < 0.5}
    hidden, inner = size(4, 224, 32), size(4, 128, 32)
    experts = min(size(2, 128), max(2, 32 * 2880 * 2880 // (hidden * inner)))
    top_k = rng.randint(1, min(8, experts))
    tokens = min(size(1, 4096), max(1, 4096 * 4 * 2880 * 2880 // (top_k * hidden * inner)))
    return {"kind": kind, "fmt": rng.choice(("mxfp4", "mxfp8")), "tokens": tokens, "top_k": top_k, "experts": experts, "hidden": hidden,
            "inner": inner, "dtype": dtype, "drop": rng.choice((0.0, 0.0, 0.1))}


# ------------------------------------------------------------------ inputs


def generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def activations(g, rows, width, dtype, spread=0.5):
    """Normal values whose columns differ in scale, a few of them by much: what a residual stream looks like."""
    scale = torch.exp(spread * torch.randn(width, generator=g, device=DEV))
    scale = torch.where(torch.rand(width, generator=g, device=DEV) < 0.01, scale * 16, scale)
    return (torch.randn(rows, width, generator=g, device=DEV) * scale).to(TYPES[dtype])


def weights(g, fmt, experts, n, k):
    """Canonical codes [experts][n][bytes of a row] and E8M0 scales [experts][n][k / 32]."""
    if fmt == "mxfp4":
        codes = torch.randint(0, 256, (experts, n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    else:
        codes = torch.randint(0, 254, (experts, n, k), generator=g, device=DEV, dtype=torch.uint8)
        codes += (codes >= 127).to(torch.uint8)   # without the two NaN codes
    lo, hi = WEIGHT_SCALES[fmt]
    return codes, torch.randint(lo, hi + 1, (experts, n, k // 32), generator=g, device=DEV, dtype=torch.uint8)


def packed(codes, scales, bits):
    """The library's weight layout of canonical codes and scales (what its packer writes on the host), laid out on the
    GPU once, as a program does when it loads a model: tiles of 8 rows x 1024 columns, codes then scales of each."""
    experts, n, width = codes.shape
    tiles, groups = -(-n // 8), scales.shape[2]
    codes = torch.nn.functional.pad(codes, (0, 0, 0, 8 * tiles - n)).view(experts, tiles, 8, width)
    scales = torch.nn.functional.pad(scales, (0, 0, 0, 8 * tiles - n)).view(experts, tiles, 8, groups)
    full, chunk, lane = groups // 32, 128 * bits, 4 * bits
    head = torch.cat([codes[..., :full * chunk].reshape(experts, tiles, 8, full, chunk).transpose(2, 3).flatten(3),
                      scales[..., :full * 32].reshape(experts, tiles, 8, full, 32).permute(0, 1, 3, 4, 2).flatten(3)], 3).flatten(2)
    last = torch.cat([codes[..., full * chunk:].flatten(2), scales[..., full * 32:].transpose(2, 3).flatten(2)], 2)
    rest = groups % 32
    last = torch.nn.functional.pad(last, (0, -(8 * rest * (lane + 1)) % 16))
    whole = torch.cat([head, last], 2).flatten(1)
    return torch.nn.functional.pad(whole, (0, -whole.shape[1] % 256)).flatten()


def interleaved(gate, up):
    """Rows of gate and up by fours, as the fused gate/up layout has them."""
    experts, n, width = gate.shape
    pad = (0, 0, 0, -n % 4)
    both = [torch.nn.functional.pad(v, pad).view(experts, -1, 4, width) for v in (gate, up)]
    return torch.stack(both, 2).view(experts, -1, width)


def routes(g, case):
    """Expert ids and weights of a router whose experts differ in popularity; -1 for a dropped slot."""
    experts, tokens, top_k = case["experts"], case["tokens"], case["top_k"]
    logits = 0.5 * torch.randn(experts, generator=g, device=DEV) + torch.randn(tokens, experts, generator=g, device=DEV)
    value, ids = torch.topk(logits, top_k, dim=1)
    ids = torch.where(torch.rand(tokens, top_k, generator=g, device=DEV) < case["drop"], -1, ids)
    return ids.to(torch.int32), torch.softmax(value, 1)


def prepare(case, seed):
    g, kind = generator(seed), case["kind"]
    s = dict(case)
    if kind == "norm":
        s["x"] = activations(g, case["rows"], case["width"], case["dtype"])
        s["res"] = activations(g, case["rows"], case["width"], case["dtype"]) if case["residual"] else None
        s["gain"] = (1 + 0.1 * torch.randn(case["width"], generator=g, device=DEV)).to(TYPES[case["dtype"]])
    elif kind == "product":
        s["x"] = activations(g, case["rows"], case["k"], case["dtype"])
        s["codes"], s["scales"] = weights(g, case["fmt"], 1, case["n"], case["k"])
        s["w"] = packed(s["codes"], s["scales"], BITS[case["fmt"]])
    elif kind == "routing":
        tokens, slots, width = case["tokens"], case["tokens"] * case["top_k"], case["width"]
        s["ids"], s["weights"] = routes(g, case)
        s["x"] = activations(g, tokens, width, case["dtype"])
        s["ys"] = activations(g, slots, width, case["dtype"])      # what the experts gave
        if case["train"]:
            s["dy"] = activations(g, tokens, width, case["dtype"])
            s["dxs"] = activations(g, slots, width, case["dtype"])   # the experts' input gradients
    else:
        s["ids"], s["weights"] = routes(g, case)
        s["x"] = activations(g, case["tokens"], case["hidden"], case["dtype"], 0.2)
        fmt, experts, hidden, inner = case["fmt"], case["experts"], case["hidden"], case["inner"]
        s["gate"], s["gate_scales"] = weights(g, fmt, experts, inner, hidden)
        s["up"], s["up_scales"] = weights(g, fmt, experts, inner, hidden)
        s["down"], s["down_scales"] = weights(g, fmt, experts, hidden, inner)
        s["w_gate_up"] = packed(interleaved(s["gate"], s["up"]), interleaved(s["gate_scales"], s["up_scales"]), BITS[fmt])
        s["w_down"] = packed(s["down"], s["down_scales"], BITS[fmt])
        # rows that the plain form keeps room for in each expert
        s["cap"] = max(1, int(torch.bincount(s["ids"].flatten().clamp(min=-1).to(torch.int64) + 1, minlength=experts + 1)[1:].max()))
    return s


# ------------------------------------------------------------------ plain forms


def group_scale(v, fmt):
    """E8M0 bytes of groups v [..., 32]: 2^(floor(log2 max|v|) - emax), 0 for a group of zeros, 255 with a value that is not finite."""
    top = v.abs().amax(-1)
    e = (torch.frexp(top).exponent - 1 - EMAX[fmt] + 127).clamp(0, 254)
    return torch.where(torch.isfinite(top), torch.where(top > 0, e, 0), 255)


def quantized(x, fmt):
    """(element values, E8M0 bytes) of x [rows][k] in groups of 32."""
    v = x.float().view(x.shape[0], -1, 32)
    e = group_scale(v, fmt)
    q = torch.ldexp(v, (127 - e).clamp(min=-127)[..., None]).clamp(-TOP[fmt], TOP[fmt])
    if fmt == "mxfp8":
        q = q.to(torch.float8_e4m3fn).float()
    else:
        a = q.abs()
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
        q = torch.copysign(torch.round(a / step) * step, q)
    return torch.where((e < 255)[..., None], q, 0.0), e


def requantized(x, fmt):
    """x [rows][k] as its microscaled form stands for it."""
    q, e = quantized(x, fmt)
    scale = torch.where(e < 255, torch.ldexp(torch.ones_like(q[..., 0]), e - 127), math.nan)
    return (q * scale[..., None]).view(x.shape)


def decoded(codes, scales, fmt):
    if fmt == "mxfp8":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        v = torch.tensor(E2M1, device=DEV)[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]
    scale = torch.ldexp(torch.ones_like(scales, dtype=torch.float32), scales.int() - 127)
    return (v.unflatten(-1, (-1, 32)) * scale[..., None]).flatten(-2)


def sorted_slots(s):
    """Slots in the order of their experts, dropped ones last: (offsets, slot of each row, row of each slot)."""
    ids, experts = s["ids"].flatten(), s["experts"]
    key = torch.where((ids >= 0) & (ids < experts), ids, experts)
    slot_of_row = torch.argsort(key, stable=True)
    row_of_slot = torch.empty_like(slot_of_row)
    row_of_slot[slot_of_row] = torch.arange(len(ids), device=DEV)
    ends = torch.searchsorted(key[slot_of_row], torch.arange(experts + 1, device=DEV, dtype=torch.int32))
    return ends, slot_of_row, row_of_slot, key < experts


def plain(s):
    kind, out = s["kind"], TYPES[s["dtype"]]
    if kind == "norm":
        v = s["x"].float() + s["res"].float() if s["residual"] else s["x"].float()
        y = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * s["gain"].float()
        got = {"sum": v.to(out)} if s["residual"] else {}
        if s["out"] == "plain":
            return {"y": y.to(out), **got}
        q, e = quantized(y, "mxfp8")
        e = torch.nn.functional.pad(e, (0, -e.shape[1] % 4)).view(s["rows"], -1, 4).transpose(0, 1)
        return {"codes": q.flatten(1).to(torch.float8_e4m3fn), "scales": e.to(torch.uint8).contiguous().view(torch.float8_e8m0fnu), **got}
    if kind == "product":
        w = decoded(s["codes"], s["scales"], s["fmt"])[0]
        return {"y": (requantized(s["x"], s["fmt"]) @ w.T).to(out)}
    offsets, slot_of_row, row_of_slot, valid = sorted_slots(s)
    token = slot_of_row // s["top_k"]
    weight = torch.where(valid, s["weights"].flatten(), 0.0)
    if kind == "routing":
        live = valid[slot_of_row][:, None]
        rows = s["ys"].float()[row_of_slot].view(s["tokens"], s["top_k"], -1)
        keep = valid.view(s["tokens"], s["top_k"], 1)
        got = {"offsets": offsets.to(torch.int32), "slot_of_row": slot_of_row.to(torch.int32),
               "row_of_slot": torch.where(valid, row_of_slot, -1 - row_of_slot).to(torch.int32),
               "xs": torch.where(live, s["x"][token], 0),
               "y": torch.where(keep, weight.view(s["tokens"], -1, 1) * rows, 0.0).sum(1).to(out)}
        if s["train"]:
            dy = s["dy"].float()
            back = s["dxs"].float()[row_of_slot].view(s["tokens"], s["top_k"], -1)
            got["dx"] = torch.where(keep, back, 0.0).sum(1).to(out)
            got["dys"] = torch.where(live, weight[slot_of_row][:, None] * dy[token], 0.0).to(out)
            got["dweights"] = torch.where(keep[..., 0], (rows * dy[:, None]).sum(-1), 0.0)
        return got
    # each expert's rows in a padded block, so that its three products are batched ones
    experts, cap, fmt = s["experts"], s["cap"], s["fmt"]
    row = torch.arange(cap, device=DEV)[None] + offsets[:-1, None]
    live = row < offsets[1:, None]
    block = slot_of_row[torch.where(live, row, 0)]
    x = requantized(s["x"], fmt)[block // s["top_k"]]
    g = torch.bmm(x, decoded(s["gate"], s["gate_scales"], fmt).transpose(1, 2))
    u = torch.bmm(x, decoded(s["up"], s["up_scales"], fmt).transpose(1, 2))
    h = requantized((g / (1 + torch.exp(-g)) * u).flatten(0, 1), fmt).view(experts, cap, -1)
    ys = torch.bmm(h, decoded(s["down"], s["down_scales"], fmt).transpose(1, 2))
    expert = torch.where(valid, s["ids"].flatten(), 0).long()
    at = expert * cap + torch.where(valid, row_of_slot - offsets[expert], 0)
    return {"y": (ys.flatten(0, 1)[at] * weight[:, None]).view(s["tokens"], s["top_k"], -1).sum(1).to(out)}


# ------------------------------------------------------------------ the framework's calls


def new(*shape, dtype=torch.uint8):
    return torch.empty(shape, dtype=dtype, device=DEV)


def called(s):
    import bit_quantized_moe_gb300 as qmv

    kind, dt, out = s["kind"], s["dtype"], TYPES[s["dtype"]]
    if kind == "norm":
        rows, width = s["rows"], s["width"]
        total = new(rows, width, dtype=out) if s["residual"] else None
        got = {"sum": total} if s["residual"] else {}
        if s["out"] == "plain":
            y = new(rows, width, dtype=out)
            qmv.qmv_rms_norm(dt, s["x"], width, s["res"], width, s["gain"], rows, width, EPS, total, "plain", y)
            return {"y": y, **got}
        y = new(qmv.qmv_act_mx_bytes("mxfp8", rows, width))
        qmv.qmv_rms_norm(dt, s["x"], width, s["res"], width, s["gain"], rows, width, EPS, total, "mxfp8", y)
        at, words = qmv.qmv_act_mx_scale_offset("mxfp8", rows, width), -(-width // 128)
        return {"codes": y[:rows * width].view(rows, width).view(torch.float8_e4m3fn),
                "scales": y[at:at + words * rows * 4].view(words, rows, 4).view(torch.float8_e8m0fnu), **got}
    if kind == "product":
        rows, n, k, fmt = s["rows"], s["n"], s["k"], s["fmt"]
        desc = qmv.wdesc(fmt, n, k)
        xq, y = new(qmv.qmv_act_mx_bytes(fmt, rows, k)), new(rows, n, dtype=out)
        qmv.qmv_quantize_act_mx(fmt, dt, s["x"], k, rows, k, xq)
        qmv.qmv_mx_product(desc, s["w"], xq, rows, None, dt, y)
        return {"y": y}
    tokens, top_k, experts = s["tokens"], s["top_k"], s["experts"]
    slots = tokens * top_k
    if kind == "routing":
        width, i32 = s["width"], torch.int32
        offsets, row_of_slot, slot_of_row = new(experts + 1, dtype=i32), new(slots, dtype=i32), new(slots, dtype=i32)
        ws = new(qmv.qmv_moe_sort_workspace_bytes(tokens, top_k, experts))
        xs, y = new(slots, width, dtype=out), new(tokens, width, dtype=out)
        qmv.qmv_moe_sort(s["ids"], tokens, top_k, experts, offsets, row_of_slot, slot_of_row, ws)
        qmv.qmv_moe_dispatch(dt, s["x"], width, tokens, top_k, width, row_of_slot, xs)
        qmv.qmv_moe_return(dt, s["ys"], s["weights"], tokens, top_k, width, row_of_slot, y, width)
        got = {"offsets": offsets, "slot_of_row": slot_of_row, "row_of_slot": row_of_slot, "xs": xs, "y": y}
        if s["train"]:
            dx, dys = new(tokens, width, dtype=out), new(slots, width, dtype=out)
            dweights = new(tokens, top_k, dtype=torch.float32)
            qmv.qmv_moe_dispatch_grad(dt, s["dxs"], tokens, top_k, width, row_of_slot, dx, width)
            qmv.qmv_moe_return_grad(dt, s["dy"], width, s["ys"], s["weights"], tokens, top_k, width, row_of_slot, dys, dweights)
            got |= {"dx": dx, "dys": dys, "dweights": dweights}
        return got
    hidden, inner, fmt = s["hidden"], s["inner"], s["fmt"]
    gate_up, down = qmv.wdesc(fmt, inner, hidden, experts), qmv.wdesc(fmt, hidden, inner, experts)
    ws = new(qmv.qmv_moe_prefill_layer_workspace_bytes(gate_up, down, tokens, top_k))
    y = new(tokens, hidden, dtype=out)
    qmv.qmv_moe_prefill_layer(gate_up, s["w_gate_up"], down, s["w_down"], dt, s["x"], hidden, s["ids"], s["weights"], tokens, top_k, ws, y)
    return {"y": y}


def run(state):
    return called(state) if own else plain(state)


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    kind, size = case["kind"], {"bf16": 2, "f16": 2, "f32": 4}[case["dtype"]]
    if kind == "norm":
        n = case["rows"] * case["width"]
        out = n * size if case["out"] == "plain" else n + n // 32
        return {"bytes": n * size * (3 if case["residual"] else 1) + out + case["width"] * size, "flops": 4 * n}
    if kind == "product":
        rows, n, k = case["rows"], case["n"], case["k"]
        matrix = n * k * BITS[case["fmt"]] // 8 + n * k // 32
        return {"bytes": rows * k * size + matrix + rows * n * size, "flops": 2 * rows * n * k}
    slots = case["tokens"] * case["top_k"]
    if kind == "routing":
        token, row, meta = case["tokens"] * case["width"] * size, slots * case["width"] * size, slots * 4
        once = 2 * token + 2 * row + 4 * meta
        # backward: dxs and dy in, dx and dys out, the rows of ys once more beside dy, the weights' gradients out
        return {"bytes": once + (2 * token + 2 * row + 2 * meta if case["train"] else 0),
                "flops": 2 * slots * case["width"] * (3 if case["train"] else 1)}
    hidden, inner = case["hidden"], case["inner"]
    one = hidden * inner * BITS[case["fmt"]] // 8 + hidden * inner // 32
    return {"bytes": 3 * one * min(case["experts"], slots) + 2 * case["tokens"] * hidden * size + slots * 8,
            "flops": 6 * slots * hidden * inner}


# ------------------------------------------------------------------ the definitions in 64 bits


def exponent(v):
    """floor(log2 v) of positive float64 values, from their bits."""
    return (v.view(torch.int64) >> 52) - 1023


def power(e):
    """2^e of whole e as float64, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def rounded64(x, fmt):
    """Element values and scales (both float64) of x [rows][k]: nearest element value, ties to the even code."""
    v = x.view(x.shape[0], -1, 32)
    top = v.abs().amax(-1)
    e = torch.where(top > 0, (exponent(top) - EMAX[fmt]).clamp(min=-127), -127)
    scale = power(e)
    a = (v.abs() / scale[..., None]).clamp(max=TOP[fmt])
    if fmt == "mxfp8":
        unit = power(exponent(a).clamp(min=-6) - 3)
        q = torch.round(a / unit) * unit
    else:
        middles = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device=DEV)
        i = torch.bucketize(a, middles)
        tie = a == middles[i.clamp(max=6)]
        q = torch.tensor(E2M1[:8], dtype=torch.float64, device=DEV)[i + (tie & (i % 2 == 1)).long()]
    return torch.where(v < 0, -q, q), scale


def matrix64(codes, scales, fmt):
    if fmt == "mxfp8":
        m, ex = (codes & 7).double(), codes >> 3 & 15
        v = torch.where(ex > 0, (8 + m) * power(ex.int() - 10), m * 2.0 ** -9)
        v = torch.where(codes >= 128, -v, v)
    else:
        both = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
        m, ex = (both & 1).double(), both >> 1 & 3
        v = torch.where(ex > 0, (2 + m) * power(ex.int() - 2), m * 0.5)
        v = torch.where(both >= 8, -v, v)
    return v * torch.repeat_interleave(power(scales.int() - 127), 32, -1)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "norm":
        v = s["x"].double()
        got = {}
        if case["residual"]:
            v = v + s["res"].double()
            got["sum"] = v
        y = v / torch.sqrt((v ** 2).sum(-1, keepdim=True) / case["width"] + EPS) * s["gain"].double()
        if case["out"] == "plain":
            return {"y": y, **got}
        q, scale = rounded64(y, "mxfp8")
        words = -(-case["width"] // 128)
        filled = torch.full((case["rows"], 4 * words), 2.0 ** -127, dtype=torch.float64, device=DEV)
        filled[:, :scale.shape[1]] = scale
        return {"codes": q.reshape(case["rows"], -1), "scales": filled.view(-1, words, 4).permute(1, 0, 2).contiguous(), **got}
    if kind == "product":
        q, scale = rounded64(s["x"].double(), case["fmt"])
        return {"y": (q * scale[..., None]).view(case["rows"], -1) @ matrix64(s["codes"][0], s["scales"][0], case["fmt"]).T}
    tokens, top_k, experts = case["tokens"], case["top_k"], case["experts"]
    ids = s["ids"].flatten().cpu().tolist()
    order = sorted(range(len(ids)), key=lambda i: (ids[i] if 0 <= ids[i] < experts else experts, i))
    slot = torch.tensor(order, device=DEV)
    live = torch.tensor([0 <= ids[i] < experts for i in order], device=DEV)
    weight = s["weights"].double().flatten()[slot] * live
    if kind == "routing":
        zero = torch.zeros(tokens, case["width"], dtype=torch.float64, device=DEV)
        got = {"offsets": None, "slot_of_row": None, "row_of_slot": None,
               "xs": s["x"].double()[slot // top_k] * live[:, None],
               "y": zero.index_add(0, slot // top_k, s["ys"].double() * weight[:, None])}
        if case["train"]:
            got["dx"] = zero.index_add(0, slot // top_k, s["dxs"].double() * live[:, None])
            got["dys"] = s["dy"].double()[slot // top_k] * weight[:, None]
            dw = torch.zeros(tokens * top_k, dtype=torch.float64, device=DEV)
            dw[slot] = (s["ys"].double() * s["dy"].double()[slot // top_k]).sum(1) * live
            got["dweights"] = dw.view(tokens, top_k)
        return got
    y = torch.zeros(tokens, case["hidden"], dtype=torch.float64, device=DEV)
    q, scale = rounded64(s["x"].double(), case["fmt"])
    x = (q * scale[..., None]).view(tokens, -1)
    at = 0
    for e in range(experts):
        n = ids.count(e)
        rows = slot[at:at + n]
        g = x[rows // top_k] @ matrix64(s["gate"][e], s["gate_scales"][e], case["fmt"]).T
        u = x[rows // top_k] @ matrix64(s["up"][e], s["up_scales"][e], case["fmt"]).T
        q, scale = rounded64(g * torch.sigmoid(g) * u, case["fmt"]) if n else (g[:, :, None], g[:, :1])
        h = (q * scale[..., None]).view(n, -1) if n else g
        y.index_add_(0, rows // top_k, h @ matrix64(s["down"][e], s["down_scales"][e], case["fmt"]).T * weight[at:at + n, None])
        at += n
    return {"y": y}
