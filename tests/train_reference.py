"""Plain 64-bit definitions of the router with its balance loss, and of E4M3 with a scale for each block of 128, for
their tests."""
import numpy as np

import rows_reference as ref


def f32(v):
    return np.asarray(v, dtype=np.float32).astype(np.float64)


# --- router -----------------------------------------------------------------------

def scores(l, score):
    """(scores, scores as shares of their sum; 0 in rows of -infinities) of logits l [tokens][experts]."""
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if score == "softmax":
            top = l.max(1, keepdims=True)
            e = np.where(l == -np.inf, 0.0, np.exp(l - np.where(top == -np.inf, 0.0, top)))
            total = e.sum(1, keepdims=True)
            p = np.where(total == 0, 0.0, e / total)
            return p, p
        s = 1 / (1 + np.exp(-l))
        # shares from logarithms, in range where the scores are not
        log = -np.logaddexp(0, -l)
        top = log.max(1, keepdims=True)
        e = np.where(l == -np.inf, 0.0, np.exp(log - np.where(top == -np.inf, 0.0, top)))
        total = e.sum(1, keepdims=True)
        return s, np.where(total == 0, 0.0, e / total)


def quotients(l, ids, score):
    """Each chosen score over the sum of the row's chosen ones (0 for slots without an expert)."""
    at = np.take_along_axis(l, np.maximum(ids, 0), 1)
    log = np.where(ids >= 0, at if score == "softmax" else -np.logaddexp(0, -at), -np.inf)
    top = log.max(1, keepdims=True)
    with np.errstate(invalid="ignore"):
        e = np.where(log == -np.inf, 0.0, np.exp(log - np.where(top == -np.inf, 0.0, top)))
        total = e.sum(1, keepdims=True)
        return np.where(total == 0, 0.0, e / np.where(total == 0, 1.0, total))


def route(l, live, top_k, score, renorm, scale):
    """(ids, weights) by the definition; rows with a NaN (softmax: or +infinity) included."""
    tokens, experts = l.shape
    bad = np.isnan(l).any(1) | ((l == np.inf).any(1) if score == "softmax" else False)
    order = np.argsort(np.where(np.isnan(l), 0, -l), axis=1, kind="stable")[:, :top_k]
    ids = np.where(np.take_along_axis(l, order, 1) == -np.inf, -1, order)
    if renorm:
        w = quotients(l, ids, score)
    else:
        w = np.take_along_axis(scores(l, score)[0], np.maximum(ids, 0), 1)
    w = scale * np.where(ids >= 0, w, 0.0)
    ids = np.where(bad[:, None], np.arange(top_k)[None], ids)
    w = np.where(bad[:, None], np.nan, w)
    return np.where(live[:, None], ids, -1).astype(np.int32), np.where(live[:, None], w, 0.0)


def balance(l, live, ids, top_k, score):
    """(counts [experts + 1], means, loss)."""
    experts = l.shape[1]
    live = live & ~(l == -np.inf).all(1)
    tokens = int(live.sum())
    used = ids[live]
    counts = np.bincount(used[(used >= 0) & (used < experts)].ravel(), minlength=experts)
    share = scores(l, score)[1]
    means = share[live].sum(0) / tokens if tokens else np.zeros(experts)
    f = counts / (top_k * tokens) if tokens else np.zeros(experts)
    return np.append(counts, tokens).astype(np.int32), means, experts * (f * means).sum()


def router_grad(l, live, ids, dweights, counts, dloss, top_k, score, renorm, scale):
    """(d logits, the sum of the magnitudes of its terms)."""
    tokens, experts = l.shape
    s, share = scores(l, score)
    other = 1 - s if score == "sigmoid" else np.ones_like(l)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            other = 1 / (1 + np.exp(l))
    d, size = np.zeros_like(l), np.zeros_like(l)
    valid = (ids >= 0) & (ids < experts)
    at = np.where(valid, ids, 0)
    rows = np.broadcast_to(np.arange(tokens)[:, None], ids.shape)
    if dweights is not None:
        g = np.where(valid, scale * dweights, 0.0)
        if renorm:
            q = quotients(l, np.where(valid, ids, -1), score)
            inner, mags = (g * q).sum(1, keepdims=True), (np.abs(g) * q).sum(1, keepdims=True)
            np.add.at(d, (rows, at), np.where(valid, q * (g - inner), 0.0))
            np.add.at(size, (rows, at), np.where(valid, q * (np.abs(g) + mags), 0.0))
            d, size = d * other, size * other
        else:
            chosen = np.take_along_axis(s, at, 1)
            np.add.at(d, (rows, at), g * chosen)
            np.add.at(size, (rows, at), np.abs(g) * chosen)
            if score == "softmax":
                d = d - s * (g * chosen).sum(1, keepdims=True)
                size = size + s * (np.abs(g) * chosen).sum(1, keepdims=True)
            else:
                d, size = d * other, size * other
    if counts is not None and counts[-1] > 0:
        f = counts[:-1] / (top_k * counts[-1])
        c = dloss * experts / counts[-1]
        inner = (share * f).sum(1, keepdims=True)
        d = d + c * share * (f - inner) * other
        size = size + abs(c) * share * (f + inner) * other
    keep = live[:, None]
    return np.where(keep, d, 0.0), np.where(keep, size, 0.0)


# --- blocks of 128 ------------------------------------------------------------------

FLOOR = 2.0 ** -116


def scales_of(top):
    """(scale, inverse) of blocks with these maxima (float64): NaN and 0 for one with an infinity or a NaN."""
    bad = ~np.isfinite(top)
    a = np.maximum(np.where(bad, 0.0, top), FLOOR)
    return np.where(bad, np.nan, f32(a / 448)), np.where(bad, 0.0, f32(448 / a))


def codes_of(x, inverse):
    with np.errstate(invalid="ignore"):
        v = np.where(inverse == 0, 0.0, x * inverse)
    return ref.nearest_codes(f32(v), "mxfp8")


def quantize_rows(x):
    """(codes [rows][K], scales [rows][ceil(K / 128)]) of x (float64)."""
    rows, K = x.shape
    v = np.pad(x, ((0, 0), (0, -K % 128))).reshape(rows, -1, 128)
    with np.errstate(invalid="ignore"):
        scale, inverse = scales_of(np.abs(v).max(-1))
    return codes_of(v, inverse[..., None]).reshape(rows, -1)[:, :K], scale


def quantize_weights(w):
    """(codes, scales [experts][ceil(N / 128)][ceil(K / 128)]) of w [experts][N][K] (float64)."""
    E, N, K = w.shape
    v = np.pad(w, ((0, 0), (0, -N % 128), (0, -K % 128))).reshape(E, -(-N // 128), 128, -(-K // 128), 128)
    with np.errstate(invalid="ignore"):
        scale, inverse = scales_of(np.abs(v).max((2, 4)))
    codes = codes_of(v, inverse[:, :, None, :, None]).reshape(E, v.shape[1] * 128, -1)
    return codes[:, :N, :K], scale


def decode_rows(codes, scales):
    return ref.element_values("mxfp8")[codes] * np.repeat(scales.astype(np.float64), 128, 1)[:, :codes.shape[1]]


def decode_weights(codes, scales):
    E, N, K = codes.shape
    s = np.repeat(np.repeat(scales.astype(np.float64), 128, 1)[:, :N], 128, 2)[:, :, :K]
    return ref.element_values("mxfp8")[codes] * s


def act_buffer(codes, scales):
    """The library's activation buffer."""
    rows, K = codes.shape
    wide = -(-K // 16) * 16
    body = np.pad(codes, ((0, 0), (0, wide - K))).reshape(-1)
    at = -(-body.size // 128) * 128
    blocks = scales.shape[1]
    tail = np.pad(scales.astype(np.float32), ((0, 0), (0, -blocks % 4))).view(np.uint8).reshape(-1)
    out = np.zeros(at + tail.size, dtype=np.uint8)
    out[:body.size] = body
    out[at:at + tail.size] = tail
    return out


def ranges(offsets, rows, experts):
    """[(first row, end)] of each expert: offsets taken into the rows, none below an earlier one."""
    if offsets is None:
        return [(0, rows)]
    got, reached = [], 0
    for e in range(experts):
        lo = max(reached, min(int(offsets[e]), rows))
        reached = max(lo, min(int(offsets[e + 1]), rows))
        got.append((lo, reached))
    return got
