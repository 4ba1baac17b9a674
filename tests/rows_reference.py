"""Plain 64-bit definitions of the many-row operators, for their tests: the
microscaled quantization of rows, products of codes and scales, the norm, the
sort by expert and the routed sums."""
import numpy as np

import oracle

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])
EMAX = {"mxfp4": 2, "mxfp8": 8}


def element_values(fmt):
    """The value of every code (NaN codes of E4M3 as NaN)."""
    if fmt == "mxfp4":
        return E2M1
    c = np.arange(256)
    m, e = c & 7, c >> 3 & 15
    v = np.where(e > 0, (8 + m) * 2.0 ** (e - 10.0), m * 2.0 ** -9)
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >= 128, -v, v)


def nearest_codes(v, fmt):
    """Codes of the nearest element values of v (float64), ties to the even code, saturating."""
    mags = element_values(fmt)[:8 if fmt == "mxfp4" else 127]
    a = np.minimum(np.abs(v), mags[-1])
    hi = np.clip(np.searchsorted(mags, a), 1, len(mags) - 1)
    lo = hi - 1
    up, down = mags[hi] - a, a - mags[lo]
    code = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    return (code + np.where(np.signbit(v), 8 if fmt == "mxfp4" else 128, 0)).astype(np.uint8)


def scale_bytes(v, fmt):
    """E8M0 bytes of groups v [..., 32] (float64)."""
    top = np.abs(v).max(-1)
    with np.errstate(invalid="ignore"):
        e = np.frexp(np.where(np.isfinite(top), top, 1.0))[1] - 1 - EMAX[fmt] + 127
    e = np.where(top > 0, np.clip(e, 0, 254), 0)
    return np.where(np.isfinite(top), e, 255).astype(np.uint8)


def quantize(x, fmt):
    """(codes [rows][K], scales [rows][K / 32]) of x (float64)."""
    v = np.asarray(x, dtype=np.float64).reshape(x.shape[0], -1, 32)
    e = scale_bytes(v, fmt)
    bad = (e == 255)[..., None]
    q = nearest_codes(np.where(bad, 0.0, v) * 2.0 ** (127.0 - e[..., None].astype(np.float64)), fmt)
    return np.where(bad, 0, q).astype(np.uint8).reshape(x.shape), e


def decode(codes, scales, fmt):
    """Values (float64) of codes [..., K] and scales [..., K / 32]."""
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return element_values(fmt)[codes] * np.repeat(s, 32, -1)


def pack_rows(codes, fmt):
    """Codes one a byte -> the canonical bytes of rows."""
    return codes if fmt == "mxfp8" else oracle.pack_nibbles(codes)


def act_buffer(codes, scales, fmt):
    """The library's activation buffer of codes [rows][K] and scales [rows][K / 32]."""
    rows, K = codes.shape
    body = pack_rows(codes, fmt).reshape(-1)
    at = -(-body.size // 128) * 128
    words = -(-K // 128)
    full = np.zeros((rows, 4 * words), dtype=np.uint8)
    full[:, :K // 32] = scales
    tail = np.ascontiguousarray(full.reshape(rows, words, 4).transpose(1, 0, 2)).reshape(-1)
    out = np.zeros(at + -(-tail.size // 16) * 16, dtype=np.uint8)
    out[:body.size] = body
    out[at:at + tail.size] = tail
    return out


def sort_slots(ids, n_experts):
    """(offsets, row_of_slot, slot_of_row) of ids [ntok][top_k]."""
    flat = np.asarray(ids).reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < n_experts), flat, n_experts)
    slot_of_row = np.argsort(key, kind="stable")
    row = np.empty(len(flat), dtype=np.int64)
    row[slot_of_row] = np.arange(len(flat))
    offsets = np.searchsorted(key[slot_of_row], np.arange(n_experts + 1))
    return offsets.astype(np.int32), np.where(key < n_experts, row, ~row).astype(np.int32), slot_of_row.astype(np.int32)


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g))
