"""The many-row operators against their 64-bit definitions.

Tolerances. Quantized codes and scales of given inputs, sorted orders and
copied rows are exact. Products are exact where every partial sum is a multiple
of one power of two below 2^24 of it (small scale ranges); otherwise the
suite's bound 1e-3 * sum|w x| holds for the fp32 result. fp32 sums of n terms
that are added one by one are within n * 2^-24 * sum|terms|. The norm's fp32
result is within 1e-5 relative (at most 64 terms a thread, a tree of 10 levels
and 6 more roundings: 80 * 2^-24 = 4.8e-6). SwiGLU in a product's epilogue is
within 2e-5 relative of the exact one of its sums: at |g| <= 80 the special
functions' exponential is within 2 + 1.16 * 80 = 95 units of 2^-23 (1.2e-5),
the division within 2, and two products follow. A quantized result of a value
known within d has a scale between those of the group's extremes and codes
between those of v - d and v + d at that scale."""
import numpy as np
import pytest
import torch

qmv = pytest.importorskip("bit_quantized_moe_gb300")
import oracle  # noqa: E402
import qmv_inputs as qi  # noqa: E402
import rows_reference as ref  # noqa: E402
from qmv_testutil import DEV, assert_close, assert_within, round_out, status_clean  # noqa: E402

pytestmark = pytest.mark.gpu

TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t.to(TORCH[dtype]) if dtype else t


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def buf(n):
    return torch.full((n,), 0xA5, dtype=torch.uint8, device=DEV)


def randn(seed, *shape):
    g = qi.rng(seed)
    return g.standard_normal(shape) * np.exp(0.5 * g.standard_normal(shape[-1:]))


def strided(values, dtype, extra):
    """Rows of `values` with `extra` elements between them, and their stride."""
    rows, K = values.shape
    t = torch.full((rows, K + extra), 7.0, dtype=TORCH[dtype], device=DEV)
    t[:, :K] = dev(values, dtype)
    return t, K + extra


def unpacked(fmt, xq, rows, K):
    c, s = qmv.qmv_act_mx_unpack(fmt, xq.cpu().numpy(), rows, K)
    return oracle.unpack_nibbles(c) if fmt == "mxfp4" else c, s


def padding_is_zero(fmt, xq, rows, K):
    """Scale bytes past K are zero."""
    words = -(-K // 128)
    at = qmv.qmv_act_mx_scale_offset(fmt, rows, K)
    tail = xq[at:at + words * rows * 4].view(words, rows, 4)[-1].cpu().numpy()
    used = K // 32 - 4 * (words - 1)
    return not tail[:, used:].any()


# --- quantization ---------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,K,extra", [(1, 32, 0), (3, 96, 0), (5, 160, 3), (17, 2880, 8), (130, 1056, 0)])
def test_quantize(fmt, dtype, rows, K, extra):
    x, ld = strided(randn(rows + K, rows, K), dtype, extra)
    xq = buf(qmv.qmv_act_mx_bytes(fmt, rows, K))
    qmv.qmv_quantize_act_mx(fmt, dtype, x, ld, rows, K, xq)
    codes, scales = unpacked(fmt, xq, rows, K)
    want_c, want_s = ref.quantize(host(x[:, :K]), fmt)
    assert np.array_equal(scales, want_s) and np.array_equal(codes, want_c)
    assert padding_is_zero(fmt, xq, rows, K)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_quantize_special_groups(fmt):
    """Zeros, subnormals, the largest numbers, ties, saturation, infinities and NaN, each in a group of its own."""
    top = ref.element_values(fmt)[7 if fmt == "mxfp4" else 126]
    rows = np.zeros((12, 32), dtype=np.float32)
    rows[1, 3] = 1e-45
    rows[2] = 2.0 ** -126
    rows[3, :4] = [3.4e38, -3.4e38, 1e30, 1.0]
    rows[4, :8] = [4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, -0.25]
    rows[5, :3] = [1.99 * 2 ** 5, -1.99 * 2 ** 5, top]
    rows[6, 9] = np.inf
    rows[7, 9] = -np.inf
    rows[8, 31] = np.nan
    rows[9, :2] = [1.0, 2.0 ** -40]
    rows[10] = -0.0
    rows[11, :2] = [2.0 ** -120, 2.0 ** -126]
    xq = buf(qmv.qmv_act_mx_bytes(fmt, 12, 32))
    qmv.qmv_quantize_act_mx(fmt, "f32", dev(rows), 32, 12, 32, xq)
    codes, scales = unpacked(fmt, xq, 12, 32)
    want_c, want_s = ref.quantize(rows.astype(np.float64), fmt)
    assert scales[6:9].reshape(-1).tolist() == [255] * 3 and not codes[6:9].any()
    assert np.array_equal(scales, want_s) and np.array_equal(codes, want_c)


# --- norm -----------------------------------------------------------------------

def quantized_close(codes, scales, y, err, fmt):
    """Codes and scales that the quantization of some values within err of y can have."""
    v, d = y.reshape(y.shape[0], -1, 32), err.reshape(y.shape[0], -1, 32)
    lo_s = ref.scale_bytes(np.maximum(np.abs(v) - d, 0), fmt)
    hi_s = ref.scale_bytes(np.abs(v) + d, fmt)
    assert (lo_s <= scales).all() and (scales <= hi_s).all()
    inv = 2.0 ** (127.0 - scales[..., None].astype(np.float64))
    val = ref.element_values(fmt)
    lo, hi = val[ref.nearest_codes((v - d) * inv, fmt)], val[ref.nearest_codes((v + d) * inv, fmt)]
    got = val[codes].reshape(v.shape)
    assert ((lo <= got) & (got <= hi)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("out", ["plain", "mxfp8", "mxfp4", "q8"])
@pytest.mark.parametrize("rows,K,extra,residual", [
    (1, 32, 0, True), (9, 256, 0, True), (3, 288, 5, True), (2, 1024, 0, False), (5, 1056, 8, True), (3, 2880, 0, True),
    (2, 4128, 1, False), (2, 7168, 0, True), (1, 8224, 0, True), (1, 32768, 0, True), (1, 65536, 0, False)])
def test_rms_norm(dtype, out, rows, K, extra, residual):
    x, ldx = strided(randn(K, rows, K), dtype, extra)
    res, ldr = strided(randn(K + 1, rows, K), dtype, 2 * extra) if residual else (None, 0)
    gain = dev(1 + 0.1 * randn(K + 2, K), dtype)
    total = torch.full_like(res, 7.0) if residual else None
    fmt = out if out.startswith("mx") else None
    n = {"plain": rows * K * x.element_size(), "q8": qmv.qmv_act_q8_bytes(rows, K)}.get(out) or qmv.qmv_act_mx_bytes(fmt, rows, K)
    y = buf(n)
    qmv.qmv_rms_norm(dtype, x, ldx, res, ldr, gain, rows, K, 1e-5, total, out, y)
    s = host(x[:, :K]) + (host(res[:, :K]) if residual else 0)
    want = s / np.sqrt((s ** 2).mean(-1, keepdims=True) + 1e-5) * host(gain)
    if residual:
        assert_within(host(total[:, :K]), s, np.abs(s) * 2.0 ** -24, dtype, "sum")
        assert (total[:, K:] == 7.0).all()
    err = 1e-5 * np.abs(want)
    if out == "plain":
        assert_within(host(y.view(TORCH[dtype]).view(rows, K)), want, err, dtype, "y")
    elif out == "q8":
        q, d = qmv.qmv_act_q8_unpack(y.cpu().numpy(), rows, K)
        d = oracle.f16_bits_to_f64(d)
        v, e = want.reshape(rows, -1, 32), err.reshape(rows, -1, 32)
        exact_d = np.abs(v).max(-1) / 127
        assert (np.abs(d - exact_d) <= exact_d * (2.0 ** -11 + 1.1e-5) + 2.0 ** -25).all()
        # q is the rounding of y / d for the unrounded d
        assert (np.abs(q.reshape(v.shape) - v / exact_d[..., None]) <= 0.5 + 127 * 2.5e-5).all()
    else:
        codes, scales = unpacked(fmt, y, rows, K)
        quantized_close(codes, scales, want, err, fmt)
        assert padding_is_zero(fmt, y, rows, K)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,K,extra", [(4, 1, 0), (3, 7, 2), (513, 31, 0), (2, 2881, 0), (1, 8191, 1)])
def test_rms_norm_odd_widths(dtype, rows, K, extra):
    x, ldx = strided(randn(K, rows, K), dtype, extra)
    res, ldr = strided(randn(K + 1, rows, K), dtype, extra)
    gain = dev(1 + 0.1 * randn(K + 2, K), dtype)
    y, total = torch.empty(rows, K, dtype=TORCH[dtype], device=DEV), torch.zeros_like(res)
    qmv.qmv_rms_norm(dtype, x, ldx, res, ldr, gain, rows, K, 1e-6, total, "plain", y)
    s = host(x[:, :K]) + host(res[:, :K])
    want = s / np.sqrt((s ** 2).mean(-1, keepdims=True) + 1e-6) * host(gain)
    assert_within(host(y), want, 1e-5 * np.abs(want), dtype, "y")
    assert_within(host(total[:, :K]), s, np.abs(s) * 2.0 ** -24, dtype, "sum")


def test_rms_norm_in_place_and_zero_row():
    """The sum may replace the residual; a row of zeros gives zeros (with eps), not NaN."""
    rows, K = 6, 2880
    x, res = dev(randn(1, rows, K), "bf16"), dev(randn(2, rows, K), "bf16")
    x[3] = 0
    res[3] = 0
    gain = dev(np.ones(K), "bf16")
    s = host(x) + host(res)
    y = torch.empty_like(x)
    qmv.qmv_rms_norm("bf16", x, K, res, K, gain, rows, K, 1e-5, res, "plain", y)
    assert_within(host(res), s, np.abs(s) * 2.0 ** -24, "bf16", "sum in place")
    want = s / np.sqrt((s ** 2).mean(-1, keepdims=True) + 1e-5)
    assert_within(host(y), want, 1e-5 * np.abs(want), "bf16", "y")
    assert not host(y)[3].any()


# --- products -------------------------------------------------------------------

def random_codes(g, fmt, shape):
    return qi.format_codes(g, fmt, shape)


def packed_weights(fmt, codes, scales):
    """codes [E][N][K] -> (descriptor, device buffer)."""
    E, N, K = codes.shape
    desc = qmv.wdesc(fmt, N, K, E)
    return desc, dev(qmv.qmv_pack_weights(desc, oracle.pack_codes(fmt, codes), scales))


# Scales of the exact products: E2M1 products are multiples of 2^-2 below 36, at scales of 2^-1 .. 2^1 each
# multiples of 2^-4 below 144; 2880 of them stay under 2^19 = 2^23 units. E4M3 products are multiples of 2^-18 and
# below 2^18: exact codes are drawn from the integers up to 15 instead (multiples of 1, at scales 1/2 .. 2 of 2^-2,
# below 900 each).
def exact_inputs(g, fmt, shape):
    codes = random_codes(g, fmt, shape)
    if fmt == "mxfp8":
        ints = ref.nearest_codes(np.arange(-15, 16, dtype=np.float64), "mxfp8")
        codes = ints[g.integers(0, len(ints), size=shape)]
    return codes, g.integers(126, 129, size=shape[:-1] + (shape[-1] // 32,), dtype=np.uint8)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("rows,N,K", [
    (1, 1, 32), (1, 8, 64), (3, 17, 96), (127, 192, 128), (128, 193, 256), (129, 40, 288), (5, 200, 1024), (130, 390, 1056),
    (64, 64, 1120), (33, 96, 1280), (300, 72, 2080), (257, 576, 2880)])
def test_product_exact(fmt, rows, N, K):
    """Every code and scale in its place: sums that fp32 holds exactly come out exactly."""
    g = qi.rng(rows * 7 + N + K)
    wc, ws = exact_inputs(g, fmt, (1, N, K))
    xc, xs = exact_inputs(g, fmt, (rows, K))
    desc, w = packed_weights(fmt, wc, ws)
    y = torch.full((rows + 1, N), 7.0, dtype=torch.float32, device=DEV)
    qmv.qmv_mx_product(desc, w, dev(ref.act_buffer(xc, xs, fmt)), rows, None, "f32", y)
    want = ref.decode(xc, xs, fmt) @ ref.decode(wc[0], ws[0], fmt).T
    assert np.abs(want).max() < 2 ** 20
    assert np.array_equal(host(y[:rows]), want)
    assert (y[rows] == 7.0).all() and status_clean()


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,N,K", [(1, 2880, 2880), (17, 516, 2048), (200, 1032, 1056), (129, 57, 7168)])
def test_product_of_quantized_rows(fmt, out, rows, N, K):
    g = qi.rng(rows + N + K)
    wc, ws = random_codes(g, fmt, (1, N, K)), qi.e8m0(g, (1, N, K // 32), 107, 122)
    desc, w = packed_weights(fmt, wc, ws)
    x = dev(randn(N, rows, K), "bf16")
    xq = buf(qmv.qmv_act_mx_bytes(fmt, rows, K))
    qmv.qmv_quantize_act_mx(fmt, "bf16", x, K, rows, K, xq)
    y = torch.empty(rows, N, dtype=TORCH[out], device=DEV)
    qmv.qmv_mx_product(desc, w, xq, rows, None, out, y)
    xv, wv = ref.decode(*ref.quantize(host(x), fmt), fmt), ref.decode(wc[0], ws[0], fmt)
    assert_close(host(y), xv @ wv.T, np.abs(xv) @ np.abs(wv).T, out, "product")


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_product_scale_range(fmt):
    """Scales far apart from row to row, at both ends of the byte's range, and NaN scales that stay in their row and column."""
    rows, N, K = 140, 200, 96
    g = qi.rng(5)
    wc, ws = exact_inputs(g, fmt, (1, N, K))
    xc, xs = exact_inputs(g, fmt, (rows, K))
    ws[0] = np.where(np.arange(N) % 2 == 0, 30, 220)[:, None] + g.integers(0, 2, size=(N, 3))
    xs[:] = np.where(np.arange(rows) % 2 == 0, 130, 120)[:, None]
    xs[4], ws[0, 6] = 0, 254
    xs[7, 1], ws[0, 9, 2] = 255, 255
    desc, w = packed_weights(fmt, wc, ws)
    y = torch.empty(rows, N, dtype=torch.float32, device=DEV)
    qmv.qmv_mx_product(desc, w, dev(ref.act_buffer(xc, xs, fmt)), rows, None, "f32", y)
    xv, wv = ref.decode(xc, xs, fmt), ref.decode(wc[0], ws[0], fmt)
    got = host(y)
    assert np.isnan(got[7]).all() and np.isnan(got[:, 9]).all()
    keep = np.ix_(np.delete(np.arange(rows), 7), np.delete(np.arange(N), 9))
    want, absum = (xv[keep[0].ravel()] @ wv[keep[1].ravel()].T, np.abs(xv[keep[0].ravel()]) @ np.abs(wv[keep[1].ravel()]).T)
    normal = absum < 2.0 ** 127
    assert np.isfinite(got[keep][normal]).all()
    # sums below the normal numbers may lose their last places
    assert (np.abs(got[keep] - want)[normal] <= 1e-3 * absum[normal] + 2.0 ** -120).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("counts", [[1], [0, 3, 0], [128, 0, 129, 1], [5, 300, 2, 0, 0, 77, 128], [0, 0], [1] * 40,
                                    [300, 0, 513, 129], [256, 1, 1000], [700],
                                    [33, 64, 65, 97, 31], [320, 449, 257, 193]])
def test_grouped_product(fmt, counts):
    """Rows of each expert by its own matrix; rows of no expert stay as they are."""
    E, N, K, tail = len(counts), 200, 1184, 5
    rows = sum(counts) + tail
    g = qi.rng(rows)
    wc, ws = exact_inputs(g, fmt, (E, N, K))
    xc, xs = exact_inputs(g, fmt, (rows, K))
    desc, w = packed_weights(fmt, wc, ws)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    y = torch.full((rows, N), 7.0, dtype=torch.float32, device=DEV)
    qmv.qmv_mx_product(desc, w, dev(ref.act_buffer(xc, xs, fmt)), rows, dev(offsets), "f32", y)
    xv = ref.decode(xc, xs, fmt)
    want = np.full((rows, N), 7.0)
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        want[a:b] = xv[a:b] @ ref.decode(wc[e], ws[e], fmt).T
    assert np.array_equal(host(y), want) and status_clean()


@pytest.mark.parametrize("counts", [[140, 3, 0, 33], [300, 290, 5, 600]])
def test_grouped_product_keeps_rows_apart(counts):
    """E4M3 rows of NaN codes, and rows with NaN scales, leave the rows after them alone, in their own tile and in later ones."""
    E, N, K, rows = len(counts), 136, 416, sum(counts)
    g = qi.rng(8)
    wc, ws = exact_inputs(g, "mxfp8", (E, N, K))
    xc, xs = exact_inputs(g, "mxfp8", (rows, K))
    bad = np.zeros(rows, dtype=bool)
    bad[:counts[0]:2] = True
    bad[-counts[-1]:-counts[-1] + 7] = True
    xc[bad], xs[:counts[0]:6] = 0x7f, 255
    desc, w = packed_weights("mxfp8", wc, ws)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    y = torch.full((rows, N), 7.0, dtype=torch.float32, device=DEV)
    qmv.qmv_mx_product(desc, w, dev(ref.act_buffer(xc, xs, "mxfp8")), rows, dev(offsets), "f32", y)
    got = host(y)
    assert np.isnan(got[bad]).all()
    xv = ref.decode(np.where(bad[:, None], 0, xc), np.where(bad[:, None], 0, xs), "mxfp8")
    for e in range(E):
        at = np.arange(offsets[e], offsets[e + 1])
        at = at[~bad[at]]
        assert np.array_equal(got[at], xv[at] @ ref.decode(wc[e], ws[e], "mxfp8").T), e


def test_grouped_product_of_many_experts():
    """The most experts that a call takes, most of them with no row or one."""
    E, N, K = qmv.MAX_SORT_EXPERTS, 24, 96
    g = qi.rng(12)
    counts = g.integers(0, 3, size=E)
    counts[17], counts[E - 1] = 150, 40
    rows = int(counts.sum())
    wc, ws = exact_inputs(g, "mxfp4", (E, N, K))
    xc, xs = exact_inputs(g, "mxfp4", (rows, K))
    desc, w = packed_weights("mxfp4", wc, ws)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    y = torch.empty(rows, N, dtype=torch.float32, device=DEV)
    qmv.qmv_mx_product(desc, w, dev(ref.act_buffer(xc, xs, "mxfp4")), rows, dev(offsets), "f32", y)
    expert = np.repeat(np.arange(E), counts)
    want = np.einsum("rk,rnk->rn", ref.decode(xc, xs, "mxfp4"), ref.decode(wc, ws, "mxfp4")[expert])
    assert np.array_equal(host(y), want) and status_clean()


@pytest.mark.parametrize("offsets", [[0, 5, 3, 9], [-7, 4, 4, 1000], [6, 6, 6, 6], [20, 30, 40, 50]])
def test_grouped_product_takes_offsets_into_its_rows(offsets):
    """Offsets that do not ascend or name rows that are not there: each expert's range is taken into [0, nrows], and what a
    descending pair names is nothing."""
    rows, E, N, K = 9, 3, 40, 64
    g = qi.rng(4)
    wc, ws = exact_inputs(g, "mxfp4", (E, N, K))
    xc, xs = exact_inputs(g, "mxfp4", (rows, K))
    desc, w = packed_weights("mxfp4", wc, ws)
    y = torch.full((rows + 2, N), 7.0, dtype=torch.float32, device=DEV)
    qmv.qmv_mx_product(desc, w, dev(ref.act_buffer(xc, xs, "mxfp4")), rows, dev(np.array(offsets, dtype=np.int32)), "f32", y)
    torch.cuda.synchronize()
    assert (y[rows:] == 7.0).all() and status_clean()


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_product_longest_k(fmt):
    """K at its limit: 256 or 512 steps a tile; entries of one magnitude, so that every partial sum is exact."""
    rows, N, K = 5, 24, 65536
    g = qi.rng(6)
    one = 2 if fmt == "mxfp4" else 0x38           # 1.0
    sign = 8 if fmt == "mxfp4" else 0x80
    wc = (one + sign * g.integers(0, 2, size=(1, N, K))).astype(np.uint8)
    xc = (one + sign * g.integers(0, 2, size=(rows, K))).astype(np.uint8)
    ws, xs = g.integers(126, 129, size=(1, N, K // 32), dtype=np.uint8), np.full((rows, K // 32), 127, dtype=np.uint8)
    desc, w = packed_weights(fmt, wc, ws)
    y = torch.empty(rows, N, dtype=torch.float32, device=DEV)
    qmv.qmv_mx_product(desc, w, dev(ref.act_buffer(xc, xs, fmt)), rows, None, "f32", y)
    assert np.array_equal(host(y), ref.decode(xc, xs, fmt) @ ref.decode(wc[0], ws[0], fmt).T)


def test_rows_past_32_bits():
    """Rows whose elements and bytes lie past 2^32 in every buffer: norm, quantization, product, dispatch and return."""
    rows, K, N = 70000, 65536, 40
    last = slice(rows - 3, rows)
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device=DEV)
    x[last] = dev(randn(1, 3, K), "bf16")
    xv = host(x[last])
    y = torch.empty_like(x)
    qmv.qmv_rms_norm("bf16", x, K, None, 0, torch.ones(K, dtype=torch.bfloat16, device=DEV), rows, K, 1e-5, None, "plain", y)
    want = xv / np.sqrt((xv ** 2).mean(-1, keepdims=True) + 1e-5)
    assert_within(host(y[last]), want, 1e-5 * np.abs(want), "bf16", "norm")
    xq = buf(qmv.qmv_act_mx_bytes("mxfp8", rows, K))
    qmv.qmv_quantize_act_mx("mxfp8", "bf16", x, K, rows, K, xq)
    codes, scales = ref.quantize(xv, "mxfp8")
    assert np.array_equal(xq[(rows - 3) * K:rows * K].view(3, K).cpu().numpy(), codes)
    g = qi.rng(2)
    wc, ws = exact_inputs(g, "mxfp8", (1, N, K))
    desc, w = packed_weights("mxfp8", wc, ws)
    out = torch.empty(rows, N, dtype=torch.float32, device=DEV)
    qmv.qmv_mx_product(desc, w, xq, rows, None, "f32", out)
    v, wv = ref.decode(codes, scales, "mxfp8"), ref.decode(wc[0], ws[0], "mxfp8")
    assert_close(host(out[last]), v @ wv.T, np.abs(v) @ np.abs(wv).T, "f32", "product")
    assert not out[:rows - 3].any()
    del xq
    row = torch.arange(rows - 1, -1, -1, dtype=torch.int32, device=DEV)   # one slot a token, in reverse
    qmv.qmv_moe_dispatch("bf16", x, K, rows, 1, K, row, y)
    assert torch.equal(y[:3], x[last].flip(0)) and not y[3:].any()
    back = torch.empty_like(x)
    qmv.qmv_moe_return("bf16", y, torch.full((rows, 1), 2.0, device=DEV), rows, 1, K, row, back, K)
    assert torch.equal(back[last], 2 * x[last]) and not back[:rows - 3].any()


@pytest.mark.parametrize("fmt,h_fmt", [("mxfp4", "mxfp4"), ("mxfp4", "mxfp8"), ("mxfp8", "mxfp4"), ("mxfp8", "mxfp8")])
@pytest.mark.parametrize("counts,N,K", [([1], 32, 32), ([0, 130, 3], 96, 96), ([129, 7], 224, 1056), ([257], 2880, 288),
                                        ([0, 400, 5, 200], 96, 1056)])
def test_gate_up_swiglu(fmt, h_fmt, counts, N, K):
    """Gate and up sums are exact here, so h is known within the special functions' error."""
    E, rows = len(counts), sum(counts)
    g = qi.rng(rows + N)
    gc, gs = exact_inputs(g, fmt, (E, N, K))
    uc, us = exact_inputs(g, fmt, (E, N, K))
    xc, xs = exact_inputs(g, fmt, (rows, K))
    gs = (gs - (9 if fmt == "mxfp8" else 4)).astype(np.uint8)   # g of a few units, where silu bends
    desc = qmv.wdesc(fmt, N, K, E)
    w = dev(qmv.qmv_pack_gate_up(desc, oracle.pack_codes(fmt, gc), gs, oracle.pack_codes(fmt, uc), us))
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    hq = buf(qmv.qmv_act_mx_bytes(h_fmt, rows, N))
    qmv.qmv_mx_gate_up_swiglu(desc, w, dev(ref.act_buffer(xc, xs, fmt)), rows, dev(offsets) if E > 1 else None, h_fmt, hq)
    xv = ref.decode(xc, xs, fmt)
    h = np.empty((rows, N))
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        gate, up = xv[a:b] @ ref.decode(gc[e], gs[e], fmt).T, xv[a:b] @ ref.decode(uc[e], us[e], fmt).T
        h[a:b] = ref.silu(gate) * up
    codes, scales = unpacked(h_fmt, hq, rows, N)
    # silu below -80 (e^-80 = 2e-35) is outside the special functions' bound: absolute there
    quantized_close(codes, scales, h, 2e-5 * np.abs(h) + 1e-25, h_fmt)
    assert padding_is_zero(h_fmt, hq, rows, N) and status_clean()


# --- routing --------------------------------------------------------------------

def drawn_ids(seed, ntok, top_k, E, drop):
    g = qi.rng(seed)
    ids = np.stack([g.permutation(E)[:top_k] if E >= top_k else g.integers(0, E, top_k) for _ in range(ntok)])
    bad = g.random(ids.shape) < drop
    return np.where(bad, g.choice([-1, E, 2 ** 31 - 1, -2 ** 31], size=ids.shape), ids).astype(np.int32)


def sorted_on_gpu(ids, E):
    n = ids.size
    offsets = torch.full((E + 1,), -9, dtype=torch.int32, device=DEV)
    row, slot = (torch.full((max(n, 4),), -9, dtype=torch.int32, device=DEV) for _ in range(2))
    qmv.qmv_moe_sort(dev(ids) if n else row, ids.shape[0], ids.shape[1], E, offsets, row, slot)
    return offsets, row[:n], slot[:n]


@pytest.mark.parametrize("ntok,top_k,E,drop", [
    (0, 2, 8, 0), (1, 1, 1, 0), (1, 1, 1, 1.0), (1, 8, 256, 0), (7, 3, 5, 0.3), (33, 4, 32, 0), (500, 2, 1024, 0.1),
    (1025, 4, 3, 0), (3001, 5, 33, 0.05), (8193, 8, 257, 0.01), (20000, 1, 1, 0)])
def test_sort(ntok, top_k, E, drop):
    ids = drawn_ids(ntok, ntok, top_k, E, drop) if ntok else np.zeros((0, top_k), dtype=np.int32)
    offsets, row, slot = sorted_on_gpu(ids, E)
    want = ref.sort_slots(ids, E)
    for got, w, what in zip((offsets, row, slot), want, ("offsets", "row_of_slot", "slot_of_row")):
        assert np.array_equal(got.cpu().numpy(), w), what


def test_sort_one_popular_expert():
    """Every slot at one expert, and at the last of 1024."""
    for e in (0, 1023):
        ids = np.full((5000, 2), e, dtype=np.int32)
        offsets, row, slot = sorted_on_gpu(ids, 1024)
        assert np.array_equal(row.cpu().numpy(), np.arange(10000)) and np.array_equal(slot.cpu().numpy(), np.arange(10000))
        assert offsets.cpu().numpy().tolist() == [0] * (e + 1) + [10000] * (1024 - e)


ROUTES = [(1, 1, 4, 8, 0), (5, 3, 4, 40, 0.3), (33, 8, 32, 2880, 0.1), (3, 2, 3, 7, 0), (130, 4, 8, 129, 0.2),
          (2, 2, 4, 7168, 1.0), (9, 5, 16, 1026, 0.1), (6, 4, 8, 9000, 0.0)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("extra", [0, 8, 3])
@pytest.mark.parametrize("ntok,top_k,E,K,drop", ROUTES)
def test_dispatch_and_return(dtype, extra, ntok, top_k, E, K, drop):
    ids = drawn_ids(K, ntok, top_k, E, drop)
    offsets, row, slot = sorted_on_gpu(ids, E)
    r = row.cpu().numpy()
    flat, valid = np.where(r >= 0, r, ~r), r >= 0
    n = ntok * top_k
    x, ld = strided(randn(1, ntok, K), dtype, extra)
    xs = torch.full((n, K), 7.0, dtype=TORCH[dtype], device=DEV)
    qmv.qmv_moe_dispatch(dtype, x, ld, ntok, top_k, K, row, xs)
    want = np.zeros((n, K))
    want[flat] = np.where(valid[:, None], np.repeat(host(x[:, :K]), top_k, 0), 0)
    assert np.array_equal(host(xs), want)

    ys = dev(randn(2, n, K), dtype)
    ys[dev(flat[~valid]).long()] = float("nan")          # what a dropped slot's row holds is not read
    weights = dev(np.abs(randn(3, ntok, top_k)).astype(np.float32))
    y = torch.full((ntok, K + extra), 7.0, dtype=TORCH[dtype], device=DEV)
    qmv.qmv_moe_return(dtype, ys, weights, ntok, top_k, K, row, y, ld)
    terms = np.where(valid[:, None], host(ys)[flat], 0) * host(weights).reshape(-1, 1)
    terms = terms.reshape(ntok, top_k, K)
    assert_within(host(y[:, :K]), terms.sum(1), (top_k + 1) * 2.0 ** -24 * np.abs(terms).sum(1), dtype, "y")
    assert (y[:, K:] == 7.0).all()

    dx = torch.full((ntok, K + extra), 7.0, dtype=TORCH[dtype], device=DEV)
    qmv.qmv_moe_dispatch_grad(dtype, ys, ntok, top_k, K, row, dx, ld)
    terms = np.where(valid[:, None], host(ys)[flat], 0).reshape(ntok, top_k, K)
    assert_within(host(dx[:, :K]), terms.sum(1), (top_k + 1) * 2.0 ** -24 * np.abs(terms).sum(1), dtype, "dx")
    assert (dx[:, K:] == 7.0).all()

    dy, ld = strided(randn(4, ntok, K), dtype, extra)
    dys = torch.full((n, K), 7.0, dtype=TORCH[dtype], device=DEV)
    dw = torch.full((ntok, top_k), 7.0, dtype=torch.float32, device=DEV)
    qmv.qmv_moe_return_grad(dtype, dy, ld, ys, weights, ntok, top_k, K, row, dys, dw)
    d = np.repeat(host(dy[:, :K]), top_k, 0)
    want = np.zeros((n, K))
    want[flat] = np.where(valid[:, None], host(weights).reshape(-1, 1) * d, 0)
    assert_within(host(dys), want, np.abs(want) * 2.0 ** -24, dtype, "dys")
    prod = np.where(valid[:, None], host(ys)[flat], 0) * d
    got = host(dw).reshape(-1)
    assert (np.abs(got - prod.sum(1)) <= (K / 32 + 16) * 2.0 ** -24 * np.abs(prod).sum(1)).all()
    assert not got[~valid].any()


@pytest.mark.parametrize("K", [64, 9])
def test_rows_that_the_call_does_not_have(K):
    """Entries of row_of_slot past the call's rows are neither written to nor read from; the others do their work."""
    ntok, top_k = 3, 2
    n = ntok * top_k
    row = dev(np.array([0, 6, ~7, 2, 1000000, ~3], dtype=np.int32))
    x = dev(randn(1, ntok, K), "f32")
    xs = torch.full((n + 2, K), 7.0, dtype=torch.float32, device=DEV)
    qmv.qmv_moe_dispatch("f32", x, K, ntok, top_k, K, row, xs)
    want = torch.full_like(xs, 7.0)
    want[0], want[2], want[3] = x[0], x[1], 0
    assert torch.equal(xs, want)
    ys, w, dy = dev(randn(2, n + 2, K), "f32"), torch.ones(ntok, top_k, device=DEV), dev(randn(3, ntok, K), "f32")
    y, dys, dw = torch.empty(ntok, K, device=DEV), torch.full_like(xs, 7.0), torch.empty(ntok, top_k, device=DEV)
    qmv.qmv_moe_return("f32", ys, w, ntok, top_k, K, row, y, K)
    assert torch.equal(y, torch.stack([ys[0], ys[2], torch.zeros_like(ys[0])]))
    qmv.qmv_moe_return_grad("f32", dy, K, ys, w, ntok, top_k, K, row, dys, dw)
    want = torch.full_like(xs, 7.0)
    want[0], want[2], want[3] = dy[0], dy[1], 0
    assert torch.equal(dys, want) and (dw.flatten()[[1, 2, 4, 5]] == 0).all() and (dw.flatten()[[0, 3]] != 0).all()
    if K % 32 == 0:
        size = qmv.qmv_act_mx_bytes("mxfp8", n, K)
        xq = torch.full((size + 256,), 0xA5, dtype=torch.uint8, device=DEV)
        qmv.qmv_moe_dispatch_mx("mxfp8", "f32", x, K, ntok, top_k, K, row, xq)
        assert (xq[size:] == 0xA5).all() and (xq[K:2 * K] == 0xA5).all() and not xq[3 * K:4 * K].any()


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("dtype,ntok,top_k,E,K,drop", [("bf16", 1, 1, 2, 32, 0), ("f16", 33, 4, 8, 2880, 0.2), ("f32", 9, 8, 16, 96, 0.1),
                                                       ("bf16", 300, 2, 4, 160, 0)])
def test_dispatch_mx_equals_dispatch_then_quantize(fmt, dtype, ntok, top_k, E, K, drop):
    ids = drawn_ids(7, ntok, top_k, E, drop)
    _, row, _ = sorted_on_gpu(ids, E)
    n = ntok * top_k
    x, ld = strided(randn(1, ntok, K), dtype, 8)
    xs = torch.empty(n, K, dtype=TORCH[dtype], device=DEV)
    qmv.qmv_moe_dispatch(dtype, x, ld, ntok, top_k, K, row, xs)
    size = qmv.qmv_act_mx_bytes(fmt, n, K)
    a, b = buf(size), buf(size)
    qmv.qmv_quantize_act_mx(fmt, dtype, xs, K, n, K, a)
    qmv.qmv_moe_dispatch_mx(fmt, dtype, x, ld, ntok, top_k, K, row, b)
    assert torch.equal(a, b)


def test_gradients_against_differences():
    """The forward is linear in x, ys and the weights, so a finite step along any direction changes
    <y, dy> by exactly the gradient's inner product with it (fp32 rounding aside)."""
    ntok, top_k, E, K = 19, 3, 8, 64
    ids = drawn_ids(3, ntok, top_k, E, 0.2)
    _, row, _ = sorted_on_gpu(ids, E)
    n = ntok * top_k
    new = lambda *s: torch.empty(*s, dtype=torch.float32, device=DEV)  # noqa: E731
    ys, w, dy = dev(randn(1, n, K), "f32"), dev(randn(2, ntok, top_k), "f32"), dev(randn(3, ntok, K), "f32")

    def loss(ys, w):
        y = new(ntok, K)
        qmv.qmv_moe_return("f32", ys, w, ntok, top_k, K, row, y, K)
        return (y.double() * dy.double()).sum().item()

    dys, dw = new(n, K), new(ntok, top_k)
    qmv.qmv_moe_return_grad("f32", dy, K, ys, w, ntok, top_k, K, row, dys, dw)
    for seed in range(4):
        a, b = dev(randn(10 + seed, n, K), "f32"), dev(randn(20 + seed, ntok, top_k), "f32")
        scale = (ys.abs().max() * dy.abs().max() * w.abs().max()).item() * n * K
        assert abs(loss(ys + a, w) - loss(ys - a, w) - 2 * (dys.double() * a.double()).sum().item()) <= 1e-6 * scale
        assert abs(loss(ys, w + b) - loss(ys, w - b) - 2 * (dw.double() * b.double()).sum().item()) <= 1e-6 * scale

    c, x = dev(randn(5, n, K), "f32"), dev(randn(6, ntok, K), "f32")
    dx = new(ntok, K)
    qmv.qmv_moe_dispatch_grad("f32", c, ntok, top_k, K, row, dx, K)

    def lin(x):
        xs = new(n, K)
        qmv.qmv_moe_dispatch("f32", x, K, ntok, top_k, K, row, xs)
        return (xs.double() * c.double()).sum().item()

    a = dev(randn(7, ntok, K), "f32")
    assert abs(lin(x + a) - lin(x - a) - 2 * (dx.double() * a.double()).sum().item()) <= 1e-6 * n * K * c.abs().max().item()


# --- the layer ------------------------------------------------------------------

def layer_case(gu_fmt, dn_fmt, dtype, ntok, top_k, E, K, N, N_down, drop, seed=0):
    g = qi.rng(seed + ntok + K)
    lo, hi = {"mxfp4": (112, 122), "mxfp8": (107, 117)}[gu_fmt]
    gc, gs = random_codes(g, gu_fmt, (E, N, K)), qi.e8m0(g, (E, N, K // 32), lo, hi)
    uc, us = random_codes(g, gu_fmt, (E, N, K)), qi.e8m0(g, (E, N, K // 32), lo, hi)
    lo, hi = {"mxfp4": (112, 122), "mxfp8": (107, 117)}[dn_fmt]
    dc, ds = random_codes(g, dn_fmt, (E, N_down, N)), qi.e8m0(g, (E, N_down, N // 32), lo, hi)
    gu = qmv.wdesc(gu_fmt, N, K, E)
    w_gu = dev(qmv.qmv_pack_gate_up(gu, oracle.pack_codes(gu_fmt, gc), gs, oracle.pack_codes(gu_fmt, uc), us))
    dn, w_dn = packed_weights(dn_fmt, dc, ds)
    ids = drawn_ids(seed, ntok, top_k, E, drop)
    weights = np.abs(randn(seed + 3, ntok, top_k)).astype(np.float32)
    x = dev(0.25 * randn(seed + 4, ntok, K), dtype)
    return gu, w_gu, dn, w_dn, x, ids, dev(weights), (gc, gs, uc, us, dc, ds)


def split_layer(gu, w_gu, dn, w_dn, dtype, x, ids, weights, E, K, N, N_down, ys_type):
    """The layer's calls one by one: (h buffer, the experts' rows, row_of_slot)."""
    (ntok, top_k), n = ids.shape, ids.size
    offsets, row, _ = sorted_on_gpu(ids, E)
    xq, hq = buf(qmv.qmv_act_mx_bytes(gu.fmt, n, K)), buf(qmv.qmv_act_mx_bytes(dn.fmt, n, N))
    ys = torch.zeros(n, N_down, dtype=TORCH[ys_type], device=DEV)
    qmv.qmv_moe_dispatch_mx(gu.fmt, dtype, x, K, ntok, top_k, K, row, xq)
    qmv.qmv_mx_gate_up_swiglu(gu, w_gu, xq, n, offsets, dn.fmt, hq)
    qmv.qmv_mx_product(dn, w_dn, hq, n, offsets, ys_type, ys)
    return hq, ys, row


@pytest.mark.parametrize("gu_fmt,dn_fmt,dtype,ntok,top_k,E,K,N,N_down,drop", [
    ("mxfp4", "mxfp4", "bf16", 1, 1, 1, 32, 32, 1, 0), ("mxfp4", "mxfp8", "bf16", 5, 2, 4, 96, 160, 40, 0.3),
    ("mxfp8", "mxfp8", "f16", 140, 2, 3, 288, 96, 200, 0), ("mxfp8", "mxfp4", "bf16", 33, 4, 32, 1056, 224, 264, 0.1),
    ("mxfp4", "mxfp4", "f16", 3, 2, 4, 64, 64, 64, 1.0)])
def test_prefill_layer(gu_fmt, dn_fmt, dtype, ntok, top_k, E, K, N, N_down, drop):
    """The layer against the definition, within the h codes' freedom: h as the gate/up call quantizes it, then its
    products, weighted, within the bounds of the product and of an fp32 sum."""
    gu, w_gu, dn, w_dn, x, ids, weights, (gc, gs, uc, us, dc, ds) = layer_case(gu_fmt, dn_fmt, dtype, ntok, top_k, E, K, N,
                                                                               N_down, drop)
    n = ntok * top_k
    ws = buf(qmv.qmv_moe_prefill_layer_workspace_bytes(gu, dn, ntok, top_k))
    y = torch.full((ntok, N_down), 7.0, dtype=TORCH[dtype], device=DEV)
    qmv.qmv_moe_prefill_layer(gu, w_gu, dn, w_dn, dtype, x, K, dev(ids), weights, ntok, top_k, ws, y)
    hq, _, _ = split_layer(gu, w_gu, dn, w_dn, dtype, x, ids, weights, E, K, N, N_down, "f32")

    off, r, slot = ref.sort_slots(ids, E)
    hc, hs = unpacked(dn_fmt, hq, n, N)
    xv = ref.decode(*ref.quantize(host(x), gu_fmt), gu_fmt)
    want, bound = np.zeros((ntok, N_down)), np.zeros((ntok, N_down))
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        tok = slot[a:b] // top_k
        wg, wu, wd = ref.decode(gc[e], gs[e], gu_fmt), ref.decode(uc[e], us[e], gu_fmt), ref.decode(dc[e], ds[e], dn_fmt)
        gate, up = xv[tok] @ wg.T, xv[tok] @ wu.T
        eg, eu = 1e-3 * np.abs(xv[tok]) @ np.abs(wg).T, 1e-3 * np.abs(xv[tok]) @ np.abs(wu).T
        h = ref.silu(gate) * up
        quantized_close(hc[a:b], hs[a:b], h, 1.1 * eg * (np.abs(up) + eu) + np.abs(ref.silu(gate)) * eu + 2e-5 * np.abs(h) + 1e-25,
                        dn_fmt)
        hv = ref.decode(hc[a:b], hs[a:b], dn_fmt)
        prod, absum = hv @ wd.T, np.abs(hv) @ np.abs(wd).T
        wt = host(weights).reshape(-1)[slot[a:b], None]
        np.add.at(want, tok, wt * prod)
        np.add.at(bound, tok, wt * (1e-3 * absum + top_k * 2.0 ** -23 * np.abs(prod)))
    assert_within(host(y), want, bound, dtype, "layer")
    assert status_clean()


@pytest.mark.parametrize("gu_fmt,dn_fmt,dtype,ntok,top_k,E,K,N,N_down,drop,ys_type", [
    ("mxfp4", "mxfp8", "bf16", 130, 4, 8, 288, 160, 264, 0.1, "f32"),
    ("mxfp8", "mxfp4", "f16", 1100, 2, 4, 96, 64, 4000, 0.05, "f16"), ("mxfp4", "mxfp4", "bf16", 4200, 2, 16, 64, 96, 1024, 0, "bf16")])
def test_prefill_layer_is_its_parts(gu_fmt, dn_fmt, dtype, ntok, top_k, E, K, N, N_down, drop, ys_type):
    """The layer equals its calls made one by one, bit for bit: with the experts' rows in fp32 up to 32 MB of them, in the
    output's type above. fp32 rows are weighted here in float64 and compared as a sum of fp32 terms."""
    gu, w_gu, dn, w_dn, x, ids, weights, _ = layer_case(gu_fmt, dn_fmt, dtype, ntok, top_k, E, K, N, N_down, drop)
    assert (ntok * top_k * N_down * 4 <= 32 << 20) == (ys_type == "f32")
    ws = buf(qmv.qmv_moe_prefill_layer_workspace_bytes(gu, dn, ntok, top_k))
    y = torch.full((ntok, N_down), 7.0, dtype=TORCH[dtype], device=DEV)
    qmv.qmv_moe_prefill_layer(gu, w_gu, dn, w_dn, dtype, x, K, dev(ids), weights, ntok, top_k, ws, y)
    _, ys, row = split_layer(gu, w_gu, dn, w_dn, dtype, x, ids, weights, E, K, N, N_down, ys_type)
    if ys_type != "f32":
        y2 = torch.empty_like(y)
        qmv.qmv_moe_return(dtype, ys, weights, ntok, top_k, N_down, row, y2, N_down)
        assert torch.equal(y, y2)
    else:
        r = row.cpu().numpy().reshape(ntok, top_k)
        terms = np.where((r >= 0)[..., None], host(ys)[np.where(r >= 0, r, ~r)], 0) * host(weights)[..., None]
        assert_within(host(y), terms.sum(1), (top_k + 1) * 2.0 ** -24 * np.abs(terms).sum(1), dtype, "layer")
    assert status_clean()


def test_layer_on_its_own_stream_and_in_a_graph():
    """Enqueued on a stream of its own, and captured once and replayed on new inputs in the same buffers."""
    args = layer_case("mxfp4", "mxfp4", "bf16", 40, 4, 8, 288, 96, 200, 0.1)
    gu, w_gu, dn, w_dn, x, ids, weights, _ = args
    ids = dev(ids)
    ws = buf(qmv.qmv_moe_prefill_layer_workspace_bytes(gu, dn, 40, 4))

    def run(y, stream=None):
        qmv.qmv_moe_prefill_layer(gu, w_gu, dn, w_dn, "bf16", x, 288, ids, weights, 40, 4, ws, y, stream)

    want, got = (torch.empty(40, 200, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    run(want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    run(got, s)
    s.synchronize()
    assert torch.equal(want, got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        run(got)
    x.copy_(dev(0.25 * randn(99, 40, 288), "bf16"))
    ids.copy_(dev(drawn_ids(99, 40, 4, 8, 0.3)))
    run(want)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(want, got) and status_clean()


def test_same_bits_every_run():
    args = layer_case("mxfp4", "mxfp8", "bf16", 300, 2, 5, 416, 160, 264, 0.05)
    gu, w_gu, dn, w_dn, x, ids, weights, _ = args
    ids = dev(ids)
    outs = []
    for _ in range(3):
        ws = buf(qmv.qmv_moe_prefill_layer_workspace_bytes(gu, dn, 300, 2))
        outs.append(torch.empty(300, 264, dtype=torch.bfloat16, device=DEV))
        qmv.qmv_moe_prefill_layer(gu, w_gu, dn, w_dn, "bf16", x, 416, ids, weights, 300, 2, ws, outs[-1])
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
