"""E4M3 with a scale for each block of 128: quantization, products and their gradients against the 64-bit definitions.

Tolerances. Codes and scales are exact. Sums that fp32 holds exactly come out exactly: integers up to 15 with scales that are
powers of two. Otherwise a block's sum is the tensor cores', whose additions truncate: at most 128 addends lose 2^-23 of
the largest partial sum each, 2^-16 of the sum of magnitudes; scaling and adding the blocks adds (blocks + 3) * 2^-24. The
weights' gradient adds products of 16-bit numbers, exact in fp32, in the same way. An output of 16 bits is the fp32
result rounded to nearest (assert_within)."""
import threading

import numpy as np
import pytest
import torch

qmv = pytest.importorskip("bit_quantized_moe_gb300")
import qmv_inputs as qi  # noqa: E402
import rows_reference as ref  # noqa: E402
import train_reference as tr  # noqa: E402
from qmv_testutil import DEV, assert_within, status_clean  # noqa: E402

pytestmark = pytest.mark.gpu

TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t.to(TORCH[dtype]) if dtype else t


def host(t):
    return t.double().cpu().numpy()


def buf(n):
    return torch.full((n,), 0xA5, dtype=torch.uint8, device=DEV)


def randn(seed, *shape):
    g = qi.rng(seed)
    return g.standard_normal(shape) * np.exp(0.5 * g.standard_normal(shape[-1:]))


def bound(depth, absum):
    return (2.0 ** -16 + (depth / 128 + 4) * 2.0 ** -24) * absum


def strided(values, dtype, extra):
    rows, K = values.shape
    t = torch.full((rows, K + extra), 7.0, dtype=TORCH[dtype], device=DEV)
    t[:, :K] = dev(values, dtype)
    return t, K + extra


INTS = ref.nearest_codes(np.arange(-15, 16, dtype=np.float64), "mxfp8")


def exact_rows(g, rows, K):
    """Codes of integers up to 15 and scales 1/2, 1 or 2."""
    return INTS[g.integers(0, 31, size=(rows, K))], 2.0 ** g.integers(-1, 2, size=(rows, -(-K // 128)))


def exact_weights(g, E, N, K):
    return INTS[g.integers(0, 31, size=(E, N, K))], 2.0 ** g.integers(-1, 2, size=(E, -(-N // 128), -(-K // 128)))


# --- quantization ---------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,K,extra", [(1, 1, 0), (3, 100, 0), (5, 128, 3), (17, 2880, 8), (130, 1000, 0), (2, 129, 0), (3, 65536, 0)])
def test_quantize_rows(dtype, rows, K, extra):
    x, ld = strided(randn(rows + K, rows, K), dtype, extra)
    xq = buf(qmv.qmv_act_b128_bytes(rows, K))
    qmv.qmv_quantize_act_b128(dtype, x, ld, rows, K, xq)
    codes, scales = qmv.qmv_act_b128_unpack(xq.cpu().numpy(), rows, K)
    wc, ws = tr.quantize_rows(host(x[:, :K]))
    assert np.array_equal(scales, ws.astype(np.float32)) and np.array_equal(codes, wc)
    wide = -(-K // 16) * 16   # rows are padded with zeros
    assert not xq[:rows * wide].view(rows, wide)[:, K:].any()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_quantize_rows_of_special_blocks(dtype):
    """Zeros, the types' ends, ties, blocks below the floor, infinities and NaN, each in a block beside an ordinary one."""
    rows = np.ones((14, 256))
    rows[0, :128] = 0
    rows[1, :128] = -0.0
    rows[2, 5] = 3e38 if dtype != "f16" else 65504
    rows[3, :128] = 2.0 ** -130 if dtype != "f16" else 2.0 ** -24
    rows[4, :128] = np.linspace(-2.0 ** -117, 2.0 ** -117, 128)
    rows[5, 7] = np.inf
    rows[6, 127] = -np.inf
    rows[7, 0] = np.nan
    rows[8, :128] = np.arange(128) * 448 / 127
    rows[9, :8] = [448, 1 / 512, 3 / 1024, 1 / 1024, 5 / 1024, 17, 19, 21]   # ties at scale 1
    rows[10, :3] = [448, 1e-10, -1e-10]
    rows[11, :128] = 448 * 1.06
    rows[12, 128:] = np.nan
    rows[13] = -448
    x = dev(rows, dtype)
    xq = buf(qmv.qmv_act_b128_bytes(14, 256))
    qmv.qmv_quantize_act_b128(dtype, x, 256, 14, 256, xq)
    codes, scales = qmv.qmv_act_b128_unpack(xq.cpu().numpy(), 14, 256)
    wc, ws = tr.quantize_rows(host(x))
    assert np.array_equal(scales, ws.astype(np.float32), equal_nan=True) and np.array_equal(codes, wc)
    assert np.isnan(scales[5:8, 0]).all() and not codes[5:8, :128].any() and np.isfinite(scales[5:8, 1]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("E,N,K", [(1, 1, 16), (2, 128, 128), (3, 130, 272), (1, 1000, 144), (5, 7, 2880)])
def test_quantize_weights(dtype, E, N, K):
    w = dev(randn(N + K, E, N, K), dtype)
    w[0, 0, 0] = 100
    if E > 1:
        w[1, -1, -1] = float("nan")
    codes, scales = buf(E * N * K + 16), torch.full((E * -(-N // 128) * -(-K // 128) + 1,), 7.0, device=DEV)
    qmv.qmv_quantize_weights_b128(dtype, w, E, N, K, codes, scales)
    wc, ws = tr.quantize_weights(host(w))
    assert np.array_equal(codes[:E * N * K].cpu().numpy().reshape(E, N, K), wc) and (codes[E * N * K:] == 0xA5).all()
    assert np.array_equal(scales[:-1].cpu().numpy(), ws.astype(np.float32).ravel(), equal_nan=True) and scales[-1] == 7.0


# --- products -------------------------------------------------------------------

SHAPES = [(1, 1, 16), (1, 8, 64), (2, 128, 128), (3, 17, 96), (16, 256, 512), (17, 130, 400), (127, 192, 128), (128, 193, 256),
          (129, 40, 288), (5, 200, 1024), (130, 390, 1056), (64, 64, 1120), (33, 96, 1280), (300, 72, 2080), (257, 576, 2880),
          (256, 256, 128), (513, 264, 144), (1, 1000, 7168), (9, 7168, 272), (640, 520, 656)]


@pytest.mark.parametrize("rows,N,K", SHAPES)
def test_product_exact(rows, N, K):
    """Every code and scale in its place: sums that fp32 holds exactly come out exactly. At K = 7168 they stay below
    900 * 7168 < 2^23 units of 1/4."""
    g = qi.rng(rows * 7 + N + K)
    wc, ws = exact_weights(g, 1, N, K)
    xc, xs = exact_rows(g, rows, K)
    y = torch.full((rows + 1, N), 7.0, dtype=torch.float32, device=DEV)
    qmv.qmv_b128_product(dev(wc), dev(ws, "f32"), 1, N, K, dev(tr.act_buffer(xc, xs)), rows, None, "f32", y)
    assert np.array_equal(host(y[:rows]), tr.decode_rows(xc, xs) @ tr.decode_weights(wc, ws)[0].T)
    assert (y[rows] == 7.0).all() and status_clean()


@pytest.mark.parametrize("rows,N,K", SHAPES + [(40, 1001, 144), (3, 7170, 32)])
def test_grad_x_exact(rows, N, K):
    g = qi.rng(rows * 5 + N + K)
    wc, ws = exact_weights(g, 1, N, K)
    dc, ds = exact_rows(g, rows, N)
    dx = torch.full((rows + 1, K), 7.0, dtype=torch.float32, device=DEV)
    qmv.qmv_b128_grad_x(dev(wc), dev(ws, "f32"), 1, N, K, dev(tr.act_buffer(dc, ds)), rows, None, "f32", dx)
    assert np.array_equal(host(dx[:rows]), tr.decode_rows(dc, ds) @ tr.decode_weights(wc, ws)[0])
    assert (dx[rows] == 7.0).all() and status_clean()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,N,K", [(1, 1, 16), (1, 8, 64), (3, 17, 96), (64, 128, 128), (63, 256, 256), (65, 130, 400),
                                      (128, 257, 272), (300, 72, 2080), (1000, 520, 144), (129, 1001, 64)])
def test_grad_w_exact(dtype, rows, N, K):
    """Integers up to 15: sums below 225 * 1000 < 2^18."""
    g = qi.rng(rows + N + K)
    dy, ld_dy = strided(g.integers(-15, 16, size=(rows, N)).astype(np.float64), dtype, -N % 8 + 8 * (N % 2))
    x, ldx = strided(g.integers(-15, 16, size=(rows, K)).astype(np.float64), dtype, 8)
    dw = torch.full((N + 1, K), 7.0, dtype=torch.float32, device=DEV)
    qmv.qmv_b128_grad_w(dtype, dy, ld_dy, x, ldx, 1, N, K, rows, None, "f32", dw)
    assert np.array_equal(host(dw[:N]), host(dy[:, :N]).T @ host(x[:, :K]))
    assert (dw[N] == 7.0).all() and status_clean()


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,N,K", [(1, 2880, 2880), (17, 516, 2048), (200, 1032, 1056), (129, 57, 7168), (600, 392, 528)])
def test_linear_and_gradients_of_random_numbers(out, rows, N, K):
    """The whole of a step: both quantizers, the product and its gradients."""
    act = "bf16" if out == "f32" else out
    w, x, dy = dev(randn(1, 1, N, K) * 0.03, act), dev(randn(2, rows, K), act), strided(randn(3, rows, N), act, -N % 8)
    codes, scales = buf(N * K), torch.empty(-(-N // 128), -(-K // 128), device=DEV)
    qmv.qmv_quantize_weights_b128(act, w, 1, N, K, codes, scales)
    wv = tr.decode_weights(*tr.quantize_weights(host(w)))[0]
    xv = tr.decode_rows(*tr.quantize_rows(host(x)))
    y, ws = torch.empty(rows, N, dtype=TORCH[act], device=DEV), buf(qmv.qmv_b128_linear_workspace_bytes(rows, K))
    qmv.qmv_b128_linear(codes, scales, 1, N, K, act, x, K, rows, None, ws, y)
    assert_within(host(y), xv @ wv.T, bound(K, np.abs(xv) @ np.abs(wv).T), act, "y")
    y2, xq = torch.empty(rows, N, dtype=TORCH[out], device=DEV), buf(qmv.qmv_act_b128_bytes(rows, K))
    qmv.qmv_quantize_act_b128(act, x, K, rows, K, xq)
    qmv.qmv_b128_product(codes, scales, 1, N, K, xq, rows, None, out, y2)
    assert_within(host(y2), xv @ wv.T, bound(K, np.abs(xv) @ np.abs(wv).T), out, "y")
    dyq, dx = buf(qmv.qmv_act_b128_bytes(rows, N)), torch.empty(rows, K, dtype=TORCH[out], device=DEV)
    qmv.qmv_quantize_act_b128(act, dy[0], dy[1], rows, N, dyq)
    qmv.qmv_b128_grad_x(codes, scales, 1, N, K, dyq, rows, None, out, dx)
    dv = tr.decode_rows(*tr.quantize_rows(host(dy[0][:, :N])))
    assert_within(host(dx), dv @ wv, bound(N, np.abs(dv) @ np.abs(wv)), out, "dx")
    dw = torch.empty(N, K, dtype=TORCH[out], device=DEV)
    qmv.qmv_b128_grad_w(act, dy[0], dy[1], x, K, 1, N, K, rows, None, out, dw)
    d = host(dy[0][:, :N])
    assert_within(host(dw), d.T @ host(x), bound(rows, np.abs(d).T @ np.abs(host(x))), out, "dw")
    assert status_clean()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,N,K,extra", [(1, 7, 16, 0), (1, 300, 2880, 3), (3, 129, 400, 1), (16, 2880, 288, 8), (15, 130, 7168, 0), (9, 64, 144, 5)])
def test_linear_is_quantize_and_product(dtype, rows, N, K, extra):
    """Rows quantized within the product's launch give the bits of the two calls; special blocks among them, any stride."""
    g = qi.rng(rows + N)
    wc, ws = exact_weights(g, 1, N, K)
    v = randn(rows + K, rows, K)
    v[0, :min(K, 128)] = 0
    v[-1, 0] = 3e4
    if rows > 3:
        v[1, 3], v[2, K - 1], v[3, 5] = np.nan, np.inf, -np.inf
    x, ld = strided(v, dtype, extra)
    w, wsd = dev(wc), dev(ws, "f32")
    y, y2 = torch.full((rows + 1, N), 7.0, dtype=TORCH[dtype], device=DEV), torch.empty(rows, N, dtype=TORCH[dtype], device=DEV)
    space = buf(qmv.qmv_b128_linear_workspace_bytes(rows, K))
    qmv.qmv_b128_linear(w, wsd, 1, N, K, dtype, x, ld, rows, None, space, y)
    xq = buf(qmv.qmv_act_b128_bytes(rows, K))
    qmv.qmv_quantize_act_b128(dtype, x, ld, rows, K, xq)
    qmv.qmv_b128_product(w, wsd, 1, N, K, xq, rows, None, dtype, y2)
    assert torch.equal(torch.nan_to_num(y[:rows], 123.0), torch.nan_to_num(y2, 123.0)) and torch.equal(y[:rows].isnan(), y2.isnan())
    assert (y[rows] == 7.0).all() and status_clean()


@pytest.mark.parametrize("counts", [[1], [0, 3, 0], [16, 0, 17, 1], [0, 40, 2, 0, 0, 7], [0, 0], [1] * 40])
def test_grouped_linear_is_quantize_and_product(counts):
    E, N, K, tail = len(counts), 200, 1184, 2
    rows = sum(counts) + tail
    g = qi.rng(rows)
    wc, ws = exact_weights(g, E, N, K)
    x = dev(randn(rows, rows, K), "bf16")
    offsets = dev(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))
    y, y2 = (torch.full((rows, N), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    qmv.qmv_b128_linear(dev(wc), dev(ws, "f32"), E, N, K, "bf16", x, K, rows, offsets, buf(qmv.qmv_b128_linear_workspace_bytes(rows, K)), y)
    xq = buf(qmv.qmv_act_b128_bytes(rows, K))
    qmv.qmv_quantize_act_b128("bf16", x, K, rows, K, xq)
    qmv.qmv_b128_product(dev(wc), dev(ws, "f32"), E, N, K, xq, rows, offsets, "bf16", y2)
    assert torch.equal(y, y2) and status_clean()


def grouped(counts, N, K, tail, seed):
    """Exact operands of experts with so many rows, and `tail` rows of none."""
    g = qi.rng(seed)
    rows = sum(counts) + tail
    wc, ws = exact_weights(g, len(counts), N, K)
    xc, xs = exact_rows(g, rows, K)
    dc, ds = exact_rows(g, rows, N)
    return rows, wc, ws, xc, xs, dc, ds, np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def check_grouped(E, N, K, rows, wc, ws, xc, xs, dc, ds, offsets, exact=True):
    """All three grouped products against the definition; rows of no expert stay as they are."""
    w, wsd, od = dev(wc), dev(ws, "f32"), dev(offsets)
    xv, dv, wv = tr.decode_rows(xc, xs), tr.decode_rows(dc, ds), tr.decode_weights(wc, ws)
    y, dx = torch.full((rows, N), 7.0, device=DEV), torch.full((rows, K), 7.0, device=DEV)
    qmv.qmv_b128_product(w, wsd, E, N, K, dev(tr.act_buffer(xc, xs)), rows, od, "f32", y)
    qmv.qmv_b128_grad_x(w, wsd, E, N, K, dev(tr.act_buffer(dc, ds)), rows, od, "f32", dx)
    ints = ref.element_values("mxfp8")
    di, xi = np.zeros((rows, -(-N // 8) * 8)), ints[xc]
    di[:, :N] = ints[dc]
    di[:, N:] = np.nan   # never read
    dw = torch.full((E, N, K), 7.0, device=DEV)
    qmv.qmv_b128_grad_w("bf16", dev(di, "bf16"), di.shape[1], dev(xi, "bf16") if K % 8 == 0 else None, K, E, N, K, rows, od, "f32", dw)
    wy, wdx, wdw = np.full((rows, N), 7.0), np.full((rows, K), 7.0), np.zeros((E, N, K))
    for e, (a, b) in enumerate(tr.ranges(offsets, rows, E)):
        wy[a:b], wdx[a:b], wdw[e] = xv[a:b] @ wv[e].T, dv[a:b] @ wv[e], ints[dc][a:b].T @ xi[a:b]
    for got, want, what in ((y, wy, "y"), (dx, wdx, "dx"), (dw, wdw, "dw")):
        assert np.array_equal(host(got), want, equal_nan=True), what
    assert status_clean()


@pytest.mark.parametrize("N,K", [(200, 1184), (129, 64), (256, 384)])
@pytest.mark.parametrize("counts", [[1], [0, 3, 0], [128, 0, 129, 1], [5, 300, 2, 0, 0, 77, 128], [0, 0], [1] * 40,
                                    [300, 0, 513, 129], [256, 1, 1000], [33, 64, 65, 97, 31], [2, 0, 1, 0, 0, 3]])
def test_grouped_products(counts, N, K):
    check_grouped(len(counts), N, K, *grouped(counts, N, K, 5, sum(counts)))


@pytest.mark.parametrize("offsets", [[-5, 10, 4, 60, 1000], [0, 0, 0, 0, 0], [300, 200, 100, 50, 0], [7, 7, 90, 40, 77],
                                     [-2147483648, 3, 2147483647, 5, 2147483647]])
def test_offsets_out_of_range_or_order(offsets):
    data = list(grouped([30, 40, 0, 20], 136, 144, 5, 3))
    data[-1] = np.array(offsets, np.int32)
    check_grouped(4, 136, 144, *data)


def test_products_of_many_experts():
    """The most experts that a call takes, most of them with no row or one."""
    E, N, K = qmv.MAX_SORT_EXPERTS, 24, 96
    g = qi.rng(12)
    counts = g.integers(0, 3, size=E)
    counts[17], counts[E - 1] = 150, 40
    check_grouped(E, N, K, *grouped([int(c) for c in counts], N, K, 3, 5))


@pytest.mark.parametrize("rows,N,K", [(33, 1000, 1040), (63, 130, 2064), (64, 2049, 144), (65, 264, 7168), (97, 1290, 272), (128, 1160, 1168)])
def test_products_of_tens_of_rows(rows, N, K):
    """Tiles of 64 rows, their depth shared by clusters of two to eight and of one."""
    check_grouped(1, N, K, *grouped([rows], N, K, 0, rows))


@pytest.mark.parametrize("counts,N,K", [([200], 7168, 2816), ([129], 2817, 7168), ([300], 4101, 4112), ([256], 4000, 4368), ([511], 4360, 2896),
                                        ([200, 100], 2600, 4112), ([0, 260], 3000, 5136), ([1000], 1032, 4112)])
def test_products_of_hundreds_of_rows(counts, N, K):
    """Two pairs of CTAs share a tile's depth, unequally where its blocks are odd in number or not of fours."""
    check_grouped(len(counts), N, K, *grouped(counts, N, K, 3 if len(counts) > 1 else 0, N))


@pytest.mark.parametrize("counts,N,K", [([4000], 1304, 1168), ([3841], 1001, 2064), ([5120], 1408, 656), ([1500, 0, 1, 2049, 255, 513], 1160, 1040),
                                        ([300] * 13, 1290, 784), ([257, 3000, 0, 1000], 776, 1936)])
def test_products_of_thousands_of_rows(counts, N, K):
    """Every pair of CTAs has its share of 256 x 256 tiles, some of them ragged in each direction, of several experts."""
    check_grouped(len(counts), N, K, *grouped(counts, N, K, 3 if len(counts) > 1 else 0, N))


def test_nan_stays_in_its_rows():
    """Rows with NaN scales or codes, and an expert whose weights are NaN, leave the others alone."""
    counts, N, K = [70, 3, 200, 33], 136, 272
    rows, wc, ws, xc, xs, dc, ds, offsets = grouped(counts, N, K, 0, 4)
    bad = np.zeros(rows, bool)
    bad[[0, 69, 71, 100, 305]] = True
    xs[bad, 1], dc[bad, 5] = np.nan, 0x7f
    wv = tr.decode_weights(wc, ws)
    ws[1] = np.nan
    xv, dv = tr.decode_rows(xc, xs), tr.decode_rows(dc, ds)
    w, wsd, od = dev(wc), dev(ws, "f32"), dev(offsets)
    y, dx = torch.empty(rows, N, device=DEV), torch.empty(rows, K, device=DEV)
    qmv.qmv_b128_product(w, wsd, 4, N, K, dev(tr.act_buffer(xc, xs)), rows, od, "f32", y)
    qmv.qmv_b128_grad_x(w, wsd, 4, N, K, dev(tr.act_buffer(dc, ds)), rows, od, "f32", dx)
    bad[70:73] = True
    assert np.isnan(host(y)[bad]).all() and np.isnan(host(dx)[bad]).all()
    for e in range(4):
        at = np.arange(offsets[e], offsets[e + 1])
        at = at[~bad[at]]
        assert np.array_equal(host(y)[at], xv[at] @ wv[e].T) and np.array_equal(host(dx)[at], dv[at] @ wv[e])
    # the weights' gradient: a NaN and an infinity of one expert's rows stay in its matrix
    ints = ref.element_values("mxfp8")
    dy, x = ints[np.where(dc == 0x7f, 0, dc)], ints[xc]
    dy[72, 3], x[71, 7], x[72, 9] = np.nan, np.inf, np.nan
    dw = torch.empty(4, N, K, device=DEV)
    qmv.qmv_b128_grad_w("f16", dev(dy, "f16"), N, dev(x, "f16"), K, 4, N, K, rows, od, "f32", dw)
    for e in (0, 2, 3):
        a, b = offsets[e], offsets[e + 1]
        assert np.array_equal(host(dw[e]), dy[a:b].T @ x[a:b]), e
    got = host(dw[1])
    assert np.isnan(got[3]).all() and np.isnan(got[:, 9]).all() and not np.isfinite(got[:, 7]).any()
    keep = np.ix_(np.delete(np.arange(N), 3), np.delete(np.arange(K), [7, 9]))
    assert np.array_equal(got[keep], (np.nan_to_num(dy[70:73]).T @ np.nan_to_num(x[70:73], posinf=0))[keep])


def test_scales_of_the_range():
    """Block scales far apart, negative ones, and zero."""
    rows, N, K = 140, 260, 400
    g = qi.rng(6)
    wc, ws = exact_weights(g, 1, N, K)
    xc, xs = exact_rows(g, rows, K)
    xs = xs * 2.0 ** g.integers(-60, 50, size=xs.shape)
    ws = ws * 2.0 ** g.integers(-30, 30, size=ws.shape)
    ws[0, 0, 1] *= -1
    ws[0, 1, 2] = 0
    xs[3] = 0
    y = torch.empty(rows, N, device=DEV)
    qmv.qmv_b128_product(dev(wc), dev(ws, "f32"), 1, N, K, dev(tr.act_buffer(xc, xs)), rows, None, "f32", y)
    xv, wv = tr.decode_rows(xc, xs), tr.decode_weights(wc, ws)[0]
    # block sums are exact; scaling and adding four blocks: 8 roundings
    assert_within(host(y), xv @ wv.T, 8 * 2.0 ** -24 * (np.abs(xv) @ np.abs(wv).T), "f32", "y")


def test_grad_w_without_rows_is_zero():
    dw = torch.full((3, 40, 48), 7.0, dtype=torch.bfloat16, device=DEV)
    x = torch.zeros(8, 48, dtype=torch.bfloat16, device=DEV)
    qmv.qmv_b128_grad_w("bf16", x, 48, x, 48, 3, 40, 48, 0, dev(np.zeros(4, np.int32)), "bf16", dw)
    assert not dw.any()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_grad_w_beside_rows_of_nan(dtype):
    """Every other expert's rows are NaN, those behind the last one too: none reaches the experts between, whatever their rows
    past the last whole 16 or 64."""
    counts = [n for m in (1, 2, 15, 16, 17, 31, 32, 33, 48, 49, 63, 64, 65, 80, 127, 129, 528, 577) for n in (m, 3 + m % 5)]
    E, N, K, rows = len(counts), 300, 272, sum(counts) + 40
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    g = qi.rng(9)
    dy, x = (g.integers(-15, 16, size=(rows, n)).astype(np.float64) for n in (N, K))
    for bad in (0, 1):
        d, v = dy.copy(), x.copy()
        for e in range(bad, E, 2):
            d[offsets[e]:offsets[e + 1]] = v[offsets[e]:offsets[e + 1]] = np.nan
        d[offsets[-1]:] = v[offsets[-1]:] = np.nan
        dyd, ld = strided(d, dtype, -N % 8)
        dw = torch.full((E, N, K), 7.0, device=DEV)
        qmv.qmv_b128_grad_w(dtype, dyd, ld, dev(v, dtype), K, E, N, K, rows, dev(offsets), "f32", dw)
        for e in range(E):
            a, b = offsets[e], offsets[e + 1]
            assert np.array_equal(host(dw[e]), d[a:b].T @ v[a:b], equal_nan=True), (bad, e)
    assert status_clean()


def test_grad_w_matches_differences():
    """L = <y, dy> of unquantized rows is linear in W: its difference along a direction is the gradient's product with it."""
    rows, N, K = 90, 136, 144
    g = qi.rng(7)
    dy, x, direction = (dev(g.standard_normal(s), "bf16") for s in ((rows, N), (rows, K), (N, K)))
    dw = torch.empty(N, K, device=DEV)
    qmv.qmv_b128_grad_w("bf16", dy, N, x, K, 1, N, K, rows, None, "f32", dw)
    w = dev(g.standard_normal((N, K)), "f32").double()
    loss = lambda w: ((x.double() @ w.T) * dy.double()).sum()  # noqa: E731
    h = 0.5
    want = (loss(w + h * direction.double()) - loss(w - h * direction.double())) / (2 * h)
    size = (dy.double().abs().T @ x.double().abs() * direction.double().abs()).sum()
    assert abs((dw.double() * direction.double()).sum() - want) <= 2.0 ** -15 * size


@pytest.mark.parametrize("rows", [1, 300])
def test_products_in_graphs_and_on_streams(rows):
    """Captured steps replay on new rows, two graphs at once; outputs equal the eager calls' bit for bit."""
    E, N, K = 3, 264, 400
    g = qi.rng(2)
    wc, ws = exact_weights(g, E, N, K)
    w, wsd = dev(wc), dev(ws, "f32")
    od = dev(np.array([0, rows // 3, rows // 3, rows], np.int32))
    runs = []
    for i in range(2):
        s = torch.cuda.Stream()
        x = torch.zeros(rows, K, dtype=torch.bfloat16, device=DEV)
        dy = torch.zeros(rows, N, dtype=torch.bfloat16, device=DEV)
        ws_buf, dyq = buf(qmv.qmv_b128_linear_workspace_bytes(rows, K)), buf(qmv.qmv_act_b128_bytes(rows, N))
        y, dx = torch.zeros(rows, N, dtype=torch.bfloat16, device=DEV), torch.zeros(rows, K, dtype=torch.bfloat16, device=DEV)
        dw = torch.zeros(E, N, K, device=DEV)

        def go(x=x, dy=dy, ws_buf=ws_buf, dyq=dyq, y=y, dx=dx, dw=dw):
            qmv.qmv_b128_linear(w, wsd, E, N, K, "bf16", x, K, rows, od, ws_buf, y)
            qmv.qmv_quantize_act_b128("bf16", dy, N, rows, N, dyq)
            qmv.qmv_b128_grad_x(w, wsd, E, N, K, dyq, rows, od, "bf16", dx)
            qmv.qmv_b128_grad_w("bf16", dy, N, x, K, E, N, K, rows, od, "f32", dw)

        with torch.cuda.stream(s):
            go()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            go()
        runs.append((s, x, dy, graph, go, (y, dx, dw)))
    wv = tr.decode_weights(wc, ws)
    for step in range(3):
        for i, (s, x, dy, graph, go, outs) in enumerate(runs):
            x.copy_(dev(randn(10 * step + i, rows, K), "bf16"))
            dy.copy_(dev(randn(10 * step + i + 5, rows, N), "bf16"))
        torch.cuda.synchronize()
        for s, x, dy, graph, go, outs in runs:
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for s, x, dy, graph, go, outs in runs:
            got = [o.clone() for o in outs]
            go()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, outs))
            xv = tr.decode_rows(*tr.quantize_rows(host(x)))
            for e, (a, b) in enumerate(tr.ranges(od.cpu().numpy(), rows, E)):
                assert_within(host(outs[0])[a:b], xv[a:b] @ wv[e].T, bound(K, np.abs(xv[a:b]) @ np.abs(wv[e]).T), "bf16", "y")
    assert status_clean()


def test_product_as_a_host_threads_first_call():
    """The tensor maps are encoded on a thread that has made no CUDA call."""
    rows, N, K = 40, 200, 272
    g = qi.rng(1)
    wc, ws = exact_weights(g, 1, N, K)
    xc, xs = exact_rows(g, rows, K)
    w, wsd, xq = dev(wc), dev(ws, "f32"), dev(tr.act_buffer(xc, xs))
    y = torch.zeros(rows, N, device=DEV)
    stream = torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    failed = []

    def go():
        try:
            qmv.qmv_b128_product(w, wsd, 1, N, K, xq, rows, None, "f32", y, stream)
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    t = threading.Thread(target=go)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not failed
    assert np.array_equal(host(y), tr.decode_rows(xc, xs) @ tr.decode_weights(wc, ws)[0].T)


def test_moe_step_of_all_calls():
    """A MoE projection's training step as it is used: router, sort, dispatch, product, return, and every gradient, against
    float64 torch on the quantized numbers."""
    tokens, experts, top_k, N, K = 150, 6, 2, 96, 160
    g = qi.rng(11)
    x, wt = dev(randn(1, tokens, K), "f32"), dev(randn(2, experts, N, K) * 0.1, "f32")
    router = dev(g.standard_normal((experts, K)) / 12, "f32")
    dout, dloss = dev(g.standard_normal((tokens, N)), "f32"), dev([0.05], "f32")
    logits = x @ router.T
    i32 = torch.int32
    ids, weights = torch.empty(tokens, top_k, dtype=i32, device=DEV), torch.empty(tokens, top_k, device=DEV)
    qmv.qmv_moe_router("f32", logits, experts, None, tokens, experts, top_k, "softmax", True, 1.0, ids, weights)
    counts, means, loss = torch.empty(experts + 1, dtype=i32, device=DEV), torch.empty(experts, device=DEV), torch.empty(1, device=DEV)
    qmv.qmv_moe_balance("f32", logits, experts, None, ids, tokens, experts, top_k, "softmax", counts, means, loss,
                        buf(qmv.qmv_moe_balance_workspace_bytes(tokens, experts)))
    slots = tokens * top_k
    offsets, row, slot = (torch.empty(n, dtype=i32, device=DEV) for n in (experts + 1, slots, slots))
    qmv.qmv_moe_sort(ids, tokens, top_k, experts, offsets, row, slot)
    assert torch.equal(offsets.diff(), counts[:-1])   # the loss counts what the sort finds
    xs, ys, out = torch.empty(slots, K, device=DEV), torch.empty(slots, N, device=DEV), torch.empty(tokens, N, device=DEV)
    codes, scales = buf(experts * N * K).view(experts, N, K), torch.empty(experts, 1, 2, device=DEV)
    qmv.qmv_quantize_weights_b128("f32", wt, experts, N, K, codes, scales)
    qmv.qmv_moe_dispatch("f32", x, K, tokens, top_k, K, row, xs)
    qmv.qmv_b128_linear(codes, scales, experts, N, K, "f32", xs, K, slots, offsets, buf(qmv.qmv_b128_linear_workspace_bytes(slots, K)), ys)
    qmv.qmv_moe_return("f32", ys, weights, tokens, top_k, N, row, out, N)
    dys, dweights = torch.empty_like(ys), torch.empty_like(weights)
    qmv.qmv_moe_return_grad("f32", dout, N, ys, weights, tokens, top_k, N, row, dys, dweights)
    dyq, dxs, dx = buf(qmv.qmv_act_b128_bytes(slots, N)), torch.empty_like(xs), torch.empty_like(x)
    qmv.qmv_quantize_act_b128("f32", dys, N, slots, N, dyq)
    qmv.qmv_b128_grad_x(codes, scales, experts, N, K, dyq, slots, offsets, "f32", dxs)
    qmv.qmv_moe_dispatch_grad("f32", dxs, tokens, top_k, K, row, dx, K)
    dys16, xs16, dw = dys.bfloat16(), xs.bfloat16(), torch.empty(experts, N, K, device=DEV)
    qmv.qmv_b128_grad_w("bf16", dys16, N, xs16, K, experts, N, K, slots, offsets, "f32", dw)
    dlogits = torch.empty_like(logits)
    qmv.qmv_moe_router_grad("f32", logits, experts, None, ids, dweights, counts, dloss, tokens, experts, top_k, "softmax", True, 1.0,
                            dlogits, experts)

    # the same in float64: quantizations by the definition, everything else by torch
    wv = torch.from_numpy(tr.decode_weights(*tr.quantize_weights(host(wt)))).to(DEV)
    xv = torch.from_numpy(tr.decode_rows(*tr.quantize_rows(host(x)))).to(DEV).requires_grad_()
    l = logits.double().requires_grad_()
    at = ids.long()
    p = torch.softmax(l, 1)
    chosen = p.gather(1, at)
    wgt = chosen / chosen.sum(1, keepdim=True)
    ys64 = torch.einsum("tk,tjnk->tjn", xv, wv[at])
    out64 = (wgt[..., None] * ys64).sum(1)
    f = torch.bincount(at.flatten(), minlength=experts).double() / slots
    loss64 = experts * (f * p.mean(0)).sum()
    ((out64 * dout.double()).sum() + 0.05 * loss64).backward()

    def near(got, want, off):
        assert (got.double() - want).abs().max() <= off * want.abs().max()

    # fp32 chains of a few hundred terms; dx takes Q(dy), off by up to 2^-4 of a value: the norm's error is below 2^-5
    near(out, out64.detach(), 2.0 ** -14)
    near(loss, loss64.detach(), 2.0 ** -18)
    near(dlogits, l.grad, 2.0 ** -12)
    assert (dx.double() - xv.grad).norm() <= 2.0 ** -5 * xv.grad.norm()
    # dW of the 16-bit rows themselves
    for e, (a, b) in enumerate(tr.ranges(offsets.cpu().numpy(), slots, experts)):
        near(dw[e], dys16[a:b].double().T @ xs16[a:b].double(), 2.0 ** -14)
    assert status_clean()
