"""The many-row operators where they can go wrong beyond ordinary inputs: numbers at the ends of their types' ranges,
infinities and NaN, offsets that name nothing, the widest layer, host threads and streams at once. Definitions and
tolerances are those of test_gpu_rows.py; what a test adds to them stands beside it."""
import threading

import numpy as np
import pytest
import torch

qmv = pytest.importorskip("bit_quantized_moe_gb300")
import oracle  # noqa: E402
import qmv_inputs as qi  # noqa: E402
import rows_reference as ref  # noqa: E402
from qmv_testutil import DEV, assert_within, status_clean  # noqa: E402
from test_gpu_rows import (TORCH, buf, dev, drawn_ids, exact_inputs, host, layer_case, packed_weights, quantized_close,  # noqa: E402
                           randn, sorted_on_gpu, split_layer, unpacked)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ntok,N_down", [(1100, 4000), (1100, 4001), (140, 32000)])
def test_layer_rows_past_f16_range_in_a_large_call(ntok, N_down):
    """fp16 calls above 32 MB of fp32 rows: a row past 65,504 is weighted as the number it is, not as infinity."""
    top_k, E, K, N = 2, 4, 96, 64
    gu, w_gu, dn, w_dn, x, ids, weights, _ = layer_case("mxfp4", "mxfp4", "f16", ntok, top_k, E, K, N, N_down, 0.05)
    assert ntok * top_k * N_down * 4 > 32 << 20
    x *= 6000.0
    weights = weights * 2.0 ** -9
    ws = buf(qmv.qmv_moe_prefill_layer_workspace_bytes(gu, dn, ntok, top_k))
    y = torch.full((ntok, N_down), 7.0, dtype=torch.float16, device=DEV)
    qmv.qmv_moe_prefill_layer(gu, w_gu, dn, w_dn, "f16", x, K, dev(ids), weights, ntok, top_k, ws, y)
    _, ys, row = split_layer(gu, w_gu, dn, w_dn, "f16", x, ids, weights, E, K, N, N_down, "f32")
    r = row.cpu().numpy().reshape(ntok, top_k)
    terms = np.where((r >= 0)[..., None], host(ys)[np.where(r >= 0, r, ~r)], 0) * host(weights)[..., None]
    large = (ys.abs() > 65520).float().mean().item()
    assert 1e-4 < large < 0.5 and torch.isfinite(ys).all() and np.abs(terms.sum(1)).max() < 60000, (large, np.abs(terms.sum(1)).max())
    # a row's elements may be rounded to fp16 (11 bits, subnormal steps of 2^-24), then weighted and summed in fp32
    bound = (2.0 ** -11 + (top_k + 1) * 2.0 ** -24) * np.abs(terms).sum(1) + 2.0 ** -25 * host(weights).sum(1)[:, None]
    assert_within(host(y), terms.sum(1), bound, "f16", "layer")
    assert status_clean()


@pytest.mark.parametrize("glu", [False, True])
def test_product_as_a_host_threads_first_call(glu):
    """A thread that has made no CUDA call may begin with a product."""
    N, K, rows = 32, 96, 5
    g = qi.rng(1)
    wc, ws = exact_inputs(g, "mxfp4", (1, N, K))
    xc, xs = exact_inputs(g, "mxfp4", (rows, K))
    desc, w = packed_weights("mxfp4", wc, ws)
    if glu:
        w = dev(qmv.qmv_pack_gate_up(desc, *[oracle.pack_codes("mxfp4", wc), ws] * 2))
    xq, y = dev(ref.act_buffer(xc, xs, "mxfp4")), buf(max(rows * N * 4, qmv.qmv_act_mx_bytes("mxfp4", rows, N)))
    stream = torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    errors = []

    def run():
        try:
            if glu:
                qmv.qmv_mx_gate_up_swiglu(desc, w, xq, rows, None, "mxfp4", y, stream)
            else:
                qmv.qmv_mx_product(desc, w, xq, rows, None, "f32", y, stream)
        except qmv.QmvError as e:
            errors.append(str(e))

    t = threading.Thread(target=run)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    if not glu:
        want = ref.decode(xc, xs, "mxfp4") @ ref.decode(wc[0], ws[0], "mxfp4").T
        assert np.array_equal(host(y[:rows * N * 4].view(torch.float32).view(rows, N)), want)
    assert status_clean()


def test_products_from_two_host_threads():
    """One kernel launched from two threads at once with the most experts and with few: each launch has the shared memory
    that it asks for, whatever the other's size."""
    N, K, rows, calls = 24, 96, 5, 4000
    errors = []
    sizes = [qmv.MAX_SORT_EXPERTS, 2]
    work = []
    for E in sizes:
        g = qi.rng(E)
        wc, ws = exact_inputs(g, "mxfp4", (E, N, K))
        xc, xs = exact_inputs(g, "mxfp4", (rows, K))
        desc, w = packed_weights("mxfp4", wc, ws)
        offsets = np.full(E + 1, rows, dtype=np.int32)
        offsets[0] = 0
        want = ref.decode(xc, xs, "mxfp4") @ ref.decode(wc[0], ws[0], "mxfp4").T
        work.append((desc, w, dev(ref.act_buffer(xc, xs, "mxfp4")), dev(offsets), want, torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [torch.zeros(rows, N, dtype=torch.float32, device=DEV) for _ in work]
    torch.cuda.synchronize()

    def run(i):
        desc, w, xq, offsets, _, stream = work[i]
        try:
            for n in range(calls):
                qmv.qmv_mx_product(desc, w, xq, rows, offsets, "f32", outs[i], stream)
                if n % 200 == 199:
                    stream.synchronize()
        except qmv.QmvError as e:
            errors.append((sizes[i], str(e)))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for out, w in zip(outs, work):
        assert np.array_equal(host(out), w[4])
    assert status_clean()


@pytest.mark.parametrize("dtype,N", [("bf16", 65600), ("f16", 70001), ("bf16", 1 << 20)])
def test_return_of_rows_past_65536_columns(dtype, N):
    """The experts' rows are as wide as a weight matrix may be high."""
    ntok, top_k, E = 3, 2, 4
    _, row, _ = sorted_on_gpu(drawn_ids(1, ntok, top_k, E, 0.2), E)
    r = row.cpu().numpy()
    flat, valid = np.where(r >= 0, r, ~r), r >= 0
    ys, weights, dy = dev(randn(2, ntok * top_k, N), dtype), dev(randn(3, ntok, top_k).astype(np.float32)), dev(randn(4, ntok, N), dtype)
    y, dx = (torch.full((ntok, N), 7.0, dtype=TORCH[dtype], device=DEV) for _ in range(2))
    qmv.qmv_moe_return(dtype, ys, weights, ntok, top_k, N, row, y, N)
    terms = np.where(valid[:, None], host(ys)[flat], 0) * host(weights).reshape(-1, 1)
    terms = terms.reshape(ntok, top_k, N)
    assert_within(host(y), terms.sum(1), (top_k + 1) * 2.0 ** -24 * np.abs(terms).sum(1), dtype, "y")
    dys, dw = torch.full_like(ys, 7.0), torch.empty(ntok, top_k, device=DEV)
    qmv.qmv_moe_return_grad(dtype, dy, N, ys, weights, ntok, top_k, N, row, dys, dw)
    d = np.repeat(host(dy), top_k, 0)
    want = np.zeros((ntok * top_k, N))
    want[flat] = np.where(valid[:, None], host(weights).reshape(-1, 1) * d, 0)
    assert_within(host(dys), want, np.abs(want) * 2.0 ** -24, dtype, "dys")
    prod = np.where(valid[:, None], host(ys)[flat], 0) * d
    # a thread's sum (one of 384 at least), then a tree
    assert (np.abs(host(dw).reshape(-1) - prod.sum(1)) <= (N / 32 + 16) * 2.0 ** -24 * np.abs(prod).sum(1)).all()


def test_layer_past_65536_columns():
    ntok, top_k, E, K, N, N_down = 3, 2, 2, 32, 32, 65600
    gu, w_gu, dn, w_dn, x, ids, weights, _ = layer_case("mxfp4", "mxfp8", "bf16", ntok, top_k, E, K, N, N_down, 0.2)
    ws = buf(qmv.qmv_moe_prefill_layer_workspace_bytes(gu, dn, ntok, top_k))
    y = torch.full((ntok, N_down), 7.0, dtype=torch.bfloat16, device=DEV)
    qmv.qmv_moe_prefill_layer(gu, w_gu, dn, w_dn, "bf16", x, K, dev(ids), weights, ntok, top_k, ws, y)
    _, ys, row = split_layer(gu, w_gu, dn, w_dn, "bf16", x, ids, weights, E, K, N, N_down, "f32")
    r = row.cpu().numpy().reshape(ntok, top_k)
    terms = np.where((r >= 0)[..., None], host(ys)[np.where(r >= 0, r, ~r)], 0) * host(weights)[..., None]
    assert_within(host(y), terms.sum(1), (top_k + 1) * 2.0 ** -24 * np.abs(terms).sum(1), "bf16", "layer")
    assert status_clean()


def norm_case(dtype, values, eps, out, ld=None):
    """(output, kept sum) of the norm of `values` without a residual, gain 1, rows `ld` apart."""
    rows, K = values.shape
    x = torch.zeros(rows, ld or K, dtype=TORCH[dtype], device=DEV)
    x[:, :K] = dev(values, dtype)
    fmt = out if out.startswith("mx") else None
    size = {"plain": rows * K * x.element_size(), "q8": qmv.qmv_act_q8_bytes(rows, K)}.get(out) or qmv.qmv_act_mx_bytes(fmt, rows, K)
    y = buf(size)
    qmv.qmv_rms_norm(dtype, x, ld or K, None, 0, torch.ones(K, dtype=TORCH[dtype], device=DEV), rows, K, eps, None, out, y)
    return host(x[:, :K]), y


# Magnitudes whose squares leave fp32: above 2^64 and below 2^-64 (eps 0: with eps the smallest rows are ordinary).
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("out", ["plain", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("K,extra", [(32, 0), (256, 0), (544, 0), (2048, 0), (2880, 0), (2880, 3), (7168, 0), (8224, 1), (65536, 0)])
def test_rms_norm_of_numbers_whose_squares_leave_the_range(dtype, out, K, extra):
    size = np.array([2.0 ** 64, 1.0, 2.0 ** 121, 2.0 ** -64, 2.0 ** 100, 2.0 ** -100, 3.0, 2.0 ** -118, 2.0 ** 63])
    s, y = norm_case(dtype, np.clip(randn(K, len(size), K), -60, 60) * size[:, None], 0.0, out, K + extra)
    want = s / np.sqrt((s ** 2).mean(-1, keepdims=True))
    err = 1e-5 * np.abs(want)
    if out == "plain":
        assert_within(host(y.view(TORCH[dtype]).view(s.shape)), want, err, dtype, "y")
    else:
        quantized_close(*unpacked(out, y, *s.shape), want, err, out)


@pytest.mark.parametrize("dtype,K", [("bf16", 31), ("f32", 2881), ("bf16", 8191), ("f32", 1025)])
def test_rms_norm_of_large_numbers_in_odd_widths(dtype, K):
    size = np.array([1.0, 2.0 ** 100, 2.0 ** 70, 2.0 ** -90])
    s, y = norm_case(dtype, np.clip(randn(K, len(size), K), -60, 60) * size[:, None], 0.0, "plain")
    want = s / np.sqrt((s ** 2).mean(-1, keepdims=True))
    assert_within(host(y.view(TORCH[dtype]).view(s.shape)), want, 1e-5 * np.abs(want), dtype, "y")


def test_rms_norm_with_eps_of_numbers_whose_squares_leave_the_range():
    """eps counts as it stands beside small rows and not beside large ones; a row of zeros without eps is 0 / 0."""
    size = np.array([2.0 ** 100, 2.0 ** -20, 2.0 ** -70, 0.0])
    for eps in (1e-5, 1e-30, 4.0, 3e38):
        s, y = norm_case("f32", np.clip(randn(3, 4, 288), -60, 60) * size[:, None], eps, "plain")
        want = s / np.sqrt((s ** 2).mean(-1, keepdims=True) + float(np.float32(eps)))
        assert_within(host(y.view(torch.float32).view(s.shape)), want, 1e-5 * np.abs(want) + 2.0 ** -149, "f32", f"eps {eps}")
    s, y = norm_case("f32", np.zeros((2, 288)), 0.0, "plain")
    assert np.isnan(host(y.view(torch.float32))).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("offsets,ranges", [
    ([0, 5, 3, 9], [(0, 5), (5, 5), (5, 9)]), ([-7, 4, 4, 1000], [(0, 4), (4, 4), (4, 9)]),
    ([6, 6, 6, 6], [(6, 6)] * 3), ([20, 30, 40, 50], [(9, 9)] * 3), ([8, 2, 0, 9], [(8, 8), (8, 8), (8, 9)])])
def test_rows_of_offsets_that_do_not_ascend(fmt, offsets, ranges):
    """Each expert's range is taken into [0, nrows] and begins no earlier than those before it end: every row has one expert
    at most, and rows of none stay as they are."""
    rows, E, N, K = 9, 3, 40, 64
    g = qi.rng(4)
    wc, ws = exact_inputs(g, fmt, (E, N, K))
    xc, xs = exact_inputs(g, fmt, (rows, K))
    desc, w = packed_weights(fmt, wc, ws)
    y = torch.full((rows + 2, N), 7.0, dtype=torch.float32, device=DEV)
    qmv.qmv_mx_product(desc, w, dev(ref.act_buffer(xc, xs, fmt)), rows, dev(np.array(offsets, dtype=np.int32)), "f32", y)
    want, xv = np.full((rows + 2, N), 7.0), ref.decode(xc, xs, fmt)
    for e, (a, b) in enumerate(ranges):
        want[a:b] = xv[a:b] @ ref.decode(wc[e], ws[e], fmt).T
    assert np.array_equal(host(y), want) and status_clean()


def test_many_descending_offsets():
    """1024 experts whose offsets fall and rise by turns: only the first pair names rows."""
    rows, E, N, K = 300, qmv.MAX_SORT_EXPERTS, 24, 32
    g = qi.rng(5)
    wc, ws = exact_inputs(g, "mxfp4", (E, N, K))
    xc, xs = exact_inputs(g, "mxfp4", (rows, K))
    desc, w = packed_weights("mxfp4", wc, ws)
    offsets = np.where(np.arange(E + 1) % 2 == 0, 0, rows).astype(np.int32)
    y = torch.full((rows, N), 7.0, dtype=torch.float32, device=DEV)
    qmv.qmv_mx_product(desc, w, dev(ref.act_buffer(xc, xs, "mxfp4")), rows, dev(offsets), "f32", y)
    assert np.array_equal(host(y), ref.decode(xc, xs, "mxfp4") @ ref.decode(wc[0], ws[0], "mxfp4").T) and status_clean()


@pytest.mark.parametrize("h_fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("rows", [40, 700])
def test_gate_up_swiglu_of_large_negative_gates(h_fmt, rows):
    """silu(g) of g from -160 to 48 beside up sums so large that the product is an ordinary number: within 12 fp32 roundings
    (four for the exponential, two for the reciprocal, six sums and products)."""
    N, K = 224, 32
    g = qi.rng(rows)
    gc, gs = np.zeros((1, N, K), dtype=np.uint8), np.full((1, N, 1), 127 + 5, dtype=np.uint8)
    gc[0, :, 0] = g.choice([12, 13], size=N)                                # -2 and -3, times 32
    gc[0, 160:, 0] = g.choice([9, 10, 11, 12, 13, 1], size=N - 160)         # groups of every size: -0.5 .. -3 and 0.5
    uc, us = exact_inputs(g, "mxfp4", (1, N, K))
    us = np.repeat(g.integers(127 + 90, 127 + 100, size=(1, N // 32, 1)), 32, axis=1).astype(np.uint8)
    xc, xs = np.zeros((rows, K), dtype=np.uint8), np.full((rows, 1), 127, dtype=np.uint8)
    xc[:, 0] = g.choice([1, 2, 3], size=rows)                               # 0.5, 1, 1.5
    desc = qmv.wdesc("mxfp4", N, K, 1)
    w = dev(qmv.qmv_pack_gate_up(desc, oracle.pack_codes("mxfp4", gc), gs, oracle.pack_codes("mxfp4", uc), us))
    hq = buf(qmv.qmv_act_mx_bytes(h_fmt, rows, N))
    qmv.qmv_mx_gate_up_swiglu(desc, w, dev(ref.act_buffer(xc, xs, "mxfp4")), rows, None, h_fmt, hq)
    xv = ref.decode(xc, xs, "mxfp4")
    gate, up = xv @ ref.decode(gc[0], gs[0], "mxfp4").T, xv @ ref.decode(uc[0], us[0], "mxfp4").T
    assert gate.min() < -100 and (np.abs(gate) < 87).any()
    h = ref.silu(gate) * up
    codes, scales = unpacked(h_fmt, hq, rows, N)
    quantized_close(codes, scales, h, 12 * 2.0 ** -24 * np.abs(h) + 2.0 ** -149, h_fmt)
    assert status_clean()


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_quantize_special_groups_of_16_bits(fmt, dtype):
    """Zeros, subnormals, the largest numbers, infinities and NaN in every column of a group, beside ordinary groups."""
    tiny, big = (2.0 ** -133, 3.3895313892515355e38) if dtype == "bf16" else (2.0 ** -24, 65504.0)
    special = [0.0, -0.0, tiny, -tiny, 37 * tiny, big, -big, np.inf, -np.inf, np.nan]
    K = 96
    v = np.tile(randn(1, 1, K), (32 * len(special), 1))
    for i, s in enumerate(special):
        for c in range(32):
            row = v[32 * i + c]
            if abs(s) < 1:
                row[32:64] = 0.0     # a group of nothing else
            row[32 + c] = s
    v[-1, 32:64] = np.where(np.arange(32) % 2, np.inf, np.nan)
    x = dev(v, dtype)
    rows = len(v)
    xq = buf(qmv.qmv_act_mx_bytes(fmt, rows, K))
    qmv.qmv_quantize_act_mx(fmt, dtype, x, K, rows, K, xq)
    codes, scales = unpacked(fmt, xq, rows, K)
    want_c, want_s = ref.quantize(host(x), fmt)
    assert (want_s == 255).sum() == 3 * 32
    assert np.array_equal(scales, want_s) and np.array_equal(codes, want_c)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("out", ["plain", "mxfp8", "mxfp4", "q8"])
@pytest.mark.parametrize("K", [96, 2880])
def test_rms_norm_of_rows_with_infinities_and_nan(dtype, out, K):
    """An infinity makes its own column NaN and the others 0, a NaN the whole row; the rows beside them stay ordinary."""
    v = randn(K, 7, K)
    v[1, 5], v[3, K - 1], v[5, 33] = np.inf, np.nan, -np.inf
    s, y = norm_case(dtype, v, 1e-5, out)
    with np.errstate(invalid="ignore"):
        want = s / np.sqrt((s ** 2).mean(-1, keepdims=True) + 1e-5)
    bad = np.isnan(want)
    assert bad[1].sum() == 1 and bad[3].all() and bad[5].sum() == 1
    err = 1e-5 * np.abs(want)
    if out == "plain":
        got = host(y.view(TORCH[dtype]).view(s.shape))
        assert np.array_equal(np.isnan(got), bad)
        assert_within(np.where(bad, 0, got), np.where(bad, 0, want), np.where(bad, 0, err), dtype, "y")
    elif out == "q8":
        q, d = qmv.qmv_act_q8_unpack(y.cpu().numpy(), *s.shape)
        d = oracle.f16_bits_to_f64(d)
        groups = bad.reshape(7, -1, 32).any(-1)
        assert np.array_equal(np.isnan(d), groups)
        exact_d = np.abs(np.where(bad, 0, want)).reshape(7, -1, 32).max(-1) / 127
        assert (np.abs(d - exact_d)[~groups] <= (exact_d * (2.0 ** -11 + 1.1e-5) + 2.0 ** -25)[~groups]).all()
        q = q.reshape(7, -1, 32)
        assert not q[1][~groups[1]].any() and not q[5][~groups[5]].any() and q[0].any()
    else:
        codes, scales = unpacked(out, y, *s.shape)
        groups = bad.reshape(7, -1, 32).any(-1)
        assert np.array_equal(scales == 255, groups) and not codes.reshape(7, -1, 32)[groups].any()
        keep = [0, 2, 4, 6]
        quantized_close(codes[keep], scales[keep], want[keep], err[keep], out)
        assert not scales[1][~groups[1]].any() and not scales[5][~groups[5]].any()


@pytest.mark.parametrize("h_fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("rows", [70, 600])
def test_gate_up_swiglu_of_nan_and_infinite_sums(h_fmt, rows):
    """A NaN gate or up sum, or an infinite one, makes its group of h NaN; the other groups and rows are as without it."""
    N, K = 128, 160
    g = qi.rng(rows)
    (gc, gs), (uc, us), (xc, xs) = (exact_inputs(g, "mxfp8", s) for s in ((1, N, K), (1, N, K), (rows, K)))
    gs = (gs - 9).astype(np.uint8)
    desc = qmv.wdesc("mxfp8", N, K, 1)

    def h_of(gs, us, xs):
        w = dev(qmv.qmv_pack_gate_up(desc, gc, gs, uc, us))
        hq = buf(qmv.qmv_act_mx_bytes(h_fmt, rows, N))
        qmv.qmv_mx_gate_up_swiglu(desc, w, dev(ref.act_buffer(xc, xs, "mxfp8")), rows, None, h_fmt, hq)
        return unpacked(h_fmt, hq, rows, N)

    codes, scales = h_of(gs, us, xs)
    assert not (scales == 255).any()
    bad_gs, bad_us, bad_xs = gs.copy(), us.copy(), xs.copy()
    bad_gs[0, 3, 1], bad_us[0, 40, 2], bad_us[0, 70], bad_xs[7, 4] = 255, 255, 254, 255   # groups 0, 1 and 2; row 7
    c, s = h_of(bad_gs, bad_us, bad_xs)
    over = np.abs(ref.decode(xc, xs, "mxfp8") @ ref.decode(uc[0], bad_us[0], "mxfp8")[70]) >= 2.0 ** 128
    assert over.sum() > rows // 2
    assert (s[:, :2] == 255).all() and (s[over, 2] == 255).all() and (s[7] == 255).all()
    other = np.delete(np.arange(rows), 7)
    c, codes = c.reshape(rows, -1, 32), codes.reshape(rows, -1, 32)
    assert np.array_equal(s[other, 3], scales[other, 3]) and np.array_equal(c[other, 3], codes[other, 3])
    assert not c[other, :2].any() and status_clean()


def test_layer_of_tokens_with_infinities_and_nan():
    """Tokens with an infinity or a NaN are NaN where an expert takes them; the others' outputs are those of a call with
    ordinary values in those places; a dropped token of NaN is zeros."""
    ntok, top_k, E, K, N, N_down = 150, 2, 3, 288, 96, 200
    gu, w_gu, dn, w_dn, x, ids, weights, _ = layer_case("mxfp4", "mxfp8", "bf16", ntok, top_k, E, K, N, N_down, 0.0)
    bad = [3, 64, 149]
    ids[64] = -1
    ws = buf(qmv.qmv_moe_prefill_layer_workspace_bytes(gu, dn, ntok, top_k))

    def run():
        y = torch.full((ntok, N_down), 7.0, dtype=torch.bfloat16, device=DEV)
        qmv.qmv_moe_prefill_layer(gu, w_gu, dn, w_dn, "bf16", x, K, dev(ids), weights, ntok, top_k, ws, y)
        return y

    want = run()
    x[3, 7], x[64], x[149, K - 1] = float("inf"), float("nan"), float("nan")
    got = run()
    keep = [t for t in range(ntok) if t not in bad]
    assert torch.equal(got[keep], want[keep])
    assert got[3].isnan().all() and got[149].isnan().all() and not got[64].any() and status_clean()


def test_layers_on_two_streams_at_once():
    """Two layers of different shapes in flight together, each with its own workspace, give what they give alone."""
    runs = []
    for args in (("mxfp4", "mxfp4", "bf16", 300, 4, 8, 288, 96, 200, 0.1), ("mxfp8", "mxfp4", "f16", 41, 2, 5, 416, 160, 264, 0.0)):
        gu, w_gu, dn, w_dn, x, ids, weights, _ = layer_case(*args)
        dtype, ntok, top_k, K = args[2], args[3], args[4], args[6]
        y = [torch.empty(ntok, args[8], dtype=TORCH[dtype], device=DEV) for _ in range(2)]
        ws = buf(qmv.qmv_moe_prefill_layer_workspace_bytes(gu, dn, ntok, top_k))
        runs.append((y, torch.cuda.Stream(), lambda out, s, a=(gu, w_gu, dn, w_dn, dtype, x, K, dev(ids), weights, ntok, top_k, ws):
                     qmv.qmv_moe_prefill_layer(*a, out, s)))
    for y, _, call in runs:
        call(y[0], None)
    torch.cuda.synchronize()
    for _ in range(30):
        for y, s, call in runs:
            call(y[1], s)
    torch.cuda.synchronize()
    assert all(torch.equal(*y) for y, _, _ in runs) and status_clean()
