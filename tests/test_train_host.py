"""Host-side tests of the router and of the products with a scale for each block of 128: the 64-bit definitions that the
GPU tests compare with, the activation buffer's layout, and the refusals, which come before anything is enqueued."""
import numpy as np
import pytest
import torch

import qmv_inputs as qi
import rows_reference as ref
import train_reference as tr

qmv = pytest.importorskip("bit_quantized_moe_gb300", reason="libqmv not built")

P = 1 << 40          # an aligned device address that no check reads
ODD = P + 4
BIG = 1 << 50


def test_scores_match_torch():
    l = qi.rng(1).standard_normal((9, 33)) * 5
    t = torch.from_numpy(l)
    assert np.allclose(tr.scores(l, "softmax")[0], torch.softmax(t, 1).numpy(), rtol=1e-14, atol=0)
    s = torch.sigmoid(t)
    got = tr.scores(l, "sigmoid")
    assert np.allclose(got[0], s.numpy(), rtol=1e-14, atol=0)
    assert np.allclose(got[1], (s / s.sum(1, keepdim=True)).numpy(), rtol=1e-13, atol=0)


def test_route_ties_and_missing_experts():
    l = np.array([[1.0, 3.0, 3.0, -np.inf], [-np.inf] * 4, [-np.inf, 2.0, -np.inf, -np.inf]])
    ids, w = tr.route(l, np.array([True] * 3), 3, "softmax", True, 2.0)
    assert ids.tolist() == [[1, 2, 0], [-1, -1, -1], [1, -1, -1]]
    assert np.allclose(w.sum(1), [2, 0, 2]) and w[0, 0] == w[0, 1] and w[2, 0] == 2.0
    ids, w = tr.route(l, np.array([True, True, False]), 1, "sigmoid", False, 1.0)
    assert ids.tolist() == [[1], [-1], [-1]] and w[2, 0] == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_router_gradient_by_differences(score, renorm):
    """The formula's gradient against central differences of what it is the gradient of."""
    g = qi.rng(3)
    tokens, experts, top_k, scale, dloss = 5, 7, 3, 2.5, 0.7
    l = g.standard_normal((tokens, experts)) * 2
    live = np.array([True, True, False, True, True])
    ids, _ = tr.route(l, live, top_k, score, renorm, scale)
    dw = g.standard_normal((tokens, top_k))
    counts, _, _ = tr.balance(l, live, ids, top_k, score)

    def total(l):
        s = tr.quotients(l, ids, score) if renorm else np.take_along_axis(tr.scores(l, score)[0], np.maximum(ids, 0), 1)
        w = np.where(ids >= 0, scale * s, 0.0)
        return (w * dw).sum() + dloss * tr.balance(l, live, ids, top_k, score)[2]

    d, _ = tr.router_grad(l, live, ids, dw, counts, dloss, top_k, score, renorm, scale)
    h = 1e-5
    for t in range(tokens):
        for e in range(experts):
            a, b = l.copy(), l.copy()
            a[t, e] += h
            b[t, e] -= h
            assert abs((total(a) - total(b)) / (2 * h) - d[t, e]) < 1e-8


def test_balance_of_an_even_router_is_one():
    l = np.zeros((8, 4))
    ids = np.array([[i % 4, (i + 1) % 4] for i in range(8)])
    counts, means, loss = tr.balance(l, np.ones(8, bool), ids, 2, "softmax")
    assert counts.tolist() == [4, 4, 4, 4, 8] and np.allclose(means, 0.25) and abs(loss - 1) < 1e-15


def test_quantized_rows_match_torch():
    x = (qi.rng(4).standard_normal((5, 200)) * 3).astype(np.float32)
    codes, scales = tr.quantize_rows(x.astype(np.float64))
    top = np.abs(np.pad(x, ((0, 0), (0, 56))).reshape(5, 2, 128)).max(-1)
    assert np.array_equal(scales.astype(np.float32), top / np.float32(448))
    v = torch.from_numpy(x * np.repeat(np.float32(448) / top, 128, 1)[:, :200])
    assert np.array_equal(codes, v.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_quantized_weights_are_rows_of_blocks():
    """A matrix of one row of blocks, every row the same maximum, quantizes as its rows do."""
    w = qi.rng(5).standard_normal((2, 130, 272))
    w[:, :, ::128] = 9.0   # the first column of each block
    codes, scales = tr.quantize_weights(w)
    rc, rs = tr.quantize_rows(w.reshape(260, 272))
    assert np.array_equal(codes.reshape(260, 272), rc)
    assert np.array_equal(np.repeat(scales, 128, 1)[:, :130].reshape(260, 3), rs)


@pytest.mark.parametrize("rows,K", [(1, 1), (3, 100), (5, 128), (7, 272), (130, 2880)])
def test_act_buffer_layout(rows, K):
    g = qi.rng(rows + K)
    codes, scales = g.integers(0, 256, size=(rows, K), dtype=np.uint8), g.standard_normal((rows, -(-K // 128))).astype(np.float32)
    buf = tr.act_buffer(codes, scales)
    assert buf.nbytes == qmv.qmv_act_b128_bytes(rows, K) == qmv.qmv_b128_linear_workspace_bytes(rows, K)
    assert qmv.qmv_act_b128_scale_offset(rows, K) % 128 == 0
    c, s = qmv.qmv_act_b128_unpack(buf, rows, K)
    assert np.array_equal(c, codes) and np.array_equal(s, scales)


def test_sizes_of_invalid_shapes_are_zero():
    for rows, K in ((-1, 32), (qmv.MAX_ROWS + 1, 32), (1, 0), (1, (1 << 20) + 1)):
        assert qmv.qmv_act_b128_bytes(rows, K) == 0 and qmv.qmv_act_b128_scale_offset(rows, K) == 0
    assert qmv.qmv_act_b128_bytes(0, 32) == 0
    assert qmv.qmv_act_b128_bytes(qmv.MAX_ROWS, 1 << 20) > 1 << 42   # past 32 bits
    for tokens, experts in ((-1, 8), (qmv.MAX_ROWS + 1, 8), (4, 0), (4, 1025)):
        assert qmv.qmv_moe_balance_workspace_bytes(tokens, experts) == 0
    assert qmv.qmv_moe_balance_workspace_bytes(0, 1) > 0


def _call(name, good, **over):
    return getattr(qmv.lib, name)(*{**good, **over}.values(), 0)


ROUTER = dict(type=0, logits=P, ldl=8, live=P, ntok=4, n=8, top_k=2, score=0, renorm=1, scale=1.0, ids=P, weights=P)
BALANCE = dict(type=0, logits=P, ldl=8, live=P, ids=P, ntok=4, n=8, top_k=2, score=0, counts=P, means=P, loss=P, ws=P, ws_bytes=BIG)
GRAD = dict(type=0, logits=P, ldl=8, live=P, ids=P, dweights=P, counts=P, dloss=P, ntok=4, n=8, top_k=2, score=0, renorm=1,
            scale=1.0, dlogits=P, ldd=8)
QUANT = dict(type=0, x=P, ldx=64, nrows=3, K=64, xq=P, xq_bytes=BIG)
QUANT_W = dict(type=0, w=P, n=2, N=64, K=64, codes=P, scales=P)
PRODUCT = dict(w=P, ws=P, n=4, N=64, K=64, xq=P, xq_bytes=BIG, nrows=3, offsets=P, out_type=0, y=P)
LINEAR = dict(w=P, ws=P, n=4, N=64, K=64, type=0, x=P, ldx=64, nrows=3, offsets=P, space=P, space_bytes=BIG, y=P)
GRAD_W = dict(type=0, dy=P, ld_dy=64, x=P, ldx=64, n=4, N=64, K=64, nrows=3, offsets=P, out_type=0, dw=P)

MATRIX = [(dict(n=0), -1), (dict(n=1025), -1), (dict(N=0), -2), (dict(N=(1 << 20) + 1), -2), (dict(K=0), -2), (dict(K=40), -2),
          (dict(K=65552), -2)]
ROWS = [(dict(nrows=-1), -1), (dict(nrows=(1 << 22) + 1), -1), (dict(offsets=None), -1), (dict(offsets=ODD), -3)]
TOKENS = [(dict(type=3), -1), (dict(ntok=-1), -1), (dict(ntok=1 << 22), -1), (dict(top_k=0), -1), (dict(top_k=9), -1),
          (dict(n=0), -1), (dict(n=1025, ldl=2000), -1), (dict(n=1, top_k=2), -1), (dict(score=2), -1), (dict(ldl=7), -2),
          (dict(logits=None), -1), (dict(logits=ODD), -3), (dict(live=ODD), -3), (dict(ids=ODD), -3)]


@pytest.mark.parametrize("name,good,bad", [
    ("qmv_moe_router", ROUTER, TOKENS + [(dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(ids=None), -1),
                                         (dict(weights=None), -1), (dict(weights=ODD), -3)]),
    ("qmv_moe_balance", BALANCE, TOKENS + [(dict(ids=None), -1), (dict(counts=None), -1), (dict(means=None), -1),
                                           (dict(loss=None), -1), (dict(ws=None), -1), (dict(ws=ODD), -3), (dict(loss=ODD), -3),
                                           (dict(ws_bytes=10), -4)]),
    ("qmv_moe_router_grad", GRAD, TOKENS + [(dict(ldd=7), -2), (dict(dlogits=None), -1), (dict(ids=None), -1),
                                            (dict(counts=None), -1), (dict(dloss=None), -1), (dict(dloss=ODD), -3),
                                            (dict(dlogits=ODD), -3), (dict(scale=float("-inf")), -1)]),
    ("qmv_quantize_act_b128", QUANT, [(dict(type=3), -1), (dict(nrows=-1), -1), (dict(nrows=1 << 23), -1), (dict(K=0), -2),
                                      (dict(K=(1 << 20) + 1, ldx=1 << 21), -2), (dict(ldx=63), -2), (dict(x=None), -1),
                                      (dict(xq=None), -1), (dict(x=ODD), -3), (dict(xq=ODD), -3), (dict(xq_bytes=256 + 47), -4)]),
    ("qmv_quantize_weights_b128", QUANT_W, MATRIX + [(dict(type=-1), -1), (dict(w=None), -1), (dict(codes=ODD), -3), (dict(scales=None), -1),
                                                     (dict(n=1024, N=1 << 20, K=65536), -2)]),
    ("qmv_b128_product", PRODUCT, MATRIX + ROWS + [(dict(out_type=3), -1), (dict(w=None), -1), (dict(ws=None), -1), (dict(y=None), -1),
                                                   (dict(ws=ODD), -3), (dict(xq=ODD), -3), (dict(xq_bytes=256 + 47), -4)]),
    ("qmv_b128_grad_x", PRODUCT, MATRIX + ROWS + [(dict(out_type=-1), -1), (dict(xq=None), -1), (dict(y=ODD), -3),
                                                  (dict(xq_bytes=256 + 47), -4), (dict(N=600, xq_bytes=3 * 600), -4)]),
    ("qmv_b128_linear", LINEAR, MATRIX + ROWS + [(dict(type=3), -1), (dict(x=None), -1), (dict(x=ODD), -3), (dict(ldx=63), -2),
                                                 (dict(space=None), -1), (dict(space_bytes=256 + 47), -4), (dict(y=None), -1)]),
    ("qmv_b128_grad_w", GRAD_W, MATRIX + ROWS + [(dict(type=2), -1), (dict(out_type=3), -1), (dict(ld_dy=63), -2), (dict(ldx=56), -2),
                                                 (dict(ld_dy=68), -2), (dict(ldx=70), -2), (dict(dy=None), -1), (dict(dw=None), -1),
                                                 (dict(x=ODD), -3), (dict(dw=ODD), -3)]),
])
def test_refusals(name, good, bad):
    for over, code in bad:
        over = {k: v for k, v in over.items() if k in good}
        assert _call(name, good, **over) == code, (over, qmv.qmv_last_error())
        assert name in qmv.qmv_last_error()


def test_no_rows_is_valid():
    for name, good in (("qmv_moe_router", ROUTER), ("qmv_moe_router_grad", GRAD)):
        assert _call(name, good, ntok=0) == 0
    for name, good in (("qmv_quantize_act_b128", QUANT), ("qmv_b128_product", PRODUCT), ("qmv_b128_grad_x", PRODUCT),
                       ("qmv_b128_linear", LINEAR)):
        assert _call(name, good, nrows=0) == 0


def test_output_tensors_that_are_too_small_are_refused():
    one = torch.zeros(BIG >> 40, dtype=torch.uint8)

    def f32(n):
        return torch.zeros(n, dtype=torch.float32)

    calls = [
        (lambda t: qmv.qmv_moe_router("f32", P, 8, P, 4, 8, 2, "softmax", True, 1.0, t, P, 0), 8, "ids"),
        (lambda t: qmv.qmv_moe_router("f32", P, 8, P, 4, 8, 2, "softmax", True, 1.0, P, t, 0), 8, "weights"),
        (lambda t: qmv.qmv_moe_balance("f32", P, 8, P, P, 4, 8, 2, "softmax", t, P, P, one, 0), 9, "counts"),
        (lambda t: qmv.qmv_moe_balance("f32", P, 8, P, P, 4, 8, 2, "softmax", P, t, P, one, 0), 8, "means"),
        (lambda t: qmv.qmv_moe_balance("f32", P, 8, P, P, 4, 8, 2, "softmax", P, P, t, one, 0), 1, "loss"),
        (lambda t: qmv.qmv_moe_router_grad("f32", P, 8, P, P, P, P, P, 4, 8, 2, "softmax", True, 1.0, t, 10, 0), 38, "dlogits"),
        (lambda t: qmv.qmv_quantize_weights_b128("f32", P, 2, 64, 64, t, P, 0), 2 * 64 * 16, "codes"),
        (lambda t: qmv.qmv_quantize_weights_b128("f32", P, 2, 129, 64, P, t, 0), 4, "scales"),
        (lambda t: qmv.qmv_b128_product(P, P, 4, 64, 64, one, 3, P, "f32", t, 0), 3 * 64, "y"),
        (lambda t: qmv.qmv_b128_linear(P, P, 4, 64, 64, "f32", P, 64, 3, P, one, t, 0), 3 * 64, "y"),
        (lambda t: qmv.qmv_b128_grad_x(P, P, 4, 64, 96, one, 3, P, "f32", t, 0), 3 * 96, "dx"),
        (lambda t: qmv.qmv_b128_grad_w("bf16", P, 64, P, 96, 4, 64, 96, 3, P, "f32", t, 0), 4 * 64 * 96, "dw"),
    ]
    for call, need, what in calls:
        with pytest.raises(qmv.QmvError) as e:
            call(f32(need)[:need - 1].clone())
        assert e.value.code == qmv.QMV_ESIZE and f" {what} " in str(e.value)
