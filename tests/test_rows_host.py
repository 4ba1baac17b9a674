"""Host-side tests of the many-row calls: the 64-bit definitions that the GPU
tests compare with, the activation buffer's layout, and the refusals, which
come before anything is enqueued."""
import numpy as np
import pytest
import torch

import oracle
import qmv_inputs as qi
import rows_reference as ref

qmv = pytest.importorskip("bit_quantized_moe_gb300", reason="libqmv not built")

P = 1 << 40          # an aligned device address that no check reads
ODD = P + 4
BIG = 1 << 50


def test_element_values_match_the_oracle():
    assert np.array_equal(ref.element_values("mxfp4"), oracle.e2m1_decode(np.arange(16, dtype=np.uint8)))
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.element_values("mxfp8"), want, equal_nan=True)


def test_nearest_codes_e4m3_match_torch():
    v = np.concatenate([np.linspace(-470, 470, 4001), np.geomspace(2.0 ** -12, 448, 4000)]).astype(np.float32)
    want = torch.from_numpy(np.clip(v, -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.nearest_codes(v.astype(np.float64), "mxfp8"), want)


def test_nearest_codes_e2m1_ties_go_to_even():
    v = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, -0.25, -5.0, 0.2500001])
    assert ref.nearest_codes(v, "mxfp4").tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 8, 14, 1]


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (5, 128), (7, 160), (130, 2880)])
def test_act_buffer_layout(fmt, rows, K):
    g = qi.rng(rows + K)
    codes = g.integers(0, 16 if fmt == "mxfp4" else 256, size=(rows, K), dtype=np.uint8)
    scales = g.integers(0, 256, size=(rows, K // 32), dtype=np.uint8)
    buf = ref.act_buffer(codes, scales, fmt)
    assert buf.nbytes == qmv.qmv_act_mx_bytes(fmt, rows, K)
    assert qmv.qmv_act_mx_scale_offset(fmt, rows, K) % 128 == 0
    c, s = qmv.qmv_act_mx_unpack(fmt, buf, rows, K)
    assert np.array_equal(c, ref.pack_rows(codes, fmt)) and np.array_equal(s, scales)


def test_act_sizes_of_invalid_shapes_are_zero():
    for fmt, rows, K in (("cb4", 1, 32), (9, 1, 32), ("mxfp4", -1, 32), ("mxfp4", qmv.MAX_ROWS + 1, 32),
                         ("mxfp8", 1, 31), ("mxfp8", 1, 0), ("mxfp8", 1, 65568)):
        assert qmv.qmv_act_mx_bytes(fmt, rows, K) == 0
        assert qmv.qmv_act_mx_scale_offset(fmt, rows, K) == 0
    # the largest buffer passes 32 bits
    assert qmv.qmv_act_mx_bytes("mxfp8", qmv.MAX_ROWS, 65536) > 1 << 38


def _call(name, good, **over):
    """The entry point with `good` arguments (in order), some of them replaced."""
    args = {**good, **over}
    return getattr(qmv.lib, name)(*[qmv.ctypes.byref(v) if isinstance(v, qmv.WDesc) else v for v in args.values()], 0)


QUANT = dict(fmt=0, type=0, x=P, ldx=64, nrows=3, K=64, xq=P, xq_bytes=BIG)
NORM = dict(type=0, x=P, ldx=64, res=P, ldr=64, gain=P, nrows=3, K=64, eps=1e-5, sum=P, out=1, y=P, y_bytes=BIG)
SORT = dict(ids=P, ntok=4, top_k=2, n=8, offsets=P, row=P, slot=P, ws=None, ws_bytes=0)
DISPATCH = dict(type=0, x=P, ldx=64, ntok=4, top_k=2, K=64, row=P, xs=P)
DISPATCH_MX = dict(fmt=0, type=0, x=P, ldx=64, ntok=4, top_k=2, K=64, row=P, xq=P, xq_bytes=BIG)
DISPATCH_GRAD = dict(type=0, dxs=P, ntok=4, top_k=2, K=64, row=P, dx=P, ldx=64)
RETURN = dict(type=0, ys=P, weights=P, ntok=4, top_k=2, N=64, row=P, y=P, ldy=64)
RETURN_GRAD = dict(type=0, dy=P, ld=64, ys=P, weights=P, ntok=4, top_k=2, N=64, row=P, dys=P, dw=P)


def product(**over):
    good = dict(desc=qmv.wdesc("mxfp4", 64, 64, 4), w=P, xq=P, xq_bytes=BIG, nrows=3, offsets=P, out_type=0, y=P)
    return _call("qmv_mx_product", good, **over)


def gate_up(**over):
    good = dict(desc=qmv.wdesc("mxfp4", 64, 64, 4), w=P, xq=P, xq_bytes=BIG, nrows=3, offsets=P, h_fmt=0, hq=P, hq_bytes=BIG)
    return _call("qmv_mx_gate_up_swiglu", good, **over)


def layer(**over):
    good = dict(gu=qmv.wdesc("mxfp4", 64, 96, 4), w_gu=P, down=qmv.wdesc("mxfp8", 96, 64, 4), w_down=P, type=0, x=P,
                ldx=96, ids=P, weights=P, ntok=3, top_k=2, ws=P, ws_bytes=BIG, y=P)
    return _call("qmv_moe_prefill_layer", good, **over)


@pytest.mark.parametrize("name,good,bad", [
    ("qmv_quantize_act_mx", QUANT, [(dict(fmt=1), -1), (dict(type=3), -1), (dict(nrows=-1), -1), (dict(nrows=1 << 23), -1),
                                    (dict(K=48), -2), (dict(K=0), -2), (dict(ldx=63), -2), (dict(x=None), -1),
                                    (dict(xq=None), -1), (dict(x=ODD), -3), (dict(xq=ODD), -3), (dict(xq_bytes=111), -4)]),
    ("qmv_rms_norm", NORM, [(dict(type=-1), -1), (dict(out=4), -1), (dict(nrows=-2), -1), (dict(K=33), -2),
                            (dict(K=65568), -2), (dict(ldx=32), -2), (dict(ldr=32), -2), (dict(eps=-1.0), -1),
                            (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1), (dict(gain=None), -1),
                            (dict(x=None), -1), (dict(y=None), -1), (dict(res=ODD), -3), (dict(sum=ODD), -3),
                            (dict(y_bytes=100), -4), (dict(out=0, y_bytes=3 * 64 * 2 - 1), -4),
                            (dict(out=3, y_bytes=3 * 80 - 1), -4)]),
    ("qmv_moe_sort", SORT, [(dict(ntok=-1), -1), (dict(top_k=0), -1), (dict(top_k=9), -1), (dict(ntok=1 << 22), -1),
                            (dict(n=0), -1), (dict(n=1025), -1), (dict(ids=None), -1), (dict(row=None), -1),
                            (dict(offsets=ODD), -3)]),
    ("qmv_moe_dispatch", DISPATCH, [(dict(type=7), -1), (dict(ntok=-1), -1), (dict(K=0), -2), (dict(ldx=60), -2),
                                    (dict(row=None), -1), (dict(xs=None), -1), (dict(xs=ODD), -3), (dict(row=ODD), -3)]),
    ("qmv_moe_dispatch_mx", DISPATCH_MX, [(dict(fmt=2), -1), (dict(K=40), -2), (dict(ldx=32), -2), (dict(x=None), -1),
                                          (dict(xq=ODD), -3), (dict(xq_bytes=10), -4)]),
    ("qmv_moe_dispatch_grad", DISPATCH_GRAD, [(dict(ldx=63), -2), (dict(dxs=None), -1), (dict(dx=ODD), -3)]),
    ("qmv_moe_return", RETURN, [(dict(ldy=63), -2), (dict(weights=None), -1), (dict(ys=ODD), -3), (dict(top_k=9), -1)]),
    ("qmv_moe_return_grad", RETURN_GRAD, [(dict(ld=1), -2), (dict(dw=None), -1), (dict(dy=ODD), -3), (dict(N=0), -2)]),
])
def test_refusals(name, good, bad):
    for over, code in bad:
        assert _call(name, good, **over) == code, (over, qmv.qmv_last_error())
        assert name in qmv.qmv_last_error()


def test_product_refusals():
    assert product(desc=qmv.wdesc("cb4", 64, 64, 4, qi.LUT_CB4)) == -1
    assert product(offsets=None) == -1                                   # dense with four experts
    assert product(desc=qmv.wdesc("mxfp4", 64, 64, 1025)) == -1
    assert product(desc=qmv.wdesc("mxfp4", 64, 40, 4)) == -2
    assert product(nrows=-1) == -1 and product(out_type=3) == -1
    assert product(w=None) == -1 and product(y=None) == -1
    assert product(xq=ODD) == -3 and product(offsets=ODD) == -3
    assert product(xq_bytes=qmv.qmv_act_mx_bytes("mxfp4", 3, 64) - 1) == -4 and gate_up(xq_bytes=7) == -4
    assert product(nrows=0) == 0                                         # nothing to do, nothing enqueued
    assert gate_up(h_fmt=1) == -1 and gate_up(hq_bytes=5) == -4
    assert gate_up(desc=qmv.wdesc("mxfp4", 48, 64, 4)) == -2             # h in groups of 32
    assert gate_up(nrows=0) == 0
    assert gate_up(hq=ODD) == -3


def test_layer_refusals():
    assert layer(down=qmv.wdesc("mxfp4", 96, 96, 4)) == -2
    assert layer(down=qmv.wdesc("mxfp4", 96, 64, 3)) == -1
    assert layer(down=qmv.wdesc("cb4", 96, 64, 4, qi.LUT_CB4)) == -1
    assert layer(type=2) == -1 and layer(ldx=95) == -2 and layer(top_k=9) == -1
    assert layer(ids=None) == -1 and layer(ws=ODD) == -3 and layer(ws_bytes=64) == -4
    assert layer(ntok=0) == 0
    gu, down = qmv.wdesc("mxfp4", 64, 96, 4), qmv.wdesc("mxfp8", 96, 64, 4)
    assert qmv.qmv_moe_prefill_layer_workspace_bytes(gu, down, 3, 2) > 0
    assert qmv.qmv_moe_prefill_layer_workspace_bytes(gu, gu, 3, 2) == 0
    assert qmv.qmv_moe_prefill_layer_workspace_bytes(gu, down, 3, 0) == 0


def test_no_rows_is_valid():
    for name, good in (("qmv_quantize_act_mx", QUANT), ("qmv_rms_norm", NORM)):
        assert _call(name, good, nrows=0) == 0
    for name, good in (("qmv_moe_dispatch", DISPATCH), ("qmv_moe_dispatch_mx", DISPATCH_MX),
                       ("qmv_moe_dispatch_grad", DISPATCH_GRAD), ("qmv_moe_return", RETURN),
                       ("qmv_moe_return_grad", RETURN_GRAD)):
        assert _call(name, good, ntok=0) == 0


def test_widths_of_the_routed_rows():
    """Dispatched rows are a product's input (K), returned ones its output (N): each takes what the product takes."""
    for name, good, ld in (("qmv_moe_return", RETURN, "ldy"), ("qmv_moe_return_grad", RETURN_GRAD, "ld")):
        assert _call(name, good, ntok=0, N=1 << 20, **{ld: 1 << 20}) == 0
        assert _call(name, good, ntok=0, N=(1 << 20) + 1, **{ld: 1 << 21}) == -2
    for name, good in (("qmv_moe_dispatch", DISPATCH), ("qmv_moe_dispatch_grad", DISPATCH_GRAD)):
        assert _call(name, good, ntok=0, K=65536, ldx=65536) == 0
        assert _call(name, good, ntok=0, K=65537, ldx=65537) == -2


def test_output_tensors_that_are_too_small_are_refused():
    """Rows and gradients whose C call takes no size: the binding compares their tensors with what the call writes."""
    desc = qmv.wdesc("mxfp4", 64, 64, 4)
    down = qmv.wdesc("mxfp8", 96, 64, 4)
    one = torch.zeros(BIG >> 40, dtype=torch.uint8)   # stands for buffers whose size the C call takes

    def f32(n):
        return torch.zeros(n, dtype=torch.float32)

    calls = [
        (lambda t: qmv.qmv_rms_norm("f32", P, 64, P, 70, P, 3, 64, 1e-5, t, "plain", one, 0), f32, 2 * 70 + 64, "sum"),
        (lambda t: qmv.qmv_mx_product(desc, P, one, 3, P, "f32", t, 0), f32, 3 * 64, "y"),
        (lambda t: qmv.qmv_moe_dispatch("f32", P, 64, 4, 2, 64, P, t, 0), f32, 8 * 64, "xs"),
        (lambda t: qmv.qmv_moe_dispatch_grad("f32", P, 4, 2, 64, P, t, 70, 0), f32, 3 * 70 + 64, "dx"),
        (lambda t: qmv.qmv_moe_return("f32", P, P, 4, 2, 64, P, t, 70, 0), f32, 3 * 70 + 64, "y"),
        (lambda t: qmv.qmv_moe_return_grad("f32", P, 64, P, P, 4, 2, 64, P, t, f32(8), 0), f32, 8 * 64, "dys"),
        (lambda t: qmv.qmv_moe_return_grad("f32", P, 64, P, P, 4, 2, 64, P, f32(512), t, 0), f32, 8, "dweights"),
        (lambda t: qmv.qmv_moe_prefill_layer(qmv.wdesc("mxfp4", 64, 96, 4), P, down, P, "bf16", P, 96, P, P, 3, 2, one, t, 0),
         lambda n: torch.zeros(n, dtype=torch.bfloat16), 3 * 96, "y"),
    ]
    for call, new, need, what in calls:
        with pytest.raises(qmv.QmvError) as e:
            call(new(need - 1))
        assert e.value.code == qmv.QMV_ESIZE and f" {what} " in str(e.value)
    # a view of rows that lie further apart holds what its storage holds from its first element on
    wide = f32(4 * 70)
    qmv._short("call", "y", wide.view(4, 70)[:, :64], 4 * (3 * 70 + 64))
    with pytest.raises(qmv.QmvError):
        qmv._short("call", "y", wide.view(4, 70)[1:, :64], 4 * (3 * 70 + 64))
