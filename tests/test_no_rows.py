"""Calls without rows or tokens, as a rank or an expert's batch without any makes them: with empty tensors, whose address is
NULL, and buffers of the sizes that the size functions give."""
import numpy as np
import pytest
import torch

qmv = pytest.importorskip("bit_quantized_moe_gb300", reason="libqmv not built")

E, N, K, TOP_K = 4, 64, 96, 2


def tensors(device):
    """What of the calls' operands does not depend on the rows."""
    return dict(w=torch.zeros(E, N, K, dtype=torch.uint8, device=device), ws=torch.zeros(E, 1, 1, device=device),
                offsets=torch.zeros(E + 1, dtype=torch.int32, device=device))


def rows(*shape, dtype=torch.bfloat16, device="cpu"):
    t = torch.empty(*shape, dtype=dtype, device=device)
    assert t.numel() == 0 and t.data_ptr() == 0
    return t


def space(n, device="cpu"):
    return torch.empty(n, dtype=torch.uint8, device=device)


def block_calls(device, stream=None):
    """(name, call) of the router and the products with a scale for each block of 128 that enqueue nothing."""
    t = tensors(device)

    def new(*shape, dtype=torch.bfloat16):
        return rows(*shape, dtype=dtype, device=device)

    def act(columns):
        return space(qmv.qmv_act_b128_bytes(0, columns), device)

    i32, f32 = torch.int32, torch.float32
    return [
        ("router", lambda: qmv.qmv_moe_router("bf16", new(0, E), E, new(0, dtype=torch.bool), 0, E, TOP_K, "softmax", True, 1.0,
                                              new(0, TOP_K, dtype=i32), new(0, TOP_K, dtype=f32), stream)),
        ("router_grad", lambda: qmv.qmv_moe_router_grad("bf16", new(0, E), E, None, new(0, TOP_K, dtype=i32), new(0, TOP_K, dtype=f32),
                                                        torch.zeros(E + 1, dtype=i32, device=device), torch.zeros(1, device=device), 0, E,
                                                        TOP_K, "softmax", True, 1.0, new(0, E), E, stream)),
        ("quantize", lambda: qmv.qmv_quantize_act_b128("bf16", new(0, K), K, 0, K, act(K), stream)),
        ("product", lambda: qmv.qmv_b128_product(t["w"], t["ws"], E, N, K, act(K), 0, t["offsets"], "bf16", new(0, N), stream)),
        ("dense product", lambda: qmv.qmv_b128_product(t["w"], t["ws"], 1, N, K, act(K), 0, None, "bf16", new(0, N), stream)),
        ("linear", lambda: qmv.qmv_b128_linear(t["w"], t["ws"], E, N, K, "bf16", new(0, K), K, 0, t["offsets"],
                                               space(qmv.qmv_b128_linear_workspace_bytes(0, K), device), new(0, N), stream)),
        ("grad_x", lambda: qmv.qmv_b128_grad_x(t["w"], t["ws"], E, N, K, act(N), 0, t["offsets"], "bf16", new(0, K), stream)),
    ]


@pytest.mark.parametrize("name", [name for name, _ in block_calls("cpu")])
def test_router_and_block_products(name):
    dict(block_calls("cpu", 0))[name]()   # the default stream's handle: nothing is enqueued


def test_unpack():
    assert qmv.lib.qmv_act_b128_unpack(None, 0, K, None, None) == 0
    codes, scales = qmv.qmv_act_b128_unpack(np.empty(0, np.uint8), 0, K)
    assert codes.shape == (0, K) and scales.shape == (0, 1)
    assert qmv.lib.qmv_act_b128_unpack(None, 1, K, None, None) == qmv.QMV_EINVAL


def test_what_does_not_depend_on_the_rows_is_still_needed():
    lib, P, odd = qmv.lib, 1 << 40, (1 << 40) + 4
    assert lib.qmv_b128_product(None, P, E, N, K, None, 0, 0, P, 0, None, 0) == -1
    assert lib.qmv_b128_product(P, None, E, N, K, None, 0, 0, P, 0, None, 0) == -1
    assert lib.qmv_b128_product(P, P, E, N, K, None, 0, 0, None, 0, None, 0) == -1   # rows of four experts need offsets
    assert lib.qmv_b128_product(odd, P, E, N, K, None, 0, 0, P, 0, None, 0) == -3
    assert lib.qmv_b128_product(P, P, E, N, 40, None, 0, 0, P, 0, None, 0) == -2
    assert lib.qmv_b128_linear(None, P, E, N, K, 0, None, K, 0, P, None, 0, None, 0) == -1
    assert lib.qmv_b128_grad_w(0, None, N, None, K, E, N, K, 0, P, 0, None, 0) == -1   # cleared all the same
    assert lib.qmv_moe_balance(0, None, E, None, None, 0, E, TOP_K, 0, None, P, P, P, 1 << 20, 0) == -1
    assert lib.qmv_moe_balance(0, None, E, None, None, 0, E, TOP_K, 0, P, P, P, None, 0, 0) == -1
    assert lib.qmv_moe_router_grad(0, None, E, None, None, None, P, None, 0, E, TOP_K, 0, 0, 1.0, None, E, 0) == -1
    assert lib.qmv_moe_router(0, None, E - 1, None, 0, E, TOP_K, 0, 0, 1.0, None, None, 0) == -2


def rows_calls(device, stream=None):
    """(name, call) of the other calls of many rows that enqueue nothing."""
    one, four = (qmv.wdesc("mxfp4", N, K, n) for n in (1, E))
    gate, down = qmv.wdesc("mxfp4", N, K, E), qmv.wdesc("mxfp8", K, N, E)
    w = torch.zeros(16, dtype=torch.uint8, device=device)   # stands for packed weights: not read
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=device)

    def new(*shape, dtype=torch.bfloat16):
        return rows(*shape, dtype=dtype, device=device)

    def act(fmt, columns):
        return space(qmv.qmv_act_mx_bytes(fmt, 0, columns), device)

    def row():
        return new(0, TOP_K, dtype=torch.int32)

    def weights():
        return new(0, TOP_K, dtype=torch.float32)

    return [
        ("quantize", lambda: qmv.qmv_quantize_act_mx("mxfp8", "bf16", new(0, K), K, 0, K, act("mxfp8", K), stream)),
        ("norm", lambda: qmv.qmv_rms_norm("bf16", new(0, K), K, new(0, K), K, torch.zeros(K, dtype=torch.bfloat16, device=device), 0, K,
                                          1e-5, new(0, K), "plain", new(0, K), stream)),
        ("norm to q8", lambda: qmv.qmv_rms_norm("bf16", new(0, K), K, None, K, torch.zeros(K, dtype=torch.bfloat16, device=device), 0, K,
                                                1e-5, None, "q8", space(0, device), stream)),
        ("product", lambda: qmv.qmv_mx_product(four, w, act("mxfp4", K), 0, offsets, "bf16", new(0, N), stream)),
        ("dense product", lambda: qmv.qmv_mx_product(one, w, act("mxfp4", K), 0, None, "f32", new(0, N, dtype=torch.float32), stream)),
        ("gate and up", lambda: qmv.qmv_mx_gate_up_swiglu(gate, w, act("mxfp4", K), 0, offsets, "mxfp8", act("mxfp8", N), stream)),
        ("dispatch", lambda: qmv.qmv_moe_dispatch("bf16", new(0, K), K, 0, TOP_K, K, row(), new(0, K), stream)),
        ("dispatch_mx", lambda: qmv.qmv_moe_dispatch_mx("mxfp4", "bf16", new(0, K), K, 0, TOP_K, K, row(), act("mxfp4", K), stream)),
        ("dispatch_grad", lambda: qmv.qmv_moe_dispatch_grad("bf16", new(0, K), 0, TOP_K, K, row(), new(0, K), K, stream)),
        ("return", lambda: qmv.qmv_moe_return("bf16", new(0, N), weights(), 0, TOP_K, N, row(), new(0, N), N, stream)),
        ("return_grad", lambda: qmv.qmv_moe_return_grad("bf16", new(0, N), N, new(0, N), weights(), 0, TOP_K, N, row(), new(0, N),
                                                        weights(), stream)),
        ("layer", lambda: qmv.qmv_moe_prefill_layer(gate, w, down, w, "bf16", new(0, K), K, row(), weights(), 0, TOP_K,
                                                    space(qmv.qmv_moe_prefill_layer_workspace_bytes(gate, down, 0, TOP_K), device),
                                                    new(0, K), stream)),
    ]


@pytest.mark.parametrize("name", [name for name, _ in rows_calls("cpu")])
def test_calls_of_many_rows(name):
    dict(rows_calls("cpu", 0))[name]()


def test_mx_unpack():
    assert qmv.lib.qmv_act_mx_unpack(0, None, 0, 64, None, None) == 0
    assert qmv.lib.qmv_act_mx_unpack(0, None, 1, 64, None, None) == qmv.QMV_EINVAL


def test_calls_of_many_rows_still_need_the_rest():
    lib, P, by = qmv.lib, 1 << 40, qmv.ctypes.byref
    four = qmv.wdesc("mxfp4", N, K, E)
    assert lib.qmv_mx_product(by(four), None, None, 0, 0, P, 0, None, 0) == -1
    assert lib.qmv_mx_product(by(four), P, None, 0, 0, None, 0, None, 0) == -1   # rows of four experts need offsets
    assert lib.qmv_rms_norm(0, None, K, None, K, None, 0, K, 1e-5, None, 0, None, 0, 0) == -1   # the gain
    assert lib.qmv_moe_sort(None, 0, TOP_K, E, None, None, None, None, 0, 0) == -1   # written all the same
    assert lib.qmv_moe_prefill_layer(by(four), P, by(qmv.wdesc("mxfp4", K, N, E)), P, 0, None, K, None, None, 0, TOP_K, None, 0, None, 0) == -1


@pytest.mark.gpu
def test_calls_of_many_rows_on_a_gpu():
    for name, call in rows_calls("cuda"):
        call()
    offsets = torch.full((E + 1,), 7, dtype=torch.int32, device="cuda")
    ids, row, slot = (rows(0, TOP_K, dtype=torch.int32, device="cuda") for _ in range(3))
    qmv.qmv_moe_sort(ids, 0, TOP_K, E, offsets, row, slot)
    assert not offsets.any() and qmv.qmv_device_status() == 0


@pytest.mark.gpu
def test_router_and_block_products_on_a_gpu():
    """The same on the device, and what is written without rows: the loss's zeros, the weights' gradient of zeros."""
    for name, call in block_calls("cuda"):
        call()
    counts, means, loss = torch.full((E + 1,), 7, dtype=torch.int32, device="cuda"), torch.full((E,), 7.0, device="cuda"), torch.full((1,), 7.0, device="cuda")
    ids = rows(0, TOP_K, dtype=torch.int32, device="cuda")
    qmv.qmv_moe_balance("bf16", rows(0, E, device="cuda"), E, None, ids, 0, E, TOP_K, "sigmoid", counts, means, loss,
                        space(qmv.qmv_moe_balance_workspace_bytes(0, E), "cuda"))
    assert not counts.any() and not means.any() and not loss.any()
    dw = torch.full((E, N, K), 7.0, dtype=torch.bfloat16, device="cuda")
    qmv.qmv_b128_grad_w("bf16", rows(0, N, device="cuda"), N, rows(0, K, device="cuda"), K, E, N, K, 0,
                        tensors("cuda")["offsets"], "bf16", dw)
    assert not dw.any() and qmv.qmv_device_status() == 0
