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
