"""The router and the products with a scale for each block of 128 where indexes pass 32 bits, and at the ends of their limits.
Operands are small integers, so that every sum is exact; rows are looked at where they lie far apart."""
import numpy as np
import pytest
import torch

qmv = pytest.importorskip("bit_quantized_moe_gb300")
import qmv_inputs as qi  # noqa: E402
import rows_reference as ref  # noqa: E402
import train_reference as tr  # noqa: E402
from qmv_testutil import DEV, status_clean  # noqa: E402

pytestmark = pytest.mark.gpu

INTS = ref.nearest_codes(np.arange(-3, 4, dtype=np.float64), "mxfp8")


def codes(seed, *shape):
    """Codes of integers up to 3 on the device."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.from_numpy(INTS).to(DEV)[torch.randint(0, 7, shape, generator=g, device=DEV)]


def values(c):
    return c.view(torch.float8_e4m3fn).double()


def act(c, seed):
    """An activation buffer of these codes, and its scales (1 or 2)."""
    rows, K = c.shape
    g = torch.Generator(device=DEV).manual_seed(seed)
    b = torch.zeros(qmv.qmv_act_b128_bytes(rows, K), dtype=torch.uint8, device=DEV)
    wide, blocks = -(-K // 16) * 16, -(-K // 128)
    b[:rows * wide].view(rows, wide)[:, :K] = c
    s = torch.randint(1, 3, (rows, blocks), generator=g, device=DEV).float()
    at, row = qmv.qmv_act_b128_scale_offset(rows, K), -(-blocks // 4) * 4
    b[at:at + rows * row * 4].view(torch.float32).view(rows, row)[:, :blocks] = s
    return b, s


def spread(c, s):
    return values(c) * torch.repeat_interleave(s, 128, 1)[:, :c.shape[1]]


def look(rows):
    return torch.tensor(sorted({0, 1, rows // 3, rows // 2 + 1, rows - 200, rows - 129, rows - 2, rows - 1}), device=DEV)


@pytest.mark.parametrize("rows,N,K", [((1 << 17) + 70, 40, 16400), ((1 << 20) + 77, 2056, 144)])
def test_rows_past_32_bits(rows, N, K):
    """Codes, and outputs, of more than 2^31 elements."""
    c, w = codes(1, rows, K), codes(2, 1, N, K)
    xq, s = act(c, 3)
    ws = torch.ones(1, -(-N // 128), -(-K // 128), device=DEV)
    at = look(rows)
    y = torch.empty(rows, N, dtype=torch.bfloat16, device=DEV)
    qmv.qmv_b128_product(w, ws, 1, N, K, xq, rows, None, "bf16", y)
    want = spread(c[at], s[at]) @ values(w[0]).T
    assert torch.equal(y[at].double(), want.to(torch.bfloat16).double())
    del y
    # the gradient of x has the roles of N and K exchanged: its outputs are rows x K
    dc = codes(4, rows, N)
    dyq, ds = act(dc, 5)
    dx = torch.empty(rows, K, dtype=torch.bfloat16, device=DEV)
    qmv.qmv_b128_grad_x(w, ws, 1, N, K, dyq, rows, None, "bf16", dx)
    assert torch.equal(dx[at].double(), (spread(dc[at], ds[at]) @ values(w[0])).to(torch.bfloat16).double())
    assert status_clean()


@pytest.mark.parametrize("rows", [9, 600])
def test_weights_past_32_bits(rows):
    """Experts whose matrices lie past 2^31 bytes, in the products and as gradients."""
    E, N, K = 70, 4096, 8208
    w = codes(1, E, N, K)
    ws = torch.ones(E, 32, 65, device=DEV)
    ends = sorted(int(v) for v in qi.rng(rows).integers(0, rows + 1, size=E - 1))
    offsets = torch.tensor([0, *ends, rows], dtype=torch.int32, device=DEV)
    c = codes(2, rows, K)
    xq, s = act(c, 3)
    y = torch.empty(rows, N, device=DEV)
    qmv.qmv_b128_product(w, ws, E, N, K, xq, rows, offsets, "f32", y)
    xv = spread(c, s)
    parts = tr.ranges(offsets.cpu().numpy(), rows, E)
    for e in (0, 1, E // 2, E - 2, E - 1):
        a, b = parts[e]
        assert torch.equal(y[a:b].double(), xv[a:b] @ values(w[e]).T), e
    dy = values(codes(4, rows, N)).bfloat16()
    dw = torch.full((E, N, K), 7.0, dtype=torch.bfloat16, device=DEV)
    qmv.qmv_b128_grad_w("bf16", dy, N, values(c).bfloat16(), K, E, N, K, rows, offsets, "bf16", dw)
    for e in (0, 1, E // 2, E - 2, E - 1):
        a, b = parts[e]
        assert torch.equal(dw[e].double(), (dy[a:b].double().T @ values(c[a:b])).to(torch.bfloat16).double()), e
    assert status_clean()


def test_quantizers_past_32_bits():
    rows, K = (1 << 20) + 3, 2064
    x = torch.randn(rows, K, dtype=torch.bfloat16, device=DEV)
    xq = torch.zeros(qmv.qmv_act_b128_bytes(rows, K), dtype=torch.uint8, device=DEV)
    qmv.qmv_quantize_act_b128("bf16", x, K, rows, K, xq)
    at = look(rows)
    wc, ws = tr.quantize_rows(x[at].double().cpu().numpy())
    assert np.array_equal(xq[:rows * K].view(rows, K)[at].cpu().numpy(), wc)
    o = qmv.qmv_act_b128_scale_offset(rows, K)
    assert np.array_equal(xq[o:].view(torch.float32).view(rows, 20)[at][:, :17].cpu().numpy(), ws.astype(np.float32))
    del xq
    # the same numbers as 8 matrices of 131,072 rows and a bit more than 2^31 elements in all
    N = 131072
    w = x[:8 * N].view(8, N, K)
    codes_, scales = torch.zeros(8, N, K, dtype=torch.uint8, device=DEV), torch.zeros(8, 1024, 17, device=DEV)
    qmv.qmv_quantize_weights_b128("bf16", w, 8, N, K, codes_, scales)
    for e in (0, 7):
        wc, ws = tr.quantize_weights(w[e:e + 1, -128:].double().cpu().numpy())
        assert np.array_equal(codes_[e, -128:].cpu().numpy(), wc[0])
        assert np.array_equal(scales[e, -1].cpu().numpy(), ws[0, 0].astype(np.float32))


def test_router_past_32_bits():
    tokens, experts, top_k, ld = 1 << 21, 1024, 2, 1032   # the most slots that a call takes
    rows = torch.randn(tokens, ld, dtype=torch.bfloat16, device=DEV)
    l = rows[:, :experts]
    ids, w = torch.empty(tokens, top_k, dtype=torch.int32, device=DEV), torch.empty(tokens, top_k, device=DEV)
    qmv.qmv_moe_router("bf16", rows, ld, None, tokens, experts, top_k, "softmax", True, 1.0, ids, w)
    at = look(tokens)
    want_ids, want = tr.route(l[at].double().cpu().numpy(), np.ones(len(at), bool), top_k, "softmax", True, 1.0)
    assert np.array_equal(ids[at].cpu().numpy(), want_ids)
    # two exponentials of differences below 10, their sum and quotient: 2 (10 + 8) + 14 roundings
    assert (np.abs(w[at].double().cpu().numpy() - want) <= 50 * 2.0 ** -24 * want).all()
    counts, means, loss = torch.empty(experts + 1, dtype=torch.int32, device=DEV), torch.empty(experts, device=DEV), torch.empty(1, device=DEV)
    ws = torch.empty(qmv.qmv_moe_balance_workspace_bytes(tokens, experts), dtype=torch.uint8, device=DEV)
    qmv.qmv_moe_balance("bf16", rows, ld, None, ids, tokens, experts, top_k, "softmax", counts, means, loss, ws)
    assert torch.equal(counts[:-1], torch.bincount(ids.flatten(), minlength=experts).int()) and counts[-1] == tokens
    d = torch.empty_like(rows)
    dl = torch.ones(1, device=DEV)
    qmv.qmv_moe_router_grad("bf16", rows, ld, None, ids, None, counts, dl, tokens, experts, top_k, "softmax", True, 1.0, d, ld)
    want, size = tr.router_grad(l[at].double().cpu().numpy(), np.ones(len(at), bool), want_ids, None, counts.cpu().numpy(), 1.0, top_k,
                                "softmax", True, 1.0)
    # stored in bf16: half a step of 2^-8 besides
    assert (np.abs(d[at, :experts].double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 150 * 2.0 ** -24 * size + 2.0 ** -133).all()


@pytest.mark.parametrize("rows", [1, 70, 700])
def test_most_columns(rows):
    """The most outputs that a matrix may have, the gradient's depth."""
    N, K = 1 << 20, 48
    w, dc, xc = codes(4, 1, N, K), codes(5, rows, N), codes(6, rows, K)
    ws = torch.ones(1, N // 128, 1, device=DEV)
    xq, xs = act(xc, 7)
    dyq, ds = act(dc, 8)
    y, dx = torch.empty(rows, N, device=DEV), torch.empty(rows, K, device=DEV)
    qmv.qmv_b128_product(w, ws, 1, N, K, xq, rows, None, "f32", y)
    qmv.qmv_b128_grad_x(w, ws, 1, N, K, dyq, rows, None, "f32", dx)
    at = torch.tensor([0, 1, 129, N // 2, N - 130, N - 1], device=DEV)
    assert torch.equal(y[:, at].double(), spread(xc, xs) @ values(w[0, at]).T)
    dv, wv, want = spread(dc, ds), values(w[0]), torch.zeros(rows, K, dtype=torch.float64, device=DEV)
    for n in range(0, N, 1 << 16):
        want += dv[:, n:n + (1 << 16)] @ wv[n:n + (1 << 16)]
    # terms of at most 18, of both signs: the sum of 2^20 wanders some 2^13, far below the 2^24 up to which fp32 is exact
    assert want.abs().max() < 2.0 ** 20 and torch.equal(dx.double(), want)
    dw = torch.empty(1, N, K, device=DEV)
    qmv.qmv_b128_grad_w("bf16", values(dc).bfloat16(), N, values(xc).bfloat16(), K, 1, N, K, rows, None, "f32", dw)
    assert torch.equal(dw[0, at].double(), values(dc[:, at]).T @ values(xc))
    assert status_clean()
