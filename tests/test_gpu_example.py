"""The example of a MoE block runs: prompt and decode on the same weights agree to the activations' quantization, and the
training step's gradients are those of torch's own indexing."""
import importlib.util
import os

import pytest
import torch

pytest.importorskip("bit_quantized_moe_gb300")
pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")


def example():
    spec = importlib.util.spec_from_file_location("moe_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


# Relative error of a product whose activations are rounded to E2M1 (a half step is up to 1/4 .. 1/8 of a value: about 0.1 in
# the root mean square) or E4M3 (1/32), twice along the layer, h's error entering once more through silu's product.
@pytest.mark.parametrize("fmt,apart", [("mxfp4", 0.35), ("mxfp8", 0.09)])
def test_moe_block(fmt, apart):
    got, loss, grads = example().main(["--tokens", "70", "--hidden", "288", "--inner", "160", "--experts", "8", "--top-k", "2",
                                       "--fmt", fmt])
    assert 0 < got < apart and loss > 0
    assert all(torch.isfinite(g.float()).all() and g.float().norm() > 0 for g in grads)


def test_routed_gradients_match_torch():
    m = example()
    tokens, experts, top_k, width = 33, 6, 3, 96
    g = torch.Generator(device=m.DEV).manual_seed(3)
    x = torch.randn(tokens, width, generator=g, device=m.DEV).bfloat16().requires_grad_()
    weights = torch.rand(tokens, top_k, generator=g, device=m.DEV).requires_grad_()
    ids = torch.rand(tokens, experts, generator=g, device=m.DEV).topk(top_k).indices
    slot = torch.argsort(ids.flatten(), stable=True)
    row = torch.empty_like(slot)
    row[slot] = torch.arange(len(slot), device=m.DEV)
    dy = torch.randn(tokens, width, generator=g, device=m.DEV).bfloat16()

    y = m.Returned.apply(m.Routed.apply(x, row.to(torch.int32), top_k), weights, row.to(torch.int32))
    mine = torch.autograd.grad(y, (x, weights), dy)
    xs = x.double()[slot // top_k]
    want = (xs[row].view(tokens, top_k, width) * weights.double()[..., None]).sum(1)
    theirs = torch.autograd.grad(want, (x, weights), dy.double())
    # bf16 steps: y, the rows' gradients and dx are each rounded once (2^-8 relative to the largest term's size)
    assert (y.double() - want).abs().max() <= 2 ** -8 * want.abs().max()
    assert (mine[0].double() - theirs[0].double()).abs().max() <= 2 * 2 ** -8 * theirs[0].double().abs().max()
    assert (mine[1].double() - theirs[1].double()).abs().max() <= 1e-5 * theirs[1].double().abs().max()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_routed_functions_take_strides_and_types_as_they_come(dtype):
    """Transposed and expanded tokens, rows, weights and gradients, in each type, give what their contiguous copies give."""
    m = example()
    tokens, experts, top_k, width = 21, 5, 3, 40
    g = torch.Generator(device=m.DEV).manual_seed(5)
    ids = torch.rand(tokens, experts, generator=g, device=m.DEV).topk(top_k).indices
    slot = torch.argsort(ids.flatten(), stable=True)
    row = torch.empty_like(slot)
    row[slot] = torch.arange(len(slot), device=m.DEV)
    row = row.to(torch.int32)

    def turned(*shape):
        return torch.randn(*reversed(shape), generator=g, device=m.DEV).to(dtype).T

    x, ys, dxs, dy = turned(tokens, width), turned(tokens * top_k, width), turned(tokens * top_k, width), turned(tokens, width)
    weights = torch.rand(top_k, tokens, generator=g, device=m.DEV).T
    one = torch.randn(1, width, generator=g, device=m.DEV).to(dtype).expand(tokens, width)

    def results(x, ys, weights, dxs, dy):
        x, ys, weights = (t.detach().requires_grad_() for t in (x, ys, weights))
        xs, y = m.Routed.apply(x, row, top_k), m.Returned.apply(ys, weights, row)
        return [xs, y, *torch.autograd.grad(xs, x, dxs), *torch.autograd.grad(y, (ys, weights), dy)]

    for tok in (x, one):
        args = (tok, ys, weights, dxs, dy)
        got, want = results(*args), results(*(t.contiguous() for t in args))
        assert all(a.dtype == b.dtype and torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(got[0], tok[slot // top_k])
