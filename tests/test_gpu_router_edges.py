"""The router, its balance loss and their gradient at the edges of what their calls allow, against the 64-bit definitions.

Tolerances. __expf is documented as off by at most 2 + |1.173 x| units in the last place: (4 + 2.4 |x|) * 2^-24 of the value.
Its argument l - top is rounded once, |x| * 2^-24 more, so that an exponential of numbers that span R is within
a = (4 + 3.4 R) * 2^-24. A sigmoid adds another exponential, at most half of its denominator, and two roundings: 1.5 a + 2 * 2^-24.
A score's share divides two such numbers, of which the lower is a sum (E / 32 additions in a lane and five levels), by a
reciprocal and a product: 3 a + (E / 32 + 12) * 2^-24. A mean of T shares adds its longest chain of additions, at most
T / 16 + 80 of them; the loss the fraction's and the product's four roundings and the additions of at most 18 numbers in a row.
A gradient's terms are products of at most three such numbers b, one of them behind a sum over the experts, with the fraction
and the loss's factor of three roundings each and the additions of the two parts: 3 b + (E / 32 + 24) * 2^-24 of the sum of their
magnitudes. Numbers below 2^-126 may be lost whole: 2^-120 is added. An output of 16 bits is the fp32 result rounded to
nearest (assert_within)."""
import numpy as np
import pytest
import torch

qmv = pytest.importorskip("bit_quantized_moe_gb300")
import qmv_inputs as qi  # noqa: E402
import train_reference as tr  # noqa: E402
from qmv_testutil import DEV, assert_within, status_clean  # noqa: E402

pytestmark = pytest.mark.gpu

MODES = [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)]


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def host(t):
    return t.double().cpu().numpy()


def share_error(l, experts, more=0):
    fine = l[np.isfinite(l)]
    span = float(max(np.abs(fine).max(), fine.max() - fine.min())) if fine.size else 0.0
    return (3 * (4 + 3.4 * span) + experts / 32 + 12 + more) * 2.0 ** -24


def logits(seed, tokens, experts, spread=2.0):
    g = qi.rng(seed)
    return (g.standard_normal((tokens, experts)) * spread + g.standard_normal(experts)).astype(np.float32)


def balance(l, ids, top_k, score):
    tokens, experts = l.shape
    counts, means, loss = torch.full((experts + 1,), 77, dtype=torch.int32, device=DEV), torch.full((experts,), 7.0, device=DEV), torch.full((1,), 7.0, device=DEV)
    ws = torch.full((qmv.qmv_moe_balance_workspace_bytes(tokens, experts),), 0xA5, dtype=torch.uint8, device=DEV)
    qmv.qmv_moe_balance("f32", l, experts, None, ids, tokens, experts, top_k, score, counts, means, loss, ws)
    return counts, means, loss


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens", [65, 1000])
@pytest.mark.parametrize("experts", [128, 129, 256, 257, 512, 640, 1024])
def test_loss_of_parts_of_several_ctas(experts, tokens, score):
    """One to eight CTAs add up the loss: none of their parts is lost, beside another stream's clusters too."""
    l = logits(experts + tokens, tokens, experts)
    ids = np.argsort(-l, axis=1, kind="stable")[:, :4].astype(np.int32)
    ld, idd = dev(l), dev(ids)
    first = balance(ld, idd, 4, score)
    wc, wm, wl = tr.balance(l.astype(np.float64), np.ones(tokens, bool), ids, 4, score)
    bound = share_error(l, experts, tokens / 16 + 80)
    assert np.array_equal(first[0].cpu().numpy(), wc)
    assert_within(host(first[1]), wm, bound * wm + 2.0 ** -120, "f32", "means")
    assert_within(host(first[2])[0], wl, (bound + 22 * 2.0 ** -24) * wl, "f32", "loss")
    slots = 1 << 16
    sort = [torch.empty(n, dtype=torch.int32, device=DEV) for n in (65, slots, slots)]
    some = torch.randint(0, 64, (slots,), dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    other, again = torch.cuda.Stream(), []
    for _ in range(50):
        with torch.cuda.stream(other):
            qmv.qmv_moe_sort(some, slots, 1, 64, *sort)
        again.append(balance(ld, idd, 4, score))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for got in again for a, b in zip(first, got))
    assert status_clean()


@pytest.mark.parametrize("score,renorm", MODES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradient_in_the_place_of_padded_strided_logits(score, renorm, dtype):
    """The logits' own place, rows further apart than they are wide, padding, and experts named twice, so that a lane's logit is
    read by many and overwritten by one: the bits of a call with a place of its own, and nothing between the rows."""
    tokens, top_k = 4000, 8
    g = qi.rng(21)
    for experts, ld in ((33, 40), (256, 257), (1000, 1024)):
        rows = dev(g.standard_normal((tokens, ld)).astype(np.float32)).to(dtype)
        ids = dev(g.integers(0, experts, size=(tokens, 1)) + g.integers(0, 3, size=(tokens, top_k))).to(torch.int32)   # some past the experts
        live = dev(g.random(tokens) < 0.9)
        dw, dl, counts = dev(g.standard_normal((tokens, top_k)).astype(np.float32)), torch.full((1,), 0.5, device=DEV), torch.zeros(experts + 1, dtype=torch.int32, device=DEV)
        counts[:-1], counts[-1] = torch.bincount(ids[ids < experts], minlength=experts), tokens
        own, place = torch.full_like(rows, 7.0), rows.clone()
        for out in (own, place):
            qmv.qmv_moe_router_grad(dtype, place, ld, live, ids, dw, counts, dl, tokens, experts, top_k, score, renorm, 1.5, out, ld)
        assert torch.equal(own[:, :experts], place[:, :experts])
        assert torch.equal(place[:, experts:], rows[:, experts:]) and (own[:, experts:] == 7.0).all()
        assert not place[~live, :experts].any()
    assert status_clean()


@pytest.mark.parametrize("score,renorm", MODES)
@pytest.mark.parametrize("spread", [1.0, 8.0, 30.0, 70.0])
def test_scores_of_logits_far_apart(score, renorm, spread):
    """Weights, means, loss and gradient where exponentials have arguments of hundreds."""
    tokens, experts, top_k = 300, 48, 6
    l = logits(int(spread), tokens, experts, spread)
    l[0] = -200 + np.arange(experts) % 3
    l[1] = 200 - np.arange(experts) % 7
    l[2] = np.where(np.arange(experts) % 2, -100, 100)
    ld, l64, live = dev(l), l.astype(np.float64), np.ones(tokens, bool)
    ids, w = torch.empty(tokens, top_k, dtype=torch.int32, device=DEV), torch.empty(tokens, top_k, device=DEV)
    qmv.qmv_moe_router("f32", ld, experts, None, tokens, experts, top_k, score, renorm, 2.5, ids, w)
    want_ids, want = tr.route(l64, live, top_k, score, renorm, 2.5)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    b = share_error(l64, experts)
    assert_within(host(w), want, b * want + 2.0 ** -120, "f32", "weights")
    counts, means, loss = balance(ld, ids, top_k, score)
    wc, wm, wl = tr.balance(l64, live, want_ids, top_k, score)
    assert np.array_equal(counts.cpu().numpy(), wc)
    c = share_error(l64, experts, tokens / 16 + 80)
    assert_within(host(means), wm, c * wm + 2.0 ** -120, "f32", "means")
    assert_within(host(loss)[0], wl, (c + 22 * 2.0 ** -24) * wl, "f32", "loss")
    dw, dl, d = dev(qi.rng(5).standard_normal((tokens, top_k)).astype(np.float32)), torch.full((1,), 0.37, device=DEV), torch.empty_like(ld)
    qmv.qmv_moe_router_grad("f32", ld, experts, None, ids, dw, counts, dl, tokens, experts, top_k, score, renorm, 2.5, d, experts)
    wd, size = tr.router_grad(l64, live, want_ids, host(dw), wc, host(dl)[0], top_k, score, renorm, 2.5)
    assert_within(host(d), wd, (3 * b + (experts / 32 + 24) * 2.0 ** -24) * size + 2.0 ** -120, "f32", "dlogits")
    assert status_clean()
