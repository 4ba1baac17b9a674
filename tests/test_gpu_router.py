"""The router, its balance loss and their gradient against the 64-bit definitions.

Tolerances. ids and counts are exact (logits are compared as they are). A weight is a quotient of exponentials: expf is
within 2 units (2^-22 relative) of its rounded argument, whose rounding adds |l - max| * 2^-24; a sum of E terms, E / 32 in
a lane and five levels, (E / 32 + 5) * 2^-24; sigmoid adds one exponential, an addition and a division; scale, division and
product 3 * 2^-24: with logits that span R, (2 (R + 8) + E / 32 + 12) * 2^-24 of the value. A mean of T shares adds the
additions of its longest chain, at most T / 16 + 16 + 64 of them. A gradient's terms are products of such numbers: the same
times the sum of the magnitudes of its terms, which cancel, and a few roundings more. Numbers below 2^-126 may be lost
whole: 2^-120 is added. An output of 16 bits is the fp32 result rounded to nearest (assert_within)."""
import numpy as np
import pytest
import torch

qmv = pytest.importorskip("bit_quantized_moe_gb300")
import qmv_inputs as qi  # noqa: E402
import train_reference as tr  # noqa: E402
from qmv_testutil import DEV, assert_within, status_clean  # noqa: E402

pytestmark = pytest.mark.gpu

TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
MODES = [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)]


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t.to(TORCH[dtype]) if dtype else t


def host(t):
    return t.double().cpu().numpy()


def rel(l, experts, more=0):
    fine = l[np.isfinite(l)]
    span = float(fine.max() - min(fine.min(), 0)) if fine.size else 0.0
    return (2 * (span + 8) + experts / 32 + 12 + more) * 2.0 ** -24


class Router:
    """One set of logits on the device (rows `extra` apart) and what the calls give for it."""

    def __init__(self, l, dtype, top_k, score, renorm, scale=1.0, live=None, extra=0):
        self.tokens, self.experts = l.shape
        t = torch.full((self.tokens, self.experts + extra), 9.0, dtype=TORCH[dtype], device=DEV)
        t[:, :self.experts] = dev(l, dtype)
        self.t, self.ld, self.l = t, self.experts + extra, host(t[:, :self.experts])
        self.dtype, self.top_k, self.mode, self.scale = dtype, top_k, (score, renorm), scale
        self.live = np.ones(self.tokens, bool) if live is None else live
        self.live_dev = None if live is None else dev(live)

    def route(self):
        ids = torch.full((self.tokens, self.top_k), 77, dtype=torch.int32, device=DEV)
        w = torch.full((self.tokens, self.top_k), 7.0, device=DEV)
        qmv.qmv_moe_router(self.dtype, self.t, self.ld, self.live_dev, self.tokens, self.experts, self.top_k, *self.mode, self.scale,
                           ids, w)
        return ids, w

    def balance(self, ids):
        counts = torch.full((self.experts + 2,), 77, dtype=torch.int32, device=DEV)
        means, loss = torch.full((self.experts + 1,), 7.0, device=DEV), torch.full((2,), 7.0, device=DEV)
        ws = torch.full((qmv.qmv_moe_balance_workspace_bytes(self.tokens, self.experts),), 0xA5, dtype=torch.uint8, device=DEV)
        qmv.qmv_moe_balance(self.dtype, self.t, self.ld, self.live_dev, ids, self.tokens, self.experts, self.top_k, self.mode[0],
                            counts, means, loss, ws)
        assert counts[-1] == 77 and means[-1] == 7 and loss[-1] == 7
        return counts[:-1], means[:-1], loss[:1]

    def grad(self, ids, dweights, counts, dloss, extra=0):
        d = torch.full((self.tokens, self.experts + extra), 7.0, dtype=TORCH[self.dtype], device=DEV)
        qmv.qmv_moe_router_grad(self.dtype, self.t, self.ld, self.live_dev, ids, dweights, counts, dloss, self.tokens, self.experts,
                                self.top_k, *self.mode, self.scale, d, self.experts + extra)
        assert (d[:, self.experts:] == 7.0).all()
        return host(d[:, :self.experts])

    def check_route(self):
        ids, w = self.route()
        want_ids, want = tr.route(self.l, self.live, self.top_k, *self.mode, self.scale)
        assert np.array_equal(ids.cpu().numpy(), want_ids)
        assert np.array_equal(np.isnan(host(w)), np.isnan(want))
        fine = ~np.isnan(want)
        assert_within(host(w)[fine], want[fine], rel(self.l, self.experts) * np.abs(want[fine]) + 2.0 ** -120, "f32", "weights")
        return ids, want_ids


def logits(seed, tokens, experts, spread=2.0):
    g = qi.rng(seed)
    return g.standard_normal((tokens, experts)) * spread + g.standard_normal(experts)


@pytest.mark.parametrize("score,renorm", MODES)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tokens,experts,top_k,extra", [(1, 1, 1, 0), (1, 32, 4, 0), (7, 5, 2, 3), (33, 33, 8, 0), (100, 64, 6, 1),
                                                        (9, 128, 8, 0), (17, 256, 8, 8), (65, 300, 3, 0), (5, 1024, 8, 0)])
def test_router_balance_and_gradient(score, renorm, dtype, tokens, experts, top_k, extra):
    l = logits(tokens + experts, tokens, experts)
    live = qi.rng(tokens).random(tokens) < 0.8 if tokens > 5 else None
    r = Router(l, dtype, top_k, score, renorm, 2.5, live, extra)
    ids, want_ids = r.check_route()
    counts, means, loss = r.balance(ids)
    wc, wm, wl = tr.balance(r.l, r.live, want_ids, top_k, score)
    bound = rel(r.l, experts, tokens / 16 + 80)
    assert np.array_equal(counts.cpu().numpy(), wc)
    assert_within(host(means), wm, bound * wm + 2.0 ** -120, "f32", "means")
    assert_within(host(loss)[0], wl, (bound + experts * 2.0 ** -24) * wl, "f32", "loss")
    dweights, dloss = dev(qi.rng(9).standard_normal((tokens, top_k)), "f32"), dev([0.37], "f32")
    for dw, c, extra in ((dweights, counts, 0), (dweights, None, 2), (None, counts, 5)):
        got = r.grad(ids, dw, c, None if c is None else dloss, extra)
        want, size = tr.router_grad(r.l, r.live, want_ids, None if dw is None else host(dw), None if c is None else wc,
                                    host(dloss)[0], top_k, score, renorm, 2.5)
        assert_within(got, want, 2 * rel(r.l, experts, 20) * size + 2.0 ** -120, dtype, "dlogits")
    assert status_clean()


@pytest.mark.parametrize("tokens,experts", [(2000, 32), (5000, 256)])
def test_balance_over_many_ctas(tokens, experts):
    """More tokens than one CTA takes; the same bits every time."""
    r = Router(logits(1, tokens, experts), "f32", 4, "softmax", True)
    ids, want_ids = r.check_route()
    first = r.balance(ids)
    wc, wm, wl = tr.balance(r.l, r.live, want_ids, 4, "softmax")
    bound = rel(r.l, experts, tokens / 16 + 80)
    assert np.array_equal(first[0].cpu().numpy(), wc)
    assert_within(host(first[1]), wm, bound * wm, "f32", "means")
    assert_within(host(first[2])[0], wl, (bound + experts * 2.0 ** -24) * wl, "f32", "loss")
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, r.balance(ids)))


@pytest.mark.parametrize("score,renorm", MODES)
def test_ties_go_to_the_lowest_expert(score, renorm):
    """Equal logits, zeros of both signs among them, in every order."""
    g = qi.rng(4)
    l = g.integers(-2, 3, size=(64, 70)).astype(np.float64)
    l[l == 0] = np.where(g.random((l == 0).sum()) < 0.5, -0.0, 0.0)
    l[3] = 0
    l[4] = -0.0
    Router(l, "f32", 8, score, renorm).check_route()


@pytest.mark.parametrize("score,renorm", MODES)
@pytest.mark.parametrize("experts", [4, 40])
def test_rows_of_special_logits(score, renorm, experts):
    """Missing experts, rows without any, infinities, NaN, the types' ends, and logits so low that their scores are 0."""
    l = logits(6, 16, experts)
    l[0] = -np.inf
    l[1, 1:] = -np.inf
    l[2, :2] = -np.inf
    l[3, 2] = np.inf
    l[4, 3] = np.nan
    l[5] = np.nan
    l[6] = -3e38
    l[7] = 3e38
    l[8] = -200 + np.arange(experts) % 3
    l[9] = 200 - np.arange(experts) % 3
    l[10, 0] = -np.finfo(np.float32).max
    l[11] = -np.inf
    l[11, 3] = np.nan
    live = np.ones(16, bool)
    live[12] = False
    l[12, 0] = np.nan
    top_k = 3
    r = Router(l, "f32", top_k, score, renorm, 1.0, live)
    ids, w = r.route()
    want_ids, want = tr.route(r.l, r.live, top_k, score, renorm, 1.0)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    got = host(w)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    fine = ~np.isnan(want)
    # differences of up to 202 in logits that count: 2 (202 + 8) + 14 roundings
    assert (np.abs(got - want)[fine] <= 440 * 2.0 ** -24 * np.abs(want[fine]) + 2.0 ** -120).all()
    # rows with a NaN do not reach the other rows' gradients
    dw = qi.rng(2).standard_normal((16, top_k))
    finite = ~(np.isnan(r.l).any(1) | ((r.l == np.inf).any(1)))
    counts, _, _ = tr.balance(r.l[finite], r.live[finite], want_ids[finite], top_k, score)
    for part in (None, counts):
        d = r.grad(ids, dev(dw, "f32"), None if part is None else dev(part), None if part is None else dev([0.5], "f32"))
        wd, size = tr.router_grad(r.l[finite], r.live[finite], want_ids[finite], host(dev(dw, "f32"))[finite], part, 0.5, top_k, score,
                                  renorm, 1.0)
        assert (np.abs(d[finite] - wd) <= 900 * 2.0 ** -24 * size + 2.0 ** -120).all()
        assert not d[12].any() and not d[0].any()
        assert np.isnan(d[~finite & live & ~((score == "sigmoid") & ~np.isnan(r.l).any(1))]).all()
    # the loss of a batch with a NaN is NaN; without those rows it is the definition's
    assert np.isnan(host(r.balance(ids)[2])[0])
    r2 = Router(l[finite], "f32", top_k, score, renorm, 1.0, live[finite])
    c2, m2, l2 = r2.balance(r2.route()[0])
    wc, wm, wl = tr.balance(r2.l, r2.live, want_ids[finite], top_k, score)
    assert np.array_equal(c2.cpu().numpy(), wc)
    assert (np.abs(host(m2) - wm) <= 500 * 2.0 ** -24 * wm + 2.0 ** -120).all()
    assert abs(host(l2)[0] - wl) <= 560 * 2.0 ** -24 * wl


def test_slots_outside_the_experts_and_named_twice():
    """ids of the caller's own: out of range on both sides, one expert in two slots."""
    r = Router(logits(8, 6, 12), "f32", 4, "softmax", True)
    ids = np.array([[0, 0, 5, 11], [-1, 12, 3, 3], [-5, 1 << 30, -2147483648, 99], [7, 7, 7, 7], [1, 2, 3, 4], [11, -1, 0, -1]], np.int32)
    dw = qi.rng(1).standard_normal((6, 4)).astype(np.float32)
    for score, renorm in MODES:
        r.mode = (score, renorm)
        counts, means, loss = r.balance(dev(ids))
        wc, wm, wl = tr.balance(r.l, r.live, ids, 4, score)
        assert np.array_equal(counts.cpu().numpy(), wc)
        assert abs(host(loss)[0] - wl) <= 2 * rel(r.l, 12, 80) * wl
        d = r.grad(dev(ids), dev(dw), counts, dev([2.0], "f32"))
        want, size = tr.router_grad(r.l, r.live, ids, dw.astype(np.float64), wc, 2.0, 4, score, renorm, 1.0)
        assert_within(d, want, 2 * rel(r.l, 12, 20) * size + 2.0 ** -120, "f32", "dlogits")


@pytest.mark.parametrize("tokens", [0, 1, 40])
def test_balance_without_a_live_token(tokens):
    """No tokens, or padding alone: zeros, and a gradient of zeros."""
    r = Router(logits(1, max(tokens, 1), 20), "bf16", 2, "sigmoid", True, 1.0, np.zeros(max(tokens, 1), bool))
    r.tokens = tokens
    ids = torch.full((max(tokens, 1), 2), 3, dtype=torch.int32, device=DEV)
    counts, means, loss = r.balance(ids)
    assert not counts.any() and not means.any() and not loss.any()
    if tokens:
        assert not r.grad(ids, torch.ones(tokens, 2, device=DEV), counts, torch.ones(1, device=DEV)).any()


def test_gradient_matches_autograd():
    """Of what the weights and the loss are, in float64 torch."""
    r = Router(logits(3, 50, 24), "f32", 3, "sigmoid", True, 2.5)
    ids, w = r.route()
    counts, means, loss = r.balance(ids)
    l = r.t.double().requires_grad_()
    s = torch.sigmoid(l)
    at = ids.long()
    chosen = s.gather(1, at)
    weights = 2.5 * chosen / chosen.sum(1, keepdim=True)
    f = counts[:-1].double() / (3 * counts[-1])
    total = 24 * (f * (s / s.sum(1, keepdim=True)).mean(0)).sum()
    dw = dev(qi.rng(5).standard_normal((50, 3)), "f32")
    (want,) = torch.autograd.grad((weights * dw.double()).sum() + 0.25 * total, l)
    got = r.grad(ids, dw, counts, dev([0.25], "f32"))
    assert np.abs(got - want.cpu().numpy()).max() <= 4 * rel(r.l, 24, 20) * float(want.abs().max())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("score,renorm", MODES)
def test_gradient_in_the_logits_place(score, renorm, dtype):
    """dlogits may be the logits themselves: the bits of a call with a place of its own."""
    for tokens, experts, top_k in ((3000, 40, 4), (9, 300, 8), (1, 1, 1)):
        r = Router(logits(tokens, tokens, experts), dtype, top_k, score, renorm, 1.5)
        ids, w = r.route()
        counts, means, loss = r.balance(ids)
        dw, dl = dev(qi.rng(3).standard_normal((tokens, top_k)), "f32"), dev([0.5], "f32")
        t = r.t.clone()
        d = torch.empty_like(t)
        for out in (d, t):
            qmv.qmv_moe_router_grad(dtype, t, experts, None, ids, dw, counts, dl, tokens, experts, top_k, score, renorm, 1.5, out, experts)
        assert torch.equal(d, t)


def test_router_in_a_graph_and_on_two_streams():
    """Captured calls replay on new logits; two graphs with a workspace each run at once."""
    tokens, experts, top_k = 700, 64, 6
    runs = []
    for i in range(2):
        s = torch.cuda.Stream()
        t = torch.zeros(tokens, experts, device=DEV)
        ids, w = torch.zeros(tokens, top_k, dtype=torch.int32, device=DEV), torch.zeros(tokens, top_k, device=DEV)
        counts, means, loss = torch.zeros(experts + 1, dtype=torch.int32, device=DEV), torch.zeros(experts, device=DEV), torch.zeros(1, device=DEV)
        ws = torch.zeros(qmv.qmv_moe_balance_workspace_bytes(tokens, experts), dtype=torch.uint8, device=DEV)
        d, dw, dl = torch.zeros_like(t), torch.ones(tokens, top_k, device=DEV), torch.ones(1, device=DEV)

        def go(t=t, ids=ids, w=w, counts=counts, means=means, loss=loss, ws=ws, d=d, dw=dw, dl=dl):
            qmv.qmv_moe_router("f32", t, experts, None, tokens, experts, top_k, "softmax", False, 1.0, ids, w)
            qmv.qmv_moe_balance("f32", t, experts, None, ids, tokens, experts, top_k, "softmax", counts, means, loss, ws)
            qmv.qmv_moe_router_grad("f32", t, experts, None, ids, dw, counts, dl, tokens, experts, top_k, "softmax", False, 1.0, d, experts)

        with torch.cuda.stream(s):
            go()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            go()
        runs.append((s, t, graph, go, (ids, w, counts, means, loss, d)))
    for step in range(3):
        for i, (s, t, graph, go, outs) in enumerate(runs):
            t.copy_(dev(logits(10 * step + i, tokens, experts), "f32"))
        torch.cuda.synchronize()
        for s, t, graph, go, outs in runs:
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for s, t, graph, go, outs in runs:
            got = [o.clone() for o in outs]
            go()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, outs))
            assert np.array_equal(got[0].cpu().numpy(), tr.route(host(t), np.ones(tokens, bool), top_k, "softmax", False, 1.0)[0])
