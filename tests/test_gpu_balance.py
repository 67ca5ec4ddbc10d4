"""The router's balance loss, counts and gradients against the definition in
64 bits."""
import pytest
import torch

from tests import _adapt as ad

pytestmark = pytest.mark.gpu


def moe():
    import int4_routed_expert_softmax_b200 as m
    return m


def inputs(T, E, k, S, mask, seed=0):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(T, E, generator=g) * 2 + torch.randn(E, generator=g)
    idx = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k].int().contiguous()
    seg = valid = None
    if S > 1:
        cuts = torch.sort(torch.randint(0, T + 1, (S - 1,), generator=g)).values
        seg = torch.cat([torch.zeros(1, dtype=torch.long), cuts, torch.tensor([T])]).int()
    if mask:
        valid = (torch.rand(T, generator=g) > 0.2).to(torch.uint8)
        idx[torch.rand(T, k, generator=g) < 0.1] = -1
        idx[torch.rand(T, k, generator=g) < 0.02] = E + 3
        if seg is not None and S > 2:  # tokens before the first and behind the last sequence
            seg[0], seg[-1] = min(2, int(seg[1])), max(T - 3, int(seg[-2]))
    w = torch.softmax(torch.randn(T, k, generator=g), dim=1)
    return logits, idx, seg, valid, torch.randn(S, generator=g), w, torch.randn(T, k, generator=g)


def cu(*ts):
    return [None if t is None else t.cuda() for t in ts]


def call(E, k, logits, idx, seg, valid, dloss, w, dw, dims=None):
    m = moe()
    T, S = logits.shape[0], 1 if seg is None else seg.numel() - 1
    d = m.dims(256, 128, E, k)
    logits, idx, seg, valid, dloss, w, dw = cu(logits, idx, seg, valid, dloss, w, dw)
    ws = m.alloc_balance_workspace(d, T, S).fill_(255)
    counts, ntok = torch.full((S, E), -9, dtype=torch.int32, device="cuda"), torch.full((S,), -9, dtype=torch.int32, device="cuda")
    pmean, loss = torch.full((S, E), 7.0, device="cuda"), torch.full((S,), 7.0, device="cuda")
    m.moe_balance_forward(d, logits, idx, counts, ntok, pmean, loss, ws, seg=seg, valid=valid)
    dl = torch.full((T + 1, E), 7.0, device="cuda")
    m.moe_balance_backward(d, logits, idx, counts, ntok, dloss, dl, seg=seg, valid=valid, w=w, dw=dw)
    assert bool((dl[T] == 7.0).all())
    return [t.cpu() for t in (counts, ntok, pmean, loss, dl[:T])]


# Probabilities: expf within 2 ulp and its argument's rounding (|v - m| 2^-24,
# here below 40), E additions, a division and a product: 2^-24 (E + 50) of p.
# Means: as many additions again at most over a CTA's tokens and warps (bounded
# by T), then 64-bit sums.
def tolerances(E, T):
    return 2.0 ** -24 * (E + 50 + min(T, 1000) + 16), 2.0 ** -24 * (3 * E + 120)


def check(E, k, case):
    logits, idx, seg, valid, dloss, w, dw = case
    got = call(E, k, *case)
    ref = ad.balance(logits, idx, E, k, seg, valid, dloss, w, dw)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    tf, tb = tolerances(E, logits.shape[0])
    assert bool(((got[2].double() - ref[2]).abs() <= tf * ref[2] + 1e-38).all())
    assert bool(((got[3].double() - ref[3]).abs() <= (tf + E * 2.0 ** -24) * ref[3].abs() + 1e-38).all())
    # the gradient's magnitude: every difference taken as a sum
    zero = torch.zeros_like(dloss)
    base = ad.balance(logits, idx, E, k, seg, valid, dloss, None, None)[4]
    p = torch.softmax(logits.double(), dim=1)
    S = dloss.numel()
    mag = torch.zeros_like(base)
    bounds = [0, logits.shape[0]] if seg is None else seg.tolist()
    for s in range(S):
        if ref[1][s] > 0:
            n = int(ref[1][s])
            f = ref[0][s].double() * E / (k * n)
            t = slice(bounds[s], bounds[s + 1])
            mag[t] = dloss[s].abs().double() / n * p[t] * (f + (p[t] @ f)[:, None])
    if dw is not None:
        kept = w.double() * (dw.double().abs() + (w.double() * dw.double().abs()).sum(1, keepdim=True))
        for i in range(logits.shape[0]):
            for s, j in enumerate(idx[i].tolist()):
                if 0 <= j < E:
                    mag[i, j] += kept[i, s]
    err = (got[4].double() - ref[4]).abs()
    assert bool((err <= tb * mag + 1e-37).all()), float((err / (mag + 1e-30)).max())


@pytest.mark.parametrize("E,k", [(1, 1), (8, 2), (16, 2), (33, 3), (90, 6), (128, 8), (160, 8), (256, 8), (257, 4),
                                 (300, 32), (384, 8), (514, 5), (1000, 7), (1024, 32)])
@pytest.mark.parametrize("T,S,mask", [(1, 1, False), (5, 2, True), (64, 1, False), (65, 4, True), (300, 7, True)])
def test_shapes(E, k, T, S, mask):
    check(E, k, inputs(T, E, k, S, mask, seed=E + T))


@pytest.mark.parametrize("T,S", [(700, 300), (2000, 1), (3000, 40), (10007, 3)])
def test_many_segments_and_long_batches(T, S):
    check(16, 2, inputs(T, 16, 2, S, True, seed=S))


@pytest.mark.parametrize("T,S", [(0, 3), (1, 2), (1, 70), (16, 16), (40, 500), (64, 64), (300, 3000)])
def test_segments_of_few_tokens_or_none(T, S):
    check(33, 3, inputs(T, 33, 3, S, T > 3, seed=T + S))


def test_without_weights_gradient():
    c = list(inputs(100, 32, 4, 3, True))
    c[5] = c[6] = None
    check(32, 4, c)


@pytest.mark.parametrize("T", [0, 40, 200])
def test_nothing_counted(T):
    """No token at all, or none that counts: zeros, not NaN."""
    E, k = 24, 3
    logits, idx, _, _, dloss, _, _ = inputs(T, E, k, 1, False)
    valid = torch.zeros(T, dtype=torch.uint8)
    got = call(E, k, logits, idx, None, valid if T else None, dloss, None, None)
    assert all(bool((t == 0).all()) for t in got)


@pytest.mark.parametrize("T", [10, 200])
def test_masked_experts(T):
    """Logits of -inf and of the type's lowest value have probability 0 and gradient 0; a row of -inf
    alone counts as a token without probabilities."""
    E, k = 40, 4
    logits, idx, _, _, dloss, _, _ = inputs(T, E, k, 1, False)
    logits[:, 5] = -float("inf")
    logits[:, 6] = torch.finfo(torch.float32).min
    logits[3] = -float("inf")
    idx[idx == 5] = 0
    idx[idx == 6] = 1
    got = call(E, k, logits, idx, None, None, dloss, None, None)
    ref = ad.balance(logits, idx, E, k, None, None, dloss)
    assert torch.equal(got[0], ref[0])
    assert float(got[2][0, 5]) == 0.0 and float(got[2][0, 6]) == 0.0
    tf, tb = tolerances(E, T)
    assert bool(((got[2].double() - ref[2]).abs() <= tf * ref[2] + 1e-38).all())
    assert bool((got[4][3] == 0).all()) and bool((got[4][:, 5:7] == 0).all())
    assert bool(torch.isfinite(got[4]).all())


def test_nan_stays_in_its_row():
    E, k, T = 256, 8, 100
    logits, idx, _, _, dloss, w, dw = inputs(T, E, k, 1, False)
    clean = call(E, k, logits, idx, None, None, dloss, w, dw)
    bad = logits.clone()
    bad[9, 17] = float("nan")
    got = call(E, k, bad, idx, None, None, dloss, w, dw)
    assert torch.equal(got[0], clean[0]) and bool(torch.isnan(got[3]).all())
    keep = torch.arange(T) != 9
    assert torch.equal(got[4][keep], clean[4][keep]) and bool(torch.isnan(got[4][9]).all())


def test_an_expert_listed_twice():
    """Its terms add up, in slot order: the same bits every time."""
    E, k, T = 64, 6, 50
    c = list(inputs(T, E, k, 1, False))
    c[1][:, 1] = c[1][:, 0]
    c[1][::2, 4] = c[1][::2, 0]
    check(E, k, c)
    assert torch.equal(call(E, k, *c)[4], call(E, k, *c)[4])


def test_gradient_by_differences():
    """d loss / d logits by central differences in 64 bits of the definition, counts held."""
    E, k, T = 12, 2, 30
    logits, idx, seg, valid, dloss, _, _ = inputs(T, E, k, 3, True)
    got = call(E, k, logits, idx, seg, valid, dloss, None, None)[4]

    def total(l):
        c, n, pm, loss, _ = ad.balance(l, idx, E, k, seg, valid)
        return float((dloss.double() * loss).sum())

    h = 1e-4
    l64 = logits.double()
    scale = float(got.abs().max())
    for t, e in [(0, 0), (4, 3), (17, 11), (29, 5)]:
        up, dn = l64.clone(), l64.clone()
        up[t, e] += h
        dn[t, e] -= h
        # third derivatives are of the gradient's size: error h^2
        assert abs((total(up) - total(dn)) / (2 * h) - float(got[t, e])) <= 1e-6 * scale


def test_in_place_misaligned_and_in_a_graph():
    m = moe()
    E, k, T, S = 256, 8, 300, 4
    logits, idx, seg, valid, dloss, w, dw = inputs(T, E, k, S, True)
    want = call(E, k, logits, idx, seg, valid, dloss, w, dw)
    d = m.dims(256, 128, E, k)
    lg, ix, sg, vl, dl, wc, dwc = cu(logits, idx, seg, valid, dloss, w, dw)
    # logits that start 4 bytes off a 16-byte boundary: the scalar loads
    off = torch.empty(T * E + 1, device="cuda")[1:].view(T, E)
    off.copy_(lg)
    ws = m.alloc_balance_workspace(d, T, S)
    counts, ntok = torch.empty(S, E, dtype=torch.int32, device="cuda"), torch.empty(S, dtype=torch.int32, device="cuda")
    pmean, loss = torch.empty(S, E, device="cuda"), torch.empty(S, device="cuda")

    def run(l, out):
        m.moe_balance_forward(d, l, ix, counts, ntok, pmean, loss, ws, seg=sg, valid=vl)
        m.moe_balance_backward(d, l, ix, counts, ntok, dl, out, seg=sg, valid=vl, w=wc, dw=dwc)

    run(off, off)
    assert torch.equal(counts.cpu(), want[0]) and torch.allclose(loss.cpu(), want[3], rtol=1e-5, atol=0)
    assert float((off.cpu() - want[4]).abs().max()) <= 1e-5 * float(want[4].abs().max())
    out = torch.zeros(T, E, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(lg, out)
    for _ in range(2):
        out.zero_()
        loss.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss.cpu(), want[3]) and torch.equal(out.cpu(), want[4])


def test_workspace_of_a_larger_batch_serves_smaller_ones():
    m = moe()
    d = m.dims(256, 128, 16, 2)
    sizes = [m.moe_balance_workspace_bytes(d, T, 3) for T in range(0, 20000, 7)]
    assert sizes == sorted(sizes)
