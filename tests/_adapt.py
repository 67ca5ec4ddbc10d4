"""Plain 64-bit forms of the adapter projection and of the balance loss, with
rounding bounds (not a test module).

Bounds: a sum of n fp32 terms in any order is off by at most n half-steps of
2^-24 relative to the sum of the terms' magnitudes; a step of a tensor-core
accumulation is counted as a whole step of 2^-23 (it may truncate), once per
MMA.  Factors carried as two tf32 or fp16 numbers are off by 2^-22.  Each bound
below is (number of steps) * 2^-23 * (the same expression over magnitudes)."""
from __future__ import annotations

import torch

STEP = 2.0 ** -23


def make_w(N, K, gen, dev="cuda"):
    """One int4 gs64 matrix as the library takes it (uint8)."""
    packed = torch.randint(0, 256, (N * K // 2,), generator=gen, device=dev, dtype=torch.uint8)
    scales = torch.exp(torch.randn(N * K // 64, generator=gen, device=dev) * 0.3 - 3.9).half()
    return torch.cat([packed, scales.view(torch.uint8)])


def dequant(W, N, K):
    raw = W[: N * K // 2].long().view(N, K // 64, 32)
    w = torch.cat([raw % 16, raw // 16], dim=2) - 8
    return (w.double() * W[N * K // 2:].view(torch.float16).double().view(N, K // 64, 1)).reshape(N, K)


def q8_0(x):
    """The dequantised Q8_0 codes of x in 64 bits (codes by the format's fp32 arithmetic)."""
    b = x.float().view(x.shape[0], -1, 32)
    d = b.abs().amax(dim=2, keepdim=True) / 127.0
    q = torch.where(d > 0, torch.round(b / d), torch.zeros_like(b)).clamp(-127, 127)
    return (q.double() * d.double()).view(x.shape[0], -1)


def own(adapter, n):
    """[T][n] one-hot (a row of zeros without an adapter)."""
    return (adapter[:, None].long() == torch.arange(n, device=adapter.device)).double()


def lora_forward(W, x, A, B, scale, adapter, N, K):
    """(out, u, bound of out, bound of u) in 64 bits."""
    n, r = A.shape[0], A.shape[1]
    What, xq, xd = dequant(W, N, K), q8_0(x), x.double()
    hot = own(adapter, n)
    out = xq @ What.t()
    mag = xq.abs() @ What.abs().t()
    u = torch.zeros(x.shape[0], r, dtype=torch.float64, device=x.device)
    um, lm = torch.zeros_like(u), torch.zeros_like(out)
    for a in range(n):
        h = hot[:, a:a + 1]
        ua, uam = xd @ A[a].double().t(), xd.abs() @ A[a].double().abs().t()
        u += h * ua
        um += h * uam
        out += h * scale[a].double() * (ua @ B[a].double().t())
        lm += h * scale[a].double().abs() * (uam @ B[a].double().abs().t())
    # base: 4 roundings of a group's term and G + 16 additions; u: K / 8 MMAs of
    # each half of the split (or K additions halved over the slices) and the
    # joins; out: u's and r / 8 MMAs of each half
    steps_u = K / 4 + 32
    return out, u, STEP * ((K / 64 + 20) * mag + (steps_u + r / 4 + 8) * lm), STEP * steps_u * um


def lora_backward(W, g, x, A, B, scale, adapter, u, N, K):
    """((dx, dA, dB), their bounds) in 64 bits; u: the given A x, or None."""
    n, r = A.shape[0], A.shape[1]
    What, gd, xd = dequant(W, N, K), g.double(), x.double()
    hot = own(adapter, n)
    T = x.shape[0]
    dx, dxm = gd @ What, gd.abs() @ What.abs()
    dA = torch.zeros(n, r, K, dtype=torch.float64, device=x.device)
    dB = torch.zeros(n, N, r, dtype=torch.float64, device=x.device)
    dAm, dBm, dxl = torch.zeros_like(dA), torch.zeros_like(dB), torch.zeros_like(dx)
    for a in range(n):
        h, s, Aa, Ba = hot[:, a:a + 1], scale[a].double(), A[a].double(), B[a].double()
        v, vm = h * s * (gd @ Ba), h * s.abs() * (gd.abs() @ Ba.abs())
        ua = u.double() if u is not None else xd @ Aa.t()
        uam = ua.abs() if u is not None else xd.abs() @ Aa.abs().t()
        dx += v @ Aa
        dxl += vm @ Aa.abs()
        dA[a], dAm[a] = v.t() @ xd, vm.t() @ xd.abs()
        dB[a], dBm[a] = s * (h * gd).t() @ ua, s.abs() * (h * gd.abs()).t() @ uam
    # v and u: L / 8 MMAs of each half, the joins and the factor; dA, dB: three
    # MMAs per 8 tokens, two split factors; dx: three MMAs per 16 of N
    sv, su = N / 4 + 32, (K / 4 + 32 if u is None else 4)
    return (dx, dA, dB), (STEP * ((3 * N / 16 + 16) * dxm + (sv + r / 4 + 8) * dxl),
                          STEP * (sv + 3 * T / 8 + 24) * dAm, STEP * (su + 3 * T / 8 + 24) * dBm)


def balance(logits, idx, E, k, seg=None, valid=None, dloss=None, w=None, dw=None):
    """(counts, ntok, pmean, loss, dlogits or None) in 64 bits, segment by segment."""
    T = logits.shape[0]
    bounds = [0, T] if seg is None else seg.tolist()
    S = len(bounds) - 1
    l64 = logits.double()
    m = l64.amax(dim=1, keepdim=True) if E else l64
    m = torch.where(m == -float("inf"), torch.zeros_like(m), m)
    e = torch.exp(l64 - m)
    tot = e.sum(dim=1, keepdim=True)
    p = torch.where(tot == 0, torch.zeros_like(e), e / tot)
    counts = torch.zeros(S, E, dtype=torch.int32)
    ntok = torch.zeros(S, dtype=torch.int32)
    pmean, loss = torch.zeros(S, E, dtype=torch.float64), torch.zeros(S, dtype=torch.float64)
    d = torch.zeros(T, E, dtype=torch.float64) if dloss is not None else None
    for s in range(S):
        f = None
        t = [i for i in range(bounds[s], bounds[s + 1]) if valid is None or valid[i]]
        for i in t:
            for j in idx[i].tolist():
                if 0 <= j < E:
                    counts[s, j] += 1
        ntok[s] = len(t)
        if t:
            f = counts[s].double() * E / (k * len(t))
            pmean[s] = p[t].sum(dim=0) / len(t)
            loss[s] = (f * pmean[s]).sum()
            if d is not None:
                d[t] = dloss[s].double() / len(t) * p[t] * (f - p[t] @ f[:, None])
    if dw is not None:
        wd, g = w.double(), dw.double()
        kept = wd * (g - (wd * g).sum(dim=1, keepdim=True))
        for i in range(T):
            for s, j in enumerate(idx[i].tolist()):
                if 0 <= j < E:
                    d[i, j] += kept[i, s]
    return counts, ntok, pmean, loss, d
