"""The int4 projection with low-rank adapters, forward and backward, against
its definition in 64 bits within bounds that count the roundings."""
import pytest
import torch

from tests import _adapt as ad

pytestmark = pytest.mark.gpu


def moe():
    import int4_routed_expert_softmax_b200 as m
    return m


def inputs(T, K, N, n, r, dtype, seed=0, ids="mixed"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x = rn(T, K)
    if T > 2:
        x[1] = 0.0          # an all-zero token
        x[2, :32] = 0.0     # an all-zero block
    W = ad.make_w(N, K, g)
    A, B = (rn(n, r, K) / K ** 0.5).to(dtype), (rn(n, N, r) * 0.1).to(dtype)
    scale = rn(n) + 1.0
    if ids == "mixed":      # every adapter, none, and numbers outside the range
        adapter = torch.randint(-2, n + 2, (T,), generator=g, device="cuda", dtype=torch.int32)
    elif ids == "none":
        adapter = torch.full((T,), -1, device="cuda", dtype=torch.int32)
    else:
        adapter = torch.full((T,), n - 1, device="cuda", dtype=torch.int32)
    return x, W, A, B, scale, adapter, rn(T, N) * 1e-3


def dirty(ws):
    return ws.fill_(255)  # NaN wherever a kernel reads what no kernel wrote


def close(got, ref, bound, what):
    err = (got.double() - ref).abs()
    assert bool((err <= bound).all()), (what, float(err.max()), float((err / bound.clamp(min=1e-300)).max()))


def forward(case, T, K, N, n, r, dtype, save=True):
    m = moe()
    x, W, A, B, scale, adapter, _ = case
    p = m.lora(K, N, n, r, dtype)
    ws = dirty(m.alloc_lora_workspace(p, T))
    out = torch.full((T + 1, N), 7.0, device="cuda")
    u = torch.full((T + 1, r), 7.0, device="cuda") if save else None
    m.moe_lora_forward(p, x, W, A, B, scale, adapter, out, ws, u=u)
    assert bool((out[T] == 7.0).all()) and (u is None or bool((u[T] == 7.0).all()))  # rows behind the last token
    return out[:T], None if u is None else u[:T]


SHAPES = [
    # T, K, N, n, r: the kernels of small batches
    (1, 64, 8, 1, 8), (1, 6144, 64, 3, 16), (2, 128, 24, 2, 8), (7, 192, 40, 4, 24), (8, 2048, 136, 40, 16),
    (9, 576, 72, 3, 128), (16, 2048, 256, 16, 16), (17, 1088, 16, 5, 64), (31, 8192, 32, 2, 40), (32, 512, 200, 33, 32),
    (33, 64, 8, 1, 8), (48, 576, 72, 3, 128), (63, 6144, 40, 20, 64), (64, 64, 2048, 1, 8),
    # tokens sorted by adapter
    (65, 64, 8, 1, 8), (66, 6144, 40, 20, 8), (128, 2048, 256, 9, 8), (385, 8192, 1000, 3, 32), (64, 192, 72, 3, 24), (65, 1088, 136, 70, 16), (127, 512, 1000, 4, 128), (200, 2048, 264, 24, 32),
    (300, 8192, 64, 2, 40), (513, 320, 2048, 8, 64), (2100, 128, 1288, 6, 16),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,K,N,n,r", SHAPES)
def test_forward(T, K, N, n, r, dtype):
    case = inputs(T, K, N, n, r, dtype, seed=T)
    out, u = forward(case, T, K, N, n, r, dtype)
    ref, uref, bo, bu = ad.lora_forward(case[1], case[0], *case[2:6], N, K)
    close(u, uref, bu, "u")
    close(out, ref, bo, "out")


@pytest.mark.parametrize("T", [5, 90])
@pytest.mark.parametrize("ids", ["none", "one"])
def test_forward_adapter_patterns(T, ids):
    case = inputs(T, 256, 72, 3, 16, torch.bfloat16, ids=ids)
    out, u = forward(case, T, 256, 72, 3, 16, torch.bfloat16)
    ref, uref, bo, bu = ad.lora_forward(case[1], case[0], *case[2:6], 72, 256)
    close(out, ref, bo, "out")
    close(u, uref, bu, "u")
    if ids == "none":
        assert bool((u == 0).all())


@pytest.mark.parametrize("T", [3, 70])
def test_projection_alone(T):
    """n_adapters = 0: no adapter tensor at all."""
    m = moe()
    case = inputs(T, 256, 72, 1, 8, torch.bfloat16, ids="none")
    p = m.lora(256, 72, 0, 8)
    out, dx = torch.empty(T, 72, device="cuda"), torch.empty(T, 256, device="cuda")
    ws = dirty(m.alloc_lora_workspace(p, T, backward=True))
    m.moe_lora_forward(p, case[0], case[1], None, None, None, None, out, ws)
    ref, _, bo, _ = ad.lora_forward(case[1], case[0], *case[2:6], 72, 256)
    close(out, ref, bo, "out")
    m.moe_lora_backward(p, case[6], case[0], case[1], None, None, None, None, ws, dx=dx)
    (rdx, _, _), (bdx, _, _) = ad.lora_backward(case[1], case[6], case[0], *case[2:6], None, 72, 256)
    close(dx, rdx, bdx, "dx")


def test_forward_does_not_see_its_neighbours():
    """A token's outputs do not depend on the batch around it beyond rounding, and one with a NaN or an
    infinity spoils only its own row."""
    T, K, N, n, r = 80, 256, 72, 3, 16
    case = inputs(T, K, N, n, r, torch.bfloat16)
    out, u = forward(case, T, K, N, n, r, torch.bfloat16)
    x = case[0].clone()
    x[7, 3], x[50, 9] = float("nan"), float("inf")
    adapter = case[5].clone()
    adapter[7] = adapter[50] = 1
    o2, u2 = forward((x, *case[1:5], adapter, case[6]), T, K, N, n, r, torch.bfloat16)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[7] = keep[50] = False
    ref, _, bo, _ = ad.lora_forward(case[1], case[0], *case[2:6], N, K)
    close(o2[keep], ref[keep], bo[keep], "out")
    assert not bool(torch.isfinite(u2[7]).any()) and not bool(torch.isfinite(u2[50]).any())
    assert not bool(torch.isfinite(o2[7]).any())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,K,N,n,r", [
    (1, 64, 8, 1, 8), (3, 128, 24, 2, 8), (16, 2048, 256, 16, 16), (33, 192, 72, 3, 24), (65, 1088, 136, 70, 16),
    (127, 512, 1000, 4, 128), (129, 320, 2048, 8, 64), (300, 8192, 64, 2, 40), (1000, 128, 1288, 6, 72)])
@pytest.mark.parametrize("save", [True, False])
def test_backward(T, K, N, n, r, dtype, save):
    m = moe()
    case = inputs(T, K, N, n, r, dtype, seed=T)
    x, W, A, B, scale, adapter, g = case
    u = forward(case, T, K, N, n, r, dtype)[1].contiguous() if save else None
    p = m.lora(K, N, n, r, dtype)
    ws = dirty(m.alloc_lora_workspace(p, T, backward=True))
    dx = torch.full((T + 1, K), 7.0, device="cuda")
    dA, dB = torch.full((n, r, K), 7.0, device="cuda"), torch.full((n, N, r), 7.0, device="cuda")
    m.moe_lora_backward(p, g, x, W, A, B, scale, adapter, ws, u=u, dx=dx, dA=dA, dB=dB)
    assert int(ws[:4].view(torch.int32)) == 0 and bool((dx[T] == 7.0).all())
    ref, bound = ad.lora_backward(W, g, x, A, B, scale, adapter, u, N, K)
    for got, want, b, name in zip((dx[:T], dA, dB), ref, bound, ("dx", "dA", "dB")):
        close(got, want, b, name)
    # each gradient alone gives the same bits
    for one in ("dx", "dA", "dB"):
        alone = {"dx": torch.empty_like(dx), "dA": torch.empty_like(dA), "dB": torch.empty_like(dB)}[one]
        m.moe_lora_backward(p, g, x, W, A, B, scale, adapter, ws, u=u, **{one: alone})
        full = {"dx": dx[:T], "dA": dA, "dB": dB}[one]
        assert torch.equal(alone[:T] if one == "dx" else alone, full), one


@pytest.mark.parametrize("power", [-60, -20, 20, 60])
def test_backward_scales_with_its_gradient(power):
    """dx of g 2^p is dx 2^p: fp16 operands do not limit the range of g."""
    m = moe()
    T, K, N = 40, 256, 72
    x, W, A, B, scale, adapter, g = inputs(T, K, N, 2, 8, torch.bfloat16)
    p = m.lora(K, N, 2, 8)
    ws = m.alloc_lora_workspace(p, T, backward=True)
    a, b = torch.empty(T, K, device="cuda"), torch.empty(T, K, device="cuda")
    m.moe_lora_backward(p, g, x, W, A, B, scale, adapter, ws, dx=a)
    m.moe_lora_backward(p, g * 2.0 ** power, x, W, A, B, scale, adapter, ws, dx=b)
    assert torch.equal(b, a * 2.0 ** power)


def test_backward_of_scales_far_apart():
    """Rows of W whose scales differ by 2^20 keep their bound."""
    m = moe()
    T, K, N = 20, 128, 64
    x, W, A, B, scale, adapter, g = inputs(T, K, N, 1, 8, torch.float16)
    s = W[N * K // 2:].view(torch.float16).view(N, K // 64)
    s[::2] = s[::2] * 512.0
    s[1::2] = s[1::2] / 512.0
    s[5] = 0.0
    g[:, ::2] *= 1e-4
    p = m.lora(K, N, 1, 8, torch.float16)
    ws = m.alloc_lora_workspace(p, T, backward=True)
    dx = torch.empty(T, K, device="cuda")
    m.moe_lora_backward(p, g, x, W, A, B, scale, adapter, ws, dx=dx)
    ref, bound = ad.lora_backward(W, g, x, A, B, scale, adapter, None, N, K)
    close(dx, ref[0], bound[0], "dx")


def test_backward_without_tokens():
    m = moe()
    p = m.lora(128, 64, 3, 8)
    _, W, A, B, scale, _, _ = inputs(4, 128, 64, 3, 8, torch.bfloat16)
    e = lambda *s: torch.empty(*s, device="cuda")
    dA, dB = torch.full((3, 8, 128), 7.0, device="cuda"), torch.full((3, 64, 8), 7.0, device="cuda")
    ws = dirty(m.alloc_lora_workspace(p, 0, backward=True))
    m.moe_lora_backward(p, e(0, 64), e(0, 128), W, A, B, scale, torch.empty(0, dtype=torch.int32, device="cuda"), ws,
                        dx=e(0, 128), dA=dA, dB=dB)
    assert bool((dA == 0).all()) and bool((dB == 0).all())
    m.moe_lora_forward(p, e(0, 128), W, A, B, scale, torch.empty(0, dtype=torch.int32, device="cuda"), e(0, 64), ws)


def test_backward_without_tokens_reads_no_input():
    """No token: g, x, W and adapter may be null, the gradients are zeros."""
    import ctypes
    m = moe()
    p = m.lora(128, 64, 3, 16, torch.float16)
    _, _, A, B, scale, _, _ = inputs(4, 128, 64, 3, 16, torch.float16)
    ws = dirty(m.alloc_lora_workspace(p, 4, backward=True))
    dA, dB = torch.full((3, 16, 128), 7.0, device="cuda"), torch.full((3, 64, 16), 7.0, device="cuda")
    rc = m.lib().moe_lora_backward(ctypes.byref(p), 0, None, None, None, A.data_ptr(), B.data_ptr(), scale.data_ptr(), None,
                                   None, None, dA.data_ptr(), dB.data_ptr(), ws.data_ptr(), ws.numel(),
                                   torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0 and not dA.any() and not dB.any()


@pytest.mark.parametrize("T", [6, 50])
def test_adapter_gradients_by_differences(T):
    """sum(g out) is linear in A and in B: central differences over steps of a
    power of two that A and B take exactly are the gradients but for rounding."""
    m = moe()
    K, N, n, r = 128, 64, 2, 8
    x, W, A, B, scale, adapter, g = inputs(T, K, N, n, r, torch.float16, seed=3)
    g = g * 1e3
    A, B = (A * 64).round() / 64, (B * 64).round() / 64
    p = m.lora(K, N, n, r, torch.float16)
    ws = m.alloc_lora_workspace(p, T, backward=True)
    dA, dB = torch.empty(n, r, K, device="cuda"), torch.empty(n, N, r, device="cuda")
    m.moe_lora_backward(p, g, x, W, A, B, scale, adapter, ws, dA=dA, dB=dB)

    def value(A_, B_):
        out = torch.empty(T, N, device="cuda")
        m.moe_lora_forward(p, x, W, A_, B_, scale, adapter, out, ws)
        return out

    _, _, bound, _ = ad.lora_forward(W, x, A.abs() + 1, B.abs() + 1, scale, adapter, N, K)
    noise = float((g.double().abs() * bound).sum())  # of either side's sum(g out)
    for at in [(0, 0, 0), (1, 7, 127), (0, 3, 70)]:
        hi, lo = A.clone(), A.clone()
        hi[at] += 1.0
        lo[at] -= 1.0
        diff = float((g.double() * (value(hi, B).double() - value(lo, B).double())).sum() / 2)
        assert abs(diff - float(dA[at])) <= noise + 1e-4 * abs(diff)
    for at in [(0, 0, 0), (1, 63, 7), (1, 20, 2)]:
        hi, lo = B.clone(), B.clone()
        hi[at] += 1.0
        lo[at] -= 1.0
        diff = float((g.double() * (value(A, hi).double() - value(A, lo).double())).sum() / 2)
        assert abs(diff - float(dB[at])) <= noise + 1e-4 * abs(diff)


@pytest.mark.parametrize("T", [4, 150])
def test_same_bits_again_on_another_stream_and_in_a_graph(T):
    m = moe()
    K, N, n, r = 512, 136, 5, 16
    case = inputs(T, K, N, n, r, torch.bfloat16)
    x, W, A, B, scale, adapter, g = case
    p = m.lora(K, N, n, r)
    ws = m.alloc_lora_workspace(p, T, backward=True)

    def outs():
        return [torch.zeros(T, N, device="cuda"), torch.zeros(T, r, device="cuda"), torch.zeros(T, K, device="cuda"),
                torch.zeros(n, r, K, device="cuda"), torch.zeros(n, N, r, device="cuda")]

    def call(o, ws):
        m.moe_lora_forward(p, x, W, A, B, scale, adapter, o[0], ws, u=o[1])
        m.moe_lora_backward(p, g, x, W, A, B, scale, adapter, ws, u=o[1], dx=o[2], dA=o[3], dB=o[4])

    first = outs()
    call(first, ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    again, ws2 = outs(), dirty(m.alloc_lora_workspace(p, T, backward=True))
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        call(again, ws2)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    graph, held = torch.cuda.CUDAGraph(), outs()
    with torch.cuda.graph(graph):
        call(held, ws)
    for _ in range(2):
        for t in held:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, held))
    # new inputs in the same buffers
    x.mul_(0.5)
    adapter.copy_(torch.flip(adapter, [0]))
    graph.replay()
    fresh = outs()
    call(fresh, ws2)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(fresh, held))


def test_two_calls_at_once_on_their_own_workspaces():
    m = moe()
    sets = []
    for i, T in enumerate((20, 260)):
        case = inputs(T, 1024, 264, 4, 16, torch.bfloat16, seed=i)
        p = m.lora(1024, 264, 4, 16)
        sets.append((p, case, m.alloc_lora_workspace(p, T), torch.empty(T, 264, device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for p, c, ws, out, s in sets:
            m.moe_lora_forward(p, *c[:6], out, ws, stream=s)
    torch.cuda.synchronize()
    for p, c, ws, out, s in sets:
        ref, _, bo, _ = ad.lora_forward(c[1], c[0], *c[2:6], 264, 1024)
        close(out, ref, bo, "out")


def test_workspace_of_a_larger_batch_serves_smaller_ones():
    m = moe()
    p = m.lora(256, 72, 3, 16)
    sizes = [m.moe_lora_workspace_bytes(p, T, True) for T in range(0, 400)]
    assert sizes == sorted(sizes)
    ws = m.alloc_lora_workspace(p, 200)
    for T in (200, 33, 32, 9, 1):
        case = inputs(T, 256, 72, 3, 16, torch.bfloat16)
        out = torch.empty(T, 72, device="cuda")
        m.moe_lora_forward(p, *case[:6], out, dirty(ws))
        ref, _, bo, _ = ad.lora_forward(case[1], case[0], *case[2:6], 72, 256)
        close(out, ref, bo, "out")


@pytest.mark.parametrize("T,what", [(1, "fwd"), (16, "fwd"), (40, "fwd"), (200, "fwd"), (1500, "fwd"), (100, "bwd"), (700, "bwd")])
def test_waits_that_run_out(T, what):
    """A short wait limit makes the kernels' waits for data give up: the status word says so, and the device,
    the workspace and later calls stay usable."""
    m = moe()
    K, N, n, r = 1024, 512, 3, 16
    case = inputs(T, K, N, n, r, torch.bfloat16)
    x, W, A, B, scale, adapter, g = case
    p = m.lora(K, N, n, r)
    ws = m.alloc_lora_workspace(p, T, backward=True)

    def call():
        if what == "fwd":
            o = torch.zeros(T, N, device="cuda")
            m.moe_lora_forward(p, x, W, A, B, scale, adapter, o, ws)
        else:
            o = torch.zeros(T, K, device="cuda")
            m.moe_lora_backward(p, g, x, W, A, B, scale, adapter, ws, dx=o)
        torch.cuda.synchronize()
        return o, int(ws[:4].view(torch.int32))

    want, status = call()
    assert status == 0
    old = m.moe_set_wait_limit(1)
    try:
        got, status = call()
    finally:
        m.moe_set_wait_limit(old)
    if T <= 64 and what == "fwd" and status == 0:  # one wait: its copies may have landed before the first look
        assert torch.equal(got, want)
    else:
        assert status == -7
    got, status = call()
    assert status == 0 and torch.equal(got, want)
