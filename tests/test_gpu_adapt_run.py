"""The adapter and balance calls together with the layer, as a fine-tuning step
uses them: the router's logits and selection, the routed experts, the shared
expert with an adapter beside each of its three matrices, the balance loss, and
the gradients back to the adapters, the hidden state and the logits.  Each step is
checked against its definition in 64 bits on the path's own inputs (a Q8_0 code
of h may flip by the rounding of what produced it, which would compare two
different steps otherwise)."""
import ctypes

import pytest
import torch

import moe_inputs as mi
from tests import _adapt as ad
from tests._common import within_tolerance

pytestmark = pytest.mark.gpu


def close(got, ref, bound):
    assert bool(((got.double() - ref).abs() <= bound).all())


@pytest.mark.parametrize("T", [5, 80])
def test_step(T):
    import int4_routed_expert_softmax_b200 as moe
    H, I, E, k, n, r = 1024, 1024, 16, 2, 3, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    d = moe.dims(H, I, E, k)
    blobs = mi.make_blobs(H, I, E + 1, 7, torch.device("cuda"))
    x, Wr = rn(T, H), rn(E, H) * 0.05
    mats = {"gate": 0, "up": 1, "down": 2}
    size = I * H // 2 + I * H // 32
    W = {m: blobs[E][i * size:(i + 1) * size] for m, i in mats.items()}
    KN = {"gate": (H, I), "up": (H, I), "down": (I, H)}
    A = {m: (rn(n, r, KN[m][0]) / KN[m][0] ** 0.5).to(torch.bfloat16) for m in mats}
    B = {m: (rn(n, KN[m][1], r) * 0.05).to(torch.bfloat16) for m in mats}
    scale, adapter = rn(n) + 1.5, torch.randint(-1, n, (T,), generator=g, device="cuda", dtype=torch.int32)
    plan = {m: moe.lora(*KN[m], n, r) for m in mats}
    ws = {m: moe.alloc_lora_workspace(plan[m], T, backward=True) for m in mats}

    # routing, and the routed experts without the shared one
    idx, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    logits, counts = torch.empty(T, E, device="cuda"), torch.zeros(E, dtype=torch.int32, device="cuda")
    moe.moe_router_topk(d, x, Wr, idx, w, logits, counts)
    table = moe.expert_table(blobs)
    routed, lws = torch.empty(T, H, device="cuda"), moe.alloc_workspace(d, T, path=moe.MOE_PATH_DECODE)
    rc = moe.lib().moe_layer_forward_ep(ctypes.byref(d), T, x.data_ptr(), Wr.data_ptr(), table.data_ptr(),
                                        routed.data_ptr(), lws.data_ptr(), lws.numel(), None, 0, E, 0,
                                        torch.cuda.current_stream().cuda_stream)
    assert rc == 0

    def project(m, inp, adapters=True):
        out, u = torch.empty(T, KN[m][1], device="cuda"), torch.empty(T, r, device="cuda")
        ids = adapter if adapters else torch.full_like(adapter, -1)
        moe.moe_lora_forward(plan[m], inp, W[m], A[m], B[m], scale, ids, out, ws[m], u=u)
        ref, uref, bo, bu = ad.lora_forward(W[m], inp, A[m], B[m], scale, ids, KN[m][1], KN[m][0])
        close(out, ref, bo)
        close(u, uref, bu)
        return out, u

    # without adapters the pieces make up the layer
    gate, up = project("gate", x, False)[0], project("up", x, False)[0]
    plain = routed + project("down", torch.nn.functional.silu(gate) * up, False)[0]
    layer = torch.empty(T, H, device="cuda")
    moe.moe_layer_forward(d, x, Wr, table, layer, moe.alloc_workspace(d, T))
    ok, rel, mx = within_tolerance(plain.cpu().numpy(), layer.cpu().numpy())
    assert ok, (rel, mx)

    # with them, forward and back
    gate, ug = project("gate", x)
    up, uu = project("up", x)
    sig = torch.sigmoid(gate)
    h = gate * sig * up
    down, ud = project("down", h)
    assert not torch.equal(down, plain - routed)

    def back(m, grad, inp, u):
        dx, dA, dB = torch.empty_like(inp), torch.empty(n, r, KN[m][0], device="cuda"), torch.empty(n, KN[m][1], r, device="cuda")
        moe.moe_lora_backward(plan[m], grad, inp, W[m], A[m], B[m], scale, adapter, ws[m], u=u, dx=dx, dA=dA, dB=dB)
        ref, bound = ad.lora_backward(W[m], grad, inp, A[m], B[m], scale, adapter, u, KN[m][1], KN[m][0])
        for got, want, b in zip((dx, dA, dB), ref, bound):
            close(got, want, b)
        return dx

    dout = rn(T, H) * 1e-2
    dh = back("down", dout, h, ud)
    dg = dh * up * (sig * (1 + gate * (1 - sig)))
    dx = back("gate", dg.contiguous(), x, ug) + back("up", (dh * gate * sig).contiguous(), x, uu)
    assert bool(torch.isfinite(dx).all())

    # the balance of the same routing, and the logits' gradient
    cnt, ntok = torch.empty(1, E, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    pm, loss = torch.empty(1, E, device="cuda"), torch.empty(1, device="cuda")
    moe.moe_balance_forward(d, logits, idx, cnt, ntok, pm, loss, moe.alloc_balance_workspace(d, T))
    assert torch.equal(cnt[0], counts) and int(ntok) == T  # the route counts that learned pins live from
    dw, dloss, dl = rn(T, k) * 1e-2, torch.tensor([0.01], device="cuda"), torch.empty(T, E, device="cuda")
    moe.moe_balance_backward(d, logits, idx, cnt, ntok, dloss, dl, w=w, dw=dw)
    ref = ad.balance(logits.cpu(), idx.cpu(), E, k, None, None, dloss.cpu(), w.cpu(), dw.cpu())
    # E + 90 roundings of 2^-24 of a probability, differences of terms of the size of their sum
    assert abs(float(loss) - float(ref[3])) <= 2.0 ** -24 * (2 * E + 90 + T) * float(ref[3])
    size = float(ref[4].abs().max())
    assert float((dl.cpu().double() - ref[4]).abs().max()) <= 2.0 ** -24 * (3 * E + 120) * 4 * size


@pytest.mark.parametrize("native", [True, False])
def test_refusals_in_device_memory(native, monkeypatch):
    """The binding's checks in C++ and in Python refuse the same tensors in the same words."""
    import int4_routed_expert_softmax_b200 as m
    from int4_routed_expert_softmax_b200 import _lib
    if not native:
        monkeypatch.setattr(_lib, "_rows_on", _lib._on)
        monkeypatch.setattr(_lib, "_addresses", _lib._adrs)
    else:
        assert _lib._addresses is not _lib._adrs  # built
    T, K, N, n, r = 4, 128, 64, 2, 8
    p = m.lora(K, N, n, r)
    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda")
    good = dict(x=z(T, K), W=z(N * K // 2 + N * K // 32, dtype=torch.uint8), A=z(n, r, K, dtype=torch.bfloat16),
                B=z(n, N, r, dtype=torch.bfloat16), scale=z(n), adapter=z(T, dtype=torch.int32), out=z(T, N) + 1,
                ws=m.alloc_lora_workspace(p, T))
    m.moe_lora_forward(p, **good)
    assert not good["out"].any()
    for name, bad, error in [
            ("x", z(T, K + 64), r"x must be \[T\]\[128\]"), ("x", z(T, K).half(), "x must be torch.float32"),
            ("x", z(K, T).t(), "x must be contiguous"), ("W", good["W"][:-1], "W has 4351 elements, needs at least 4352"),
            ("A", good["A"].half(), "A must be torch.bfloat16"), ("B", good["B"].cpu(), "B must be in device memory"),
            ("scale", None, "scale is required"), ("adapter", good["adapter"].long(), "adapter must be torch.int32"),
            ("out", z(T, 2 * N)[:, ::2], "out must be contiguous"), ("u", z(T * r - 1), "u has 31 elements, needs at least 32"),
            ("ws", None, "ws is required")]:
        with pytest.raises(ValueError, match=error):
            m.moe_lora_forward(p, **{**good, name: bad})
    with pytest.raises(TypeError, match="scale must be a torch.Tensor"):
        m.moe_lora_forward(p, **{**good, "scale": 1.0})
    d = m.dims(256, 128, 16, 2)
    i32 = lambda *s: z(*s, dtype=torch.int32)
    bal = dict(logits=z(T, 16), idx=i32(T, 2), counts=i32(16), ntok=i32(1), pmean=z(16), loss=z(1),
               ws=m.alloc_balance_workspace(d, T))
    m.moe_balance_forward(d, **bal)
    assert int(bal["ntok"]) == T
    for name, bad, error in [("seg", i32(1), "seg has 1 elements, needs at least 2"),
                             ("seg", i32(3), "counts has 16 elements, needs at least 32"),
                             ("valid", z(T), "valid must be torch.uint8"), ("idx", i32(T, 1), "idx has 4 elements")]:
        with pytest.raises(ValueError, match=error):
            m.moe_balance_forward(d, **{**bal, name: bad})
    with pytest.raises(TypeError, match="seg must be a torch.Tensor"):
        m.moe_balance_forward(d, **{**bal, "seg": [0, 4]})
