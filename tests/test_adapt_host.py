"""Refusals of the adapter and balance calls, in the C ABI and in the binding.
Everything here is decided on the host: no GPU."""
import ctypes

import pytest
import torch

import int4_routed_expert_softmax_b200 as moe

P = ctypes.c_void_p
OK, BAD_ARG, SHAPE, WORKSPACE = 0, -1, -2, -4


@pytest.fixture(scope="module")
def lib():
    from int4_routed_expert_softmax_b200 import build
    build.build()
    return moe.lib()


def fwd(lib, p, T=4, x=4096, W=4096, A=4096, B=4096, scale=4096, adapter=4096, out=4096, u=None, ws=4096, n=1 << 40):
    return lib.moe_lora_forward(ctypes.byref(p), T, x, W, A, B, scale, adapter, out, u, ws, n, None)


def bwd(lib, p, T=4, g=4096, x=4096, W=4096, A=4096, B=4096, scale=4096, adapter=4096, u=None, dx=4096, dA=4096,
        dB=4096, ws=4096, n=1 << 40):
    return lib.moe_lora_backward(ctypes.byref(p), T, g, x, W, A, B, scale, adapter, u, dx, dA, dB, ws, n, None)


def test_lora_dims(lib):
    good = moe.lora(6144, 2048, 16, 16)
    assert moe.moe_lora_workspace_bytes(good, 16) > 0
    for K, N, n, r in [(0, 64, 1, 8), (96, 64, 1, 8), (8256, 64, 1, 8), (128, 0, 1, 8), (128, 12, 1, 8),
                       (128, 8200, 1, 8), (128, 64, -1, 8), (128, 64, 4097, 8), (128, 64, 1, 0), (128, 64, 1, 12),
                       (128, 64, 1, 136), (-64, 64, 1, 8)]:
        p = moe.lora(K, N, n, r)
        assert fwd(lib, p) == SHAPE and bwd(lib, p) == SHAPE, (K, N, n, r)
        assert moe.moe_lora_workspace_bytes(p, 16) == 0
        with pytest.raises(moe.MoeError):
            moe.alloc_lora_workspace(p, 16, device="cpu")
    bad = moe.MoeLoraDims(128, 64, 1, 8, 2)  # no such type
    assert fwd(lib, bad) == BAD_ARG and moe.moe_lora_workspace_bytes(bad, 4) == 0
    with pytest.raises(ValueError, match="float16 or bfloat16"):
        moe.lora(128, 64, 1, 8, torch.float32)
    assert lib.moe_lora_forward(None, 1, 4096, 4096, 4096, 4096, 4096, 4096, 4096, None, 4096, 1 << 40, None) == BAD_ARG
    assert moe.moe_lora_workspace_bytes(good, 1 << 19) > 0 and moe.moe_lora_workspace_bytes(good, (1 << 19) + 1) == 0
    assert moe.moe_lora_workspace_bytes(good, -1) == 0
    assert moe.moe_lora_workspace_bytes(good, 64, True) >= moe.moe_lora_workspace_bytes(good, 64)


def test_lora_forward_arguments(lib):
    p = moe.lora(128, 64, 2, 8)
    assert fwd(lib, p, T=-1) == BAD_ARG
    for name in ("x", "W", "A", "B", "scale", "adapter", "out", "ws"):
        assert fwd(lib, p, **{name: None}) == BAD_ARG, name
    for name in ("x", "W", "A", "B", "out"):
        assert fwd(lib, p, **{name: 4096 + 8}) == BAD_ARG, name
    assert fwd(lib, p, ws=4096 + 64) == WORKSPACE
    assert fwd(lib, p, n=moe.moe_lora_workspace_bytes(p, 4) - 1) == WORKSPACE
    assert fwd(lib, p, T=0, x=None, W=None, A=None, B=None, out=None, ws=None, n=0) == OK


def test_lora_backward_arguments(lib):
    p = moe.lora(128, 64, 2, 8)
    assert bwd(lib, p, T=-1) == BAD_ARG
    for name in ("g", "x", "W", "A", "B", "scale", "adapter", "ws"):
        assert bwd(lib, p, **{name: None}) == BAD_ARG, name
    for name in ("g", "x", "W", "A", "B", "dx", "dA", "dB"):
        assert bwd(lib, p, **{name: 4096 + 8}) == BAD_ARG, name
    assert bwd(lib, p, ws=4096 + 64) == WORKSPACE
    assert bwd(lib, p, n=moe.moe_lora_workspace_bytes(p, 4, True) - 256) == WORKSPACE


def bal(lib, d, T=4, S=1, seg=None, logits=4096, idx=4096, counts=4096, ntok=4096, pmean=4096, loss=4096, ws=4096,
        n=1 << 40):
    return lib.moe_balance_forward(ctypes.byref(d), T, S, seg, logits, idx, None, counts, ntok, pmean, loss, ws, n, None)


def balb(lib, d, T=4, S=1, seg=None, logits=4096, idx=4096, counts=4096, ntok=4096, dloss=4096, w=None, dw=None,
         dlogits=4096):
    return lib.moe_balance_backward(ctypes.byref(d), T, S, seg, logits, idx, None, counts, ntok, dloss, w, dw, dlogits, None)


def test_balance_arguments(lib):
    d = moe.dims(256, 128, 16, 2)
    bad = moe.dims(256, 128, 16, 17)
    assert bal(lib, bad) == SHAPE and balb(lib, bad) == SHAPE
    assert moe.moe_balance_workspace_bytes(bad, 4) == 0 and moe.moe_balance_workspace_bytes(d, -1) == 0
    assert moe.moe_balance_workspace_bytes(d, 4, 0) == 0 and moe.moe_balance_workspace_bytes(d, 4, 65536) == 0
    for f in (bal, balb):
        assert f(lib, d, T=-1) == BAD_ARG and f(lib, d, S=0) == BAD_ARG
        assert f(lib, d, S=2) == BAD_ARG                       # more than one segment, no offsets
        assert f(lib, d, S=65536, seg=4096) == SHAPE
        assert f(lib, d, logits=4098) == BAD_ARG
    for name in ("logits", "idx", "counts", "ntok", "pmean", "loss", "ws"):
        assert bal(lib, d, **{name: None}) == BAD_ARG, name
    assert bal(lib, d, ws=4096 + 64) == WORKSPACE
    for name in ("logits", "counts", "ntok", "dloss", "dlogits"):
        assert balb(lib, d, **{name: None}) == BAD_ARG, name
    assert balb(lib, d, w=4096) == BAD_ARG and balb(lib, d, dw=4096) == BAD_ARG  # they come together
    assert balb(lib, d, w=4096, dw=4096, idx=None) == BAD_ARG
    assert balb(lib, d, dlogits=4097) == BAD_ARG
    assert balb(lib, d, T=0, logits=None, idx=None, counts=None, ntok=None, dloss=None, dlogits=None) == OK


def test_lora_refuses_a_misaligned_u(lib):
    """The backward reads u in 16-byte pieces."""
    p = moe.lora(128, 64, 2, 8)
    for at in (4096 + 4, 4096 + 8):
        assert fwd(lib, p, u=at) == BAD_ARG and bwd(lib, p, u=at) == BAD_ARG


def test_balance_refuses_more_tokens_than_its_indexes_hold(lib):
    d, most = moe.dims(256, 128, 16, 2), 1 << 25
    for T in (most + 1, 2 ** 31 - 1):
        assert bal(lib, d, T=T) == SHAPE and balb(lib, d, T=T) == SHAPE
        assert moe.moe_balance_workspace_bytes(d, T) == 0
    assert moe.moe_balance_workspace_bytes(d, most, 65535) > 0


def test_binding_refuses_host_tensors_and_wrong_types():
    p = moe.lora(128, 64, 2, 8)
    x, W = torch.zeros(4, 128), torch.zeros(64 * 64 + 256, dtype=torch.uint8)
    A, B = torch.zeros(2, 8, 128, dtype=torch.bfloat16), torch.zeros(2, 64, 8, dtype=torch.bfloat16)
    sc, ad, out, ws = torch.ones(2), torch.zeros(4, dtype=torch.int32), torch.zeros(4, 64), torch.zeros(9, dtype=torch.uint8)
    with pytest.raises(ValueError, match="x must be in device memory"):
        moe.moe_lora_forward(p, x, W, A, B, sc, ad, out, ws)
    with pytest.raises(ValueError, match="x must be in device memory"):
        moe.moe_lora_backward(p, out, x, W, A, B, sc, ad, ws)
    with pytest.raises(TypeError, match="x must be a torch.Tensor"):
        moe.moe_lora_forward(p, x.numpy(), W, A, B, sc, ad, out, ws)
    d = moe.dims(256, 128, 16, 2)
    lg, ix = torch.zeros(4, 16), torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="logits must be in device memory"):
        moe.moe_balance_forward(d, lg, ix, ix, ix, lg, lg, ws)
    with pytest.raises(ValueError, match="logits must be in device memory"):
        moe.moe_balance_backward(d, lg, ix, ix, ix, lg, lg)
