"""The training entry points refuse bad arguments with the documented status before
any HIP call (CPU only: the non-NULL pointers are never dereferenced)."""
import ctypes
import math
import os

import pytest
import torch

import routing_grouped_expert_amd as moe
from routing_grouped_expert_amd import _native as N

FAKE, MISALIGNED = 0x10000, 0x10008


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(N.LIB_PATH):
        from routing_grouped_expert_amd.build import build
        build()
    return N.load()


def routing(fields=None, w_dtype=N.MOE_BF16):
    r = N.MoeRouting(*([FAKE] * 8), w_dtype)
    for k, v in (fields or {}).items():
        setattr(r, k, v)
    return ctypes.byref(r)


SHAPES = [{"h": 0}, {"h": 12}, {"i": 4}, {"i": -8}, {"k": 0}, {"k": 17}, {"e": 0}, {"e": 257},
          {"n": -1}, {"n": 1 << 30},
          {"n": 1 << 20, "h": 1024},                     # x of 2^31 bytes
          {"n": 1 << 16, "k": 4, "i": 2048, "h": 8},     # h of 2^31 bytes
          {"n": 1, "k": 1, "i": 1 << 21, "h": 8},        # inter
          {"h": 1 << 16, "i": 1 << 14}]                  # an expert's w13


def test_experts_train_and_backward(lib):
    def train(x=FAKE, dt=N.MOE_BF16, n=33, h=128, w13=FAKE, w2=FAKE, e=8, i=256, k=2,
              act=N.MOE_ACT_SILU, layout=N.MOE_W13_PACKED, r=None, out=FAKE, hs=FAKE, ws=FAKE,
              size=1 << 40):
        return lib.moe_experts_train(x, dt, n, h, w13, w2, e, i, k, act, layout, None,
                                     r or routing(), out, hs, ws, size, None)

    def backward(x=FAKE, dt=N.MOE_BF16, n=33, h=128, w13=FAKE, w2=FAKE, e=8, i=256, k=2,
                 act=N.MOE_ACT_SILU, layout=N.MOE_W13_PACKED, r=None, out=FAKE, hs=FAKE, ws=FAKE,
                 size=1 << 40, d=FAKE, dw13=FAKE, dw2=FAKE, dw=FAKE):
        return lib.moe_experts_backward(d, x, hs, dt, n, h, w13, w2, e, i, k, act, layout, None,
                                        r or routing(), out, dw13, dw2, dw, ws, size, None)
    for call in (train, backward):
        for bad in SHAPES:
            assert call(**bad) == N.MOE_ERR_SHAPE, bad
        for p in ("x", "w13", "w2", "out", "hs"):
            assert call(**{p: None}) == N.MOE_ERR_NULL, p
            assert call(**{p: MISALIGNED}) == N.MOE_ERR_ALIGN, p
        for f in ("offsets", "col_sorted", "row_sorted", "gate_scal"):
            assert call(r=routing({f: None})) == N.MOE_ERR_NULL, f
            assert call(r=routing({f: MISALIGNED})) == N.MOE_ERR_ALIGN, f
        assert call(dt=2) == N.MOE_ERR_DTYPE
        assert call(r=routing(w_dtype=4)) == N.MOE_ERR_DTYPE
        assert call(act=5) == N.MOE_ERR_UNSUPPORTED
        assert call(layout=3) == N.MOE_ERR_UNSUPPORTED
        assert call(act=N.MOE_ACT_RELU2, layout=N.MOE_W13_INTERLEAVED) == N.MOE_ERR_UNSUPPORTED
        assert call(ws=None) == N.MOE_ERR_WORKSPACE
        assert call(ws=MISALIGNED) == N.MOE_ERR_ALIGN
    need = lib.moe_experts_backward_workspace_bytes(33, 2, 128, 256, N.MOE_BF16)
    assert need >= 66 * (2 * 256 * 2 + 256 * 2 + 256 * 4)
    assert backward(size=need - 1) == N.MOE_ERR_WORKSPACE
    assert train(size=lib.moe_workspace_bytes(33, 8, 2, 128, 256, N.MOE_BF16) - 1) == \
        N.MOE_ERR_WORKSPACE
    for p in ("d", "dw13", "dw2", "dw"):
        assert backward(**{p: None}) == N.MOE_ERR_NULL, p
        assert backward(**{p: MISALIGNED}) == N.MOE_ERR_ALIGN, p
    assert train(None, n=0, w13=None, w2=None, out=None, hs=None, ws=None, size=0) == N.MOE_OK
    # without tokens the weight gradients are still written
    assert backward(n=0, dw13=None) == N.MOE_ERR_NULL
    for bad in ((-1, 2, 128, 256), (33, 0, 128, 256), (33, 17, 128, 256), (33, 2, 12, 256),
                (33, 2, 128, 0)):
        assert lib.moe_experts_backward_workspace_bytes(*bad, N.MOE_BF16) == 0, bad
    assert lib.moe_experts_backward_workspace_bytes(33, 2, 128, 256, 9) == 0


def _tensor(**kw):
    t = N.MoeAdamwTensor(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, 100, N.MOE_BF16, N.MOE_F32)
    for k, v in kw.items():
        setattr(t, k, v)
    return (N.MoeAdamwTensor * 1)(t)


def test_adamw(lib):
    def call(tensors=None, count=1, **kw):
        a = N.MoeAdamw(1e-3, 0.9, 0.999, 1e-8, 0.1, 1, None, None, 0.0, 32, 0, 0)
        for k, v in kw.items():
            setattr(a, k, v)
        return lib.moe_adamw(_tensor() if tensors is None else tensors, count, ctypes.byref(a),
                             None)
    assert lib.moe_adamw(_tensor(), 1, None, None) == N.MOE_ERR_NULL
    assert call(count=0) == N.MOE_OK and call(_tensor(n=0, p=None, grad=None)) == N.MOE_OK
    assert lib.moe_adamw(None, 1, ctypes.byref(N.MoeAdamw(1e-3, 0.9, 0.999, 1e-8, 0.1, 1, None,
                                                          None, 0.0, 32, 0, 0)), None) == \
        N.MOE_ERR_NULL
    assert call(count=-1) == N.MOE_ERR_SHAPE
    nan, inf = math.nan, math.inf
    for bad in ({"lr": -1.0}, {"lr": nan}, {"lr": inf}, {"beta1": 1.0}, {"beta1": nan},
                {"beta2": -0.1}, {"beta2": 1 - 1e-12}, {"eps": -1e-9}, {"eps": inf},
                {"weight_decay": nan}, {"step": 0}, {"step": -3}, {"step": 1 << 31},
                {"grad_norm": FAKE}, {"grad_norm": FAKE, "max_norm": -1.0},
                {"grad_norm": FAKE, "max_norm": nan}):
        assert call(**bad) == N.MOE_ERR_SHAPE, bad
    for off in (2, 4):
        assert call(grad_norm=FAKE + off, max_norm=1.0) == N.MOE_ERR_ALIGN
    assert call(step_on_device=FAKE + 1) == N.MOE_ERR_ALIGN
    for bad in ({"state_bits": 16}, {"stochastic": 2}):
        assert call(**bad) == N.MOE_ERR_UNSUPPORTED, bad
    for f in ("p", "grad", "m", "v"):
        assert call(_tensor(**{f: None})) == N.MOE_ERR_NULL, f
        assert call(_tensor(**{f: MISALIGNED})) == N.MOE_ERR_ALIGN, f
    assert call(_tensor(master=MISALIGNED)) == N.MOE_ERR_ALIGN
    for f in ("m_scale", "v_scale"):
        assert call(_tensor(**{f: None}), state_bits=8) == N.MOE_ERR_NULL, f
        assert call(_tensor(**{f: MISALIGNED}), state_bits=8) == N.MOE_ERR_ALIGN, f
    for bad in ({"n": -1}, {"n": 1 << 36}):
        assert call(_tensor(**bad)) == N.MOE_ERR_SHAPE, bad
    for bad in ({"p_dtype": 2}, {"grad_dtype": -1}):
        assert call(_tensor(**bad)) == N.MOE_ERR_DTYPE, bad


def test_grad_norm(lib):
    def call(tensors=None, out=FAKE, ws=FAKE, size=1 << 30):
        return lib.moe_grad_norm(_tensor() if tensors is None else tensors, 1, out, ws, size, None)
    assert call(_tensor(grad=None)) == N.MOE_ERR_NULL
    assert call(_tensor(grad=MISALIGNED)) == N.MOE_ERR_ALIGN
    assert call(_tensor(grad_dtype=3)) == N.MOE_ERR_DTYPE
    assert call(_tensor(n=-1)) == N.MOE_ERR_SHAPE
    assert call(out=None) == N.MOE_ERR_NULL and call(out=MISALIGNED) == N.MOE_ERR_ALIGN
    assert call(ws=None) == N.MOE_ERR_WORKSPACE and call(size=0) == N.MOE_ERR_WORKSPACE
    assert lib.moe_grad_norm_workspace_bytes(_tensor(n=-1), 1) == 0
    many = lib.moe_grad_norm_workspace_bytes(_tensor(n=1 << 30), 1)
    assert many >= (1 << 30) // 32768 * 8


def test_python_side_refuses_tensors_off_the_gpu():
    p = torch.ones(16)
    s = moe.moe_adamw_state([p], 8, master=True)
    assert s.m[0].dtype == torch.float8_e4m3fn and s.m_scale[0].shape == (1,)
    assert s.master == [None]
    assert moe.moe_adamw_state([p.bfloat16()], master=True).master[0].dtype == torch.float32
    with pytest.raises(ValueError):
        moe.moe_adamw([p], [p.clone()], s, lr=1e-3, step=1)
    with pytest.raises(ValueError):
        moe.moe_grad_norm([p])
    with pytest.raises(ValueError):
        moe.moe_adamw_state([p], 4)
