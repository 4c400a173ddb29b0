"""The row and block-norm entry points refuse bad arguments with the documented
status before any HIP call, and their Python side refuses bad tensors (CPU only:
the non-NULL pointers are never dereferenced)."""
import ctypes
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


def test_row_calls(lib):
    def dispatch(x=FAKE, dt=N.MOE_BF16, n=33, h=128, k=2, r=None, o=FAKE):
        return lib.moe_dispatch(x, dt, n, h, k, r or routing(), o, None)

    def combine(y=FAKE, dt=N.MOE_BF16, n=33, h=128, k=2, r=None, o=FAKE):
        return lib.moe_combine_weighted(y, dt, n, h, k, r or routing(), o, None)

    def backward(y=FAKE, dt=N.MOE_BF16, n=33, h=128, k=2, r=None, o=FAKE, dw=FAKE, d=FAKE):
        return lib.moe_combine_weighted_backward(d, y, dt, n, h, k, r or routing(), o, dw, None)

    for call in (dispatch, combine, backward):
        assert call(None, n=0, o=None) == N.MOE_OK
        assert call(None) == N.MOE_ERR_NULL
        assert call(o=None) == N.MOE_ERR_NULL
        assert call(o=MISALIGNED) == N.MOE_ERR_ALIGN
        assert call(MISALIGNED) == N.MOE_ERR_ALIGN
        assert call(dt=3) == N.MOE_ERR_DTYPE
        assert call(r=routing({"row_sorted": None})) == N.MOE_ERR_NULL
        assert call(r=routing({"row_sorted": MISALIGNED})) == N.MOE_ERR_ALIGN
        for bad in ({"h": 0}, {"h": 12}, {"h": -8}, {"k": 0}, {"k": 17}, {"n": -1},
                    {"n": 1 << 30, "k": 2}, {"h": (1 << 24) + 8}):
            assert call(**bad) == N.MOE_ERR_SHAPE, bad
        # more 16-byte chunks than a grid has threads
        assert call(n=1 << 23, h=1 << 14, k=1) == N.MOE_ERR_SHAPE
    assert backward(n=1 << 24, h=8, k=1) == N.MOE_ERR_SHAPE
    for call in (combine, backward):
        assert call(r=routing({"topk_w": None})) == N.MOE_ERR_NULL
        assert call(r=routing(w_dtype=5)) == N.MOE_ERR_DTYPE
    assert backward(dw=None) == N.MOE_ERR_NULL
    assert backward(d=None) == N.MOE_ERR_NULL
    assert lib.moe_dispatch(FAKE, N.MOE_BF16, 3, 8, 2, None, FAKE, None) == N.MOE_ERR_NULL

    def softmax(d=FAKE, n=33, e=8, k=2, r=None, o=FAKE):
        return lib.moe_route_backward(d, n, e, k, r or routing(), o, None)
    assert softmax(None, n=0, o=None) == N.MOE_OK
    assert softmax(None) == N.MOE_ERR_NULL
    assert softmax(o=MISALIGNED) == N.MOE_ERR_ALIGN
    assert softmax(r=routing({"topk_idx": None})) == N.MOE_ERR_NULL
    assert softmax(r=routing(w_dtype=9)) == N.MOE_ERR_DTYPE
    for bad in ({"e": 0}, {"e": 257}, {"k": 9}, {"n": -1}, {"n": 1 << 25, "e": 128}):
        assert softmax(**bad) == N.MOE_ERR_SHAPE, bad


def norm_struct(w_post=FAKE, w_pre=FAKE, gate=None, kind=N.MOE_GATE_NONE, scale=1.0, eps=1e-6):
    return ctypes.byref(N.MoeBlockNorm(w_post, w_pre, gate, kind, scale, eps))


def test_block_norm_calls(lib):
    def fwd(x=FAKE, y=FAKE, dt=N.MOE_BF16, n=33, h=128, s=None, xo=FAKE, no=FAKE, rp=FAKE):
        return lib.moe_block_norm(x, y, dt, n, h, s or norm_struct(), xo, no, rp, FAKE, None)

    def bwd(x=FAKE, y=FAKE, dt=N.MOE_BF16, n=33, h=128, s=None, xo=FAKE, no=FAKE, rp=FAKE,
            dx=FAKE, dy=FAKE, dwp=FAKE, dg=FAKE, ws=FAKE, wsb=1 << 30):
        return lib.moe_block_norm_backward(xo, no, x, y, dt, n, h, s or norm_struct(), rp, FAKE,
                                           dx, dy, dwp, FAKE, dg, ws, wsb, None)

    nan, inf = float("nan"), float("inf")
    for call in (fwd, bwd):
        assert call(None) == N.MOE_ERR_NULL
        assert call(MISALIGNED) == N.MOE_ERR_ALIGN
        assert call(y=MISALIGNED) == N.MOE_ERR_ALIGN
        assert call(dt=2) == N.MOE_ERR_DTYPE
        assert call(no=None) == N.MOE_ERR_NULL
        assert call(no=MISALIGNED) == N.MOE_ERR_ALIGN
        for bad in ({"h": 0}, {"h": 100}, {"h": 16392}, {"n": -1}, {"n": 1 << 31}):
            assert call(**bad) == N.MOE_ERR_SHAPE, bad
        for s in (norm_struct(eps=0.0), norm_struct(eps=-1.0), norm_struct(eps=nan),
                  norm_struct(eps=inf), norm_struct(scale=nan), norm_struct(scale=inf)):
            assert call(s=s) == N.MOE_ERR_SHAPE
        assert call(s=norm_struct(gate=FAKE, kind=3)) == N.MOE_ERR_UNSUPPORTED
        assert call(s=norm_struct(kind=N.MOE_GATE_TOKEN)) == N.MOE_ERR_NULL
        assert call(s=norm_struct(w_pre=MISALIGNED)) == N.MOE_ERR_ALIGN
        # the parts that need the block's output, and nothing to do at all
        assert call(y=None) == N.MOE_ERR_NULL
        assert call(y=None, s=norm_struct(w_post=None, gate=FAKE, kind=1)) == N.MOE_ERR_NULL
        assert call(y=None, s=norm_struct(w_post=None, w_pre=None)) == N.MOE_ERR_NULL
    assert fwd(None, None, n=0) == N.MOE_OK
    assert fwd(xo=None) == N.MOE_ERR_NULL
    assert lib.moe_block_norm(FAKE, FAKE, N.MOE_BF16, 3, 8, None, FAKE, FAKE, FAKE, FAKE,
                              None) == N.MOE_ERR_NULL
    assert bwd(xo=None, s=norm_struct(w_pre=None)) == N.MOE_ERR_NULL
    assert bwd(rp=None) == N.MOE_ERR_NULL
    assert bwd(dx=None) == N.MOE_ERR_NULL
    assert bwd(dy=None) == N.MOE_ERR_NULL
    assert bwd(dwp=None) == N.MOE_ERR_NULL
    assert bwd(dg=None, s=norm_struct(gate=FAKE, kind=N.MOE_GATE_TOKEN)) == N.MOE_ERR_NULL
    assert bwd(dg=None, n=0, s=norm_struct(gate=FAKE, kind=N.MOE_GATE_CHANNEL)) == N.MOE_ERR_NULL
    assert bwd(ws=None) == N.MOE_ERR_WORKSPACE
    assert bwd(wsb=64) == N.MOE_ERR_WORKSPACE
    assert bwd(ws=MISALIGNED) == N.MOE_ERR_ALIGN


def test_block_norm_workspace(lib):
    ws = lib.moe_block_norm_workspace_bytes
    assert ws(0, 8, N.MOE_BF16) > 0
    assert ws(1, 8, N.MOE_F32) >= 3 * 8 * 4
    assert ws(1 << 20, 16384, N.MOE_BF16) >= 3 * 16384 * 4
    for bad in ((-1, 8), (1 << 31, 8), (4, 0), (4, 12), (4, 16392)):
        assert ws(*bad, N.MOE_BF16) == 0
    assert ws(4, 8, 7) == 0


def test_python_side_refuses_host_tensors():
    x = torch.zeros(4, 16)
    r = moe.Routing.empty(4, 8, 2, torch.float32, "cpu")
    for call in (lambda: moe.moe_dispatch(x, r), lambda: moe.moe_combine_weighted(x, r),
                 lambda: moe.moe_combine_weighted_backward(x, x, r),
                 lambda: moe.moe_route_backward(x, r),
                 lambda: moe.moe_block_norm(x, w_pre=x[0]),
                 lambda: moe.moe_block_norm_backward(x, x, x, w_pre=x[0], rstd_pre=x[0])):
        with pytest.raises(ValueError, match="GPU"):
            call()


def int4(q=FAKE, s=FAKE, z=FAKE):
    return ctypes.byref(N.MoeInt4Weights(q, s, z))


def test_int4_calls(lib):
    def experts(x=FAKE, n=33, h=128, w13=None, w2=None, e=8, i=256, k=2, g=64,
                act=N.MOE_ACT_SILU, layout=N.MOE_W13_PACKED, r=None, o=FAKE, ws=FAKE,
                wsb=1 << 30):
        return lib.moe_experts_int4(x, n, h, w13 or int4(), w2 or int4(z=None), e, i, k, g, act,
                                    layout, None, r or routing(), o, ws, wsb, None)

    def forward(x=FAKE, n=33, h=128, w13=None, w2=None, e=8, i=256, k=2, g=64,
                act=N.MOE_ACT_SILU, layout=N.MOE_W13_PACKED, r=None, o=FAKE, ws=FAKE,
                wsb=1 << 30):
        return lib.moe_forward_int4(x, FAKE, n, h, w13 or int4(), w2 or int4(z=None), e, i, k, g,
                                    act, layout, None, r or routing(), o, ws, wsb, None)

    for call in (experts, forward):
        assert call(None, n=0, o=None) == N.MOE_OK
        assert call(None) == N.MOE_ERR_NULL
        assert call(MISALIGNED) == N.MOE_ERR_ALIGN
        assert call(o=None) == N.MOE_ERR_NULL
        assert call(w13=int4(q=None)) == N.MOE_ERR_NULL
        assert call(w2=int4(s=None)) == N.MOE_ERR_NULL
        assert call(w2=int4(z=MISALIGNED)) == N.MOE_ERR_ALIGN
        for bad in ({"g": 16}, {"g": 0}, {"g": 96}, {"h": 96}, {"i": 96}, {"h": 0}, {"k": 9},
                    {"e": 257}, {"n": -1}, {"n": 1 << 24, "h": 1024}):
            assert call(**bad) == N.MOE_ERR_SHAPE, bad
        assert call(act=5) == N.MOE_ERR_UNSUPPORTED
        assert call(act=N.MOE_ACT_RELU2, layout=N.MOE_W13_INTERLEAVED) == N.MOE_ERR_UNSUPPORTED
        assert call(r=routing({"offsets": None})) == N.MOE_ERR_NULL
        assert call(ws=None) == N.MOE_ERR_WORKSPACE
        assert call(wsb=1024) == N.MOE_ERR_WORKSPACE
    need = lib.moe_int4_workspace_bytes(33, 8, 2, 128, 256)
    assert need >= 66 * 256 * 2 + 66 * 128 * 4
    assert lib.moe_int4_workspace_bytes(33, 8, 9, 128, 256) == 0
    assert lib.moe_int4_workspace_bytes(33, 8, 2, 100, 256) == 0

    def quantize(w=FAKE, dt=N.MOE_F32, e=4, rows=33, k=128, g=64, q=FAKE, s=FAKE, z=None):
        return lib.moe_quantize_int4(w, dt, e, rows, k, g, q, s, z, None)
    assert quantize(None) == N.MOE_ERR_NULL
    assert quantize(q=None) == N.MOE_ERR_NULL
    assert quantize(s=MISALIGNED) == N.MOE_ERR_ALIGN
    assert quantize(z=MISALIGNED) == N.MOE_ERR_ALIGN
    assert quantize(dt=4) == N.MOE_ERR_DTYPE
    for bad in ({"e": 0}, {"rows": 0}, {"k": 96}, {"k": 0}, {"g": 48}, {"g": 0},
                {"e": 1 << 30, "rows": 1 << 20}):
        assert quantize(**bad) == N.MOE_ERR_SHAPE, bad

    def dequantize(w=None, e=4, rows=33, k=128, g=64, o=FAKE):
        return lib.moe_dequantize_int4(w or int4(), e, rows, k, g, o, None)
    assert dequantize(int4(q=None)) == N.MOE_ERR_NULL
    assert dequantize(int4(z=MISALIGNED)) == N.MOE_ERR_ALIGN
    assert dequantize(o=None) == N.MOE_ERR_NULL
    assert dequantize(k=100) == N.MOE_ERR_SHAPE


def test_block_forward_call(lib):
    def block(x=FAKE, wg=FAKE, n=33, h=128, e=8, i=256, k=2, dt=N.MOE_BF16, act=N.MOE_ACT_SILU,
              layout=N.MOE_W13_PACKED, s=None, lg=FAKE, r=None, xo=FAKE, ws=FAKE, wsb=1 << 30):
        return lib.moe_block_forward(x, wg, dt, n, h, FAKE, FAKE, e, i, k, act, layout, None,
                                     s or norm_struct(), lg, r or routing(w_dtype=dt), xo, ws,
                                     wsb, None)
    assert block(None, n=0, xo=None, ws=None) == N.MOE_OK
    assert block(None) == N.MOE_ERR_NULL
    assert block(wg=None) == N.MOE_ERR_NULL
    assert block(lg=None) == N.MOE_ERR_NULL
    assert block(xo=None) == N.MOE_ERR_NULL
    assert block(xo=MISALIGNED) == N.MOE_ERR_ALIGN
    assert block(s=norm_struct(w_pre=None)) == N.MOE_ERR_NULL
    assert block(s=norm_struct(eps=0.0)) == N.MOE_ERR_SHAPE
    assert block(s=norm_struct(kind=N.MOE_GATE_CHANNEL)) == N.MOE_ERR_NULL
    assert block(r=routing({"col_sum": None})) == N.MOE_ERR_NULL
    for bad in ({"h": 100}, {"h": 16392}, {"k": 9}, {"e": 257}, {"i": 12}, {"n": -1}):
        assert block(**bad) == N.MOE_ERR_SHAPE, bad
    assert block(dt=5) == N.MOE_ERR_DTYPE
    assert block(act=N.MOE_ACT_RELU2, layout=N.MOE_W13_INTERLEAVED) == N.MOE_ERR_UNSUPPORTED
    inner = lib.moe_workspace_bytes(33, 8, 2, 128, 256, N.MOE_BF16)
    assert block(ws=None) == N.MOE_ERR_WORKSPACE
    assert block(wsb=inner) == N.MOE_ERR_WORKSPACE
    assert block(ws=MISALIGNED) == N.MOE_ERR_ALIGN
