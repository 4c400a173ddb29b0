"""MI355X (gfx950) MoE-layer forward: routing metadata, grouped expert FFN and
combine, all in hand-written HIP kernels behind the C ABI of ``libmoe.so``.

This module is a thin binding over that ABI: it checks tensor placement and
dtypes, allocates outputs and workspaces with torch, and passes raw device
pointers plus the current HIP stream.  Every step of the layer runs in the
library's kernels; there is no other implementation behind these functions, and
they raise if the library is missing.

    routing = moe_route(logits, topk)
    out = moe_experts(x, w13, w2, routing, act="silu", layout="packed")
    out, routing = moe_forward(x, logits, w13, w2, topk, act="swiglu_oai",
                               layout="interleaved",
                               params={"alpha": 1.702, "beta": 1.0, "limit": 7.0})

With the router's gate weight ``w_gate [E, H]`` the routing step also computes
the logits (router GEMM): ``logits, routing = moe_gate_route(x, w_gate, topk)``;
``moe_gate_forward`` runs the whole layer from ``x`` and ``w_gate``.

One GPU of an expert-parallel group (experts [lo, lo + n) of the layer's E,
weights w13 [n, ...], w2 [n, ...]) uses the ``_ep`` variants; summing their
outputs over the group's shares gives the layer output:

    routing = moe_route_ep(logits, topk, lo, n)
    out = moe_experts_ep(x, w13, w2, routing, act="silu")
    out, routing = moe_forward_ep(x, logits, w13, w2, topk, lo, act="silu")

Expert products that run elsewhere (a training step) take their rows from
``moe_dispatch`` and give them back to ``moe_combine_weighted``; the gradients
are calls of their own (this package registers nothing with autograd):

    x_sorted = moe_dispatch(x, routing)                  # rows by expert
    out = moe_combine_weighted(y_sorted, routing)        # topk_w applied
    d_y_sorted, d_topk_w = moe_combine_weighted_backward(d_out, y_sorted, routing)
    d_logits = moe_route_backward(d_topk_w, routing)
    d_x = moe_combine(d_x_sorted, routing)               # gradient of the dispatch

The norms around the layer, with the gate and the residual sum, are one call:

    s = moe_block_norm(x, y, w_post=w_post, gate=gate, w_pre=w_next, residual_scale=0.22)
    g = moe_block_norm_backward(d_x_out, d_n_out, x, y, w_post=w_post, gate=gate, w_pre=w_next,
                                residual_scale=0.22, rstd_post=s.rstd_post,
                                rstd_pre=s.rstd_pre)

``moe_block_forward`` runs the whole block from its residual stream.  Expert
weights of 4-bit codes with a scale and a zero point a group, for decoding:

    w13_q, w13_s, w13_z = moe_quantize_int4(w13, group=128)
    w2_q, w2_s, w2_z = moe_quantize_int4(w2, group=128)
    out = moe_experts_int4(x, w13_q, w13_s, w13_z, w2_q, w2_s, w2_z, routing, act="silu")
"""
from __future__ import annotations

import ctypes
from dataclasses import InitVar, dataclass
from typing import Optional

import torch

from . import _native as N

__all__ = ["Routing", "MoeError", "Prepared", "moe_route", "moe_experts", "moe_experts_w13",
           "moe_experts_w2", "moe_experts_w2_rows", "moe_combine", "prepare_experts_w2_rows",
           "prepare_combine", "moe_forward", "moe_forward_noalloc", "prepare_forward_noalloc",
           "prepare_route", "prepare_experts",
           "prepare_experts_w13", "prepare_experts_w2", "prepare_forward",
           "moe_route_ep", "moe_experts_ep", "moe_forward_ep", "prepare_route_ep",
           "prepare_experts_ep", "prepare_forward_ep", "moe_gate_route", "moe_gate_forward",
           "prepare_gate_route", "prepare_gate_forward", "moe_experts_weighted_input",
           "prepare_experts_weighted_input", "moe_quantize_mxfp4", "moe_experts_mxfp4",
           "moe_forward_mxfp4", "prepare_experts_mxfp4", "prepare_forward_mxfp4",
           "moe_dispatch", "moe_combine_weighted", "moe_combine_weighted_backward",
           "moe_route_backward", "prepare_dispatch", "prepare_combine_weighted",
           "prepare_combine_weighted_backward", "prepare_route_backward", "BlockNorm",
           "BlockNormGrads", "moe_block_norm", "moe_block_norm_backward", "prepare_block_norm",
           "prepare_block_norm_backward", "moe_block_norm_workspace_bytes", "moe_block_forward",
           "prepare_block_forward", "moe_quantize_int4",
           "moe_dequantize_int4", "moe_experts_int4", "moe_forward_int4", "prepare_experts_int4",
           "prepare_forward_int4", "moe_int4_workspace_bytes",
           "moe_workspace_bytes", "moe_status_str", "ACTS", "LAYOUTS"]

_DT = {torch.float32: N.MOE_F32, torch.bfloat16: N.MOE_BF16}
ACTS = {"silu": N.MOE_ACT_SILU, "swiglu_oai": N.MOE_ACT_SWIGLU_OAI, "relu2": N.MOE_ACT_RELU2}
LAYOUTS = {"packed": N.MOE_W13_PACKED, "interleaved": N.MOE_W13_INTERLEAVED}
_PBITS = {"alpha": N.MOE_PARAM_ALPHA, "beta": N.MOE_PARAM_BETA, "limit": N.MOE_PARAM_LIMIT}


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {moe_status_str(status)} (status {status})")


def moe_status_str(status: int) -> str:
    return N.load().moe_status_str(status).decode()


def _check(status: int, where: str):
    if status != N.MOE_OK:
        raise MoeError(status, where)


def _dt(t: torch.Tensor) -> int:
    if t.dtype not in _DT:
        raise TypeError(f"unsupported dtype {t.dtype}; expected float32 or bfloat16")
    return _DT[t.dtype]


def _dev(*ts: torch.Tensor):
    dev = ts[0].device
    for t in ts:
        if t.device.type != "cuda" or t.device != dev:
            raise ValueError("all tensors must be on the same GPU")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
    return dev


def _shapes(x, w13, w2, act, out=None, logits=None, n_experts=None):
    """Every buffer size the kernels assume, checked before any launch.
    ``n_experts`` is the logits' expert count when w13/w2 hold only a share."""
    if act not in ACTS:
        raise ValueError(f"unknown activation {act!r}")
    if x.dim() != 2 or w13.dim() != 3 or w2.dim() != 3:
        raise ValueError("expected x [N, H], w13 [E, nI, H], w2 [E, H, I]")
    n, hidden = x.shape
    e, h2, inter = w2.shape
    rows = inter if act == "relu2" else 2 * inter
    if h2 != hidden or tuple(w13.shape) != (e, rows, hidden):
        raise ValueError(f"w13 {tuple(w13.shape)} / w2 {tuple(w2.shape)} do not match "
                         f"x {tuple(x.shape)} and act {act!r}")
    if not (x.dtype == w13.dtype == w2.dtype):
        raise TypeError("x, w13 and w2 must share a dtype")
    if out is not None and (tuple(out.shape) != (n, hidden) or out.dtype != x.dtype):
        raise ValueError("out must be [N, H] in the layer dtype")
    if logits is not None and (logits.dim() != 2 or
                               tuple(logits.shape) != (n, e if n_experts is None else n_experts)):
        raise ValueError("logits must be [N, E]")


def _check_routing(routing: "Routing", n: int, e: int, k: int, fills: Optional[int] = None):
    """Buffers of the sizes that n tokens, e experts and k slots need.  ``fills``:
    the call writes the routing, of a layer of that many experts."""
    m = n * k
    want = {"topk_idx": (n, k), "topk_w": (n, k), "bitmatrix": (n, (e + 31) // 32),
            "col_sum": (e,), "offsets": (e + 1,), "col_sorted": (m,), "row_sorted": (m,),
            "gate_scal": (m,)}
    for f, shp in want.items():
        t = getattr(routing, f)
        if tuple(t.shape) != shp or not t.is_contiguous():
            raise ValueError(f"routing.{f} must be contiguous {shp}, got {tuple(t.shape)}")
    if routing.gate_scal.dtype != routing.topk_w.dtype:
        raise TypeError("routing.topk_w and gate_scal must share a dtype")
    if fills is not None and fills != e:
        routing.layer_experts = fills
    elif fills is not None:
        vars(routing).pop("layer_experts", None)


def _stream(dev, stream) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    return ctypes.c_void_p(s.cuda_stream)


@dataclass
class Routing:
    """Routing metadata of one layer (device tensors); field meanings as in moe.h."""

    topk_idx: torch.Tensor    # [N, k] int32
    topk_w: torch.Tensor      # [N, k] logits dtype
    bitmatrix: torch.Tensor   # [N, ceil(E/32)] int32 (uint32 bit patterns)
    col_sum: torch.Tensor     # [E] int32
    offsets: torch.Tensor     # [E+1] int32
    col_sorted: torch.Tensor  # [N*k] int32
    row_sorted: torch.Tensor  # [N*k] int32
    gate_scal: torch.Tensor   # [N*k] logits dtype
    # the layer's expert count in the routing of an expert share; None: whole layer.
    # (An attribute of a share's routing only, so that the fields stay all tensors.)
    layer_experts: InitVar[Optional[int]] = None

    def __post_init__(self, layer_experts):
        if layer_experts is not None:
            self.layer_experts = layer_experts

    @classmethod
    def empty(cls, n_tokens: int, n_experts: int, topk: int, dtype: torch.dtype,
              device) -> "Routing":
        i32 = dict(dtype=torch.int32, device=device)
        m = n_tokens * topk
        return cls(
            topk_idx=torch.empty(n_tokens, topk, **i32),
            topk_w=torch.empty(n_tokens, topk, dtype=dtype, device=device),
            bitmatrix=torch.empty(n_tokens, (n_experts + 31) // 32, **i32),
            col_sum=torch.empty(n_experts, **i32),
            offsets=torch.empty(n_experts + 1, **i32),
            col_sorted=torch.empty(m, **i32),
            row_sorted=torch.empty(m, **i32),
            gate_scal=torch.empty(m, dtype=dtype, device=device),
        )

    @property
    def n_experts(self) -> int:
        return self.col_sum.numel()

    @property
    def topk(self) -> int:
        return self.topk_idx.shape[1]

    def tensors(self) -> tuple:
        return (self.topk_idx, self.topk_w, self.bitmatrix, self.col_sum, self.offsets,
                self.col_sorted, self.row_sorted, self.gate_scal)

    def as_c(self) -> N.MoeRouting:
        return N.MoeRouting(*(t.data_ptr() for t in self.tensors()), _dt(self.topk_w))


def _params(params: Optional[dict]) -> Optional[N.MoeActParams]:
    if not params:
        return None
    p = N.MoeActParams(1.0, 0.0, 0.0, 0)
    for k, v in params.items():
        if k not in _PBITS:
            raise ValueError(f"unknown activation parameter {k!r}")
        if v is None:
            continue  # unset: the kernel keeps its plain-SwiGLU default
        setattr(p, k, float(v))
        p.set |= _PBITS[k]
    return p


def moe_workspace_bytes(n_tokens: int, n_experts: int, topk: int, hidden: int = 0,
                        inter: int = 0, dtype: torch.dtype = torch.bfloat16) -> int:
    b = N.load().moe_workspace_bytes(n_tokens, n_experts, topk, hidden, inter, _DT[dtype])
    if b == 0:
        raise MoeError(N.MOE_ERR_SHAPE, "moe_workspace_bytes")
    return b


def _workspace(ws, nbytes: int, device) -> torch.Tensor:
    if ws is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    if ws.numel() * ws.element_size() < nbytes:
        raise MoeError(N.MOE_ERR_WORKSPACE, "workspace")
    return ws


class Prepared:
    """One validated C-ABI call with its arguments marshalled once; calling it
    re-enqueues the same work (same buffers, same stream) without re-checking
    or re-converting anything on the Python side."""

    def __init__(self, name: str, args: tuple, keep: tuple, result):
        self._fn = getattr(N.load(), name)
        self._name = name
        self._args = args
        self._keep = keep          # ctypes structs and tensors the pointers refer to
        self.result = result

    def __call__(self):
        st = self._fn(*self._args)
        if st != N.MOE_OK:
            raise MoeError(st, self._name)
        return self.result


def _nbytes(t: torch.Tensor) -> int:
    return t.numel() * t.element_size()


def _share(e: int, local_offset: int, n_local: int):
    if not (0 <= local_offset and 1 <= n_local and local_offset + n_local <= e):
        raise ValueError(f"expert share [{local_offset}, {local_offset + n_local}) is not "
                         f"inside [0, {e})")


def prepare_route(logits: torch.Tensor, topk: int, *, routing: Optional[Routing] = None,
                  workspace: Optional[torch.Tensor] = None, stream=None,
                  _share_of: Optional[tuple] = None) -> Prepared:
    dev = _dev(logits)
    if logits.dim() != 2:
        raise ValueError("logits must be [N, E]")
    n, e = logits.shape
    lo, nl = _share_of if _share_of is not None else (0, e)
    _share(e, lo, nl)
    if routing is None:
        routing = Routing.empty(n, nl, topk, logits.dtype, dev)
    _check_routing(routing, n, nl, topk, fills=e)
    ws = _workspace(workspace, moe_workspace_bytes(n, e, topk, 0, 0, logits.dtype), dev)
    r = routing.as_c()
    if _share_of is None:
        args = (logits.data_ptr(), _dt(logits), n, e, topk, ctypes.byref(r), ws.data_ptr(),
                _nbytes(ws), _stream(dev, stream))
        return Prepared("moe_route", args, (r, logits, ws, routing), routing)
    args = (logits.data_ptr(), _dt(logits), n, e, topk, lo, nl, ctypes.byref(r), ws.data_ptr(),
            _nbytes(ws), _stream(dev, stream))
    return Prepared("moe_route_ep", args, (r, logits, ws, routing), routing)


def prepare_route_ep(logits: torch.Tensor, topk: int, local_offset: int, n_local: int, *,
                     routing: Optional[Routing] = None, workspace: Optional[torch.Tensor] = None,
                     stream=None) -> Prepared:
    return prepare_route(logits, topk, routing=routing, workspace=workspace, stream=stream,
                         _share_of=(local_offset, n_local))


def moe_route_ep(logits: torch.Tensor, topk: int, local_offset: int, n_local: int, *,
                 routing: Optional[Routing] = None, workspace: Optional[torch.Tensor] = None,
                 stream=None) -> Routing:
    """Routing for the expert share [local_offset, local_offset + n_local) of
    ``logits [N, E]``: global top-k, metadata over the local experts (moe.h)."""
    return prepare_route_ep(logits, topk, local_offset, n_local, routing=routing,
                            workspace=workspace, stream=stream)()


def moe_route(logits: torch.Tensor, topk: int, *, routing: Optional[Routing] = None,
              workspace: Optional[torch.Tensor] = None, stream=None) -> Routing:
    """Top-k gating and routing metadata for ``logits [N, E]`` (see moe.h)."""
    return prepare_route(logits, topk, routing=routing, workspace=workspace, stream=stream)()


def prepare_experts(x, w13, w2, routing: Routing, act: str, layout: str = "packed",
                    params: Optional[dict] = None, *, out=None, workspace=None,
                    stream=None, _ep: bool = False) -> Prepared:
    dev = _dev(x, w13, w2)
    _shapes(x, w13, w2, act, out)
    n, hidden = x.shape
    e, inter = w2.shape[0], w2.shape[2]
    k = routing.topk
    _check_routing(routing, n, e, k)
    if out is None:
        out = torch.empty_like(x)
    # the experts' workspace does not depend on the expert count (any E >= k)
    ws = _workspace(workspace, moe_workspace_bytes(n, max(e, k), k, hidden, inter, x.dtype),
                    dev)
    r = routing.as_c()
    p = _params(params)
    args = (x.data_ptr(), _dt(x), n, hidden, w13.data_ptr(), w2.data_ptr(), e, inter, k,
            ACTS[act], LAYOUTS[layout], ctypes.byref(p) if p else None, ctypes.byref(r),
            out.data_ptr(), ws.data_ptr(), _nbytes(ws), _stream(dev, stream))
    return Prepared("moe_experts_ep" if _ep else "moe_experts", args,
                    (r, p, x, w13, w2, out, ws, routing), out)


def prepare_experts_ep(x, w13, w2, routing: Routing, act: str, layout: str = "packed",
                       params: Optional[dict] = None, *, out=None, workspace=None,
                       stream=None) -> Prepared:
    return prepare_experts(x, w13, w2, routing, act, layout, params, out=out,
                           workspace=workspace, stream=stream, _ep=True)


def moe_experts_ep(x: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor, routing: Routing,
                   act: str, layout: str = "packed", params: Optional[dict] = None, *,
                   out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """Expert FFN of one expert share (w13/w2 hold its n_local experts) from a
    moe_route_ep routing; tokens with no slot in the share get zero rows."""
    return prepare_experts_ep(x, w13, w2, routing, act, layout, params, out=out,
                              workspace=workspace, stream=stream)()


def moe_experts(x: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor, routing: Routing,
                act: str, layout: str = "packed", params: Optional[dict] = None, *,
                out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """Grouped expert FFN + weighted combine from existing routing metadata."""
    return prepare_experts(x, w13, w2, routing, act, layout, params, out=out,
                           workspace=workspace, stream=stream)()


def prepare_experts_w13(x, w13, routing: Routing, act: str, layout: str = "packed",
                        params: Optional[dict] = None, *, act_out=None,
                        stream=None) -> Prepared:
    dev = _dev(x, w13)
    n, hidden = x.shape
    e, k = routing.n_experts, routing.topk
    inter = w13.shape[1] if act == "relu2" else w13.shape[1] // 2
    _shapes(x, w13, torch.empty(e, hidden, inter, device="meta", dtype=x.dtype), act)
    _check_routing(routing, n, e, k)
    if act_out is None:
        act_out = torch.empty(n * k, inter, dtype=x.dtype, device=dev)
    if tuple(act_out.shape) != (n * k, inter) or act_out.dtype != x.dtype:
        raise ValueError("act_out must be [N*k, inter] in the layer dtype")
    r = routing.as_c()
    p = _params(params)
    args = (x.data_ptr(), _dt(x), n, hidden, w13.data_ptr(), e, inter, k, ACTS[act],
            LAYOUTS[layout], ctypes.byref(p) if p else None, ctypes.byref(r),
            act_out.data_ptr(), _stream(dev, stream))
    return Prepared("moe_experts_w13", args, (r, p, x, w13, act_out, routing), act_out)


def moe_experts_w13(x: torch.Tensor, w13: torch.Tensor, routing: Routing, act: str,
                    layout: str = "packed", params: Optional[dict] = None, *,
                    act_out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Grouped GEMM with w13 + activation; returns the sorted activation rows
    ``[N*k, inter]`` that moe_experts_w2 consumes."""
    return prepare_experts_w13(x, w13, routing, act, layout, params, act_out=act_out,
                               stream=stream)()


def prepare_experts_w2(act_in, w2, routing: Routing, *, out=None, workspace=None,
                       stream=None) -> Prepared:
    dev = _dev(act_in, w2)
    e, hidden, inter = w2.shape
    k = routing.topk
    n = routing.topk_idx.shape[0]
    if tuple(act_in.shape) != (n * k, inter) or act_in.dtype != w2.dtype:
        raise ValueError("act_in must be [N*k, inter] in the layer dtype")
    _check_routing(routing, n, e, k)
    if out is None:
        out = torch.empty(n, hidden, dtype=w2.dtype, device=dev)
    if tuple(out.shape) != (n, hidden) or out.dtype != w2.dtype:
        raise ValueError("out must be [N, hidden] in the layer dtype")
    ws = _workspace(workspace, moe_workspace_bytes(n, e, k, hidden, inter, w2.dtype), dev)
    r = routing.as_c()
    args = (act_in.data_ptr(), _dt(act_in), n, hidden, w2.data_ptr(), e, inter, k,
            ctypes.byref(r), out.data_ptr(), ws.data_ptr(), _nbytes(ws), _stream(dev, stream))
    return Prepared("moe_experts_w2", args, (r, act_in, w2, out, ws, routing), out)


def moe_experts_w2(act_in: torch.Tensor, w2: torch.Tensor, routing: Routing, *,
                   out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """Grouped GEMM with w2 + routing weight + combine into ``out [N, hidden]``."""
    return prepare_experts_w2(act_in, w2, routing, out=out, workspace=workspace,
                              stream=stream)()


def prepare_experts_w2_rows(act_in, w2, routing: Routing, *, y_sorted=None,
                            stream=None) -> Prepared:
    dev = _dev(act_in, w2)
    e, hidden, inter = w2.shape
    k = routing.topk
    n = routing.topk_idx.shape[0]
    if tuple(act_in.shape) != (n * k, inter) or act_in.dtype != w2.dtype:
        raise ValueError("act_in must be [N*k, inter] in the layer dtype")
    _check_routing(routing, n, e, k)
    if y_sorted is None:
        y_sorted = torch.empty(n * k, hidden, dtype=w2.dtype, device=dev)
    if tuple(y_sorted.shape) != (n * k, hidden) or y_sorted.dtype != w2.dtype:
        raise ValueError("y_sorted must be [N*k, hidden] in the layer dtype")
    _dev(act_in, y_sorted)
    r = routing.as_c()
    args = (act_in.data_ptr(), _dt(act_in), n, hidden, w2.data_ptr(), e, inter, k,
            ctypes.byref(r), y_sorted.data_ptr(), _stream(dev, stream))
    return Prepared("moe_experts_w2_rows", args, (r, act_in, w2, y_sorted, routing), y_sorted)


def moe_experts_w2_rows(act_in: torch.Tensor, w2: torch.Tensor, routing: Routing, *,
                        y_sorted: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Grouped GEMM with w2 + routing weight into the sorted rows ``[N*k, hidden]``
    (no combine); rows past the routed ones are left as they were."""
    return prepare_experts_w2_rows(act_in, w2, routing, y_sorted=y_sorted, stream=stream)()


def prepare_combine(y_sorted, routing: Routing, *, out=None, stream=None) -> Prepared:
    dev = _dev(y_sorted)
    n, k = routing.topk_idx.shape
    if y_sorted.dim() != 2 or y_sorted.shape[0] != n * k:
        raise ValueError("y_sorted must be [N*k, hidden]")
    hidden = y_sorted.shape[1]
    rs = routing.row_sorted
    if tuple(rs.shape) != (n * k,) or rs.dtype != torch.int32 or not rs.is_contiguous():
        raise ValueError("routing.row_sorted must be contiguous int32 [N*k]")
    if out is None:
        out = torch.empty(n, hidden, dtype=y_sorted.dtype, device=dev)
    if tuple(out.shape) != (n, hidden) or out.dtype != y_sorted.dtype:
        raise ValueError("out must be [N, hidden] in the dtype of y_sorted")
    _dev(y_sorted, out, rs)
    r = routing.as_c()
    args = (y_sorted.data_ptr(), _dt(y_sorted), n, hidden, k, ctypes.byref(r), out.data_ptr(),
            _stream(dev, stream))
    return Prepared("moe_combine", args, (r, y_sorted, out, routing), out)


def moe_combine(y_sorted: torch.Tensor, routing: Routing, *, out: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """Scatter-combine ``out[t] = sum_j y_sorted[row_sorted[t*k + j]]`` (slot order,
    fp32 sum, one rounding; slots with row_sorted = -1 skipped)."""
    return prepare_combine(y_sorted, routing, out=out, stream=stream)()


def prepare_forward(x, logits, w13, w2, topk: int, act: str, layout: str = "packed",
                    params: Optional[dict] = None, *, out=None, routing=None, workspace=None,
                    stream=None) -> Prepared:
    dev = _dev(x, logits, w13, w2)
    _shapes(x, w13, w2, act, out, logits)
    n, hidden = x.shape
    e, inter = w2.shape[0], w2.shape[2]
    if logits.dtype != x.dtype:
        raise TypeError("moe_forward takes logits in the layer dtype")
    if routing is None:
        routing = Routing.empty(n, e, topk, logits.dtype, dev)
    _check_routing(routing, n, e, topk, fills=e)
    if out is None:
        out = torch.empty_like(x)
    ws = _workspace(workspace, moe_workspace_bytes(n, e, topk, hidden, inter, x.dtype), dev)
    r = routing.as_c()
    p = _params(params)
    args = (x.data_ptr(), logits.data_ptr(), _dt(x), n, hidden, w13.data_ptr(), w2.data_ptr(),
            e, inter, topk, ACTS[act], LAYOUTS[layout], ctypes.byref(p) if p else None,
            ctypes.byref(r), out.data_ptr(), ws.data_ptr(), _nbytes(ws), _stream(dev, stream))
    return Prepared("moe_forward", args, (r, p, x, logits, w13, w2, out, ws, routing),
                    (out, routing))


def prepare_forward_noalloc(x, logits, w13, w2, topk: int, act: str, layout: str = "packed",
                            params: Optional[dict] = None, *, out=None, routing=None,
                            stream=None) -> Prepared:
    dev = _dev(x, logits, w13, w2)
    _shapes(x, w13, w2, act, out, logits)
    n, hidden = x.shape
    e, inter = w2.shape[0], w2.shape[2]
    if logits.dtype != x.dtype:
        raise TypeError("moe_forward_noalloc takes logits in the layer dtype")
    if routing is None:
        routing = Routing.empty(n, e, topk, logits.dtype, dev)
    _check_routing(routing, n, e, topk, fills=e)
    if out is None:
        out = torch.empty_like(x)
    r = routing.as_c()
    p = _params(params)
    args = (x.data_ptr(), logits.data_ptr(), _dt(x), n, hidden, w13.data_ptr(), w2.data_ptr(),
            e, inter, topk, ACTS[act], LAYOUTS[layout], ctypes.byref(p) if p else None,
            ctypes.byref(r), out.data_ptr(), _stream(dev, stream))
    return Prepared("moe_forward_noalloc", args, (r, p, x, logits, w13, w2, out, routing),
                    (out, routing))


def moe_forward_noalloc(x: torch.Tensor, logits: torch.Tensor, w13: torch.Tensor,
                        w2: torch.Tensor, topk: int, act: str, layout: str = "packed",
                        params: Optional[dict] = None, *, out: Optional[torch.Tensor] = None,
                        routing: Optional[Routing] = None, stream=None):
    """moe_forward with no workspace argument: the intermediates live in the
    library's static per-GPU scratch (MOE_NOALLOC_SCRATCH_BYTES).  With ``out``
    and ``routing`` given, nothing is allocated; calls that overlap on one GPU
    race.  Returns (out, routing)."""
    return prepare_forward_noalloc(x, logits, w13, w2, topk, act, layout, params, out=out,
                                   routing=routing, stream=stream)()


def prepare_forward_ep(x, logits, w13, w2, topk: int, local_offset: int, act: str,
                       layout: str = "packed", params: Optional[dict] = None, *, out=None,
                       routing=None, workspace=None, stream=None) -> Prepared:
    dev = _dev(x, logits, w13, w2)
    n, hidden = x.shape
    e = logits.shape[1]
    nl, inter = w2.shape[0], w2.shape[2]
    _shapes(x, w13, w2, act, out, logits, n_experts=e)
    _share(e, local_offset, nl)
    if logits.dtype != x.dtype:
        raise TypeError("moe_forward_ep takes logits in the layer dtype")
    if routing is None:
        routing = Routing.empty(n, nl, topk, logits.dtype, dev)
    _check_routing(routing, n, nl, topk, fills=e)
    if out is None:
        out = torch.empty_like(x)
    ws = _workspace(workspace, moe_workspace_bytes(n, e, topk, hidden, inter, x.dtype), dev)
    r = routing.as_c()
    p = _params(params)
    args = (x.data_ptr(), logits.data_ptr(), _dt(x), n, hidden, w13.data_ptr(), w2.data_ptr(),
            e, local_offset, nl, inter, topk, ACTS[act], LAYOUTS[layout],
            ctypes.byref(p) if p else None, ctypes.byref(r), out.data_ptr(), ws.data_ptr(),
            _nbytes(ws), _stream(dev, stream))
    return Prepared("moe_forward_ep", args, (r, p, x, logits, w13, w2, out, ws, routing),
                    (out, routing))


def moe_forward_ep(x: torch.Tensor, logits: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor,
                   topk: int, local_offset: int, act: str, layout: str = "packed",
                   params: Optional[dict] = None, *, out: Optional[torch.Tensor] = None,
                   routing: Optional[Routing] = None, workspace: Optional[torch.Tensor] = None,
                   stream=None):
    """moe_route_ep then moe_experts_ep for the share of w13/w2's experts that
    starts at ``local_offset``; returns ``(out, routing)``."""
    return prepare_forward_ep(x, logits, w13, w2, topk, local_offset, act, layout, params,
                              out=out, routing=routing, workspace=workspace, stream=stream)()


def moe_forward(x: torch.Tensor, logits: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor,
                topk: int, act: str, layout: str = "packed", params: Optional[dict] = None, *,
                out: Optional[torch.Tensor] = None, routing: Optional[Routing] = None,
                workspace: Optional[torch.Tensor] = None, stream=None):
    """Routing then experts on one stream; returns ``(out, routing)``."""
    return prepare_forward(x, logits, w13, w2, topk, act, layout, params, out=out,
                           routing=routing, workspace=workspace, stream=stream)()


def _gate_args(x, w_gate, logits):
    dev = _dev(x, w_gate)
    if x.dim() != 2 or w_gate.dim() != 2 or x.shape[1] != w_gate.shape[1]:
        raise ValueError("expected x [N, H] and w_gate [E, H]")
    if x.dtype != w_gate.dtype:
        raise TypeError("x and w_gate must share a dtype")
    n, e = x.shape[0], w_gate.shape[0]
    if logits is None:
        logits = torch.empty(n, e, dtype=x.dtype, device=dev)
    _dev(x, logits)
    if tuple(logits.shape) != (n, e) or logits.dtype != x.dtype:
        raise ValueError("logits must be [N, E] in the layer dtype")
    return dev, n, e, logits


def prepare_gate_route(x: torch.Tensor, w_gate: torch.Tensor, topk: int, *,
                       logits: Optional[torch.Tensor] = None, routing: Optional[Routing] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None) -> Prepared:
    dev, n, e, logits = _gate_args(x, w_gate, logits)
    if routing is None:
        routing = Routing.empty(n, e, topk, x.dtype, dev)
    _check_routing(routing, n, e, topk, fills=e)
    ws = _workspace(workspace, moe_workspace_bytes(n, e, topk, x.shape[1], 0, x.dtype), dev)
    r = routing.as_c()
    args = (x.data_ptr(), w_gate.data_ptr(), _dt(x), n, x.shape[1], e, topk, logits.data_ptr(),
            ctypes.byref(r), ws.data_ptr(), _nbytes(ws), _stream(dev, stream))
    return Prepared("moe_gate_route", args, (r, x, w_gate, logits, ws, routing),
                    (logits, routing))


def moe_gate_route(x: torch.Tensor, w_gate: torch.Tensor, topk: int, *,
                   logits: Optional[torch.Tensor] = None, routing: Optional[Routing] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None):
    """Router GEMM ``logits = x . w_gate^T`` then the routing step; returns
    ``(logits, routing)`` (see moe.h)."""
    return prepare_gate_route(x, w_gate, topk, logits=logits, routing=routing,
                              workspace=workspace, stream=stream)()


def prepare_gate_forward(x, w_gate, w13, w2, topk: int, act: str, layout: str = "packed",
                         params: Optional[dict] = None, *, out=None, logits=None, routing=None,
                         workspace=None, stream=None) -> Prepared:
    dev, n, e, logits = _gate_args(x, w_gate, logits)
    _dev(x, w13, w2)
    _shapes(x, w13, w2, act, out, logits)
    hidden, inter = x.shape[1], w2.shape[2]
    if routing is None:
        routing = Routing.empty(n, e, topk, x.dtype, dev)
    _check_routing(routing, n, e, topk, fills=e)
    if out is None:
        out = torch.empty_like(x)
    ws = _workspace(workspace, moe_workspace_bytes(n, e, topk, hidden, inter, x.dtype), dev)
    r = routing.as_c()
    p = _params(params)
    args = (x.data_ptr(), w_gate.data_ptr(), _dt(x), n, hidden, w13.data_ptr(), w2.data_ptr(),
            e, inter, topk, ACTS[act], LAYOUTS[layout], ctypes.byref(p) if p else None,
            logits.data_ptr(), ctypes.byref(r), out.data_ptr(), ws.data_ptr(), _nbytes(ws),
            _stream(dev, stream))
    return Prepared("moe_gate_forward", args,
                    (r, p, x, w_gate, w13, w2, out, logits, ws, routing), (out, logits, routing))


def moe_gate_forward(x: torch.Tensor, w_gate: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor,
                     topk: int, act: str, layout: str = "packed", params: Optional[dict] = None,
                     *, out: Optional[torch.Tensor] = None, logits: Optional[torch.Tensor] = None,
                     routing: Optional[Routing] = None, workspace: Optional[torch.Tensor] = None,
                     stream=None):
    """The whole layer from the token rows and the router's gate weight;
    returns ``(out, logits, routing)``."""
    return prepare_gate_forward(x, w_gate, w13, w2, topk, act, layout, params, out=out,
                                logits=logits, routing=routing, workspace=workspace,
                                stream=stream)()


def prepare_experts_weighted_input(x, w13, w2, routing: Routing, act: str,
                                   layout: str = "packed", params: Optional[dict] = None, *,
                                   out=None, workspace=None, stream=None) -> Prepared:
    dev = _dev(x, w13, w2)
    _shapes(x, w13, w2, act, out)
    n, hidden = x.shape
    e, inter = w2.shape[0], w2.shape[2]
    k = routing.topk
    _check_routing(routing, n, e, k)
    if out is None:
        out = torch.empty_like(x)
    # the scaled input rows xs [N*k, hidden] follow the experts' workspace
    need = moe_workspace_bytes(n, max(e, k), k, hidden, inter, x.dtype) \
        + (n * k * hidden * x.element_size() + 255) // 256 * 256
    ws = _workspace(workspace, need, dev)
    r = routing.as_c()
    p = _params(params)
    args = (x.data_ptr(), _dt(x), n, hidden, w13.data_ptr(), w2.data_ptr(), e, inter, k,
            ACTS[act], LAYOUTS[layout], ctypes.byref(p) if p else None, ctypes.byref(r),
            out.data_ptr(), ws.data_ptr(), _nbytes(ws), _stream(dev, stream))
    return Prepared("moe_experts_weighted_input", args, (r, p, x, w13, w2, out, ws, routing), out)


def moe_experts_weighted_input(x: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor,
                               routing: Routing, act: str, layout: str = "packed",
                               params: Optional[dict] = None, *,
                               out: Optional[torch.Tensor] = None,
                               workspace: Optional[torch.Tensor] = None,
                               stream=None) -> torch.Tensor:
    """Expert FFN with the routing weight applied to each entry's input row
    (rounded to the layer dtype) instead of its output (see moe.h)."""
    return prepare_experts_weighted_input(x, w13, w2, routing, act, layout, params, out=out,
                                          workspace=workspace, stream=stream)()


def moe_quantize_mxfp4(w: torch.Tensor, *, stream=None):
    """MXFP4 expert weights from ``w [E, rows, K]`` (K a multiple of 32): returns
    ``(q [E, rows, K/2] uint8, scales [E, K/32, rows] uint8)`` (see moe.h)."""
    dev = _dev(w)
    if w.dim() != 3:
        raise ValueError("expected w [E, rows, K]")
    e, rows, k = w.shape
    q = torch.empty(e, rows, k // 2, dtype=torch.uint8, device=dev)
    sc = torch.empty(e, k // 32, rows, dtype=torch.uint8, device=dev)
    _check(N.load().moe_quantize_mxfp4(w.data_ptr(), _dt(w), e, rows, k, q.data_ptr(),
                                       sc.data_ptr(), _stream(dev, stream)), "moe_quantize_mxfp4")
    return q, sc


def _mxfp4_shapes(x, w13_q, w13_s, w2_q, w2_s, act):
    """Codes and scales as moe_quantize_mxfp4 lays them out; returns (E, inter)."""
    if x.dtype != torch.bfloat16:
        raise TypeError("MXFP4 weights run a bf16 layer")
    for t in (w13_q, w13_s, w2_q, w2_s):
        if t.dtype != torch.uint8 or t.dim() != 3:
            raise TypeError("MXFP4 codes and scales are 3-D uint8 tensors")
    n, h = x.shape
    e, hh, half_i = w2_q.shape
    inter = 2 * half_i
    rows = inter if act == "relu2" else 2 * inter
    want = {"w13_q": (e, rows, h // 2), "w13_s": (e, h // 32, rows),
            "w2_q": (e, h, inter // 2), "w2_s": (e, inter // 32, h)}
    got = {"w13_q": w13_q, "w13_s": w13_s, "w2_q": w2_q, "w2_s": w2_s}
    if hh != h or h % 32 or inter % 32:
        raise ValueError("hidden and inter must be multiples of 32 and match x")
    for k, shp in want.items():
        if tuple(got[k].shape) != shp:
            raise ValueError(f"{k} must be {shp}, got {tuple(got[k].shape)}")
    return e, inter


def prepare_experts_mxfp4(x, w13_q, w13_s, w2_q, w2_s, routing: Routing, act: str,
                          layout: str = "packed", params: Optional[dict] = None, *, out=None,
                          workspace=None, stream=None) -> Prepared:
    dev = _dev(x, w13_q, w13_s, w2_q, w2_s)
    if act not in ACTS:
        raise ValueError(f"unknown activation {act!r}")
    e, inter = _mxfp4_shapes(x, w13_q, w13_s, w2_q, w2_s, act)
    n, hidden = x.shape
    k = routing.topk
    _check_routing(routing, n, e, k)
    if out is None:
        out = torch.empty_like(x)
    ws = _workspace(workspace, moe_workspace_bytes(n, max(e, k), k, hidden, inter, x.dtype), dev)
    r = routing.as_c()
    p = _params(params)
    args = (x.data_ptr(), _dt(x), n, hidden, w13_q.data_ptr(), w13_s.data_ptr(), w2_q.data_ptr(),
            w2_s.data_ptr(), e, inter, k, ACTS[act], LAYOUTS[layout],
            ctypes.byref(p) if p else None, ctypes.byref(r), out.data_ptr(), ws.data_ptr(),
            _nbytes(ws), _stream(dev, stream))
    return Prepared("moe_experts_mxfp4", args,
                    (r, p, x, w13_q, w13_s, w2_q, w2_s, out, ws, routing), out)


def moe_experts_mxfp4(x: torch.Tensor, w13_q: torch.Tensor, w13_s: torch.Tensor,
                      w2_q: torch.Tensor, w2_s: torch.Tensor, routing: Routing, act: str,
                      layout: str = "packed", params: Optional[dict] = None, *,
                      out: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """moe_experts with MXFP4 expert weights (codes and scales from
    moe_quantize_mxfp4); bf16 layer (see moe.h)."""
    return prepare_experts_mxfp4(x, w13_q, w13_s, w2_q, w2_s, routing, act, layout, params,
                                 out=out, workspace=workspace, stream=stream)()


def prepare_forward_mxfp4(x, logits, w13_q, w13_s, w2_q, w2_s, topk: int, act: str,
                          layout: str = "packed", params: Optional[dict] = None, *, out=None,
                          routing=None, workspace=None, stream=None) -> Prepared:
    dev = _dev(x, logits, w13_q, w13_s, w2_q, w2_s)
    if act not in ACTS:
        raise ValueError(f"unknown activation {act!r}")
    e, inter = _mxfp4_shapes(x, w13_q, w13_s, w2_q, w2_s, act)
    n, hidden = x.shape
    if logits.dtype != x.dtype or tuple(logits.shape) != (n, e):
        raise ValueError("logits must be [N, E] in the layer dtype")
    if routing is None:
        routing = Routing.empty(n, e, topk, x.dtype, dev)
    _check_routing(routing, n, e, topk, fills=e)
    if out is None:
        out = torch.empty_like(x)
    ws = _workspace(workspace, moe_workspace_bytes(n, e, topk, hidden, inter, x.dtype), dev)
    r = routing.as_c()
    p = _params(params)
    args = (x.data_ptr(), logits.data_ptr(), _dt(x), n, hidden, w13_q.data_ptr(),
            w13_s.data_ptr(), w2_q.data_ptr(), w2_s.data_ptr(), e, inter, topk, ACTS[act],
            LAYOUTS[layout], ctypes.byref(p) if p else None, ctypes.byref(r), out.data_ptr(),
            ws.data_ptr(), _nbytes(ws), _stream(dev, stream))
    return Prepared("moe_forward_mxfp4", args,
                    (r, p, x, logits, w13_q, w13_s, w2_q, w2_s, out, ws, routing),
                    (out, routing))


def moe_forward_mxfp4(x: torch.Tensor, logits: torch.Tensor, w13_q: torch.Tensor,
                      w13_s: torch.Tensor, w2_q: torch.Tensor, w2_s: torch.Tensor, topk: int,
                      act: str, layout: str = "packed", params: Optional[dict] = None, *,
                      out: Optional[torch.Tensor] = None, routing: Optional[Routing] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None):
    """Routing then the MXFP4-weight experts on one stream; returns ``(out, routing)``."""
    return prepare_forward_mxfp4(x, logits, w13_q, w13_s, w2_q, w2_s, topk, act, layout, params,
                                 out=out, routing=routing, workspace=workspace, stream=stream)()


# ------------------------------------------------- rows into sorted order and back
#
# The calls below marshal their arguments once for both forms: moe_X runs them
# right away, prepare_X keeps them in a Prepared.  A decoding step is a chain of
# kernels of a few microseconds, so what moe_X does on the host is kept short:
# raw device indexes and stream handles instead of torch's objects for them.

class _Call:
    """One checked C call: its device, name, arguments, and what they refer to."""

    __slots__ = ("dev", "name", "args", "keep", "result")

    def __init__(self, dev: int, name: str, args: tuple, keep: tuple, result):
        self.dev, self.name, self.args, self.keep, self.result = dev, name, args, keep, result

    def run(self):
        fn = getattr(N.load(), self.name)
        if torch._C._cuda_getDevice() == self.dev:
            st = fn(*self.args)
        else:
            with torch.cuda.device(self.dev):
                st = fn(*self.args)
        if st != N.MOE_OK:
            raise MoeError(st, self.name)
        return self.result

    def prepared(self) -> Prepared:
        return _DevicePrepared(self.dev, self.name, self.args, self.keep, self.result)


class _DevicePrepared(Prepared):
    """A Prepared whose launches go to the device of its tensors, whichever
    device is current when it is called."""

    def __init__(self, dev: int, name: str, args: tuple, keep: tuple, result):
        super().__init__(name, args, keep, result)
        self._dev = dev

    def __call__(self):
        if torch.cuda.current_device() == self._dev:
            return super().__call__()
        with torch.cuda.device(self._dev):
            return super().__call__()


def _index(*ts: torch.Tensor) -> int:
    """Device index of tensors that must be contiguous on one GPU."""
    dev = ts[0].get_device()
    for t in ts:
        if t.get_device() != dev or not t.is_contiguous():
            break
    else:
        if dev >= 0:
            return dev
    if any(t.get_device() != dev for t in ts) or dev < 0:
        raise ValueError("all tensors must be on the same GPU")
    raise ValueError("tensors must be contiguous")


def _raw_stream(dev: int, stream) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _like(t: torch.Tensor, stream) -> torch.Tensor:
    """New memory like ``t`` that belongs to the stream the call runs on."""
    if stream is None:
        return torch.empty_like(t)
    with torch.cuda.stream(stream):
        return torch.empty_like(t)


def _new(like: torch.Tensor, shape, dtype, stream) -> torch.Tensor:
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _is(t: torch.Tensor, shape, dtype, dev: int, name: str):
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {tuple(shape)} {dtype} on GPU {dev}, got "
                         f"{tuple(t.shape)} {t.dtype} on {t.device}")


def _output(t, like: torch.Tensor, shape, dtype, stream, name: str) -> torch.Tensor:
    """The caller's output tensor, checked, or new memory."""
    if t is None:
        return _new(like, shape, dtype, stream)
    _is(t, shape, dtype, like.get_device(), name)
    return t


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _scratch(ws, like: torch.Tensor, nbytes: int, stream) -> torch.Tensor:
    if ws is None:
        return _new(like, nbytes, torch.uint8, stream)
    _index(like, ws)
    return _workspace(ws, nbytes, None)


def _new_routing(n: int, e: int, topk: int, like: torch.Tensor, stream) -> Routing:
    if stream is None:
        return Routing.empty(n, e, topk, like.dtype, like.device)
    with torch.cuda.stream(stream):
        return Routing.empty(n, e, topk, like.dtype, like.device)


def _row_routing(routing: Routing, dev: int, order: torch.Tensor, name: str, weights: bool):
    """Checks the routing fields a row call reads (`order`: row_sorted or
    topk_idx); returns (N, k, topk_w's pointer or None, its dtype)."""
    n, k = routing.topk_idx.shape
    if order.numel() != n * k or order.get_device() != dev or not order.is_contiguous():
        raise ValueError(f"routing.{name} must be contiguous with N*k = {n * k} entries on the "
                         f"GPU of the rows")
    if order.dtype is not torch.int32:
        raise TypeError(f"routing.{name} must be int32")
    if not weights:
        return n, k, None, 0
    w = routing.topk_w
    if w.shape != (n, k) or w.get_device() != dev or not w.is_contiguous():
        raise ValueError("routing.topk_w must be contiguous [N, k] on the GPU of the rows")
    return n, k, w.data_ptr(), _dt(w)


def _dispatch(x, routing, x_sorted, stream) -> _Call:
    dev, order = _index(x), routing.row_sorted
    n, k, _, _ = _row_routing(routing, dev, order, "row_sorted", False)
    if x.dim() != 2 or x.shape[0] != n:
        raise ValueError("x must be [N, hidden] with the routing's N")
    hidden = x.shape[1]
    x_sorted = _output(x_sorted, x, (n * k, hidden), x.dtype, stream, "x_sorted")
    r = N.MoeRouting(row_sorted=order.data_ptr())
    args = (x.data_ptr(), _dt(x), n, hidden, k, ctypes.byref(r), x_sorted.data_ptr(),
            _raw_stream(dev, stream))
    return _Call(dev, "moe_dispatch", args, (r, x, x_sorted, routing), x_sorted)


def prepare_dispatch(x: torch.Tensor, routing: Routing, *,
                     x_sorted: Optional[torch.Tensor] = None, stream=None) -> Prepared:
    return _dispatch(x, routing, x_sorted, stream).prepared()


def moe_dispatch(x: torch.Tensor, routing: Routing, *, x_sorted: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """Token rows into expert-sorted order: ``x_sorted[row_sorted[t*k + j]] = x[t]``
    (``[N*k, hidden]``; rows that no slot points to are left as they were).  The
    gradient with respect to ``x`` is ``moe_combine(d_x_sorted, routing)``."""
    return _dispatch(x, routing, x_sorted, stream).run()


def _combine_weighted(y_sorted, routing, out, stream) -> _Call:
    dev, order = _index(y_sorted), routing.row_sorted
    n, k, w, wdt = _row_routing(routing, dev, order, "row_sorted", True)
    if y_sorted.dim() != 2 or y_sorted.shape[0] != n * k:
        raise ValueError("y_sorted must be [N*k, hidden]")
    hidden = y_sorted.shape[1]
    out = _output(out, y_sorted, (n, hidden), y_sorted.dtype, stream, "out")
    r = N.MoeRouting(topk_w=w, row_sorted=order.data_ptr(), w_dtype=wdt)
    args = (y_sorted.data_ptr(), _dt(y_sorted), n, hidden, k, ctypes.byref(r), out.data_ptr(),
            _raw_stream(dev, stream))
    return _Call(dev, "moe_combine_weighted", args, (r, y_sorted, out, routing), out)


def prepare_combine_weighted(y_sorted: torch.Tensor, routing: Routing, *,
                             out: Optional[torch.Tensor] = None, stream=None) -> Prepared:
    return _combine_weighted(y_sorted, routing, out, stream).prepared()


def moe_combine_weighted(y_sorted: torch.Tensor, routing: Routing, *,
                         out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Expert rows back into token order with the routing weights applied:
    ``out[t] = sum_j topk_w[t, j] * y_sorted[row_sorted[t*k + j]]`` (slot order,
    fp32 sum, one rounding; slots with row_sorted = -1 skipped)."""
    return _combine_weighted(y_sorted, routing, out, stream).run()


def _combine_weighted_backward(d_out, y_sorted, routing, d_y_sorted, d_topk_w, stream) -> _Call:
    dev, order = _index(d_out, y_sorted), routing.row_sorted
    n, k, w, wdt = _row_routing(routing, dev, order, "row_sorted", True)
    if y_sorted.dim() != 2 or y_sorted.shape[0] != n * k:
        raise ValueError("y_sorted must be [N*k, hidden]")
    hidden = y_sorted.shape[1]
    if tuple(d_out.shape) != (n, hidden) or d_out.dtype != y_sorted.dtype:
        raise ValueError("d_out must be [N, hidden] in the dtype of y_sorted")
    if d_y_sorted is None:
        d_y_sorted = _like(y_sorted, stream)
    else:
        _is(d_y_sorted, (n * k, hidden), y_sorted.dtype, dev, "d_y_sorted")
    d_topk_w = _output(d_topk_w, y_sorted, (n, k), torch.float32, stream, "d_topk_w")
    r = N.MoeRouting(topk_w=w, row_sorted=order.data_ptr(), w_dtype=wdt)
    args = (d_out.data_ptr(), y_sorted.data_ptr(), _dt(y_sorted), n, hidden, k, ctypes.byref(r),
            d_y_sorted.data_ptr(), d_topk_w.data_ptr(), _raw_stream(dev, stream))
    return _Call(dev, "moe_combine_weighted_backward", args,
                 (r, d_out, y_sorted, d_y_sorted, d_topk_w, routing), (d_y_sorted, d_topk_w))


def prepare_combine_weighted_backward(d_out: torch.Tensor, y_sorted: torch.Tensor,
                                      routing: Routing, *,
                                      d_y_sorted: Optional[torch.Tensor] = None,
                                      d_topk_w: Optional[torch.Tensor] = None,
                                      stream=None) -> Prepared:
    return _combine_weighted_backward(d_out, y_sorted, routing, d_y_sorted, d_topk_w,
                                      stream).prepared()


def moe_combine_weighted_backward(d_out: torch.Tensor, y_sorted: torch.Tensor, routing: Routing,
                                  *, d_y_sorted: Optional[torch.Tensor] = None,
                                  d_topk_w: Optional[torch.Tensor] = None, stream=None):
    """Gradient of moe_combine_weighted: returns ``(d_y_sorted [N*k, hidden],
    d_topk_w [N, k] fp32)``; rows that no slot points to are left as they were and
    skipped slots get a zero weight gradient (see moe.h)."""
    return _combine_weighted_backward(d_out, y_sorted, routing, d_y_sorted, d_topk_w,
                                      stream).run()


def _route_backward(d_topk_w, routing, n_experts, d_logits, stream) -> _Call:
    dev, order = _index(d_topk_w), routing.topk_idx
    n, k, w, wdt = _row_routing(routing, dev, order, "topk_idx", True)
    if tuple(d_topk_w.shape) != (n, k) or d_topk_w.dtype != torch.float32:
        raise ValueError("d_topk_w must be fp32 [N, k]")
    layer = routing.layer_experts
    e = n_experts if n_experts is not None else routing.n_experts if layer is None else layer
    if layer is not None and e != layer:
        raise ValueError(f"the routing is a share's of a layer of {layer} experts, not {e}")
    d_logits = _output(d_logits, d_topk_w, (n, e), routing.topk_w.dtype, stream, "d_logits")
    r = N.MoeRouting(topk_idx=order.data_ptr(), topk_w=w, w_dtype=wdt)
    args = (d_topk_w.data_ptr(), n, e, k, ctypes.byref(r), d_logits.data_ptr(),
            _raw_stream(dev, stream))
    return _Call(dev, "moe_route_backward", args, (r, d_topk_w, d_logits, routing), d_logits)


def prepare_route_backward(d_topk_w: torch.Tensor, routing: Routing,
                           n_experts: Optional[int] = None, *,
                           d_logits: Optional[torch.Tensor] = None, stream=None) -> Prepared:
    return _route_backward(d_topk_w, routing, n_experts, d_logits, stream).prepared()


def moe_route_backward(d_topk_w: torch.Tensor, routing: Routing,
                       n_experts: Optional[int] = None, *,
                       d_logits: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of the routing weights with respect to the router logits
    ``[N, E]`` (zeros for experts that were not selected).  ``n_experts``: the
    layer's expert count, by default the routing's own (that of the whole layer also
    where moe_route_ep or moe_forward_ep filled it for a share)."""
    return _route_backward(d_topk_w, routing, n_experts, d_logits, stream).run()


# ------------------------------------------------- norms around a block

@dataclass
class BlockNorm:
    """Outputs of moe_block_norm; None for what the call does not have."""

    x_out: Optional[torch.Tensor]      # [N, H]
    n_out: Optional[torch.Tensor]      # [N, H]
    rstd_post: Optional[torch.Tensor]  # [N] fp32
    rstd_pre: Optional[torch.Tensor]   # [N] fp32


@dataclass
class BlockNormGrads:
    """Outputs of moe_block_norm_backward; None for what the call does not have."""

    d_x: torch.Tensor                  # [N, H]
    d_y: Optional[torch.Tensor]        # [N, H]
    d_w_post: Optional[torch.Tensor]   # [H] fp32
    d_w_pre: Optional[torch.Tensor]    # [H] fp32
    d_gate: Optional[torch.Tensor]     # fp32 in the shape of the gate


def moe_block_norm_workspace_bytes(n_tokens: int, hidden: int,
                                   dtype: torch.dtype = torch.bfloat16) -> int:
    b = N.load().moe_block_norm_workspace_bytes(n_tokens, hidden, _DT[dtype])
    if b == 0:
        raise MoeError(N.MOE_ERR_SHAPE, "moe_block_norm_workspace_bytes")
    return b


def _block_norm_args(x, y, w_post, w_pre, gate, residual_scale, eps):
    """Checks what both directions take; returns (device, n, hidden, C struct)."""
    here = [t for t in (x, y, w_post, w_pre, gate) if t is not None]
    dev, dtype = _index(*here), x.dtype
    if x.dim() != 2:
        raise ValueError("x must be [N, hidden]")
    for t in here:
        if t.dtype is not dtype:
            raise TypeError("x, y, the weights and the gate must share a dtype")
    n, hidden = shape = x.shape
    if y is not None:
        if y.shape != shape:
            raise ValueError("y must have the shape of x")
    elif w_post is not None or gate is not None:
        raise ValueError("w_post and gate need the block's output y")
    elif w_pre is None:
        raise ValueError("nothing to do without y and w_pre")
    post = pre = gp = None
    kind = N.MOE_GATE_NONE
    if w_post is not None:
        if w_post.shape != (hidden,):
            raise ValueError("w_post must be [hidden]")
        post = w_post.data_ptr()
    if w_pre is not None:
        if w_pre.shape != (hidden,):
            raise ValueError("w_pre must be [hidden]")
        pre = w_pre.data_ptr()
    if gate is not None:
        if gate.shape == (n, 1):
            kind = N.MOE_GATE_TOKEN
        elif gate.shape == (hidden,):
            kind = N.MOE_GATE_CHANNEL
        else:
            raise ValueError("gate must be [N, 1] (a value per token) or [hidden] (per channel)")
        gp = gate.data_ptr()
    return dev, n, hidden, N.MoeBlockNorm(post, pre, gp, kind, residual_scale, eps)


def _block_norm(x, y, w_post, w_pre, gate, residual_scale, eps, x_out, n_out, rstd_post, rstd_pre,
                stream) -> _Call:
    dev, n, hidden, c = _block_norm_args(x, y, w_post, w_pre, gate, residual_scale, eps)
    f32, xo, no, rpost, rpre = torch.float32, None, None, None, None
    if y is not None:
        if x_out is None:
            x_out = _like(x, stream)
        else:
            _is(x_out, x.shape, x.dtype, dev, "x_out")
        xo = x_out.data_ptr()
    elif x_out is not None:
        raise ValueError("the call has no x_out")
    if w_pre is not None:
        if n_out is None:
            n_out = _like(x, stream)
        else:
            _is(n_out, x.shape, x.dtype, dev, "n_out")
        no = n_out.data_ptr()
        rstd_pre = _output(rstd_pre, x, (n,), f32, stream, "rstd_pre")
        rpre = rstd_pre.data_ptr()
    elif n_out is not None or rstd_pre is not None:
        raise ValueError("the call has no n_out and rstd_pre")
    if w_post is not None:
        rstd_post = _output(rstd_post, x, (n,), f32, stream, "rstd_post")
        rpost = rstd_post.data_ptr()
    elif rstd_post is not None:
        raise ValueError("the call has no rstd_post")
    args = (x.data_ptr(), _ptr(y), _dt(x), n, hidden, ctypes.byref(c), xo, no, rpost, rpre,
            _raw_stream(dev, stream))
    res = BlockNorm(x_out, n_out, rstd_post, rstd_pre)
    return _Call(dev, "moe_block_norm", args, (c, x, y, w_post, w_pre, gate, res), res)


def prepare_block_norm(x: torch.Tensor, y: Optional[torch.Tensor] = None, *,
                       w_post: Optional[torch.Tensor] = None,
                       w_pre: Optional[torch.Tensor] = None,
                       gate: Optional[torch.Tensor] = None, residual_scale: float = 1.0,
                       eps: float = 1e-6, x_out: Optional[torch.Tensor] = None,
                       n_out: Optional[torch.Tensor] = None,
                       rstd_post: Optional[torch.Tensor] = None,
                       rstd_pre: Optional[torch.Tensor] = None, stream=None) -> Prepared:
    return _block_norm(x, y, w_post, w_pre, gate, residual_scale, eps, x_out, n_out, rstd_post,
                       rstd_pre, stream).prepared()


def moe_block_norm(x: torch.Tensor, y: Optional[torch.Tensor] = None, *,
                   w_post: Optional[torch.Tensor] = None, w_pre: Optional[torch.Tensor] = None,
                   gate: Optional[torch.Tensor] = None, residual_scale: float = 1.0,
                   eps: float = 1e-6, x_out: Optional[torch.Tensor] = None,
                   n_out: Optional[torch.Tensor] = None,
                   rstd_post: Optional[torch.Tensor] = None,
                   rstd_pre: Optional[torch.Tensor] = None, stream=None) -> BlockNorm:
    """Norms around a block in one pass: ``x_out = x + residual_scale * gate *
    rmsnorm(y, w_post)`` and ``n_out = rmsnorm(x_out, w_pre)``, the input of the
    next block.  Without ``y`` it is the norm ahead of a block alone, without
    ``w_pre`` the step after a block alone, without ``w_post`` the block's output
    enters unnormed.  ``gate``: ``[N, 1]`` (a value per token) or ``[hidden]``
    (per channel).  ``x_out`` may be ``x`` (see moe.h)."""
    return _block_norm(x, y, w_post, w_pre, gate, residual_scale, eps, x_out, n_out, rstd_post,
                       rstd_pre, stream).run()


def _block_norm_backward(d_x_out, d_n_out, x, y, w_post, w_pre, gate, residual_scale, rstd_post,
                         rstd_pre, d_x, d_y, d_w_post, d_w_pre, d_gate, workspace,
                         stream) -> _Call:
    # the gradient takes the saved rstds, so eps no longer matters
    dev, n, hidden, c = _block_norm_args(x, y, w_post, w_pre, gate, residual_scale, 1.0)
    dtype, f32, rows, token, width = x.dtype, torch.float32, x.shape, (n,), (hidden,)
    ins = [None] * 4   # d_x_out, d_n_out, rstd_post, rstd_pre
    outs = [None] * 4  # d_y, d_w_post, d_w_pre, d_gate
    if d_x_out is not None:
        _is(d_x_out, rows, dtype, dev, "d_x_out")
        ins[0] = d_x_out.data_ptr()
    elif w_pre is None:
        raise ValueError("no gradient flows in: d_x_out or w_pre with d_n_out is needed")
    if w_pre is not None:
        if d_n_out is None or rstd_pre is None:
            raise ValueError("d_n_out and the forward call's rstd_pre go with w_pre")
        _is(d_n_out, rows, dtype, dev, "d_n_out")
        _is(rstd_pre, token, f32, dev, "rstd_pre")
        ins[1], ins[3] = d_n_out.data_ptr(), rstd_pre.data_ptr()
        d_w_pre = _output(d_w_pre, x, width, f32, stream, "d_w_pre")
        outs[2] = d_w_pre.data_ptr()
    elif d_n_out is not None or d_w_pre is not None:
        raise ValueError("d_n_out and d_w_pre go with w_pre")
    if w_post is not None:
        if rstd_post is None:
            raise ValueError("the forward call's rstd_post goes with w_post")
        _is(rstd_post, token, f32, dev, "rstd_post")
        ins[2] = rstd_post.data_ptr()
        d_w_post = _output(d_w_post, x, width, f32, stream, "d_w_post")
        outs[1] = d_w_post.data_ptr()
    elif d_w_post is not None:
        raise ValueError("d_w_post goes with w_post")
    if gate is not None:
        d_gate = _output(d_gate, x, gate.shape, f32, stream, "d_gate")
        outs[3] = d_gate.data_ptr()
    elif d_gate is not None:
        raise ValueError("d_gate goes with gate")
    if d_x is None:
        d_x = _like(x, stream)
    else:
        _is(d_x, rows, dtype, dev, "d_x")
    if y is not None:
        if d_y is None:
            d_y = _like(x, stream)
        else:
            _is(d_y, rows, dtype, dev, "d_y")
        outs[0] = d_y.data_ptr()
    elif d_y is not None:
        raise ValueError("d_y goes with y")
    dt = _dt(x)
    need = N.load().moe_block_norm_workspace_bytes(n, hidden, dt)
    if need == 0:
        raise MoeError(N.MOE_ERR_SHAPE, "moe_block_norm_backward")
    ws = _scratch(workspace, x, need, stream)
    args = (ins[0], ins[1], x.data_ptr(), _ptr(y), dt, n, hidden, ctypes.byref(c), ins[2], ins[3],
            d_x.data_ptr(), *outs, ws.data_ptr(), _nbytes(ws), _raw_stream(dev, stream))
    res = BlockNormGrads(d_x, d_y, d_w_post, d_w_pre, d_gate)
    return _Call(dev, "moe_block_norm_backward", args,
                 (c, d_x_out, d_n_out, x, y, w_post, w_pre, gate, rstd_post, rstd_pre, res, ws),
                 res)


def prepare_block_norm_backward(d_x_out: Optional[torch.Tensor], d_n_out: Optional[torch.Tensor],
                                x: torch.Tensor, y: Optional[torch.Tensor] = None, *,
                                w_post: Optional[torch.Tensor] = None,
                                w_pre: Optional[torch.Tensor] = None,
                                gate: Optional[torch.Tensor] = None,
                                residual_scale: float = 1.0,
                                rstd_post: Optional[torch.Tensor] = None,
                                rstd_pre: Optional[torch.Tensor] = None,
                                d_x: Optional[torch.Tensor] = None,
                                d_y: Optional[torch.Tensor] = None,
                                d_w_post: Optional[torch.Tensor] = None,
                                d_w_pre: Optional[torch.Tensor] = None,
                                d_gate: Optional[torch.Tensor] = None,
                                workspace: Optional[torch.Tensor] = None,
                                stream=None) -> Prepared:
    return _block_norm_backward(d_x_out, d_n_out, x, y, w_post, w_pre, gate, residual_scale,
                                rstd_post, rstd_pre, d_x, d_y, d_w_post, d_w_pre, d_gate,
                                workspace, stream).prepared()


def moe_block_norm_backward(d_x_out: Optional[torch.Tensor], d_n_out: Optional[torch.Tensor],
                            x: torch.Tensor, y: Optional[torch.Tensor] = None, *,
                            w_post: Optional[torch.Tensor] = None,
                            w_pre: Optional[torch.Tensor] = None,
                            gate: Optional[torch.Tensor] = None, residual_scale: float = 1.0,
                            rstd_post: Optional[torch.Tensor] = None,
                            rstd_pre: Optional[torch.Tensor] = None,
                            d_x: Optional[torch.Tensor] = None,
                            d_y: Optional[torch.Tensor] = None,
                            d_w_post: Optional[torch.Tensor] = None,
                            d_w_pre: Optional[torch.Tensor] = None,
                            d_gate: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None,
                            stream=None) -> BlockNormGrads:
    """Gradient of moe_block_norm from the gradients of ``x_out`` (None: zero) and
    ``n_out`` (with ``w_pre``), the forward call's arguments and its rstds.  The
    gradients of the weights and the gate are fp32 (see moe.h)."""
    return _block_norm_backward(d_x_out, d_n_out, x, y, w_post, w_pre, gate, residual_scale,
                                rstd_post, rstd_pre, d_x, d_y, d_w_post, d_w_pre, d_gate,
                                workspace, stream).run()


def _block_forward(x, w_gate, w13, w2, topk, act, layout, params, w_pre, w_post, gate,
                   residual_scale, eps, x_out, logits, routing, workspace, stream) -> _Call:
    if w_pre is None:
        raise ValueError("w_pre, the weight of the norm ahead of the block, is needed")
    # (x stands for the block's output, which has its shape)
    dev, n, hidden, c = _block_norm_args(x, x, w_post, w_pre, gate, residual_scale, eps)
    _index(x, w_gate, w13, w2)
    if w_gate.dim() != 2 or w_gate.shape[1] != hidden or w_gate.dtype != x.dtype:
        raise ValueError("w_gate must be [E, hidden] in the dtype of x")
    _shapes(x, w13, w2, act)
    e, inter = w2.shape[0], w2.shape[2]
    if w_gate.shape[0] != e:
        raise ValueError("w_gate and the experts differ in their number")
    if layout not in LAYOUTS:
        raise ValueError(f"unknown w13 layout {layout!r}")
    x_out = _output(x_out, x, (n, hidden), x.dtype, stream, "x_out")
    logits = _output(logits, x, (n, e), x.dtype, stream, "logits")
    if routing is None:
        routing = _new_routing(n, e, topk, x, stream)
    _check_routing(routing, n, e, topk, fills=e)
    _index(x, *routing.tensors())
    need = (moe_workspace_bytes(n, e, topk, hidden, inter, x.dtype) + 255) // 256 * 256 \
        + (n * hidden * x.element_size() + 255) // 256 * 256
    ws = _scratch(workspace, x, need, stream)
    r = routing.as_c()
    p = _params(params)
    args = (x.data_ptr(), w_gate.data_ptr(), _dt(x), n, hidden, w13.data_ptr(), w2.data_ptr(), e,
            inter, topk, ACTS[act], LAYOUTS[layout], ctypes.byref(p) if p else None,
            ctypes.byref(c), logits.data_ptr(), ctypes.byref(r), x_out.data_ptr(), ws.data_ptr(),
            _nbytes(ws), _raw_stream(dev, stream))
    return _Call(dev, "moe_block_forward", args,
                 (r, p, c, x, w_gate, w13, w2, w_pre, w_post, gate, x_out, logits, ws, routing),
                 (x_out, logits, routing))


def prepare_block_forward(x: torch.Tensor, w_gate: torch.Tensor, w13: torch.Tensor,
                          w2: torch.Tensor, topk: int, act: str, layout: str = "packed",
                          params: Optional[dict] = None, *, w_pre: torch.Tensor,
                          w_post: Optional[torch.Tensor] = None,
                          gate: Optional[torch.Tensor] = None, residual_scale: float = 1.0,
                          eps: float = 1e-6, x_out: Optional[torch.Tensor] = None,
                          logits: Optional[torch.Tensor] = None,
                          routing: Optional[Routing] = None,
                          workspace: Optional[torch.Tensor] = None, stream=None) -> Prepared:
    return _block_forward(x, w_gate, w13, w2, topk, act, layout, params, w_pre, w_post, gate,
                          residual_scale, eps, x_out, logits, routing, workspace,
                          stream).prepared()


def moe_block_forward(x: torch.Tensor, w_gate: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor,
                      topk: int, act: str, layout: str = "packed", params: Optional[dict] = None,
                      *, w_pre: torch.Tensor, w_post: Optional[torch.Tensor] = None,
                      gate: Optional[torch.Tensor] = None, residual_scale: float = 1.0,
                      eps: float = 1e-6, x_out: Optional[torch.Tensor] = None,
                      logits: Optional[torch.Tensor] = None, routing: Optional[Routing] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None):
    """The block around the layer: norm, moe_gate_forward, norm, gate and residual
    sum (see moe.h); returns ``(x_out, logits, routing)``.  ``x_out`` may be ``x``."""
    return _block_forward(x, w_gate, w13, w2, topk, act, layout, params, w_pre, w_post, gate,
                          residual_scale, eps, x_out, logits, routing, workspace, stream).run()


# ------------------------------------------------- 4-bit expert weights with group scales

_INT4_GROUPS = (32, 64, 128)


def moe_quantize_int4(w: torch.Tensor, group: int = 128, *, zeros: bool = True, stream=None):
    """4-bit weights from ``w [E, rows, K]`` (K a multiple of ``group``, 32, 64 or
    128): returns ``(q [E, rows, K/2] uint8, scales [E, K/group, rows] bf16,
    zeros [E, K/group, rows] uint8)``; the last is None without ``zeros``
    (symmetric codes, see moe.h)."""
    dev = _index(w)
    if w.dim() != 3:
        raise ValueError("expected w [E, rows, K]")
    e, rows, k = w.shape
    if group not in _INT4_GROUPS or k % group:
        raise ValueError("group must be 32, 64 or 128 and divide K")
    q = _output(None, w, (e, rows, k // 2), torch.uint8, stream, "q")
    s = _output(None, w, (e, k // group, rows), torch.bfloat16, stream, "scales")
    z = _output(None, w, (e, k // group, rows), torch.uint8, stream, "zeros") if zeros else None
    args = (w.data_ptr(), _dt(w), e, rows, k, group, q.data_ptr(), s.data_ptr(), _ptr(z),
            _raw_stream(dev, stream))
    return _Call(dev, "moe_quantize_int4", args, (w,), (q, s, z)).run()


def _int4_weights(q, s, z, name: str):
    """Checks one weight array; returns (E, rows, K, group, the C struct)."""
    if q.dtype is not torch.uint8 or s.dtype is not torch.bfloat16 or q.dim() != 3 or s.dim() != 3:
        raise TypeError(f"{name}: expected uint8 codes [E, rows, K/2] and bf16 scales "
                        f"[E, K/group, rows]")
    e, rows, half = q.shape
    es, ng, rs = s.shape
    k = 2 * half
    group = k // ng if ng else 0
    if group not in _INT4_GROUPS or k != ng * group or es != e or rs != rows:
        raise ValueError(f"{name}: scales {tuple(s.shape)} do not give groups of 32, 64 or 128 "
                         f"of codes {tuple(q.shape)}")
    if z is None:
        return e, rows, k, group, N.MoeInt4Weights(q.data_ptr(), s.data_ptr(), None)
    if z.dtype is not torch.uint8 or z.shape != s.shape:
        raise ValueError(f"{name}: zeros must be uint8 in the shape of the scales")
    return e, rows, k, group, N.MoeInt4Weights(q.data_ptr(), s.data_ptr(), z.data_ptr())


def moe_dequantize_int4(q: torch.Tensor, scales: torch.Tensor,
                        zeros: Optional[torch.Tensor] = None, *,
                        out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """bf16 weights ``[E, rows, K]`` of 4-bit codes, scales and zero points."""
    dev = _index(q, scales) if zeros is None else _index(q, scales, zeros)
    e, rows, k, group, c = _int4_weights(q, scales, zeros, "w")
    out = _output(out, q, (e, rows, k), torch.bfloat16, stream, "out")
    args = (ctypes.byref(c), e, rows, k, group, out.data_ptr(), _raw_stream(dev, stream))
    return _Call(dev, "moe_dequantize_int4", args, (c, q, scales, zeros), out).run()


def moe_int4_workspace_bytes(n_tokens: int, n_experts: int, topk: int, hidden: int,
                             inter: int) -> int:
    b = N.load().moe_int4_workspace_bytes(n_tokens, n_experts, topk, hidden, inter)
    if b == 0:
        raise MoeError(N.MOE_ERR_SHAPE, "moe_int4_workspace_bytes")
    return b


def _int4_layer(x, w13, w2, act, layout):
    """Checks the layer; returns (device, n, hidden, E, inter, group, structs)."""
    dev = _index(x, *[t for t in (*w13, *w2) if t is not None])
    if act not in ACTS:
        raise ValueError(f"unknown activation {act!r}")
    if layout not in LAYOUTS:
        raise ValueError(f"unknown w13 layout {layout!r}")
    if x.dim() != 2 or x.dtype != torch.bfloat16:
        raise TypeError("4-bit weights run a bf16 layer: x must be bf16 [N, hidden]")
    n, hidden = x.shape
    e, rows, k, group, c13 = _int4_weights(*w13, "w13")
    e2, h2, inter, group2, c2 = _int4_weights(*w2, "w2")
    if k != hidden or h2 != hidden or e2 != e or rows != (inter if act == "relu2" else 2 * inter):
        raise ValueError(f"w13 [{e}, {rows}, {k}] / w2 [{e2}, {h2}, {inter}] do not match "
                         f"x {tuple(x.shape)} and act {act!r}")
    if group != group2:
        raise ValueError(f"w13 and w2 must share a group size, got {group} and {group2}")
    return dev, n, hidden, e, inter, group, c13, c2


def _experts_int4(x, w13, w2, routing, act, layout, params, out, workspace, stream) -> _Call:
    if routing.layer_experts is not None:
        raise ValueError("moe_experts_int4 takes the whole layer's routing, not an expert share's "
                         "(moe_route_ep)")
    dev, n, hidden, e, inter, group, c13, c2 = _int4_layer(x, w13, w2, act, layout)
    k = routing.topk
    off, col, row, scal = (routing.offsets, routing.col_sorted, routing.row_sorted,
                           routing.gate_scal)
    if _index(off, col, row, scal) != dev:
        raise ValueError("the routing must be on the GPU of x")
    if off.numel() != e + 1 or not col.numel() == row.numel() == scal.numel() == n * k:
        raise ValueError(f"the routing is not one of {n} tokens and {e} experts")
    if not off.dtype is col.dtype is row.dtype is torch.int32:
        raise TypeError("the routing's offsets, col_sorted and row_sorted must be int32")
    if out is None:
        out = _like(x, stream)
    else:
        _is(out, x.shape, x.dtype, dev, "out")
    ws = _scratch(workspace, x, moe_int4_workspace_bytes(n, e, k, hidden, inter), stream)
    r = N.MoeRouting(None, None, None, None, off.data_ptr(), col.data_ptr(), row.data_ptr(),
                     scal.data_ptr(), _dt(scal))
    p = _params(params)
    args = (x.data_ptr(), n, hidden, ctypes.byref(c13), ctypes.byref(c2), e, inter, k, group,
            ACTS[act], LAYOUTS[layout], ctypes.byref(p) if p else None, ctypes.byref(r),
            out.data_ptr(), ws.data_ptr(), _nbytes(ws), _raw_stream(dev, stream))
    return _Call(dev, "moe_experts_int4", args, (r, p, c13, c2, x, w13, w2, out, ws, routing), out)


def prepare_experts_int4(x: torch.Tensor, w13_q: torch.Tensor, w13_s: torch.Tensor,
                         w13_z: Optional[torch.Tensor], w2_q: torch.Tensor, w2_s: torch.Tensor,
                         w2_z: Optional[torch.Tensor], routing: Routing, act: str,
                         layout: str = "packed", params: Optional[dict] = None, *,
                         out: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None, stream=None) -> Prepared:
    return _experts_int4(x, (w13_q, w13_s, w13_z), (w2_q, w2_s, w2_z), routing, act, layout,
                         params, out, workspace, stream).prepared()


def moe_experts_int4(x: torch.Tensor, w13_q: torch.Tensor, w13_s: torch.Tensor,
                     w13_z: Optional[torch.Tensor], w2_q: torch.Tensor, w2_s: torch.Tensor,
                     w2_z: Optional[torch.Tensor], routing: Routing, act: str,
                     layout: str = "packed", params: Optional[dict] = None, *,
                     out: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """moe_experts with 4-bit expert weights (codes, scales and zero points as
    moe_quantize_int4 gives them, zeros None for symmetric codes); bf16 layer,
    shaped for decode-sized batches (see moe.h).  ``routing`` is the whole layer's:
    one of an expert share is refused."""
    return _experts_int4(x, (w13_q, w13_s, w13_z), (w2_q, w2_s, w2_z), routing, act, layout,
                         params, out, workspace, stream).run()


def _forward_int4(x, logits, w13, w2, topk, act, layout, params, out, routing, workspace,
                  stream) -> _Call:
    dev, n, hidden, e, inter, group, c13, c2 = _int4_layer(x, w13, w2, act, layout)
    _index(x, logits)
    if logits.dtype != x.dtype or tuple(logits.shape) != (n, e):
        raise ValueError("logits must be [N, E] in the layer dtype")
    if routing is None:
        routing = _new_routing(n, e, topk, x, stream)
    _check_routing(routing, n, e, topk, fills=e)
    _index(x, *routing.tensors())
    out = _output(out, x, (n, hidden), x.dtype, stream, "out")
    ws = _scratch(workspace, x, moe_int4_workspace_bytes(n, e, topk, hidden, inter), stream)
    r = routing.as_c()
    p = _params(params)
    args = (x.data_ptr(), logits.data_ptr(), n, hidden, ctypes.byref(c13), ctypes.byref(c2), e,
            inter, topk, group, ACTS[act], LAYOUTS[layout], ctypes.byref(p) if p else None,
            ctypes.byref(r), out.data_ptr(), ws.data_ptr(), _nbytes(ws), _raw_stream(dev, stream))
    return _Call(dev, "moe_forward_int4", args,
                 (r, p, c13, c2, x, logits, w13, w2, out, ws, routing), (out, routing))


def prepare_forward_int4(x: torch.Tensor, logits: torch.Tensor, w13_q: torch.Tensor,
                         w13_s: torch.Tensor, w13_z: Optional[torch.Tensor], w2_q: torch.Tensor,
                         w2_s: torch.Tensor, w2_z: Optional[torch.Tensor], topk: int, act: str,
                         layout: str = "packed", params: Optional[dict] = None, *,
                         out: Optional[torch.Tensor] = None, routing: Optional[Routing] = None,
                         workspace: Optional[torch.Tensor] = None, stream=None) -> Prepared:
    return _forward_int4(x, logits, (w13_q, w13_s, w13_z), (w2_q, w2_s, w2_z), topk, act, layout,
                         params, out, routing, workspace, stream).prepared()


def moe_forward_int4(x: torch.Tensor, logits: torch.Tensor, w13_q: torch.Tensor,
                     w13_s: torch.Tensor, w13_z: Optional[torch.Tensor], w2_q: torch.Tensor,
                     w2_s: torch.Tensor, w2_z: Optional[torch.Tensor], topk: int, act: str,
                     layout: str = "packed", params: Optional[dict] = None, *,
                     out: Optional[torch.Tensor] = None, routing: Optional[Routing] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None):
    """Routing then the 4-bit experts on one stream; returns ``(out, routing)``."""
    return _forward_int4(x, logits, (w13_q, w13_s, w13_z), (w2_q, w2_s, w2_z), topk, act, layout,
                         params, out, routing, workspace, stream).run()
