"""CPU oracle for the MoE layer forward: TEST INFRASTRUCTURE ONLY.

A plain, slow, obviously-correct numpy (float64) statement of what the GPU path
computes.  Only ``tests/``, ``__graft_entry__.smoke()`` and the ``cpu_baseline``
leg of ``bench.py`` may import it.  It shares no code with the HIP library or its
Python binding, and imports neither.

* :mod:`oracle.routing` -- top-k gating with softmax over the selected logits and
  the routing metadata built from it (bitmatrix, per-expert histogram, ragged
  offsets, stable expert-sorted gather/scatter indices, permuted gate weights).
* :mod:`oracle.ffn` -- the expert FFN (SiLU-gated, SwiGLU-OAI, ReLU^2) run as the
  masked per-expert loop, the weighted combine, and the sorted-dispatch variant.
* :mod:`oracle.ffn` also gives the layer with the routing weight on the input
  rows (``moe_ffn_weighted_input``).
* :mod:`oracle.quant` -- MXFP4 expert weights: E2M1 codes with one E8M0 scale
  per 32 weights along K (quantise, dequantise), and 4-bit codes with a scale and
  a zero point per group of weights.
* :mod:`oracle.routing` also gives the router logits from the gate weight
  (``gate_logits``, ``route_gate``).
* both also give one GPU's expert-parallel share (``route_ep``,
  ``moe_ffn_share``): the selected experts remapped to local ids, -1 outside.

* :mod:`oracle.block` -- rows into expert-sorted order and back with the routing
  weights, the norms around a block, and the gradients of both.

* :mod:`oracle.train` -- the gradient of the expert FFN and the AdamW step.

Every function is pinned by ``tests/test_oracle_*.py`` against brute force,
library routines, closed forms, invariants and the hand-derived fixtures in
``tests/golden/``; the one part with no such pin (the SwiGLU-OAI formula relative
to the pages) is marked "parity unpinned" where it is defined.
"""
from .routing import (RoutingRef, bitmatrix, gate_logits, histogram, offsets_from_hist,
                      remap_to_share, route, route_ep, route_gate, round_to_dtype, sorted_indices,
                      topk_select, topk_softmax)
from .quant import (dequantize_int4, dequantize_mxfp4, e2m1_decode, e2m1_encode, quantize_int4,
                    quantize_mxfp4)
from .block import (block_norm, block_norm_grad, combine_weighted, combine_weighted_grad,
                    dispatch, rms_norm, topk_weight_grad)
from .ffn import (activation, moe_ffn, moe_ffn_share, moe_ffn_sorted,
                  moe_ffn_weighted_input, split_gate_up)
from .train import (activation_grad, adamw, block_scale, clip_coefficient, e4m3_values,
                    join_gate_up, moe_ffn_grad)

__all__ = [
    "RoutingRef", "route", "topk_select", "topk_softmax", "bitmatrix", "histogram",
    "offsets_from_hist", "sorted_indices", "round_to_dtype", "remap_to_share", "route_ep",
    "gate_logits", "route_gate",
    "activation", "split_gate_up", "moe_ffn", "moe_ffn_sorted", "moe_ffn_share",
    "moe_ffn_weighted_input", "quantize_mxfp4", "dequantize_mxfp4", "e2m1_encode",
    "e2m1_decode", "dispatch", "combine_weighted", "combine_weighted_grad", "topk_weight_grad",
    "rms_norm", "block_norm", "block_norm_grad", "quantize_int4", "dequantize_int4",
    "activation_grad", "join_gate_up", "moe_ffn_grad", "adamw", "clip_coefficient",
    "e4m3_values", "block_scale",
]
