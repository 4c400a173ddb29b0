"""The 4-bit oracle: closed forms and properties of the quantiser (CPU)."""
import numpy as np
import pytest
import torch

import oracle


def test_representable_weights_come_back():
    rng = np.random.default_rng(0)
    for zeros, lo, hi in ((True, -7, 8), (False, -7, 7)):
        c = rng.integers(lo, hi + 1, size=(3, 64)).astype(np.float32)
        c[:, [0, 32]], c[:, [1, 33]] = lo, hi  # each group reaches both ends
        w = c * np.float32(0.25)
        q, s, z = oracle.quantize_int4(torch.from_numpy(w), 32, zeros)
        assert np.array_equal(s, np.full((3, 2), 0.25, np.float32))
        assert np.array_equal(oracle.dequantize_int4(q, s, z, 32), w)


def test_packing_and_the_default_zero_point():
    q = np.array([[0x21, 0xF0] * 8], dtype=np.uint8)  # codes 1 2 0 15 ...
    v = oracle.dequantize_int4(q, np.array([[0.5]]), None, 32)
    assert np.array_equal(v[0, :4], (np.array([1, 2, 0, 15]) - 8) * 0.5)
    z = np.array([[3]], dtype=np.uint8)
    assert np.array_equal(oracle.dequantize_int4(q, np.array([[0.5]]), z, 32), v + 2.5)


@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_error_is_about_half_a_step(group, zeros):
    g = torch.Generator().manual_seed(group)
    w = torch.randn(5, 256, generator=g) * 0.02
    w[0] = 0
    w[1] = w[1].abs()
    q, s, z = oracle.quantize_int4(w, group, zeros)
    err = np.abs(oracle.dequantize_int4(q, s, z, group) - w.numpy()).reshape(5, -1, group)
    # half a step for the code; the scale's rounding to bf16 (2^-8) may cut off up to
    # 15 * 2^-8 of a step at the ends, and the rounded zero point half a step more
    assert (err <= s[..., None] * (0.5 + 15 / 256 + (0.5 if zeros else 0.0))).all()
    assert not err[0].any()
