"""The block norm's gradient row by row: what a row's values may and may not reach."""
import pytest
import torch

from routing_grouped_expert_amd import moe_block_norm, moe_block_norm_backward
from tests.test_block_norm_gpu import _dev, _inputs

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _bad_rows(t):
    return set((~torch.isfinite(t)).any(1).nonzero()[:, 0].tolist())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("h", [72, 520, 1416])
@pytest.mark.parametrize("gate", ["none", "token", "channel"])
def test_unnormed_branch_gradient_does_not_see_y(gate, h, dt):
    """Without w_post and w_pre d_y = scale * gate * d_x_out, whatever y holds; the
    scale is a power of two, so the product rounds once and the bits are equal."""
    print(f"[norm-rows] {gate} h={h} {dt}", flush=True)
    a, d = _inputs(23, h, dt, gate, post=False, pre=False, seed=h)
    a["y"][3, 5] = float("inf")
    a["y"][11] = float("nan")
    a["y"][20, h - 1] = -float("inf")
    da, dd = _dev(a), _dev(d)
    g = moe_block_norm_backward(dd["d_x_out"], None, **da, residual_scale=0.5)
    want = 0.5 * dd["d_x_out"].float()
    if gate != "none":
        want = want * da["gate"].float()
    assert torch.equal(g.d_y, want.to(da["y"].dtype))
    assert torch.equal(g.d_x, dd["d_x_out"])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("post", [0, 1])
def test_non_finite_values_fill_their_own_rows_only(post, dt):
    """With a norm a row's gradient depends on all of the row: those rows and no others."""
    a, d = _inputs(40, 136, dt, "channel", post=bool(post), seed=9)
    a["x"][3, 7] = float("inf")
    a["y"][11, 0] = float("nan")
    da, dd = _dev(a), _dev(d)
    f = moe_block_norm(**da)
    g = moe_block_norm_backward(dd["d_x_out"], dd["d_n_out"], **da, rstd_post=f.rstd_post,
                                rstd_pre=f.rstd_pre)
    for t in (f.x_out, f.n_out, g.d_x, g.d_y):
        assert _bad_rows(t) == {3, 11}
