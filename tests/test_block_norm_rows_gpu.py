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


# the first widths of every kernel (16-byte chunks a row: 129, 257, 386, 513, 769,
# 1025, 2049 and more), where a workgroup takes one row at a time
WIDE = [("bf16", 1032), ("bf16", 2056), ("bf16", 3104), ("bf16", 4104), ("bf16", 6152),
        ("bf16", 8200), ("bf16", 16384), ("f32", 520), ("f32", 1032), ("f32", 1544),
        ("f32", 2056), ("f32", 3080), ("f32", 4104), ("f32", 8200)]


@pytest.mark.parametrize("dt,h", WIDE)
def test_later_rows_of_a_workgroup_are_like_its_first(dt, h):
    """A launch has at most 512 (backward) or 2048 (forward) workgroups of one row:
    4500 rows give each several turns, calls of 500 rows one.  Every row's outputs have
    the same bits; the sums over the rows are the same fp32 terms in another order, off
    by at most n 2^-24 of the terms' magnitudes on either side."""
    print(f"[norm-turns] {dt} h={h}", flush=True)
    n, part = 4500, 500
    g = torch.Generator("cuda").manual_seed(h)

    def rnd(*shape, std=1.0, mean=0.0):
        t = torch.randn(*shape, generator=g, device=DEV) * std + mean
        return t.to({"bf16": torch.bfloat16, "f32": torch.float32}[dt])

    w = {"w_post": rnd(h, std=0.3, mean=1.0), "w_pre": rnd(h, std=0.3, mean=1.0),
         "gate": rnd(h, std=0.5), "residual_scale": 0.5}
    x, y, dx, dn = rnd(n, h, std=2.0), rnd(n, h), rnd(n, h, std=0.1), rnd(n, h, std=0.1)

    def both(s):
        f = moe_block_norm(x[s], y[s], **w)
        b = moe_block_norm_backward(dx[s], dn[s], x[s], y[s], **w, rstd_post=f.rstd_post,
                                    rstd_pre=f.rstd_pre)
        return f, b

    f, b = both(slice(0, n))
    sums = {k: torch.zeros(h, dtype=torch.float64, device=DEV)
            for k in ("d_w_pre", "d_w_post", "d_gate")}
    terms = {k: v.clone() for k, v in sums.items()}
    for i in range(0, n, part):
        s = slice(i, i + part)
        pf, pb = both(s)
        for k in ("x_out", "n_out", "rstd_post", "rstd_pre"):
            assert torch.equal(getattr(f, k)[s], getattr(pf, k)), (k, i)
        for k in ("d_x", "d_y"):
            assert torch.equal(getattr(b, k)[s], getattr(pb, k)), (k, i)
        yh = y[s].double() * pf.rstd_post.double()[:, None]
        z = yh * w["w_post"].double()
        xh = (x[s].double() + 0.5 * w["gate"].double() * z) * pf.rstd_pre.double()[:, None]
        sd = 0.5 * pb.d_x.double()
        terms["d_w_pre"] += (dn[s].double() * xh).abs().sum(0)
        terms["d_w_post"] += (sd * w["gate"].double() * yh).abs().sum(0)
        terms["d_gate"] += (sd * z).abs().sum(0)
        for k in sums:
            sums[k] += getattr(pb, k).double()
    for k in sums:
        # (the terms are taken from rounded outputs: 1 % covers it)
        err = (getattr(b, k).double() - sums[k]).abs()
        assert (err <= 1.01 * 2 * n * 2.0 ** -24 * terms[k]).all(), k
