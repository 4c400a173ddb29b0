"""Measured cases of the operators around and inside a mixture-of-experts block.

Three groups of operators, each in a plain form (elementary torch operations in
32 bits, rounded once at the end) and as this package's calls:

* sorted rows: token rows into expert-sorted order (``moe_dispatch``), the rows
  back into token order with the routing weights applied
  (``moe_combine_weighted``), and the gradient of that step down to the router
  logits (``moe_combine_weighted_backward``, ``moe_route_backward``);
* block norms: the norm after a block with its gate, the residual scale and the
  residual sum, and the norm ahead of the next block, in one pass
  (``moe_block_norm``), and its gradient (``moe_block_norm_backward``);
* 4-bit experts: the expert FFN of decode-sized batches with 4-bit weights, one
  scale and zero point per group of weights (``moe_experts_int4``).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-6


# ---------------------------------------------------------------- cases

def _rows(kind, n, h, e, k, dtype, wdtype, zipf):
    return {"kind": kind, "n": n, "h": h, "e": e, "k": k, "dtype": dtype, "wdtype": wdtype,
            "zipf": zipf}


def _norm(kind, n, h, dtype, gate, scale, post=True, pre=True, branch=True):
    return {"kind": kind, "n": n, "h": h, "dtype": dtype, "gate": gate, "scale": scale,
            "post": post, "pre": pre, "branch": branch}


def _int4(n, h, i, e, k, group, zeros, act, layout):
    return {"kind": "int4", "n": n, "h": h, "i": i, "e": e, "k": k, "group": group,
            "zeros": zeros, "act": act, "layout": layout, "dtype": "bf16", "wdtype": "bf16",
            "zipf": 0.0}


def listed():
    def named(name, c):
        return {"name": name, **c}

    return [
        # a small fp32 layer: what a call costs when there is next to nothing to move
        named("dispatch_tiny", _rows("dispatch", 33, 128, 8, 2, "f32", "f32", 0.0)),
        # a training or prompt batch of a 64-expert top-8 layer with skewed routing
        named("dispatch_prompt", _rows("dispatch", 16384, 4096, 64, 8, "bf16", "bf16", 1.1)),
        # a decoding step of 33 sequences on a 128-expert top-4 layer
        named("combine_step", _rows("combine", 33, 2880, 128, 4, "bf16", "bf16", 0.0)),
        # a prompt of 4096 tokens on the same layer, routing weights kept in fp32
        named("combine_prompt", _rows("combine", 4096, 2880, 128, 4, "bf16", "f32", 0.0)),
        # an fp32 training step with an odd token count and odd sizes
        named("combine_grad_odd", _rows("combine_grad", 4095, 1416, 40, 6, "f32", "f32", 0.5)),
        # a training step of the 64-expert top-8 layer: the largest case
        named("combine_grad_train", _rows("combine_grad", 16384, 4096, 64, 8, "bf16", "bf16",
                                          1.1)),
        # the norms between two blocks while one token is decoded
        named("norm_token", _norm("norm", 1, 2880, "bf16", "none", 1.0)),
        # the same for a prompt, with a learned gate per channel and a residual scale
        named("norm_prompt", _norm("norm", 16384, 4096, "bf16", "channel", 0.22)),
        # an fp32 training step of a narrow model, one gate value per token, odd token count
        named("norm_grad_odd", _norm("norm_grad", 4099, 512, "f32", "token", 1.0)),
        # the training step that goes with norm_prompt
        named("norm_grad_train", _norm("norm_grad", 16384, 4096, "bf16", "channel", 0.22)),
        # one token decoded through a 128-expert top-4 layer held in 4 bits
        named("int4_token", _int4(1, 2880, 2880, 128, 4, 64, True, "swiglu_oai", "interleaved")),
        # a decoding step of 32 sequences on the 64-expert top-8 layer, symmetric codes
        named("int4_step", _int4(32, 4096, 1536, 64, 8, 128, False, "silu", "packed")),
    ]


def _log_int(rng, lo, hi, mult=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo // mult, round(v / mult)) * mult


def draw(rng):
    kind = rng.choice(["dispatch", "combine", "combine_grad", "norm", "norm_grad", "int4"])
    while True:
        if kind == "int4":
            group = rng.choice([32, 64, 128])
            e = _log_int(rng, 4, 128)
            k = rng.randint(1, min(e, 8))
            act = rng.choice(["silu", "swiglu_oai", "relu2"])
            c = _int4(_log_int(rng, 1, 128), _log_int(rng, 256, 4096, group),
                      _log_int(rng, 256, 4096, group), e, k, group, rng.random() < 0.5, act,
                      "packed" if act == "relu2" else rng.choice(["packed", "interleaved"]))
            if 1.5 * c["i"] * c["h"] * e <= 1.7e9:
                return c
            continue
        dtype = rng.choice(["bf16", "bf16", "f32"])
        n, h = _log_int(rng, 1, 16384), _log_int(rng, 64, 8192, 8)
        if kind in ("norm", "norm_grad"):
            branch = rng.random() < 0.8
            c = _norm(kind, n, h, dtype,
                      rng.choice(["none", "token", "channel"]) if branch else "none",
                      rng.choice([1.0, 0.22, 0.5]) if branch else 1.0,
                      branch and rng.random() < 0.75, not branch or rng.random() < 0.75, branch)
        else:
            e = _log_int(rng, 2, 256)
            k = rng.randint(1, min(e, 16))
            c = _rows(kind, n, h, e, k, dtype, rng.choice([dtype, "f32"]),
                      rng.choice([0.0, 0.0, 0.5, 1.1]))
        if work(c)["bytes"] <= 2.3e9:
            return c


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _routing(g, c):
    """Routing metadata as a routing step leaves it, from random logits (a
    Zipf-like bias per expert where ``zipf`` is set)."""
    n, e, k = c["n"], c["e"], c["k"]
    logits = _randn(g, n, e)
    if c["zipf"]:
        rank = torch.randperm(e, generator=g, device="cuda").float() + 1.0
        logits = logits - c["zipf"] * rank.log()
    dt = DTYPES[c["wdtype"]]
    val, idx = logits.to(dt).sort(dim=1, descending=True, stable=True)
    topk_idx = idx[:, :k].to(torch.int32).contiguous()
    topk_w = torch.softmax(val[:, :k].float(), 1).to(dt).contiguous()
    flat = topk_idx.reshape(-1).long()
    col_sorted = flat.sort(stable=True)[1]
    row_sorted = torch.empty_like(col_sorted)
    row_sorted[col_sorted] = torch.arange(n * k, device="cuda")
    col_sum = torch.bincount(flat, minlength=e)
    offsets = torch.cat([col_sum.new_zeros(1), col_sum.cumsum(0)])
    words = (e + 31) // 32
    bits = torch.zeros(n, words * 32, dtype=torch.int64, device="cuda")
    bits.scatter_(1, topk_idx.long(), 1)
    shifts = torch.arange(32, device="cuda")
    bitmatrix = (bits.view(n, words, 32) << shifts).sum(2)
    return {"topk_idx": topk_idx, "topk_w": topk_w,
            "bitmatrix": torch.where(bitmatrix >= 2 ** 31, bitmatrix - 2 ** 32, bitmatrix)
            .to(torch.int32),
            "col_sum": col_sum.to(torch.int32), "offsets": offsets.to(torch.int32),
            "col_sorted": col_sorted.to(torch.int32), "row_sorted": row_sorted.to(torch.int32),
            "gate_scal": topk_w.reshape(-1)[col_sorted].contiguous()}


def _codes(g, e, rows, k, group, zeros):
    """4-bit codes, group scales and zero points of one weight array: codes two
    to a byte (the even element in the low nibble), scales and zero points
    group-major per expert; without zero points the zero is 8."""
    q = torch.randint(0, 256, (e, rows, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = (0.5 + torch.rand(e, k // group, rows, generator=g, device="cuda")) / (4.6 * k ** 0.5)
    z = None
    if zeros:
        z = torch.randint(5, 11, (e, k // group, rows), generator=g, device="cuda",
                          dtype=torch.uint8)
    return q, s.to(torch.bfloat16), z


def prepare(case, seed):
    c, g = case, _gen(seed)
    n, h, dt = c["n"], c["h"], DTYPES[c["dtype"]]
    s = {"case": c}
    if c["kind"] in ("dispatch", "combine", "combine_grad", "int4"):
        s["routing"] = _routing(g, c)
    if c["kind"] in ("dispatch", "int4"):
        s["x"] = _randn(g, n, h).to(dt)
    if c["kind"] in ("combine", "combine_grad"):
        s["y_sorted"] = _randn(g, n * c["k"], h).to(dt)
    if c["kind"] == "combine_grad":
        s["d_out"] = (_randn(g, n, h) / 64).to(dt)
    if c["kind"] == "int4":
        rows = c["i"] if c["act"] == "relu2" else 2 * c["i"]
        s["w13"] = _codes(g, c["e"], rows, h, c["group"], c["zeros"])
        s["w2"] = _codes(g, c["e"], h, c["i"], c["group"], c["zeros"])
        s["params"] = {"alpha": 1.702, "beta": 1.0, "limit": 7.0} if c["act"] == "swiglu_oai" \
            else {}
    if c["kind"] in ("norm", "norm_grad"):
        # a residual stream has a few channels far above the others
        chan = 1.0 + 20.0 * (torch.rand(h, generator=g, device="cuda") < 0.01)
        s["x"] = (_randn(g, n, h) * chan).to(dt)
        s["y"] = (_randn(g, n, h) * 0.7).to(dt) if c["branch"] else None
        s["w_post"] = (1.0 + 0.2 * _randn(g, h)).to(dt) if c["post"] else None
        s["w_pre"] = (1.0 + 0.2 * _randn(g, h)).to(dt) if c["pre"] else None
        s["gate"] = None
        if c["gate"] == "token":
            s["gate"] = torch.sigmoid(_randn(g, n, 1)).to(dt)
        elif c["gate"] == "channel":
            s["gate"] = (0.5 + 0.2 * _randn(g, h)).to(dt)
    if c["kind"] == "norm_grad":
        s["d_x_out"] = (_randn(g, n, h) / 64).to(dt)
        s["d_n_out"] = (_randn(g, n, h) / 64).to(dt) if c["pre"] else None
        # what the forward pass saved for this one
        f = _norm_values(s)
        s["rstd_post"], s["rstd_pre"] = f["rstd_post"], f["rstd_pre"]
    return s


# ---------------------------------------------------------------- plain forms

def _norm_values(s):
    """The block norm in fp32: every value the outputs and the gradient need."""
    c = s["case"]
    x = s["x"].float()
    f = {"rstd_post": None, "rstd_pre": None, "n": None}
    if s["y"] is not None:
        z = s["y"].float()
        if s["w_post"] is not None:
            f["rstd_post"] = torch.rsqrt((z * z).mean(1) + EPS)
            z = z * f["rstd_post"][:, None] * s["w_post"].float()
        f["z"] = z
        b = z if s["gate"] is None else z * s["gate"].float()
        x = x + c["scale"] * b
    f["x"] = x
    if s["w_pre"] is not None:
        f["rstd_pre"] = torch.rsqrt((x * x).mean(1) + EPS)
        f["n"] = x * f["rstd_pre"][:, None] * s["w_pre"].float()
    return f


def _plain_norm(s):
    f, dt = _norm_values(s), s["x"].dtype
    return {"x_out": f["x"].to(dt) if s["y"] is not None else None,
            "n_out": f["n"].to(dt) if f["n"] is not None else None,
            "rstd_post": f["rstd_post"], "rstd_pre": f["rstd_pre"]}


def _rms_grad(u, r, w, d):
    """Gradient of u * r * w, r = 1 / rms(u), with respect to u and w."""
    uh, du = u * r[:, None], d * w
    return r[:, None] * (du - uh * (du * uh).mean(1, keepdim=True)), (d * uh).sum(0)


def _plain_norm_grad(s):
    c, dt = s["case"], s["x"].dtype
    out = {"d_x": None, "d_y": None, "d_w_pre": None, "d_w_post": None, "d_gate": None}
    x, d = s["x"].float(), s["d_x_out"].float()
    if s["y"] is not None:
        y = s["y"].float()
        z = y
        if s["w_post"] is not None:
            z = y * s["rstd_post"][:, None] * s["w_post"].float()
        x = x + c["scale"] * (z if s["gate"] is None else z * s["gate"].float())
    if s["w_pre"] is not None:
        dx, out["d_w_pre"] = _rms_grad(x, s["rstd_pre"], s["w_pre"].float(),
                                       s["d_n_out"].float())
        d = d + dx
    out["d_x"] = d.to(dt)
    if s["y"] is not None:
        dz = c["scale"] * d
        if s["gate"] is not None:
            dg = dz * z
            out["d_gate"] = dg.sum(1, keepdim=True) if c["gate"] == "token" else dg.sum(0)
            dz = dz * s["gate"].float()
        if s["w_post"] is not None:
            dz, out["d_w_post"] = _rms_grad(y, s["rstd_post"], s["w_post"].float(), dz)
        out["d_y"] = dz.to(dt)
    return out


def _plain_rows(s):
    c, r = s["case"], s["routing"]
    n, k, h = c["n"], c["k"], c["h"]
    row = r["row_sorted"].long()
    if c["kind"] == "dispatch":
        return s["x"][r["col_sorted"].long() // k]
    w = r["topk_w"].float()
    y = s["y_sorted"][row].view(n, k, h).float()
    if c["kind"] == "combine":
        return (y * w[:, :, None]).sum(1).to(s["y_sorted"].dtype)
    d = s["d_out"].float()
    dw = (y * d[:, None, :]).sum(2)
    dy = torch.empty_like(s["y_sorted"])
    dy[row] = (w[:, :, None] * d[:, None, :]).view(n * k, h).to(dy.dtype)
    dl = w * (dw - (w * dw).sum(1, keepdim=True))
    d_logits = torch.zeros(n, c["e"], device="cuda").scatter_(1, r["topk_idx"].long(), dl)
    return {"d_y_sorted": dy, "d_topk_w": dw, "d_logits": d_logits.to(r["topk_w"].dtype)}


def _values(w, group, pick=None):
    """fp32 weights [E, rows, K] (of the picked experts) from codes, scales and zeros."""
    q, s, z = (t if t is None or pick is None else t[pick] for t in w)
    e, rows, half = q.shape
    v = torch.stack([q & 15, q >> 4], -1).view(e, rows, 2 * half // group, group).float()
    zero = 8.0 if z is None else z.float().transpose(1, 2)[..., None]
    return ((v - zero) * s.float().transpose(1, 2)[..., None]).view(e, rows, 2 * half)


def _act(u, act, layout, p):
    """Activation of w13 products u [B, rows, cols] -> [B, inter, cols]."""
    if act == "relu2":
        return torch.relu(u) ** 2
    b, rows, cols = u.shape
    if layout == "packed":
        gate, up = u[:, :rows // 2], u[:, rows // 2:]
    else:
        gate, up = u[:, 0::2], u[:, 1::2]
    if act == "swiglu_oai":
        gate = gate.clamp(max=p["limit"])
        up = up.clamp(-p["limit"], p["limit"])
        return gate * torch.sigmoid(p["alpha"] * gate) * (up + p["beta"])
    return gate * torch.sigmoid(gate) * up


def _plain_int4(s):
    c, r = s["case"], s["routing"]
    n, k, e, h = c["n"], c["k"], c["e"], c["h"]
    x = s["x"].float()
    eidx = r["topk_idx"].long()
    if n * k <= e:
        # few entries: each one's expert is picked out and applied to its row
        pick = eidx.reshape(-1)
        cols = x.repeat_interleave(k, 0)[:, :, None]
        a = _act(torch.bmm(_values(s["w13"], c["group"], pick), cols), c["act"], c["layout"],
                 s["params"])
        y = torch.bmm(_values(s["w2"], c["group"], pick), a.contiguous())[:, :, 0].view(n, k, h)
    else:
        # every expert is applied to every token; each token's are picked out
        cols = x.t().contiguous()[None].expand(e, h, n).contiguous()
        a = _act(torch.bmm(_values(s["w13"], c["group"]), cols), c["act"], c["layout"],
                 s["params"])
        y = torch.bmm(_values(s["w2"], c["group"]), a.contiguous())  # [E, H, N]
        y = y[eidx, :, torch.arange(n, device="cuda")[:, None]]
    return (y * r["topk_w"].float()[:, :, None]).sum(1).to(torch.bfloat16)


# ---------------------------------------------------------------- run

def _own_run(s):
    import routing_grouped_expert_amd as moe

    c, kind = s["case"], s["case"]["kind"]
    if kind in ("norm", "norm_grad"):
        args = {"w_pre": s["w_pre"], "w_post": s["w_post"], "gate": s["gate"],
                "residual_scale": c["scale"]}
        if kind == "norm":
            r = moe.moe_block_norm(s["x"], s["y"], eps=EPS, **args)
            return {"x_out": r.x_out, "n_out": r.n_out, "rstd_post": r.rstd_post,
                    "rstd_pre": r.rstd_pre}
        r = moe.moe_block_norm_backward(s["d_x_out"], s["d_n_out"], s["x"], s["y"],
                                        rstd_post=s["rstd_post"], rstd_pre=s["rstd_pre"], **args)
        return {"d_x": r.d_x, "d_y": r.d_y, "d_w_pre": r.d_w_pre, "d_w_post": r.d_w_post,
                "d_gate": r.d_gate}
    routing = moe.Routing(**s["routing"])
    if kind == "dispatch":
        return moe.moe_dispatch(s["x"], routing)
    if kind == "combine":
        return moe.moe_combine_weighted(s["y_sorted"], routing)
    if kind == "combine_grad":
        dy, dw = moe.moe_combine_weighted_backward(s["d_out"], s["y_sorted"], routing)
        return {"d_y_sorted": dy, "d_topk_w": dw,
                "d_logits": moe.moe_route_backward(dw, routing)}
    return moe.moe_experts_int4(s["x"], *s["w13"], *s["w2"], routing, c["act"], c["layout"],
                                s["params"])


def run(state):
    if own:
        return _own_run(state)
    kind = state["case"]["kind"]
    if kind == "norm":
        return _plain_norm(state)
    if kind == "norm_grad":
        return _plain_norm_grad(state)
    if kind == "int4":
        return _plain_int4(state)
    return _plain_rows(state)


# ---------------------------------------------------------------- least work

def work(case):
    c = case
    n, h, es = c["n"], c["h"], SIZE[c["dtype"]]
    if c["kind"] in ("norm", "norm_grad"):
        grad = c["kind"] == "norm_grad"
        if grad:  # x, d_x_out, (y), (d_n_out) in; d_x, (d_y) out
            arrays = 3 + 2 * c["branch"] + c["pre"]
        else:     # x, (y) in; (x_out), (n_out) out
            arrays = 1 + 2 * c["branch"] + c["pre"]
        return {"bytes": arrays * n * h * es + 4 * n * (c["post"] + c["pre"]),
                "flops": (16 if grad else 8) * n * h}
    m, ws = n * c["k"], SIZE[c["wdtype"]]
    if c["kind"] == "dispatch":
        return {"bytes": (n + m) * h * es + 4 * m, "flops": 0}
    if c["kind"] == "combine":
        return {"bytes": (n + m) * h * es + (4 + ws) * m, "flops": 2 * m * h}
    if c["kind"] == "combine_grad":
        return {"bytes": (n + 2 * m) * h * es + (12 + ws) * m + n * c["e"] * ws,
                "flops": 3 * m * h}
    # the experts that at least one token takes, expected for even routing
    e, i = c["e"], c["i"]
    used = e * (1 - (1 - c["k"] / e) ** n)
    sets = 2 if c["act"] != "relu2" else 1
    weights = (sets + 1) * i * h
    per = 0.5 + (2 + c["zeros"]) / c["group"]
    return {"bytes": used * weights * per + 2 * n * h * es, "flops": 2 * m * weights}


# ---------------------------------------------------------------- 64 bits

def _exact_norm(c, s):
    """Row by row from the definitions: u / sqrt(mean(u^2) + eps) * w."""
    x = s["x"].double()
    res = {"x_out": None, "n_out": None, "rstd_post": None, "rstd_pre": None}
    if c["branch"]:
        b = s["y"].double()
        if c["post"]:
            rms = (b.square().sum(1, keepdim=True) / c["h"] + EPS).sqrt()
            res["rstd_post"] = (1.0 / rms)[:, 0]
            b = b / rms * s["w_post"].double()
        if c["gate"] != "none":
            b = b * s["gate"].double()
        x = x + b * c["scale"]
        res["x_out"] = x
    if c["pre"]:
        rms = (x.square().sum(1, keepdim=True) / c["h"] + EPS).sqrt()
        res["rstd_pre"] = (1.0 / rms)[:, 0]
        res["n_out"] = x / rms * s["w_pre"].double()
    return res


def _exact_norm_grad(c, s):
    """Reverse-mode differentiation of the definition in 64 bits."""
    names = [p for p in ("x", "y", "w_pre", "w_post", "gate") if s[p] is not None]
    leaf = {p: s[p].double().requires_grad_() for p in names}
    f = _exact_norm(c, {**{p: None for p in ("y", "w_pre", "w_post", "gate")}, **leaf})
    x_out = f["x_out"] if f["x_out"] is not None else leaf["x"]
    total = (x_out * s["d_x_out"].double()).sum()
    if c["pre"]:
        total = total + (f["n_out"] * s["d_n_out"].double()).sum()
    got = dict(zip(names, torch.autograd.grad(total, [leaf[p] for p in names])))
    return {"d_x": got["x"], "d_y": got.get("y"), "d_w_pre": got.get("w_pre"),
            "d_w_post": got.get("w_post"), "d_gate": got.get("gate")}


def _exact_rows(c, s):
    """Slot by slot: slot j of every token at a time."""
    r, k, h = s["routing"], c["k"], c["h"]
    row, w = r["row_sorted"].view(-1, k).long(), r["topk_w"].double()
    if c["kind"] == "dispatch":
        out = torch.zeros(c["n"] * k, h, dtype=torch.float64, device="cuda")
        for j in range(k):
            out[row[:, j]] = s["x"].double()
        return out
    if c["kind"] == "combine":
        out = torch.zeros(c["n"], h, dtype=torch.float64, device="cuda")
        for j in range(k):
            out += w[:, j:j + 1] * s["y_sorted"][row[:, j]].double()
        return out
    d = s["d_out"].double()
    dy = torch.zeros(c["n"] * k, h, dtype=torch.float64, device="cuda")
    dw = torch.zeros_like(w)
    for j in range(k):
        dy[row[:, j]] = w[:, j:j + 1] * d
        dw[:, j] = (s["y_sorted"][row[:, j]].double() * d).sum(1)
    # d softmax_i / d logit_j = p_i (delta_ij - p_j) over the chosen experts
    jac = torch.diag_embed(w) - w[:, :, None] * w[:, None, :]
    dl = (jac * dw[:, :, None]).sum(1)
    d_logits = torch.zeros(c["n"], c["e"], dtype=torch.float64, device="cuda")
    d_logits[torch.arange(c["n"], device="cuda")[:, None], r["topk_idx"].long()] = dl
    return {"d_y_sorted": dy, "d_topk_w": dw, "d_logits": d_logits}


def _exact_int4(c, s):
    """Expert by expert, the tokens that chose it."""
    def matrix(w, e):
        q, sc, z = w
        low, high = (q[e] & 15).double(), (q[e] >> 4).double()
        v = torch.stack([low, high], 2).flatten(1)
        scale = sc[e].double().t().repeat_interleave(c["group"], 1)
        zero = 8.0 if z is None else z[e].double().t().repeat_interleave(c["group"], 1)
        return scale * (v - zero)

    r, p = s["routing"], s["params"]
    out = torch.zeros(c["n"], c["h"], dtype=torch.float64, device="cuda")
    for e in range(c["e"]):
        tok, slot = torch.nonzero(r["topk_idx"] == e, as_tuple=True)
        if tok.numel() == 0:
            continue
        u = s["x"][tok].double() @ matrix(s["w13"], e).t()
        if c["act"] == "relu2":
            a = u.clamp(min=0).square()
        else:
            g, up = (u[:, :c["i"]], u[:, c["i"]:]) if c["layout"] == "packed" \
                else (u[:, ::2], u[:, 1::2])
            alpha, beta = p.get("alpha", 1.0), p.get("beta", 0.0)
            lim = p.get("limit", math.inf)
            g, up = g.clamp(max=lim), up.clamp(min=-lim, max=lim)
            a = g / (1 + torch.exp(-alpha * g)) * (up + beta)
        out[tok] += r["topk_w"][tok, slot].double()[:, None] * (a @ matrix(s["w2"], e).t())
    return out


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "norm":
        return _exact_norm(case, s)
    if kind == "norm_grad":
        return _exact_norm_grad(case, s)
    if kind == "int4":
        return _exact_int4(case, s)
    return _exact_rows(case, s)
