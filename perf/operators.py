"""Measured cases of the operators around the expert dispatch: the RMS norm in front of it and its gradient, the router's
balance loss with its gradient, and the linear layers (router projection, shared expert, routed experts) with their epilogue.

`run` computes a case with plain torch operations in 32 bits, or, with `own` set, through the package's entry points.
"""
import math

import torch

own = False

F8 = torch.float8_e4m3fn
SCORES = ("softmax", "sigmoid")
ACTS = ("none", "silu", "gelu", "swiglu")


# ---- cases ---------------------------------------------------------------------


def listed():
    return [
        # one token of a decode step enters an MoE block: residual added, normalised, handed on in bf16 (router) and e4m3 (experts)
        dict(name="norm_one_token", op="norm", rows=1, hidden=7168, residual=True, out="both", gamma="bf16"),
        # the same at the prefill batch, 8 ranks x 4096 tokens
        dict(name="norm_prefill", op="norm", rows=32768, hidden=7168, residual=True, out="both", gamma="bf16"),
        # gradient of the norm on a short, odd training batch of the small configuration's width
        dict(name="norm_backward_short", op="norm_backward", rows=517, hidden=1024, residual=True, gamma="fp32"),
        # and on 8 x 2048 training tokens
        dict(name="norm_backward_train", op="norm_backward", rows=16384, hidden=7168, residual=True, gamma="fp32"),
        # balance loss and gradient over one decode-sized micro-batch, top 8 of 256 experts
        dict(name="balance_micro", op="balance", tokens=1024, experts=256, topk=8, score="softmax", seqs=1, mask=0.0),
        # sequence-wise loss over packed sequences of uneven length, skewed experts and dropped slots
        dict(name="balance_packed", op="balance", tokens=32768, experts=64, topk=6, score="softmax", seqs=9, mask=0.05),
        # the largest training batch, 8 ranks x 16384 tokens, sigmoid scores
        dict(name="balance_large", op="balance", tokens=131072, experts=256, topk=8, score="sigmoid", seqs=32, mask=0.0),
        # router projection of the decode batch, 8 x 128 tokens, fp32 logits
        dict(name="router_logits", op="linear", type="bf16", groups=0, tokens=1024, topk=1, cin=7168, cout=256, act="none", bias=False, residual=False, out="fp32"),
        # one token through a shared dense layer with bias, activation and residual
        dict(name="dense_one_token", op="linear", type="bf16", groups=0, tokens=1, topk=1, cin=7168, cout=2048, act="gelu", bias=True, residual=True, out="bf16"),
        # one rank's 32 experts on the prefill batch: gate and up products with SwiGLU
        dict(name="experts_up_prefill", op="linear", type="bf16", groups=32, tokens=4096, topk=8, cin=7168, cout=2048, act="swiglu", bias=False, residual=False, out="bf16"),
        # the same experts' down product from e4m3 rows
        dict(name="experts_down_fp8", op="linear", type="e4m3", groups=32, tokens=4096, topk=8, cin=2048, cout=7168, act="none", bias=False, residual=False, out="bf16"),
        # one rank's experts on the FP8 decode batch, output quantised again for the down product
        dict(name="experts_up_decode_fp8", op="linear", type="e4m3", groups=32, tokens=128, topk=8, cin=7168, cout=2048, act="swiglu", bias=False, residual=False, out="e4m3"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "norm_backward", "balance", "linear", "linear", "linear"))
    if op in ("norm", "norm_backward"):
        hidden = 128 * rng.randint(1, 64)
        c = dict(op=op, rows=_log(rng, 1, min(32768 if op == "norm" else 16384, 32768 * 7168 // hidden)), hidden=hidden,
                 residual=rng.random() < 0.7, gamma=rng.choice(("bf16", "fp32")))
        return dict(c, out=rng.choice(("bf16", "e4m3", "both"))) if op == "norm" else c
    if op == "balance":
        experts = rng.choice((rng.randint(2, 64), 32 * rng.randint(2, 12), rng.randint(65, 1024)))
        tokens = _log(rng, 1, 131072 * 256 // max(256, experts))
        return dict(op=op, tokens=tokens, experts=experts, topk=rng.randint(1, min(10, experts)), score=rng.choice(SCORES),
                    seqs=_log(rng, 1, min(64, tokens)), mask=rng.choice((0.0, 0.05, 0.3)))
    kind = rng.choice(("bf16", "e4m3"))
    groups = rng.choice((0, 0, rng.randint(1, 8), rng.randint(9, 64)))
    cin = 128 * rng.randint(1, 56) if kind == "e4m3" else 8 * rng.randint(8, 896)
    out = rng.choice(("bf16", "bf16", "fp32", "e4m3"))
    cout = 128 * rng.randint(1, 32) if out == "e4m3" else rng.choice((rng.randint(1, 512), 8 * rng.randint(16, 512), 128 * rng.randint(1, 32)))
    topk = rng.randint(1, min(8, groups)) if groups else 1
    tokens = _log(rng, 1, max(1, min(16384, 16384 // topk)))
    return dict(op=op, type=kind, groups=groups, tokens=tokens, topk=topk, cin=cin, cout=cout, act=rng.choice(ACTS),
                bias=rng.random() < 0.5, residual=rng.random() < 0.4, out=out)


# ---- inputs ----------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32 if dtype == F8 else dtype) * scale).to(dtype)


def _quantised(g, rows, k, scale, block_rows):
    """e4m3 [rows, k] of normal values and one fp32 scale for each block of block_rows x 128."""
    s = (0.5 + torch.rand(-(-rows // block_rows), k // 128, generator=g, device="cuda")) * (scale * 4.5 / 448)
    q = torch.empty(rows, k, dtype=F8, device="cuda")
    part = max(1, (1 << 27) // k)
    for r in range(0, rows, part):
        q[r:r + part] = (torch.randn(min(part, rows - r), k, generator=g, device="cuda") * 99.0).clamp_(-448, 448).to(F8)
    return q, s


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case=case)
    if op in ("norm", "norm_backward"):
        n, h = case["rows"], case["hidden"]
        gamma = 1 + 0.2 * torch.randn(h, generator=g, device="cuda")
        s["gamma"] = gamma if case["gamma"] == "fp32" else gamma.bfloat16()
        s["eps"] = 1e-6
        s["x"] = _randn(g, n, h, scale=1.5)
        s["res"] = _randn(g, n, h) if case["residual"] else None
        empty = lambda t, *shape: torch.empty(*shape, dtype=t, device="cuda")  # noqa: E731
        if op == "norm":
            s["h"] = empty(torch.bfloat16, n, h) if case["residual"] else None
            s["y"] = empty(torch.bfloat16, n, h) if case["out"] != "e4m3" else None
            s["q"] = empty(F8, n, h) if case["out"] != "bf16" else None
            s["q_scale"] = empty(torch.float32, n, h // 128) if case["out"] != "bf16" else None
            s["rstd"] = empty(torch.float32, n)
        else:
            s["dy"] = _randn(g, n, h)
            s["rstd"] = (s["x"].float().square().mean(1) + s["eps"]).rsqrt()
            s["dx"], s["dgamma"] = empty(torch.bfloat16, n, h), empty(torch.float32, h)
            if own:
                from combine_top_group_b200 import ep
                s["ws"] = empty(torch.uint8, ep.ep_rmsnorm_backward_workspace_bytes(n, h))
    elif op == "balance":
        n, e, k, q = case["tokens"], case["experts"], case["topk"], case["seqs"]
        bias = -0.3 * torch.log1p(torch.arange(e, device="cuda", dtype=torch.float32))
        s["logits"] = torch.randn(n, e, generator=g, device="cuda") + bias
        idx = s["logits"].topk(k, dim=1).indices.int()
        drop = torch.rand(n, k, generator=g, device="cuda") < case["mask"]
        s["idx"] = torch.where(drop, -1, idx).contiguous()
        cuts = (torch.rand(q - 1, generator=g, device="cuda") * n).long().sort().values
        ends = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), cuts, torch.full((1,), n, dtype=torch.long, device="cuda")])
        s["seq_off"] = ends.int()
        s["seq"] = torch.repeat_interleave(torch.arange(q, device="cuda"), ends[1:] - ends[:-1], output_size=n)
        s["coef"] = 1e-2
        s["grad"] = torch.rand(1, generator=g, device="cuda") + 0.5
        s["loss"], s["counts"] = torch.empty(1, device="cuda"), torch.empty(q, e, dtype=torch.int32, device="cuda")
        s["prob"], s["dlogits"] = torch.empty(q, e, device="cuda"), torch.empty(n, e, device="cuda")
        if own:
            from combine_top_group_b200 import ep
            s["ws"] = torch.empty(ep.ep_balance_loss_workspace_bytes(n, e, q), dtype=torch.uint8, device="cuda")
            s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    else:
        e, t, k, cin, cout = case["groups"], case["tokens"], case["topk"], case["cin"], case["cout"]
        wide = cout * (2 if case["act"] == "swiglu" else 1)
        groups = max(1, e)
        if e:
            logits = torch.randn(t, e, generator=g, device="cuda") - 0.1 * torch.log1p(torch.arange(e, device="cuda", dtype=torch.float32))
            top = logits.topk(k, dim=1)
            s["idx"], s["idx_w"] = top.indices.int().contiguous(), top.values.softmax(1).contiguous()
            counts = torch.bincount(s["idx"].flatten().long(), minlength=e)
        else:
            counts = torch.full((1,), t, device="cuda")
        rows = t * k
        s["counts"] = counts
        s["most"] = int(counts.max())  # the plain form's padded length
        s["expert"] = torch.repeat_interleave(torch.arange(groups, device="cuda"), counts, output_size=rows)
        s["place"] = torch.arange(rows, device="cuda") - (counts.cumsum(0) - counts)[s["expert"]]
        if case["type"] == "e4m3":
            s["x"], s["x_scale"] = _quantised(g, rows, cin, 1.0, 1)
            per = wide // cout
            blocks = -(-cout // 128)
            w, ws = _quantised(g, groups * wide, cin, cin ** -0.5, 128)
            ws = ws[:1].expand(groups * per * blocks, -1) * (0.5 + torch.rand(groups * per * blocks, 1, generator=g, device="cuda"))
            s["w"], s["w_scale"] = w.view(groups, wide, cin), ws.reshape(groups, per * blocks, cin // 128).contiguous()
        else:
            s["x"], s["x_scale"] = _randn(g, rows, cin), None
            s["w"], s["w_scale"] = _randn(g, groups, wide, cin, scale=cin ** -0.5), None
        s["bias"] = torch.randn(groups, wide, generator=g, device="cuda") * 0.1 if case["bias"] else None
        s["res"] = _randn(g, rows, cout) if case["residual"] else None
        kind = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": F8}[case["out"]]
        s["out"] = torch.empty(rows, cout, dtype=kind, device="cuda")
        s["out_scale"] = torch.empty(rows, cout // 128, device="cuda") if case["out"] == "e4m3" else None
        if own:
            from combine_top_group_b200 import ep
            s["buf"] = ep.ep_buffer_create(ep.ep_default_config(1, t, 128, groups, k), device="cuda")
            if e:
                ep.ep_get_layout(s["buf"], t, topk_idx=s["idx"], topk_w=s["idx_w"])
    return s


# ---- plain forms -------------------------------------------------------------------


def _e4m3_blocks(y):
    """e4m3 values and one fp32 scale for each 128 channels, by the dispatch's rule."""
    b = y.view(y.shape[0], -1, 128)
    amax = b.abs().amax(2, keepdim=True).clamp_min(1e-4)
    return (b * (448.0 / amax)).clamp(-448, 448).to(F8).view(y.shape), (amax / 448.0).squeeze(2)


def _norm_plain(s):
    v = s["x"].float()
    if s["res"] is not None:
        v = v + s["res"].float()
    rstd = torch.rsqrt(v.square().mean(1) + s["eps"])
    y = v * rstd[:, None] * s["gamma"].float()
    q, scale = _e4m3_blocks(y) if s["q"] is not None else (None, None)
    return dict(h=v.bfloat16() if s["h"] is not None else None, y=y.bfloat16() if s["y"] is not None else None, q=q, q_scale=scale, rstd=rstd)


def _norm_backward_plain(s):
    n = s["x"].float() * s["rstd"][:, None]
    dy = s["dy"].float()
    t = dy * s["gamma"].float()
    dx = (t - n * (t * n).mean(1, keepdim=True)) * s["rstd"][:, None]
    if s["res"] is not None:
        dx = dx + s["res"].float()
    return dict(dx=dx.bfloat16(), dgamma=(dy * n).sum(0))


def _balance_plain(s):
    c = s["case"]
    n, e, k, q = c["tokens"], c["experts"], c["topk"], c["seqs"]
    z = s["logits"]
    if c["score"] == "softmax":
        a = (z - z.amax(1, keepdim=True)).exp()
        d = a
    else:
        a = torch.sigmoid(z)
        d = a * torch.sigmoid(-z)
    total = a.sum(1, keepdim=True)
    p = a / total
    at = torch.where(s["idx"] >= 0, s["seq"][:, None] * e + s["idx"], q * e)
    counts = torch.zeros(q * e + 1, dtype=torch.int64, device=z.device).index_add_(0, at.flatten().long(), torch.ones(n * k, dtype=torch.int64, device=z.device))
    counts = counts[:-1].view(q, e)
    off = s["seq_off"].long()
    length = (off[1:] - off[:-1]).clamp_min(1)[:, None]
    member = (s["seq"][None, :] == torch.arange(q, device=z.device)[:, None]).float()
    prob = (member @ p) / length
    f = counts.float() * (e / k) / length
    loss = (s["coef"] / q) * (f * prob).sum().view(1)
    ft = f[s["seq"]]
    dp = (ft - (ft * p).sum(1, keepdim=True)) / total * d
    dlogits = dp * (s["grad"] * (s["coef"] / q) / length[s["seq"]])
    return dict(loss=loss, counts=counts.int(), prob=prob, dlogits=dlogits)


def _activated(z, act, cout):
    if act == "swiglu":
        gate, up = z[:, :cout], z[:, cout:]
        return gate * torch.sigmoid(gate) * up
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    return z


def _block_scaled(w, scale, cout):
    """Weights in fp32: each 128 x 128 block of each half of cout rows times its scale."""
    g, wide, cin = w.shape
    s = scale.view(g, wide // cout, -1, cin // 128).repeat_interleave(128, 2)[:, :, :cout].reshape(g, wide, cin // 128, 1)
    return (w.float().view(g, wide, cin // 128, 128) * s).view(g, wide, cin)


def _linear_plain(s):
    c = s["case"]
    x, w, cout = s["x"].float(), s["w"], c["cout"]
    if s["x_scale"] is not None:
        x = (x.view(x.shape[0], -1, 128) * s["x_scale"][:, :, None]).view(x.shape)
        w = _block_scaled(w, s["w_scale"], cout)
    else:
        w = w.float()
    padded = torch.zeros(w.shape[0], s["most"], x.shape[1], device=x.device)
    padded[s["expert"], s["place"]] = x
    z = torch.bmm(padded, w.transpose(1, 2))[s["expert"], s["place"]]
    if s["bias"] is not None:
        z = z + s["bias"][s["expert"]]
    y = _activated(z, c["act"], cout)
    if s["res"] is not None:
        y = y + s["res"].float()
    if c["out"] == "e4m3":
        q, scale = _e4m3_blocks(y)
        return dict(out=q, out_scale=scale)
    return dict(out=y.bfloat16() if c["out"] == "bf16" else y)


# ---- the package's entry points -------------------------------------------------------


def _run_own(s):
    from combine_top_group_b200 import ep
    c = s["case"]
    if c["op"] == "norm":
        ep.ep_rmsnorm(s["x"], s["gamma"], s["eps"], residual=s["res"], h=s["h"], y=s["y"], q=s["q"], q_scale=s["q_scale"], rstd=s["rstd"])
        return {k: s[k] for k in ("h", "y", "q", "q_scale", "rstd")}
    if c["op"] == "norm_backward":
        ep.ep_rmsnorm_backward(s["x"], s["rstd"], s["gamma"], s["dy"], s["dx"], s["dgamma"], s["ws"], dh=s["res"])
        return {k: s[k] for k in ("dx", "dgamma")}
    if c["op"] == "balance":
        score = ep.EP_SCORE_SOFTMAX if c["score"] == "softmax" else ep.EP_SCORE_SIGMOID
        ep.ep_balance_loss(s["logits"], s["idx"], score, s["coef"], s["loss"], s["counts"], s["ws"], s["err"], seq_off=s["seq_off"], prob=s["prob"])
        ep.ep_balance_loss_backward(s["logits"], s["counts"], c["topk"], score, s["coef"], s["dlogits"], seq_off=s["seq_off"], grad_loss=s["grad"])
        return {k: s[k] for k in ("loss", "counts", "prob", "dlogits")}
    act = {"none": ep.EP_ACT_NONE, "silu": ep.EP_ACT_SILU, "gelu": ep.EP_ACT_GELU, "swiglu": ep.EP_ACT_SWIGLU}[c["act"]]
    more = dict(x_scale=s["x_scale"], w_scale=s["w_scale"], bias=s["bias"], residual=s["res"], out_scale=s["out_scale"], act=act)
    if c["groups"]:
        ep.ep_expert_linear(s["buf"], c["tokens"], s["x"], s["w"], s["out"], **more)
    else:
        ep.ep_linear(s["buf"], s["x"], s["w"], s["out"], **more)
    return {k: s[k] for k in ("out", "out_scale")}


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _norm_plain, "norm_backward": _norm_backward_plain, "balance": _balance_plain, "linear": _linear_plain}[state["case"]["op"]](state)


# ---- what a pass cannot do without -------------------------------------------------------


def work(case):
    if case["op"] == "norm":
        n, h = case["rows"], case["hidden"]
        per = 2 + (4 if case["residual"] else 0) + {"bf16": 2, "e4m3": 1 + 4 / 128, "both": 3 + 4 / 128}[case["out"]]
        return dict(bytes=n * h * per + h * (2 if case["gamma"] == "bf16" else 4) + 4 * n, flops=5 * n * h)
    if case["op"] == "norm_backward":
        n, h = case["rows"], case["hidden"]
        return dict(bytes=n * h * (8 if case["residual"] else 6) + 4 * n + h * (6 if case["gamma"] == "bf16" else 8), flops=9 * n * h)
    if case["op"] == "balance":
        n, e, k, q = case["tokens"], case["experts"], case["topk"], case["seqs"]
        return dict(bytes=8 * n * e + 4 * n * k + 8 * q * e, flops=9 * n * e)
    g, t, k, cin, cout = max(1, case["groups"]), case["tokens"], case["topk"], case["cin"], case["cout"]
    rows, wide = t * k, cout * (2 if case["act"] == "swiglu" else 1)
    hit = min(g, rows)  # experts that hold rows, at most
    b = 2 if case["type"] == "bf16" else 1
    size = {"bf16": 2, "fp32": 4, "e4m3": 1 + 4 / 128}[case["out"]]
    more = (4 * hit * wide if case["bias"] else 0) + (2 * rows * cout if case["residual"] else 0)
    scales = (4 * rows * cin // 128 + 4 * hit * wide * cin // 16384) if b == 1 else 0
    return dict(bytes=rows * cin * b + hit * wide * cin * b + rows * cout * size + more + scales, flops=2 * rows * wide * cin)


# ---- definitions in 64 bits -------------------------------------------------------------


def _quantised_exactly(y):
    parts = y.split(128, dim=1)
    scale = torch.stack([torch.clamp(p.abs().max(dim=1).values, min=1e-4) / 448 for p in parts], dim=1)
    q = torch.cat([(p / scale[:, i:i + 1]).clamp(-448, 448) for i, p in enumerate(parts)], dim=1)
    return q.to(F8), scale


def _exact_norm(s, want):
    v = s["x"].double() if s["res"] is None else s["x"].double() + s["res"].double()
    rms = ((v * v).sum(dim=1) / v.shape[1] + s["eps"]).sqrt()
    y = v / rms.unsqueeze(1) * s["gamma"].double().unsqueeze(0)
    q, scale = _quantised_exactly(y) if want != "bf16" else (None, None)
    return dict(h=v if s["res"] is not None else None, y=y if want != "e4m3" else None, q=q, q_scale=scale, rstd=1 / rms)


def _exact_norm_backward(s):
    h, r, dy, gamma = s["x"].double(), s["rstd"].double().unsqueeze(1), s["dy"].double(), s["gamma"].double()
    inner = (dy * gamma * h).sum(dim=1, keepdim=True)
    dx = r * gamma * dy - h * inner * r ** 3 / h.shape[1]
    if s["res"] is not None:
        dx += s["res"].double()
    return dict(dx=dx, dgamma=(dy * h * r).sum(dim=0))


def _exact_balance(s):
    c = s["case"]
    e, k, q = c["experts"], c["topk"], c["seqs"]
    off = s["seq_off"].tolist()
    loss = torch.zeros(1, dtype=torch.float64, device="cuda")
    counts, prob = torch.zeros(q, e, dtype=torch.int32, device="cuda"), torch.zeros(q, e, dtype=torch.float64, device="cuda")
    grads = []
    for i in range(q):
        lo, hi = off[i], off[i + 1]
        if lo == hi:
            continue
        z = s["logits"][lo:hi].double()
        ids = s["idx"][lo:hi]
        n = torch.bincount(ids[ids >= 0].long(), minlength=e)
        f = n.double() * e / (k * (hi - lo))
        if c["score"] == "softmax":
            p = z.softmax(dim=1)
            slope = p
        else:
            sig = z.sigmoid()
            p = sig / sig.sum(dim=1, keepdim=True)
            slope = p * (1 - sig)
        counts[i], prob[i] = n.int(), p.mean(dim=0)
        loss += s["coef"] / q * torch.dot(f, prob[i])
        grads.append(slope * (f - p @ f.unsqueeze(1).expand(-1, 1) * torch.ones_like(f)) * (s["grad"].double() * s["coef"] / q / (hi - lo)))
    return dict(loss=loss, counts=counts, prob=prob, dlogits=torch.cat(grads))


def _exact_linear(s):
    c = s["case"]
    cout, parts, at = c["cout"], [], 0
    for g, n in enumerate(s["counts"].tolist()):
        x, w = s["x"][at:at + n].double(), s["w"][g].double()
        if s["x_scale"] is not None:
            x = x * s["x_scale"][at:at + n].double().repeat_interleave(128, dim=1)
            blocks = -(-cout // 128)
            scale = s["w_scale"][g].double().repeat_interleave(128, dim=1)
            row = torch.arange(w.shape[0], device="cuda")
            w = w * scale[row // cout * blocks + row % cout // 128]
        z = x @ w.t()
        if s["bias"] is not None:
            z += s["bias"][g].double()
        if c["act"] == "swiglu":
            z = torch.nn.functional.silu(z[:, :cout]) * z[:, cout:]
        elif c["act"] == "silu":
            z = torch.nn.functional.silu(z)
        elif c["act"] == "gelu":
            z = torch.nn.functional.gelu(z)
        if s["res"] is not None:
            z += s["res"][at:at + n].double()
        parts.append(z)
        at += n
    y = torch.cat(parts)
    if c["out"] == "e4m3":
        q, scale = _quantised_exactly(y)
        return dict(out=q, out_scale=scale)
    return dict(out=y, out_scale=None)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s, case["out"])
    return {"norm_backward": _exact_norm_backward, "balance": _exact_balance, "linear": _exact_linear}[case["op"]](s)
