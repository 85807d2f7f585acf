"""The operators' measured cases, their plain forms and their definition in 64 bits.

Two families:

* ``ce_*``: softmax cross entropy of hidden rows against a large vocabulary with
  the output projection inside (logits ``hidden @ W.T / T`` are not an input and
  not an output).  ``ce_score`` gives the loss, the row losses and the
  log-sum-exps; ``ce_train`` the loss and the gradients of hidden and W in one
  call; ``ce_rows`` the row losses and then the gradients for a given upstream
  gradient per row.
* ``norm_*``: the norms after and before a block, its gate and its residual
  scale in one pass over the rows: ``u = norm(block) * post``,
  ``v = x + scale * gate * u``, ``y = norm(v) * pre``, and the gradients.

``own`` selects the calls of this repository's operators; without it ``run``
computes the plain form in 32 bits.
"""
import math

import torch

own = False

IGNORE = -100
W_STD = 0.02      # spread of the output projection's entries


# ---------------------------------------------------------------- cases
def _ce(name, op, N, H, V, ignored=0.0, smooth=0.0, z=0.0, T=1.0, weighted=False, reduction="mean"):
    return {"name": name, "op": op, "N": N, "H": H, "V": V, "ignored": ignored, "smooth": smooth,
            "z": z, "T": T, "weighted": weighted, "reduction": reduction}


def _norm(name, op, N, H, post=True, gate=False, pre=True, dv=True, x32=False, w32=False,
          dy32=False, scale=1.0, offset=0.0):
    return {"name": name, "op": op, "N": N, "H": H, "post": post, "gate": gate, "pre": pre,
            "dv": dv, "x32": x32, "w32": w32, "dy32": dy32, "scale": scale, "offset": offset}


def listed():
    return [
        # one token scored against a full vocabulary (serving: the log-probability of a forced token)
        _ce("ce_score_one_token", "ce_score", 1, 4096, 128256),
        # a prompt scored for its perplexity, part of it template text that does not count
        _ce("ce_score_prompt", "ce_score", 8192, 4096, 128256, ignored=0.2),
        # the smallest training step: launch latency counts
        _ce("ce_train_tiny", "ce_train", 256, 256, 4096),
        # an ordinary step of a small student: odd row count and vocabulary, smoothing, summed
        _ce("ce_train_odd", "ce_train", 1531, 1024, 50257, ignored=0.1, smooth=0.1, reduction="sum"),
        # instruction tuning at the widest vocabulary: ragged H tiles, a third of the rows ignored, z-loss
        _ce("ce_train_wide_vocab", "ce_train", 4096, 2880, 201088, ignored=0.35, z=1e-4),
        # the largest step: several chunks of rows, weighted rows
        _ce("ce_train_large", "ce_train", 16384, 4096, 128256, ignored=0.05, weighted=True),
        # token log-probabilities and their gradient for a policy objective
        _ce("ce_rows_policy", "ce_rows", 2048, 2048, 128256, ignored=0.25, T=1.25),
        # single-token decode between two blocks
        _norm("norm_fwd_one_token", "norm_fwd", 1, 4096, gate=True, scale=0.22),
        # a prefill or training forward of one block boundary
        _norm("norm_fwd_rows", "norm_fwd", 16384, 4096, gate=True, scale=0.22),
        # the last norm before the head: no post-norm, 32-bit residual stream, ragged rows
        _norm("norm_bwd_last", "norm_bwd", 4001, 2880, post=False, dv=False, x32=True, w32=True, dy32=True),
        # a small batch's backward at a block boundary
        _norm("norm_bwd_small", "norm_bwd", 300, 1024, gate=True, w32=True, offset=1.0),
        # the backward of a long batch at a block boundary
        _norm("norm_bwd_rows", "norm_bwd", 16384, 4096, gate=True, scale=0.22),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ce_score", "ce_train", "ce_rows", "norm_fwd", "norm_bwd"])
    if op.startswith("ce"):
        while True:
            N = _log_uniform(rng, 1, 16384)
            H = 8 * _log_uniform(rng, 8, 512)
            V = _log_uniform(rng, 300, 201088)
            if N * H * V <= 16384 * 4096 * 128256 and N * V <= 16384 * 128256:
                break
        c = _ce("", op, N, H, V, ignored=rng.choice([0.0, 0.05, 0.3, 0.6]),
                smooth=rng.choice([0.0, 0.0, 0.1]), z=rng.choice([0.0, 0.0, 1e-4]),
                T=rng.choice([1.0, 1.0, 0.7, 2.0]), weighted=rng.random() < 0.3,
                reduction=rng.choice(["mean", "sum"]))
        if op == "ce_rows":
            c["weighted"] = False
    else:
        while True:
            N = _log_uniform(rng, 1, 65536)
            H = 8 * _log_uniform(rng, 8, 1024)
            if N * H <= 16384 * 4096:
                break
        post, pre = rng.choice([(True, True), (False, True), (True, False), (True, True)])
        c = _norm("", op, N, H, post=post, gate=rng.random() < 0.5, pre=pre,
                  dv=rng.random() < 0.6 or not pre, x32=rng.random() < 0.3,
                  w32=rng.random() < 0.5, dy32=rng.random() < 0.3,
                  scale=rng.choice([1.0, 0.22, 0.5]), offset=rng.choice([0.0, 1.0]))
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    N, H = case["N"], case["H"]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=dev) * std

    s = {"case": case}
    if case["op"].startswith("ce"):
        V = case["V"]
        W = normal(V, H, std=W_STD).bfloat16()
        labels = torch.randint(0, V, (N,), generator=g, device=dev)
        # a student that has learned something: the label's logit stands out by 0 to 12
        lift = torch.rand(N, 1, generator=g, device=dev) * (12.0 / (W_STD * W_STD * H))
        hidden = (normal(N, H) + lift * W[labels].float()).bfloat16()
        drop = torch.rand(N, generator=g, device=dev) < case["ignored"]
        drop[0] = False
        s |= {"W": W, "hidden": hidden, "labels": torch.where(drop, IGNORE, labels)}
        if case["weighted"]:
            s["weight"] = torch.rand(N, generator=g, device=dev) + 0.5
        if case["op"] == "ce_rows":
            s["row_grad"] = normal(N) / N      # advantages: either sign
    else:
        xt = torch.float32 if case["x32"] else torch.bfloat16
        wt = torch.float32 if case["w32"] else torch.bfloat16
        around = 1.0 - case["offset"]
        s["x"] = (normal(N, H) * 2.0).to(xt)
        s["block"] = normal(N, H, std=0.7).bfloat16()
        if case["post"]:
            s["post"] = (around + normal(H, std=0.1)).to(wt)
        if case["gate"]:
            s["gate"] = normal(H, std=0.5).to(wt)
        if case["pre"]:
            s["pre"] = (around + normal(H, std=0.1)).to(wt)
        if case["op"] == "norm_bwd":
            if case["pre"]:
                s["dy"] = normal(N, H, std=1e-2).to(torch.float32 if case["dy32"] else torch.bfloat16)
            if case["dv"]:
                s["dv"] = normal(N, H, std=1e-2).to(xt)
    return s


# ---------------------------------------------------------------- plain forms
def _plain_ce(s):
    c, op = s["case"], s["case"]["op"]
    h, W, labels = s["hidden"].float(), s["W"].float(), s["labels"]
    V, eps, lam, T = c["V"], c["smooth"], c["z"], c["T"]
    valid = labels != IGNORE
    at = torch.where(valid, labels, 0)[:, None]
    a = (h @ W.t()) / T
    top = a.amax(1, keepdim=True)
    e = torch.exp(a - top)
    total = e.sum(1, keepdim=True)
    lse = top + torch.log(total)
    row = lse - (1 - eps) * a.gather(1, at) + lam * lse * lse
    if eps:
        row = row - eps * a.mean(1, keepdim=True)
    row_loss = torch.where(valid, row[:, 0], 0.0)
    lse_out = torch.where(valid, lse[:, 0], 0.0)
    count = valid.sum()
    share = 1.0 / torch.clamp(count, min=1).float() if c["reduction"] == "mean" else 1.0
    weight = s.get("weight")
    loss = ((row_loss if weight is None else row_loss * weight).sum() * share).reshape(1)
    if op == "ce_score":
        return {"loss": loss, "row_loss": row_loss, "lse": lse_out}
    if op == "ce_rows":
        k = s["row_grad"]
    else:
        k = share if weight is None else weight * share
    k = torch.where(valid, k, 0.0)[:, None]
    del a
    G = e.mul_((1 + 2 * lam * lse) / total)
    if eps:
        G -= eps / V
    G.scatter_add_(1, at, torch.full_like(lse, -(1 - eps)))
    G *= k / T
    dH, dW = (G @ W).bfloat16(), (G.t() @ h).bfloat16()
    if op == "ce_rows":
        return {"row_loss": row_loss, "dH": dH, "dW": dW}
    return {"loss": loss, "row_loss": row_loss, "dH": dH, "dW": dW}


NORM_EPS = 1e-6


def _plain_norm(s):
    c = s["case"]
    off, scale = c["offset"], c["scale"]
    x, b = s["x"].float(), s["block"].float()
    post = s["post"].float() + off if c["post"] else None
    gate = s["gate"].float() if c["gate"] else None
    pre = s["pre"].float() + off if c["pre"] else None
    u = b
    if c["post"]:
        rb = torch.rsqrt((b * b).mean(1, keepdim=True) + NORM_EPS)
        bn = b * rb
        u = bn * post
    v = x + scale * (u * gate if c["gate"] else u)
    if c["pre"]:
        rv = torch.rsqrt((v * v).mean(1, keepdim=True) + NORM_EPS)
        vn = v * rv
    if c["op"] == "norm_fwd":
        out = {"v": v.to(s["x"].dtype)}
        if c["pre"]:
            out["y"] = (vn * pre).bfloat16()
        return out
    out = {}
    dv = s["dv"].float() if c["dv"] else 0.0
    if c["pre"]:
        dy = s["dy"].float()
        t = dy * pre
        dv = dv + rv * (t - vn * (vn * t).mean(1, keepdim=True))
        out["dpre"] = (dy * vn).sum(0)
    out["dx"] = dv.to(s["x"].dtype)
    du = scale * dv
    if c["gate"]:
        out["dgate"] = (du * u).sum(0)
        du = du * gate
    if c["post"]:
        out["dpost"] = (du * bn).sum(0)
        t = du * post
        du = rb * (t - bn * (bn * t).mean(1, keepdim=True))
    out["dblock"] = du.bfloat16()
    return out


# ---------------------------------------------------------------- the framework's calls
def _own_ce(s):
    from chunked_kl_loss_tcgen05_b200.torch_api import fused_ce_bwd, fused_ce_fwd, fused_ce_fwd_bwd
    c = s["case"]
    kw = dict(T=c["T"], label_smoothing=c["smooth"], z_loss=c["z"], ignore_index=IGNORE, check=False)
    h, W, labels = s["hidden"], s["W"], s["labels"]
    if c["op"] == "ce_score":
        loss, row_loss, lse = fused_ce_fwd(h, W, labels, row_weight=s.get("weight"),
                                           reduction=c["reduction"], **kw)
        return {"loss": loss, "row_loss": row_loss, "lse": lse}
    if c["op"] == "ce_train":
        loss, row_loss, dH, dW = fused_ce_fwd_bwd(h, W, labels, row_weight=s.get("weight"),
                                                  reduction=c["reduction"],
                                                  grad_dtype=torch.bfloat16, **kw)
        return {"loss": loss, "row_loss": row_loss, "dH": dH, "dW": dW}
    _, row_loss, lse = fused_ce_fwd(h, W, labels, reduction="sum", **kw)
    dH, dW = fused_ce_bwd(h, W, labels, lse, s["row_grad"], grad_dtype=torch.bfloat16, **kw)
    return {"row_loss": row_loss, "dH": dH, "dW": dW}


def _own_norm(s):
    from chunked_kl_loss_tcgen05_b200.torch_api import block_norm_bwd, block_norm_fwd
    c = s["case"]
    kw = dict(post_weight=s.get("post"), gate=s.get("gate"), pre_weight=s.get("pre"),
              scale=c["scale"], post=c["post"], pre=c["pre"], eps=NORM_EPS,
              weight_offset=c["offset"])
    if c["op"] == "norm_fwd":
        v, y = block_norm_fwd(s["x"], s["block"], **kw)
        return {"v": v, "y": y} if c["pre"] else {"v": v}
    dx, dblock, dpost, dgate, dpre = block_norm_bwd(s["x"], s["block"], dy=s.get("dy"),
                                                    dv=s.get("dv"), **kw)
    out = {"dx": dx, "dblock": dblock, "dpost": dpost, "dgate": dgate, "dpre": dpre}
    return {k: t for k, t in out.items() if t is not None}


def run(state):
    if state["case"]["op"].startswith("ce"):
        return _own_ce(state) if own else _plain_ce(state)
    return _own_norm(state) if own else _plain_norm(state)


# ---------------------------------------------------------------- what a pass needs
def work(case):
    N, H = case["N"], case["H"]
    if case["op"].startswith("ce"):
        V = case["V"]
        n = max(1.0, N * (1.0 - case["ignored"]))
        if case["op"] == "ce_score":
            return {"bytes": 2 * (n * H + V * H) + 16 * N, "flops": 2 * n * H * V}
        return {"bytes": 4 * (n * H + V * H) + 16 * N, "flops": 6 * n * H * V}
    xb = 4 if case["x32"] else 2
    if case["op"] == "norm_fwd":
        per = 2 * xb + 2 + (2 if case["pre"] else 0)
        return {"bytes": per * N * H, "flops": 10 * N * H}
    per = 2 * xb + 4 + (xb if case["dv"] else 0)
    if case["pre"]:
        per += 4 if case["dy32"] else 2
    return {"bytes": per * N * H, "flops": 30 * N * H}


# ---------------------------------------------------------------- 64 bits
def _exact_ce(s):
    """l = -sum_v t_v log q_v + z log(Z)^2 with the smoothed target t; rows in blocks."""
    c, op = s["case"], s["case"]["op"]
    N, V, T = c["N"], c["V"], c["T"]
    W64 = s["W"].double()
    keep = (s["labels"] != IGNORE).nonzero()[:, 0]
    denom = float(max(1, keep.numel())) if c["reduction"] == "mean" else 1.0
    f64 = dict(dtype=torch.float64, device=W64.device)
    losses, lses = torch.zeros(N, **f64), torch.zeros(N, **f64)
    dH = torch.zeros(N, c["H"], **f64)
    dW = torch.zeros(V, c["H"], **f64)
    coef = torch.ones(N, **f64)
    if c["weighted"]:
        coef = s["weight"].double()
    step = max(1, 200_000_000 // V)
    for i in range(0, keep.numel(), step):
        rows = keep[i:i + step]
        h = s["hidden"][rows].double()
        z = torch.mm(h, W64.t()).div_(T)
        logZ = torch.logsumexp(z, 1)
        logq = z.sub_(logZ[:, None])
        y = s["labels"][rows]
        picked = logq[torch.arange(len(rows), device=y.device), y]
        losses[rows] = -(1 - c["smooth"]) * picked - c["smooth"] * logq.mean(1) + c["z"] * logZ ** 2
        lses[rows] = logZ
        if op == "ce_score":
            continue
        up = s["row_grad"].double()[rows] if op == "ce_rows" else coef[rows] / denom
        D = logq.exp_() * (1 + 2 * c["z"] * logZ)[:, None] - c["smooth"] / V
        D[torch.arange(len(rows), device=y.device), y] -= 1 - c["smooth"]
        D *= up[:, None] / T
        dH[rows] = D @ W64
        dW.addmm_(D.t(), h)
    loss = (coef * losses).sum().div(denom).reshape(1)
    if op == "ce_score":
        return {"loss": loss, "row_loss": losses, "lse": lses}
    if op == "ce_rows":
        return {"row_loss": losses, "dH": dH, "dW": dW}
    return {"loss": loss, "row_loss": losses, "dH": dH, "dW": dW}


def _exact_norm(s):
    """The forward in 64 bits, and its gradients by differentiation."""
    c = s["case"]
    bwd = c["op"] == "norm_bwd"
    t = {k: s[k].double().requires_grad_(bwd) for k in ("x", "block", "post", "gate", "pre") if k in s}
    u = t["block"]
    if c["post"]:
        u = u / (u.square().mean(-1, keepdim=True) + NORM_EPS).sqrt() * (t["post"] + c["offset"])
    if c["gate"]:
        u = t["gate"] * u
    v = t["x"] + c["scale"] * u
    y = None
    if c["pre"]:
        y = v / (v.square().mean(-1, keepdim=True) + NORM_EPS).sqrt() * (t["pre"] + c["offset"])
    if not bwd:
        return {"v": v, "y": y} if c["pre"] else {"v": v}
    total = 0.0
    if c["pre"]:
        total = total + (y * s["dy"].double()).sum()
    if c["dv"]:
        total = total + (v * s["dv"].double()).sum()
    names = list(t)
    grads = torch.autograd.grad(total, [t[k] for k in names])
    return {"d" + k: g for k, g in zip(names, grads)}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_ce(s) if case["op"].startswith("ce") else _exact_norm(s)
