"""Workloads of the operators at the end of a packed, adaptively normalised network: the
affine layer norm of the last hidden rows, and the softmax cross entropy over a vocabulary
whose logits (hidden rows times the head's weight) are never kept.

Every case is one pass through one operator. ``own`` chooses between the plain form
(elementary torch operations in fp32) and the library's calls.
"""
import math

import torch

own = False

EPS = 1e-6
IGNORE = -100
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _norm(name, way, dtype, R, D, affine=True):
    return {"name": name, "op": "norm", "way": way, "dtype": dtype, "R": R, "D": D, "affine": affine}


def _loss(name, way, N, V, D, ignored=0.0, zloss=False):
    return {"name": name, "op": "loss", "way": way, "dtype": "bf16", "N": N, "V": V, "D": D,
            "ignored": ignored, "zloss": zloss}


def listed():
    return [
        # One row: the norm of a sampler's single new token.
        _norm("norm-fwd-bf16-1x1536", "fwd", "bf16", 1, 1536),
        # A short ragged batch in training: launch latency and the weight gradient's reduction.
        _norm("norm-train-bf16-257x1152", "train", "bf16", 257, 1152),
        # fp32 rows whose width is no whole number of warps.
        _norm("norm-train-f32-8190x2040", "train", "f32", 8190, 2040),
        # One long video sequence in training.
        _norm("norm-train-bf16-32760x1536", "train", "bf16", 32760, 1536),
        # The same length at a large model's width, inference only.
        _norm("norm-fwd-bf16-32760x5120", "fwd", "bf16", 32760, 5120),
        # The likelihood of one token under a small vocabulary.
        _loss("loss-fwd-1x1000x512", "fwd", 1, 1000, 512),
        # A few tokens in training: one row tile, latency and the weight's bytes.
        _loss("loss-train-96x8192x1024", "train", 96, 8192, 1024),
        # A validation batch: losses only.
        _loss("loss-fwd-4096x32000x1536", "fwd", 4096, 32000, 1536),
        # A large vocabulary on a ragged batch: the vocabulary goes in several pieces.
        _loss("loss-train-1023x131072x1024", "train", 1023, 131072, 1024, zloss=True),
        # Masked-token training: half of the rows carry no loss; odd row and vocabulary counts.
        _loss("loss-train-4095x50257x1536-half", "train", 4095, 50257, 1536, ignored=0.5),
        # A full training batch.
        _loss("loss-train-8192x50257x2048", "train", 8192, 50257, 2048),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.4:
        return {"op": "norm", "way": rng.choice(["fwd", "train"]), "dtype": rng.choice(["bf16", "f32"]),
                "R": _spread(rng, 1, 32760), "D": 8 * _spread(rng, 8, 640),
                "affine": rng.random() < 0.8}
    return {"op": "loss", "way": rng.choice(["fwd", "train", "train"]), "dtype": "bf16",
            "N": _spread(rng, 1, 8192), "V": _spread(rng, 16, 50257), "D": 8 * _spread(rng, 8, 256),
            "ignored": rng.choice([0.0, 0.0, 0.15, 0.5, 0.85]), "zloss": rng.random() < 0.25}


def _active(case):
    return case["N"] - int(case["N"] * case["ignored"])


def work(case):
    if case["op"] == "norm":
        e = 2 if case["dtype"] == "bf16" else 4
        rows, D = case["R"] * case["D"], case["D"]
        nbytes = 2 * rows * e + 8 * case["R"] + (2 * D * e if case["affine"] else 0)
        flops = 8 * rows
        if case["way"] == "train":  # dy read, dx written (x, mean and rstd are at hand); fp32 dweight, dbias
            nbytes += 2 * rows * e + (8 * D if case["affine"] else 0)
            flops += 14 * rows
        return {"bytes": nbytes, "flops": flops}
    N, V, D, n = case["N"], case["V"], case["D"], _active(case)
    nbytes = 2 * (n * D + V * D) + 8 * N + 8 * N
    flops = 2 * n * V * D + 4 * n * V
    if case["way"] == "train":  # dx and dweight written; dloss (and dlse) read
        nbytes += 2 * (N * D + V * D) + 4 * N * (2 if case["zloss"] else 1)
        flops += 4 * n * V * D + 4 * n * V
    return {"bytes": nbytes, "flops": flops}


def _inputs(case, seed):
    """The case's inputs from the seed alone, and nothing of either form."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    dt = DTYPES[case["dtype"]]
    if case["op"] == "norm":
        R, D = case["R"], case["D"]
        # Residual-stream rows: a scale of their own, a shared offset per channel.
        s = {"x": (normal(R, D) * (0.5 + 2 * torch.rand(R, 1, generator=g, device="cuda"))
                   + normal(1, D)).to(dt),
             "weight": None, "bias": None}
        if case["affine"]:
            s["weight"] = (1 + 0.2 * normal(D)).to(dt)
            s["bias"] = (0.1 * normal(D)).to(dt)
        if case["way"] == "train":
            s["dy"] = (0.02 * normal(R, D)).to(dt)
        return s
    N, V, D = case["N"], case["V"], case["D"]
    s = {"x": normal(N, D).to(dt), "weight": (1.5 / math.sqrt(D) * normal(V, D)).to(dt),
         "target": torch.randint(V, (N,), generator=g, device="cuda", dtype=torch.int64)}
    n = _active(case)
    if n < N:
        s["target"][torch.randperm(N, generator=g, device="cuda")[n:]] = IGNORE
    if case["way"] == "train":
        # A mean over the rows that count, each with a weight of its own (as a noise level gives).
        s["dloss"] = (0.5 + 1.5 * torch.rand(N, generator=g, device="cuda")) / max(n, 1)
        s["dlse"] = 1e-2 * normal(N) / max(n, 1) if case["zloss"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if not own:
        return s
    import adaln_layernorm_modulate_gb300 as A

    def f32(*shape):
        return torch.empty(*shape, dtype=torch.float32, device="cuda")

    x, dt = s["x"], A.ADALN_BF16 if case["dtype"] == "bf16" else A.ADALN_F32
    nb = 0
    if case["op"] == "norm":
        R, D = case["R"], case["D"]
        s["y"], s["mean"], s["rstd"] = torch.empty_like(x), f32(R), f32(R)
        if case["way"] == "train":
            s["dx"] = torch.empty_like(x)
            s["dweight"], s["dbias"] = (f32(D), f32(D)) if case["affine"] else (None, None)
            nb = A.adaln_layernorm_bwd_workspace_size(R, D, dt)
    else:
        N, V, D = case["N"], case["V"], case["D"]
        s["loss"], s["lse"] = f32(N), f32(N)
        nb = A.adaln_linear_xent_fwd_workspace_size(N, V, D, dt)
        if case["way"] == "train":
            s["dx"], s["dweight"] = torch.empty_like(x), torch.empty_like(s["weight"])
            nb = max(nb, A.adaln_linear_xent_bwd_workspace_size(N, V, D, dt))
    s["workspace"], s["workspace_bytes"] = torch.empty(nb, dtype=torch.uint8, device="cuda"), nb
    return s


def run(state):
    if state["case"]["op"] == "norm":
        return _norm_own(state) if own else _norm_plain(state)
    return _loss_own(state) if own else _loss_plain(state)


def _norm_plain(s):
    x = s["x"].float()
    D = x.shape[1]
    mean = x.sum(1) / D
    d = x - mean[:, None]
    rstd = 1 / torch.sqrt((d * d).sum(1) / D + EPS)
    xhat = d * rstd[:, None]
    y = xhat
    if s["weight"] is not None:
        y = xhat * s["weight"].float() + s["bias"].float()
    out = {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}
    if "dy" in s:
        dy = s["dy"].float()
        g = dy if s["weight"] is None else dy * s["weight"].float()
        m1 = g.sum(1, keepdim=True) / D
        m2 = (g * xhat).sum(1, keepdim=True) / D
        out["dx"] = (rstd[:, None] * (g - m1 - xhat * m2)).to(s["x"].dtype)
        if s["weight"] is not None:
            out["dweight"], out["dbias"] = (dy * xhat).sum(0), dy.sum(0)
    return out


def _norm_own(s):
    import adaln_layernorm_modulate_gb300 as A
    R, D = s["case"]["R"], s["case"]["D"]
    A.adaln_layernorm_fwd(s["x"], s["weight"], s["bias"], s["y"], s["mean"], s["rstd"], R, D, EPS)
    out = {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    if "dy" in s:
        A.adaln_layernorm_bwd(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"], s["dx"], s["dweight"],
                              s["dbias"], s["workspace"], s["workspace_bytes"], R, D)
        out["dx"] = s["dx"]
        if s["weight"] is not None:
            out["dweight"], out["dbias"] = s["dweight"], s["dbias"]
    return out


def _loss_plain(s):
    x, w, target = s["x"].float(), s["weight"].float(), s["target"]
    counts = target != IGNORE
    rows = torch.arange(x.shape[0], device=x.device)
    column = torch.where(counts, target, torch.zeros_like(target))
    logits = x @ w.t()
    top = logits.max(1).values
    lse = top + torch.log(torch.exp(logits - top[:, None]).sum(1))
    loss = lse - logits[rows, column]
    zero = torch.zeros_like(lse)
    out = {"loss": torch.where(counts, loss, zero), "lse": torch.where(counts, lse, zero)}
    if "dloss" in s:
        dloss = torch.where(counts, s["dloss"], zero)
        dlse = zero if s["dlse"] is None else torch.where(counts, s["dlse"], zero)
        d = torch.exp(logits - lse[:, None]) * (dloss + dlse)[:, None]
        d[rows, column] -= dloss
        out["dx"] = (d @ w).to(s["x"].dtype)
        out["dweight"] = (d.t() @ x).to(s["weight"].dtype)
    return out


def _loss_own(s):
    import adaln_layernorm_modulate_gb300 as A
    N, V, D = s["case"]["N"], s["case"]["V"], s["case"]["D"]
    A.adaln_linear_xent_fwd(s["x"], s["weight"], s["target"], s["loss"], s["lse"], N, V, D, IGNORE,
                            s["workspace"], s["workspace_bytes"])
    out = {"loss": s["loss"], "lse": s["lse"]}
    if "dloss" in s:
        A.adaln_linear_xent_bwd(s["x"], s["weight"], s["target"], s["lse"], s["dloss"], s["dlse"], s["dx"],
                                s["dweight"], N, V, D, IGNORE, s["workspace"], s["workspace_bytes"])
        out["dx"], out["dweight"] = s["dx"], s["dweight"]
    return out


def exact(case, seed):
    """The definitions in 64 bits, a block of rows at a time."""
    s = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v
         for k, v in _inputs(case, seed).items()}
    if case["op"] == "norm":
        x, D = s["x"], case["D"]
        var, mean = torch.var_mean(x, dim=1, correction=0)
        std = torch.sqrt(var + EPS)
        gain = s["weight"] if case["affine"] else torch.ones(D, dtype=x.dtype, device=x.device)
        xhat = (x - mean.unsqueeze(1)) / std.unsqueeze(1)
        out = {"y": xhat * gain + (s["bias"] if case["affine"] else 0), "mean": mean, "rstd": 1 / std}
        if case["way"] == "train":
            # The Jacobian of a standardised row is (I - 11'/D - xhat xhat'/D) / std.
            v = s["dy"] * gain
            v = v - xhat * torch.einsum("rd,rd->r", v, xhat).div(D).unsqueeze(1) - v.mean(1, keepdim=True)
            out["dx"] = v / std.unsqueeze(1)
            if case["affine"]:
                out["dweight"] = torch.einsum("rd,rd->d", s["dy"], xhat)
                out["dbias"] = s["dy"].sum(0)
        return out
    N, x, w, target = case["N"], s["x"], s["weight"], s["target"]
    out = {"loss": x.new_zeros(N), "lse": x.new_zeros(N)}
    train = case["way"] == "train"
    if train:
        out["dx"], out["dweight"] = torch.zeros_like(x), torch.zeros_like(w)
    keep = torch.nonzero(target != IGNORE).squeeze(1)
    for rows in keep.split(2048):
        h, t = x[rows], target[rows]
        z = torch.mm(h, w.t())
        lse = torch.logsumexp(z, dim=1)
        out["lse"][rows] = lse
        out["loss"][rows] = lse - z.gather(1, t.unsqueeze(1)).squeeze(1)
        if train:
            up = s["dloss"][rows]
            both = up if s["dlse"] is None else up + s["dlse"][rows]
            z = z.sub_(lse.unsqueeze(1)).exp_().mul_(both.unsqueeze(1))
            z.scatter_add_(1, t.unsqueeze(1), -up.unsqueeze(1))
            out["dx"][rows] = torch.mm(z, w)
            out["dweight"] += torch.mm(z.t(), h)
    return out
