"""Workloads of the self-attention between two adaptively normalised blocks: the norms of queries
and keys for each head with their rotation by positions of several axes (time, height, width), and
softmax attention over packed sequences of different lengths, with grouped heads, causal or not.

Every case is one pass through one operator. ``own`` chooses between the plain form
(elementary torch operations in fp32) and the library's calls.
"""
import math

import torch

own = False

EPS = 1e-6
THETA = 10000.0
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _rope(name, way, dtype, R, Hq, Hk, d, axes, start=0):
    return {"name": name, "op": "rope", "way": way, "dtype": dtype, "R": R, "Hq": Hq, "Hk": Hk, "d": d,
            "axes": axes, "start": start}


def _attn(name, way, lens_q, lens_k, Hq, Hk, d, causal=False):
    return {"name": name, "op": "attn", "way": way, "dtype": "bf16", "lens_q": lens_q, "lens_k": lens_k,
            "Hq": Hq, "Hk": Hk, "d": d, "causal": causal}


def _packed(*runs):
    return " ".join(" ".join([str(n)] * times) for n, times in runs)


MIXED = _packed((256, 32), (1024, 8), (4096, 2))
ODD = "4095 2049 1 1001 513 77 8191"


def listed():
    return [
        # One new token of a sampler.
        _rope("rope-fwd-bf16-1x12x128", "fwd", "bf16", 1, 12, 12, 128, "44 42 42", start=4096),
        # A short ragged batch of images in training, heads of an odd width, keys in groups.
        _rope("rope-train-bf16-257x16x72", "train", "bf16", 257, 16, 4, 72, "36 36"),
        # fp32 activations, one axis, positions far out; part of each head is not rotated.
        _rope("rope-train-f32-8190x8x64", "train", "f32", 8190, 8, 8, 64, "48", start=500000),
        # One long video sequence in training.
        _rope("rope-train-bf16-32760x12x128", "train", "bf16", 32760, 12, 12, 128, "44 42 42"),
        # The same length at a large model's width, inference only.
        _rope("rope-fwd-bf16-32760x40x128", "fwd", "bf16", 32760, 40, 40, 128, "44 42 42"),
        # A few short captions in training: latency counts.
        _attn("attn-train-causal-short", "train", "17 0 130 5 1", "17 0 130 5 1", 4, 2, 64, causal=True),
        # One query that reads a whole video (attention pooling, a new token over a long cache).
        _attn("attn-fwd-1-over-32760", "fwd", "1", "32760", 12, 12, 128),
        # Video rows that attend to a text's 512 rows, in training.
        _attn("attn-train-32760-over-512", "train", "32760", "512", 12, 12, 128),
        # Packed buckets of several lengths in training.
        _attn("attn-train-packed-24576x12x128", "train", MIXED, MIXED, 12, 12, 128),
        # Text of ragged lengths, causal, grouped heads, in training.
        _attn("attn-train-causal-15927x16x64", "train", ODD, ODD, 16, 4, 64, causal=True),
        # A long sequence in training.
        _attn("attn-train-16384x12x128", "train", "16384", "16384", 12, 12, 128),
        # One long video sequence, inference only.
        _attn("attn-fwd-32760x12x128", "fwd", "32760", "32760", 12, 12, 128),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _split(rng, d):
    """Up to three even widths of axes within a head of d elements."""
    n, left, axes = rng.randint(1, 3), d, []
    for i in range(n):
        w = 2 * rng.randint(1, max(1, (left - 2 * (n - 1 - i)) // 2)) if rng.random() < 0.3 else left // (n - i) // 2 * 2
        axes.append(max(w, 2))
        left -= axes[-1]
    return " ".join(str(w) for w in axes)


def draw(rng):
    if rng.random() < 0.4:
        way, d = rng.choice(["fwd", "train"]), 8 * rng.randint(2, 16)
        Hq = _spread(rng, 1, 16 if way == "train" else 40)
        return {"op": "rope", "way": way, "dtype": rng.choice(["bf16", "f32"]), "R": _spread(rng, 1, 32760),
                "Hq": Hq, "Hk": rng.randint(1, Hq), "d": d, "axes": _split(rng, d),
                "start": _spread(rng, 1, 1 << 20)}
    way, causal = rng.choice(["fwd", "train", "train"]), rng.random() < 0.4
    Hk, group = rng.randint(1, 4), rng.choice([1, 1, 2, 4])
    d = rng.choice([32, 64, 72, 80, 96, 128, 128])
    longest, rows, lens_q, lens_k = _spread(rng, 16, 8192), 0, [], []
    for _ in range(_spread(rng, 1, 40)):
        nq = _spread(rng, 1, longest)
        nk = nq if causal or rng.random() < 0.7 else _spread(rng, 1, longest)
        if rows + max(nq, nk) > 20000:
            break
        rows += max(nq, nk)
        lens_q.append(str(nq))
        lens_k.append(str(nk))
    return {"op": "attn", "way": way, "dtype": "bf16", "lens_q": " ".join(lens_q), "lens_k": " ".join(lens_k),
            "Hq": Hk * group, "Hk": Hk, "d": d, "causal": causal}


def _lens(case, which):
    return [int(n) for n in case[which].split()]


def _axes(case):
    return [int(w) for w in case["axes"].split()]


def work(case):
    Hq, Hk, d = case["Hq"], case["Hk"], case["d"]
    if case["op"] == "rope":
        e = 2 if case["dtype"] == "bf16" else 4
        n = case["R"] * (Hq + Hk) * d
        nbytes, flops = 2 * n * e + 4 * case["R"] * len(_axes(case)) + 2 * d * e, 7 * n
        if case["way"] == "train":  # the outputs' gradients read, dq and dk written (q and k are at hand)
            nbytes += 2 * n * e + 8 * d
            flops += 14 * n
        return {"bytes": nbytes, "flops": flops}
    lq, lk = _lens(case, "lens_q"), _lens(case, "lens_k")
    pairs = sum(n * (n + 1) // 2 if case["causal"] else n * m for n, m in zip(lq, lk))
    q, k = sum(lq) * Hq * d, sum(lk) * Hk * d
    nbytes, flops = 2 * (2 * q + 2 * k) + 4 * sum(lq) * Hq, 4 * pairs * Hq * d
    if case["way"] == "train":  # dout read; dq, dk and dv written
        nbytes += 2 * (2 * q + 2 * k)
        flops += 10 * pairs * Hq * d
    return {"bytes": nbytes, "flops": flops}


def _inputs(case, seed):
    """The case's inputs from the seed alone, and nothing of either form. Queries, keys and values
    are parts of the rows of a joint projection where they have the same rows."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    dt, Hq, Hk, d = DTYPES[case["dtype"]], case["Hq"], case["Hk"], case["d"]
    if case["op"] == "rope":
        R = case["R"]
        # Projected rows: a scale of their own, a shared offset a channel.
        rows = (normal(R, (Hq + 2 * Hk) * d) * (0.5 + 2 * torch.rand(R, 1, generator=g, device="cuda"))
                + 0.3 * normal(1, (Hq + 2 * Hk) * d)).to(dt)
        s = {"q": rows[:, : Hq * d].view(R, Hq, d), "k": rows[:, Hq * d: (Hq + Hk) * d].view(R, Hk, d),
             "q_weight": (1 + 0.2 * normal(d)).to(dt), "k_weight": (1 + 0.2 * normal(d)).to(dt)}
        # Positions on a grid (time; rows of 30; columns of 52), row by row.
        i, n = torch.arange(R, device="cuda"), len(_axes(case))
        grid = [i // 1560, i // 52 % 30, i % 52] if n == 3 else [i // 52, i % 52] if n == 2 else [i]
        s["pos"] = (torch.stack(grid, 1) + case["start"]).to(torch.int32)
        if case["way"] == "train":
            s["dq_out"], s["dk_out"] = (0.02 * normal(R, Hq, d)).to(dt), (0.02 * normal(R, Hk, d)).to(dt)
        return s
    lq, lk = _lens(case, "lens_q"), _lens(case, "lens_k")
    Rq, Rk = sum(lq), sum(lk)
    # Normalised queries and keys whose products spread over a few units, rows of values. Keys lie near a
    # direction of their own sequence, so that queries weigh them unevenly.
    q = (1.4 * normal(Rq, Hq, d)).to(dt)
    k = (1.0 * normal(Rk, Hk, d) + 0.4 * normal(1, Hk, d)).to(dt)
    if lq == lk:
        v = normal(Rk, (Hq + 2 * Hk) * d).to(dt)[:, (Hq + Hk) * d:].view(Rk, Hk, d)
    else:
        v = normal(Rk, 2 * Hk * d).to(dt)[:, Hk * d:].view(Rk, Hk, d)
    cu = [torch.tensor([0] + x, device="cuda").cumsum(0).to(torch.int32) for x in (lq, lk)]
    s = {"q": q, "k": k, "v": v, "cu_q": cu[0], "cu_k": cu[1]}
    if case["way"] == "train":
        s["dout"] = (0.02 * normal(Rq, Hq, d)).to(dt)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if not own:
        return s
    import adaln_layernorm_modulate_gb300 as A

    def fresh(t):
        return torch.empty(t.shape, dtype=t.dtype, device="cuda")

    Hq, Hk, d = case["Hq"], case["Hk"], case["d"]
    dt = A.ADALN_BF16 if case["dtype"] == "bf16" else A.ADALN_F32
    nb = 0
    if case["op"] == "rope":
        s["q_out"], s["k_out"] = fresh(s["q"]), fresh(s["k"])
        if case["way"] == "train":
            s["dq"], s["dk"] = fresh(s["q"]), fresh(s["k"])
            s["dq_weight"], s["dk_weight"] = (torch.empty(d, device="cuda") for _ in range(2))
            nb = A.adaln_qk_norm_rope_bwd_workspace_size(case["R"], Hq, Hk, d, dt)
    else:
        Rq, Rk, nseg = s["q"].shape[0], s["k"].shape[0], s["cu_q"].numel() - 1
        s["o"], s["lse"] = fresh(s["q"]), torch.empty(Hq, Rq, device="cuda")
        nb = A.adaln_attention_fwd_workspace_size(nseg, Rq, Rk, Hq, Hk, d, dt)
        if case["way"] == "train":
            s["dq"], s["dk"], s["dv"] = fresh(s["q"]), fresh(s["k"]), fresh(s["v"])
            nb = max(nb, A.adaln_attention_bwd_workspace_size(nseg, Rq, Rk, Hq, Hk, d, dt))
    s["workspace"], s["workspace_bytes"] = torch.empty(nb, dtype=torch.uint8, device="cuda"), nb
    return s


def run(state):
    if state["case"]["op"] == "rope":
        return _rope_own(state) if own else _rope_plain(state)
    return _attn_own(state) if own else _attn_plain(state)


def _turns(s, width):
    """cos and sin of the angles of every pair of a head, [R, 1, pairs]: the angles in 64 bits."""
    case, angles = s["case"], []
    for a, w in enumerate(_axes(case)):
        i = torch.arange(w // 2, device="cuda", dtype=torch.float64)
        angles.append(s["pos"][:, a: a + 1].double() * torch.exp(-2 * i / w * math.log(THETA)))
    rest = (width - sum(_axes(case))) // 2
    angles.append(torch.zeros(s["pos"].shape[0], rest, device="cuda", dtype=torch.float64))
    angle = torch.cat(angles, 1).unsqueeze(1)
    return torch.cos(angle).float(), torch.sin(angle).float()


def _turn(x, c, s):
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)


def _rope_plain(s):
    d = s["case"]["d"]
    cos, sin = _turns(s, d)
    out = {}
    for n in ("q", "k"):
        x, w = s[n].float(), s[n + "_weight"].float()
        rstd = 1 / torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS)
        xhat = x * rstd
        out[n + "_out"] = _turn(xhat * w, cos, sin).to(s[n].dtype)
        if "dq_out" in s:
            dy = _turn(s["d" + n + "_out"].float(), cos, -sin)
            g = dy * w
            out["d" + n] = (rstd * (g - xhat * ((g * xhat).sum(-1, keepdim=True) / d))).to(s[n].dtype)
            out["d" + n + "_weight"] = (dy * xhat).sum((0, 1))
    return out


def _rope_own(s):
    import adaln_layernorm_modulate_gb300 as A
    c = s["case"]
    R, Hq, Hk, d = c["R"], c["Hq"], c["Hk"], c["d"]
    axes = _axes(c)
    ld = s["q"].stride(0)
    A.adaln_qk_norm_rope_fwd(s["q"], s["k"], s["q_weight"], s["k_weight"], s["pos"], s["q_out"], s["k_out"],
                             R, Hq, Hk, d, ld, ld, Hq * d, Hk * d, axes, THETA, EPS)
    out = {n: s[n] for n in ("q_out", "k_out")}
    if "dq_out" in s:
        A.adaln_qk_norm_rope_bwd(s["dq_out"], s["dk_out"], s["q"], s["k"], s["q_weight"], s["k_weight"], s["pos"],
                                 s["dq"], s["dk"], s["dq_weight"], s["dk_weight"], s["workspace"],
                                 s["workspace_bytes"], R, Hq, Hk, d, Hq * d, Hk * d, ld, ld, Hq * d, Hk * d,
                                 axes, THETA, EPS)
        out.update({n: s[n] for n in ("dq", "dq_weight", "dk", "dk_weight")})
    return out


def _blocks(case):
    """Segments, a block of heads at a time: first rows and lengths, query heads, key heads."""
    Hq, Hk = case["Hq"], case["Hk"]
    group, a, b = Hq // Hk, 0, 0
    for n, m in zip(_lens(case, "lens_q"), _lens(case, "lens_k")):
        step = max(1, min(Hk, (1 << 28) // max(1, n * m * group)))
        if n or m:
            for h in range(0, Hk, step):
                e = min(Hk, h + step)
                yield a, n, b, m, slice(h * group, e * group), slice(h, e)
        a, b = a + n, b + m


def _attn_plain(s):
    case = s["case"]
    group, d = case["Hq"] // case["Hk"], case["d"]
    scale = 1 / math.sqrt(d)
    dt, train = s["q"].dtype, "dout" in s
    out = {"o": torch.empty_like(s["q"]),
           "lse": torch.empty(case["Hq"], s["q"].shape[0], dtype=torch.float32, device="cuda")}
    if train:
        out["dq"] = torch.empty_like(s["q"])
        out["dk"], out["dv"] = (torch.empty(s["k"].shape, dtype=dt, device="cuda") for _ in range(2))
    for a, n, b, m, hq, hk in _blocks(case):
        q = s["q"][a: a + n, hq].float().transpose(0, 1)
        k, v = (s[x][b: b + m, hk].float().transpose(0, 1) for x in ("k", "v"))
        kr, vr = (x.repeat_interleave(group, 0) for x in (k, v))
        z = q @ kr.transpose(1, 2) * scale
        if case["causal"]:
            seen = torch.arange(m, device="cuda") <= torch.arange(n, device="cuda")[:, None] + (m - n)
            z = torch.where(seen, z, torch.full_like(z, -math.inf))
        top = z.max(2, keepdim=True).values
        p = torch.exp(z - top)
        total = p.sum(2, keepdim=True)
        p = p / total
        o = p @ vr
        out["o"][a: a + n, hq] = o.to(dt).transpose(0, 1)
        out["lse"][hq, a: a + n] = (top + torch.log(total)).squeeze(2)
        if train:
            do = s["dout"][a: a + n, hq].float().transpose(0, 1)
            dp = do @ vr.transpose(1, 2)
            dz = p * (dp - (do * o).sum(2, keepdim=True)) * scale
            out["dq"][a: a + n, hq] = (dz @ kr).to(dt).transpose(0, 1)
            heads = k.shape[0]
            dk = (dz.transpose(1, 2) @ q).view(heads, group, m, d).sum(1)
            dv = (p.transpose(1, 2) @ do).view(heads, group, m, d).sum(1)
            out["dk"][b: b + m, hk] = dk.to(dt).transpose(0, 1)
            out["dv"][b: b + m, hk] = dv.to(dt).transpose(0, 1)
    return out


def _attn_own(s):
    import adaln_layernorm_modulate_gb300 as A
    c = s["case"]
    Hq, Hk, d, causal = c["Hq"], c["Hk"], c["d"], c["causal"]
    Rq, Rk, nseg = s["q"].shape[0], s["k"].shape[0], s["cu_q"].numel() - 1
    scale, ldv = 1 / math.sqrt(d), s["v"].stride(0)
    A.adaln_attention_fwd(s["q"], s["k"], s["v"], s["o"], s["lse"], s["cu_q"], s["cu_k"], nseg, Rq, Rk, Hq, Hk, d,
                          Hq * d, Hk * d, ldv, Hq * d, scale, causal, s["workspace"], s["workspace_bytes"])
    out = {"o": s["o"], "lse": s["lse"]}
    if "dout" in s:
        A.adaln_attention_bwd(s["dout"], s["q"], s["k"], s["v"], s["o"], s["lse"], s["dq"], s["dk"], s["dv"],
                              s["cu_q"], s["cu_k"], nseg, Rq, Rk, Hq, Hk, d, Hq * d, Hq * d, Hk * d, ldv, Hq * d,
                              Hq * d, Hk * d, Hk * d, scale, causal, s["workspace"], s["workspace_bytes"])
        out.update({n: s[n] for n in ("dq", "dk", "dv")})
    return out


def exact(case, seed):
    """The definitions in 64 bits."""
    s = _inputs(case, seed)
    Hq, Hk, d = case["Hq"], case["Hk"], case["d"]
    train = case["way"] == "train"
    if case["op"] == "rope":
        # Pairs as complex numbers, times e^(i angle); gradients by the chain rule through the graph.
        angle, at = torch.zeros(case["R"], d // 2, dtype=torch.float64, device="cuda"), 0
        for a, w in enumerate(_axes(case)):
            freq = torch.tensor([THETA ** (-2.0 * i / w) for i in range(w // 2)], dtype=torch.float64, device="cuda")
            angle[:, at: at + w // 2] = torch.outer(s["pos"][:, a].double(), freq)
            at += w // 2
        unit = torch.polar(torch.ones_like(angle), angle).unsqueeze(1)
        out = {}
        for n in ("q", "k"):
            x = s[n].double().contiguous().requires_grad_(train)
            w = s[n + "_weight"].double().requires_grad_(train)
            y = x * w / torch.sqrt(torch.mean(torch.square(x), -1, keepdim=True) + EPS)
            y = torch.view_as_real(torch.view_as_complex(y.unflatten(-1, (d // 2, 2))) * unit).flatten(-2)
            out[n + "_out"] = y.detach()
            if train:
                out["d" + n], out["d" + n + "_weight"] = torch.autograd.grad(y, (x, w), s["d" + n + "_out"].double())
        return out
    lq, lk = _lens(case, "lens_q"), _lens(case, "lens_k")
    flops = sum(n * m for n, m in zip(lq, lk)) * Hq * d * (14 if train else 4)
    if flops > 1.2e13:  # the fp64 rate is about 1 TFLOP/s
        return None
    zero = {x: torch.zeros(s[x].shape, dtype=torch.float64, device="cuda") for x in ("q", "k", "v")}
    out = {"o": torch.zeros_like(zero["q"]),
           "lse": torch.zeros(Hq, sum(lq), dtype=torch.float64, device="cuda")}
    if train:
        out["dq"], out["dk"], out["dv"] = zero["q"], zero["k"], zero["v"]
    a = b = 0
    for n, m in zip(lq, lk):
        rows, keys = slice(a, a + n), slice(b, b + m)
        for h in range(Hq if n and m else 0):
            kv = h * Hk // Hq
            q, k, v = s["q"][rows, h].double(), s["k"][keys, kv].double(), s["v"][keys, kv].double()
            z = torch.mm(q, k.t()).div_(math.sqrt(d))
            if case["causal"]:
                z.masked_fill_(torch.ones(n, m, dtype=torch.bool, device="cuda").triu(m - n + 1), -math.inf)
            lse = torch.logsumexp(z, 1)
            out["lse"][h, rows] = lse
            p = z.sub_(lse.unsqueeze(1)).exp_()
            out["o"][rows, h] = torch.mm(p, v)
            if train:
                do = s["dout"][rows, h].double()
                out["dv"][keys, kv] += torch.mm(p.t(), do)
                dp = torch.mm(do, v.t())
                # The Jacobian of a softmax row is diag(p) - p p'.
                dp -= torch.einsum("nm,nm->n", p, dp).unsqueeze(1)
                dz = dp.mul_(p).div_(math.sqrt(d))
                out["dq"][rows, h] = torch.mm(dz, k)
                out["dk"][keys, kv] += torch.mm(dz.t(), q)
        a, b = a + n, b + m
    return out
