"""The affine layer norm against its definition in 64 bits (torch, on the tensors' device),
its gradients against differences of that definition, and its refusals.

Tolerances. u = 2^-24 is half a step of fp32, h = finfo(dtype).eps / 2 half a step of the
output's type. An output is rounded once (h * |value|); the fp32 work before it adds a few
roundings of each of its terms, taken at the terms' absolute sizes: the row statistics come from
sums of depth at most D / 32 + 10 (a lane's elements, then trees), and a column sum is a chain of
at most R / 64 + 64 additions (a tile's rows, then its pieces)."""
import pytest
import torch

import adaln_layernorm_modulate_gb300 as A

U = 2.0 ** -24
EPS = 1e-6


def test_shape_pointer_and_eps_checks():
    L = A.lib()
    ok = [16] * 6
    assert L.adaln_layernorm_fwd(*ok, 4, 12, EPS, 1, None) == 2
    assert L.adaln_layernorm_fwd(*ok, 4, 16392, EPS, 1, None) == 2
    assert L.adaln_layernorm_fwd(*ok, 4, 64, EPS, 2, None) == 1
    assert L.adaln_layernorm_fwd(*ok, -1, 64, EPS, 1, None) == 1
    assert L.adaln_layernorm_fwd(*ok, 2 ** 62, 64, EPS, 1, None) == 1
    assert L.adaln_layernorm_fwd(*ok, 4, 64, 0.0, 1, None) == 1
    assert L.adaln_layernorm_fwd(*ok, 4, 64, float("nan"), 1, None) == 1
    assert L.adaln_layernorm_fwd(None, 16, 16, 16, 16, 16, 4, 64, EPS, 1, None) == 1
    assert L.adaln_layernorm_fwd(16, 16, 16, 16, None, 16, 4, 64, EPS, 1, None) == 1
    assert L.adaln_layernorm_fwd(16, 18, 16, 16, 16, 16, 4, 64, EPS, 1, None) == 3
    assert L.adaln_layernorm_fwd(16, 16, 24, 16, 16, 16, 4, 64, EPS, 1, None) == 3
    assert L.adaln_layernorm_fwd(*ok, 0, 64, EPS, 1, None) == 0
    b = [16] * 8
    assert L.adaln_layernorm_bwd(*b, 256, 1 << 20, 4, 12, 1, None) == 2
    assert L.adaln_layernorm_bwd(*b, 256, 1 << 20, -4, 64, 1, None) == 1
    assert L.adaln_layernorm_bwd(None, *b[1:], 256, 1 << 20, 4, 64, 1, None) == 1
    assert L.adaln_layernorm_bwd(16, 16, 16, 16, 16, 16, 24, 16, 256, 1 << 20, 4, 64, 1, None) == 3
    assert L.adaln_layernorm_bwd(*b, None, 1 << 20, 4, 64, 1, None) == 4
    assert L.adaln_layernorm_bwd(*b, 256, 100, 4, 64, 1, None) == 4
    assert A.adaln_layernorm_bwd_workspace_size(4, 12, 1) == 0
    assert A.adaln_layernorm_bwd_workspace_size(-1, 64, 1) == 0


def test_cpu_tensors_and_module_text():
    from adaln_layernorm_modulate_gb300.autograd import LayerNorm
    m = LayerNorm(64, bias=False)
    assert "64, eps=1e-06, weight=True, bias=False" in repr(m)
    with pytest.raises(ValueError):
        m(torch.zeros(2, 64))


def definition(x, w, b, dy):
    x, dy = x.double(), dy.double()
    D = x.shape[1]
    one = torch.ones(D, dtype=torch.float64, device=x.device)
    w = one if w is None else w.double()
    b = 0 * one if b is None else b.double()
    mean = x.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + torch.tensor(EPS, dtype=torch.float32).double())
    xhat = (x - mean) * rstd
    g = dy * w
    dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    return dict(y=xhat * w + b, mean=mean, rstd=rstd, xhat=xhat, g=g, dx=dx, dw=(dy * xhat).sum(0), db=dy.sum(0),
                w=w, b=b)


def inputs(R, D, dtype, weight, bias, seed=0, kind="rows"):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(R, D, generator=g, device="cuda")
    if kind == "offset":  # a mean that dwarfs the spread
        x = x * 0.5 + 200 * torch.randn(R, 1, generator=g, device="cuda")
    if kind == "constant":  # no spread at all: xhat is 0
        x = torch.randn(R, 1, generator=g, device="cuda").expand(R, D)
    x = x.to(dtype).contiguous()
    w = (1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(dtype) if weight else None
    b = torch.randn(D, generator=g, device="cuda").to(dtype) if bias else None
    dy = torch.randn(R, D, generator=g, device="cuda").to(dtype)
    return x, w, b, dy


def call(x, w, b, dy, want_w=True, want_b=True):
    R, D = x.shape
    dt = A.ADALN_BF16 if x.dtype == torch.bfloat16 else A.ADALN_F32
    nan = float("nan")
    y, dx = torch.full_like(x, nan), torch.full_like(x, nan)
    mean, rstd = (torch.full((R,), nan, device="cuda") for _ in range(2))
    dw, db = (torch.full((D,), nan, device="cuda") for _ in range(2))
    A.adaln_layernorm_fwd(x, w, b, y, mean, rstd, R, D, EPS)
    nb = A.adaln_layernorm_bwd_workspace_size(R, D, dt)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    A.adaln_layernorm_bwd(dy, x, mean, rstd, w, dx, dw if want_w else None, db if want_b else None, ws, nb, R, D)
    assert A.adaln_read_status(ws) == 0
    return dict(y=y, mean=mean, rstd=rstd, dx=dx, dw=dw, db=db)


def check(x, w, b, dy, got, want_w=True, want_b=True):
    R, D = x.shape
    r = definition(x, w, b, dy)
    h = torch.finfo(x.dtype).eps / 2 if x.dtype == torch.bfloat16 else U
    depth = D / 32 + 10
    peak = (x.double() - x[:, :1].double()).abs().amax(1, keepdim=True) + x[:, :1].double().abs()
    spread = (x.double() - x[:, :1].double()).abs().amax(1, keepdim=True)
    # mean: an average of d = x - x0 (depth roundings of its size), then x0 + it rounded
    e_mean = U * (depth * spread + 2 * peak)
    assert ((got["mean"].double()[:, None] - r["mean"]).abs() <= e_mean).all()
    # rstd: half the variance's relative error (centred squares; the mean's error is second order)
    e_rstd = r["rstd"] * U * (depth + 8) + r["rstd"] ** 3 * (U * depth * spread) ** 2
    assert ((got["rstd"].double()[:, None] - r["rstd"]).abs() <= e_rstd).all()
    e_xhat = U * (depth + 8) * (r["rstd"] * spread + r["xhat"].abs())
    e_y = h * r["y"].abs() + 2 * (r["w"].abs() * e_xhat + 3 * U * ((r["xhat"] * r["w"]).abs() + r["b"].abs()))
    assert ((got["y"].double() - r["y"]).abs() <= e_y).all()
    # The backward takes the forward's mean as rounded to fp32: xhat moves by up to e_mean * rstd.
    e_xb = e_xhat + e_mean * r["rstd"]
    ga = r["g"].abs()
    e_mgx = (ga * e_xb).mean(1, keepdim=True) + U * (depth + 4) * (r["g"] * r["xhat"]).abs().mean(1, keepdim=True)
    mgx = (r["g"] * r["xhat"]).mean(1, keepdim=True).abs()
    e_dx = r["rstd"] * (4 * U * ga + U * (depth + 4) * ga.mean(1, keepdim=True) + r["xhat"].abs() * e_mgx
                        + e_xb * mgx + 4 * U * r["xhat"].abs() * mgx)
    e_dx = e_dx + h * r["dx"].abs() + e_rstd / r["rstd"] * r["dx"].abs() * 4
    assert ((got["dx"].double() - r["dx"]).abs() <= 2 * e_dx).all()
    chain = R / 64 + 64
    if want_w:
        e = U * chain * (dy.double() * r["xhat"]).abs().sum(0) + (dy.double().abs() * e_xb).sum(0)
        assert ((got["dw"].double() - r["dw"]).abs() <= e).all()
    if want_b:
        assert ((got["db"].double() - r["db"]).abs() <= U * chain * dy.double().abs().sum(0)).all()


SHAPES = [(1, 8), (1, 1536), (2, 64), (5, 264), (257, 1152), (3, 16384), (300, 2040), (4099, 640), (700, 5120)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("R,D", SHAPES, ids=["%dx%d" % s for s in SHAPES])
def test_matches_the_definition(R, D, dtype):
    a = inputs(R, D, dtype, True, True, seed=R + D)
    check(*a, call(*a))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["offset", "constant"])
def test_rows_with_little_spread(kind):
    a = inputs(130, 1536, torch.float32, True, True, seed=3, kind=kind)
    check(*a, call(*a))


@pytest.mark.gpu
@pytest.mark.parametrize("weight,bias", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("R,D", [(9, 768), (2000, 512)])
def test_optional_weight_bias_and_gradients(weight, bias, R, D):
    a = inputs(R, D, torch.bfloat16, weight, bias, seed=5)
    full = call(*a)
    check(*a, full)
    for want_w, want_b in ((True, False), (False, True), (False, False)):
        part = call(*a, want_w, want_b)
        check(*a, part, want_w, want_b)
        assert torch.equal(part["dx"], full["dx"])
        # What is not wanted is not written.
        assert torch.equal(part["dw"], full["dw"]) if want_w else part["dw"].isnan().all()
        assert torch.equal(part["db"], full["db"]) if want_b else part["db"].isnan().all()


@pytest.mark.gpu
def test_one_bad_row_stays_alone():
    x, w, b, dy = inputs(64, 1536, torch.bfloat16, True, True, seed=7)
    clean = call(x, w, b, dy)
    x[10, 3] = float("nan")
    x[20, 5] = float("inf")
    got = call(x, w, b, dy)
    rows = [i for i in range(64) if i not in (10, 20)]
    assert torch.equal(got["y"][rows], clean["y"][rows]) and torch.equal(got["dx"][rows], clean["dx"][rows])
    assert got["y"][10].isnan().all() and got["y"][20].isnan().any()


@pytest.mark.gpu
def test_no_rows():
    x = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16)
    got = call(x, None, None, x)
    assert (got["dw"] == 0).all() and (got["db"] == 0).all()


@pytest.mark.gpu
def test_autograd_matches_the_calls_and_differences():
    from adaln_layernorm_modulate_gb300.autograd import LayerNorm, layer_norm
    x, w, b, dy = inputs(66, 512, torch.float32, True, True, seed=11)
    direct = call(x, w, b, dy)
    xs = x.view(6, 11, 512).transpose(0, 1)  # not contiguous
    m = LayerNorm(512, device="cuda")
    with torch.no_grad():
        m.weight.copy_(w)
        m.bias.copy_(b)
    leaf = xs.clone(memory_format=torch.preserve_format).requires_grad_(True)
    y = m(leaf)
    y.backward(dy.view(6, 11, 512).transpose(0, 1))
    back = lambda t: t.transpose(0, 1).reshape(66, 512)
    assert torch.equal(back(y.detach()), direct["y"]) and torch.equal(back(leaf.grad), direct["dx"])
    # Differences of the 64-bit definition along one direction of each input. Central, step s:
    # the remainder is s^2 / 6 of a third derivative of order 1 a row.
    g = torch.Generator("cuda").manual_seed(1)
    s = 1e-4
    loss = lambda x_, w_, b_: (definition(x_, w_, b_, dy)["y"] * dy.double()).sum()
    args, grads = [x.double(), w.double(), b.double()], [direct["dx"], direct["dw"], direct["db"]]
    for i in range(3):
        v = torch.randn(args[i].shape, generator=g, device="cuda", dtype=torch.float64)
        up, dn = list(args), list(args)
        up[i], dn[i] = args[i] + s * v, args[i] - s * v
        want = (loss(*up) - loss(*dn)) / (2 * s)
        size = (grads[i].double() * v).norm()
        assert ((grads[i].double() * v).sum() - want).abs() <= 1e-4 * size + 66 * 512 * s * s
    with pytest.raises(ValueError):
        layer_norm(x, w[:256])
    with pytest.raises(TypeError):
        layer_norm(x, w.bfloat16())


@pytest.mark.gpu
def test_side_stream_and_graph_replay():
    x, w, b, dy = inputs(257, 1152, torch.bfloat16, True, True, seed=13)
    want = call(x, w, b, dy)
    R, D = x.shape
    out = {k: torch.empty_like(v) for k, v in want.items()}
    nb = A.adaln_layernorm_bwd_workspace_size(R, D, A.ADALN_BF16)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")

    def both():
        A.adaln_layernorm_fwd(x, w, b, out["y"], out["mean"], out["rstd"], R, D, EPS)
        A.adaln_layernorm_bwd(dy, x, out["mean"], out["rstd"], w, out["dx"], out["dw"], out["db"], ws, nb, R, D)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(out[k], want[k]) for k in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for v in out.values():
        v.zero_()
    graph.replay()
    assert all(torch.equal(out[k], want[k]) for k in want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 1152, 5120, 16384])
def test_a_workspace_holds_every_smaller_batch(D, dtype):
    dt = A.ADALN_BF16 if dtype == torch.bfloat16 else A.ADALN_F32
    sizes = [A.adaln_layernorm_bwd_workspace_size(R, D, dt) for R in range(0, 2000)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    x, w, b, dy = inputs(sms, D, dtype, True, True, seed=17)
    want = call(x, w, b, dy)
    dx, dw, db = (torch.empty_like(want[k]) for k in ("dx", "dw", "db"))
    nb = sizes[sms + 1]
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    A.adaln_layernorm_bwd(dy, x, want["mean"], want["rstd"], w, dx, dw, db, ws, nb, sms, D)
    assert torch.equal(dx, want["dx"]) and torch.equal(dw, want["dw"]) and torch.equal(db, want["db"])
