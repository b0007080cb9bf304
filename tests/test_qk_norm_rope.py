"""Head norms with rotation by positions against their definition in 64 bits (torch, on the tensors'
device), its gradients against differences of that definition, and its refusals.

Tolerances. u = 2^-24 is half a step of fp32, h = finfo(dtype).eps / 2 half a step of the output's
type. An output is rounded once (h * |value|). Before it, in fp32: a sum of squares of at most 256
terms over lanes of eight (a chain of 4, then at most 7 additions: 12 u, half of it after the root),
the root, the products with rstd and weight (4 u), and the rotation: an angle good to 2^-32 of a turn
rounded to fp32 as half turns (pi u), its cosine and sine (2 steps each, 4 u), two products and a sum
(3 u). Together less than 24 u of the pair's size. Positions up to p put p * 2^-50 on top, the frequencies'
own rounding on both sides."""
import pytest
import torch

import adaln_layernorm_modulate_gb300 as A

U = 2.0 ** -24
EPS = 1e-6
THETA = 10000.0


def axes_array(*widths):
    import ctypes
    arr = (ctypes.c_int32 * len(widths))(*widths)
    return arr, ctypes.addressof(arr)


def test_shape_pointer_and_argument_checks():
    L = A.lib()
    arr, ax = axes_array(16, 48)

    def fwd(q=16, k=16, qw=16, kw=16, pos=16, qo=16, ko=16, R=4, Hq=2, Hk=1, d=64, ql=128, kl=64, qol=128, kol=64,
            axes=ax, n=2, theta=THETA, eps=EPS, norm=1, dt=1):
        return L.adaln_qk_norm_rope_fwd(q, k, qw, kw, pos, qo, ko, R, Hq, Hk, d, ql, kl, qol, kol, axes, n, theta, eps,
                                        norm, dt, None)

    assert [fwd(d=v) for v in (0, 4, 12, 264)] == [2] * 4
    assert fwd(dt=2) == 1 and fwd(R=-1) == 1 and fwd(Hq=-1) == 1 and fwd(Hq=20000) == 1
    assert [fwd(eps=v) for v in (0.0, -1.0, float("inf"), float("nan"))] == [1] * 4
    assert [fwd(theta=v) for v in (0.5, float("inf"), float("nan"))] == [1] * 3
    assert fwd(q=None) == 1 and fwd(ko=None) == 1 and fwd(axes=None) == 1 and fwd(n=0) == 1 and fwd(n=9) == 1
    assert fwd(q=24) == 3 and fwd(qo=8) == 3 and fwd(qw=18) == 3 and fwd(pos=18) == 3
    assert fwd(ql=127) == 3 and fwd(ql=120) == 1 and fwd(kol=56) == 1 and fwd(R=2 ** 60) == 1
    assert fwd(norm=0) == 1  # weights without a norm
    for bad in ((16, 56), (15, 16), (-2, 16)):
        keep, p = axes_array(*bad)
        assert fwd(axes=p) == 1
    assert fwd(R=0, q=None) == 0 and fwd(Hq=0, Hk=0, q=None, k=None) == 0

    def bwd(ptr=(16,) * 11, ws=256, nb=1 << 24, R=4, ld=(128, 64) * 3, n=2, norm=1, eps=EPS, d=64):
        return L.adaln_qk_norm_rope_bwd(*ptr, ws, nb, R, 2, 1, d, *ld, ax, n, THETA, eps, norm, 1, None)

    assert bwd(d=12) == 2 and bwd(R=-1) == 1 and bwd(eps=0.0) == 1
    assert bwd(ptr=(None,) + (16,) * 10) == 1 and bwd(ptr=(16, 16, None) + (16,) * 8) == 1
    assert bwd(ptr=(16,) * 7 + (24,) + (16,) * 3) == 3 and bwd(ptr=(16,) * 10 + (18,)) == 3
    assert bwd(ld=(120, 64) + (128, 64) * 2) == 1 and bwd(norm=0) == 1
    assert A.adaln_qk_norm_rope_bwd_workspace_size(4, 2, 1, 12, 1) == 0
    assert A.adaln_qk_norm_rope_bwd_workspace_size(-4, 2, 1, 64, 1) == 0


def test_cpu_tensors_and_module_text():
    from adaln_layernorm_modulate_gb300.autograd import QKNormRope
    m = QKNormRope(64, (16, 24, 24))
    assert "64, axes=(16, 24, 24), theta=10000, eps=1e-06" in repr(m)
    with pytest.raises(ValueError):
        m(torch.zeros(3, 2, 64), torch.zeros(3, 1, 64), torch.zeros(3, 3, dtype=torch.int32))


def angles(pos, axes, d):
    parts = [pos[:, a: a + 1].double() * torch.tensor([THETA ** (-2.0 * i / w) for i in range(w // 2)],
                                                      dtype=torch.float64, device=pos.device)
             for a, w in enumerate(axes)]
    t = torch.cat(parts, 1) if parts else torch.zeros(pos.shape[0], 0, dtype=torch.float64, device=pos.device)
    return torch.nn.functional.pad(t, (0, d // 2 - t.shape[1])).unsqueeze(1)


def turned(x, t):
    z = torch.view_as_complex(x.double().unflatten(-1, (-1, 2)).contiguous())
    return torch.view_as_real(z * torch.polar(torch.ones_like(t), t)).flatten(-2)


def pair_size(x):
    """Every element's pair's size."""
    return x.unflatten(-1, (-1, 2)).norm(dim=-1, keepdim=True).expand(*x.shape[:-1], x.shape[-1] // 2, 2).flatten(-2)


def definition(x, w, t, norm=True):
    x = x.double()
    if not norm:
        return turned(x, t)
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + torch.tensor(EPS, dtype=torch.float32).double())
    return turned(y if w is None else y * w.double(), t)


def inputs(R, Hq, Hk, d, axes, dtype, weights=True, far=3000, seed=0, rotate=True):
    g = torch.Generator("cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
    rows = (rand(R, (Hq + 2 * Hk) * d) * (0.2 + 3 * torch.rand(R, 1, generator=g, device="cuda"))).to(dtype)
    q, k = rows[:, : Hq * d].view(R, Hq, d), rows[:, Hq * d: (Hq + Hk) * d].view(R, Hk, d)
    w = [(1 + 0.3 * rand(d)).to(dtype) if weights else None for _ in range(2)]
    pos = torch.randint(-far, far + 1, (R, len(axes)), generator=g, device="cuda", dtype=torch.int32) if rotate else None
    return dict(q=q, k=k, w=w, pos=pos, axes=axes, dq_out=rand(R, Hq, d).to(dtype), dk_out=rand(R, Hk, d).to(dtype))


def ld(t):
    return t.stride(0) if t.shape[0] > 1 else t.shape[1] * t.shape[2]


def call(i, norm=True, sums=True):
    q, k, axes = i["q"], i["k"], i["axes"]
    (R, Hq, d), Hk = q.shape, k.shape[1]
    dt = A.ADALN_BF16 if q.dtype == torch.bfloat16 else A.ADALN_F32
    nan = float("nan")
    pad = 16  # rows of outputs lie further apart than they are wide: what is between stays
    wide = {n: torch.full((R, h * d + pad), nan, dtype=q.dtype, device="cuda")
            for n, h in (("q_out", Hq), ("k_out", Hk), ("dq", Hq), ("dk", Hk))}
    lds = {n: v.shape[1] for n, v in wide.items()}
    dw = [torch.full((d,), nan, device="cuda") if sums and i["w"][s] is not None else None for s in range(2)]
    A.adaln_qk_norm_rope_fwd(q, k, *i["w"], i["pos"], wide["q_out"], wide["k_out"], R, Hq, Hk, d, ld(q), ld(k),
                             lds["q_out"], lds["k_out"], axes, THETA, EPS, norm)
    nb = A.adaln_qk_norm_rope_bwd_workspace_size(R, Hq, Hk, d, dt)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    A.adaln_qk_norm_rope_bwd(i["dq_out"], i["dk_out"], q if norm else None, k if norm else None, *i["w"], i["pos"],
                             wide["dq"], wide["dk"], *dw, ws, nb, R, Hq, Hk, d, Hq * d, Hk * d, ld(q), ld(k),
                             lds["dq"], lds["dk"], axes, THETA, EPS, norm)
    assert A.adaln_read_status(ws) == 0
    out = {}
    for n, v in wide.items():
        assert v[:, v.shape[1] - pad:].isnan().all(), "wrote between the rows of " + n
        out[n] = v[:, : v.shape[1] - pad].reshape(R, (v.shape[1] - pad) // d, d)
    out["dq_w"], out["dk_w"] = dw
    return out


def check(i, got, norm=True, far=3000, chain=None):
    d = i["q"].shape[2]
    t = angles(i["pos"], i["axes"], d) if i["pos"] is not None else torch.zeros(i["q"].shape[0], 1, d // 2,
                                                                               dtype=torch.float64, device="cuda")
    dtype = i["q"].dtype
    h = torch.finfo(dtype).eps / 2
    e_rel = 24 * U + far * 2.0 ** -50
    for n, w in (("q", i["w"][0]), ("k", i["w"][1])):
        x, dout = i[n], i["d" + n + "_out"]
        ref = definition(x, w, t, norm)
        assert ((got[n + "_out"].double() - ref).abs() <= h * ref.abs() + e_rel * pair_size(ref) + 1e-38).all(), n
        dy = turned(dout, -t)
        e_dy = e_rel * pair_size(dy)
        xd = x.double()
        if not norm:
            assert ((got["d" + n].double() - dy).abs() <= h * dy.abs() + e_dy + 1e-38).all(), "d" + n
            continue
        rstd = 1 / torch.sqrt((xd * xd).mean(-1, keepdim=True) + torch.tensor(EPS, dtype=torch.float32).double())
        xhat, g = xd * rstd, dy if w is None else dy * w.double()
        one = torch.ones(d, dtype=torch.float64, device="cuda") if w is None else w.double().abs()
        m = (g * xhat).mean(-1, keepdim=True)
        ref = rstd * (g - xhat * m)
        # the mean: its terms' errors and a sum of 12 additions; twice for the products around it
        e_m = 2 * ((e_dy * one + 24 * U * g.abs()) * xhat.abs()).mean(-1, keepdim=True)
        err = h * ref.abs() + 2 * rstd * (e_dy * one + 24 * U * (g.abs() + (xhat * m).abs()) + xhat.abs() * e_m)
        assert ((got["d" + n].double() - ref).abs() <= err + 1e-38).all(), "d" + n
        if got["d" + n + "_w"] is not None and w is not None:
            terms = dy * xhat
            length = chain or terms.shape[0] * terms.shape[1]
            err = ((e_dy + 24 * U * dy.abs()) * xhat.abs() + U * (length + 64) * terms.abs()).sum((0, 1))
            assert ((got["d" + n + "_w"].double() - terms.sum((0, 1))).abs() <= err + 1e-38).all(), "d" + n + "_w"


CASES = [
    (1, 1, 1, 8, (8,)), (1, 12, 12, 128, (44, 42, 42)), (3, 5, 1, 16, (4, 4)), (2, 3, 2, 24, (24,)),
    (7, 2, 2, 32, (8, 8, 8, 8)), (257, 16, 4, 72, (36, 36)), (33, 8, 8, 64, (48,)), (130, 4, 1, 128, (16, 56, 56)),
    (65, 3, 3, 136, (100, 2)), (19, 2, 1, 200, (40, 160)), (40, 7, 3, 256, (64, 96, 96)), (1000, 12, 4, 128, (2,)),
    (5000, 3, 2, 48, (0, 16, 32)),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,Hq,Hk,d,axes", CASES)
def test_against_the_definition(R, Hq, Hk, d, axes, dtype):
    i = inputs(R, Hq, Hk, d, axes, dtype, seed=R + d)
    check(i, call(i))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_many_rows(dtype):
    # More tokens than groups of lanes at once: every group takes several, in a chain of at most
    # 30000 / 2000 tokens of 6 heads (at least 152 CTAs of 16 groups).
    i = inputs(30000, 6, 6, 128, (44, 42, 42), dtype, seed=5)
    check(i, call(i), chain=6 * 15 + 152 * 8 // 32)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_without_weights_rotation_or_norm(dtype):
    for kw, norm in ((dict(weights=False), True), (dict(rotate=False), True), (dict(weights=False), False),
                     (dict(weights=False, rotate=False), False)):
        i = inputs(50, 4, 2, 64, (16, 24, 24), dtype, seed=6, **kw)
        got = call(i, norm)
        check(i, got, norm)
        if not norm and i["pos"] is None:
            assert torch.equal(got["q_out"], i["q"]) and torch.equal(got["dk"], i["dk_out"])


@pytest.mark.gpu
def test_far_positions():
    # Angles of up to 2^31 radians; the definition's own product is off by as much as the frequencies'
    # rounding, 2^31 * 2^-52 each.
    for far in (1 << 20, (1 << 31) - 1):
        i = inputs(300, 2, 2, 64, (32, 32), torch.float32, far=far, seed=7)
        check(i, call(i), far=far)


@pytest.mark.gpu
def test_one_side_alone():
    i = inputs(70, 4, 2, 64, (64,), torch.bfloat16, seed=8)
    both = call(i)
    R, d = 70, 64
    for n, H, s in (("q", 4, 0), ("k", 2, 1)):
        out, dx, dw = torch.empty_like(both[n + "_out"]), torch.empty_like(both["d" + n]), torch.empty(d, device="cuda")
        nb = A.adaln_qk_norm_rope_bwd_workspace_size(R, H, 0, d, 1)
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        x, w, up = i[n], i["w"][s], i["d" + n + "_out"]
        if n == "q":
            A.adaln_qk_norm_rope_fwd(x, None, w, None, i["pos"], out, None, R, H, 0, d, ld(x), 0, H * d, 0, (64,))
            A.adaln_qk_norm_rope_bwd(up, None, x, None, w, None, i["pos"], dx, None, dw, None, ws, nb, R, H, 0, d,
                                     H * d, 0, ld(x), 0, H * d, 0, (64,))
        else:
            A.adaln_qk_norm_rope_fwd(None, x, None, w, i["pos"], None, out, R, 0, H, d, 0, ld(x), 0, H * d, (64,))
            A.adaln_qk_norm_rope_bwd(None, up, None, x, None, w, i["pos"], None, dx, None, dw, ws, nb, R, 0, H, d,
                                     0, H * d, 0, ld(x), 0, H * d, (64,))
        assert torch.equal(out, both[n + "_out"]) and torch.equal(dx, both["d" + n])
        # The same sums in another order: at most R * H additions either way, of terms whose sizes add to this.
        size = (up.float().abs() * (x.float().abs() / x.float().pow(2).mean(-1, keepdim=True).sqrt())).sum((0, 1))
        assert ((dw - both["d" + n + "_w"]).abs() <= 4 * U * R * H * size.max()).all()


@pytest.mark.gpu
def test_no_rows():
    i = inputs(0, 2, 2, 64, (64,), torch.bfloat16)
    got = call(i)
    assert (got["dq_w"] == 0).all() and (got["dk_w"] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_of_zeros_and_bad_values(dtype):
    i = inputs(20, 3, 3, 64, (64,), dtype, seed=9)
    i["q"][4] = 0
    check(i, call(i))
    want = call(i)
    i["q"][7, 1, 5] = float("nan")
    i["k"][9, 2, 3] = float("inf")
    got = call(i)
    rows = torch.arange(20, device="cuda")
    assert got["q_out"][7, 1].isnan().all() and not got["q_out"][7, 0].isnan().any()
    for n, r in (("q", 7), ("k", 9)):
        assert torch.equal(got[n + "_out"][rows != r], want[n + "_out"][rows != r])
        assert torch.equal(got["d" + n][rows != r], want["d" + n][rows != r])


@pytest.mark.gpu
def test_differences_of_the_definition():
    i = inputs(40, 3, 2, 64, (16, 24, 16), torch.float32, seed=10)
    got = call(i)
    t = angles(i["pos"], i["axes"], 64)
    g = torch.Generator("cuda").manual_seed(4)
    s = 1e-5
    for n, w in (("q", i["w"][0]), ("k", i["w"][1])):
        up = i["d" + n + "_out"].double()
        x, wd = i[n].double(), w.double()
        for grad, f, at in ((got["d" + n], lambda v: (definition(v, wd, t) * up).sum(), x),
                            (got["d" + n + "_w"], lambda v: (definition(x, v, t) * up).sum(), wd)):
            v = torch.randn(at.shape, generator=g, device="cuda", dtype=torch.float64)
            want = (f(at + s * v) - f(at - s * v)) / (2 * s)
            # rounding of the differences (values near 1e3 in 64 bits over 2e-5) and their s^2 remainder
            assert ((grad.double() * v).sum() - want).abs() <= 1e-5 * (grad.double() * v).norm() + 1e-5


@pytest.mark.gpu
def test_autograd_matches_the_calls():
    from adaln_layernorm_modulate_gb300.autograd import QKNormRope, qk_norm_rope
    i = inputs(60, 4, 2, 64, (32, 32), torch.bfloat16, seed=11)
    want = call(i)
    rows = i["q"]._base.clone().requires_grad_(True)  # the joint projection
    q, k, _ = rows.view(6, 10, -1).split([256, 128, 128], dim=-1)
    m = QKNormRope(64, (32, 32), device="cuda", dtype=torch.bfloat16)
    with torch.no_grad():
        m.q_weight.copy_(i["w"][0])
        m.k_weight.copy_(i["w"][1])
    pos = i["pos"].view(6, 10, 2).long()
    qo, ko = m(q.unflatten(-1, (4, 64)), k.unflatten(-1, (2, 64)), pos)
    assert torch.equal(qo.reshape(60, 4, 64), want["q_out"]) and torch.equal(ko.reshape(60, 2, 64), want["k_out"])
    torch.autograd.backward([qo, ko], [i["dq_out"].view(6, 10, 4, 64), i["dk_out"].view(6, 10, 2, 64)])
    assert torch.equal(rows.grad[:, :256].reshape(60, 4, 64), want["dq"])
    assert torch.equal(rows.grad[:, 256:384].reshape(60, 2, 64), want["dk"])
    assert (rows.grad[:, 384:] == 0).all()
    assert torch.equal(m.q_weight.grad, want["dq_w"].bfloat16()) and torch.equal(m.k_weight.grad, want["dk_w"].bfloat16())
    # Heads that do not lie side by side, and an output that is not used.
    qt = i["q"].transpose(0, 1).contiguous().transpose(0, 1).requires_grad_(True)
    qo, _ = qk_norm_rope(qt, i["k"], i["pos"], (32, 32), *i["w"])
    qo.backward(i["dq_out"])
    assert torch.equal(qt.grad, want["dq"])
    with pytest.raises(TypeError):
        qk_norm_rope(i["q"], i["k"].float(), i["pos"], (32, 32))
    with pytest.raises(TypeError):
        qk_norm_rope(i["q"], i["k"], i["pos"].float(), (32, 32))
    with pytest.raises(ValueError):
        qk_norm_rope(i["q"], i["k"], i["pos"], (64,))
    with pytest.raises(ValueError):
        qk_norm_rope(i["q"], i["k"][:30], i["pos"], (32, 32))
    with pytest.raises(A.AdalnError):
        qk_norm_rope(i["q"], i["k"], i["pos"], (32, 34))


@pytest.mark.gpu
def test_values_of_every_lane_count_agree_with_a_wider_batch():
    # A row's results do not depend on the rows or heads beside it (items of other sizes).
    i = inputs(4000, 6, 2, 40, (20, 20), torch.bfloat16, seed=13)
    want = call(i)
    j = {n: (v[:3] if torch.is_tensor(v) else v) for n, v in i.items()}
    got = call(j)
    assert all(torch.equal(got[n], want[n][:3]) for n in ("q_out", "k_out", "dq", "dk"))


@pytest.mark.gpu
def test_repeat_side_stream_and_graph_replay():
    i = inputs(500, 6, 3, 128, (44, 42, 42), torch.bfloat16, seed=12)
    want = call(i)
    again = call(i)
    assert all(torch.equal(again[n], want[n]) for n in want)
    R, Hq, Hk, d = 500, 6, 3, 128
    out = {n: torch.empty_like(v) for n, v in want.items()}
    nb = A.adaln_qk_norm_rope_bwd_workspace_size(R, Hq, Hk, d, 1)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")

    def both():
        A.adaln_qk_norm_rope_fwd(i["q"], i["k"], *i["w"], i["pos"], out["q_out"], out["k_out"], R, Hq, Hk, d,
                                 ld(i["q"]), ld(i["k"]), Hq * d, Hk * d, i["axes"])
        A.adaln_qk_norm_rope_bwd(i["dq_out"], i["dk_out"], i["q"], i["k"], *i["w"], i["pos"], out["dq"], out["dk"],
                                 out["dq_w"], out["dk_w"], ws, nb, R, Hq, Hk, d, Hq * d, Hk * d, ld(i["q"]),
                                 ld(i["k"]), Hq * d, Hk * d, i["axes"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(out[n], want[n]) for n in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for v in out.values():
        v.fill_(0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out[n], want[n]) for n in want)


@pytest.mark.gpu
@pytest.mark.parametrize("norm", [True, False])
def test_outputs_changed_in_place(norm):
    # Halving is exact, forward and backward.
    from adaln_layernorm_modulate_gb300.autograd import qk_norm_rope
    i = inputs(30, 4, 2, 64, (32, 32), torch.bfloat16, weights=norm, seed=14)
    want = call(i, norm=norm, sums=norm)
    q, k = (i[n].clone().requires_grad_(True) for n in "qk")
    qo, ko = qk_norm_rope(q, k, i["pos"], (32, 32), *i["w"], norm=norm)
    qo.mul_(0.5)
    ko *= 2
    torch.autograd.backward([qo, ko], [i["dq_out"], i["dk_out"]])
    assert torch.equal(qo.detach(), 0.5 * want["q_out"]) and torch.equal(ko.detach(), 2 * want["k_out"])
    assert torch.equal(q.grad, 0.5 * want["dq"]) and torch.equal(k.grad, 2 * want["dk"])


@pytest.mark.gpu
def test_node_without_rows_or_heads():
    from adaln_layernorm_modulate_gb300.autograd import QKNormRope
    m = QKNormRope(64, (64,), device="cuda", dtype=torch.bfloat16)
    for shape, heads in (((0, 5), 2), ((3, 0), 2), ((3, 5), 0), ((0,), 0)):
        q = torch.ones(*shape, 2, 64, dtype=torch.bfloat16, device="cuda", requires_grad=True)
        k = torch.ones(*shape, heads, 64, dtype=torch.bfloat16, device="cuda", requires_grad=True)
        qo, ko = m(q, k, torch.zeros(*shape, 1, dtype=torch.int32, device="cuda"))
        assert qo.shape == q.shape and ko.shape == k.shape
        (qo.sum() + ko.sum()).backward()
        assert q.grad.shape == q.shape and k.grad.shape == k.shape and (m.k_weight.grad == 0).all()
        m.zero_grad()
