"""The softmax cross entropy over a vocabulary against its definition in 64 bits (torch, on the
tensors' device), its gradients against differences of that definition, and its refusals.

Tolerances. h = 2^-8 is half a step of bf16. A tensor-core sum of K products takes K / 16 steps,
each off by at most 2^-22 of the sum of the terms' absolute values (two units of fp32, whatever
the direction of its rounding). The exponentials are good to 2^-20 relative (their argument, at
most 30 or so, is rounded to fp32). dz is rounded to bf16 (h of its value), dx and dweight once;
below 2^-126, the smallest normal value of fp32 and bf16 alike, any of them may be 0 instead."""
import math

import pytest
import torch

import adaln_layernorm_modulate_gb300 as A

H = 2.0 ** -8
TINY = 2.0 ** -126
IGNORE = -100


def test_checks_before_any_device_work():
    L = A.lib()
    f = lambda x=16, w=16, t=16, lo=16, ls=16, N=4, V=10, D=64, ws=256, nb=1 << 30, dt=1: L.adaln_linear_xent_fwd(
        x, w, t, lo, ls, N, V, D, IGNORE, ws, nb, dt, None)
    assert f(D=12) == 2 and f(D=16392) == 2 and f(dt=0) == 2 and f(dt=7) == 1
    assert f(N=-1) == 1 and f(V=0) == 1 and f(V=2 ** 31) == 1 and f(N=2 ** 31) == 1
    assert f(x=None) == 1 and f(w=None) == 1 and f(t=None) == 1 and f(lo=None) == 1 and f(ls=None) == 1
    assert f(x=24) == 3 and f(w=24) == 3 and f(t=20) == 3 and f(lo=18) == 3 and f(ws=272) == 3
    assert f(ws=None) == 4 and f(nb=1000) == 4
    b = lambda x=16, w=16, t=16, ls=16, up=16, ul=16, dx=16, dw=16, N=4, V=10, D=64, ws=256, nb=1 << 30, dt=1: \
        L.adaln_linear_xent_bwd(x, w, t, ls, up, ul, dx, dw, N, V, D, IGNORE, ws, nb, dt, None)
    assert b(D=12) == 2 and b(dt=0) == 2 and b(N=-1) == 1 and b(V=0) == 1
    assert b(x=None) == 1 and b(w=None) == 1 and b(t=None) == 1 and b(ls=None) == 1 and b(up=None) == 1
    assert b(dx=None, dw=None) == 1
    assert b(dx=24) == 3 and b(dw=24) == 3 and b(ul=18) == 3 and b(t=20) == 3
    assert b(ws=None) == 4 and b(nb=1000) == 4


def test_workspace_sizes():
    for size in (A.adaln_linear_xent_fwd_workspace_size, A.adaln_linear_xent_bwd_workspace_size):
        assert size(4, 10, 12, 1) == 0 and size(4, 10, 64, 0) == 0 and size(-1, 10, 64, 1) == 0
        assert size(0, 1, 8, 1) > 0
        # Far below the logits it stands for (fp32: 6.4 GB).
        assert size(16384, 100000, 1024, 1) < 0.5e9
        assert size(1 << 20, 1 << 17, 8192, 1) > 1 << 33  # sizes past 32 bits


def test_python_refusals():
    from adaln_layernorm_modulate_gb300.autograd import linear_cross_entropy
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(10, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        linear_cross_entropy(x, w, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):
        linear_cross_entropy(x, w, torch.zeros(4, dtype=torch.int64), reduction="avg")


def inputs(N, V, D, ignored=0.0, seed=0, scale=1.5):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(N, D, generator=g, device="cuda").bfloat16()
    w = (scale / D ** 0.5 * torch.randn(V, D, generator=g, device="cuda")).bfloat16()
    t = torch.randint(V, (N,), generator=g, device="cuda")
    t[torch.rand(N, generator=g, device="cuda") < ignored] = IGNORE
    up = 0.5 + torch.rand(N, generator=g, device="cuda")
    ul = 0.1 * torch.randn(N, generator=g, device="cuda")
    return x, w, t, up, ul


def call(x, w, t, up, ul, want_x=True, want_w=True, status=0, backward=True):
    (N, D), V = x.shape, w.shape[0]
    nan = float("nan")
    loss, lse = (torch.full((N,), nan, device="cuda") for _ in range(2))
    nb = max(A.adaln_linear_xent_fwd_workspace_size(N, V, D, 1), A.adaln_linear_xent_bwd_workspace_size(N, V, D, 1))
    ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda")  # whatever it holds: NaN
    A.adaln_linear_xent_fwd(x, w, t, loss, lse, N, V, D, IGNORE, ws, nb)
    assert A.adaln_read_status(ws) == status
    if not backward:
        return loss, lse
    dx = torch.full_like(x, nan) if want_x else None
    dw = torch.full_like(w, nan) if want_w else None
    ws.fill_(0xFF)
    A.adaln_linear_xent_bwd(x, w, t, lse, up, ul, dx, dw, N, V, D, IGNORE, ws, nb)
    assert A.adaln_read_status(ws) == status
    return loss, lse, dx, dw


def check(x, w, t, up, ul, got):
    """Every output against the definition, rows that carry no loss among them."""
    (N, D), V = x.shape, w.shape[0]
    loss, lse, dx, dw = got
    on = (t >= 0) & (t < V)
    off = ~on
    assert (loss[off] == 0).all() and (lse[off] == 0).all()
    if dx is not None:
        assert (dx[off] == 0).all()
    xd, wd, td = x[on].double(), w.double(), t[on]
    upd = up[on].double()
    uld = torch.zeros_like(upd) if ul is None else ul[on].double()
    z = xd @ wd.t()
    L = torch.logsumexp(z, 1)
    p = torch.exp(z - L[:, None])
    rows = torch.arange(len(td), device="cuda")
    steps = D / 16 + 16
    e_z = 2.0 ** -22 * steps * (xd.abs() @ wd.abs().t()).amax(1) if len(td) else L
    # The sum of exponentials: 2^-20 relative and a chain of at most V / 16 + 64 additions.
    e_l = e_z + 2.0 ** -20 + 2.0 ** -24 * (V / 16 + 64) + 2.0 ** -23 * L.abs()
    assert ((lse[on].double() - L).abs() <= e_l).all()
    zt = z[rows, td]
    assert ((loss[on].double() - (L - zt)).abs() <= e_l + e_z + 2.0 ** -23 * (L - zt).abs()).all()
    dz = p * (upd + uld)[:, None]
    e_dz = dz.abs() * (e_l + e_z + 2.0 ** -19)[:, None]
    dz[rows, td] -= upd
    e_dz[rows, td] += 2.0 ** -23 * upd
    e_dz += H * dz.abs() + TINY
    for out, want, err, big, frob in (
            (None if dx is None else dx[on], lambda: dz @ wd, lambda: e_dz @ wd.abs(),
             lambda: 2.0 ** -22 * (V / 16 + 32) * (dz.abs() @ wd.abs()),
             lambda: ((dz ** 2) @ (wd ** 2)).sum() ** 0.5),
            (dw, lambda: dz.t() @ xd, lambda: e_dz.t() @ xd.abs(),
             lambda: 2.0 ** -22 * (N / 16 + 32) * (dz.t().abs() @ xd.abs()),
             lambda: ((dz ** 2).t() @ (xd ** 2)).sum() ** 0.5)):
        if out is None:
            continue
        ref = want()
        e = (out.double() - ref).abs()
        assert (e <= err() + big() + H * ref.abs() + TINY).all()
        # The roundings are independent: together they stay near h of the root of the squares
        # (and e_z, the same for a row's whole dz, near its part).
        assert e.norm() <= 2 * (H * frob() + H * ref.norm()) + 2 * (e_l.max() + e_z.max() if len(td) else 0) * ref.norm()


CASES = [(1, 1, 8), (1, 1000, 512), (3, 16, 64), (2, 300, 72), (128, 256, 64), (130, 257, 72), (129, 513, 200),
         (300, 5000, 768), (96, 8192, 1024), (40, 300, 4096), (5, 40, 16384), (1, 9000, 264)]


@pytest.mark.gpu
@pytest.mark.parametrize("N,V,D", CASES, ids=["%dx%dx%d" % c for c in CASES])
def test_matches_the_definition(N, V, D):
    a = inputs(N, V, D, seed=N + V)
    check(*a, call(*a))


@pytest.mark.gpu
@pytest.mark.parametrize("ignored", [0.15, 0.5, 0.9])
@pytest.mark.parametrize("N,V,D", [(37, 700, 128), (700, 1025, 264)])
def test_rows_without_a_loss(N, V, D, ignored):
    a = inputs(N, V, D, ignored, seed=7)
    check(*a, call(*a))


@pytest.mark.gpu
@pytest.mark.parametrize("N", [0, 1, 200])
def test_no_row_carries_a_loss(N):
    x, w, t, up, ul = inputs(N, 600, 128, seed=8)
    t.fill_(IGNORE)
    loss, lse, dx, dw = call(x, w, t, up, ul)
    assert (loss == 0).all() and (lse == 0).all() and (dx == 0).all() and (dw == 0).all()


@pytest.mark.gpu
def test_several_pieces_of_the_vocabulary():
    a = inputs(8192, 9001, 72, 0.3, seed=9)
    check(*a, call(*a))


@pytest.mark.gpu
@pytest.mark.parametrize("N,V,D,ignored", [(8192, 20001, 72, 0.3), (2049, 70000, 136, 0.0)])
def test_dz_in_several_pieces(N, V, D, ignored):
    # dz of the whole vocabulary would take more than the 256 MiB of a piece: dx adds up over
    # launches, dweight comes piece by piece, the last one narrower.
    assert N * V * 2 > 256 << 20
    x, w, t, up, ul = inputs(N, V, D, ignored, seed=20)
    t[0], t[1], t[2] = 0, V - 1, V // 2
    full = call(x, w, t, up, ul)
    check(x, w, t, up, ul, full)
    assert torch.equal(call(x, w, t, up, ul, want_w=False)[2], full[2])
    assert torch.equal(call(x, w, t, up, ul, want_x=False)[3], full[3])


@pytest.mark.gpu
def test_many_rows_of_one_word():
    # A word that is every other row's target: more rows than dweight corrects one by one.
    x, w, t, up, ul = inputs(1500, 3000, 136, 0.1, seed=21)
    t[::2] = 77
    t[1:9] = 78  # eight rows and some chance ones: at and past the limit
    check(x, w, t, up, ul, call(x, w, t, up, ul))


@pytest.mark.gpu
def test_what_rows_without_a_loss_hold_does_not_matter():
    x, w, t, up, ul = inputs(140, 900, 128, 0.4, seed=10)
    want = call(x, w, t, up, ul)
    off = t == IGNORE
    x[off], up[off], ul[off] = float("nan"), float("inf"), float("nan")
    got = call(x, w, t, up, ul)
    assert all(torch.equal(g, v) for g, v in zip(got, want))


@pytest.mark.gpu
def test_one_bad_row_stays_alone():
    x, w, t, up, ul = inputs(140, 900, 128, seed=11)
    want = call(x, w, t, up, ul)
    x[5, 3] = float("nan")
    got = call(x, w, t, up, ul)
    rows = torch.arange(140, device="cuda") != 5
    assert got[0][5].isnan() and got[1][5].isnan() and got[2][5].isnan().all()
    assert all(torch.equal(g[rows], v[rows]) for g, v in zip(got[:3], want[:3]))


@pytest.mark.gpu
def test_extreme_logits():
    # Logits of several hundred: exp overflows without the maximum taken out, and all but a few
    # probabilities are 0.
    x, w, t, up, ul = inputs(64, 500, 64, seed=12, scale=300.0)
    check(x, w, t, up, ul, call(x, w, t, up, ul))


@pytest.mark.gpu
def test_bad_targets_are_recorded_and_carry_no_loss():
    x, w, t, up, ul = inputs(300, 400, 64, seed=13)
    t[17], t[200], t[299] = 400, -1, 2 ** 40
    check(x, w, t, up, ul, call(x, w, t, up, ul, status=9))


@pytest.mark.gpu
def test_optional_outputs_and_dlse():
    x, w, t, up, ul = inputs(200, 700, 136, 0.2, seed=14)
    full = call(x, w, t, up, ul)
    assert torch.equal(call(x, w, t, up, ul, want_w=False)[2], full[2])
    assert torch.equal(call(x, w, t, up, ul, want_x=False)[3], full[3])
    check(x, w, t, up, None, call(x, w, t, up, None))
    zero = torch.zeros_like(up)
    check(x, w, t, zero, ul, call(x, w, t, zero, ul))


@pytest.mark.gpu
def test_offsets_past_32_bits():
    # weight and dweight of 2.3e9 elements; the last words of the vocabulary hold the targets.
    N, V, D = 4, 140000, 16384
    g = torch.Generator("cuda").manual_seed(15)
    x = torch.randn(N, D, generator=g, device="cuda").bfloat16()
    w = torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
    tail = (0.02 * torch.randn(64, D, generator=g, device="cuda")).bfloat16()
    w[-64:] = tail
    t = torch.tensor([V - 1, V - 64, V - 7, 0], device="cuda")
    up = torch.ones(N, device="cuda")
    loss, lse, dx, dw = call(x, w, t, up, None)
    z = torch.cat([torch.zeros(N, 1, dtype=torch.float64, device="cuda"), x.double() @ tail.double().t()], 1)
    weight = torch.ones(65, dtype=torch.float64, device="cuda")
    weight[0] = V - 64  # the words whose weight is zero have one logit, 0
    L = torch.log((torch.exp(z) * weight).sum(1))
    e_z = 2.0 ** -22 * (D / 16 + 16) * (x.double().abs() @ tail.double().abs().t()).amax(1)
    assert ((lse.double() - L).abs() <= e_z + 2.0 ** -20 + 2.0 ** -24 * (V / 16 + 64) + 2.0 ** -23 * L).all()
    dz = torch.exp(z[:, 1:] - L[:, None])
    hot = torch.zeros_like(dz)
    hot[0, 63] = hot[1, 0] = hot[2, 57] = 1
    ref = (dz - hot).t() @ x.double()
    err = ((dz - hot).abs() * (H + 2 * e_z.max() + 2.0 ** -18)).t() @ x.double().abs()
    assert ((dw[-64:].double() - ref).abs() <= err + H * ref.abs()).all()
    rest = dw[: V - 64].float().abs().amax(1)  # tiny probabilities everywhere, -1 at word 0
    assert (rest[1:] <= 1.2 * N * 6 / V).all() and rest[0] >= 1


@pytest.mark.gpu
def test_differences_of_the_definition():
    from adaln_layernorm_modulate_gb300.autograd import linear_cross_entropy
    x, w, t, _, _ = inputs(60, 300, 64, 0.25, seed=16)
    x, w = x.requires_grad_(True), w.requires_grad_(True)
    linear_cross_entropy(x, w, t, z_loss=1e-2).backward()
    keep = t != IGNORE

    def loss(x_, w_):
        z = x_[keep] @ w_.t()
        L = torch.logsumexp(z, 1)
        return (L - z[torch.arange(int(keep.sum())), t[keep]] + 1e-2 * L * L).mean()

    xd, wd = x.detach().double(), w.detach().double()
    g = torch.Generator("cuda").manual_seed(3)
    s = 1e-4  # central: the remainder is of order s^2
    for a, b, grad in ((xd, wd, x.grad), (wd, xd, w.grad)):
        v = torch.randn(a.shape, generator=g, device="cuda", dtype=torch.float64)
        f = (lambda q: loss(q, b)) if a is xd else (lambda q: loss(b, q))
        want = (f(a + s * v) - f(a - s * v)) / (2 * s)
        size = (grad.double() * v).norm()  # independent roundings of h each, in dz and at the end
        assert ((grad.double() * v).sum() - want).abs() <= 4 * H * size + 1e-5


@pytest.mark.gpu
def test_autograd_matches_the_calls():
    from adaln_layernorm_modulate_gb300.autograd import linear_cross_entropy
    x, w, t, up, ul = inputs(132, 700, 128, 0.3, seed=17)
    want = call(x, w, t, up, None)
    xs = x.view(12, 11, 128).transpose(0, 1).clone(memory_format=torch.preserve_format).requires_grad_(True)
    ts = t.view(12, 11).transpose(0, 1)
    wp = w.clone().requires_grad_(True)
    loss = linear_cross_entropy(xs, wp, ts, reduction="none", check_targets=True)
    assert loss.shape == ts.shape and not xs.is_contiguous()
    loss.backward(up.view(12, 11).transpose(0, 1))
    # Another order of the rows: dweight's sums differ, everything of a row does not.
    assert torch.equal(loss.detach().transpose(0, 1).reshape(-1), want[0])
    assert torch.equal(xs.grad.transpose(0, 1).reshape(132, 128), want[2])
    assert (wp.grad.double() - want[3].double()).norm() <= 2 * H * want[3].double().norm()
    frozen = linear_cross_entropy(x, wp.detach().requires_grad_(True), t, reduction="sum")
    frozen.backward()
    assert x.grad is None
    assert linear_cross_entropy(x, w, torch.full_like(t, IGNORE)).item() == 0.0
    with pytest.raises(A.AdalnError):
        linear_cross_entropy(x, w, torch.full_like(t, 700), check_targets=True)
    with pytest.raises(TypeError):
        linear_cross_entropy(x.float(), w.float(), t)
    with pytest.raises(ValueError):
        linear_cross_entropy(x, w, t.int())


@pytest.mark.gpu
def test_repeat_side_stream_and_graph_replay():
    x, w, t, up, ul = inputs(500, 3000, 320, 0.2, seed=18)
    want = call(x, w, t, up, ul)
    assert all(torch.equal(g, v) for g, v in zip(call(x, w, t, up, ul), want))
    (N, D), V = x.shape, w.shape[0]
    out = [torch.empty_like(v) for v in want]
    nb = max(A.adaln_linear_xent_fwd_workspace_size(N, V, D, 1), A.adaln_linear_xent_bwd_workspace_size(N, V, D, 1))
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")

    def both():
        A.adaln_linear_xent_fwd(x, w, t, out[0], out[1], N, V, D, IGNORE, ws, nb)
        A.adaln_linear_xent_bwd(x, w, t, out[1], up, ul, out[2], out[3], N, V, D, IGNORE, ws, nb)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(g, v) for g, v in zip(out, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for v in out:
        v.zero_()
    graph.replay()
    assert all(torch.equal(g, v) for g, v in zip(out, want))


@pytest.mark.gpu
def test_outputs_stay_inside_their_buffers():
    x, w, t, up, ul = inputs(77, 333, 72, 0.2, seed=19)
    (N, D), V = x.shape, w.shape[0]
    guard = 4096

    def fenced(n, dtype):
        whole = torch.full((n + 2 * guard,), 7.0, dtype=dtype, device="cuda")
        return whole, whole[guard:guard + n]

    nb = max(A.adaln_linear_xent_fwd_workspace_size(N, V, D, 1), A.adaln_linear_xent_bwd_workspace_size(N, V, D, 1))
    bufs = [fenced(N, torch.float32), fenced(N, torch.float32), fenced(N * D, torch.bfloat16),
            fenced(V * D, torch.bfloat16), fenced(nb // 4, torch.float32)]
    loss, lse, dx, dw, ws = (b[1] for b in bufs)
    A.adaln_linear_xent_fwd(x, w, t, loss, lse, N, V, D, IGNORE, ws, nb)
    A.adaln_linear_xent_bwd(x, w, t, lse, up, ul, dx, dw, N, V, D, IGNORE, ws, nb)
    check(x, w, t, up, ul, (loss, lse, dx.view(N, D), dw.view(V, D)))
    for whole, part in bufs:
        assert (whole[:guard] == 7).all() and (whole[guard + part.numel():] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("N", [255, 1020])
def test_equal_target_gradients_leave_no_scale_error(N):
    # A mean's dloss: the same for all rows, and with small probabilities dz of the target nearly so.
    # (1 - p) / N lies almost halfway between two bf16 values here. Half of the rows have one word
    # as their target; a rounding that goes the same way in all of them would scale its gradient.
    V, D, word, n = 3000, 512, 77, (N + 1) // 2
    g = torch.Generator("cuda").manual_seed(22)
    x = (torch.randn(1, D, generator=g, device="cuda") + 0.5 * torch.randn(N, D, generator=g, device="cuda")).bfloat16()
    w = (0.2 / D ** 0.5 * torch.randn(V, D, generator=g, device="cuda")).bfloat16()
    t = torch.randint(V, (N,), generator=g, device="cuda")
    t[::2] = word
    up = torch.full((N,), 1.0 / N, device="cuda")
    got = call(x, w, t, up, None)
    check(x, w, t, up, None, got)
    z = x.double() @ w.double().t()
    dz = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))[:, word] * up.double()
    dz[t == word] -= up[0].double()
    ref = dz @ x.double()
    # A rounding of a row's dz errs by up to a step (2 H), either way: the deviation of their sum is
    # H / sqrt(n) of it; that of the result's own D roundings, along the result, H / sqrt(D). Four of each.
    scale = (got[3][word].double() @ ref) / (ref @ ref) - 1
    assert scale.abs() <= 4 * H * (n ** -0.5 + D ** -0.5) < 0.9 * H  # to nearest it is 0.9 H


@pytest.mark.gpu
@pytest.mark.parametrize("V", [1, 2, 300, 5000])
def test_losses_of_confident_rows(V):
    # All logits are 16384 but the target's, 6 to 13 more: lse has steps of 2^-9 there, the loss,
    # log(1 + (V - 1) exp(-6 ..)), must not. The products are sums of small integers: exact.
    N, D = 40, 64
    t = torch.arange(N, device="cuda") % min(V, 8)
    x = torch.zeros(N, D, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = w[:, 0] = 128
    x[torch.arange(N, device="cuda"), 1 + t] = 1
    for k in range(min(V, 8)):
        w[k, 1 + k] = 6 + k
    loss, _ = call(x, w, t, torch.ones(N, device="cuda"), None, backward=False)
    z = x.double() @ w.double().t()
    want = torch.logsumexp(z, 1) - z.gather(1, t[:, None]).squeeze(1)
    # The sum is 1 and the others: exponentials good to 2^-20 and at most V / 16 + 64 additions, then
    # a logarithm and its result, and a difference of the maximum, which is exact.
    assert (loss >= 0).all()
    rel = 2.0 ** -20 + 2.0 ** -24 * (V / 16 + 64)
    assert ((loss.double() - want).abs() <= rel + 2.0 ** -22 * want).all()


@pytest.mark.gpu
@pytest.mark.parametrize("power", [10, 20, 60])
def test_losses_of_very_large_logits(power):
    # Logits of 2^20, 2^40 and 2^120, exact: two words share the maximum of every row, the others lie
    # at half of it and at its negative.
    N, V, D = 20, 130, 64
    x = torch.zeros(N, D, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
    x[:, 3] = 2.0 ** power
    w[:, 3] = -(2.0 ** power)
    w[70:, 3] = 2.0 ** (power - 1)
    w[5, 3] = w[101, 3] = 2.0 ** power
    t = torch.tensor([5, 101, 80, 7], device="cuda").repeat(5)
    loss, lse = call(x, w, t, torch.ones(N, device="cuda"), None, backward=False)
    top = 2.0 ** (2 * power)
    want = (torch.tensor([0.0, 0.0, top / 2, 2 * top], dtype=torch.float64, device="cuda") + math.log(2.0)).repeat(5)
    assert ((loss.double() - want).abs() <= 2.0 ** -22 * want).all()
    assert ((lse.double() - (top + math.log(2.0))).abs() <= 2.0 ** -22 * top).all()


@pytest.mark.gpu
@pytest.mark.parametrize("power", [10, 20, 60])
def test_gradients_of_very_large_logits(power):
    # The same logits; a row's lse is what fp32 leaves of it, and dz = exp(z - lse) by that.
    V, D = 130, 64
    x = torch.zeros(1, D, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
    x[:, 3] = 2.0 ** power
    w[:, 3] = -(2.0 ** power)
    w[70:, 3] = 2.0 ** (power - 1)
    w[5, 3] = w[101, 3] = 2.0 ** power
    one = torch.ones(1, device="cuda")
    _, lse, _, dw = call(x, w, torch.tensor([80], device="cuda"), one, None)
    want = torch.exp(w[:, 3].double() * 2.0 ** power - lse.double())
    want[80] -= 1
    want *= 2.0 ** power
    # Rounded as dz and as dweight (a word of one row has the first back, but not the words that
    # are no target), an exponential good to 2^-20.
    assert ((dw[:, 3].double() - want).abs() <= (2 * H + 2.0 ** -19) * want.abs() + TINY).all()
    assert (dw[:, :3] == 0).all() and (dw[:, 4:] == 0).all()


@pytest.mark.gpu
def test_the_mean_is_over_the_rows_that_carry_a_loss():
    from adaln_layernorm_modulate_gb300.autograd import linear_cross_entropy
    x, w, t, _, _ = inputs(300, 400, 64, 0.2, seed=23)
    t[17], t[200], t[299] = 400, -1, 2 ** 40  # no words: they carry none
    on = (t >= 0) & (t < 400)
    rows = linear_cross_entropy(x, w, t, reduction="none")
    assert torch.equal(linear_cross_entropy(x, w, t), rows.sum() / on.sum())
    # ignore_index may be a word of the vocabulary.
    t[on] = t[on].clamp(max=398)
    t[:5] = 399
    on = (t >= 0) & (t < 399)
    rows = linear_cross_entropy(x, w, t, ignore_index=399, reduction="none")
    assert torch.equal(linear_cross_entropy(x, w, t, ignore_index=399), rows.sum() / on.sum())


def pieces(N, V):
    """The vocabulary pieces of a backward, from the limits in the library's source."""
    import os
    import re
    src = open(os.path.join(os.path.dirname(A.__file__), "csrc", "adaln.cu")).read()
    mib, = re.findall(r"kProbsBytes = \(int64_t\)(\d+) << 20;", src)
    least, = re.findall(r"kMinPiece = (\d+);", src)
    rows = -(-max(N, 1) // 256) * 256
    wide = max((int(mib) << 20) // 2 // rows // 256 * 256, int(least))
    return -(-V // wide)


def test_the_tests_vocabularies_go_in_several_pieces():
    assert pieces(8192, 20001) == 2 and pieces(2049, 70000) == 2 and pieces(8191, 17000) == 2
    assert pieces(2500, 120001) == 3 and pieces(8192, 9001) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("N,V,D,ignored,n", [(600, 9000, 1288, 0.0, 1), (8191, 17000, 648, 0.4, 2),
                                             (4100, 24, 264, 0.1, 1), (3000, 256, 640, 0.0, 1),
                                             (2500, 120001, 328, 0.2, 3)])
def test_full_tiles(N, V, D, ignored, n):
    # Both gradients from 256-column tiles with several tiles and K steps each way, in one piece and
    # in more; thousands of rows of a few words.
    assert pieces(N, V) == n
    x, w, t, up, ul = inputs(N, V, D, ignored, seed=24)
    t[0], t[1] = 0, V - 1
    check(x, w, t, up, ul, call(x, w, t, up, ul))


@pytest.mark.parametrize("V,D", [(1, 8), (300, 64), (8192, 1024), (32000, 1536), (50257, 2048), (131072, 1024),
                                 (1 << 20, 4096)])
def test_a_workspace_holds_every_smaller_batch(V, D):
    for size in (A.adaln_linear_xent_fwd_workspace_size, A.adaln_linear_xent_bwd_workspace_size):
        sizes = [size(n, V, D, 1) for n in list(range(0, 600, 37)) + list(range(768, 40000, 256))]
        assert all(a <= b for a, b in zip(sizes, sizes[1:]))


@pytest.mark.gpu
def test_a_smaller_batch_in_a_larger_ones_workspace():
    # 2560 rows keep dz of all 50257 words at once, 2816 rows in two pieces; 512 rows have narrower
    # tiles, and so more partial sums of the forward, than 768.
    V, D = 50257, 64
    assert pieces(2560, V) == 1 and pieces(2816, V) == 2
    for most, N, words in ((2816, 2560, V), (768, 512, 8192)):
        x, w, t, up, ul = inputs(N, words, D, 0.1, seed=25)
        want = call(x, w, t, up, ul)
        loss, lse, dx, dw = (torch.empty_like(v) for v in want)
        for forward in (True, False):
            size = A.adaln_linear_xent_fwd_workspace_size if forward else A.adaln_linear_xent_bwd_workspace_size
            nb = size(most, words, D, 1)
            ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
            if forward:
                A.adaln_linear_xent_fwd(x, w, t, loss, lse, N, words, D, IGNORE, ws, nb)
            else:
                A.adaln_linear_xent_bwd(x, w, t, lse, up, ul, dx, dw, N, words, D, IGNORE, ws, nb)
        assert all(torch.equal(a, b) for a, b in zip((loss, lse, dx, dw), want))


@pytest.mark.gpu
@pytest.mark.parametrize("ignored", [0.0, 0.3])
@pytest.mark.parametrize("N,V,D", [(4096, 24, 256), (8192, 16, 520), (20001, 5, 264), (3001, 300, 1032),
                                   (2000, 100, 4104), (700, 2, 72), (9, 1, 8), (40000, 900, 72)])
def test_words_of_many_rows_keep_their_targets_remainders(N, V, D, ignored):
    # Every target's rounding is given back in fp32, however many rows a word has: what is left is the
    # rounding of the other elements of dz, and the result's.
    x, w, t, up, ul = inputs(N, V, D, ignored, seed=26)
    got = call(x, w, t, up, ul)
    check(x, w, t, up, ul, got)
    again = call(x, w, t, up, ul, want_x=False)
    assert torch.equal(again[3], got[3])
    on = (t >= 0) & (t < V)
    xd, td = x[on].double(), t[on]
    z = xd @ w.double().t()
    dz = torch.exp(z - torch.logsumexp(z, 1, keepdim=True)) * (up + ul)[on].double()[:, None]
    rows = torch.arange(len(td), device="cuda")
    others = dz.clone()
    others[rows, td] = 0
    dz[rows, td] -= up[on].double()
    ref = dz.t() @ xd
    # A rounding is even over its half step: h / sqrt(3) at most, root mean square, all independent. A
    # twentieth more for the sample of D * V of them (a quarter below 10,000), and the fp32 sums.
    size = (H ** 2 / 3 * (ref.norm() ** 2 + ((others ** 2).t() @ xd ** 2).sum())) ** 0.5
    fp32 = 2.0 ** -18 * (dz.t().abs() @ xd.abs()).norm()
    assert (got[3].double() - ref).norm() <= (1.05 if D * V > 10000 else 1.25) * size + fp32


@pytest.mark.gpu
def test_words_of_many_and_of_very_many_rows():
    # More rows than are looked at together: words of a few hundred rows go by lists, the others not.
    N, V, D = 30000, 400, 136
    x, w, t, up, ul = inputs(N, V, D, 0.1, seed=28)
    t[::3] = torch.where(t[::3] == IGNORE, t[::3], t[::3] % 4)
    t[7:7 + 512 * 2:2] = 399
    t[N - 1] = 399
    got = call(x, w, t, up, ul)
    check(x, w, t, up, ul, got)
    assert all(torch.equal(a, b) for a, b in zip(call(x, w, t, up, ul), got))


@pytest.mark.gpu
@pytest.mark.parametrize("N,V,D", [(300, 16, 2048), (2000, 24, 2048)])
def test_losses_of_wide_rows_and_few_words_keep_a_millionth(N, V, D):
    # The tensor cores cut a sum after each 16 products, always towards zero, so that the errors of
    # D / 16 steps add up. Losses of a few words (2 or 3) show it most; 2^-20 of them is asked for.
    x, w, t, up, ul = inputs(N, V, D, seed=27)
    loss, lse = call(x, w, t, up, ul, backward=False)
    z = x.double() @ w.double().t()
    L = torch.logsumexp(z, 1)
    want = L - z.gather(1, t[:, None]).squeeze(1)
    assert (lse.double() - L).norm() <= 2.0 ** -20 * L.norm()
    assert (loss.double() - want).norm() <= 2.0 ** -20 * want.norm()
