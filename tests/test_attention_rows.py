"""What reaches a row of attention and what does not: other rows of its tile, other segments, queries that
see no key; that every output is written, and nothing that is not asked for."""
import math

import pytest
import torch

import adaln_layernorm_modulate_gb300 as A
from tests.test_attention import CASES, call, check, inputs

GRADS = ("o", "dq", "dk", "dv")
H, U = 2.0 ** -8, 2.0 ** -24


def changed(i, **rows):
    """A copy of the inputs; name -> (rows, factor)."""
    j = {n: (v.clone() if torch.is_tensor(v) else v) for n, v in i.items()}
    for n, (at, f) in rows.items():
        j[n][at] = (j[n][at].float() * f).bfloat16()
    return j


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens_q,lens_k,causal", [([70, 60], [600, 600], False), ([9, 200], [3000, 300], False),
                                                  ([270, 300], [900, 300], True), ([1, 500], [5000, 500], False)])
def test_finite_neighbours_do_not_matter(lens_q, lens_k, causal, d):
    # The second segment's queries share a tile with the first one's; their scores on its keys differ by
    # hundreds from tile to tile. The keys grow along the segment, so that the maxima do.
    i = inputs(lens_q, lens_k, 4, 2, d, seed=40)
    n, m = lens_q[0], lens_k[0]
    ramp = 0.5 + torch.arange(m, device="cuda")[:, None, None] / m
    i = changed(i, k=(slice(0, m), ramp))
    want = call(i, causal)
    got = call(changed(i, q=(slice(n, None), 50), dout=(slice(n, None), 7), v=(slice(m, None), 3)), causal)
    for x, at in (("o", n), ("dq", n), ("dk", m), ("dv", m)):
        assert torch.equal(got[x][:at], want[x][:at]), x
    assert torch.equal(got["lse"][:, :n], want["lse"][:, :n])


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,m,causal", [(128, 700, False), (1000, 1000, True), (5, 4000, False)])
def test_a_row_does_not_depend_on_the_rows_beside_it(n, m, causal, d):
    i = inputs([n], [m], 2, 1, d, seed=41)
    want = call(i, causal)
    odd = torch.arange(n, device="cuda") % 2 == 1
    got = call(changed(i, q=(odd, 40), dout=(odd, 3)), causal)
    for x in ("o", "dq"):
        assert torch.equal(got[x][~odd], want[x][~odd]), x
    assert torch.equal(got["lse"][:, ~odd], want["lse"][:, ~odd])


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(CASES))
def test_every_output_is_written(name):
    # (check() takes a dq that is NaN throughout for one that was not asked for.)
    lens_q, lens_k, Hq, Hk, d, causal = CASES[name]
    i = inputs(lens_q, lens_q if lens_k is None else lens_k, Hq, Hk, d, seed=50 + len(name))
    got = call(i, causal)
    assert not any(got[n].isnan().any() for n in GRADS + ("lse",))
    check(i, got, causal)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens_q,lens_k", [([300, 129], [200, 40]), ([400, 5, 90], [150, 5, 0]), ([2000], [700])])
@pytest.mark.parametrize("q_value,dout_value", [(1.0, math.inf), (1.0, math.nan), (math.nan, 1.0), (-math.inf, math.nan)])
def test_queries_that_see_no_key(lens_q, lens_k, d, q_value, dout_value):
    # Causal, more queries than keys: the first queries of a segment see nothing. They may hold anything.
    i = inputs(lens_q, lens_k, 4, 2, d, seed=42)
    want = call(i, True)
    none = torch.cat([torch.arange(n, device="cuda") < n - m for n, m in zip(lens_q, lens_k)])
    got = call(changed(i, q=(none, q_value), dout=(none, dout_value)), True)
    for n in GRADS:
        assert torch.equal(got[n], want[n]), n
    assert torch.equal(got["lse"], want["lse"])
    assert (got["o"][none] == 0).all() and (got["dq"][none] == 0).all() and (got["lse"][:, none] == -math.inf).all()


@pytest.mark.gpu
def test_a_list_that_is_not_wanted_is_not_made():
    # 2000 segments of a query and a key: an entry of 32 bytes each in either work list.
    i = inputs([1] * 2000, [1] * 2000, 2, 2, 64, seed=43)
    (R, H, d), nseg = i["q"].shape, 2000
    o, lse = torch.empty_like(i["q"]), torch.empty(H, R, device="cuda")
    nb = max(f(nseg, R, R, H, H, d, 1) for f in (A.adaln_attention_fwd_workspace_size, A.adaln_attention_bwd_workspace_size))
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    A.adaln_attention_fwd(i["q"], i["k"], i["v"], o, lse, i["cu_q"], i["cu_k"], nseg, R, R, H, H, d, *[H * d] * 4,
                          0.125, False, ws, nb)
    written = {}
    for name, want_q, want_kv in (("both", True, True), ("q", True, False), ("kv", False, True)):
        dx = [torch.empty_like(i["q"]) for _ in range(3)]
        ws.fill_(255)
        A.adaln_attention_bwd(i["dout"], i["q"], i["k"], i["v"], o, lse, dx[0] if want_q else None,
                              *(dx[1:] if want_kv else (None, None)), i["cu_q"], i["cu_k"], nseg, R, R, H, H, d,
                              *[H * d] * 8, 0.125, False, ws, nb)
        assert A.adaln_read_status(ws) == 0
        written[name] = int((ws != 255).sum())
    # (Numbers below 2000 have no byte of 255 but their lowest, one in 256 of them.)
    assert written["both"] - written["q"] >= 2000 * 28 and written["both"] - written["kv"] >= 2000 * 28, written


@pytest.mark.gpu
@pytest.mark.parametrize("want_q", [True, False])
def test_one_list_alone_checks_the_tables_too(want_q):
    i = inputs([40, 60], [40, 60], 2, 2, 64, seed=44)
    j = dict(i, cu_q=torch.tensor([0, 60, 40], dtype=torch.int32, device="cuda"))
    got = call(j, status=6, want_q=want_q, want_kv=not want_q)
    assert all(t.isnan().all() for t in got.values())


@pytest.mark.gpu
def test_workspace_has_no_room_for_pieces_that_cannot_be():
    # Units of fewer than eight steps are never cut. 32 segments of 256: the status, work lists and
    # statistics of the rows, nothing else.
    R, H, d = 32 * 256, 12, 128
    fwd, bwd = A.adaln_attention_fwd_workspace_size, A.adaln_attention_bwd_workspace_size
    assert fwd(32, R, 7 * 128, H, H, d, 1) <= 65536
    assert bwd(32, 7 * 128, 7 * 128, H, H, d, 1) <= 65536 + 8 * H * 7 * 128
    assert fwd(32, R, 8 * 128, H, H, d, 1) > 1 << 20 and bwd(32, R, R, H, H, d, 1) > 1 << 20


@pytest.mark.gpu
@pytest.mark.parametrize("n", [896, 897])  # seven tiles, eight
@pytest.mark.parametrize("d", [64, 128])
def test_both_sides_of_the_pieces_border(n, d):
    for heads, kv in ((1, 1), (3, 3), (2, 1)):
        i = inputs([n], [n], heads, kv, d, seed=45)
        check(i, call(i))
        check(i, call(i, True), True)


@pytest.mark.gpu
@pytest.mark.parametrize("N,M", [(5, 0), (0, 7), (0, 0), (5, 7)])
@pytest.mark.parametrize("packed", [False, True])
def test_node_with_gradients_of_one_side(N, M, packed):
    # A side that wants its gradient may have no rows.
    from adaln_layernorm_modulate_gb300.autograd import attention
    for wanted in ("q", "k", "v", "kv"):
        q, k, v = (torch.randn(3, n, h, 64, device="cuda", dtype=torch.bfloat16) for n, h in ((N, 4), (M, 2), (M, 2)))
        cu = [torch.arange(4, device="cuda", dtype=torch.int32) * n for n in (N, M)] if packed else []
        x = [(t.flatten(0, 1) if packed else t).requires_grad_(n in wanted) for n, t in zip("qkv", (q, k, v))]
        attention(*x, *cu, check_tables=True).sum().backward()
        for n, t in zip("qkv", x):
            assert (t.grad is None) == (n not in wanted)
            assert t.grad is None or (t.grad.shape == t.shape and not t.grad.isnan().any())
            assert t.grad is None or (N and M) or (t.grad == 0).all()


def average_errors(i, causal):
    """Errors of dq, dk and dv in the 2-norm, over what independent roundings leave: results and dz (for dv: p) are
    off by at most H of each value, H / sqrt(3) in the mean square where all have the worst mantissa."""
    got = call(i, causal)
    q, k, v, do = (i[n].double() for n in ("q", "k", "v", "dout"))
    group, scale = q.shape[1] // k.shape[1], q.shape[2] ** -0.5
    bad, size = torch.zeros(3, dtype=torch.float64), torch.zeros(3, dtype=torch.float64)
    a = b = 0
    for n, m in zip(i["lens_q"], i["lens_k"]):
        Q, D = (t[a: a + n].transpose(0, 1) for t in (q, do))
        K, V = (t[b: b + m].repeat_interleave(group, 1).transpose(0, 1) for t in (k, v))
        z = scale * Q @ K.transpose(1, 2)
        if causal:
            z = z.masked_fill(torch.ones(n, m, dtype=torch.bool, device="cuda").triu(m - n + 1), -math.inf)
        p = torch.softmax(z, 2).nan_to_num(0)
        dp = D @ V.transpose(1, 2)
        dz = scale * p * (dp - (p * dp).sum(2, keepdim=True))
        shared = lambda t: t.unflatten(0, (-1, group)).sum(1)
        ref = dz @ K, shared(dz.transpose(1, 2) @ Q), shared(p.transpose(1, 2) @ D)
        terms = (dz ** 2) @ K ** 2, shared((dz ** 2).transpose(1, 2) @ Q ** 2), shared((p ** 2).transpose(1, 2) @ D ** 2)
        for x, (name, r0, r1) in enumerate((("dq", a, a + n), ("dk", b, b + m), ("dv", b, b + m))):
            bad[x] += (got[name][r0:r1].double().transpose(0, 1) - ref[x]).square().sum().cpu()
            size[x] += (ref[x].square().sum() + terms[x].sum()).cpu()
        a, b = a + n, b + m
    return (bad / (size * H ** 2 / 3)).sqrt()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [8, 40, 64, 128])
@pytest.mark.parametrize("n,m,causal", [(400, 2, False), (400, 3, False), (77, 16, False), (200, 32, False), (2, 2, True),
                                        (3, 3, True), (17, 17, True), (31, 33, True), (40, 8, True)])
def test_gradients_of_rows_of_few_keys(n, m, causal, d):
    # dp - delta is a difference of near values there: delta of a rounded o would be off by as much as dz is.
    # Many short segments of other lengths among them, so that groups of rows hold several.
    times = max(1, 1200 // n)
    lens_q, lens_k = [n] * times + [0, n, 1, 5], [m] * times + [m, 0, 1, 4]
    i = inputs(lens_q, lens_k, 4, 2, d, seed=46)
    # More roundings than a thousand, so that their mean square is near its expectation; fp32's own errors are
    # far below.
    assert (average_errors(i, causal) <= 1.1).all()


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [False, True])
def test_rows_of_one_key_have_no_gradient(causal):
    # p = 1 and dp = delta: what is left is the difference of two sums of d products in fp32, 2 (d / 16 + 12) U of
    # their sizes, and p's own error of 2^-20.
    i = inputs([1] * 700, [1] * 700, 4, 2, 64, seed=47)
    got = call(i, causal)
    dp = (i["dout"].double().unflatten(1, (2, 2)).abs() * i["v"].double().abs()[:, :, None]).sum(3, keepdim=True)
    err = 64 ** -0.5 * (2 * 16 * U + 2.0 ** -20) * dp
    K, Q = i["k"].double().abs()[:, :, None], i["q"].double().abs().unflatten(1, (2, 2))
    assert (got["dq"].double().abs().unflatten(1, (2, 2)) <= err * K).all()
    assert (got["dk"].double().abs() <= (err * Q).sum(2)).all()
