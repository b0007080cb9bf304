"""Attention over packed sequences against its definition in 64 bits (torch, on the tensors' device), its
gradients against differences of that definition, and its refusals.

Tolerances. H = 2^-8 is half a step of bf16, U = 2^-24 of fp32. The tensor cores cut a sum towards
zero after every 16 products: 2^-23 of what has been summed each time, so a sum of n products is
off by at most 2^-23 (n / 16 + 1) of its terms' sizes.
  z    that, over d terms, and the rounding of the exponent's argument and of its reference: 8 U of the
       largest score of the row; exp2 itself 2^-21.
  p    the exponential of a difference of two such (relative: twice z's error), rounded to bf16: H.
  o    a sum of p v over the row's keys: p's relative error and the sum's own on sum p |v|, rounded once: H.
  dz   p (dp - delta): dp as z; delta = dout . o with o's error, and 24 U for its own sum; p's
       relative error; rounded to bf16: H.
  dq, dk, dv   sums of dz k, dz q, p dout with these errors, rounded once."""
import math

import pytest
import torch

import adaln_layernorm_modulate_gb300 as A

H, U = 2.0 ** -8, 2.0 ** -24


def test_shape_pointer_and_argument_checks():
    L = A.lib()

    def fwd(p=(16,) * 7, nseg=2, Rq=8, Rk=8, Hq=4, Hk=2, d=64, ld=(256, 128, 128, 256), scale=0.1, ws=256, nb=1 << 30,
            dt=1):
        return L.adaln_attention_fwd(*p, nseg, Rq, Rk, Hq, Hk, d, *ld, scale, 0, ws, nb, dt, None)

    assert [fwd(d=v) for v in (0, 4, 12, 136)] == [2] * 4 and fwd(dt=0) == 2 and fwd(dt=3) == 1
    assert fwd(nseg=-1) == 1 and fwd(Rq=-1) == 1 and fwd(Rk=2 ** 31) == 1 and fwd(Hk=3) == 1 and fwd(Hk=0) == 1
    assert fwd(Hq=0) == 1 and fwd(Hq=2, Hk=4) == 1
    assert [fwd(scale=v) for v in (0.0, -1.0, float("inf"), float("nan"))] == [1] * 4
    assert fwd(nseg=0) == 1  # rows without a segment
    assert fwd(p=(16,) * 5 + (None, 16), Rq=7) == 1  # no table, and no equal lengths
    assert fwd(p=(16,) * 6 + (None,), Rk=7) == 1
    for i in range(5):
        p = [16] * 7
        p[i] = None
        assert fwd(p=tuple(p)) == 1, i
        p[i] = 18
        assert fwd(p=tuple(p)) == 3, i
    assert fwd(p=(16,) * 5 + (18, 16)) == 3
    for i in range(4):
        ld = [256, 128, 128, 256]
        ld[i] -= 8
        assert fwd(ld=tuple(ld)) == 1, i
        ld[i] += 9
        assert fwd(ld=tuple(ld)) == 3, i

    def bwd(p=(16,) * 11, Rq=8, Rk=8, ld=(256, 256, 128, 128, 256, 256, 128, 128), scale=0.1, d=64, dt=1):
        return L.adaln_attention_bwd(*p, 2, Rq, Rk, 4, 2, d, *ld, scale, 0, 256, 1 << 30, dt, None)

    assert bwd(d=12) == 2 and bwd(dt=0) == 2 and bwd(scale=0.0) == 1 and bwd(Rq=-1) == 1
    for i in range(6):
        p = [16] * 11
        p[i] = None
        assert bwd(p=tuple(p)) == 1, i
    assert bwd(p=(16,) * 7 + (None,) + (16,) * 3) == 1  # dk and dv go together
    assert bwd(p=(16,) * 6 + (None,) * 3 + (16,) * 2) == 1
    for i in range(8):
        ld = [256, 256, 128, 128, 256, 256, 128, 128]
        ld[i] -= 8
        assert bwd(ld=tuple(ld)) == 1, i
    assert A.adaln_attention_fwd_workspace_size(2, 8, 8, 4, 2, 12, 1) == 0
    assert A.adaln_attention_bwd_workspace_size(2, 8, 8, 4, 3, 64, 1) == 0


def test_refusals_of_the_node():
    from adaln_layernorm_modulate_gb300.autograd import attention
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        attention(x, x, x, torch.tensor([0, 4]))


def inputs(lens_q, lens_k, Hq, Hk, d, seed=0, spread=1.2, joint=False):
    g = torch.Generator("cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
    Rq, Rk = sum(lens_q), sum(lens_k)
    if joint:
        rows = (spread * rand(Rq, (Hq + 2 * Hk) * d)).bfloat16()
        q, k, v = (t.unflatten(1, (-1, d)) for t in rows.split([Hq * d, Hk * d, Hk * d], 1))
    else:
        q, k, v = (spread * rand(Rq, Hq, d)).bfloat16(), (spread * rand(Rk, Hk, d)).bfloat16(), rand(Rk, Hk, d).bfloat16()
    cu = [torch.tensor([0] + list(x), device="cuda").cumsum(0).to(torch.int32) for x in (lens_q, lens_k)]
    return dict(q=q, k=k, v=v, dout=rand(Rq, Hq, d).bfloat16(), cu_q=cu[0], cu_k=cu[1], lens_q=lens_q, lens_k=lens_k)


def ld(t):
    return t.stride(0) if t.shape[0] > 1 else t.shape[1] * t.shape[2]


def call(i, causal=False, scale=None, status=0, pad=16, dense=False, want_q=True, want_kv=True):
    q, k, v, dout = i["q"], i["k"], i["v"], i["dout"]
    (Rq, Hq, d), (Rk, Hk, _) = q.shape, k.shape
    nseg = i["cu_q"].numel() - 1
    scale = d ** -0.5 if scale is None else scale
    cu_q, cu_k = (None, None) if dense else (i["cu_q"], i["cu_k"])
    nan = float("nan")
    wide = {n: torch.full((R, h * d + pad), nan, dtype=torch.bfloat16, device="cuda")
            for n, R, h in (("o", Rq, Hq), ("dq", Rq, Hq), ("dk", Rk, Hk), ("dv", Rk, Hk))}
    lse = torch.full((Hq, Rq), nan, device="cuda")
    nb = A.adaln_attention_fwd_workspace_size(nseg, Rq, Rk, Hq, Hk, d, 1)
    ws = torch.full((nb,), 255, dtype=torch.uint8, device="cuda")
    lo, lk = Hq * d + pad, Hk * d + pad
    A.adaln_attention_fwd(q, k, v, wide["o"], lse, cu_q, cu_k, nseg, Rq, Rk, Hq, Hk, d, ld(q), ld(k), ld(v), lo, scale,
                          causal, ws, nb)
    assert A.adaln_read_status(ws) == status
    nb = A.adaln_attention_bwd_workspace_size(nseg, Rq, Rk, Hq, Hk, d, 1)
    ws = torch.full((nb,), 255, dtype=torch.uint8, device="cuda")
    A.adaln_attention_bwd(dout, q, k, v, wide["o"], lse, wide["dq"] if want_q else None, wide["dk"] if want_kv else None,
                          wide["dv"] if want_kv else None, cu_q, cu_k, nseg, Rq, Rk, Hq, Hk, d, ld(dout), ld(q), ld(k),
                          ld(v), lo, lo, lk, lk, scale, causal, ws, nb)
    assert A.adaln_read_status(ws) == status
    out = {"lse": lse}
    for n, t in wide.items():
        if pad:
            assert t[:, t.shape[1] - pad:].isnan().all(), "wrote between the rows of " + n
        out[n] = t[:, : t.shape[1] - pad].unflatten(1, (-1, d))
    return out


def check(i, got, causal=False, scale=None):
    q, k, v, dout = (i[n].double() for n in ("q", "k", "v", "dout"))
    (Rq, Hq, d), (Rk, Hk, _) = q.shape, k.shape
    scale = d ** -0.5 if scale is None else scale
    group = Hq // Hk
    cut = lambda n: 2.0 ** -23 * (n / 16 + 1)
    a = b = 0
    off = []

    def near(name, x, ref, err, where):
        bad = ((x.double() - ref).abs() > err + 1e-30) | (x.isnan() & ~ref.isnan())
        if bad.any():
            worst = ((x.double() - ref).abs() / (err + 1e-30)).nan_to_num(1e9).max().item()
            off.append((name, where, int(bad.sum()), worst))

    for s, (n, m) in enumerate(zip(i["lens_q"], i["lens_k"])):
        seen = torch.ones(n, m, dtype=torch.bool, device="cuda")
        if causal:
            seen = seen.tril(m - n)
        some = seen.any(1) if m else torch.zeros(n, dtype=torch.bool, device="cuda")
        for kv in range(Hk):
            K, V = k[b: b + m, kv], v[b: b + m, kv]
            dk, dv, e_dk, e_dv = (torch.zeros(m, d, dtype=torch.float64, device="cuda") for _ in range(4))
            for h in range(kv * group, (kv + 1) * group):
                Q, D = q[a: a + n, h], dout[a: a + n, h]
                z = scale * Q @ K.t()
                e_z = cut(d) * scale * Q.abs() @ K.abs().t()
                z = z.masked_fill(~seen, -math.inf)
                top = torch.where(some[:, None], z.masked_fill(~seen, 0).abs().amax(1, keepdim=True) if m else 0, 0)
                e_z = (e_z.amax(1, keepdim=True) if m else 0) + 8 * U * top + 2.0 ** -21
                lse = torch.logsumexp(z, 1) if m else torch.full((n,), -math.inf, device="cuda")
                p = torch.where(seen, torch.exp(z - torch.where(some, lse, 0)[:, None]), 0)
                e_p = 2 * e_z
                o = p @ V
                e_o = (H + 2 * e_p + cut(m) + 4 * U) * (p @ V.abs()) + H * o.abs()
                where = (s, h, n, m)
                gl = got["lse"][h, a: a + n]
                assert ((gl == -math.inf) == ~some).all(), where
                near("lse", gl[some], lse[some], (e_z.flatten()[some] if m else 0) + U * (m / 16 + 64) + 2 * U * lse[some].abs(), where)
                near("o", got["o"][a: a + n, h], o, e_o, where)
                dp = D @ V.t()
                delta = (D * o).sum(1, keepdim=True)
                e_delta = (D.abs() * (e_o + 24 * U * o.abs())).sum(1, keepdim=True)
                e_dp = cut(d) * D.abs() @ V.abs().t()
                dz = p * (dp - delta)
                e_dz = p * (e_dp + e_delta + (e_p + 4 * U) * (dp - delta).abs())
                e_dz = e_dz + H * (dz.abs() + e_dz)
                dq = scale * dz @ K
                e_dq = scale * (e_dz @ K.abs() + cut(m) * dz.abs() @ K.abs())
                if not got["dq"].isnan().all() or n == 0:
                    near("dq", got["dq"][a: a + n, h], dq, e_dq + H * (dq.abs() + e_dq), where)
                dk += scale * dz.t() @ Q
                e_dk += scale * (e_dz.t() @ Q.abs() + cut(n * group) * dz.abs().t() @ Q.abs())
                dv += p.t() @ D
                e_dv += (p * (H + e_p * (1 + H) + cut(n * group))).t() @ D.abs()
            near("dk", got["dk"][b: b + m, kv], dk, e_dk + H * (dk.abs() + e_dk), (s, kv, n, m))
            near("dv", got["dv"][b: b + m, kv], dv, e_dv + H * (dv.abs() + e_dv), (s, kv, n, m))
        a, b = a + n, b + m
    assert not off, off[:8]


# Queries, keys (None: the same), heads, key heads, elements of a head, causal.
CASES = {
    "one": ([1], [1], 1, 1, 8, False),
    "tile": ([128], [128], 1, 1, 64, False),
    "tile-wide": ([128], [128], 1, 1, 128, False),
    "two-tiles": ([256], [256], 2, 1, 128, False),
    "causal-tile": ([128], None, 1, 1, 64, True),
    "causal": ([500], None, 2, 2, 128, True),
    "ragged": ([17, 0, 130, 5, 1], None, 4, 2, 64, True),
    "ragged-full": ([17, 0, 130, 5, 1, 384, 129], None, 3, 3, 128, False),
    "cross": ([300, 1, 77], [5, 200, 128], 4, 4, 64, False),
    "no-keys": ([50, 200, 3], [0, 100, 0], 2, 1, 64, False),
    "no-queries": ([0, 40, 0], [300, 10, 7], 2, 2, 72, False),
    "more-queries-causal": ([300, 129], [100, 1], 4, 2, 64, True),
    "more-keys-causal": ([100, 1, 200], [700, 300, 201], 4, 1, 128, True),
    "odd-heads": ([200, 260], None, 6, 2, 24, True),
    "d80": ([333], [257], 2, 2, 80, False),
    "d96": ([260], [400], 2, 2, 96, True),
    "d120": ([140, 3], None, 3, 1, 120, True),
    "d16": ([1000], [900], 2, 2, 16, False),
    "groups": ([700, 90], None, 16, 2, 64, True),
    "split-1": ([1], [5000], 3, 3, 128, False),
    "split-causal": ([40], [3000], 2, 2, 64, True),
    "split-ragged": ([3, 2], [2000, 1], 2, 1, 72, False),
    "many": ([(7 * s) % 61 for s in range(90)], None, 2, 2, 64, True),
    "pieces": ([1100, 40], [2300, 700], 3, 3, 64, False),
    "pieces-causal": ([3000, 1500], None, 2, 1, 128, True),
    "pieces-groups": ([40, 1500], [1000, 1200], 8, 1, 72, False),
    "pieces-many": ([9, 700, 0, 2100, 130], [4000, 1, 50, 1030, 0], 1, 1, 32, False),
    "full-waves": ([2500, 1300], None, 12, 4, 64, False),
    "full-waves-wide": ([2000, 777, 1400], None, 12, 12, 128, True),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(CASES))
def test_against_the_definition(name):
    lens_q, lens_k, Hq, Hk, d, causal = CASES[name]
    i = inputs(lens_q, lens_q if lens_k is None else lens_k, Hq, Hk, d, seed=len(name))
    check(i, call(i, causal), causal)


@pytest.mark.gpu
def test_average_errors():
    # Roundings of different terms are independent: together they stay near one rounding's size.
    i = inputs([2000], [2000], 2, 2, 128, seed=1, spread=1.0)
    got = call(i)
    q, k, v, do = (i[n].double().transpose(0, 1) for n in ("q", "k", "v", "dout"))
    p = torch.softmax(128 ** -0.5 * q @ k.transpose(1, 2), 2)
    o = p @ v
    dp = do @ v.transpose(1, 2)
    dz = 128 ** -0.5 * p * (dp - (do * o).sum(2, keepdim=True))
    ref = dict(o=o, dq=dz @ k, dk=dz.transpose(1, 2) @ q, dv=p.transpose(1, 2) @ do)
    for n, r in ref.items():
        r = r.transpose(0, 1)
        assert (got[n].double() - r).norm() <= H * r.norm(), n


@pytest.mark.gpu
def test_scores_far_apart():
    # Scores of several hundred: all but a few probabilities are 0, maxima grow along the row.
    i = inputs([300], [600], 2, 2, 64, seed=2, spread=9.0)
    check(i, call(i), False)
    g = torch.arange(600, device="cuda")[:, None, None] / 40.0
    i["k"] = (i["k"].float() * g).bfloat16()
    check(i, call(i), False)
    i = inputs([300], [300], 2, 2, 64, seed=3)
    check(i, call(i, True, 3.0), True, 3.0)


@pytest.mark.gpu
def test_neighbours_do_not_matter():
    lens = [100, 200, 60, 129]
    i = inputs(lens, lens, 4, 2, 64, seed=4)
    want = call(i, True)
    for bad in (1, 3):
        j = {n: (v.clone() if torch.is_tensor(v) else v) for n, v in i.items()}
        rows = slice(sum(lens[:bad]), sum(lens[: bad + 1]))
        for n in ("q", "k", "v", "dout"):
            j[n][rows] = float("nan") if bad == 1 else float("inf")
        got = call(j, True)
        keep = torch.ones(sum(lens), dtype=torch.bool, device="cuda")
        keep[rows] = False
        for n in ("o", "dq", "dk", "dv"):
            assert torch.equal(got[n][keep], want[n][keep]), n
        assert torch.equal(got["lse"][:, keep], want["lse"][:, keep])
        assert got["o"][rows].isnan().all()


@pytest.mark.gpu
def test_dense_is_packed_with_equal_lengths():
    i = inputs([150] * 3, [70] * 3, 4, 2, 128, seed=5)
    want, got = call(i), call(i, dense=True)
    assert all(torch.equal(got[n], want[n]) for n in want)


@pytest.mark.gpu
def test_parts_of_a_joint_projection():
    i = inputs([90, 200], [90, 200], 4, 2, 64, seed=6, joint=True)
    assert i["q"].stride(0) == 8 * 64
    check(i, call(i, True), True)


@pytest.mark.gpu
def test_optional_gradients():
    i = inputs([90, 200], [200, 90], 4, 2, 64, seed=7)
    want = call(i)
    a, b = call(i, want_kv=False), call(i, want_q=False)
    assert torch.equal(a["dq"], want["dq"]) and a["dk"].isnan().all() and a["dv"].isnan().all()
    assert torch.equal(b["dk"], want["dk"]) and torch.equal(b["dv"], want["dv"]) and b["dq"].isnan().all()


@pytest.mark.gpu
@pytest.mark.parametrize("table", [[1, 40, 100], [0, 60, 40], [0, 40, 99], [0, 40, 101], [0, -5, 100], [0, 200, 100],
                                   [0, 2 ** 31 - 1, 100]])
def test_malformed_tables_compute_nothing(table):
    i = inputs([40, 60], [40, 60], 2, 2, 64, seed=8)
    for which in ("cu_q", "cu_k"):
        j = dict(i, **{which: torch.tensor(table, dtype=torch.int32, device="cuda")})
        got = call(j, status=6)
        assert all(t.isnan().all() for t in got.values())


@pytest.mark.gpu
def test_no_rows():
    for lens_q, lens_k in (([], []), ([0, 0], [0, 0]), ([5, 6], [0, 0]), ([0, 0], [5, 6])):
        i = inputs(lens_q, lens_k, 2, 2, 64)
        got = call(i)
        assert all((got[n] == 0).all() for n in ("o", "dq", "dk", "dv")) and (got["lse"] == -math.inf).all()


@pytest.mark.gpu
def test_offsets_past_32_bits():
    # Keys and values of 2.4e9 elements each; the rows near the end hold the weight.
    n, heads, d = 600_000, 32, 128
    g = torch.Generator("cuda").manual_seed(9)
    k = torch.zeros(n, heads, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros(n, heads, d, dtype=torch.bfloat16, device="cuda")
    q = torch.randn(2, heads, d, generator=g, device="cuda").bfloat16()
    k[-300:] = (8 * torch.randn(300, heads, d, generator=g, device="cuda")).bfloat16()
    v[-300:] = torch.randn(300, heads, d, generator=g, device="cuda").bfloat16()
    o, lse = torch.empty_like(q), torch.empty(heads, 2, device="cuda")
    cu_q, cu_k = (torch.tensor(t, dtype=torch.int32, device="cuda") for t in ([0, 1, 2], [0, 100, n]))
    nb = A.adaln_attention_fwd_workspace_size(2, 2, n, heads, heads, d, 1)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    args = (cu_q, cu_k, 2, 2, n, heads, heads, d)
    hd = heads * d
    A.adaln_attention_fwd(q, k, v, o, lse, *args, hd, hd, hd, hd, d ** -0.5, False, ws, nb)
    assert A.adaln_read_status(ws) == 0
    z = torch.einsum("hd,nhd->hn", q[1].double(), k[-300:].double()) * d ** -0.5
    z = torch.cat([z, torch.full((heads, 1), math.log(n - 400), device="cuda", dtype=torch.float64)], 1)
    L = torch.logsumexp(z, 1)
    p = torch.exp(z - L[:, None])[:, :300]
    ref = torch.einsum("hn,nhd->hd", p, v[-300:].double())
    size = torch.einsum("hn,nhd->hd", p, v[-300:].double().abs())
    e_z = 2.0 ** -23 * 9 * z.abs().amax() * 40 + 2.0 ** -21
    assert ((lse[:, 1].double() - L).abs() <= e_z + 2.0 ** -24 * n / 16).all() and (o[0] == 0).all()
    assert ((o[1].double() - ref).abs() <= (2 * H + 4 * e_z + 2.0 ** -23 * n / 16) * size).all()
    dout = torch.randn(2, heads, d, generator=g, device="cuda").bfloat16()
    dq, dk, dv = torch.empty_like(q), torch.full_like(k, float("nan")), torch.full_like(v, float("nan"))
    nb = A.adaln_attention_bwd_workspace_size(2, 2, n, heads, heads, d, 1)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    A.adaln_attention_bwd(dout, q, k, v, o, lse, dq, dk, dv, *args, hd, hd, hd, hd, hd, hd, hd, hd, d ** -0.5, False,
                          ws, nb)
    assert A.adaln_read_status(ws) == 0
    want = p.t()[:, :, None] * dout[1].double()
    assert ((dv[-300:].double() - want).abs() <= (3 * H + 4 * e_z) * want.abs() + 1e-30).all()
    assert not dk[-300:].isnan().any() and not dk[:: n // 50].isnan().any()


@pytest.mark.gpu
def test_differences_of_the_definition():
    from adaln_layernorm_modulate_gb300.autograd import attention
    i = inputs([60, 130], [60, 130], 4, 2, 64, seed=10)
    x = [i[n].clone().requires_grad_(True) for n in ("q", "k", "v")]
    o = attention(*x, i["cu_q"], causal=True, check_tables=True)
    o.backward(i["dout"])

    def f(q, k, v):
        total = 0
        for a, b in ((0, 60), (60, 190)):
            K, V = (t[a:b].repeat_interleave(2, 1).transpose(0, 1) for t in (k, v))
            z = 0.125 * q[a:b].transpose(0, 1) @ K.transpose(1, 2)
            z = z.masked_fill(torch.ones(b - a, b - a, dtype=torch.bool, device="cuda").triu(1), -math.inf)
            total = total + ((torch.softmax(z, 2) @ V).transpose(0, 1) * i["dout"][a:b].double()).sum()
        return total

    at = [t.detach().double() for t in x]
    g = torch.Generator("cuda").manual_seed(3)
    s = 1e-4
    for j in range(3):
        v = torch.randn(at[j].shape, generator=g, device="cuda", dtype=torch.float64)
        up, down = list(at), list(at)
        up[j], down[j] = at[j] + s * v, at[j] - s * v
        want = (f(*up) - f(*down)) / (2 * s)
        grad = x[j].grad.double()
        # independent roundings: of p or dz and at the end
        assert ((grad * v).sum() - want).abs() <= 4 * H * (grad * v).norm() + 1e-4


@pytest.mark.gpu
def test_autograd_matches_the_calls():
    from adaln_layernorm_modulate_gb300.autograd import attention
    i = inputs([100, 30], [40, 260], 4, 2, 64, seed=11)
    want = call(i, pad=0)
    q, k, v = (i[n].clone().requires_grad_(True) for n in ("q", "k", "v"))
    o, lse = attention(q, k, v, i["cu_q"].long(), i["cu_k"], return_lse=True)
    o.backward(i["dout"])
    assert torch.equal(o, want["o"]) and torch.equal(lse, want["lse"]) and not lse.requires_grad
    assert all(torch.equal(t.grad, want["d" + n]) for n, t in (("q", q), ("k", k), ("v", v)))
    # Dense, heads that do not lie side by side; an expanded gradient.
    i = inputs([48] * 3, [48] * 3, 4, 2, 64, seed=12)
    want = call(i, True, pad=0)
    q, k, v = (i[n].unflatten(0, (3, 48)).transpose(1, 2).contiguous().transpose(1, 2).requires_grad_(True)
               for n in ("q", "k", "v"))
    o = attention(q, k, v, causal=True)
    assert torch.equal(o.flatten(0, 1), want["o"])
    o.backward(i["dout"].view(3, 48, 4, 64))
    assert all(torch.equal(t.grad.flatten(0, 1), want["d" + n]) for n, t in (("q", q), ("k", k), ("v", v)))
    attention(q, k, v).sum().backward()
    frozen = attention(q.detach(), k.detach(), v.detach().requires_grad_(True))
    frozen.sum().backward()
    with pytest.raises(TypeError):
        attention(q.float(), k.float(), v.float())
    with pytest.raises(ValueError):
        attention(q, k, v[:, :40])
    with pytest.raises(ValueError):
        attention(q, k, v, i["cu_q"])
    with pytest.raises(A.AdalnError):
        attention(q[:, :, :3], k, v)
    with pytest.raises(A.AdalnError):
        attention(i["q"], i["k"], i["v"], i["cu_q"] + 1, check_tables=True)


@pytest.mark.gpu
@pytest.mark.parametrize("lens_k", [[300, 40], [3000, 3000]])
def test_repeat_side_stream_and_graph_replay(lens_k):
    i = inputs([300, 40] if lens_k[0] < 1000 else [3, 2], lens_k, 2, 1, 128, seed=13)
    want = call(i, pad=0)
    again = call(i, pad=0)
    assert all(torch.equal(again[n], want[n]) for n in want)
    (Rq, Hq, d), (Rk, Hk, _) = i["q"].shape, i["k"].shape
    out = {n: torch.empty_like(v) for n, v in want.items()}
    sizes = (2, Rq, Rk, Hq, Hk, d)
    nb = max(A.adaln_attention_fwd_workspace_size(*sizes, 1), A.adaln_attention_bwd_workspace_size(*sizes, 1))
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    lq, lk = Hq * d, Hk * d

    def both():
        A.adaln_attention_fwd(i["q"], i["k"], i["v"], out["o"], out["lse"], i["cu_q"], i["cu_k"], *sizes, lq, lk, lk, lq,
                              d ** -0.5, False, ws, nb)
        A.adaln_attention_bwd(i["dout"], i["q"], i["k"], i["v"], out["o"], out["lse"], out["dq"], out["dk"], out["dv"],
                              i["cu_q"], i["cu_k"], *sizes, lq, lq, lk, lk, lq, lq, lk, lk, d ** -0.5, False, ws, nb)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(out[n], want[n]) for n in want)
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    for g in (graph, other):  # two graphs with one workspace
        with torch.cuda.graph(g):
            both()
    for v in out.values():
        v.fill_(0)
    for _ in range(3):
        graph.replay()
        other.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out[n], want[n]) for n in want)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_calls_back_to_back(d):
    # Many steps a CTA, kernels queued behind each other: warps run apart as far as the barriers let them.
    i = inputs([9000, 3000], [500, 260], 8, 4, d, seed=15)
    want = call(i, pad=0)
    (Rq, Hq, _), (Rk, Hk, _) = i["q"].shape, i["k"].shape
    sizes = (2, Rq, Rk, Hq, Hk, d)
    nb = A.adaln_attention_bwd_workspace_size(*sizes, 1)
    runs = []
    for _ in range(12):
        out = {n: torch.empty_like(want[n]) for n in ("dq", "dk", "dv")}
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        runs.append((out, ws))
    torch.cuda.synchronize()
    lq, lk = Hq * d, Hk * d
    for out, ws in runs:
        A.adaln_attention_bwd(i["dout"], i["q"], i["k"], i["v"], want["o"], want["lse"], out["dq"], out["dk"], out["dv"],
                              i["cu_q"], i["cu_k"], *sizes, lq, lq, lk, lk, lq, lq, lk, lk, d ** -0.5, False, ws, nb)
    for out, ws in runs:
        assert A.adaln_read_status(ws) == 0
        assert all(torch.equal(out[n], want[n]) for n in out)


@pytest.mark.gpu
def test_two_streams_at_once():
    sets = [inputs([900, 300], [900, 300], 4, 2, 64, seed=30), inputs([5, 400], [3000, 200], 2, 2, 128, seed=31)]
    want = [call(i, pad=0) for i in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for n, i in enumerate(sets):
            with torch.cuda.stream(streams[n]):
                (Rq, Hq, d), (Rk, Hk, _) = i["q"].shape, i["k"].shape
                sizes = (2, Rq, Rk, Hq, Hk, d)
                out = {m: torch.empty_like(t) for m, t in want[n].items()}
                nb = max(A.adaln_attention_fwd_workspace_size(*sizes, 1), A.adaln_attention_bwd_workspace_size(*sizes, 1))
                ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
                lq, lk, sc = Hq * d, Hk * d, d ** -0.5
                A.adaln_attention_fwd(i["q"], i["k"], i["v"], out["o"], out["lse"], i["cu_q"], i["cu_k"], *sizes, lq, lk, lk, lq,
                                      sc, False, ws, nb)
                A.adaln_attention_bwd(i["dout"], i["q"], i["k"], i["v"], out["o"], out["lse"], out["dq"], out["dk"], out["dv"],
                                      i["cu_q"], i["cu_k"], *sizes, lq, lq, lk, lk, lq, lq, lk, lk, sc, False, ws, nb)
                got[n].append((out, ws))
    torch.cuda.synchronize()
    for n in range(2):
        for out, ws in got[n]:
            assert A.adaln_read_status(ws) == 0
            assert all(torch.equal(out[m], want[n][m]) for m in out), n


@pytest.mark.gpu
def test_thousands_of_segments():
    # More segments than the work list keeps on chip. Rows of at most one tile of keys do not depend on what they
    # are packed with.
    lens = [(7 * s) % 23 for s in range(2500)]
    i = inputs(lens, lens, 2, 1, 64, seed=32)
    whole = call(i, True, pad=0)
    cut = sum(lens[:900])
    for rows, part in ((slice(0, cut), lens[:900]), (slice(cut, None), lens[900:])):
        cu = torch.tensor([0] + part, device="cuda").cumsum(0).to(torch.int32)
        j = dict({n: i[n][rows] for n in ("q", "k", "v", "dout")}, cu_q=cu, cu_k=cu, lens_q=part, lens_k=part)
        got = call(j, True, pad=0)
        assert all(torch.equal(got[n], whole[n][rows]) for n in ("o", "dq", "dk", "dv"))
        assert torch.equal(got["lse"], whole["lse"][:, rows])
    few = dict({n: i[n][:cut] for n in ("q", "k", "v", "dout")}, lens_q=lens[:60], lens_k=lens[:60])
    rows = sum(lens[:60])
    few = {n: (t[:rows] if torch.is_tensor(t) else t) for n, t in few.items()}
    check(few, {n: (t[:, :rows] if n == "lse" else t[:rows]) for n, t in whole.items()}, True)


@pytest.mark.gpu
def test_one_workspace_for_changing_inputs():
    # What a call leaves in the workspace, or a cache holds of it, is nothing to the next.
    lens = [([700, 300], [700, 300]), ([200, 800], [500, 500]), ([999, 1], [1, 999])]
    sets = [inputs(q, k, 4, 2, 64, seed=20 + n) for n, (q, k) in enumerate(lens)]
    want = [call(i, pad=0) for i in sets]
    sizes = (2, 1000, 1000, 4, 2, 64)
    nb = max(A.adaln_attention_fwd_workspace_size(*sizes, 1), A.adaln_attention_bwd_workspace_size(*sizes, 1))
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    outs = [{n: torch.empty_like(t) for n, t in want[x % 3].items()} for x in range(15)]
    torch.cuda.synchronize()
    for x, out in enumerate(outs):
        i = sets[x % 3]
        A.adaln_attention_fwd(i["q"], i["k"], i["v"], out["o"], out["lse"], i["cu_q"], i["cu_k"], *sizes, 256, 128, 128, 256,
                              0.125, False, ws, nb)
        A.adaln_attention_bwd(i["dout"], i["q"], i["k"], i["v"], out["o"], out["lse"], out["dq"], out["dk"], out["dv"],
                              i["cu_q"], i["cu_k"], *sizes, 256, 256, 128, 128, 256, 256, 128, 128, 0.125, False, ws, nb)
    for x, out in enumerate(outs):
        assert all(torch.equal(out[n], want[x % 3][n]) for n in out), x


@pytest.mark.gpu
def test_workspaces_hold_fewer_rows_too():
    for Hq, nseg in ((1, 1), (3, 1), (12, 4), (40, 2)):
        for size in (A.adaln_attention_fwd_workspace_size, A.adaln_attention_bwd_workspace_size):
            last = 0
            for R in (0, 1, 5, 100, 127, 128, 129, 500, 1000, 5000, 19000, 20000, 100000):
                now = size(nseg, R, R, Hq, Hq, 64, 1)
                assert now >= last, (Hq, nseg, R)
                last = now


@pytest.mark.gpu
def test_with_head_norms_and_rotation():
    """The operators as a block uses them: a joint projection's rows through the head norms, the rotation
    and attention, and back."""
    from adaln_layernorm_modulate_gb300.autograd import attention, qk_norm_rope
    lens, Hq, Hk, d = [70, 1, 200], 4, 2, 64
    g = torch.Generator("cuda").manual_seed(14)
    R = sum(lens)
    rows = torch.randn(R, (Hq + 2 * Hk) * d, generator=g, device="cuda").bfloat16().requires_grad_(True)
    w = [(1 + 0.2 * torch.randn(d, generator=g, device="cuda")).bfloat16().requires_grad_(True) for _ in range(2)]
    pos = torch.cat([torch.stack([torch.arange(n, device="cuda") // 10, torch.arange(n, device="cuda") % 10], 1) for n in lens])
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    dout = torch.randn(R, Hq, d, generator=g, device="cuda").bfloat16()
    q, k, v = (t.unflatten(1, (-1, d)) for t in rows.split([Hq * d, Hk * d, Hk * d], 1))
    q, k = qk_norm_rope(q, k, pos, (32, 32), *w)
    attention(q, k, v, cu).backward(dout)

    rd, wd = rows.detach().double().requires_grad_(True), [t.detach().double().requires_grad_(True) for t in w]
    q, k, v = (t.unflatten(1, (-1, d)) for t in rd.split([Hq * d, Hk * d, Hk * d], 1))
    freq = 10000.0 ** (-torch.arange(0, 32, 2, device="cuda", dtype=torch.float64) / 32)
    t = torch.cat([pos[:, :1] * freq, pos[:, 1:] * freq], 1)[:, None]
    out = []
    for x, wx in ((q, wd[0]), (k, wd[1])):
        y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * wx
        a, b = y[..., 0::2], y[..., 1::2]
        out.append(torch.stack([a * t.cos() - b * t.sin(), a * t.sin() + b * t.cos()], -1).flatten(-2))
    q, k = out
    o = []
    for a, b in ((0, 70), (70, 71), (71, 271)):
        K, V = (x[a:b].repeat_interleave(2, 1).transpose(0, 1) for x in (k, v))
        o.append((torch.softmax(0.125 * q[a:b].transpose(0, 1) @ K.transpose(1, 2), 2) @ V).transpose(0, 1))
    torch.cat(o).backward(dout.double())
    # A handful of bf16 roundings in the chain (q', k', p, dz, their gradients), independent between elements.
    for got, want in ((rows.grad, rd.grad), (w[0].grad, wd[0].grad), (w[1].grad, wd[1].grad)):
        assert (got.double() - want).norm() <= 6 * H * want.norm()


@pytest.mark.gpu
@pytest.mark.parametrize("B,N,M", [(0, 5, 7), (3, 0, 7), (3, 5, 0), (0, 0, 0)])
def test_node_without_rows(B, N, M):
    from adaln_layernorm_modulate_gb300.autograd import attention
    q, k, v = (torch.randn(B, n, h, 64, device="cuda", dtype=torch.bfloat16).requires_grad_(True)
               for n, h in ((N, 4), (M, 2), (M, 2)))
    for causal in (False, True):
        o, lse = attention(q, k, v, causal=causal, return_lse=True, check_tables=True)
        assert o.shape == q.shape and lse.shape == (4, B, N) and (o == 0).all() and (lse == -math.inf).all()
        o.sum().backward()
        assert all(t.grad.shape == t.shape and (t.grad == 0).all() for t in (q, k, v))
