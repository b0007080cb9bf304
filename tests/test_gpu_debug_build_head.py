"""The affine layer norm and the vocabulary loss under the index-checked debug build: no check
fails and every output is bitwise the release library's."""
import pytest

from tests.test_gpu_debug_build import debug_lib, library  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


def _norm(A, R, D, code, weight=True):
    import torch
    g = torch.Generator("cuda").manual_seed(R + D)
    dt = torch.bfloat16 if code == 1 else torch.float32
    x, dy = (torch.randn(R, D, generator=g, device="cuda").to(dt) for _ in range(2))
    w, b = (torch.randn(D, generator=g, device="cuda").to(dt) for _ in range(2))
    if not weight:
        w = b = None
    y, dx = torch.zeros_like(x), torch.zeros_like(x)
    mean, rstd, dw, db = (torch.zeros(n, device="cuda") for n in (R, R, D, D))
    nb = A.adaln_layernorm_bwd_workspace_size(R, D, code)
    ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    A.adaln_layernorm_fwd(x, w, b, y, mean, rstd, R, D)
    A.adaln_layernorm_bwd(dy, x, mean, rstd, w, dx, dw, db, ws, nb, R, D)
    return y, mean, rstd, dx, dw, db


def _loss(A, N, V, D, ignored):
    import torch
    g = torch.Generator("cuda").manual_seed(N + V)
    x = torch.randn(N, D, generator=g, device="cuda").bfloat16()
    w = (torch.randn(V, D, generator=g, device="cuda") / D ** 0.5).bfloat16()
    t = torch.randint(V, (N,), generator=g, device="cuda")
    t[torch.rand(N, generator=g, device="cuda") < ignored] = -100
    up, ul, loss, lse = (torch.rand(N, generator=g, device="cuda") for _ in range(4))
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    nb = max(A.adaln_linear_xent_fwd_workspace_size(N, V, D, 1), A.adaln_linear_xent_bwd_workspace_size(N, V, D, 1))
    ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    A.adaln_linear_xent_fwd(x, w, t, loss, lse, N, V, D, -100, ws, nb)
    A.adaln_linear_xent_bwd(x, w, t, lse, up, ul, dx, dw, N, V, D, -100, ws, nb)
    assert A.adaln_read_status(ws) == 0
    return loss, lse, dx, dw


CASES = {
    "norm-bf16-257x1536": lambda A: _norm(A, 257, 1536, 1),
    "norm-bf16-5x264": lambda A: _norm(A, 5, 264, 1, weight=False),
    "norm-f32-300x2040": lambda A: _norm(A, 300, 2040, 0),
    "norm-f32-21x16384": lambda A: _norm(A, 21, 16384, 0),
    "norm-bf16-40x16384": lambda A: _norm(A, 40, 16384, 1),
    "loss-1x1x8": lambda A: _loss(A, 1, 1, 8, 0.0),
    "loss-130x257x72": lambda A: _loss(A, 130, 257, 72, 0.3),
    "loss-700x1025x264": lambda A: _loss(A, 700, 1025, 264, 0.5),
    "loss-50x700x128-none": lambda A: _loss(A, 50, 700, 128, 2.0),
    "loss-1000x30000x64": lambda A: _loss(A, 1000, 30000, 64, 0.1),
}


@pytest.mark.parametrize("name", sorted(CASES))
def test_debug_build_checks_pass_and_match_the_release_build(debug_lib, name):  # noqa: F811
    import torch
    with library("release") as A:
        want = CASES[name](A)
    with library("debug") as A:
        got = CASES[name](A)
        word = A.adaln_debug_read(reset=True)
    assert word == 0, {v: n for v, n in A.DEBUG_CLASSES.items() if word & v}
    assert all(torch.equal(a, b) for a, b in zip(want, got))


# A vocabulary in two pieces, the last one narrower; 256-column tiles of dx and dweight.
PIECES = {
    "loss-8192x20001x72": lambda A: _loss(A, 8192, 20001, 72, 0.3),
    "loss-8192x17000x520": lambda A: _loss(A, 8192, 17000, 520, 0.0),
}


@pytest.mark.parametrize("name", sorted(PIECES))
def test_debug_build_checks_pass_over_several_pieces(debug_lib, name):  # noqa: F811
    import torch

    from tests.test_linear_xent import pieces
    N, V = (int(v) for v in name.split("-")[1].split("x")[:2])
    assert pieces(N, V) == 2
    with library("release") as A:
        want = PIECES[name](A)
    with library("debug") as A:
        got = PIECES[name](A)
        word = A.adaln_debug_read(reset=True)
    assert word == 0, {v: n for v, n in A.DEBUG_CLASSES.items() if word & v}
    assert all(torch.equal(a, b) for a, b in zip(want, got))


# Words of many rows: looked for among all targets, in one look and in three, and listed.
WORDS = {
    "loss-3000x20x264": lambda A: _loss(A, 3000, 20, 264, 0.1),
    "loss-20000x300x72": lambda A: _loss(A, 20000, 300, 72, 0.3),
    "loss-20000x9x72": lambda A: _loss(A, 20000, 9, 72, 0.3),
    "loss-900x70x2056": lambda A: _loss(A, 900, 70, 2056, 0.0),
}


@pytest.mark.parametrize("name", sorted(WORDS))
def test_debug_build_checks_pass_with_words_of_many_rows(debug_lib, name):  # noqa: F811
    import torch
    with library("release") as A:
        want = WORDS[name](A)
    with library("debug") as A:
        got = WORDS[name](A)
        word = A.adaln_debug_read(reset=True)
    assert word == 0, {v: n for v, n in A.DEBUG_CLASSES.items() if word & v}
    assert all(torch.equal(a, b) for a, b in zip(want, got))
