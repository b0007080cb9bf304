"""The head norms with rotation and attention under the index-checked debug build: no check fails and every
output is bitwise the release library's."""
import pytest

from tests.test_gpu_debug_build import debug_lib, library  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


def _rope(A, R, Hq, Hk, d, axes, code):
    import torch
    g = torch.Generator("cuda").manual_seed(R + d)
    dt = torch.bfloat16 if code == 1 else torch.float32
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dt)
    q, k, dqo, dko = (rand(R, h * d) for h in (Hq, Hk, Hq, Hk))
    w = [rand(d) for _ in range(2)]
    pos = torch.randint(-999, 999, (R, len(axes)), generator=g, device="cuda", dtype=torch.int32)
    out = [torch.zeros_like(x) for x in (q, k, q, k)]
    dw = [torch.zeros(d, device="cuda") for _ in range(2)]
    nb = A.adaln_qk_norm_rope_bwd_workspace_size(R, Hq, Hk, d, code)
    ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    lq, lk = Hq * d, Hk * d
    A.adaln_qk_norm_rope_fwd(q, k, *w, pos, out[0], out[1], R, Hq, Hk, d, lq, lk, lq, lk, axes)
    A.adaln_qk_norm_rope_bwd(dqo, dko, q, k, *w, pos, out[2], out[3], *dw, ws, nb, R, Hq, Hk, d, lq, lk, lq, lk, lq, lk,
                             axes)
    assert A.adaln_read_status(ws) == 0
    return (*out, *dw)


def _attention(A, lens_q, lens_k, Hq, Hk, d, causal):
    import torch

    from tests.test_attention import call, inputs
    i = inputs(lens_q, lens_k, Hq, Hk, d, seed=sum(lens_q) + d)
    got = call(i, causal, pad=0)
    return tuple(got[n] for n in sorted(got))


CASES = {
    "rope-bf16-257x6x72": lambda A: _rope(A, 257, 6, 2, 72, (36, 36), 1),
    "rope-bf16-5x1x8": lambda A: _rope(A, 5, 1, 1, 8, (8,), 1),
    "rope-f32-300x4x128": lambda A: _rope(A, 300, 4, 4, 128, (44, 42, 42), 0),
    "rope-f32-70x3x256": lambda A: _rope(A, 70, 3, 2, 256, (100,), 0),
    "attention-ragged-causal": lambda A: _attention(A, [17, 0, 130, 5, 1], [17, 0, 130, 5, 1], 4, 2, 64, True),
    "attention-cross": lambda A: _attention(A, [300, 1, 77], [5, 200, 128], 2, 1, 128, False),
    "attention-pieces": lambda A: _attention(A, [3, 200], [5000, 2500], 2, 2, 72, False),
    "attention-pieces-causal": lambda A: _attention(A, [2000, 1111], [2000, 1111], 2, 1, 128, True),
    "attention-no-keys": lambda A: _attention(A, [50, 3], [0, 0], 1, 1, 24, False),
    "attention-many": lambda A: _attention(A, [7 * s % 61 for s in range(600)], [5 * s % 71 for s in range(600)], 2, 2, 64, False),
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
