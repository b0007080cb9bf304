"""The autograd node over libadaln: it runs the same kernels as the C-ABI calls (bitwise
equal results), its gradients match the oracle, and it refuses CPU tensors."""
import numpy as np
import pytest

import synth
from tests import gpu_harness as H


def test_cpu_tensors_are_refused():
    import torch

    from adaln_layernorm_modulate_gb300.autograd import AdaLNModulate
    m = AdaLNModulate(1e-6)
    assert "eps=1e-06, save_stats=True" in repr(m)
    x = torch.zeros(1, 4, 64)
    with pytest.raises(ValueError):
        m(x, torch.zeros(1, 64), torch.zeros(1, 64))


CASES = {
    "dense-bf16-2x300x1536": lambda: synth.dense("a", 201, synth.BF16, 2, 300, 1536,
                                                 x_mode=synth.ROWS_SCALED, dy_std=0.02),
    "packed-f32-d264": lambda: synth.make("a", 202, synth.F32, 264, [5, 90, 0, 33], [1, 1, 0, 2], 3),
}


@pytest.mark.gpu
@pytest.mark.parametrize("save_stats", [True, False], ids=["saved-stats", "recomputed-stats"])
@pytest.mark.parametrize("name", sorted(CASES))
def test_autograd_matches_direct_calls_and_oracle(orc, name, save_stats):
    import torch

    import adaln_layernorm_modulate_gb300 as A
    from adaln_layernorm_modulate_gb300.autograd import adaln_modulate
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    w = CASES[name]()
    d = H.upload(w)
    packed = w.dense is None
    x = d.x if packed else d.x.view(w.dense[0], w.dense[1], w.D)
    x = x.clone().requires_grad_(True)
    shift = d.shift.clone().requires_grad_(True)
    scale = d.scale.clone().requires_grad_(True)
    dy = d.dy if packed else d.dy.view(w.dense[0], w.dense[1], w.D)
    if packed:
        y = adaln_modulate(x, shift, scale, d.cu, d.mod, eps=H.EPS, check_tables=True, save_stats=save_stats)
    else:
        y = adaln_modulate(x, shift, scale, eps=H.EPS, save_stats=save_stats)
    y.backward(dy)

    # Same kernels as the C-ABI path: bitwise equal.
    y2, mean2, rstd2, _ = H.gpu_fwd(d)
    dx2, dsh2, dsc2, _ = H.gpu_bwd(d, mean2, rstd2)
    assert torch.equal(y.detach().reshape(w.R, w.D), y2)
    assert torch.equal(x.grad.reshape(w.R, w.D), dx2)
    assert torch.equal(shift.grad, dsh2.to(shift.dtype))
    assert torch.equal(scale.grad, dsc2.to(scale.dtype))

    # And the oracle, within the operator's tolerances.
    ry, rmean, rrstd = orc.fwd(w.x, w.shift, w.scale, w.dtype, w.cu_seqlens, w.mod_idx, w.nmod, eps=H.EPS)
    H.check_io(H.to_host(y.detach().reshape(w.R, w.D), w.dtype), ry, w.dtype, orc, "y")
    m32, r32 = H.round_f32(rmean), H.round_f32(rrstd)
    rdx, rdsh, rdsc = orc.bwd(w.dy, w.x, m32, r32, w.scale, w.dtype, w.cu_seqlens, w.mod_idx, w.nmod)
    extra = H.stat_shift_bound(_dx_terms(w, m32, r32))
    H.check_io(H.to_host(x.grad.reshape(w.R, w.D), w.dtype), rdx, w.dtype, orc, "dx", extra=extra)
    tol = H.grad_tol(w.dtype) if w.dtype == synth.F32 else 4e-3  # rounded once to bf16
    assert H.rel_l2(H.to_host(shift.grad.float(), 0), rdsh) <= tol
    assert H.rel_l2(H.to_host(scale.grad.float(), 0), rdsc) <= tol


def _dx_terms(w, mean, rstd):
    x = synth.widen(w.x, w.dtype)
    dy = synth.widen(w.dy, w.dtype)
    m_of_row = np.repeat(w.mod_idx, np.diff(w.cu_seqlens))
    g = dy * (1 + synth.widen(w.scale, w.dtype)[m_of_row])
    xhat = (x - mean[:, None]) * rstd[:, None]
    return rstd, mean, xhat, g.mean(axis=1), (g * xhat).mean(axis=1)


class Context:
    """What a node's forward keeps for its backward."""
    needs_input_grad = (True,) * 8

    def save_for_backward(self, *tensors):
        self.saved_tensors = tensors

    def mark_non_differentiable(self, *tensors):
        pass

    def set_materialize_grads(self, value):
        pass


@pytest.mark.parametrize("node", ["dense", "packed", "packed-recomputed", "norm", "loss"])
def test_nodes_launch_on_their_tensors_device(monkeypatch, node):
    # Tensors on device 1 while device 0 is current: every call of the library has to see device 1
    # as the current one. No GPU: the tensors hold nothing, the calls and the current device are fakes.
    import torch
    from torch._subclasses.fake_tensor import FakeTensorMode

    from adaln_layernorm_modulate_gb300 import autograd as G
    current, seen = [0], []

    class Device:
        def __init__(self, device):
            self.index = device.index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *error):
            current[0] = self.before

    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", Device)
    for name in dir(G):
        if name.startswith("adaln_") and name != "adaln_modulate":
            def call(*args, name=name):
                seen.append((name, current[0]))
                return 256 if name.endswith("_size") else 0
            monkeypatch.setattr(G, name, call)
    with FakeTensorMode():
        make = lambda *shape, dtype=torch.bfloat16: torch.empty(*shape, dtype=dtype, device="cuda:1")
        ctx, row, table = Context(), make(12, 64), make(3, 64)
        if node == "dense":
            x = make(3, 4, 64)
            G.AdaLNModulateFunction.forward(ctx, x, table, table)
            G.AdaLNModulateFunction.backward(ctx, x, None, None)
        elif node.startswith("packed"):
            cu, mod = make(4, dtype=torch.int32), make(3, dtype=torch.int32)
            G.AdaLNModulateFunction.forward(ctx, row, table, table, cu, mod, 1e-6, True, node == "packed")
            G.AdaLNModulateFunction.backward(ctx, row, None, None)
        elif node == "norm":
            G.LayerNormFunction.forward(ctx, row, make(64), make(64))
            G.LayerNormFunction.backward(ctx, row)
        else:
            target, up = make(12, dtype=torch.int64), make(12, dtype=torch.float32)
            G.LinearCrossEntropyFunction.forward(ctx, row, make(100, 64), target, -100, True)
            G.LinearCrossEntropyFunction.backward(ctx, up, None)
    assert len(seen) >= 3 and all(device == 1 for _, device in seen), seen
    assert current == [0]


def test_modulation_tables_of_another_device_are_refused():
    import torch
    from torch._subclasses.fake_tensor import FakeTensorMode

    from adaln_layernorm_modulate_gb300.autograd import AdaLNModulateFunction
    with FakeTensorMode():
        x, near = (torch.empty(1, 4, 64, device="cuda:0"), torch.empty(1, 64, device="cuda:0"))
        for far in (torch.empty(1, 64), torch.empty(1, 64, device="cuda:1")):
            for tables in ((near, far), (far, near)):
                with pytest.raises(ValueError, match="one device"):
                    AdaLNModulateFunction.forward(Context(), x, *tables)


@pytest.mark.parametrize("shift,scale,cu,mod", [((3, 56), (3, 64), 4, 3), ((3, 64), (2, 64), 4, 3), ((64,), (64,), 4, 3),
                                                ((3, 64), (3, 64), 3, 3), ((3, 64), (3, 64), 4, 4),
                                                ((3, 64), (3, 64), 0, 0)])
def test_packed_tables_of_other_shapes_are_refused(shift, scale, cu, mod):
    # The kernels would read past the shorter of them.
    import torch
    from torch._subclasses.fake_tensor import FakeTensorMode

    from adaln_layernorm_modulate_gb300.autograd import AdaLNModulateFunction
    with FakeTensorMode():
        make = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device="cuda")
        with pytest.raises(ValueError, match="packed input"):
            AdaLNModulateFunction.forward(Context(), make(9, 64), make(*shift), make(*scale),
                                          make(cu, dtype=torch.int32), make(mod, dtype=torch.int32))
