"""The example model with self-attention: the packed AdaLN node, the head norms with rotation, attention,
the affine layer norm and the vocabulary loss in one step. It runs, and its gradients agree with the same
model's in plain torch."""
import pytest
import torch


def test_refuses_heads_it_cannot_have():
    from adaln_layernorm_modulate_gb300 import masked_lm as M
    for dim, heads in ((128, 3), (96, 8), (512, 2)):
        with pytest.raises(ValueError):
            M.MaskedLM(50, dim, device="cpu", heads=heads)


@pytest.mark.gpu
def test_it_runs():
    from adaln_layernorm_modulate_gb300.masked_lm import train
    assert all(v == v for v in train(5, heads=4))


@pytest.mark.gpu
def test_gradients_agree_with_plain_torch():
    from adaln_layernorm_modulate_gb300 import masked_lm as M
    from adaln_layernorm_modulate_gb300.autograd import linear_cross_entropy
    torch.manual_seed(2)
    model = M.MaskedLM(301, 128, heads=2)
    gen = torch.Generator().manual_seed(2)
    lens = [33, 1, 190, 20]
    seen, target, t, cu, mod = M.batch(gen, lens, 301)
    linear_cross_entropy(model(seen, t, cu, mod), model.head, target).backward()
    got = {n: p.grad.double() for n, p in model.named_parameters()}

    # The same model in fp64 on the bf16 values of the parameters.
    p = {n: v.detach().double().requires_grad_(True) for n, v in model.named_parameters()}
    x = p["embed.weight"][seen]
    cond = torch.stack([t, t * t], 1).double()
    shift, scale = (cond @ p["modulation.weight"].t() + p["modulation.bias"]).chunk(2, dim=1)
    row = torch.repeat_interleave(torch.arange(4, device="cuda"), (cu[1:] - cu[:-1]).long())

    def norm(v):
        d = v - v.mean(1, keepdim=True)
        return d / torch.sqrt((d * d).mean(1, keepdim=True) + 1e-6)

    y = norm(x) * (1 + scale[row]) + shift[row]
    place = torch.cat([torch.arange(n, device="cuda", dtype=torch.float64) for n in lens])
    angle = place[:, None] * 10000.0 ** (-torch.arange(0, 64, 2, device="cuda", dtype=torch.float64) / 64)

    def turned(v, w):  # [R, 2, 64]
        v = v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6) * w
        a, b, c, s = v[..., 0::2], v[..., 1::2], angle.cos()[:, None], angle.sin()[:, None]
        return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)

    q, k, v = (u.unflatten(1, (2, 64)) for u in (y @ p["qkv.weight"].t() + p["qkv.bias"]).chunk(3, dim=1))
    q, k = turned(q, p["rope.q_weight"]), turned(k, p["rope.k_weight"])
    z = torch.einsum("ihd,jhd->hij", q, k) / 8
    z = z.masked_fill(row[:, None] != row[None, :], float("-inf"))
    o = torch.einsum("hij,jhd->ihd", torch.softmax(z, 2), v).flatten(1)
    x = x + o @ p["out.weight"].t() + p["out.bias"]
    near = torch.cat([y, torch.roll(y, 1, 0), torch.roll(y, -1, 0)], dim=1)
    mid = torch.nn.functional.silu(near @ p["up.weight"].t() + p["up.bias"])
    out = x + mid @ p["down.weight"].t() + p["down.bias"]
    z = (norm(out) * p["norm.weight"] + p["norm.bias"]) @ p["head"].t()
    keep = target != M.IGNORE
    loss = (torch.logsumexp(z[keep], 1) - z[keep].gather(1, target[keep][:, None]).squeeze(1)).mean()
    loss.backward()
    # bf16 activations: about twenty roundings of 2^-8 in the chain, independent between elements.
    for name, v in p.items():
        assert (got[name] - v.grad).norm() <= 20 * 2.0 ** -8 * v.grad.norm() + 1e-6, name
