"""The example model: the packed AdaLN node, the affine layer norm and the vocabulary loss train
together, and their gradients agree with the same model's in plain torch."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_the_loss_falls():
    from adaln_layernorm_modulate_gb300.masked_lm import train
    losses = train(40)
    assert all(v == v for v in losses)
    assert sum(losses[-5:]) / 5 < 0.75 * losses[0]


def test_gradients_agree_with_plain_torch():
    from adaln_layernorm_modulate_gb300 import masked_lm as M
    from adaln_layernorm_modulate_gb300.autograd import linear_cross_entropy
    torch.manual_seed(1)
    model = M.MaskedLM(301, 128)
    gen = torch.Generator().manual_seed(1)
    seen, target, t, cu, mod = M.batch(gen, [33, 1, 90, 20], 301)
    h = model(seen, t, cu, mod)
    linear_cross_entropy(h, model.head, target).backward()
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
    near = torch.cat([y, torch.roll(y, 1, 0), torch.roll(y, -1, 0)], dim=1)
    mid = torch.nn.functional.silu(near @ p["up.weight"].t() + p["up.bias"])
    out = x + mid @ p["down.weight"].t() + p["down.bias"]
    z = (norm(out) * p["norm.weight"] + p["norm.bias"]) @ p["head"].t()
    keep = target != M.IGNORE
    loss = (torch.logsumexp(z[keep], 1) - z[keep].gather(1, target[keep][:, None]).squeeze(1)).mean()
    loss.backward()
    # bf16 activations: about ten roundings of 2^-8 in the chain, independent between elements.
    for name, v in p.items():
        assert (got[name] - v.grad).norm() <= 10 * 2.0 ** -8 * v.grad.norm() + 1e-6, name
