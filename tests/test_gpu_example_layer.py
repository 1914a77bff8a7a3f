"""The linear attention layer of examples/decay_attention_layer.py, in fp32, against the same layer written as a
recurrence in float64 and differentiated by autograd.

Tolerance: the longest sums here have 2^8 terms, each sum is off by at most 2^8 2^-24 of its summands' absolute values,
six follow one another, and a norm divides by a deviation of at least 1/4 of the summands here: 6 * 4 * 2^-16 = 4e-4 of the
largest value.
"""

import pytest

from tests.gpu_util import ss_module

pytestmark = pytest.mark.gpu
TOL = 4e-4


@pytest.fixture(scope="module")
def ex():
    ss_module()
    from examples import decay_attention_layer
    return decay_attention_layer


def _near(got, ref, what):
    worst = float((got.double() - ref).abs().max() / ref.abs().max())
    assert worst < TOL, f"{what}: {worst:.3g}"


def _plain(layer, params, x, lengths):
    import torch
    from torch.nn import functional as F
    B, L, D = x.shape
    H, G, K = layer.H, layer.G, layer.K
    xn = F.layer_norm(x, (D,), params["n_scale"], params["n_bias"], 1e-5)
    q, k, v = (t.unflatten(-1, (-1, K)) for t in (xn @ params["W"]).split([G * K, G * K, H * K], dim=-1))
    q, k = q.repeat_interleave(H // G, 2), k.repeat_interleave(H // G, 2)
    g = -F.softplus(xn @ params["Wg"] + params["bg"])
    S, outs = x.new_zeros(B, H, K, K), []
    for t in range(L):
        live = (t < lengths)[:, None, None]
        S = torch.where(live[..., None], torch.exp(g[:, t])[..., None, None] * S + k[:, t, :, :, None] * v[:, t, :, None, :], S)
        outs.append(torch.where(live, K ** -0.5 * torch.einsum("bhkv,bhk->bhv", S, q[:, t]), 0.0))
    on = F.layer_norm(torch.stack(outs, 1), (K,), params["h_scale"], params["h_bias"], 1e-5)
    return x + on.flatten(2) @ params["Wo"]


@pytest.mark.parametrize("L, heads, groups, width", [(37, 4, 2, 16), (130, 3, 3, 24)])
def test_layer_against_autograd(ex, L, heads, groups, width):
    import torch
    B, D = 3, 64
    gen = torch.Generator(device="cuda").manual_seed(L)
    layer = ex.DecayAttentionLayer(D, heads, groups, width, dtype=torch.float32, seed=1)
    x = torch.randn(B, L, D, generator=gen, device="cuda")
    dy = torch.randn(B, L, D, generator=gen, device="cuda")
    lengths = torch.tensor([L, L // 2, 1], device="cuda", dtype=torch.int32)
    params = {n: t.double().requires_grad_() for n, t in layer.params.items()}
    xr = x.double().requires_grad_()
    ref = _plain(layer, params, xr, lengths)
    live = (torch.arange(L, device="cuda")[None, :] < lengths[:, None])[..., None]
    dy = torch.where(live, dy, 0.0)
    (ref * dy.double()).sum().backward()
    y, _, saved = layer.forward(x, lengths, train=True)
    grads, dx = layer.backward(dy, saved)
    _near(torch.where(live, y, 0.0), torch.where(live, ref.detach(), 0.0), "y")
    _near(dx, xr.grad, "dx")
    for n in grads:
        _near(grads[n], params[n].grad, n)


def test_decode_continues_a_prompt(ex):
    import torch
    layer = ex.DecayAttentionLayer(64, 4, 2, 32, dtype=torch.float32, seed=2)
    x = torch.randn(2, 90, 64, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    whole, _, _ = layer.forward(x)
    _near(ex.decode(layer, x, 75), whole.double(), "y")


def test_training_lowers_the_loss(ex):
    import torch
    layer = ex.DecayAttentionLayer(128, 4, 2, 32)
    x = torch.randn(3, 200, 128, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda").bfloat16()
    lengths = torch.tensor([200, 33, 0], device="cuda", dtype=torch.int32)
    losses = ex.train(layer, x, x.float() + torch.roll(x.float(), 1, dims=1), lengths, steps=10)
    assert losses[-1] < losses[0]
