"""The layer of examples/delta_rule_layer.py, in fp32, against the same layer written as a recurrence in float64 and
differentiated by autograd.

Tolerance: the rule's outputs are sums of at most 32 products whose operands are off by 2^-22 and whose absolute values sum
to about one (keys, queries of length one, beta below one: no step makes an error larger; scale K^-1/2); a group norm
multiplies that by eps^-1/2 = 316 at most: 316 * 32 * 2^-22 = 2.4e-3 of the largest value.  The layer norm and projections
around it (sums of 2^8 terms, 2^-16) add 6 * 2^-16: 2.5e-3.
"""

import pytest

from tests.gpu_util import ss_module

pytestmark = pytest.mark.gpu
TOL = 2.5e-3


@pytest.fixture(scope="module")
def ex():
    ss_module()
    from examples import delta_rule_layer
    return delta_rule_layer


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
    q, k = (K ** -0.5 * t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-5) for t in (q, k))
    q, k = q.repeat_interleave(H // G, 2), k.repeat_interleave(H // G, 2)
    g = -F.softplus(xn @ params["Wg"] + params["bg"])
    beta = torch.sigmoid(xn @ params["Wb"])
    S, outs = x.new_zeros(B, H, K, K), []
    for t in range(L):
        live = (t < lengths)[:, None, None]
        Sd = torch.exp(g[:, t])[..., None, None] * S
        r = v[:, t] - torch.einsum("bhkv,bhk->bhv", Sd, k[:, t])
        S = torch.where(live[..., None], Sd + beta[:, t, :, None, None] * k[:, t, :, :, None] * r[:, :, None, :], S)
        outs.append(torch.where(live, K ** -0.5 * torch.einsum("bhkv,bhk->bhv", S, q[:, t]), 0.0))
    o = torch.stack(outs, 1).flatten(2)
    on = F.silu(F.group_norm(o.reshape(B * L, H * K), H, params["h_scale"], params["h_bias"], 1e-5))
    return x + on.view(B, L, -1) @ params["Wo"]


@pytest.mark.parametrize("L, heads, groups, width", [(37, 4, 2, 16), (130, 3, 3, 24), (65, 2, 1, 32)])
def test_layer_against_autograd(ex, L, heads, groups, width):
    import torch
    B, D = 3, 64
    gen = torch.Generator(device="cuda").manual_seed(L)
    layer = ex.DeltaRuleLayer(D, heads, groups, width, dtype=torch.float32, seed=1)
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
    layer = ex.DeltaRuleLayer(64, 4, 2, 32, dtype=torch.float32, seed=2)
    x = torch.randn(2, 90, 64, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    whole, _, _ = layer.forward(x)
    _near(ex.decode(layer, x, 75), whole.double(), "y")


def test_training_runs_in_bf16(ex):
    import math

    import torch
    layer = ex.DeltaRuleLayer(128, 4, 2, 32)
    x = torch.randn(3, 200, 128, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda").bfloat16()
    lengths = torch.tensor([200, 33, 0], device="cuda", dtype=torch.int32)
    losses = ex.train(layer, x, x.float() + torch.roll(x.float(), 1, dims=1), lengths, steps=3)
    assert len(losses) == 3 and all(math.isfinite(v) for v in losses)
