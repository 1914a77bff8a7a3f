"""A layer of linear attention with a decay for each head, trained for a few steps and then decoded from.

    xn = layer_norm(x);  q, k, v = columns of xn W;  g = -softplus(xn Wg + bg)
    o  = linear attention of q, k, v with log decays g;  y = x + (layer norm of each head's o) Wo

Both norms, the attention, their gradients and the single-token step are this package's kernels; the projections are
plain matrix products.  Run it as `python examples/decay_attention_layer.py`.
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mamba_selective_ssm_gb300 as ss  # noqa: E402

EPS = 1e-5


class DecayAttentionLayer:
    """``heads`` heads of ``width`` columns; ``groups`` sets of q and k, each shared by heads / groups heads."""

    def __init__(self, dim, heads, groups, width, dtype=torch.bfloat16, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.H, self.G, self.K, self.dtype = heads, groups, width, dtype
        inner, qk = heads * width, groups * width

        def normal(rows, cols):
            return torch.randn(rows, cols, generator=gen, device="cuda") * rows ** -0.5

        self.params = {
            "n_scale": torch.ones(dim, device="cuda"), "n_bias": torch.zeros(dim, device="cuda"),
            "W": normal(dim, 2 * qk + inner), "Wg": 0.1 * normal(dim, heads), "bg": torch.linspace(-4.0, 0.0, heads, device="cuda"),
            "h_scale": torch.ones(width, device="cuda"), "h_bias": torch.zeros(width, device="cuda"),
            "Wo": normal(inner, dim),
        }

    def _project(self, x):
        """x [tokens, dim] -> its norm with the statistics, the projection and the decays' argument."""
        p = self.params
        xn, mean, rstd = ss.layernorm_fwd(x, p["n_scale"], p["n_bias"], EPS)
        return xn, mean, rstd, xn @ p["W"].to(self.dtype), xn.float() @ p["Wg"] + p["bg"]

    def _qkv(self, z):
        """q, k, v as column ranges of the projection [..., 2 G K + H K]."""
        qk = self.G * self.K
        q, k, v = z[..., :qk], z[..., qk:2 * qk], z[..., 2 * qk:]
        return (t.unflatten(-1, (-1, self.K)) for t in (q, k, v))

    def forward(self, x, lengths=None, h0=None, train=False):
        """x [B, L, dim] -> y, the state after each row's last token, and what ``backward`` needs (None unless ``train``)."""
        B, L, D = x.shape
        p = self.params
        xn, mean, rstd, z, a = self._project(x.view(B * L, D))
        q, k, v = self._qkv(z.view(B, L, -1))
        g = -torch.nn.functional.softplus(a).view(B, L, self.H)
        o, ckpt, h = ss.linattn_fwd(q, k, v, g, h0=h0, lengths=lengths, want_ckpt=train)
        on, omean, orstd = ss.layernorm_fwd(o.view(-1, self.K), p["h_scale"], p["h_bias"], EPS)
        y = x + (on.view(B * L, -1) @ p["Wo"].to(self.dtype)).view(B, L, D)
        saved = (x, lengths, xn, mean, rstd, q, k, v, a, g, o, ckpt, on, omean, orstd) if train else None
        return y, h, saved

    def backward(self, dy, saved):
        """Gradients of the parameters (fp32) and of x, for the gradient dy [B, L, dim] of y."""
        x, lengths, xn, mean, rstd, q, k, v, a, g, o, ckpt, on, omean, orstd = saved
        B, L, D = x.shape
        p, dt = self.params, self.dtype
        gr = {}
        dy2 = dy.reshape(B * L, D)
        gr["Wo"] = on.view(B * L, -1).float().t() @ dy2.float()
        don = (dy2 @ p["Wo"].to(dt).t()).view(-1, self.K)
        do, gr["h_scale"], gr["h_bias"] = ss.layernorm_bwd(don, o.view(-1, self.K), p["h_scale"], omean, orstd)
        s = ss.linattn_bwd(q, k, v, g, ckpt, do.to(dt).view(o.shape), lengths=lengths, want_dh0=False)
        dz = torch.cat([s[n].reshape(B * L, -1) for n in ("dq", "dk", "dv")], dim=1)
        da = -s["dg"].view(B * L, -1) * torch.sigmoid(a)
        gr["W"], gr["Wg"], gr["bg"] = xn.float().t() @ dz.float(), xn.float().t() @ da, da.sum(0)
        dxn = (dz @ p["W"].to(dt).t()).float() + da @ p["Wg"].t()
        dx, gr["n_scale"], gr["n_bias"] = ss.layernorm_bwd(dxn.to(dt), x.view(B * L, D), p["n_scale"], mean, rstd)
        return gr, dy + dx.view(B, L, D).to(dt)

    def step(self, x, h):
        """One token for each sequence: x [B, dim] -> y [B, dim], the state h [B, H, K, K] in place."""
        p = self.params
        _, _, _, z, a = self._project(x)
        q, k, v = (t.contiguous() for t in self._qkv(z))
        o = ss.linattn_step(q, k, v, -torch.nn.functional.softplus(a), h)
        on, _, _ = ss.layernorm_fwd(o.view(-1, self.K), p["h_scale"], p["h_bias"], EPS, want_stats=False)
        return x + on.view(x.shape[0], -1) @ p["Wo"].to(self.dtype)


def train(layer, x, target, lengths, steps):
    """Gradient descent on the mean squared error of the tokens within their rows; the losses."""
    B, L, D = x.shape
    rate = D / 16  # the error's curvature in Wo is 2 / D times that of the normed heads, whose largest eigenvalue is a few units
    live = (torch.arange(L, device="cuda")[None, :] < lengths[:, None])[..., None]
    n = live.sum() * D
    losses = []
    for _ in range(steps):
        y, _, saved = layer.forward(x, lengths, train=True)
        e = torch.where(live, y.float() - target, 0.0)
        losses.append(float((e * e).sum() / n))
        grads, _ = layer.backward((2.0 * e / n).to(x.dtype), saved)
        for name, g in grads.items():
            layer.params[name] -= rate * g
    return losses


def decode(layer, x, prompt):
    """The first ``prompt`` tokens in one call, the others one at a time: y [B, L, dim]."""
    y, h, _ = layer.forward(x[:, :prompt].contiguous())
    ys = [y]
    for t in range(prompt, x.shape[1]):
        ys.append(layer.step(x[:, t].contiguous(), h)[:, None])
    return torch.cat(ys, dim=1)


def main():
    torch.manual_seed(0)
    B, L, D = 4, 1000, 512
    layer = DecayAttentionLayer(D, heads=8, groups=2, width=64)
    x = torch.randn(B, L, D, device="cuda", dtype=torch.bfloat16)
    target = x.float() + torch.roll(x.float(), 1, dims=1)  # a token's own value and the one's before
    lengths = torch.tensor([L, 700, 1, 0], device="cuda", dtype=torch.int32)
    losses = train(layer, x, target, lengths, steps=30)
    print("loss " + " ".join(f"{v:.3f}" for v in losses[::5] + losses[-1:]))
    whole, _, _ = layer.forward(x)
    apart = (decode(layer, x, L - 20) - whole).float().abs().max()
    print(f"prefill and decode against one call: {float(apart):.3g} of {float(whole.float().abs().max()):.3g} at most")


if __name__ == "__main__":
    main()
