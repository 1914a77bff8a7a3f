"""A layer of the gated delta rule, trained for a few steps and then decoded from.

    xn = layer_norm(x);  q, k, v = columns of xn W, each head's q and k of length one
    g = -softplus(xn Wg + bg),  beta = sigmoid(xn Wb)
    o = gated delta rule of q, k, v with log decays g and rates beta
    y = x + silu(group norm of o, a head a group) Wo

The norms, the rule, their gradients and the single-token step are this package's kernels; the projections are plain
matrix products.  Run it as `python examples/delta_rule_layer.py`.
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mamba_selective_ssm_gb300 as ss  # noqa: E402

EPS = 1e-5


class DeltaRuleLayer:
    """``heads`` heads of ``width`` columns; ``groups`` sets of q and k, each shared by heads / groups heads."""

    def __init__(self, dim, heads, groups, width, dtype=torch.bfloat16, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.H, self.G, self.K, self.dtype = heads, groups, width, dtype
        inner, qk = heads * width, groups * width

        def normal(rows, cols):
            return torch.randn(rows, cols, generator=gen, device="cuda") * rows ** -0.5

        self.unit = torch.full((width,), width ** -0.5, device="cuda")  # an RMS norm with it makes a row's length one
        self.params = {
            "n_scale": torch.ones(dim, device="cuda"), "n_bias": torch.zeros(dim, device="cuda"),
            "W": normal(dim, 2 * qk + inner), "Wg": 0.1 * normal(dim, heads), "bg": torch.linspace(-4.0, 0.0, heads, device="cuda"),
            "Wb": normal(dim, heads), "h_scale": torch.ones(inner, device="cuda"), "h_bias": torch.zeros(inner, device="cuda"),
            "Wo": normal(inner, dim),
        }

    def _project(self, x):
        """x [tokens, dim] -> its norm with the statistics, q and k [tokens G, K] before and after theirs, v, and the
        arguments of the decays and rates."""
        p = self.params
        xn, mean, rstd = ss.layernorm_fwd(x, p["n_scale"], p["n_bias"], EPS)
        z = xn @ p["W"].to(self.dtype)
        qk = 2 * self.G * self.K
        raw = z[:, :qk].reshape(-1, self.K)
        unit, rms = ss.rmsnorm_fwd(raw, self.unit, EPS)
        xf = xn.float()
        return xn, mean, rstd, raw, rms, unit.view(-1, 2, self.G, self.K), z[:, qk:], xf @ p["Wg"] + p["bg"], xf @ p["Wb"]

    def forward(self, x, lengths=None, h0=None, train=False):
        """x [B, L, dim] -> y, the state after each row's last token, and what ``backward`` needs (None unless ``train``)."""
        B, L, D = x.shape
        p = self.params
        xn, mean, rstd, raw, rms, unit, v, a, b = self._project(x.view(B * L, D))
        q, k = (unit[:, i].unflatten(0, (B, L)) for i in range(2))
        v = v.unflatten(0, (B, L)).unflatten(-1, (self.H, self.K))
        g, beta = -torch.nn.functional.softplus(a).view(B, L, self.H), torch.sigmoid(b).view(B, L, self.H)
        o, ckpt, h = ss.deltarule_fwd(q, k, v, g, beta, h0=h0, lengths=lengths, want_ckpt=train)
        on, omean, orstd = ss.groupnorm_fwd(o.view(B * L, -1), p["h_scale"], p["h_bias"], self.H, EPS, silu=True)
        y = x + (on @ p["Wo"].to(self.dtype)).view(B, L, D)
        saved = (x, lengths, xn, mean, rstd, raw, rms, q, k, v, a, g, beta, o, ckpt, on, omean, orstd) if train else None
        return y, h, saved

    def backward(self, dy, saved):
        """Gradients of the parameters (fp32) and of x, for the gradient dy [B, L, dim] of y."""
        x, lengths, xn, mean, rstd, raw, rms, q, k, v, a, g, beta, o, ckpt, on, omean, orstd = saved
        B, L, D = x.shape
        p, dt = self.params, self.dtype
        gr = {}
        dy2 = dy.reshape(B * L, D)
        gr["Wo"] = on.float().t() @ dy2.float()
        do, gr["h_scale"], gr["h_bias"] = ss.groupnorm_bwd(dy2 @ p["Wo"].to(dt).t(), o.view(B * L, -1), p["h_scale"], p["h_bias"],
                                                           omean, orstd, self.H, silu=True)
        s = ss.deltarule_bwd(q, k, v, g, beta, ckpt, do.to(dt).view(o.shape), lengths=lengths, want_dh0=False)
        dunit = torch.stack([s["dq"], s["dk"]], dim=2).view(-1, self.K)
        draw, _ = ss.rmsnorm_bwd(dunit, raw, self.unit, rms)
        dz = torch.cat([draw.to(dt).view(B * L, -1), s["dv"].reshape(B * L, -1)], dim=1)
        da = -s["dg"].view(B * L, -1) * torch.sigmoid(a)
        bt = beta.view(B * L, -1)
        db = s["dbeta"].view(B * L, -1) * bt * (1.0 - bt)
        xf = xn.float()
        gr["W"], gr["Wg"], gr["bg"], gr["Wb"] = xf.t() @ dz.float(), xf.t() @ da, da.sum(0), xf.t() @ db
        dxn = (dz @ p["W"].to(dt).t()).float() + da @ p["Wg"].t() + db @ p["Wb"].t()
        dx, gr["n_scale"], gr["n_bias"] = ss.layernorm_bwd(dxn.to(dt), x.view(B * L, D), p["n_scale"], mean, rstd)
        return gr, dy + dx.view(B, L, D).to(dt)

    def step(self, x, h):
        """One token for each sequence: x [B, dim] -> y [B, dim], the state h [B, H, K, K] in place."""
        p = self.params
        _, _, _, _, _, unit, v, a, b = self._project(x)
        o = ss.deltarule_step(unit[:, 0].contiguous(), unit[:, 1].contiguous(), v.unflatten(-1, (self.H, self.K)).contiguous(),
                              -torch.nn.functional.softplus(a), torch.sigmoid(b), h)
        on, _, _ = ss.groupnorm_fwd(o.view(x.shape[0], -1), p["h_scale"], p["h_bias"], self.H, EPS, silu=True, want_stats=False)
        return x + on @ p["Wo"].to(self.dtype)


def train(layer, x, target, lengths, steps, rate=4.0):
    """Gradient descent on the mean squared error of the tokens within their rows; the losses."""
    B, L, D = x.shape
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
    layer = DeltaRuleLayer(D, heads=8, groups=2, width=64)
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
