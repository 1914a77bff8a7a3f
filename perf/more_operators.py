"""The gated delta rule (prefill, training step, single-token step) and group norm with an activation (forward, backward): cases, inputs,
plain forms and 64-bit values.

The rule per batch row, head h (q, k shared by H/G heads), token t < length, with S: [K, V] and scale = K^-1/2:
    r_t = v_t - exp(g_t) S_{t-1}^T k_t        S_t = exp(g_t) S_{t-1} + beta_t k_t r_t^T        o_t = scale * S_t^T q_t
and, for a loss whose gradients at o and at the last state are `do` and `dh_last`, the gradients of q, k, v, g, beta and of the first state.

The norm over x [N, M, C] per sample n and group of C / groups channels, statistics over the M positions and the group's channels:
    y = act((x - mean) * rstd * scale + bias)        act: SiLU or nothing
"""

import math

import torch

own = False

EPS = 1e-5
CHUNK = 64  # tokens per chunk of the plain form
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases


def _rule(name, op, B, L, H, G, K, V, dtype, decay=True, carry=False, ragged=False, packed=False, strong=False):
    return {"name": name, "op": op, "B": B, "L": L, "H": H, "G": G, "K": K, "V": V, "dtype": dtype, "decay": decay,
            "carry": carry, "ragged": ragged, "packed": packed, "strong": strong}


def _norm(name, op, N, M, C, groups, dtype, silu=True):
    return {"name": name, "op": op, "N": N, "M": M, "C": C, "groups": groups, "dtype": dtype, "silu": silu}


def listed():
    return [
        # a batch of short prompts of unequal length (an empty one and one of a single token among them) before decoding, odd head sizes
        _rule("delta_prefill_ragged", "prefill", 5, 77, 6, 3, 40, 72, "bf16", carry=True, ragged=True),
        # one long prompt on the long-context layer's width (d_inner 2048, 16384 tokens), q and k shared by four heads each
        _rule("delta_prefill_long", "prefill", 1, 16384, 32, 8, 128, 64, "bf16"),
        # a batch of prompts on the 1.4B layer's width (d_inner 4096), q, k and v cut out of one projection
        _rule("delta_prefill_layer", "prefill", 4, 2048, 32, 32, 128, 128, "bf16", packed=True),
        # one training step of that layer: forward with checkpoints, then all gradients
        _rule("delta_train_layer", "train", 4, 2048, 32, 32, 128, 128, "bf16", packed=True),
        # a long sequence trained in pieces: a state comes in and a gradient of the state arrives at the end; beta up to 2
        _rule("delta_train_long", "train", 1, 8192, 32, 4, 128, 64, "bf16", carry=True, strong=True),
        # the 130M layer in fp32 (d_inner 1536, 24 heads of 64), the rule without a decay
        _rule("delta_train_130m_f32", "train", 8, 2048, 24, 24, 64, 64, "f32", decay=False),
        # one sequence being decoded: latency
        _rule("delta_step_one", "step", 1, 1, 32, 32, 128, 128, "bf16", carry=True),
        # a server's batch of sequences being decoded
        _rule("delta_step_batch", "step", 96, 1, 32, 8, 128, 128, "bf16", carry=True),
        # the norm over each head's output of the 1.4B layer, token by token, with its activation
        _norm("norm_fwd_tokens", "norm_fwd", 8192, 1, 4096, 32, "bf16"),
        # the same width normalised over whole sequences, as around a convolution
        _norm("norm_fwd_sequences", "norm_fwd", 4, 2048, 4096, 32, "bf16"),
        # their backward passes; the sequences' on the 130M layer's width in fp32
        _norm("norm_bwd_tokens", "norm_bwd", 8192, 1, 4096, 32, "bf16"),
        _norm("norm_bwd_sequences_f32", "norm_bwd", 8, 2048, 1536, 24, "f32"),
    ]


def _log(rng, lo, hi):
    n = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))
    return n - (n > lo and n % 1024 == 0)  # the round sizes are listed


def draw(rng):
    op = rng.choice(["prefill", "prefill", "train", "train", "step", "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("norm"):
        groups = rng.choice([1, 2, 4, 8, 24, 32, 32, _log(rng, 1, 128)])
        per = rng.choice([4, 8, 16, 32, 64, 128, 128, _log(rng, 1, 256)])
        C = groups * per
        while C % 8:  # channels come in eights
            C *= 2
            groups *= 2
        N = _log(rng, 1, 8192)
        M = 1 if rng.random() < 0.4 else _log(rng, 1, 16384)
        most = (1 << 25) // C // (1 if dtype == "bf16" else 2)
        N = max(1, min(N, most))
        return {"op": op, "N": N, "M": max(1, min(M, most // N)), "C": C, "groups": groups, "dtype": dtype, "silu": rng.random() < 0.7}
    K, V = (rng.choice([rng.choice([64, 128]), 8 * rng.randint(1, 16)]) for _ in range(2))
    G = _log(rng, 1, 32)
    H = G * rng.choice([r for r in (1, 1, 2, 3, 4, 8, 16, 32) if G * r <= 64])
    decay, carry, ragged, packed, strong = rng.random() < 0.75, rng.random() < 0.5, rng.random() < 0.4, rng.random() < 0.5, rng.random() < 0.3
    step = op == "step"
    if step:
        B, L = min(_log(rng, 1, 256), max(1, 96 * 32 * 128 * 128 // (H * K * V))), 1
    else:  # tokens: no more than the largest listed cases have, of tokens or of work
        most = min(4 * 2048 * 32 // H, (4 * 2048 * 32 * 128 * 128 if dtype == "bf16" else 8 * 2048 * 24 * 64 * 64) // (H * K * V))
        most -= most // 16
        L = min(_log(rng, 1, 16384), most)
        B = min(_log(rng, 1, 64), max(1, most // L))
    return {"op": op, "B": B, "L": L, "H": H, "G": G, "K": K, "V": V, "dtype": dtype, "decay": decay, "carry": carry or step,
            "ragged": ragged and not step, "packed": packed and not step, "strong": strong}


# ---------------------------------------------------------------- inputs


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DT[case["dtype"]]

    def normal(*shape, dtype=dt):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)

    s = {"op": case["op"]}
    if case["op"].startswith("norm"):
        N, M, C, n = case["N"], case["M"], case["C"], case["groups"]
        f = torch.float32
        x = (normal(N, M, C, dtype=f) * 1.5 + 0.3 * normal(N, 1, C, dtype=f)).to(dt)  # a channel has a mean of its own
        s |= {"x": x, "scale": 1 + 0.1 * normal(C, dtype=f), "bias": 0.1 * normal(C, dtype=f), "groups": n, "silu": case["silu"]}
        if case["op"] == "norm_bwd":  # what the forward saved
            xd = x.double().view(N, M, n, C // n)
            s |= {"dy": normal(N, M, C), "mean": xd.mean((1, 3)).float(), "rstd": (xd.var((1, 3), unbiased=False) + EPS).rsqrt().float()}
        return s
    B, L, H, G, K, V = (case[k] for k in "BLHGKV")
    s["g"] = None
    if case["decay"]:  # -a_h * dt with the step sizes of the scan's layers: softplus(0.5 eps + bias), bias of [1e-3, 1e-1]
        u = torch.empty(H, device="cuda").uniform_(math.log(1e-3), math.log(1e-1), generator=gen).exp()
        a = torch.empty(H, device="cuda").uniform_(1.0, 16.0, generator=gen)
        dts = torch.nn.functional.softplus(0.5 * normal(B, L, H, dtype=torch.float32) + torch.log(torch.expm1(u)))
        s["g"] = -(a * dts)
    s["beta"] = torch.sigmoid(normal(B, L, H, dtype=torch.float32)) * (2.0 if case["strong"] else 1.0)
    s["K"], s["V"], s["G"], s["H"] = K, V, G, H
    q, k, v = (torch.randn(B, L, n, w, generator=gen, device="cuda") for n, w in ((G, K), (G, K), (H, V)))
    k = k + 0.5 * torch.randn(B, 1, G, K, generator=gen, device="cuda")  # keys of a sequence resemble one another
    q, k = (t / t.norm(dim=-1, keepdim=True) for t in (q, k))  # the rule's layers feed it rows of length one
    if case["packed"]:
        s["qkv"] = torch.cat([t.flatten(2) for t in (q, k, v)], -1).to(dt)
    else:
        s["q"], s["k"], s["v"] = q.to(dt), k.to(dt), v.to(dt)
    s["h"] = normal(B, H, K, V, dtype=torch.float32) if case["carry"] or case["op"] == "step" else None
    if case["op"] == "step":
        for n in "qkv":
            s[n] = s[n][:, 0].contiguous()
        s["g"] = s["g"][:, 0].contiguous() if case["decay"] else None
        s["beta"] = s["beta"][:, 0].contiguous()
    s["lengths"] = None
    if case["ragged"]:
        n = torch.randint(0, L + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        n[0] = L
        n[1:2] = 0
        n[2:3] = 1
        s["lengths"] = n
    if case["op"] == "train":
        s["do"] = normal(B, L, H, V)
        s["dh_last"] = 0.1 * normal(B, H, K, V, dtype=torch.float32) if case["carry"] else None
    return s


def _qkv(s):
    """q, k, v as the program has them: three tensors, or views of one projection's output."""
    if "qkv" not in s:
        return s["q"], s["k"], s["v"]
    gk = s["G"] * s["K"]
    q, k, v = s["qkv"].split([gk, gk, s["H"] * s["V"]], dim=-1)
    return q.unflatten(-1, (s["G"], s["K"])), k.unflatten(-1, (s["G"], s["K"])), v.unflatten(-1, (s["H"], s["V"]))


# ---------------------------------------------------------------- one pass


def run(s):
    if own:
        import mamba_selective_ssm_gb300 as ss

        if s["op"] == "norm_fwd":
            y, mean, rstd = ss.groupnorm_fwd(s["x"], s["scale"], s["bias"], s["groups"], EPS, silu=s["silu"])
            return {"y": y, "mean": mean, "rstd": rstd}
        if s["op"] == "norm_bwd":
            dx, dscale, dbias = ss.groupnorm_bwd(s["dy"], s["x"], s["scale"], s["bias"], s["mean"], s["rstd"], s["groups"], silu=s["silu"])
            return {"dx": dx, "dscale": dscale, "dbias": dbias}
        if s["op"] == "step":  # the state advances in place, pass after pass
            return {"o": ss.deltarule_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["h"]), "h": s["h"]}
        q, k, v = _qkv(s)
        train = s["op"] == "train"
        o, ckpt, h_last = ss.deltarule_fwd(q, k, v, s["g"], s["beta"], h0=s["h"], lengths=s["lengths"], want_ckpt=train)
        if not train:
            return {"o": o, "h_last": h_last}
        d = ss.deltarule_bwd(q, k, v, s["g"], s["beta"], ckpt, s["do"], dh_last=s["dh_last"], lengths=s["lengths"])
        return {"o": o, "h_last": h_last, "dq": d["dq"], "dk": d["dk"], "dv": d["dv"], "dg": d["dg"], "dbeta": d["dbeta"], "dh0": d["dh0"]}
    if s["op"] == "norm_fwd":
        return _norm_fwd(s["x"], s["scale"], s["bias"], s["groups"], s["silu"])
    if s["op"] == "norm_bwd":
        return _norm_bwd(s["dy"], s["x"], s["scale"], s["bias"], s["mean"], s["rstd"], s["silu"])
    if s["op"] == "step":
        return _step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["h"])
    return _chunked(*_qkv(s), s["g"], s["beta"], s["h"], s["lengths"], s.get("do"), s.get("dh_last"))


def _norm_fwd(x, scale, bias, groups, silu):
    N, M, C = x.shape
    f = x.float().view(N, M, groups, C // groups)
    mean = f.mean((1, 3))
    d = f - mean[:, None, :, None]
    rstd = ((d * d).mean((1, 3)) + EPS).rsqrt()
    y = (d * rstd[:, None, :, None]).view(N, M, C) * scale + bias
    return {"y": (y / (1 + (-y).exp()) if silu else y).to(x.dtype), "mean": mean, "rstd": rstd}


def _norm_bwd(dy, x, scale, bias, mean, rstd, silu):
    N, M, C = x.shape
    n = mean.shape[1]
    xh = ((x.float().view(N, M, n, C // n) - mean[:, None, :, None]) * rstd[:, None, :, None]).view(N, M, C)
    g = dy.float()
    if silu:
        y = xh * scale + bias
        p = 1 / (1 + (-y).exp())
        g = g * p * (1 + y * (1 - p))
    w, xg = (g * scale).view(N, M, n, C // n), xh.view(N, M, n, C // n)
    dx = rstd[:, None, :, None] * (w - w.mean((1, 3), keepdim=True) - xg * (w * xg).mean((1, 3), keepdim=True))
    return {"dx": dx.reshape(N, M, C), "dscale": (g * xh).sum((0, 1)), "dbias": g.sum((0, 1))}


def _step(q, k, v, g, beta, h):
    B, H, V = v.shape
    G, K = q.shape[1:]
    q, k = (t.float()[:, :, None].expand(B, G, H // G, K).reshape(B, H, K) for t in (q, k))
    if g is not None:
        h.mul_(g.exp()[:, :, None, None])
    r = v.float() - (k[..., None] * h).sum(2)
    h.add_((beta[..., None] * k)[..., None] * r[:, :, None])
    return {"o": ((q[..., None] * h).sum(2) * K**-0.5).to(v.dtype), "h": h}


def _inverse(A):
    """(I + A)^-1 of strictly lower triangular A [..., C, C], C a power of two: blocks of twice the size from pairs of inverted ones."""
    C = A.shape[-1]
    X = torch.eye(C, device=A.device, dtype=A.dtype).expand_as(A).clone()
    s = 1
    while s < C:
        n = C // (2 * s)
        Xb, Ab = X.unflatten(-1, (n, 2, s)).unflatten(-4, (n, 2, s)), A.unflatten(-1, (n, 2, s)).unflatten(-4, (n, 2, s))
        d = torch.arange(n, device=A.device)
        lo, hi, a = Xb[..., d, 0, :, d, 0, :], Xb[..., d, 1, :, d, 1, :], Ab[..., d, 1, :, d, 0, :]
        Xb[..., d, 1, :, d, 0, :] = -(hi @ a @ lo)
        s *= 2
    return X


def _chunked(q, k, v, g, beta, h0, lengths, do, dh_last):
    """The chunked form in 32 bits: inside a chunk products and one triangular inverse, from chunk to chunk the state."""
    B, L, G, K = q.shape
    H, V = v.shape[2:]
    C, dt, scale = CHUNK, v.dtype, K**-0.5
    n = -(-L // C)
    live = torch.arange(n * C, device=q.device) < (lengths[:, None] if lengths is not None else L)  # [B, n*C]
    live = live.expand(B, n * C)

    def lay(t):  # [B, L, heads, W] -> [B, H, n, C, W] in 32 bits, nothing past a row's end
        t = torch.nn.functional.pad(t.float(), (0, 0, 0, 0, 0, n * C - L))
        t = torch.where(live[:, :, None, None], t, 0.0)
        t = t[:, :, :, None].expand(B, n * C, t.shape[2], H // t.shape[2], t.shape[3]).flatten(2, 3)
        return t.unflatten(1, (n, C)).permute(0, 3, 1, 2, 4).contiguous()

    def back(t):  # [B, H, n, C, W] -> [B, L, H, W]
        return t.permute(0, 2, 3, 1, 4).reshape(B, n * C, H, t.shape[-1])[:, :L]

    q, k, v, beta = lay(q), lay(k), lay(v), lay(beta[..., None])
    c = (torch.zeros_like(beta[..., 0]) if g is None else lay(g[..., None])[..., 0]).double().cumsum(-1)
    lower = torch.ones(C, C, device=q.device, dtype=torch.bool).tril()
    D = (c[..., :, None] - c[..., None, :]).masked_fill(~lower, -math.inf).exp().float()
    into, rest, whole = c.exp().float()[..., None], (c[..., -1:] - c).exp().float()[..., None], c[..., -1].exp().float()[..., None, None]
    Ds = D.tril(-1)
    kk, qk = k @ k.mT, q @ k.mT
    P, A = qk * D * scale, kk * Ds
    inv = _inverse(A * beta.mT)  # r = inv (v - into * k S)
    S = torch.zeros(B, H, K, V, device=q.device) if h0 is None else h0.clone()
    Ss, rs, os = [], [], []
    for m in range(n):
        r = inv[:, :, m] @ (v[:, :, m] - into[:, :, m] * (k[:, :, m] @ S))
        u = beta[:, :, m] * r
        os.append(P[:, :, m] @ u + scale * into[:, :, m] * (q[:, :, m] @ S))
        if do is not None:
            Ss.append(S)
            rs.append(r)
        S = whole[:, :, m] * S + (rest[:, :, m] * k[:, :, m]).mT @ u
    out = {"o": back(torch.stack(os, 2)).to(dt), "h_last": S}
    if do is None:
        return out
    do = lay(do)
    S, r = torch.stack(Ss, 2), torch.stack(rs, 2)
    u = beta * r
    inv = _inverse(beta * A).mT  # the gradient of u through the chunk's later r: inv du
    U = torch.zeros(B, H, K, V, device=q.device) if dh_last is None else dh_last.clone()
    Us, dus = [], []
    for m in reversed(range(n)):
        Us.append(U)
        du = inv[:, :, m] @ (P[:, :, m].mT @ do[:, :, m] + rest[:, :, m] * (k[:, :, m] @ U))
        dus.append(du)
        U = whole[:, :, m] * U + (scale * into[:, :, m] * q[:, :, m]).mT @ do[:, :, m] - (into[:, :, m] * k[:, :, m]).mT @ (beta[:, :, m] * du)
    dh0 = U
    U, du = torch.stack(Us[::-1], 2), torch.stack(dus[::-1], 2)  # the gradient of the state leaving a chunk, and of its u
    dv = beta * du
    dP, dA = (do @ u.mT) * D * scale, -(dv @ u.mT) * Ds
    qi, ri, wi = scale * into * (do @ S.mT), -into * (dv @ S.mT), rest * (u @ U.mT)
    dq, dk = dP @ k + qi, dA @ k + ri + dP.mT @ q + dA.mT @ k + wi
    # a decay counts in every product of a token at or after it with one before it
    E = (dP * qk + dA * kk).double().tril(-1)
    a, b = ((q * qi).sum(-1) + (k * ri).sum(-1)).double(), (k * wi).sum(-1).double()
    after = a + E.sum(-1) - E.sum(-2)
    dg = after.flip(-1).cumsum(-1).flip(-1) + b.cumsum(-1) - b + (whole[..., 0] * (S * U).sum((-1, -2))[..., None]).double()
    dg = back(torch.where(live.view(B, 1, n, C), dg, 0.0)[..., None])[..., 0]
    share = lambda t: back(t).unflatten(2, (G, H // G)).sum(3).to(dt)  # noqa: E731
    return out | {"dq": share(dq), "dk": share(dk), "dv": back(dv).to(dt), "dg": None if g is None else dg.float(),
                  "dbeta": back((r * du).sum(-1, keepdim=True))[..., 0].contiguous(), "dh0": dh0}


# ---------------------------------------------------------------- work


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("norm"):
        n, C, R = case["N"] * case["M"] * case["C"], case["C"], case["N"] * case["groups"]
        if case["op"] == "norm_fwd":
            return {"bytes": 2 * n * e + 8 * C + 8 * R, "flops": 12 * n}
        return {"bytes": 2 * n * e + 4 * n + 16 * C + 8 * R, "flops": 24 * n}
    B, L, H, G, K, V = (case[k] for k in "BLHGKV")
    qk, vo, st = B * L * G * K * e, B * L * H * V * e, 4 * B * H * K * V
    g = 4 * B * L * H * (2 if case["decay"] else 1)  # beta, and the log decay
    if case["op"] == "step":
        return {"bytes": 2 * qk + 2 * vo + g + 2 * st, "flops": 7 * B * H * K * V}
    carry = st if case["carry"] else 0
    fwd = {"bytes": 2 * qk + 2 * vo + g + st + carry, "flops": 6 * B * L * H * K * V}
    if case["op"] == "prefill":
        return fwd
    # the backward reads q, k, v, do, g, beta (and the arriving gradient) and writes those of q, k, v, g, beta and of the first state
    return {"bytes": fwd["bytes"] + 4 * qk + 3 * vo + 2 * g + st + carry, "flops": fwd["flops"] + 14 * B * L * H * K * V}


# ---------------------------------------------------------------- 64 bits, from the recurrence


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        N, M, C, n = case["N"], case["M"], case["C"], case["groups"]
        x = s["x"].double().transpose(1, 2).reshape(N, n, C // n * M)  # a row for each sample and group
        chan = lambda t: t.double().view(n, C // n, 1).expand(n, C // n, M).reshape(1, n, -1)  # noqa: E731
        rows = lambda t: t.view(N, C, M).transpose(1, 2)  # noqa: E731
        w, b = chan(s["scale"]), chan(s["bias"])
        if case["op"] == "norm_fwd":
            var, mean = torch.var_mean(x, dim=2, correction=0)
            r = 1.0 / torch.sqrt(var + EPS)
            y = torch.addcmul(b, (x - mean.unsqueeze(2)) * r.unsqueeze(2), w)
            return {"y": rows(y * torch.sigmoid(y) if case["silu"] else y), "mean": mean, "rstd": r}
        m, r = s["mean"].double().unsqueeze(2), s["rstd"].double().unsqueeze(2)
        d = s["dy"].double().transpose(1, 2).reshape(N, n, -1)
        if case["silu"]:
            y = (x - m) * r * w + b
            e = torch.sigmoid(y)
            d = d * (e + y * e * torch.sigmoid(-y))
        p, t = (d * w).sum(2, keepdim=True), (d * w * (x - m)).sum(2, keepdim=True)
        size = M * (C // n)
        dx = r * d * w - r * p / size - r**3 * (x - m) * t / size
        return {"dx": rows(dx), "dscale": torch.einsum("nmc,nmc->c", rows(d), rows((x - m) * r)), "dbias": torch.einsum("nmc->c", rows(d))}
    B, L, H, G, K, V = (case[k] for k in "BLHGKV")
    R, BH = H // G, B * H
    if case["op"] == "step":
        for t in ("q", "k", "v", "g", "beta"):
            s[t] = s[t].unsqueeze(1) if s[t] is not None else None
    q, k, v = (t.double() for t in _qkv(s))
    q, k = q.repeat_interleave(R, 2) / math.sqrt(K), k.repeat_interleave(R, 2)
    n = s["lengths"].tolist() if s["lengths"] is not None else [L] * B
    g = s["g"].double() if s["g"] is not None else torch.zeros(B, L, H, device="cuda", dtype=torch.float64)
    live = torch.zeros(B, L, 1, 1, device="cuda", dtype=torch.float64)
    for b, m in enumerate(n):
        live[b, :m] = 1
    # a token past its row's end neither decays nor writes nor reads
    q, k, v, g, beta = q * live, k * live, v * live, g * live[..., 0], s["beta"].double() * live[..., 0]
    q, k, v, e, beta = (t.transpose(0, 1).reshape(L, BH, -1).contiguous() for t in (q, k, v, g.exp().unsqueeze(-1), beta.unsqueeze(-1)))
    S = s["h"].double().reshape(BH, K, V).clone() if s["h"] is not None else torch.zeros(BH, K, V, device="cuda", dtype=torch.float64)

    def rows(t):  # [L, B*H, W] -> [B, L, H, W]
        return t.view(L, B, H, -1).transpose(0, 1)

    def step(S, t):  # in place; what the token finds in the decayed state
        S.mul_(e[t].unsqueeze(-1))
        r = v[t] - torch.bmm(k[t].unsqueeze(1), S).squeeze(1)
        return r

    def write(S, t, r):
        S.baddbmm_((beta[t] * k[t]).unsqueeze(2), r.unsqueeze(1))

    o = torch.empty(L, BH, V, device="cuda", dtype=torch.float64)
    every = max(1, math.isqrt(L))
    marks = []
    for t in range(L):
        if case["op"] == "train" and t % every == 0:
            marks.append(S.clone())
        write(S, t, step(S, t))
        torch.bmm(q[t].unsqueeze(1), S, out=o[t].unsqueeze(1))
    if case["op"] == "step":
        return {"o": rows(o)[:, 0], "h": S.view(B, H, K, V)}
    out = {"o": rows(o), "h_last": S.view(B, H, K, V).clone()}
    if case["op"] == "prefill":
        return out
    do = (s["do"].double() * live).transpose(0, 1).reshape(L, BH, V).contiguous()
    U = s["dh_last"].double().reshape(BH, K, V).clone() if s["dh_last"] is not None else torch.zeros(BH, K, V, device="cuda", dtype=torch.float64)
    dq, dk, dv, dg, db = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty_like(e), torch.empty_like(beta)
    for m in range(len(marks) - 1, -1, -1):
        S, found = marks[m], []  # the decayed states of this stretch of tokens, before their writes
        for t in range(m * every, min(L, (m + 1) * every)):
            r = step(S, t)
            found.append((S.clone(), r))
            write(S, t, r)
            torch.bmm(S, do[t].unsqueeze(2), out=dq[t].unsqueeze(2))
        for t in range(min(L, (m + 1) * every) - 1, m * every - 1, -1):
            Sd, r = found[t - m * every]
            U.baddbmm_(q[t].unsqueeze(2), do[t].unsqueeze(1))
            Uk = torch.bmm(k[t].unsqueeze(1), U).squeeze(1)
            db[t] = (Uk * r).sum(1, keepdim=True)
            dr = beta[t] * Uk
            dv[t] = dr
            dk[t] = (beta[t].unsqueeze(-1) * torch.bmm(U, r.unsqueeze(2)) - torch.bmm(Sd, dr.unsqueeze(2))).squeeze(2)
            U.baddbmm_(k[t].unsqueeze(2), dr.unsqueeze(1), alpha=-1)
            dg[t] = torch.bmm(U.view(BH, 1, K * V), Sd.view(BH, K * V, 1)).squeeze(2)
            U.mul_(e[t].unsqueeze(-1))
    share = lambda t: rows(t).reshape(B, L, G, R, K).sum(3)  # noqa: E731
    alive = live[..., 0]
    return out | {"dq": share(dq) / math.sqrt(K), "dk": share(dk), "dv": rows(dv), "dg": rows(dg)[..., 0] * alive if s["g"] is not None else None,
                  "dbeta": rows(db)[..., 0] * alive, "dh0": U.view(B, H, K, V)}
