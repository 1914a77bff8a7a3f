"""Linear attention with a decay for each head (prefill, training step, single-token step) and layer norm (forward, backward):
cases, inputs, plain forms and 64-bit values.

The model per batch row, head h (q, k shared by H/G heads), token t < length:
    S_t = exp(g_t) S_{t-1} + k_t v_t^T        o_t = scale * S_t^T q_t        S: [K, V], scale = K^-1/2
and, for a loss whose gradients at o and at the last state are `do` and `dh_last`, the gradients of q, k, v, g and of the first state.
"""

import math

import torch

own = False

EPS = 1e-5
CHUNK = 64  # tokens per chunk of the plain form
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases


def _attn(name, op, B, L, H, G, K, V, dtype, decay="token", carry=False, ragged=False, packed=False):
    return {"name": name, "op": op, "B": B, "L": L, "H": H, "G": G, "K": K, "V": V, "dtype": dtype, "decay": decay,
            "carry": carry, "ragged": ragged, "packed": packed}


def _norm(name, op, rows, dim, dtype):
    return {"name": name, "op": op, "rows": rows, "dim": dim, "dtype": dtype}


def listed():
    return [
        # a batch of short prompts of unequal length (an empty one and one of a single token among them) before decoding, odd head sizes
        _attn("prefill_ragged", "prefill", 5, 77, 6, 3, 40, 72, "bf16", carry=True, ragged=True),
        # one long prompt, q and k shared by all heads, on the long-context layer's width (d_inner 2048, 16384 tokens)
        _attn("prefill_long_shared", "prefill", 1, 16384, 32, 1, 128, 64, "bf16"),
        # a batch of prompts on the 1.4B layer's width (d_inner 4096), q, k and v cut out of one projection
        _attn("prefill_layer", "prefill", 4, 2048, 32, 32, 128, 128, "bf16", packed=True),
        # one training step of that layer: forward with checkpoints, then all gradients
        _attn("train_layer", "train", 4, 2048, 32, 32, 128, 128, "bf16", packed=True),
        # a long sequence trained in pieces: a state comes in and a gradient of the state arrives at the end
        _attn("train_long_shared", "train", 1, 8192, 32, 4, 128, 64, "bf16", carry=True),
        # the 130M layer in fp32 (d_inner 1536, 24 heads of 64), one decay per head
        _attn("train_130m_f32", "train", 8, 2048, 24, 24, 64, 64, "f32", decay="head"),
        # one sequence being decoded: latency
        _attn("step_one", "step", 1, 1, 32, 32, 128, 128, "bf16", carry=True),
        # a server's batch of sequences being decoded
        _attn("step_batch", "step", 96, 1, 32, 8, 128, 128, "bf16", carry=True),
        # the norm before the 1.4B layer, and over each head's output of it
        _norm("norm_fwd_layer", "norm_fwd", 8192, 2048, "bf16"),
        _norm("norm_fwd_heads", "norm_fwd", 262144, 128, "bf16"),
        # their backward passes; the 130M layer's in fp32
        _norm("norm_bwd_heads", "norm_bwd", 262144, 128, "bf16"),
        _norm("norm_bwd_130m_f32", "norm_bwd", 16384, 768, "f32"),
    ]


def _log(rng, lo, hi):
    n = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))
    return n - (n > lo and n % 1024 == 0)  # the round sizes are listed


def draw(rng):
    op = rng.choice(["prefill", "prefill", "train", "train", "step", "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("norm"):
        dim = rng.choice([2 ** rng.randint(4, 13), 768, 8 * (2 * _log(rng, 1, 512) - 1)])
        rows = min(_log(rng, 1, 262144), (1 << 25) // dim // (1 if dtype == "bf16" else 2))
        return {"op": op, "rows": max(1, rows), "dim": dim, "dtype": dtype}
    K, V = (rng.choice([rng.choice([64, 128]), 8 * rng.randint(1, 16)]) for _ in range(2))
    G = _log(rng, 1, 32)
    H = G * rng.choice([r for r in (1, 1, 2, 3, 4, 8, 16, 32) if G * r <= 64])
    decay, carry, ragged, packed = rng.choice(["token", "token", "head"]), rng.random() < 0.5, rng.random() < 0.4, rng.random() < 0.5
    step = op == "step"
    if step:
        B, L = min(_log(rng, 1, 256), max(1, 96 * 32 * 128 * 128 // (H * K * V))), 1
    else:  # tokens: no more than the largest listed cases have, of tokens or of work
        most = min(4 * 2048 * 32 // H, (4 * 2048 * 32 * 128 * 128 if dtype == "bf16" else 8 * 2048 * 24 * 64 * 64) // (H * K * V))
        most -= most // 16
        L = min(_log(rng, 1, 16384), most)
        B = min(_log(rng, 1, 64), max(1, most // L))
    return {"op": op, "B": B, "L": L, "H": H, "G": G, "K": K, "V": V, "dtype": dtype, "decay": decay, "carry": carry or step,
            "ragged": ragged and not step, "packed": packed and not step}


# ---------------------------------------------------------------- inputs


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DT[case["dtype"]]

    def normal(*shape, dtype=dt):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)

    s = {"op": case["op"]}
    if case["op"].startswith("norm"):
        R, N = case["rows"], case["dim"]
        x = (normal(R, N, dtype=torch.float32) * 1.5 + 0.3 * normal(R, 1, dtype=torch.float32)).to(dt)  # a row has a mean of its own
        s |= {"x": x, "scale": 1 + 0.1 * normal(N, dtype=torch.float32), "bias": 0.1 * normal(N, dtype=torch.float32)}
        if case["op"] == "norm_bwd":  # what the forward saved
            xd = x.double()
            s |= {"dy": normal(R, N), "mean": xd.mean(1).float(), "rstd": (xd.var(1, unbiased=False) + EPS).rsqrt().float()}
        return s
    B, L, H, G, K, V = (case[k] for k in "BLHGKV")
    if case["decay"] == "token":  # -a_h * dt with the step sizes of the scan's layers: softplus(0.5 eps + bias), bias of [1e-3, 1e-1]
        u = torch.empty(H, device="cuda").uniform_(math.log(1e-3), math.log(1e-1), generator=gen).exp()
        a = torch.empty(H, device="cuda").uniform_(1.0, 16.0, generator=gen)
        dts = torch.nn.functional.softplus(0.5 * normal(B, L, H, dtype=torch.float32) + torch.log(torch.expm1(u)))
        s["g"] = -(a * dts)
    else:  # memories of 2^5 to 2^12 tokens, one for each head
        s["g"] = torch.log1p(-torch.exp2(-torch.empty(H, device="cuda").uniform_(5.0, 12.0, generator=gen)))
    s["K"], s["V"], s["G"], s["H"] = K, V, G, H
    if case["packed"]:
        s["qkv"] = normal(B, L, 2 * G * K + H * V)
    else:
        s["q"], s["k"], s["v"] = normal(B, L, G, K), normal(B, L, G, K), normal(B, L, H, V)
    s["h"] = normal(B, H, K, V, dtype=torch.float32) if case["carry"] or case["op"] == "step" else None
    if case["op"] == "step":
        for n in "qkv":
            s[n] = s[n][:, 0].contiguous()
        s["g"] = s["g"][:, 0].contiguous() if case["decay"] == "token" else s["g"]
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
            y, mean, rstd = ss.layernorm_fwd(s["x"], s["scale"], s["bias"], EPS)
            return {"y": y, "mean": mean, "rstd": rstd}
        if s["op"] == "norm_bwd":
            dx, dscale, dbias = ss.layernorm_bwd(s["dy"], s["x"], s["scale"], s["mean"], s["rstd"])
            return {"dx": dx, "dscale": dscale, "dbias": dbias}
        if s["op"] == "step":  # the state advances in place, pass after pass
            return {"o": ss.linattn_step(s["q"], s["k"], s["v"], s["g"], s["h"]), "h": s["h"]}
        q, k, v = _qkv(s)
        train = s["op"] == "train"
        o, ckpt, h_last = ss.linattn_fwd(q, k, v, s["g"], h0=s["h"], lengths=s["lengths"], want_ckpt=train)
        if not train:
            return {"o": o, "h_last": h_last}
        d = ss.linattn_bwd(q, k, v, s["g"], ckpt, s["do"], dh_last=s["dh_last"], lengths=s["lengths"])
        return {"o": o, "h_last": h_last, "dq": d["dq"], "dk": d["dk"], "dv": d["dv"], "dg": d["dg"], "dh0": d["dh0"]}
    if s["op"] == "norm_fwd":
        return _norm_fwd(s["x"], s["scale"], s["bias"])
    if s["op"] == "norm_bwd":
        return _norm_bwd(s["dy"], s["x"], s["scale"], s["mean"], s["rstd"])
    if s["op"] == "step":
        return _step(s["q"], s["k"], s["v"], s["g"], s["h"])
    return _chunked(*_qkv(s), s["g"], s["h"], s["lengths"], s.get("do"), s.get("dh_last"))


def _norm_fwd(x, scale, bias):
    f = x.float()
    mean = f.mean(1)
    c = f - mean[:, None]
    rstd = ((c * c).mean(1) + EPS).rsqrt()
    return {"y": (c * rstd[:, None] * scale + bias).to(x.dtype), "mean": mean, "rstd": rstd}


def _norm_bwd(dy, x, scale, mean, rstd):
    xh = (x.float() - mean[:, None]) * rstd[:, None]
    g = dy.float()
    w = g * scale
    dx = rstd[:, None] * (w - w.mean(1, keepdim=True) - xh * (w * xh).mean(1, keepdim=True))
    return {"dx": dx, "dscale": (g * xh).sum(0), "dbias": g.sum(0)}


def _step(q, k, v, g, h):
    B, H, V = v.shape
    G, K = q.shape[1:]
    q, k = (t.float()[:, :, None].expand(B, G, H // G, K).reshape(B, H, K) for t in (q, k))
    h.mul_(g.exp().expand(B, H)[:, :, None, None]).add_(k[..., None] * v.float()[:, :, None])
    return {"o": ((q[..., None] * h).sum(2) * K**-0.5).to(v.dtype), "h": h}


def _chunked(q, k, v, g, h0, lengths, do, dh_last):
    """The chunked form in 32 bits: inside a chunk the masked product of scores, across chunks one product with the chunks' decays."""
    B, L, G, K = q.shape
    H, V = v.shape[2:]
    R, C, dt, scale = H // G, CHUNK, v.dtype, K**-0.5
    n = -(-L // C)
    live = torch.arange(n * C, device=q.device) < (lengths[:, None] if lengths is not None else L)  # [B, n*C]
    live = live.expand(B, n * C)

    def lay(t):  # [B, L, heads, W] -> [B, G, heads/G, n, C, W] in 32 bits, nothing past a row's end
        t = torch.nn.functional.pad(t.float(), (0, 0, 0, 0, 0, n * C - L))
        t = torch.where(live[:, :, None, None], t, 0.0)
        return t.unflatten(1, (n, C)).unflatten(3, (G, -1)).permute(0, 3, 4, 1, 2, 5)

    def back(t):  # the reverse, rounded once
        return t.permute(0, 3, 4, 1, 2, 5).reshape(B, n * C, -1, t.shape[-1])[:, :L].contiguous()

    q, k, v = lay(q), lay(k), lay(v)
    per_head = g.dim() == 1
    gl = lay(g.expand(B, L, H)[..., None])[..., 0].double()  # [B, G, R, n, C]
    c = gl.cumsum(-1)
    lower = torch.ones(C, C, device=q.device, dtype=torch.bool).tril()
    D = (c[..., :, None] - c[..., None, :]).masked_fill(~lower, -math.inf).exp().float()
    into, rest = c.exp().float()[..., None], (c[..., -1:] - c).exp().float()[..., None]
    P = (q @ k.mT) * D * scale
    # states: [h0, what each chunk adds]; S[m] enters chunk m, S[n] is the last
    E = torch.nn.functional.pad(c[..., -1].cumsum(-1), (1, 0))
    across = (E[..., :, None] - E[..., None, :]).masked_fill(~torch.ones(n + 1, n + 1, device=q.device, dtype=torch.bool).tril(), -math.inf).exp().float()
    first = torch.zeros(B, G, R, 1, K, V, device=q.device) if h0 is None else h0.view(B, G, R, 1, K, V)
    S = (across @ torch.cat([first, (k * rest).mT @ v], 3).flatten(4)).unflatten(4, (K, V))
    o = P @ v + scale * into * (q @ S[:, :, :, :n])
    out = {"o": back(o).to(dt), "h_last": S[:, :, :, n].reshape(B, H, K, V)}
    if do is None:
        return out
    do = lay(do)
    last = torch.zeros(B, G, R, 1, K, V, device=q.device) if dh_last is None else dh_last.view(B, G, R, 1, K, V)
    U = (across.mT @ torch.cat([scale * (q * into).mT @ do, last], 3).flatten(4)).unflatten(4, (K, V))
    S, U0, U = S[:, :, :, :n], U[:, :, :, 0], U[:, :, :, 1:]  # the state entering a chunk, the gradient of the one leaving it
    dP = (do @ v.mT) * D * scale
    qi, ki = scale * into * (do @ S.mT), rest * (v @ U.mT)
    dq, dk, dv = dP @ k + qi, dP.mT @ q + ki, P.mT @ do + rest * (k @ U)
    M = (dP * (q @ k.mT)).double()
    before = M.cumsum(-1) - M  # [i, t]: sum over j < t
    dg = torch.where(lower, before, 0.0).sum(-2)
    a, b = (q * qi).sum(-1).double(), (k * ki).sum(-1).double()
    dg = dg + a.flip(-1).cumsum(-1).flip(-1) + b.cumsum(-1) - b + (c[..., -1].exp() * (S * U).sum((-1, -2)).double())[..., None]
    dg = torch.where(live.view(B, 1, 1, n, C), dg, 0.0)
    dg = back(dg[..., None])[..., 0]
    out |= {"dq": back(dq.sum(2, keepdim=True)).to(dt), "dk": back(dk.sum(2, keepdim=True)).to(dt), "dv": back(dv).to(dt),
            "dg": (dg.sum((0, 1)) if per_head else dg).float(), "dh0": U0.reshape(B, H, K, V)}
    return out


# ---------------------------------------------------------------- work


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("norm"):
        n, R, N = case["rows"] * case["dim"], case["rows"], case["dim"]
        if case["op"] == "norm_fwd":
            return {"bytes": 2 * n * e + 8 * N + 8 * R, "flops": 8 * n}
        return {"bytes": 2 * n * e + 4 * n + 12 * N + 8 * R, "flops": 14 * n}
    B, L, H, G, K, V = (case[k] for k in "BLHGKV")
    qk, vo, st = B * L * G * K * e, B * L * H * V * e, 4 * B * H * K * V
    g = 4 * (B * L * H if case["decay"] == "token" else H)
    if case["op"] == "step":
        return {"bytes": 2 * qk + 2 * vo + g + 2 * st, "flops": 5 * B * H * K * V}
    carry = st if case["carry"] else 0
    fwd = {"bytes": 2 * qk + 2 * vo + g + st + carry, "flops": 4 * B * L * H * K * V}
    if case["op"] == "prefill":
        return fwd
    # the backward reads q, k, v, do, g (and the arriving gradient) and writes those of q, k, v, g and of the first state
    return {"bytes": fwd["bytes"] + 4 * qk + 3 * vo + 2 * g + st + carry, "flops": fwd["flops"] + 10 * B * L * H * K * V}


# ---------------------------------------------------------------- 64 bits, from the recurrence


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_fwd":
        x = s["x"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0)
        r = 1.0 / torch.sqrt(var + EPS)
        return {"y": torch.addcmul(s["bias"].double(), (x - mean.unsqueeze(1)) * r.unsqueeze(1), s["scale"].double()), "mean": mean, "rstd": r}
    if case["op"] == "norm_bwd":
        x, dy, w = s["x"].double(), s["dy"].double(), s["scale"].double()
        m, r, N = s["mean"].double().unsqueeze(1), s["rstd"].double().unsqueeze(1), case["dim"]
        p, t = torch.einsum("rn,n->r", dy, w), torch.einsum("rn,rn,n->r", dy, x - m, w)
        return {"dx": r * dy * w - r * p.unsqueeze(1) / N - r**3 * (x - m) * t.unsqueeze(1) / N,
                "dscale": torch.einsum("rn,rn->n", dy, (x - m) * r), "dbias": torch.einsum("rn->n", dy)}
    B, L, H, G, K, V = (case[k] for k in "BLHGKV")
    if case["op"] == "step":
        h = torch.exp(s["g"].double()).expand(B, H).reshape(B, H, 1, 1) * s["h"].double()
        h = h + torch.einsum("bhk,bhv->bhkv", s["k"].double().repeat_interleave(H // G, 1), s["v"].double())
        return {"o": torch.einsum("bhk,bhkv->bhv", s["q"].double().repeat_interleave(H // G, 1), h) / math.sqrt(K), "h": h}
    q, k, v = (t.double() for t in _qkv(s))
    q, k = q.repeat_interleave(H // G, 2) / math.sqrt(K), k.repeat_interleave(H // G, 2)
    n = s["lengths"].tolist() if s["lengths"] is not None else [L] * B
    g = s["g"].double().expand(B, L, H).clone()
    do = s["do"].double() if "do" in s else None
    q, k, v = q.clone(), k.clone(), v.clone()
    do = do.clone() if do is not None else None
    for b, m in enumerate(n):  # a token past its row's end neither decays nor adds nor reads
        for t in (q, k, v, g) + ((do,) if do is not None else ()):
            t[b, m:] = 0
    q, k, v, e = (t.transpose(0, 1).reshape(L, B * H, -1).contiguous() for t in (q, k, v, g.exp().unsqueeze(-1)))
    S = s["h"].double().reshape(B * H, K, V).clone() if s["h"] is not None else torch.zeros(B * H, K, V, device="cuda", dtype=torch.float64)
    o = torch.empty(L, B * H, V, device="cuda", dtype=torch.float64)

    def rows(t):  # [L, B*H, W] -> [B, L, H, W]
        return t.view(L, B, H, -1).transpose(0, 1)

    if do is not None:
        do = do.transpose(0, 1).reshape(L, B * H, V).contiguous()
        dq = torch.empty(L, B * H, K, device="cuda", dtype=torch.float64)
    first = S.clone()
    for t in range(L):
        S.mul_(e[t].unsqueeze(-1)).baddbmm_(k[t].unsqueeze(2), v[t].unsqueeze(1))
        torch.bmm(q[t].unsqueeze(1), S, out=o[t].unsqueeze(1))
        if do is not None:
            torch.bmm(S, do[t].unsqueeze(2), out=dq[t].unsqueeze(2))
    out = {"o": rows(o), "h_last": S.view(B, H, K, V)}
    if do is None:
        return out
    U = s["dh_last"].double().reshape(B * H, K, V).clone() if s["dh_last"] is not None else torch.zeros_like(S)
    # through the decays' running sum c_t: dL/dc_t = q_t.dq_t - k_t.dk_t, and <S, dL/dS> at the end; dg is its sum over later tokens
    end = (S * U).sum((1, 2))
    dk, dv = torch.empty_like(k), torch.empty_like(v)
    for t in range(L - 1, -1, -1):
        U.baddbmm_(q[t].unsqueeze(2), do[t].unsqueeze(1))
        torch.bmm(U, v[t].unsqueeze(2), out=dk[t].unsqueeze(2))
        torch.bmm(k[t].unsqueeze(1), U, out=dv[t].unsqueeze(1))
        U.mul_(e[t].unsqueeze(-1))
    dc = (q * dq).sum(-1) - (k * dk).sum(-1)
    dg = rows((dc.flip(0).cumsum(0).flip(0) + end).unsqueeze(-1))[..., 0].contiguous()
    for b, m in enumerate(n):
        dg[b, m:] = 0
    share = lambda t: rows(t).reshape(B, L, G, H // G, K).sum(3)  # noqa: E731
    return out | {"dq": share(dq) / math.sqrt(K), "dk": share(dk), "dv": rows(dv), "dg": dg.sum((0, 1)) if case["decay"] == "head" else dg,
                  "dh0": U.view(B, H, K, V)}
