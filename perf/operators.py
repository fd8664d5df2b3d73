"""Cases, inputs, plain forms and work of the operators around retention: layer norm
(forward with the residual, backward with the weight's gradient), rotary positions, and
linear attention whose decay is set for each head and token (chunked over prompts, one step
over single tokens).

With ``own`` false, ``run`` computes an operator from elementary torch operations in 32
bits (decay exponents and rotation angles in 64); with ``own`` true it calls the package.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64              # tokens a chunk of the plain form of linear attention
RESET = -200.0          # exp of it is 0 in 32 bits: stands for a decay of exactly 0


# ---- cases ------------------------------------------------------------------------------

def listed():
    return [
        # the norm before a layer while a batch of 32 sequences decodes: latency
        {"name": "norm_decode", "op": "norm", "rows": 32, "d": 4096, "type": "bf16",
         "residual": True, "affine": True},
        # the same norm over two 8192-token training sequences
        {"name": "norm_train", "op": "norm", "rows": 16384, "d": 4096, "type": "bf16",
         "residual": True, "affine": True},
        # its gradients, the residual stream's own gradient joined
        {"name": "norm_back_train", "op": "norm_back", "rows": 16384, "d": 4096, "type": "bf16",
         "residual": True, "affine": True},
        # gradients in float32 at an odd width and an odd number of rows, no residual
        {"name": "norm_back_odd", "op": "norm_back", "rows": 3001, "d": 1537, "type": "f32",
         "residual": False, "affine": True},
        # q and k of one decode step, each sequence at a position of its own
        {"name": "rotary_decode", "op": "rotary", "B": 64, "N": 1, "Hq": 32, "Hk": 8, "d": 128,
         "rot": 128, "type": "bf16", "half": True, "token_major": True, "back": False,
         "scaled": False, "pos": "sequence"},
        # a long prompt, half of each head rotated, angles stretched for a long context
        {"name": "rotary_prompt", "op": "rotary", "B": 1, "N": 16384, "Hq": 32, "Hk": 8, "d": 128,
         "rot": 64, "type": "bf16", "half": True, "token_major": True, "back": False,
         "scaled": True, "pos": "first"},
        # gradients of rotated float32 heads of retention's own width and order
        {"name": "rotary_back", "op": "rotary", "B": 2, "N": 2047, "Hq": 16, "Hk": 16, "d": 256,
         "rot": 256, "type": "f32", "half": False, "token_major": False, "back": True,
         "scaled": False, "pos": "token"},
        # a batch of decode steps on states in a pool with free slots
        {"name": "step_batch", "op": "step", "B": 128, "H": 16, "Hq": 16, "Hk": 16, "Hv": 16,
         "dk": 256, "dv": 512, "type": "bf16", "pool": 144, "fade": 16.0},
        # one sequence decoding: latency
        {"name": "step_one", "op": "step", "B": 1, "H": 16, "Hq": 16, "Hk": 16, "Hv": 16,
         "dk": 128, "dv": 128, "type": "f32", "pool": 4, "fade": 1.0},
        # one long prompt on heads of retention's width
        {"name": "prompt_long", "op": "prompt", "S": 1, "tokens": 8192, "packed": False,
         "ragged": False, "H": 16, "Hq": 16, "Hk": 16, "Hv": 16, "dk": 256, "dv": 512,
         "type": "bf16", "token_major": True, "fade": 16.0, "resets": False, "start": False},
        # prompts of many lengths packed end to end, q and k shared by groups of four heads
        {"name": "prompt_packed", "op": "prompt", "S": 13, "tokens": 14001, "packed": True,
         "ragged": True, "H": 32, "Hq": 8, "Hk": 8, "Hv": 32, "dk": 64, "dv": 128,
         "type": "bf16", "token_major": True, "fade": 16.0, "resets": False, "start": True},
        # a padded float32 batch with document borders inside its rows, odd head sizes
        {"name": "prompt_f32_odd", "op": "prompt", "S": 3, "tokens": 2001, "packed": False,
         "ragged": True, "H": 5, "Hq": 5, "Hk": 1, "Hv": 5, "dk": 48, "dv": 81,
         "type": "f32", "token_major": False, "fade": 4.0, "resets": True, "start": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_back", "rotary", "step", "prompt", "prompt"])
    kind = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm_back"):
        d = _log_int(rng, 64, 8192)
        if rng.random() < 0.7:
            d = max(64, d // 8 * 8)
        rows = min(_log_int(rng, 1, 16384), (1 << 25) // d)
        return {"op": op, "rows": rows, "d": d, "type": kind, "residual": rng.random() < 0.6,
                "affine": rng.random() < 0.8}
    if op == "rotary":
        B, d = _log_int(rng, 1, 64), 2 * _log_int(rng, 16, 128)
        Hk = rng.choice([1, 2, 3, 8, 16])
        Hq = Hk * rng.choice([1, 2, 4])
        N = min(_log_int(rng, 1, 8192), max(1, (1 << 26) // (B * (Hq + Hk) * d)))
        rot = d if rng.random() < 0.5 else 2 * rng.randint(1, d // 2)
        return {"op": op, "B": B, "N": N, "Hq": Hq, "Hk": Hk, "d": d, "rot": rot, "type": kind,
                "half": rng.random() < 0.5, "token_major": rng.random() < 0.5,
                "back": rng.random() < 0.3, "scaled": rng.random() < 0.4,
                "pos": rng.choice(["first", "sequence", "token"])}
    dk = rng.choice([16, 33, 48, 64, 64, 80, 128, 128, 192, 256])
    dv = rng.choice([16, 40, 64, 64, 81, 128, 128, 256, 512])
    H = rng.choice([1, 3, 4, 8, 16, 32])
    shared = [h for h in (1, 2, 3, 4, 8, H) if H % h == 0]
    heads = {"H": H, "Hq": rng.choice([H, rng.choice(shared)]),
             "Hk": rng.choice([H, rng.choice(shared)]), "Hv": rng.choice([H, rng.choice(shared)])}
    if op == "step":
        B = min(_log_int(rng, 1, 256), max(1, (1 << 27) // (H * dk * dv)))
        return {"op": op, "B": B, **heads, "dk": dk, "dv": dv, "type": kind,
                "pool": B + rng.randint(0, 17), "fade": rng.choice([1.0, 4.0, 16.0])}
    S = _log_int(rng, 1, 16)
    most = 8192 if kind == "bf16" else 2048
    most = max(S, min(most, (1 << 29) // (H * (dk + dv) * 12), (1 << 34) // (H * dk * dv)))
    return {"op": op, "S": S, "tokens": max(S, _log_int(rng, S, most)), "packed": rng.random() < 0.5,
            "ragged": rng.random() < 0.6, **heads, "dk": dk, "dv": dv, "type": kind,
            "token_major": rng.random() < 0.5, "fade": rng.choice([1.0, 4.0, 16.0]),
            "resets": rng.random() < 0.3, "start": rng.random() < 0.5}


# ---- inputs -----------------------------------------------------------------------------

def _lengths(case, seed):
    """Tokens of each of the S sequences: equal shares, or spread over a factor of about 8."""
    S, T = case["S"], case["tokens"]
    if not case["ragged"]:
        return [T // S + (1 if s < T % S else 0) for s in range(S)] if case["packed"] else [T // S] * S
    rng = np.random.default_rng([seed, 3])
    share = np.exp(rng.uniform(0.0, math.log(8.0), S))
    n = np.maximum(1, np.floor(share / share.sum() * T).astype(int))
    if case["packed"]:
        n[int(np.argmax(n))] += T - int(n.sum())
    return [int(x) for x in n]


def _longest(case):
    """Rows of a padded batch: fixed by the case, not by the seed."""
    S, T = case["S"], case["tokens"]
    if S == 1:
        return T
    return min(T, 8 * T // (S + 7) + 1) if case["ragged"] else T // S


def _heads(gen, B, H, N, d, dtype, token_major):
    """[B, H, N, d] values, in memory head-major or (as a projection leaves them) token-major."""
    shape = (B, N, H, d) if token_major else (B, H, N, d)
    x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)
    return x.transpose(1, 2) if token_major else x


def _theta(rot, scaled):
    """Angles of the rotated pairs; stretched 8-fold where a pair turns less than once in
    4096 positions, left alone where it turns 32 times, in between in proportion."""
    j = np.arange(rot // 2, dtype=np.float64)
    th = 10000.0 ** (-2.0 * j / rot)
    if not scaled:
        return th, 1.0
    turns = 4096.0 * th / (2.0 * math.pi)
    keep = np.clip((turns - 1.0) / 31.0, 0.0, 1.0)
    return th * (keep + (1.0 - keep) / 8.0), 0.1 * math.log(8.0) + 1.0


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    c, op, dt = case, case["op"], TYPES[case["type"]]

    def randn(*shape, dtype=dt, std=1.0, mean=0.0):
        x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)
        return (x * std + mean).to(dtype)

    s = {"case": dict(c)}
    if op in ("norm", "norm_back"):
        s["x"] = randn(c["rows"], c["d"], std=1.5, mean=0.25)
        s["w"] = randn(c["d"], dtype=torch.float32, std=0.2, mean=1.0) if c["affine"] else None
        s["b"] = randn(c["d"], dtype=torch.float32, std=0.2) if c["affine"] else None
        if op == "norm":
            s["r"] = randn(c["rows"], c["d"]) if c["residual"] else None
        else:
            s["dy"] = randn(c["rows"], c["d"])
            s["dh"] = randn(c["rows"], c["d"]) if c["residual"] else None
        return s
    if op == "rotary":
        B, N = c["B"], c["N"]
        s["q"] = _heads(gen, B, c["Hq"], N, c["d"], dt, c["token_major"])
        s["k"] = _heads(gen, B, c["Hk"], N, c["d"], dt, c["token_major"])
        s["theta"], s["magnitude"] = _theta(c["rot"], c["scaled"])
        first = torch.randint(0, 100000, (B,), generator=gen, device=DEV)
        s["pos0"], s["pos"] = 11 + int(seed) % 1000, None
        if c["pos"] == "sequence":
            s["pos"] = first
        elif c["pos"] == "token":
            s["pos"] = (first[:, None] + torch.arange(N, device=DEV)[None]) % 65536
        return s
    S = c["B"] if op == "step" else c["S"]
    H, dk, dv = c["H"], c["dk"], c["dv"]
    s["scale"] = 1.0 / math.sqrt(dk)
    if op == "step":
        for name, h, d in (("q", c["Hq"], dk), ("k", c["Hk"], dk), ("v", c["Hv"], dv)):
            s[name] = _heads(gen, S, h, 1, d, dt, False)
        s["g"] = torch.nn.functional.logsigmoid(randn(S, H, 1, dtype=torch.float32, mean=2.0)) / c["fade"]
        s["state"] = randn(c["pool"], H, dk, dv, dtype=torch.float32)
        order = np.random.default_rng([seed, 5]).permutation(c["pool"])[:S]
        s["slots"] = torch.tensor(order.astype(np.int32), device=DEV)
        return s
    lens = _lengths(c, seed)
    B, N = (1, c["tokens"]) if c["packed"] else (S, _longest(c))
    for name, h, d in (("q", c["Hq"], dk), ("k", c["Hk"], dk), ("v", c["Hv"], dv)):
        s[name] = _heads(gen, B, h, N, d, dt, c["token_major"])
    g = torch.nn.functional.logsigmoid(randn(B, H, N, dtype=torch.float32, mean=2.0)) / c["fade"]
    if c["resets"]:
        g[torch.rand((B, 1, N), generator=gen, device=DEV).expand(B, H, N) < 0.01] = -math.inf
    s["g"] = g
    s["start"] = randn(S, H, dk, dv, dtype=torch.float32) if c["start"] else None
    s["lens"], s["cu"], s["longest"] = None, None, max(lens)
    if c["packed"]:
        s["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32), device=DEV)
    else:
        lens = [min(n, N) for n in lens]
        s["longest"] = max(lens)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV) if c["ragged"] else None
        # rows past a sequence's length belong to nobody: they stay as they are here
        s["out"] = torch.zeros_like(s["v"][:, :1].expand(B, H, N, dv), memory_format=torch.contiguous_format)
    return s


# ---- the operators, plain or the package's ----------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return _own(op, s)
    return {"norm": _norm, "norm_back": _norm_back, "rotary": _rotary, "step": _step,
            "prompt": _prompt}[op](s)


def _own(op, s):
    import linear_recurrent_sequence_rn_amd as rn
    c = s["case"]
    if op == "norm":
        if s["r"] is None:
            return {"out": rn.rn_layernorm(s["x"], s["w"], s["b"])}
        out, total = rn.rn_layernorm(s["x"], s["w"], s["b"], residual=s["r"])
        return {"out": out, "sum": total}
    if op == "norm_back":
        got = rn.rn_layernorm_backward(s["dy"], s["x"], s["w"], dsum=s["dh"])
        return {"dx": got["dx"], "dw": got["dweight"], "db": got["dbias"]}
    if op == "rotary":
        q, k = rn.rn_rotary(s["q"], s["k"], s["theta"], pos0=s["pos0"], pos=s["pos"],
                            half=c["half"], inverse=c["back"], magnitude=s["magnitude"])
        return {"q": q, "k": k}
    if op == "step":
        out = rn.rn_linear_attention_step(s["q"], s["k"], s["v"], s["g"], s["state"],
                                          slots=s["slots"], qk_scale=s["scale"])
        return {"out": out, "state": s["state"]}
    out, state = rn.rn_linear_attention_chunked(
        s["q"], s["k"], s["v"], s["g"], qk_scale=s["scale"], lengths=s["lens"],
        cu_seqlens=s["cu"], max_len=s["longest"], state_in=s["start"], state_out=True,
        out=None if c["packed"] else s["out"])
    return {"out": out, "state": state}


def _norm(s, eps=1e-5):
    h = s["x"].float()
    if s["r"] is not None:
        h = h + s["r"].float()
    m = h.mean(-1, keepdim=True)
    y = (h - m) * torch.rsqrt((h - m).square().mean(-1, keepdim=True) + eps)
    if s["w"] is not None:
        y = y * s["w"] + s["b"]
    out = {"out": y.to(s["x"].dtype)}
    if s["r"] is not None:
        out["sum"] = h.to(s["x"].dtype)
    return out


def _norm_back(s, eps=1e-5):
    x, dy = s["x"].float(), s["dy"].float()
    xc = x - x.mean(-1, keepdim=True)
    rstd = torch.rsqrt(xc.square().mean(-1, keepdim=True) + eps)
    xh = xc * rstd
    g = dy if s["w"] is None else dy * s["w"]
    dx = (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True)) * rstd
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * xh).sum(0), "db": dy.sum(0)}


def _positions(s, N, B):
    t = torch.arange(N, device=DEV)[None]
    if s["pos"] is None:
        return (t + s["pos0"]).expand(B, N)
    return s["pos"][:, None] + t if s["pos"].dim() == 1 else s["pos"]


def _rotary(s):
    c = s["case"]
    rot, half = c["rot"], c["half"]
    theta = torch.from_numpy(s["theta"]).to(DEV)
    a = _positions(s, c["N"], c["B"]).double()[:, None, :, None] * theta
    cos = (a.cos() * s["magnitude"]).float()
    sin = (a.sin() * s["magnitude"]).float()
    if c["back"]:
        sin = -sin

    def turn(x):
        y = x.float()
        if half:
            u, w = y[..., : rot // 2], y[..., rot // 2: rot]
            z = torch.cat((u * cos - w * sin, u * sin + w * cos), -1)
        else:
            u, w = y[..., 0:rot:2], y[..., 1:rot:2]
            z = torch.stack((u * cos - w * sin, u * sin + w * cos), -1).flatten(-2)
        return torch.cat((z, y[..., rot:]), -1).to(x.dtype)

    return {"q": turn(s["q"]), "k": turn(s["k"])}


def _spread(x, H):
    """The H heads' own copies of heads that groups of them share, in 32 bits."""
    x = x.float()
    return x if x.shape[1] == H else x.repeat_interleave(H // x.shape[1], 1)


def _step(s):
    H = s["case"]["H"]
    q, k, v = (_spread(s[n], H) for n in "qkv")
    at = s["slots"].long()
    S = s["state"][at] * s["g"].exp()[..., None] + k.transpose(-1, -2) * v
    s["state"][at] = S
    o = (q * s["scale"]) @ S
    return {"out": o.to(s["v"].dtype), "state": s["state"]}


def _prompt(s):
    """Chunks of 64 tokens: products inside each, and one product of the chunks' decays with
    the chunks' own states for the states between them."""
    c = s["case"]
    H, S, dk, dv = c["H"], c["S"], c["dk"], c["dv"]
    C = CHUNK
    nc = -(-s["longest"] // C)
    t = torch.arange(nc * C, device=DEV)[None].expand(S, -1)
    if c["packed"]:
        cu = s["cu"].long()
        n, row, seq = (cu[1:] - cu[:-1])[:, None], t + cu[:-1, None], torch.zeros_like(t)
    else:
        n = s["lens"].long()[:, None] if s["lens"] is not None else torch.full((S, 1), s["longest"], device=DEV)
        row, seq = t, torch.arange(S, device=DEV)[:, None].expand(S, nc * C)
    live = t < n
    row = torch.where(live, row, 0)

    def take(x):          # [B, h, N, d] -> [S, H, nc, C, d], zeros behind each sequence
        x = x.transpose(1, 2)[seq, row]
        x = torch.where(live[..., None, None], x, 0).transpose(1, 2)
        return _spread(x, H).reshape(S, H, nc, C, -1)

    q, k, v = take(s["q"]), take(s["k"]), take(s["v"])
    g = s["g"].transpose(1, 2)[seq, row].double().clamp_min(RESET)
    g = torch.where(live[..., None], g, 0.0).transpose(1, 2).reshape(S, H, nc, C)
    cum = g.cumsum(-1)
    tri = torch.ones(C, C, dtype=torch.bool, device=DEV).tril()
    D = torch.where(tri, (cum[..., :, None] - cum[..., None, :]), -math.inf).exp().float()
    o = ((q @ k.transpose(-1, -2)) * D) @ v
    w = (cum[..., -1:] - cum).exp().float()
    U = (k * w[..., None]).transpose(-1, -2) @ v
    first = torch.zeros_like(U[:, :, :1]) if s["start"] is None else s["start"][:, :, None]
    U = torch.cat((first, U), 2).reshape(S, H, nc + 1, dk * dv)
    G = torch.cat((torch.zeros_like(cum[..., :1, -1]), cum[..., -1].cumsum(-1)), -1)
    tri = torch.ones(nc + 1, nc + 1, dtype=torch.bool, device=DEV).tril()
    M = torch.where(tri, G[..., :, None] - G[..., None, :], -math.inf).exp().float()
    states = (M @ U).reshape(S, H, nc + 1, dk, dv)
    o = o + (q @ states[:, :, :-1]) * cum.exp().float()[..., None]
    o = (o * s["scale"]).reshape(S, H, nc * C, dv).transpose(1, 2)[live].to(s["v"].dtype)
    if c["packed"]:
        out = torch.empty((c["tokens"], H, dv), dtype=o.dtype, device=DEV)
        out[row[live]] = o
        out = out[None].transpose(1, 2)
    else:
        out = s["out"]
        out.transpose(1, 2)[seq[live], row[live]] = o
    return {"out": out, "state": states[:, :, -1].contiguous()}


# ---- the definitions in 64 bits ---------------------------------------------------------

def exact(case, seed):
    c, op = case, case["op"]
    s = prepare(case, seed)
    if op == "norm":
        h = s["x"].double() + (0.0 if s["r"] is None else s["r"].double())
        var, mean = torch.var_mean(h, -1, correction=0, keepdim=True)
        y = (h - mean) / (var + 1e-5).sqrt()
        if s["w"] is not None:
            y = y * s["w"].double() + s["b"].double()
        return {"out": y} if s["r"] is None else {"out": y, "sum": h}
    if op == "norm_back":
        # the differential of y = z / n, z = x - mean, n = sqrt(|z|^2 / d + eps), transposed
        z = s["x"].double()
        z = z - z.sum(-1, keepdim=True) / c["d"]
        n = (z.pow(2).sum(-1, keepdim=True) / c["d"] + 1e-5).sqrt()
        dy = s["dy"].double()
        a = dy if s["w"] is None else dy * s["w"].double()
        b = a / n - z * (a * z).sum(-1, keepdim=True) / (c["d"] * n.pow(3))
        dx = b - b.sum(-1, keepdim=True) / c["d"]
        if s["dh"] is not None:
            dx = dx + s["dh"].double()
        return {"dx": dx, "dw": (dy * (z / n)).sum(0), "db": dy.sum(0)}
    if op == "rotary":
        p = s["pos"]
        if p is None:
            p = torch.full((c["B"],), s["pos0"], device=DEV)
        if p.dim() == 1:
            p = p[:, None] + torch.arange(c["N"], device=DEV)
        th = torch.tensor(s["theta"], dtype=torch.float64, device=DEV)
        z = torch.polar(torch.full((), s["magnitude"], dtype=torch.float64, device=DEV).expand(c["B"], c["N"], len(th)),
                        p[..., None].double() * th)[:, None]
        z = z.conj() if c["back"] else z
        out = {}
        for name in ("q", "k"):
            x = s[name].double().clone()
            lo, hi = (slice(0, c["rot"] // 2), slice(c["rot"] // 2, c["rot"])) if c["half"] else \
                (slice(0, c["rot"], 2), slice(1, c["rot"], 2))
            y = torch.complex(x[..., lo], x[..., hi]) * z
            x[..., lo], x[..., hi] = y.real, y.imag
            out[name] = x
        return out

    def each(x):
        return x.double()[:, torch.arange(c["H"], device=DEV) // (c["H"] // x.shape[1])]

    if op == "step":
        pool, at = s["state"].double(), s["slots"].long()
        S = pool[at]
        S = torch.exp(s["g"].double())[..., None] * S + torch.einsum("bhnd,bhne->bhde", each(s["k"]), each(s["v"]))
        pool[at] = S
        return {"out": (each(s["q"])[:, :, 0, :, None] * S).sum(-2)[:, :, None] * s["scale"], "state": pool}
    # the recurrence, token by token: about 60 microseconds and 40 bytes of traffic a value
    if s["longest"] * (6e-5 + c["S"] * c["H"] * c["dk"] * c["dv"] * 40 / 3e12) > 20:
        return None
    q, k, v, a = each(s["q"]), each(s["k"]), each(s["v"]), torch.exp(s["g"].double())
    S = torch.zeros((c["S"], c["H"], c["dk"], c["dv"]), dtype=torch.float64, device=DEV)
    if s["start"] is not None:
        S += s["start"]
    out = s["out"].double() if not c["packed"] else torch.zeros((1, c["H"], c["tokens"], c["dv"]), dtype=torch.float64, device=DEV)
    if c["packed"]:
        first = s["cu"][:-1].long()
        n = s["cu"][1:].long() - first
        seq = torch.zeros_like(first)
    else:
        seq = torch.arange(c["S"], device=DEV)
        first = torch.zeros_like(seq)
        n = torch.full_like(seq, s["longest"]) if s["lens"] is None else s["lens"].long()
    by_length = torch.argsort(n, descending=True)
    left = n[by_length].tolist()
    seq, first, S = seq[by_length], first[by_length], S[by_length]
    m = len(left)
    for t in range(s["longest"]):
        while left[m - 1] <= t:
            m -= 1
        at, row = seq[:m], first[:m] + t
        S[:m] *= a[at, :, row][..., None, None]
        S[:m] += k[at, :, row][..., None] * v[at, :, row][..., None, :]
        out[at, :, row] = torch.matmul(q[at, :, row][..., None, :], S[:m]).squeeze(-2) * s["scale"]
    state = torch.empty_like(S)
    state[by_length] = S
    return {"out": out, "state": state}


# ---- work -------------------------------------------------------------------------------

def work(case):
    c, op = case, case["op"]
    e = 2 if c["type"] == "bf16" else 4
    if op in ("norm", "norm_back"):
        n = c["rows"] * c["d"]
        wide = (4 if c["residual"] else 2) if op == "norm" else (4 if c["residual"] else 3)
        par = c["d"] * 4 * ((2 if c["affine"] else 0) if op == "norm" else (3 if c["affine"] else 2))
        return {"bytes": n * e * wide + par, "flops": n * (8 if op == "norm" else 14)}
    if op == "rotary":
        n = c["B"] * c["N"] * (c["Hq"] + c["Hk"])
        return {"bytes": 2 * n * c["d"] * e, "flops": 3 * n * c["rot"]}
    rows = c["B"] if op == "step" else c["tokens"]
    io = rows * e * (c["Hq"] * c["dk"] + c["Hk"] * c["dk"] + c["Hv"] * c["dv"] + c["H"] * c["dv"])
    io += rows * c["H"] * 4
    state = 4 * c["H"] * c["dk"] * c["dv"] * (c["B"] if op == "step" else c["S"])
    times = 2 if op == "step" or c["start"] else 1
    return {"bytes": io + state * times, "flops": 4 * rows * c["H"] * c["dk"] * c["dv"]}
